"""What the draft operators launch, on the CPU (see test_launches_cpu.py): every
launch fits a dispatch wherever a call is taken, calls are refused where one would
not, and a split product's slices lie in the workspace that the library asks for.
Pointers passed here are never dereferenced."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from test_launches_cpu import CHILD, HERE, MOST_ITEMS, ROOT, work_items
from vocab_argmax_amd import _build

P = 0x7F0000010000          # aligned, never dereferenced
WS = 0x7E0000000000
HUGE = 1 << 50
F32, BF16 = 0, 1
OK = 0


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host C++ compiler")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    so = str(tmp_path_factory.mktemp("record") / "launch_record.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    f"-I{rocm}/include", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}",
                    os.path.join(HERE, "launch_record.cc"), "-ldl", "-o", so], check=True)
    child = CHILD.replace("vpa.head_lib()", "vpa.draft_lib()")

    def run(calls):
        first = os.environ.get("LD_PRELOAD")
        env = dict(os.environ, LD_PRELOAD=f"{so}:{first}" if first else so,
                   PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
        res = subprocess.run([sys.executable, "-c", child], input=json.dumps(calls), text=True,
                             capture_output=True, env=env, timeout=600)
        assert res.returncode == 0, res.stderr[-4000:]
        return json.loads(res.stdout)
    return run


def verify(r, k, v, dt=BF16, q=True):
    return ["vpa_sampled_verify", [P, dt, v, [v, v, 1], r, k, P if k else None,
                                   P if q and k else None, dt, v, P if k else None, P, None, WS,
                                   HUGE, P, P, P, None]]


def distill(n, v, dt=BF16):
    return ["vpa_distill_loss", [P, dt, v, [v, v, 1], n, P, P, 8, 1, 1.0, WS, HUGE, P, P, None]]


def distill_backward(n, v, dt=BF16):
    return ["vpa_distill_loss_backward", [P, dt, v, [v, v, 1], n, P, P, 8, 1.0, P, P, P + 4096, v,
                                          v, None]]


def distill_both(n, v, dt=BF16):
    return ["vpa_distill_loss_and_grad", [P, dt, v, [v, v, 1], n, P, P, 8, 1, 1.0, P, WS, HUGE, P,
                                          P, P + 4096, v, v, None]]


def rms(n, c, dt=BF16, fp8=False):
    a = [P, c, dt, None, 0, P, dt, n, c, 1e-6, None, 0, P + 4096, c]
    return (["vpa_rms_norm_fp8", a + [P, (c + 127) // 128, None]] if fp8
            else ["vpa_rms_norm", a + [P, None]])


def rms_backward(n, c, dt=BF16, need="xw"):
    return ["vpa_rms_norm_backward", [P, c, P, c, dt, P, dt, P, None, 0, n, c,
                                      P + 4096 if "x" in need else None, c,
                                      P if "w" in need else None, WS, HUGE, None]]


def quant(n, c, dt=BF16, rows=1):
    return ["vpa_quantize_fp8", [P, c, dt, n, c, rows, P, c, P, (c + 127) // 128, None]]


def linear(n, m, k, odt=BF16, ws_bytes=HUGE):
    ld, b = (k + 15) // 16 * 16, (k + 127) // 128
    return ["vpa_head_linear_fp8", [P, ld, P, b, P, ld, P, b, None, None, 0, n, m, k, 0, P, m, odt,
                                    WS, ws_bytes, None]]


def test_calls_that_are_taken_fit_a_dispatch(record):
    calls = [verify(r, k, v, dt, q) for r in (1, 64, 65, 170, 4096, 100000) for k in (0, 1, 5, 70)
             for v in (1, 1000, 200064) for dt in (F32, BF16) for q in (False, True)]
    calls += [make(n, v, dt) for n in (1, 127, 128, 4096, 1 << 17)
              for v in (1, 1000, 50257, 200064, (1 << 24) - 1) for dt in (F32, BF16)
              for make in (distill, distill_backward, distill_both)]
    calls += [f(n, c, dt) for n in (1, 4096, 1 << 22, (1 << 31) - 1) for c in (1, 513, 4096)
              for dt in (F32, BF16) for f in (rms, lambda *a: rms(*a, fp8=True), rms_backward)]
    calls += [quant(n, c, dt, rows) for n in (1, 4096, 1 << 17) for c in (1, 4096, 1 << 15)
              for dt in (F32, BF16) for rows in (1, 128)]
    calls += [linear(n, m, k, odt) for n in (1, 16, 17, 64, 65, 4096, 1 << 17)
              for m in (1, 4096, 50257, 200064) for k in (1, 130, 2048) for odt in (F32, BF16)]
    taken = 0
    for call, (status, message, got) in zip(calls, record(calls)):
        if status == OK:
            taken += 1
            assert got and max(map(work_items, got)) <= MOST_ITEMS, (call, got)
        else:
            assert "exceed one dispatch" in message and not got, (call, message, got)
    assert taken > len(calls) * 0.9


def test_calls_beyond_a_dispatch_are_refused(record):
    calls = [verify(1 << 24, 0, 1), distill_backward(1 << 24, 4096), distill(1 << 25, 50),
             rms(1 << 22, 16385), rms_backward(1 << 22, 8193), quant(1 << 24, 1 << 15),
             linear(1 << 23, 1 << 16, 64), linear(40, 1 << 30, 16), linear(16, 1 << 30, 16),
             linear(1 << 22, 1 << 16, 64, odt=F32)]
    for call, (status, message, got) in zip(calls, record(calls)):
        assert status != OK and "exceed one dispatch" in message and not got, (call, message, got)


def test_products_keep_to_their_workspace(record):
    """The slices of a split product, as the kernel that joins them is told, lie in the
    workspace of the size that the library asks for, and a byte less is refused."""
    sizes = [(n, m, k) for n in (1, 16, 17, 32, 33, 64, 65, 130, 300, 1000, 2048, 4340)
             for m in (1, 16, 515, 4096, 8192, 50257) for k in (1, 130, 2047, 8192, 40000)]
    need = record([["vpa_head_linear_fp8_workspace", list(s)] for s in sizes])
    split = 0
    for odt in (BF16, F32):
        calls = [linear(*s, odt, n[0]) for s, n in zip(sizes, need)]
        for call, (status, message, got) in zip(calls, record(calls)):
            given = call[1][-2]
            assert status == OK, (call, message)
            for l in got:
                if "gemm_join_kernel" in l["name"]:
                    split += 1
                    assert l["part"] >= WS and l["part"] + l["part_bytes"] <= WS + given, (call, l)
    assert split > 20
    # of the two result types at least one needs all of it
    short = [[linear(*s, odt, n[0] - 1) for odt in (BF16, F32)] for s, n in zip(sizes, need) if n[0]]
    got = record([c for pair in short for c in pair])
    for i in range(len(short)):
        bad = [r for r in got[2 * i:2 * i + 2] if r[0] != OK]
        assert bad and all("workspace" in r[1] for r in bad), short[i]
