"""What the head operators launch, on the CPU: a preloaded library
(launch_record.cc) takes the place of the HIP runtime's kernel launch and
writes each one down, so that the sizes of a launch and the part of the
workspace that its arguments give it can be compared with what the call
checked and asked for.  Pointers passed here are never dereferenced."""
import json
import os
import shutil
import subprocess
import sys

import pytest

from vocab_argmax_amd import _build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

# Runs `calls` (name, arguments) with recorded launches -> one list per call:
# [status, message, launches].
CHILD = """
import ctypes, json, sys
import vocab_argmax_amd as vpa
here = ctypes.CDLL(None)
class Launch(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 192), ("grid", ctypes.c_uint32 * 3),
                ("block", ctypes.c_uint32 * 3), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("slices", ctypes.c_int64), ("part", ctypes.c_uint64),
                ("part_bytes", ctypes.c_int64), ("chunks", ctypes.c_int64)]
here.launches_get.restype = ctypes.POINTER(Launch)
lib = vpa.head_lib()
out = []
for name, args in json.load(sys.stdin):
    here.launches_clear()
    args = [vpa.Vocab(*a) if isinstance(a, list) else a for a in args]
    r = getattr(lib, name)(*args)
    got = []
    for i in range(here.launches_count()):
        l = here.launches_get(i).contents
        got.append(dict(name=l.name.decode(), grid=list(l.grid), block=list(l.block), m=l.m, n=l.n,
                        k=l.k, slices=l.slices, part=l.part, part_bytes=l.part_bytes,
                        chunks=l.chunks))
    out.append([r, vpa.last_error() if r else "", got])
json.dump(out, sys.stdout)
"""

P = 0x7F0000010000          # aligned, never dereferenced
WS = 0x7E0000000000
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

    def run(calls):
        first = os.environ.get("LD_PRELOAD")
        env = dict(os.environ, LD_PRELOAD=f"{so}:{first}" if first else so,
                   PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
        res = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps(calls), text=True,
                             capture_output=True, env=env, timeout=600)
        assert res.returncode == 0, res.stderr[-4000:]
        return json.loads(res.stdout)
    return run


def linear(rows, outer, inner, dt=BF16, ws_bytes=0, act=0, ldx=None, ldw=None):
    return ["vpa_head_linear", [P, ldx or inner, P, ldw or inner, None, None, 0, dt, rows, outer,
                                inner, act, P, outer, dt, None, 0, WS, ws_bytes, None]]


def linear_backward(rows, outer, inner, dt=BF16, ws_bytes=0, act=0, ldg=None, ldx=None, ldw=None,
                    need="xwb"):
    return ["vpa_head_linear_backward",
            [P, ldg or outer, P, ldx or inner, P, ldw or inner, P, outer, dt, rows, outer, inner,
             act, P if "x" in need else None, inner, P if "w" in need else None, inner,
             P if "b" in need else None, WS, ws_bytes, None]]


def work_items(launch):
    n = 1
    for g, b in zip(launch["grid"], launch["block"]):
        n *= g * b
    return n


def products_within(record, sizes, make, workspace):
    """Every launch of each size's call keeps to the workspace it was given,
    the size that the library itself asks for."""
    need = record([[workspace, [dt, *size]] for size, dt in sizes])
    calls = [make(*size, dt=dt, ws_bytes=n[0], act=act)
             for (size, dt), n in zip(sizes, need) for act in (0, 3)]
    for call, (status, message, got) in zip(calls, record(calls)):
        given = call[1][-2]
        assert status == OK, (call, message)
        assert got, call
        for l in got:
            assert l["part_bytes"] == 0 or (
                l["part"] >= WS and l["part"] + l["part_bytes"] <= WS + given), (call, l)


THIN = [((rows, outer, inner), dt)
        for dt in (BF16, F32) for rows in (1, 16, 17, 32, 33, 40, 64, 65, 300)
        for outer in (1, 2, 3, 8, 513, 32000, 50257, 151936)
        for inner in (1, 2, 3, 8, 513, 50257) if outer * inner < 1 << 28]


def test_products_of_thin_operands_keep_to_their_workspace(record):
    """A weight or x of one column has a stride of 1 both ways: its layout, and
    with it the slices of the product, is not to be read from the strides."""
    products_within(record, THIN, linear_backward, "vpa_head_linear_backward_workspace")
    products_within(record, THIN, linear, "vpa_head_linear_workspace")


MOST_ITEMS = (1 << 32) - 1  # of one dispatch
HUGE = 1 << 50


def test_large_products_are_not_refused(record):
    """Scoring and training batches of a wide vocabulary, two-launch plans
    among them: every launch fits a dispatch, so every call is taken."""
    calls = [make(rows, outer, inner, dt=dt, ws_bytes=HUGE)
             for rows in (16, 64, 4096, 65536, 90000, 131072, 1 << 20) for outer in (50257, 200064)
             for inner in (64, 2047, 2048) for dt in (BF16, F32)
             for make in (linear, linear_backward)]
    calls += [linear(40, 1 << 28, 64, ws_bytes=HUGE), linear(40, 64, 1 << 28, ws_bytes=HUGE)]
    for call, (status, message, got) in zip(calls, record(calls)):
        assert status == OK, (call, message)
        assert max(map(work_items, got)) <= MOST_ITEMS, call


def test_products_beyond_a_dispatch_are_refused(record):
    """A call is refused exactly where one of its launches would not fit."""
    edge = 1 << 30                      # columns: a workgroup of 256 takes 64 of them
    calls = [linear(40, edge - 64, 8, ws_bytes=HUGE), linear(40, edge, 8, ws_bytes=HUGE),
             linear(16, edge - 64, 8, ws_bytes=HUGE), linear(16, edge, 8, ws_bytes=HUGE),
             linear(1 << 21, 1 << 16, 64, ws_bytes=HUGE), linear(1 << 23, 1 << 16, 64, ws_bytes=HUGE)]
    for i, (call, (status, message, got)) in enumerate(zip(calls, record(calls))):
        if i % 2:
            assert status != OK and "exceed one dispatch" in message and not got, (call, got)
        else:
            assert status == OK and max(map(work_items, got)) <= MOST_ITEMS, (call, message, got)


ORDINARY = [((rows, outer, inner), dt) for dt in (BF16, F32) for rows in (1, 24, 130, 2048, 4340)
            for outer in (96, 4090, 8192, 50257) for inner in (200, 4088, 8192)]


def test_ordinary_products_keep_to_their_workspace(record):
    products_within(record, ORDINARY, linear_backward, "vpa_head_linear_backward_workspace")
    products_within(record, ORDINARY, linear, "vpa_head_linear_workspace")


def norm(rows, cols, dt=BF16):
    return ["vpa_layer_norm", [P, cols, dt, P, P, dt, rows, cols, 1e-5, P, cols, P, P, None]]


def norm_backward(rows, cols, dt=BF16, need="xwb"):
    return ["vpa_layer_norm_backward",
            [P, cols, P, cols, dt, P, dt, P, P, rows, cols, P + 4096 if "x" in need else None, cols,
             P if "w" in need else None, P if "b" in need else None, WS, HUGE, None]]


def test_norms_of_many_rows_are_not_refused(record):
    """Rows that registers hold are walked by a grid of bounded size: any number
    of them is taken.  Longer rows are a workgroup each and end at 2^22 - 1."""
    some = [(1 << 22) - 1, 1 << 22, (1 << 22) + 5, 1 << 26, (1 << 31) - 1]
    calls = [make(rows, cols, dt=dt) for rows in some for dt in (BF16, F32)
             for cols in (1, 64, 513, 2048, 2049, 8192 if dt == BF16 else 4096)
             for make in (norm, norm_backward)]
    calls += [norm(1 << 23, 16384), norm((1 << 22) - 1, 16385), norm_backward((1 << 22) - 1, 8193),
              norm_backward(1 << 23, 8193, need="w")]
    for call, (status, message, got) in zip(calls, record(calls)):
        assert status == OK and got, (call, message)
        assert max(map(work_items, got)) <= MOST_ITEMS, call
    calls = [norm(1 << 22, 16385), norm_backward(1 << 22, 8193), norm(1 << 22, 8193, dt=F32)]
    for call, (status, message, got) in zip(calls, record(calls)):
        assert status != OK and "exceed one dispatch" in message and not got, call


def test_cuts_that_the_gpu_tests_mean(record):
    """test_head_edges_gpu.py is about rows that a workgroup reads in several
    chunks, by the kernel of 8 vectors a thread and by the one of 2."""
    from test_head_edges_gpu import CHUNKED
    def logprobs(n, v, dt):
        return ["vpa_token_logprobs", [P, dt, v, [v, v, 1], n, P, 1, 5, WS, HUGE, P, P, P, P, P,
                                       None]]
    calls = [logprobs(c[0], c[1], dt) for c in CHUNKED for dt in (BF16, F32)]
    want = [c[2 if dt == BF16 else 3] for c in CHUNKED for dt in (BF16, F32)]
    for call, vecs, (status, message, got) in zip(calls, want, record(calls)):
        assert status == OK, message
        part = [l for l in got if "logprob_part_kernel" in l["name"]]
        assert len(part) == 1 and part[0]["chunks"] >= 2 and part[0]["k"] == vecs, (call, part)


def test_backward_needs_what_it_says(record):
    """vpa_head_linear_backward_need is what the call checks, to the byte, and
    every launch keeps to it."""
    some = [((rows, outer, inner), act, ldg, need, dt)
            for rows, outer, inner in ((40, 512, 4096), (64, 50257, 2), (300, 4090, 785),
                                       (2048, 8192, 2047), (4096, 4352, 4096))
            for act in (0, 3) for ldg in (outer, (outer + 7) // 8 * 8, (outer + 7) // 8 * 8 + 1)
            for need in ("xwb", "x", "w", "b", "xw") for dt in (BF16, F32)]
    need = record([["vpa_head_linear_backward_need",
                    [dt, *size, int(act != 0 or ldg % (8 if dt == BF16 else 4) != 0)] +
                    [int(c in want) for c in "xwb"]] for size, act, ldg, want, dt in some])
    exact, short = [], []
    for (size, act, ldg, want, dt), (n, _, _) in zip(some, need):
        exact.append(linear_backward(*size, dt=dt, ws_bytes=n, act=act, ldg=ldg, need=want))
        short.append(linear_backward(*size, dt=dt, ws_bytes=n - 1, act=act, ldg=ldg, need=want))
    for call, (status, message, got) in zip(exact, record(exact)):
        assert status == OK and got, (call, message)
        for l in got:
            assert l["part_bytes"] == 0 or (
                l["part"] >= WS and l["part"] + l["part_bytes"] <= WS + call[1][-2]), (call, l)
    for (n, _, _), call, (status, message, got) in zip(need, short, record(short)):
        assert n == 0 or (status != OK and "workspace" in message and not got), call
