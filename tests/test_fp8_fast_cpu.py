"""The 8-bit product's fast form on the CPU: it refuses what the product refuses, its
launches fit a dispatch, and its slices lie in the workspace of the size it asks for."""
import pytest

import test_draft_cpu as base
import vocab_argmax_amd as vpa
from test_draft_launches_cpu import BF16, F32, HUGE, OK, WS, linear, record  # noqa: F401
from test_launches_cpu import MOST_ITEMS, work_items

REFUSALS = base.test_head_linear_fp8_rejects.pytestmark[0].args[1]


@pytest.mark.parametrize("kw,status", REFUSALS)
def test_refusals(monkeypatch, kw, status):
    class Fast:
        vpa_head_linear_fp8 = staticmethod(
            lambda *args: base.Calls().vpa_head_linear_fp8_fast(*args))
    monkeypatch.setattr(base, "lib", Fast())
    base.test_head_linear_fp8_rejects(kw, status)


def test_workspaces():
    lib = vpa.draft_lib()
    f = lib.vpa_head_linear_fp8_fast_workspace
    for bad in ((0, 4, 4), (-1, 4, 4), (4, 0, 4), (4, 4, 0), (1 << 31, 4, 4), (4, 1 << 31, 4)):
        assert f(*bad) == 0
    for n in (1, 64, 65, 512, 1000, 2048, 4096):
        for m in (16, 4096, 8192):
            for k in (130, 4096, 40000):
                assert f(n, m, k) == vpa.draft_call().vpa_head_linear_fp8_fast_workspace(n, m, k)
                assert f(n, m, k) >= lib.vpa_head_linear_fp8_workspace(n, m, k)


def fast(call):
    return ["vpa_head_linear_fp8_fast", call[1]]


def test_launches(record):  # noqa: F811
    sizes = [(n, m, k) for n in (1, 64, 65, 130, 300, 1000, 2048, 4340, 1 << 17)
             for m in (1, 515, 4096, 8192, 50257) for k in (1, 130, 2047, 8192, 40000)]
    need = record([["vpa_head_linear_fp8_fast_workspace", list(s)] for s in sizes])
    sizes_given = [n[0] for n in need]
    split = short = 0
    for odt in (BF16, F32):
        calls = [fast(linear(*s, odt, n)) for s, n in zip(sizes, sizes_given)]
        for call, (status, message, got) in zip(calls, record(calls)):
            assert status == OK, (call, message)
            assert got and max(map(work_items, got)) <= MOST_ITEMS, (call, got)
            for l in got:
                if "gemm_join_kernel" in l["name"]:
                    split += 1
                    assert l["part"] >= WS and l["part"] + l["part_bytes"] <= WS + call[1][-2], (call, l)
        calls = [fast(linear(*s, odt, n - 1)) for s, n in zip(sizes, sizes_given) if n]
        short += sum("workspace" in r[1] for r in record(calls))
    assert split > 20 and short > 20


def test_calls_beyond_a_dispatch_are_refused(record):  # noqa: F811
    calls = [fast(linear(1 << 23, 1 << 16, 64)), fast(linear(1 << 22, 1 << 16, 64, odt=F32))]
    for call, (status, message, got) in zip(calls, record(calls)):
        assert status != OK and "exceed one dispatch" in message and not got, (call, message, got)
