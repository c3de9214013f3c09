"""The 8-bit product's fast form: the checks of test_rms_fp8_gpu.py, whose tolerances
know the instruction's cut, at the sizes at which kernels, tiles and slices change."""
import functools

import pytest
import torch

import test_fp8_plans_gpu as plans
import test_rms_fp8_gpu as base
import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, half, near

pytestmark = pytest.mark.gpu


@pytest.fixture
def fast(monkeypatch):
    monkeypatch.setattr(vpa, "head_linear_fp8", functools.partial(vpa.head_linear_fp8, fast=True))


@pytest.mark.parametrize("n,k,m", [c for c in base.FP8_CASES if c[0] > 16] + plans.PLANS)
def test_head_linear_fp8(fast, n, k, m):
    base.test_head_linear_fp8(n, k, m)


def test_infinities_and_nan(fast):
    base.test_head_linear_fp8_carries_infinities_and_nan()


@pytest.mark.parametrize("n,k,m", [(20, 1000, 500), (64, 4096, 1000), (300, 1024, 700)])
def test_other_results_are_the_same(n, k, m):
    """Up to 64 rows, and to fp32."""
    _, x, xs, w, ws = base.operands(n, n, k, m, wild=True)
    for dtype in (F32, BF) if n <= 64 else (F32,):
        assert torch.equal(vpa.head_linear_fp8(x, xs, w, ws, out_dtype=dtype, fast=True),
                           vpa.head_linear_fp8(x, xs, w, ws, out_dtype=dtype))


def test_the_cut_keeps_to_its_bound():
    """7 * 2^-13 of sum |x w|, where every group of 8 holds products that cancel."""
    from test_fp8_sums_gpu import operands
    for n, k, m in ((65, 256, 130), (300, 512, 16500), (2048, 384, 4096)):
        x, xs, w, ws, z = operands(n, n, k, m)
        mag = x.double().abs() @ w.double().abs().T
        tol = base.CUT * mag
        near(vpa.head_linear_fp8(x, xs, w, ws, fast=True), z, tol + half(BF) * (z.abs() + tol), "cut")


@pytest.mark.parametrize("n,k,m", [(128, 4096, 4096), (512, 4096, 4096), (1000, 8192, 8192),
                                   (2048, 40000, 515), (129, 2100, 5500)])
def test_workspace_streams_and_graphs(n, k, m):
    _, x, xs, w, ws = base.operands(11, n, k, m)
    want = vpa.head_linear_fp8(x, xs, w, ws, fast=True)
    need = vpa.draft_lib().vpa_head_linear_fp8_fast_workspace(n, m, k)
    assert need >= vpa.draft_lib().vpa_head_linear_fp8_workspace(n, m, k)
    buf = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert torch.equal(vpa.head_linear_fp8(x, xs, w, ws, workspace=buf[:need], fast=True), want)
    assert bool((buf[need:] == 0x5A).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = vpa.head_linear_fp8(x, xs, w, ws, fast=True, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    xx = x.clone().view(torch.uint8)
    ld = (k + 15) // 16 * 16
    xg = torch.zeros((n, ld), dtype=torch.uint8, device=DEV)
    xg[:, :k] = xx
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vpa.head_linear_fp8(xg.view(vpa.FP8)[:, :k], xs, w, ws, fast=True)
    for turn in range(3):
        xg[:, :k] = xx if turn != 1 else xx.flip(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, vpa.head_linear_fp8(xg.view(vpa.FP8)[:, :k], xs, w, ws, fast=True)), turn
