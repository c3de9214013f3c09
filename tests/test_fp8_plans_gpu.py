"""8-bit products at the sizes at which their tiles, slices and stages change: the
checks of test_rms_fp8_gpu.py, against 64 bits with its tolerances."""
import pytest
import torch

import test_rms_fp8_gpu as base
import vocab_argmax_amd as vpa

pytestmark = pytest.mark.gpu

PLANS = [  # rows, inner, outer
    # 64-tiles of a few blocks of rows, in slices, whole, and with an end in each
    (65, 4096, 4096), (128, 4200, 2048), (130, 1100, 515), (192, 4095, 4096), (256, 300, 4096),
    (66, 7, 3), (65, 1, 64), (1000, 200, 1000), (16384, 130, 64),
    # 128-tiles in one round of workgroups
    (512, 4200, 4096), (1000, 1030, 4090), (1024, 1100, 4096), (70, 130, 16450), (129, 2100, 11008),
    # past it
    (1025, 600, 4096), (260, 300, 16500),
] + [  # fewer stages than buffers, as many, and one more, with and without a last one cut off
    (257, k, 4000) for k in (100, 128, 250, 256, 384, 500, 512, 520, 640, 700)
] + [(200, k, 300) for k in (100, 128, 256, 300, 384, 500, 512, 640)]


@pytest.mark.parametrize("n,k,m", PLANS)
def test_plans(n, k, m):
    base.test_head_linear_fp8(n, k, m)


@pytest.mark.parametrize("n,k,m,slices", [
    (128, 4096, 4096, 2), (512, 4096, 4096, 2), (129, 2100, 11008, 0), (129, 2100, 5500, 2)])
def test_slices_keep_to_their_workspace_and_repeat(n, k, m, slices):
    _, x, xs, w, ws = base.operands(11, n, k, m)
    for dtype in (torch.bfloat16, torch.float32):
        want = vpa.head_linear_fp8(x, xs, w, ws, out_dtype=dtype)
        need = vpa.draft_lib().vpa_head_linear_fp8_workspace(n, m, k)
        assert need == slices * n * m * 4
        buf = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(vpa.head_linear_fp8(x, xs, w, ws, out_dtype=dtype,
                                                   workspace=buf[:need]), want)
        assert bool((buf[need:] == 0x5A).all())
