"""The norm over the whole range of its types: rows whose squares, or the sum of
them, lie outside of fp32."""
import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, U, gen, half, near, randn

pytestmark = pytest.mark.gpu

COLS = [7, 64, 513, 4096, 8192, 16384, 20000]


def rows(c, dtype):
    """Rows around 1e-30 .. 1e36, one of a single size, one with a small half."""
    x = randn(gen(c), 8, c)
    for i, scale in enumerate((1e-30, 1e-24, 1e-12, 3e17, 1e19, 1e30, 1e36)):
        x[i] *= scale
    x[7] = 2.0 ** 64
    x[7, ::2] = 2.0 ** -60
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", COLS)
def test_rows_of_any_size(c, dtype):
    """The mean of squares is of 64 bits, so rstd is off by the roundings of its own few fp32
    steps (half a step each: the mean's mantissa, its root, the inverse), y by two products'."""
    x = rows(c, dtype)
    d = x.double()
    rstd = 1 / d.square().mean(1, keepdim=True).sqrt()
    got = vpa.rms_norm(x, eps=0.0, with_rstd=True)
    near(got.rstd[:, None], rstd, 4 * U * rstd, "rstd")
    want = d * rstd
    tol = 6 * U * want.abs()
    # (results of the last row's small half lie below fp32's normal range: a step of 2^-149)
    near(got.y, want, tol + half(dtype) * want.abs() + 2.0 ** -133, "y")
    q = vpa.rms_norm_fp8(x, eps=0.0)
    pad = torch.nn.functional.pad(want.abs(), (0, -c % 128)).view(8, -1, 128).amax(2)
    pad = pad.clamp(min=2.0 ** -100)                     # the least that a scale is made of
    near(q.scale, pad / 448.0, 8 * U * pad / 448.0, "scale")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", COLS)
def test_gradients_of_rows_of_any_size(c, dtype):
    """grad_x is of the size of rstd: 1e-30 for rows around 1e30.  Sums over a row as in the other
    tests of the norm: `depth` terms one after another."""
    x = rows(c, dtype)
    # (below 1e-12 and at 1e36 the results leave bf16 and fp32 or come near to it)
    x = x[2:6]
    g = randn(gen(c + 1), 4, c, dtype=dtype)
    rstd = vpa.rms_norm(x, eps=0.0, with_rstd=True).rstd
    d = x.double()
    r = 1 / d.square().mean(1, keepdim=True).sqrt()
    xh, u = d * r, g.double()
    mean = (u * xh).mean(1, keepdim=True)
    want = r * (u - xh * mean)
    depth = min(c, 70) + c / 64 + 16
    rel = (depth + 12) * U
    tol = r * (rel * u.abs() + xh.abs() * (rel * (u * xh).abs().mean(1, keepdim=True) +
                                           rel * mean.abs())) + 2 * U * want.abs()
    gx, gw = vpa.rms_norm_backward(g, x, rstd)
    near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
    w = (u * xh).sum(0)
    tol = (4 + 16) * U * (u * xh).abs().sum(0)
    near(gw, w, tol + half(dtype) * (w.abs() + tol), "grad_weight")


def test_the_sum_keeps_small_rows_apart_from_eps():
    """eps counts next to squares far below fp32's range."""
    x = torch.full((1, 300), 2.0 ** -80, device=DEV)
    got = vpa.rms_norm(x, eps=2.0 ** -120, with_rstd=True)
    near(got.rstd, torch.full((1,), 2.0 ** 60, dtype=torch.float64, device=DEV), 4 * U * 2.0 ** 60, "rstd")
    got = vpa.rms_norm(x, eps=0.0, with_rstd=True)
    assert float(got.rstd) == 2.0 ** 80 and bool((got.y == 1).all())


@pytest.mark.parametrize("c", [100, 4096, 20000])
def test_the_ends_of_the_range(c):
    """Roots below 2^-128 have an infinite rstd; the largest finite rows have their norm."""
    x = torch.zeros((3, c), device=DEV)
    x[1] = 2.0 ** -140
    x[2] = torch.finfo(F32).max
    got = vpa.rms_norm(x, eps=0.0, with_rstd=True)
    assert bool(got.rstd[:2].isinf().all()) and bool(got.y[0].isnan().all())
    assert bool(got.y[1].isinf().all())
    # (1 / the largest lies below the normal numbers, at a step of 2^-149)
    near(got.rstd[2:], torch.full((1,), 2.0 ** -128, dtype=torch.float64, device=DEV), 2.0 ** -148, "rstd")
    near(got.y[2:], torch.ones((1, c), dtype=torch.float64, device=DEV), 2.0 ** -20, "y")
