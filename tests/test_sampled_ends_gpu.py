"""Draws of the sampled verification at the ends of their random numbers, and draft
distributions that hold NaN."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, NEG, gen, randn

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("u", [1.0, 1.5, math.inf])
@pytest.mark.parametrize("v", [900, 5000, 50257])
def test_random_numbers_from_1_on_draw_the_last_weight(v, u, dtype):
    """Whatever the order of the sums: columns at the end whose weights are too small to change a
    sum of 64 bits, and a masked one after them."""
    r = 500
    x = randn(gen(v), r, v, scale=3.0)
    x[:, v - 40:] = -60.0
    x[:, v - 3:] = NEG
    x = x.to(dtype)
    none = torch.zeros((r, 0), device=DEV)
    su = torch.full((r,), u, dtype=F64, device=DEV)
    out, _, _ = vpa.sampled_verify(x, v, v, 1, none.int(), none, su)
    assert bool((out[:, 0] == v - 4).all()), out[:, 0][out[:, 0] != v - 4].tolist()[:5]
    # and of max(p - q, 0)
    x = x.repeat_interleave(2, 0)
    q = torch.full((r, v), 0.5 / v, device=DEV)
    q[:, v - 6:] = 0.0
    ids = torch.zeros((r, 1), dtype=torch.int32, device=DEV)
    q[:, 0] = 1.0
    out, n, _ = vpa.sampled_verify(x, v, v, 1, ids, torch.ones((r, 1), device=DEV), su, draft_probs=q)
    assert bool((n == 1).all()) and bool((out[:, 0] == v - 4).all())


def test_nan_in_a_draft_distribution():
    """A draft whose probability is NaN is not accepted; a column with NaN has no weight."""
    v = 3000
    x = randn(gen(2), 4, v)
    q = torch.zeros((2, v), device=DEV)
    q[0, 5] = math.nan
    q[1, 7] = 1.0
    q[1, :7] = math.nan
    ids = torch.tensor([[5], [7]], dtype=torch.int32, device=DEV)
    for s in (0.0, 0.5, 1.0):
        out, n, _ = vpa.sampled_verify(x, v, v, 1, ids, torch.full((2, 1), 0.999, device=DEV),
                                       torch.full((2,), s, dtype=F64, device=DEV), draft_probs=q)
        assert n.tolist() == [1, 1]
        w = x[0::2].double().softmax(1)
        w[0, 5] = 0
        w[1, :8] = 0
        c = w.cumsum(1)
        for i in range(2):
            want = v - 1 if s == 1 else int((c[i] > s * c[i, -1]).int().argmax())
            assert int(out[i, 0]) == want
