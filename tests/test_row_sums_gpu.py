"""Sums of exponentials over long rows: their error does not grow with the vocabulary.

Equal logits c below several maxima of 0, so that every wavefront measures from 0:
equal terms are rounded in the same direction in every lane, which random ones hide."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, U

pytestmark = pytest.mark.gpu


def row_sum(v, c):
    tops = -(-v // 256)
    return tops + (v - tops) * math.exp(c)


def logits(n, v, c, dtype):
    x = torch.full((n, v), c, dtype=dtype, device=DEV)
    x[:, ::256] = 0.0
    return x


# an element's power: z = c log2(e) rounded (|z| < 8: 2^-22 ln 2 < 3 u), log2(e) itself (1 u), the
# instruction (2 u); a vector's 8 terms in fp32 (4 u), a chunk's 20 vectors (10 u: a step of u of
# the sums so far, half of the whole on average); 64-bit sums rounded once (1 u), joined over
# wavefronts and segments (3 + 6 u).  The tightest a sum of chunks in fp32 would do is 100 u.
SUM = 30 * U


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v", [(1024, 2 ** 21), (3, 2 ** 24 - 1), (130, 151936), (1100, 200064)])
def test_distill(n, v, dtype):
    """The loss against a maximum's column is ln s, and the gradient of the others 1 / s of theirs."""
    for c in (-1.0, -2.5, -3.0):
        x = logits(n, v, c, dtype)
        ids = torch.zeros((n, 1), dtype=torch.int32, device=DEV)
        lp = torch.zeros((n, 1), device=DEV)
        s = row_sum(v, c)
        want = math.log(s)
        loss, _ = vpa.distill_loss(x, v, v, 1, ids, lp)
        off = float((loss.double() - want).abs().max())
        assert off <= SUM + U * want, f"loss, c {c}: {off / U:.1f} u"
        one = torch.ones(n, device=DEV)
        loss, d = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, one, out=x)
        off = float((loss.double() - want).abs().max())
        assert off <= SUM + U * want, f"loss at once, c {c}: {off / U:.1f} u"
        # a power (6 u) and two products more; bf16's rounding is half a step, 2^-8
        g = math.exp(c) / s
        off = float((d[:, 1::256].double() / g - 1).abs().max())
        assert off <= SUM + 10 * U + (2.0 ** -8 if dtype is BF else 0), f"gradient, c {c}: {off / U:.1f} u"
        del x, d
