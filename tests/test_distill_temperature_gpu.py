"""A teacher softened by the temperature as well as the student, in the two ways that
the documentation names, against 64 bits."""
import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import DEV, SUM, U, gen, near, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [0.5, 1.0, 2.0, 5.0])
def test_softened_teachers(t):
    n, v, k = 20, 300, 8
    g = gen(int(10 * t))
    x, y = randn(g, n, v, scale=2.0), randn(g, n, v, scale=2.0)
    q = torch.log_softmax(x.double() / t, 1)
    p = torch.log_softmax(y.double() / t, 1)
    # log probabilities of fp32: half a step each, on values up to 40; the sums as SUM says
    tol = SUM + 40 * 8 * U
    soft = vpa.token_logprobs(y / t, v, v, 1, n_top=k)
    ids, own = soft.top_ids, p.gather(1, soft.top_ids.long())
    lq = q.gather(1, ids.long())
    # without a tail: of the softened logits, and of the others' log probabilities / t
    w = torch.log_softmax(own, 1)
    want = (w.exp() * (w - lq)).sum(1)
    near(vpa.distill_loss(x, v, v, 1, ids, soft.top_logprobs, temperature=t)[0], want, tol, "softened")
    hard = vpa.token_logprobs(y, v, v, 1, n_top=k)
    assert torch.equal(hard.top_ids, ids)
    near(vpa.distill_loss(x, v, v, 1, ids, hard.top_logprobs / t, temperature=t)[0], want, tol, "l / t")
    # with one: what the softened teacher leaves to all other columns
    others = torch.ones((n, v), dtype=torch.bool, device=DEV).scatter(1, ids.long(), False)
    q0 = q.masked_fill(~others, -float("inf")).logsumexp(1)
    p0 = p.masked_fill(~others, -float("inf")).logsumexp(1)
    want = (own.exp() * (own - lq)).sum(1) + p0.exp() * (p0 - q0)
    # p_0 is what 8 probabilities of fp32 logarithms leave of 1: its logarithm's error counts
    # p_0 times, so it is theirs
    near(vpa.distill_loss(x, v, v, 1, ids, soft.top_logprobs, tail=True, temperature=t)[0], want,
         tol, "softened, tail")
