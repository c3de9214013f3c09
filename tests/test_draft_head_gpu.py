"""GPU tests of examples/draft_head.py: the head's operators run together."""
import pytest
import torch

import vocab_argmax_amd as vpa
from examples.draft_head import DraftHead

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# A chain of at most 8 operators on fp32, each off by at most 2 (n + 2) u of its
# sums of |terms|, n <= 523 terms; over random data such a sum is about sqrt(n)
# of the result's size: 8 * 2 * 525 * 2^-24 * 23 < 2^-6 of a result's norm.
CHAIN = 2.0 ** -6


def close(got, want, what):
    err = (got.double() - want).norm() / want.norm()
    assert got.shape == want.shape and float(err) <= CHAIN, (what, float(err))


def reference(head, x, targets, entropy_weight):
    """The same loss and gradients by autograd in 64 bits on the CPU."""
    p = {k: t.double().cpu().requires_grad_() for k, t in head.params.items()}
    x = x.double().cpu().requires_grad_()
    c = (x.shape[1],)
    norm = torch.nn.functional.layer_norm
    h = norm(x, c, p["norm1.weight"], p["norm1.bias"], 1e-5)
    b = h + torch.nn.functional.silu(h @ p["block.weight"].T + p["block.bias"])
    y = norm(b, c, p["norm2.weight"], p["norm2.bias"], 1e-5)
    logp = (y @ p["vocab.weight"].T).log_softmax(1)
    t = targets.long().cpu()
    lp = torch.where(t >= 0, logp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    loss = -(lp.mean() - entropy_weight * (logp.exp() * logp).sum(1).mean())
    loss.backward()
    return loss.detach(), {k: t.grad for k, t in p.items()}, x.grad, logp.detach()


def inputs(n, k, v, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(n, k, generator=g, device=DEV).to(dtype)
    return x, torch.randint(-1, v, (n,), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("n,k,v,s", [(1, 64, 131, 1), (7, 96, 515, 3), (40, 130, 523, 2)])
def test_loss_and_gradients(n, k, v, s):
    head = DraftHead(k, v, s, torch.float32, DEV, seed=n)
    x, targets = inputs(n, k, v, torch.float32, 5 + n)
    loss, grads, dx = head.loss_and_grads(x, targets, 0.25)
    want, wg, wx, logp = reference(head, x, targets, 0.25)
    close(loss.cpu(), want, "loss")
    for name in grads:
        close(grads[name].cpu(), wg[name], name)
    close(dx.cpu(), wx, "x")
    ids, r = head.decode(x, 3)
    close(r.logprobs.cpu(), logp.max(1).values, "greedy log probabilities")
    assert torch.equal(ids, r.top_ids[:, 0])


def test_training_learns_its_rows_and_verifies_them():
    """bf16, 64 rows: after some steps every row's greedy token is its target,
    and a verification that drafts the targets accepts all of them."""
    v, k = 5003, 3
    head = DraftHead(256, v, 2, torch.bfloat16, DEV, seed=3)
    x, targets = inputs(64, 256, v, torch.bfloat16, 9)
    targets.clamp_(min=0)
    first = head.train_step(x, targets, 1.0).item()
    for _ in range(60):
        last = head.train_step(x, targets, 1.0).item()
    assert last < 0.1 * first
    ids, r = head.decode(x)
    assert torch.equal(ids, targets) and torch.equal(r.top_ids[:, 0], targets)
    drafts = targets.view(16, k + 1)[:, :k].contiguous()
    out, sampled, rejected, tg, lp = head.verify(x, drafts)
    assert torch.equal(tg.view(-1), targets) and torch.equal(out.view(-1), targets)
    assert bool((sampled == k + 1).all()) and bool((rejected == 0).all())
    assert torch.equal(lp.view(-1), r.logprobs)
