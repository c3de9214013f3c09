"""Calls of the draft operators that their documentation allows at its edges: the
largest vocabulary, the smallest and largest temperatures, calls on two streams at
once, graphs that share a workspace, one tensor in several places."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
MOST = 2 ** 24 - 1
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def teacher(g, n, v, k):
    ids = torch.stack([torch.randperm(v, generator=g, device=DEV)[:k] for _ in range(n)]).int()
    lp = torch.log_softmax(randn(g, n, k), 1) - 0.3
    return ids, lp


def distill_64(x, ids, lp, tail, t):
    """(loss, gradient) in 64 bits."""
    x = x.double().requires_grad_()
    logq = torch.log_softmax(x / t, 1)
    lp = lp.double()
    if not tail:
        lp = torch.log_softmax(lp, 1)
    p = lp.exp()
    loss = (p * (lp - logq.gather(1, ids.long()))).sum(1)
    if tail:
        p0 = 1 - p.sum(1)
        others = torch.ones_like(x, dtype=torch.bool).scatter(1, ids.long(), False)
        logq0 = torch.logsumexp(logq.masked_fill(~others, -math.inf), 1)
        loss = loss + p0 * (p0.log() - logq0)
    return loss.detach(), torch.autograd.grad(loss.sum(), x)[0]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_largest_vocabulary_draws_exactly(dtype):
    """Equal logits: every weight is 1, sums are whole numbers, and the token is the whole part of
    u V."""
    x = torch.zeros((1, MOST), dtype=dtype, device=DEV)
    none = torch.zeros((1, 0), dtype=torch.int32, device=DEV)
    for u in (0.0, 0.25, 0.5 + 2.0 ** -30, 12345678.5 / MOST, 1 - 2.0 ** -53):
        out, n, r = vpa.sampled_verify(x, MOST, MOST, 1, none, none.float(),
                                       torch.tensor([u], dtype=F64, device=DEV))
        assert int(out[0, 0]) == min(int(u * MOST), MOST - 1) and int(n) == 1 and int(r) == 0


def test_the_largest_vocabulary_distills():
    """Equal logits: q = 1 / V everywhere.  The sum of ones in fp32 is exact up to 2^24; logarithms
    are of 64 bits, and the results have one rounding."""
    x = torch.zeros((1, MOST), dtype=F32, device=DEV)
    ids = torch.tensor([[5, MOST - 1, -1]], dtype=torch.int32, device=DEV)
    lp = torch.tensor([[0.5, 0.25, 0.1]], device=DEV).log()
    one = torch.ones(1, device=DEV)
    loss, d = vpa.distill_loss_and_grad(x, MOST, MOST, 1, ids, lp, one)
    p = torch.tensor([2 / 3, 1 / 3], dtype=F64)
    want = float((p * (p.log() + math.log(MOST))).sum())
    assert abs(float(loss) - want) < 4 * U * want
    q = 1 / MOST
    assert abs(float(d[0, 5]) - (q - 2 / 3)) < 8 * U and abs(float(d[0, -1]) - (q - 1 / 3)) < 8 * U
    rest = d[0, 6:-1]
    assert float((rest.double() - q).abs().max()) < 16 * U * q


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("t", [2.0 ** -100, 1e-20, 1e-9, 1e-6, 1e-3, 1e3, 1e20, 3e38])
@pytest.mark.parametrize("n,v", [(3, 1000), (2, 40000), (5, 200000)])
def test_temperatures(n, v, t, tail):
    """Logits are small whole numbers: their differences are exact, a power's exponent has an error
    of 2 u of itself and powers of a sum that count have exponents above -40, so a loss is off by
    (100 + 8) u, a sum of v terms by 16 u more, relative to the loss and 1 (q sums to 1)."""
    g = gen(int(v + n))
    x = torch.randint(-8, 9, (n, v), generator=g, device=DEV).to(BF)
    ids, lp = teacher(g, n, v, 9)
    want, wd = distill_64(x.float(), ids, lp, tail, float(torch.tensor(t, dtype=F32)))
    one = torch.ones(n, device=DEV)
    t32 = float(torch.tensor(t, dtype=F32))
    loss, stats = vpa.distill_loss(x, v, v, 1, ids, lp, tail, t32)
    tol = 128 * U * (1 + want.abs())
    assert bool(((loss.double() - want).abs() <= tol).all())
    both, d = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, one, tail, t32)
    assert bool(((both.double() - want).abs() <= tol).all())
    d2 = vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, one, t32)
    # bf16 results: half a step (2^-8, or of the subnormals 2^-134), and 256 u of the terms q P and
    # p, at most 1 / t each
    for y in (d, d2):
        tol = 2.0 ** -8 * 1.01 * wd.abs() + 512 * U / t32 + 2.0 ** -133
        assert bool(((y.double() - wd).abs() <= tol).all())


@pytest.mark.parametrize("t,step,base", [
    (2.0 ** -100, 1.0, 0.0), (1e-20, 1.0, 0.0), (1e-20, 1.0, 1000.0), (1e-9, 1.0, 7.0),
    (1e-6, 0.5, 100.0), (1e-4, 1.0, -60.0), (1.0, 4096.0, 3e10), (1.0, 2.0 ** 70, -1e30),
    (1e-3, 2.0 ** 100, 1e37)])
@pytest.mark.parametrize("v", [50, 5000, 151936])
def test_nothing_but_the_largest_logits_counts(v, t, step, base):
    """Logits that are far apart next to the temperature: the largest ones, n of them, have
    probability 1 / n each and all others 0, so every sum is a whole number."""
    g = gen(v)
    x = torch.randint(-5, 3, (6, v), generator=g, device=DEV).float() * step + base
    top = x.max(1, keepdim=True).values
    ties = x == top
    count = ties.sum(1).double()
    first = ties.int().argmax(1).int()
    u = torch.rand(3, generator=g, device=DEV, dtype=F64)
    t3 = torch.full((3,), t, device=DEV)
    # requests of a draft and a bonus row: drafts of probability 1 / n, accepted just below it
    drafts = first[0::2].reshape(3, 1).contiguous()
    n = count[0::2]
    for near, accepted in ((0.999, 1), (1.001, 0)):
        au = (near / n).float().reshape(3, 1)
        out, num, _ = vpa.sampled_verify(x, v, v, 1, drafts, au, u, temperature=t3)
        assert num.tolist() == [2 if accepted or m == 1 and near / m < 1 else 1 for m in n.tolist()]
        for r in range(3):
            row = 2 * r + int(num[r]) - 1
            w = ties[row].double()
            if int(num[r]) == 1:
                w[drafts[r, 0]] = 0
            if float(w.sum()) == 0:
                want = int(drafts[r, 0])
            else:
                want = int((w.cumsum(0) > u[r] * w.sum()).int().argmax())
            assert int(out[r, int(num[r]) - 1]) == want
    # the loss against the first of them: ln n, from sums of ones
    lp = torch.zeros((6, 1), device=DEV)
    one = torch.ones(6, device=DEV)
    loss, d = vpa.distill_loss_and_grad(x, v, v, 1, first.reshape(6, 1), lp, one, False, t)
    # (the two calls cut a row differently, so they may differ in the last bits)
    for y in (loss, vpa.distill_loss(x, v, v, 1, first.reshape(6, 1), lp, False, t)[0]):
        assert bool(((y.double() - count.log()).abs() <= 4 * U * (1 + count.log())).all())
    want = ties.double() / count[:, None]
    want.scatter_add_(1, first.reshape(6, 1).long(), torch.full((6, 1), -1.0, dtype=F64, device=DEV))
    t32 = float(torch.tensor(t, dtype=F32))
    assert bool(((d.double() - want / t32).abs() <= 16 * U / t32).all())


def test_two_streams_at_once():
    g = gen(3)
    x = randn(g, 96, 50257, dtype=BF) * 3
    ids, lp = teacher(g, 96, 50257, 8)
    dids = torch.randint(0, 50257, (24, 3), generator=g, device=DEV, dtype=torch.int32)
    u, s = torch.rand(24, 3, generator=g, device=DEV), torch.rand(24, generator=g, device=DEV, dtype=F64)
    w8, ws = vpa.quantize_fp8(randn(g, 4096, 2048), 128)
    h = randn(g, 96, 2048, dtype=BF)

    def step(**kw):
        out = list(vpa.sampled_verify(x, 50257, 50257, 1, dids, u, s, **kw))
        out += list(vpa.distill_loss(x, 50257, 50257, 1, ids, lp, True, **kw))
        n = vpa.rms_norm_fp8(h, residual=h, **kw)
        out += [n.scale, n.summed, vpa.head_linear_fp8(n.y, n.scale, w8, ws, **kw)]
        return out
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step())
    torch.cuda.synchronize()
    for out in got[0] + got[1]:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_graphs_that_share_a_workspace():
    g = gen(4)
    v = 151936
    xs = [randn(g, 20, v, dtype=BF) for _ in range(2)]
    t = [teacher(g, 20, v, 5) for _ in range(2)]
    dids = torch.randint(0, v, (4, 4), generator=g, device=DEV, dtype=torch.int32)
    u, s = torch.zeros(4, 4, device=DEV), torch.rand(4, generator=g, device=DEV, dtype=F64)
    need = max(vpa.sampled_verify_workspace(v, v, 1, 4, 4), vpa.distill_workspace(v, v, 1, 20))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    calls = [lambda: vpa.sampled_verify(xs[0], v, v, 1, dids, u, s, workspace=ws),
             lambda: vpa.distill_loss(xs[1], v, v, 1, *t[1], True, workspace=ws),
             lambda: vpa.sampled_verify(xs[1], v, v, 1, dids, u, s, workspace=ws)]
    want = [[a.clone() for a in f()] for f in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in calls:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(f())
        graphs.append(gr)
    for turn in range(4):
        for i in ((0, 1, 2), (2, 1, 0))[turn % 2]:
            graphs[i].replay()
        calls[turn % 3]()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w)), turn


@pytest.mark.parametrize("c", [100, 2048, 8191, 20000])
def test_one_tensor_in_several_places(c):
    g = gen(c)
    x, w = randn(g, 70, c, dtype=BF), randn(g, c, dtype=BF)
    want = vpa.rms_norm(x * 2, w)
    got = vpa.rms_norm(x, w, residual=x)
    assert torch.equal(got.y, want.y) and torch.equal(got.summed, x * 2)
    a = x.clone()
    got = vpa.rms_norm(a, w, residual=a, summed=a)
    assert got.summed is a and torch.equal(a, x * 2) and torch.equal(got.y, want.y)
    a = x.clone()
    q, q0 = vpa.rms_norm_fp8(a, w, residual=a, summed=a), vpa.rms_norm_fp8(x * 2, w)
    assert torch.equal(q.scale, q0.scale) and torch.equal(q.y.float(), q0.y.float())
    # the gradient of y that is also that of the sum, replaced by the gradient of x
    r = vpa.rms_norm(x, w, with_rstd=True).rstd
    gr = randn(g, 70, c, dtype=BF)
    gx, gw = vpa.rms_norm_backward(gr, x, r, w, gr)
    b = gr.clone()
    assert torch.equal(vpa.rms_norm_backward(b, x, r, w, b, need_weight=False, out=b)[0], gx)
    b = gr.clone()
    out, gw2 = vpa.rms_norm_backward(gr, x, r, w, b, out=b)
    assert out is b and torch.equal(b, gx) and torch.equal(gw, gw2)


@pytest.mark.parametrize("n,v", [(3, 1000), (2, 50257), (70, 50257), (2, 151937), (130, 151937)])
def test_gradient_in_the_logits_place(n, v):
    g = gen(v)
    x = randn(g, n, v, dtype=BF)
    ids, lp = teacher(g, n, v, 64)
    one = torch.rand(n, generator=g, device=DEV)
    loss, d = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, one, True)
    y = x.clone()
    loss2, d2 = vpa.distill_loss_and_grad(y, v, v, 1, ids, lp, one, True, out=y)
    assert d2 is y and torch.equal(d, y) and torch.equal(loss, loss2)
    _, stats = vpa.distill_loss(x, v, v, 1, ids, lp, True)
    want = vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, one)
    y = x.clone()
    assert torch.equal(vpa.distill_loss_backward(y, v, v, 1, ids, lp, stats, one, out=y), want)
