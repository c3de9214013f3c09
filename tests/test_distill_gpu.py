"""GPU tests of the distillation loss and its gradient against their
definition in 64 bits, with derived tolerances (see test_head_gpu.py)."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, NEG, SUM, U, gen, half, near, randn, strided

pytestmark = pytest.mark.gpu


def oracle(x, vocab, ids, lp, tail, temp, g=None):
    """(loss, gradient by x[:, :vocab] or None) row by row, by definition."""
    x, lp, ids = x[:, :vocab].double().cpu(), lp.double().cpu(), ids.cpu().long()
    n = x.shape[0]
    loss = torch.zeros(n, dtype=torch.float64)
    grad = torch.zeros_like(x)
    for i in range(n):
        bad = bool(((ids[i] < -1) | (ids[i] >= vocab)).any())
        use = ids[i] >= 0
        if not bool(use.any()) and not bad:
            continue
        y = lp[i][use]
        bad |= bool((y.isnan() | (y == math.inf)).any())
        bad |= bool((x[i].isnan() | (x[i] == math.inf)).any())
        if bad:
            loss[i] = grad[i] = math.nan
            continue
        if tail:
            p = y.exp()
        else:
            p = (y - y.max()).exp() if bool((y > NEG).any()) else torch.zeros_like(y)
            p = p / p.sum() if bool((y > NEG).any()) else p
        p0 = max(0.0, 1.0 - float(p.sum())) if tail else 0.0
        total = float(p.sum()) + p0
        if not bool((x[i] > NEG).any()):
            loss[i] = math.inf if total > 0 else 0.0
            continue
        z = x[i] / temp
        logq = z - z.logsumexp(0)
        at = ids[i][use]
        named = torch.zeros(vocab, dtype=torch.bool)
        named[at] = True
        term = torch.where(p > 0, p * (torch.where(p > 0, p, 1.0).log() - logq[at]), 0.0)
        loss[i] = term.sum()
        d = logq.exp() * total
        if p0 > 0:
            rest = logq.masked_fill(named, NEG)
            lq0 = rest.logsumexp(0) if bool((rest > NEG).any()) else torch.tensor(NEG)
            loss[i] += p0 * (math.log(p0) - float(lq0)) if float(lq0) > NEG else math.inf
            if float(lq0) > NEG:
                d -= p0 * (rest - lq0).exp()
        d.index_add_(0, at, -p)
        grad[i] = d / temp
    if g is not None:
        grad = grad * g.double().cpu()[:, None]
    return loss.to(DEV), grad.to(DEV)


def make(seed, n, v, cols, k, dtype, shift=0.0):
    g = gen(seed)
    x = randn(g, n, cols, scale=2.0)
    x[torch.arange(n, device=DEV), torch.randint(0, v, (n,), generator=g, device=DEV)] += \
        12 * torch.rand(n, generator=g, device=DEV)
    x = (x + shift).to(dtype)
    y = x[:, :v].float() + randn(g, n, v)
    y = y.masked_fill(y.isnan(), NEG)
    best = y.topk(min(k, v), dim=1)
    lp = best.values - y.logsumexp(1, keepdim=True)
    ids = best.indices.to(torch.int32)
    if k > v:
        ids = torch.nn.functional.pad(ids, (0, k - v), value=-1)
        lp = torch.nn.functional.pad(lp, (0, k - v), value=float("nan"))
    x[:, v:] = float("nan")                              # padding is never read
    return x, ids, lp, torch.rand(n, generator=g, device=DEV) + 0.5


def tolerances(x, v, loss, grad, temp, dtype, g):
    """s and s_o are off by SUM relative (each exponential by (|z| + 2) u too, which its weight
    2^-|z| takes away), z itself by its rounding: 2 u |x - M| / t <= 2 u span / t for what a row's
    exponentials are measured from.  The loss is a mean of such logarithms with weights that sum
    to 1; its own 64-bit terms add nothing.  A gradient's two terms are off by that relative to
    themselves, and are at most |grad| + 2 p apart from it: below, terms are at most 2 g / t."""
    fin = torch.where(torch.isfinite(x[:, :v].double()), x[:, :v].double(), 0.0)
    span = (fin.amax(1) - fin.amin(1)) / temp
    rel = SUM + 8 * U * (1 + span) + 4 * U * fin.abs().amax(1) / temp
    t_loss = rel + 2 * U * loss.abs().nan_to_num(0, 0, 0)
    size = g.double().abs() / temp
    t_grad = 3 * (rel * size)[:, None] * torch.ones_like(grad)
    return t_loss, t_grad + half(dtype) * (grad.abs().nan_to_num(0, 0, 0) + t_grad)


def check(x, v, w, s, ids, lp, tail, temp, g, what=""):
    loss, grad = oracle(x, v, ids, lp, tail, temp, g)
    t_loss, t_grad = tolerances(x, v, loss, grad, temp, x.dtype, g)
    got, stats = vpa.distill_loss(x, v, w, s, ids, lp, tail, temp)
    near(got, loss, t_loss, what + " loss")
    d = vpa.distill_loss_backward(x, v, w, s, ids, lp, stats, g, temp)
    near(d[:, :v], grad, t_grad, what + " gradient")
    assert bool((d[:, v:] == 0).all()), what + " padding"
    l2, d2 = vpa.distill_loss_and_grad(x, v, w, s, ids, lp, g, tail, temp)
    near(l2, loss, t_loss, what + " loss at once")
    near(d2[:, :v], grad, t_grad, what + " gradient at once")
    assert bool((d2[:, v:] == 0).all()), what + " padding at once"
    return got, d


CASES = [  # rows, vocab, width, shards, top
    (1, 1, 1, 1, 1), (3, 2, 1, 2, 1), (2, 7, 3, 3, 5), (3, 5, 6, 1, 9), (5, 64, 64, 1, 64),
    (4, 1000, 125, 8, 64), (1, 4097, 4097, 1, 20), (3, 8191, 4100, 2, 8), (2, 16385, 5462, 3, 64),
    (33, 50257, 16753, 3, 20), (2, 151936, 76032, 2, 5), (3, 200064, 25008, 8, 64),
    (300, 300, 300, 1, 3), (1500, 2000, 2007, 1, 8), (300, 40000, 40000, 1, 20),
]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v,w,s,k", CASES)
def test_distill(n, v, w, s, k, dtype, tail):
    x, ids, lp, g = make(n * v + k, n, v, w * s, k, dtype)
    temp = 0.7 if k == 20 else 1.0 if k != 8 else 2.5
    _, d = check(x, v, w, s, ids, lp, tail, temp, g, "whole rows")
    # odd strides, rows that are not aligned: the same columns, other lanes
    xs = strided(x[:, :v], 3, 1)
    check(xs, v, w, s, ids, lp, tail, temp, g, "strided rows")


def test_teachers_of_any_kind():
    """Ids twice, fewer tokens, none, probabilities of 0, sums above 1, ids outside, NaN."""
    v, k = 700, 6
    x, ids, lp, g = make(1, 10, v, v + 3, k, F32)
    ids[0, 3] = ids[0, 1]                                # the same token twice
    ids[1, 2:] = -1
    ids[2] = -1                                          # a padding position ...
    x[2, 5] = math.nan                                   # ... whatever it holds
    lp[3] = NEG                                          # the teacher gives nothing
    lp[4, 1] = NEG
    lp[5] = -0.2                                         # sums above 1
    ids[6, 4] = v
    ids[7, 0] = -2
    lp[8, 2] = math.nan
    lp[9] = lp[9] + 900.0                                # logits for log probabilities
    for tail in (False, True):
        a = slice(0, 9) if tail else slice(0, 10)
        loss, d = check(x[a], v, v, 1, ids[a].contiguous(), lp[a].contiguous(), tail, 1.0,
                        g[a].contiguous(), f"tail {tail}")
        assert loss[2] == 0 and bool((d[2] == 0).all())
        assert bool(loss[[6, 7, 8]].isnan().all()) and bool(d[6:9, :v].isnan().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [600, 30000])
def test_students_of_any_kind(v, dtype):
    """Masked columns named and not, all columns masked but the named, rows of the type's lowest
    value, all -inf, NaN and +inf among the named and among the others."""
    k = 4
    x, ids, lp, g = make(2, 12, v, v, k, dtype)
    ids = torch.stack([torch.tensor([7, 300, v - 1, 12], dtype=torch.int32, device=DEV)] * 12)
    lp = torch.tensor([[-0.5, -1.5, -2.5, -3.5]], device=DEV).repeat(12, 1)
    at = ids[0].long()
    x[0, 300] = NEG                                      # the loss is +inf
    x[1, ::3] = NEG
    x[1, at] = 1.0
    x[2, :] = NEG
    x[2, at] = torch.tensor([1.0, 2.0, 3.0, -1.0], device=DEV).to(dtype)   # nothing but the named
    x[3, :] = torch.finfo(dtype).min
    x[4, :] = NEG
    x[5, 100] = math.nan
    x[6, 300] = math.nan
    x[7, 100] = math.inf
    x[8, 300] = math.inf
    x[9, :] = torch.finfo(dtype).min
    x[9, at] = 2.0
    x[10, at] += 60.0                                    # the others are far below
    x[11, :] -= 60.0
    x[11, 100] = 60.0                                    # the named are
    for tail in (False, True):
        check(x, v, v, 1, ids, lp, tail, 1.0, g, f"tail {tail}")


@pytest.mark.parametrize("v", [5000, 100000])
def test_a_sure_student_keeps_the_tails_digits(v):
    """What a student leaves outside of the named tokens, e^-30 and less, is not the difference of
    two sums: the gradient over it is right relative to its own size."""
    x = randn(gen(3), 4, v)
    ids = torch.tensor([[17, 2000, 4999]], dtype=torch.int32, device=DEV).repeat(4, 1)
    lp = torch.log(torch.tensor([[0.6, 0.3, 0.05]], device=DEV)).repeat(4, 1)
    for i, lift in enumerate((20.0, 45.0, 90.0, 200.0)):
        x[i, ids[0].long()] += lift
    g = torch.ones(4, device=DEV)
    loss, grad = oracle(x, v, ids, lp, True, 1.0, g)
    got, stats = vpa.distill_loss(x, v, v, 1, ids, lp, True, 1.0)
    # each logarithm is off by SUM and by the rounding of z, |z| <= 210
    near(got, loss, SUM + 210 * 4 * U + 2 * U * loss, "loss")
    d = vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, g)
    others = torch.ones(v, dtype=torch.bool, device=DEV)
    others[ids[0].long()] = False
    want = grad[:, others]
    # r(c) to SUM and its z's rounding (|z| <= 12); p_0 = 0.05 from three exponentials of fp32
    # logarithms, half a step each on values up to 3
    near(d[:, others], want, want.abs() * (SUM + 12 * 4 * U + 16 * U + 0.95 / 0.05 * 4 * U), "gradient")


def test_gradient_against_differences():
    v, k = 40, 5
    x, ids, lp, g = make(4, 3, v, v, k, F32)
    h = 2.0 ** -6
    for tail in (False, True):
        for temp in (1.0, 2.0):
            _, stats = vpa.distill_loss(x, v, v, 1, ids, lp, tail, temp)
            d = vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, g, temp).double()
            for c in (0, 7, int(ids[0, 0]), int(ids[1, 3]), v - 1):
                e = torch.zeros_like(x)
                e[:, c] = h
                up = vpa.distill_loss(x + e, v, v, 1, ids, lp, tail, temp)[0].double()
                down = vpa.distill_loss(x - e, v, v, 1, ids, lp, tail, temp)[0].double()
                # the third derivatives of a log-sum are below 1, of the loss at most 2 of them
                tol = g.double() * (2 * h * h / 6 + 2 * (SUM + 40 * U) * 2 / h)
                near(d[:, c], g.double() * (up - down) / (2 * h), tol, f"column {c}")


@pytest.mark.parametrize("dtype,n,v", [(BF, 5, 3000), (F32, 2, 50257), (BF, 700, 20000)])
def test_gradient_in_the_logits_place_and_other_tensors(dtype, n, v):
    x, ids, lp, g = make(5, n, v, v + 5, 8, dtype)
    loss, stats = vpa.distill_loss(x, v, v, 1, ids, lp, True)
    want = vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, g)
    l2, both = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, g, True)
    a = x.clone()
    assert vpa.distill_loss_backward(a, v, v, 1, ids, lp, stats, g, out=a) is a
    assert torch.equal(a, want)
    a = x.clone()
    l3, d3 = vpa.distill_loss_and_grad(a, v, v, 1, ids, lp, g, True, out=a)
    assert d3 is a and torch.equal(a, both) and torch.equal(l2, l3)
    out = strided(torch.zeros_like(x), 9, 1)
    wide = out.as_strided((n, out.stride(0)), (out.stride(0), 1))
    vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, g, True, out=out)
    assert torch.equal(out, both)
    assert bool(wide[:-1, x.shape[1]:].isnan().all()), "past the gradient's columns"


@pytest.mark.parametrize("n,v", [(3, 1000), (4, 151936), (600, 50257)])
def test_repeats_streams_graphs_and_workspaces(n, v):
    x, ids, lp, g = make(6, n, v, v, 8, BF)
    need = vpa.distill_workspace(v, v, 1, n)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)

    def step(x, **kw):
        loss, stats = vpa.distill_loss(x, v, v, 1, ids, lp, True, **kw)
        return (loss, vpa.distill_loss_backward(x, v, v, 1, ids, lp, stats, g),
                *vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, g, True, **kw))
    want = step(x)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(step(x), want))
    assert all(torch.equal(a, b) for a, b in zip(step(x, workspace=ws[:need]), want))
    assert bool((ws[need:] == 0x5A).all())
    if need:
        with pytest.raises(vpa.VpaError, match="workspace"):
            step(x, workspace=ws[:need - 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, d = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, g, True, stream=side)
    side.synchronize()
    assert torch.equal(loss, want[2]) and torch.equal(d, want[3])
    x2 = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x2)
    for turn in range(3):
        x2.copy_(x if turn != 1 else x * 0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(x2))), turn


def test_empty_batch():
    x = torch.zeros((0, 50), device=DEV)
    ids, lp = torch.zeros((0, 3), dtype=torch.int32, device=DEV), torch.zeros((0, 3), device=DEV)
    loss, stats = vpa.distill_loss(x, 50, 50, 1, ids, lp)
    assert loss.shape == (0,)
    g = torch.zeros(0, device=DEV)
    assert vpa.distill_loss_backward(x, 50, 50, 1, ids, lp, stats, g).shape == (0, 50)
    assert vpa.distill_loss_and_grad(x, 50, 50, 1, ids, lp, g)[1].shape == (0, 50)


def test_refusals():
    x, ids, lp, g = make(7, 4, 100, 104, 3, BF)
    vpa.distill_loss(x, 100, 100, 1, ids, lp)
    stats = vpa.distill_loss(x, 100, 100, 1, ids, lp)[1]
    for args, kw, err in (
            ((x[:, :99], 100, 100, 1, ids, lp), {}, ValueError),
            ((x, 100, 100, 1, ids.long(), lp), {}, TypeError),
            ((x, 100, 100, 1, ids, lp.double()), {}, TypeError),
            ((x, 100, 100, 1, ids[:, :2], lp), {}, ValueError),
            ((x, 100, 100, 1, ids[:3].contiguous(), lp), {}, ValueError),
            ((x, 100, 100, 1, ids.cpu(), lp), {}, ValueError),
            ((x, 100, 100, 1, ids[:, :0].contiguous(), lp[:, :0].contiguous()), {}, vpa.VpaError),
            ((x, 100, 40, 2, ids, lp), {}, vpa.VpaError),
            ((x, 100, 100, 1, ids, lp), dict(temperature=0.0), vpa.VpaError),
            ((x, 100, 100, 1, ids, lp), dict(temperature=math.inf), vpa.VpaError),
            ((x, 100, 100, 1, ids, lp), dict(temperature=math.nan), vpa.VpaError),
            ((x.half(), 100, 100, 1, ids, lp), {}, TypeError)):
        with pytest.raises(err):
            vpa.distill_loss(*args, **kw)
    wide = torch.zeros((4, 65), device=DEV)
    with pytest.raises(vpa.VpaError):
        vpa.distill_loss(x, 100, 100, 1, wide.to(torch.int32), wide)
    with pytest.raises(ValueError):
        vpa.distill_loss_backward(x, 100, 100, 1, ids, lp, stats[:, :7], g)
    with pytest.raises(ValueError):
        vpa.distill_loss_backward(x, 100, 100, 1, ids, lp, stats, g[:3])
    with pytest.raises(ValueError):
        vpa.distill_loss_and_grad(x, 100, 100, 1, ids, lp, g, out=x[:, :100])
    with pytest.raises(TypeError):
        vpa.distill_loss_and_grad(x, 100, 100, 1, ids, lp, g, out=x.float())
    moved = x.as_strided((4, 104), (100, 1)) if x.is_contiguous() else x
    with pytest.raises((ValueError, vpa.VpaError)):
        vpa.distill_loss_and_grad(x, 100, 100, 1, ids, lp, g, out=moved)


def test_offsets_past_32_bits():
    v, n = 200064, 11000                                 # 2.2e9 elements
    x = torch.zeros((n, v), dtype=BF, device=DEV)
    rows = torch.tensor([0, 10733, 10734, n - 1], device=DEV)
    some, ids4, lp4, g4 = make(8, 4, v, v, 8, BF)
    x[rows] = some
    ids = torch.full((n, 8), -1, dtype=torch.int32, device=DEV)
    lp = torch.zeros((n, 8), device=DEV)
    ids[rows], lp[rows] = ids4, lp4
    g = torch.ones(n, device=DEV)
    g[rows] = g4
    want_l, want_d = oracle(some, v, ids4, lp4, True, 1.0, g4)
    t_loss, t_grad = tolerances(some, v, want_l, want_d, 1.0, BF, g4)
    loss, d = vpa.distill_loss_and_grad(x, v, v, 1, ids, lp, g, True, out=x)
    near(loss[rows], want_l, t_loss, "loss")
    near(d[rows], want_d, t_grad, "gradient")
    loss[rows] = 0
    assert bool((loss == 0).all())
    d[rows] = 0
    assert not bool(d.view(torch.int16).any())
