"""GPU tests of the head's operators against plain 64-bit forms.

Tolerances are derived, not tuned.  h(t) is half a step of type t relative to
a value (torch.finfo(t).eps / 2); u = 2^-24 is fp32's.  A sum of n terms in
fp32, however ordered, is off by at most n u sum |terms|; the matrix cores
may drop what is below the last bit, a whole step: 2 u.
"""
import math

import pytest
import torch

import vocab_argmax_amd as vpa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
NEG = float("-inf")


def half(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def strided(t, pad, offset=0):
    """t's values in a wider buffer: row stride t.shape[1] + pad, starting
    `offset` elements in (so that rows need not be aligned)."""
    r, c = t.shape
    buf = torch.full((r * (c + pad) + offset + pad,), float("nan"), dtype=t.dtype, device=DEV)
    view = buf[offset:].as_strided((r, c), (c + pad, 1))
    view.copy_(t)
    return view


def near(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, what
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = bad.nonzero()[0].tolist()
        t = torch.as_tensor(tol, device=DEV).expand_as(want)[tuple(i)].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i} got "
                             f"{got[tuple(i)].item()!r}, want {want[tuple(i)].item()!r}, tol {t:.3g}")


# ---------------------------------------------------------------------------
# token log probabilities
# ---------------------------------------------------------------------------

def logprob_oracle(x, vocab, tok, n_top):
    """(logprobs, lse, entropy, top_ids, top_logprobs) in 64 bits by definition."""
    x = x[:, :vocab].double()
    n = x.shape[0]
    bad = (x.isnan() | (x == math.inf)).any(1)
    empty = (x == NEG).all(1)
    m = x.masked_fill(x.isnan(), NEG).amax(1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    d = x - m
    s = d.exp().sum(1, keepdim=True)
    logp = d - s.log()                          # all -inf: -inf - -inf
    logp[empty] = NEG
    logp[bad] = math.nan
    p = logp.exp()
    ent = -torch.where(p == 0, 0.0, p * logp).sum(1)
    ent[bad] = math.nan
    lse = (m + s.log())[:, 0]
    lse[empty], lse[bad] = NEG, math.nan
    lp = None
    if tok is not None:
        t = tok.long().view(n, -1)
        ok = (t >= 0) & (t < vocab)
        lp = torch.where(ok, logp.gather(1, t.clamp(0, vocab - 1)),
                         torch.where(t == -1, 0.0, math.nan)).view(tok.shape)
    # the argmax order: NaN first, then by value, lower id first (a stable sort)
    ids = x.sort(dim=1, descending=True, stable=True).indices[:, :n_top] if n_top else None
    tops = logp.gather(1, ids) if n_top else None
    return lp, lse, ent, ids, tops


# s: at most 64 terms a thread in a row, then trees; each 2^z is off by
# (|z| + 2) u relative, and terms with a large |z| weigh 2^-|z|: |z| 2^z <= 0.54
SUM = (64 + 32) * U


def check_logprobs(r, x, vocab, tok, n_top, what):
    lp, lse, ent, ids, tops = logprob_oracle(x, vocab, tok, n_top)
    if tok is not None:
        near(r.logprobs, lp, SUM + 4 * U * lp.abs().nan_to_num(0, 0, 0), what + " logprobs")
    near(r.lse, lse, SUM + 4 * U * lse.abs().nan_to_num(0, 0, 0), what + " lse")
    near(r.entropy, ent, 3 * SUM * (1 + ent.abs().nan_to_num(0, 0, 0)), what + " entropy")
    if n_top:
        assert torch.equal(r.top_ids.long(), ids), what + " top_ids"
        near(r.top_logprobs, tops, SUM + 4 * U * tops.abs().nan_to_num(0, 0, 0),
             what + " top_logprobs")


LOGPROB_CASES = [  # rows, vocab, width, shards, tokens, top
    (1, 1, 1, 1, 1, 1), (3, 2, 1, 2, 1, 2), (2, 7, 3, 3, 2, 5), (5, 64, 64, 1, 1, 64),
    (4, 1000, 125, 8, 64, 64), (1, 4097, 4097, 1, 1, 20), (3, 8191, 4100, 2, 3, 8),
    (2, 16385, 5462, 3, 1, 64), (33, 50257, 16753, 3, 1, 20), (2, 151936, 76032, 2, 1, 5),
    (7, 200064, 25008, 8, 4, 0), (300, 300, 300, 1, 1, 3), (1500, 20000, 20000, 1, 1, 5),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v,w,s,t,top", LOGPROB_CASES)
def test_token_logprobs(n, v, w, s, t, top, dtype):
    g = gen(n * v + t)
    x = randn(g, n, w * s, dtype=dtype, scale=3.0)
    x[:, v:] = float("nan")                              # padding is never read
    tok = torch.randint(0, v, (n, t), generator=g, device=DEV, dtype=torch.int32)
    check_logprobs(vpa.token_logprobs(x, v, w, s, tok, top), x, v, tok, top, "whole rows")
    one = tok[:, 0].contiguous()
    xs = strided(x[:, :v], 3, 1)                         # odd stride, rows not aligned
    r = vpa.token_logprobs(xs, v, w, s, one, min(top, 2))
    check_logprobs(r, x, v, one, min(top, 2), "strided rows")
    # shard by shard, then joined in rank order
    parts = []
    for k in range(s):
        xr = x[:, k * w:(k + 1) * w]
        parts.append(vpa.logprob_stats(xr, v, w, s, tok, top, first_shard=k, n_local=1))
    rec = torch.cat(parts)
    assert torch.equal(rec, vpa.logprob_stats(x, v, w, s, tok, top))
    check_logprobs(vpa.combine_logprobs(rec, v, w, tok, top), x, v, tok, top, "sharded rows")


def special_rows(dtype, v):
    """Rows whose masks, infinities, NaN and ties could go wrong."""
    g = gen(v)
    x = randn(g, 16, v, dtype=dtype, scale=2.0)
    low = torch.finfo(dtype).min
    x[0] = NEG                                           # the mask leaves nothing
    x[1] = low                                           # masked with the lowest value
    x[2] = NEG
    x[2, v // 2] = -7.0                                  # one token left
    x[3, ::2] = NEG
    x[4, ::2] = low
    x[5, v - 1] = float("nan")
    x[6] = float("nan")
    x[7, v // 3] = float("inf")
    x[8] = 1.25                                          # all equal
    x[9] = torch.arange(v, device=DEV).to(dtype)         # ascending
    x[10] = -torch.arange(v, device=DEV).to(dtype)       # descending
    x[11] = 0.0
    x[11, ::3] = -0.0                                    # equal to +0 in the order
    x[12, 0] = 3.0e38
    x[13] = x[13] * 1e30
    x[14, :] = NEG
    x[14, :min(v, 3)] = low                              # lowest values beside masked ones
    x[15, v // 2:] = NEG
    return x


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v,s,top", [(5, 2, 5), (1000, 3, 20), (9000, 2, 64), (40000, 5, 8)])
def test_special_rows(v, s, top, dtype):
    x = special_rows(dtype, v)
    w = -(-v // s)
    tok = torch.tensor([[0, v // 2, v - 1, -1, v, v + 70000, -2]] * 16, dtype=torch.int32, device=DEV)
    buf = torch.full((16, w * s), float("nan"), dtype=dtype, device=DEV)
    buf[:, :v] = x
    r = vpa.token_logprobs(buf, v, w, s, tok, top)
    check_logprobs(r, x, v, tok, top, "special")
    rec = vpa.logprob_stats(buf, v, w, s, tok, top)
    check_logprobs(vpa.combine_logprobs(rec, v, w, tok, top), x, v, tok, top, "special, sharded")


def grad_oracle(x, v, tok, gl, ge, stats):
    """The formula in 64 bits, and the sum of its terms' magnitudes."""
    xd = x[:, :v].double()
    mx, ls, h = (stats[:, i:i + 1].double() for i in range(3))
    empty = (mx == NEG) & (ls == 0)
    lp = (xd - mx) - ls
    p = lp.exp()
    t = tok.long().view(x.shape[0], -1)
    ok = (t >= 0) & (t < v)
    g = torch.where(ok, gl.double().view(t.shape), 0.0)
    e = torch.zeros_like(mx) if ge is None else ge.double()[:, None]
    lpe = torch.where(lp == NEG, 0.0, lp)
    d = torch.where(lp == NEG, 0.0, -p * (g.sum(1, keepdim=True) + e * (lpe + h)))
    mag = p * (g.abs().sum(1, keepdim=True) + e.abs() * (lpe.abs() + h.abs()))
    hot, hot_mag = torch.zeros_like(d), torch.zeros_like(d)
    hot.scatter_add_(1, t.clamp(0, v - 1), g)
    hot_mag.scatter_add_(1, t.clamp(0, v - 1), g.abs())
    d = torch.where(empty, 0.0, d + hot)
    # p is off by (|log p| + 2) 2 u relative, the rest by a few roundings; at
    # most 64 given tokens are summed
    tol = (2 * (lpe.abs() + 2) + 8) * U * mag + 66 * U * (hot_mag + mag)
    return d, tol.nan_to_num(0, 0, 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v,w,s,t", [(1, 1, 1, 1, 1), (3, 7, 4, 2, 3), (4, 1000, 125, 8, 64),
                                       (5, 50257, 16753, 3, 2), (2, 16385, 16400, 1, 1)])
def test_logprobs_backward(n, v, w, s, t, dtype):
    g = gen(7 * v + n)
    x = randn(g, n, w * s, dtype=dtype, scale=3.0)
    x[:, v:] = float("nan")
    if v > 100:
        x[0, 10:60] = NEG
    tok = torch.randint(0, v, (n, t), generator=g, device=DEV, dtype=torch.int32)
    if t > 1:
        tok[:, 1] = tok[:, 0]                            # one token twice
        tok[0, t - 1] = -1
    gl, ge = randn(g, n, t), randn(g, n, scale=0.1)
    r = vpa.token_logprobs(x, v, w, s, tok)
    for e in (ge, None):
        want, tol = grad_oracle(x, v, tok, gl, e, r.row_stats)
        tol = tol + half(dtype) * want.abs() + torch.finfo(F32).tiny
        got = vpa.token_logprobs_backward(x, v, w, s, tok, r.row_stats, gl, e)
        near(got[:, :v], want, tol, "gradient")
        assert bool((got[:, v:] == 0).all())
        # shard by shard
        parts = [vpa.token_logprobs_backward(x[:, k * w:(k + 1) * w], v, w, s, tok, r.row_stats,
                                             gl, e, first_shard=k, n_local=1) for k in range(s)]
        assert torch.equal(torch.cat(parts, 1), got)
        # unaligned strided rows, replaced in place
        xs = strided(x, 5, 1)
        got2 = vpa.token_logprobs_backward(xs, v, w, s, tok, r.row_stats, gl, e, out=xs)
        assert got2.data_ptr() == xs.data_ptr() and torch.equal(xs, got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_of_special_rows(dtype):
    v = 1000
    x = special_rows(dtype, v)
    tok = torch.tensor([[0, v // 2, -1, v + 5]] * 16, dtype=torch.int32, device=DEV)
    gl = randn(gen(3), 16, 4)
    ge = randn(gen(4), 16)
    r = vpa.token_logprobs(x, v, v, 1, tok)
    want, tol = grad_oracle(x, v, tok, gl, ge, r.row_stats)
    got = vpa.token_logprobs_backward(x, v, v, 1, tok, r.row_stats, gl, ge)
    near(got, want, tol + half(dtype) * want.abs().nan_to_num(0, 0, 0) + torch.finfo(F32).tiny,
         "special gradient")
    assert bool((got[0] == 0).all())                     # nothing left: no gradient
    for row in (5, 6, 7):
        assert bool(got[row].isnan().all())


def test_logprob_gradient_against_differences():
    """The gradient is the difference quotient of the forward call's loss."""
    v = 50
    x = randn(gen(1), 2, v)
    tok = torch.tensor([[3, 3], [49, 0]], dtype=torch.int32, device=DEV)
    gl, ge = randn(gen(2), 2, 2), randn(gen(3), 2)
    r = vpa.token_logprobs(x, v, v, 1, tok)
    got = vpa.token_logprobs_backward(x, v, v, 1, tok, r.row_stats, gl, ge).double()
    h = 2.0 ** -7

    def loss(d):
        q = vpa.token_logprobs(x + d, v, v, 1, tok)
        return (q.logprobs.double() * gl).sum(1) + q.entropy.double() * ge
    scale = 1 + gl.abs().sum(1) + ge.abs() * 8
    for c in (0, 3, 17, 49):
        d = torch.zeros_like(x)
        d[:, c] = h
        quot = (loss(d) - loss(-d)) / (2 * h)
        # the third derivative is below 4 scale; the losses are off by SUM scale each
        tol = 4 * scale * h * h / 6 + 4 * SUM * scale / h
        near(got[:, c], quot, tol, f"column {c}")


# ---------------------------------------------------------------------------
# the head's products
# ---------------------------------------------------------------------------

ACT = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z / (1 + (-z).exp()),
       "gelu": lambda z: 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))}


def slope(act, z):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        q = 1 / (1 + (-z).exp())
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * (-z * z / 2).exp() / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


LINEAR_CASES = [  # rows, inner, outer
    (1, 1, 1), (1, 7, 3), (1, 4096, 4096), (2, 64, 50), (3, 65, 129), (5, 1000, 1001),
    (16, 512, 256), (17, 2048, 640), (32, 2048, 1000), (33, 96, 77), (64, 1024, 512),
    (65, 130, 260), (128, 256, 256), (129, 257, 255), (256, 512, 768), (300, 64, 1031),
    (512, 2048, 513), (1000, 72, 520),
]


def linear_oracle(x, w, b, act, r):
    """y in 64 bits and a bound on the fp32 computation's error before y's rounding."""
    xd, wd = x.double(), w.double()
    z = xd @ wd.T
    dz = (x.shape[1] + 2) * 2 * U * (xd.abs() @ wd.abs().T)
    if b is not None:
        z = z + b.double()
    dz = dz + 2 * U * z.abs()
    y = ACT[act](z)
    # |act'| <= 1.13; the activation itself is off by a few steps of its terms
    # (2^z within 1 + |z| steps, and 1 / (1 + e) damps a large |z|; erf within 4)
    dy = 1.13 * dz + (0 if act in ("none", "relu") else 12 * U * (z.abs() + 1))
    if r is not None:
        y = y + r.double()
        dy = dy + U * y.abs()
    return z, dz, y, dy


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,k,m", LINEAR_CASES)
def test_head_linear(n, k, m, dtype):
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=dtype), randn(g, m, k, dtype=dtype, scale=k ** -0.5)
    b, r = randn(g, m, dtype=dtype), randn(g, n, m, dtype=dtype)
    acts = ("none", "relu", "gelu", "silu")
    for i, (act, bias, res) in enumerate((a, bb, rr) for a in acts for bb, rr in
                                         ((None, None), (b, r))):
        z, dz, y, dy = linear_oracle(x, w, bias, act, res)
        got = vpa.head_linear(x, w, bias, act, res)
        near(got, y, dy + half(dtype) * (y.abs() + dy), f"{act} {i}")
    # fp32 output, the kept pre-activation, odd strides, rows not aligned
    z, dz, y, dy = linear_oracle(x, w, b, "silu", r)
    out = torch.full((n, m + 3), 7.0, device=DEV)
    y32, pre = vpa.head_linear(strided(x, 3, 1), strided(w, 1, 3), b, "silu", strided(r, 5, 2),
                               out=out[:, 1:m + 1], with_pre=True)
    near(y32, y, dy + U * y.abs(), "fp32 output")
    near(pre, z, dz + half(dtype) * (z.abs() + dz), "pre")
    assert bool((out[:, 0] == 7.0).all()) and bool((out[:, m + 1:] == 7.0).all())
    # in the residual's place
    rr = strided(r, 8)
    vpa.head_linear(x, w, b, "silu", rr, out=rr)
    near(rr, y, dy + half(dtype) * (y.abs() + dy), "in place")


def test_head_linear_carries_infinities_and_nan():
    """Operands that are not finite show in the rows and columns they reach only."""
    g = gen(5)
    x, w = randn(g, 40, 200, dtype=BF), randn(g, 70, 200, dtype=BF)
    x[3, 199] = float("nan")
    w[5, 0] = float("inf")
    y = vpa.head_linear(x, w)
    want = (x.double() @ w.double().T)
    assert torch.equal(y.isnan(), want.isnan()) and bool(y[3].isnan().all())
    assert torch.equal(y.isinf(), want.isinf())
    x32, w32 = x.float(), w.float()
    y = vpa.head_linear(x32, w32)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("n,k,m", [(1, 1, 1), (1, 129, 70), (3, 65, 129), (64, 256, 320),
                                   (100, 130, 1031), (257, 512, 600), (513, 96, 2049)])
def test_head_linear_backward(n, k, m, act, dtype):
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=dtype), randn(g, m, k, dtype=dtype, scale=k ** -0.5)
    b, gr = randn(g, m, dtype=dtype), randn(g, n, m, dtype=dtype)
    _, pre = vpa.head_linear(x, w, b, act, with_pre=True)
    s = slope(act, pre.double())
    dz = gr.double() * s
    # dz: a few steps of the slope's terms, then (with an activation) its rounding
    z = pre.double().abs()
    off = 0 * dz if act == "none" else gr.double().abs() * 16 * U * (1 + z)
    rounded = off if act == "none" else off + half(dtype) * (dz.abs() + off)
    xs, ws, gs = (strided(t, 3, 1) for t in (x, w, gr))
    for args in ((gr, x, w), (gs, xs, ws)):
        gx, gw, gb = vpa.head_linear_backward(*args, pre, act)
        want = dz @ w.double()
        tol = rounded @ w.double().abs() + (m + 2) * 2 * U * (dz.abs() @ w.double().abs())
        near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
        want = dz.T @ x.double()
        tol = rounded.T @ x.double().abs() + (n + 2) * 2 * U * (dz.T.abs() @ x.double().abs())
        near(gw, want, tol + half(dtype) * (want.abs() + tol), "grad_weight")
        want = dz.sum(0)
        tol = off.sum(0) + (n + 2) * U * dz.abs().sum(0)
        near(gb, want, tol + half(dtype) * (want.abs() + tol), "grad_bias")
    only = vpa.head_linear_backward(gr, x, w, pre, act, need_x=False, need_bias=False)
    assert only[0] is None and only[2] is None and torch.equal(
        only[1], vpa.head_linear_backward(gr, x, w, pre, act)[1])


def test_linear_gradient_against_differences():
    g = gen(11)
    x, w, b = randn(g, 3, 5), randn(g, 4, 5), randn(g, 4)
    gr = randn(g, 3, 4)
    for act in ("silu", "gelu"):
        y, pre = vpa.head_linear(x, w, b, act, with_pre=True)
        gx, gw, gb = vpa.head_linear_backward(gr, x, w, pre, act)
        h = 2.0 ** -6

        def loss(dx, dw):
            return (vpa.head_linear(x + dx, w + dw, b, act).double() * gr).sum()
        size = float(gr.abs().sum()) * 40
        tol = size * (h * h + 16 * U / h)
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        dx[1, 2] = h
        near(gx[1, 2], (loss(dx, 0 * dw) - loss(-dx, 0 * dw)) / (2 * h), tol, act)
        dw[3, 4] = h
        near(gw[3, 4], (loss(0 * dx, dw) - loss(0 * dx, -dw)) / (2 * h), tol, act)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

NORM_CASES = [(1, 1), (1, 2), (3, 7), (2, 63), (5, 64), (4, 257), (33, 1000), (7, 1601),
              (32, 4096), (3, 8192), (2, 12289), (1, 70001), (700, 520), (2100, 96)]


def norm_bound(c):
    """Roundings of one row's sum: a thread's share, the tree, and the rest."""
    return (math.ceil(c / 64) + 32) * U


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("n,c", NORM_CASES)
def test_layer_norm(n, c, dtype, wdtype):
    g = gen(n * 100003 + c)
    x = (randn(g, n, c) * 2 + 3).to(dtype)
    w, b = randn(g, c, dtype=wdtype), randn(g, c, dtype=wdtype)
    eps = 1e-5
    xd = x.double()
    mu = xd.mean(1, keepdim=True)
    var = (xd - mu).square().mean(1, keepdim=True)
    rs = 1 / (var + eps).sqrt()
    k = norm_bound(c)
    dmu = k * xd.abs().mean(1, keepdim=True)             # error of the mean
    # relative error of rstd: half of the variance's, to which the mean's adds its square
    drs = k + 0.5 * (dmu * dmu + 2 * U * dmu * rs.reciprocal()) / (var + eps)
    for ww, bb in ((None, None), (w, b), (w, None), (None, b)):
        scale = 1.0 if ww is None else ww.double()
        shift = 0.0 if bb is None else bb.double()
        want = (xd - mu) * rs * scale + shift
        part = ((xd - mu) * rs * scale).abs()
        tol = (rs * dmu) * abs(scale) + part * (drs + 4 * U) + U * want.abs()
        got, mean, rstd = vpa.layer_norm(x, ww, bb, eps, with_stats=True)
        near(got, want, tol + half(dtype) * (want.abs() + tol), "y")
        near(mean, mu[:, 0], dmu[:, 0], "mean")
        near(rstd, rs[:, 0], rs[:, 0] * (drs[:, 0] + 4 * U), "rstd")
        xs = strided(x, 3, 1)
        assert torch.equal(vpa.layer_norm(xs, ww, bb, eps), got)
        vpa.layer_norm(xs, ww, bb, eps, out=xs)          # in place
        assert torch.equal(xs, got)


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("n,c", NORM_CASES)
def test_layer_norm_backward(n, c, dtype, wdtype):
    g = gen(n * 100003 + c + 1)
    x = (randn(g, n, c) * 2 + 3).to(dtype)
    w, gr = randn(g, c, dtype=wdtype), randn(g, n, c, dtype=dtype)
    _, mean, rstd = vpa.layer_norm(x, w, None, with_stats=True)
    rs = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * rs
    gd = gr.double()
    k = norm_bound(c)
    for ww in (w, None):
        u = gd * (1.0 if ww is None else ww.double())
        a, b = u.mean(1, keepdim=True), (u * xh).mean(1, keepdim=True)
        aa, bb = u.abs().mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
        want = rs * (u - a - xh * b)
        tol = rs * (8 * U * (u.abs() + aa + xh.abs() * bb) + k * (aa + xh.abs() * bb))
        gx, gw, gb = vpa.layer_norm_backward(gr, x, mean, rstd, ww)
        near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
        ot = dtype if ww is None else wdtype
        assert gw.dtype == gb.dtype == ot
        want = (gd * xh).sum(0)
        tol = (n + 6) * U * (gd * xh).abs().sum(0)
        near(gw, want, tol + half(ot) * (want.abs() + tol), "grad_weight")
        want = gd.sum(0)
        tol = (n + 2) * U * gd.abs().sum(0)
        near(gb, want, tol + half(ot) * (want.abs() + tol), "grad_bias")
        # strided, unaligned; each output alone
        got = vpa.layer_norm_backward(strided(gr, 3, 1), strided(x, 1, 3), mean, rstd, ww)
        assert all(torch.equal(p, q) for p, q in zip(got, (gx, gw, gb)))
        only = vpa.layer_norm_backward(gr, x, mean, rstd, ww, need_weight=False, need_bias=False)
        assert torch.equal(only[0], gx) and only[1] is None and only[2] is None
        only = vpa.layer_norm_backward(gr, x, mean, rstd, ww, need_x=False, need_bias=False)
        assert torch.equal(only[1], gw) and only[0] is None and only[2] is None


def test_layer_norm_of_constant_and_special_rows():
    x = torch.full((4, 300), 5.0, device=DEV)
    x[1, 7] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e6 + torch.arange(300, device=DEV) % 2
    y = vpa.layer_norm(x)
    assert bool((y[0] == 0).all()) and bool(y[1].isnan().all()) and bool(y[2].isnan().all())
    want = torch.nn.functional.layer_norm(x[3:].double(), (300,))
    # the mean is exact to a step of 1e6 = 2^-4; the spread is 1
    near(y[3:], want, 2.0 ** -3, "large mean")
    assert bool(vpa.layer_norm(x[:1], eps=0.0).isnan().all())   # 0 / 0


# ---------------------------------------------------------------------------
# streams, graphs, empty batches, determinism
# ---------------------------------------------------------------------------

def _head_step(x, nw, nb, w, tok, gl):
    """Norm, residual block, LM head, log probabilities and every gradient."""
    h, mean, rstd = vpa.layer_norm(x, nw, nb, with_stats=True)
    logits = vpa.head_linear(h, w)
    r = vpa.token_logprobs(logits, w.shape[0], w.shape[0], 1, tok, n_top=4)
    d = vpa.token_logprobs_backward(logits, w.shape[0], w.shape[0], 1, tok, r.row_stats, gl)
    gh, gw, gb = vpa.head_linear_backward(d, h, w)
    gx, gnw, gnb = vpa.layer_norm_backward(gh, x, mean, rstd, nw)
    return r.logprobs, r.entropy, r.top_ids, gx, gw, gb, gnw, gnb


def _step_inputs(n, k, v, seed):
    g = gen(seed)
    return (randn(g, n, k, dtype=BF), randn(g, k, dtype=F32), randn(g, k, dtype=F32),
            randn(g, v, k, dtype=BF, scale=k ** -0.5),
            torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32), randn(g, n))


@pytest.mark.parametrize("n", [1, 24, 300])
def test_step_repeats_bit_for_bit_and_replays_from_a_graph(n):
    ins = _step_inputs(n, 512, 5003, n)
    want = _head_step(*ins)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(_head_step(*ins), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _head_step(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _head_step(*ins)
    for rep in range(3):
        new = _step_inputs(n, 512, 5003, 900 + rep)
        for t, s in zip(ins, new):
            t.copy_(s)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, _head_step(*ins))), rep


def test_explicit_stream():
    ins = _step_inputs(40, 256, 3001, 5)
    want = _head_step(*ins)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, nw, nb, w, tok, gl = ins
    h, mean, rstd = vpa.layer_norm(x, nw, nb, with_stats=True, stream=side)
    logits = vpa.head_linear(h, w, stream=side)
    r = vpa.token_logprobs(logits, 3001, 3001, 1, tok, n_top=4, stream=side)
    d = vpa.token_logprobs_backward(logits, 3001, 3001, 1, tok, r.row_stats, gl, stream=side)
    gh, gw, gb = vpa.head_linear_backward(d, h, w, stream=side)
    gx, gnw, gnb = vpa.layer_norm_backward(gh, x, mean, rstd, nw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    got = (r.logprobs, r.entropy, r.top_ids, gx, gw, gb, gnw, gnb)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_batches():
    x = torch.empty((0, 64), dtype=BF, device=DEV)
    w = randn(gen(1), 32, 64, dtype=BF)
    assert vpa.layer_norm(x).shape == (0, 64)
    y, pre = vpa.head_linear(x, w, activation="silu", with_pre=True)
    assert y.shape == pre.shape == (0, 32)
    gx, gw, gb = vpa.head_linear_backward(y, x, w, pre, "silu")
    assert gx.shape == (0, 64) and bool((gw == 0).all()) and bool((gb == 0).all())
    e = torch.empty(0, device=DEV)
    gx, gw, gb = vpa.layer_norm_backward(x, x, e, e)
    assert gx.shape == (0, 64) and bool((gw == 0).all()) and bool((gb == 0).all())
    tok = torch.empty(0, dtype=torch.int32, device=DEV)
    r = vpa.token_logprobs(y, 32, 32, 1, tok, 3)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3)
    rec = vpa.logprob_stats(y, 32, 16, 2, tok, 3)
    assert rec.shape == (2, 0, 10)
    assert vpa.combine_logprobs(rec, 32, 16, tok, 3).lse.shape == (0,)
    assert vpa.token_logprobs_backward(y, 32, 32, 1, tok, r.row_stats, r.logprobs).shape == (0, 32)


def test_no_tokens_and_only_the_entropy():
    v = 500
    x = randn(gen(9), 6, v)
    r = vpa.token_logprobs(x, v, v, 1)
    assert r.logprobs is None and r.top_ids is None
    lp, lse, ent, _, _ = logprob_oracle(x, v, None, 0)
    near(r.entropy, ent, 3 * SUM * (1 + ent), "entropy")
    ge = randn(gen(10), 6)
    got = vpa.token_logprobs_backward(x, v, v, 1, None, r.row_stats, None, ge)
    want, tol = grad_oracle(x, v, torch.full((6, 1), -1, device=DEV), torch.zeros(6, 1, device=DEV),
                            ge, r.row_stats)
    near(got, want, tol + U * want.abs() + torch.finfo(F32).tiny, "entropy gradient")


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31 and 2^32 bytes of the buffer."""
    v, n = 200064, 11000                                 # 2.2e9 elements, 4.4 GB
    x = torch.zeros((n, v), dtype=BF, device=DEV)
    rows = torch.tensor([0, 5368, 10735, n - 1], device=DEV)
    vals = randn(gen(2), 4, v, dtype=BF, scale=3.0)
    x[rows] = vals
    tok = torch.randint(0, v, (n,), generator=gen(3), device=DEV, dtype=torch.int32)
    r = vpa.token_logprobs(x, v, v, 1, tok, 2)
    sub = vpa.token_logprobs(vals, v, v, 1, tok[rows].contiguous(), 2)
    for a, b in ((r.logprobs, sub.logprobs), (r.lse, sub.lse), (r.entropy, sub.entropy),
                 (r.top_ids, sub.top_ids)):
        near(a[rows], b.double(), 4 * SUM * (1 + b.abs().double()), "rows far into the buffer")
    gl = torch.ones(n, device=DEV)
    vpa.token_logprobs_backward(x, v, v, 1, tok, r.row_stats, gl, out=x)
    want, tol = grad_oracle(vals, v, tok[rows], gl[rows], None, r.row_stats[rows])
    near(x[rows], want, tol + half(BF) * want.abs() + torch.finfo(F32).tiny, "gradient")


# ---------------------------------------------------------------------------
# the kernels that the sizes above do not reach, workspaces, refusals
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,k,m", [
    (9, 72, 32800), (16, 520, 33001),       # few rows of a wide weight
    (40, 4096, 300), (61, 8200, 130),       # few rows, slices of k
    (2900, 200, 2901),                      # 256-tiles with ragged edges
    (4090, 136, 4340), (4340, 136, 4090),   # whole rounds of tiles, and the rest
    (4096, 1024, 4096), (200, 6000, 260),   # many stages; slices of k of larger tiles
])
def test_head_linear_tiles(n, k, m):
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=BF), randn(g, m, k, dtype=BF, scale=k ** -0.5)
    b, r = randn(g, m, dtype=BF), randn(g, n, m, dtype=BF)
    z, dz, y, dy = linear_oracle(x, w, b, "gelu", r)
    got, pre = vpa.head_linear(x, w, b, "gelu", r, with_pre=True)
    near(got, y, dy + half(BF) * (y.abs() + dy), "y")
    near(pre, z, dz + half(BF) * (z.abs() + dz), "pre")
    near(vpa.head_linear(x, w, b, "gelu", r, out_dtype=F32), y, dy + U * y.abs(), "fp32 y")
    for _ in range(3):
        assert torch.equal(vpa.head_linear(x, w, b, "gelu", r), got)


@pytest.mark.parametrize("n,k,m,pad", [(136, 4088, 4340, 0), (2048, 1024, 4097, 0),
                                       (1030, 520, 2904, 8), (4096, 256, 264, 0),
                                       (2000, 1024, 2048, 1)])
def test_head_linear_backward_tiles(n, k, m, pad):
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=BF), randn(g, m, k, dtype=BF, scale=k ** -0.5)
    gr = randn(g, n, m, dtype=BF)
    args = (strided(gr, pad), strided(x, pad), strided(w, pad)) if pad else (gr, x, w)
    gx, gw, gb = vpa.head_linear_backward(*args)
    gd, xd, wd = gr.double(), x.double(), w.double()
    want = gd @ wd
    tol = (m + 2) * 2 * U * (gd.abs() @ wd.abs())
    near(gx, want, tol + half(BF) * (want.abs() + tol), "grad_x")
    want = gd.T @ xd
    tol = (n + 2) * 2 * U * (gd.abs().T @ xd.abs())
    near(gw, want, tol + half(BF) * (want.abs() + tol), "grad_weight")
    want = gd.sum(0)
    tol = (n + 2) * U * gd.abs().sum(0)
    near(gb, want, tol + half(BF) * (want.abs() + tol), "grad_bias")
    for _ in range(3):
        again = vpa.head_linear_backward(*args)
        assert all(torch.equal(a, c) for a, c in zip(again, (gx, gw, gb)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v,s,top", [(2, 150001, 3, 20), (66, 20011, 2, 64), (700, 3001, 1, 7)])
def test_masks_that_leave_few_tokens(n, v, s, top, dtype):
    """Row i keeps i % (top + 3) columns, the first, the last or any; the
    masked ones are -inf or the type's lowest value."""
    g = gen(n + v)
    w = -(-v // s)
    x = randn(g, n, w * s, dtype=dtype, scale=2.0)
    order = torch.rand((n, v), generator=g, device=DEV).argsort(1)
    rank = torch.empty_like(order).scatter_(
        1, order, torch.arange(v, device=DEV).expand(n, v).contiguous())
    col = torch.arange(v, device=DEV).expand(n, v)
    i = torch.arange(n, device=DEV)[:, None]
    rank = torch.where(i % 3 == 0, col, torch.where(i % 3 == 1, v - 1 - col, rank))
    low = torch.where(i % 2 == 0, NEG, torch.finfo(dtype).min).to(dtype)
    x[:, :v] = torch.where(rank < i % (top + 3), x[:, :v], low)
    tok = torch.randint(0, v, (n, 2), generator=g, device=DEV, dtype=torch.int32)
    check_logprobs(vpa.token_logprobs(x, v, w, s, tok, top), x, v, tok, top, "masked")


def test_workspaces_of_the_caller():
    g = gen(77)
    n, k, v = 100, 1000, 30011
    ins = _step_inputs(n, 1000, 30011, 4)
    x, nw, nb, w, tok, gl = ins
    garbage = lambda size: torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    from vocab_argmax_amd import head
    logits = vpa.head_linear(x, w)
    ws = vpa.logprobs_workspace(v, v, 1, n, 20)
    a, b = vpa.token_logprobs(logits, v, v, 1, tok, 20), vpa.token_logprobs(
        logits, v, v, 1, tok, 20, workspace=garbage(ws))
    assert torch.equal(a.logprobs, b.logprobs) and torch.equal(a.top_ids, b.top_ids)
    x2, w2 = randn(g, 40, 8192, dtype=BF), randn(g, 256, 8192, dtype=BF)
    ws = head._linear_workspace(vpa.VPA_BF16, 40, 256, 8192)
    assert ws > 0
    assert torch.equal(vpa.head_linear(x2, w2), vpa.head_linear(x2, w2, workspace=garbage(ws)))
    with pytest.raises(vpa.VpaError):
        vpa.head_linear(x2, w2, workspace=garbage(ws - 1))
    gr = randn(g, n, v, dtype=BF)
    ws = head._linear_grad_workspace(vpa.VPA_BF16, n, v, k)
    got = vpa.head_linear_backward(gr, x, w, workspace=garbage(ws))
    assert all(torch.equal(p, q) for p, q in zip(got, vpa.head_linear_backward(gr, x, w)))
    with pytest.raises(vpa.VpaError):
        vpa.head_linear_backward(gr, x, w, workspace=garbage(1))
    _, mean, rstd = vpa.layer_norm(x, nw, nb, with_stats=True)
    ws = head._norm_grad_workspace(n, k)
    got = vpa.layer_norm_backward(x, x, mean, rstd, nw, workspace=garbage(ws))
    assert all(torch.equal(p, q) for p, q in zip(got, vpa.layer_norm_backward(x, x, mean, rstd, nw)))
    with pytest.raises(vpa.VpaError):
        vpa.layer_norm_backward(x, x, mean, rstd, nw, workspace=garbage(ws - 1))
    with pytest.raises(ValueError):
        vpa.head_linear(x2, w2, workspace=torch.empty(1 << 24, dtype=torch.uint8))


def test_refusals():
    """Each is refused before anything is launched."""
    g = gen(8)
    x, w = randn(g, 4, 64, dtype=BF), randn(g, 32, 64, dtype=BF)
    tok = torch.zeros(4, dtype=torch.int32, device=DEV)
    wide = torch.zeros(4, 200, dtype=BF, device=DEV)
    r = vpa.token_logprobs(wide, 200, 100, 2, tok)
    e = torch.zeros(4, device=DEV)
    bad = [
        lambda: vpa.token_logprobs(wide[:, :120], 200, 100, 2, tok),     # stride 200, too narrow
        lambda: vpa.token_logprobs(wide[:, ::2], 100, 100, 1, tok),
        lambda: vpa.token_logprobs(wide[:1].expand(4, 200), 200, 100, 2, tok),
        lambda: vpa.token_logprobs(wide, 200, 100, 2, tok.long()),
        lambda: vpa.token_logprobs(wide, 200, 100, 2, tok[:3]),
        lambda: vpa.token_logprobs(wide, 200, 100, 2, tok.cpu()),
        lambda: vpa.token_logprobs(wide, 200, 100, 2, tok, 65),
        lambda: vpa.token_logprobs(wide, 200, 100, 2, tok, -1),
        lambda: vpa.token_logprobs(wide, 200, 50, 2, tok),
        lambda: vpa.token_logprobs(wide.half(), 200, 100, 2, tok),
        lambda: vpa.token_logprobs(wide, 200, 100, 2,
                                   torch.zeros(4, 65, dtype=torch.int32, device=DEV)),
        lambda: vpa.logprob_stats(wide[:, :99], 200, 100, 2, tok, first_shard=1),
        lambda: vpa.logprob_stats(wide, 200, 100, 2, tok, first_shard=2, n_local=1),
        lambda: vpa.combine_logprobs(torch.zeros(2, 4, 9, dtype=torch.int32, device=DEV), 200, 100,
                                     tok),
        lambda: vpa.token_logprobs_backward(wide, 200, 100, 2, tok, r.row_stats, None),
        lambda: vpa.token_logprobs_backward(wide[:, :120], 200, 100, 2, tok, r.row_stats, e),
        lambda: vpa.token_logprobs_backward(wide, 200, 100, 2, tok, r.row_stats[:3], e),
        lambda: vpa.token_logprobs_backward(wide, 200, 100, 2, tok, r.row_stats, e.to(BF)),
        lambda: vpa.head_linear(x, w[:, :63]),
        lambda: vpa.head_linear(x, w.float()),
        lambda: vpa.head_linear(x, w.T),
        lambda: vpa.head_linear(x, w.cpu()),
        lambda: vpa.head_linear(x, w, w[0, :31]),
        lambda: vpa.head_linear(x, w, activation="tanh"),
        lambda: vpa.head_linear(x, w, residual=x),
        lambda: vpa.head_linear(x, w, residual=w[:1, :32].expand(4, 32)),
        lambda: vpa.head_linear(x, w, out=torch.empty(4, 32, dtype=torch.float16, device=DEV)),
        lambda: vpa.head_linear(x, w, out_dtype=torch.float16),
        lambda: vpa.head_linear_backward(wide[:, :32], x, w, activation="silu"),
        lambda: vpa.head_linear_backward(wide[:, :32], x[:3], w),
        lambda: vpa.layer_norm(x, e),
        lambda: vpa.layer_norm(x, w[0], w[0].float()),
        lambda: vpa.layer_norm(x, w[0].half()),
        lambda: vpa.layer_norm(x, eps=float("nan")),
        lambda: vpa.layer_norm(x, eps=-1.0),
        lambda: vpa.layer_norm(x[0]),
        lambda: vpa.layer_norm_backward(x, x, e[:3], e),
        lambda: vpa.layer_norm_backward(x, x.float(), e, e),
    ]
    for i, call in enumerate(bad):
        try:
            call()
        except (ValueError, TypeError, vpa.VpaError):
            continue
        raise AssertionError(f"call {i} was not refused")


@pytest.mark.parametrize("n,k,m", [(1000, 1027, 2100), (2050, 2047, 1030)])
def test_rows_that_are_not_aligned(n, k, m):
    """inner is odd: operands are copied to aligned rows, or not, where the
    caller's rows are aligned already; the results are the same."""
    g = gen(n + k)
    x, w = randn(g, n, k, dtype=BF), randn(g, m, k, dtype=BF, scale=k ** -0.5)
    gr = randn(g, n, m, dtype=BF)
    pad = -k % 64
    xa, wa = strided(x, pad), strided(w, pad)
    z, dz, y, dy = linear_oracle(x, w, None, "silu", gr)
    got = vpa.head_linear(x, w, None, "silu", gr)
    near(got, y, dy + half(BF) * (y.abs() + dy), "y")
    gd, xd, wd = gr.double(), x.double(), w.double()
    grads = vpa.head_linear_backward(gr, x, w, need_bias=False)[:2]
    want = gd @ wd
    tol = (m + 2) * 2 * U * (gd.abs() @ wd.abs())
    near(grads[0], want, tol + half(BF) * (want.abs() + tol), "grad_x")
    want = gd.T @ xd
    tol = (n + 2) * 2 * U * (gd.abs().T @ xd.abs())
    near(grads[1], want, tol + half(BF) * (want.abs() + tol), "grad_weight")
    for a, b in ((xa, wa), (x, wa), (xa, w)):
        near(vpa.head_linear(a, b, None, "silu", gr), y, dy + half(BF) * (y.abs() + dy), "aligned")
        other = vpa.head_linear_backward(gr, a, b, need_bias=False)[:2]
        assert all(torch.equal(p, q) for p, q in zip(other, grads))


def test_product_offsets_past_32_bits():
    """Logits, their gradient and a weight of more than 2^32 bytes."""
    n, k, m = 11000, 64, 200064                          # 2.2e9 logits, 4.4 GB
    g = gen(21)
    x, w = randn(g, n, k, dtype=BF), randn(g, m, k, dtype=BF, scale=k ** -0.5)
    rows = torch.tensor([0, 5367, 5368, 10735, n - 1], device=DEV)
    y = vpa.head_linear(x, w)
    _, _, want, dy = linear_oracle(x[rows], w, None, "none", None)
    near(y[rows], want, dy + half(BF) * (want.abs() + dy), "rows of logits")
    cols = torch.tensor([0, 1, 99999, m - 1], device=DEV)
    _, _, want, dy = linear_oracle(x, w[cols], None, "none", None)
    near(y[:, cols], want, dy + half(BF) * (want.abs() + dy), "columns of logits")
    gx, gw, gb = vpa.head_linear_backward(y, x, w)
    gd = y[rows].double()
    want = gd @ w.double()
    tol = (m + 2) * 2 * U * (gd.abs() @ w.double().abs())
    near(gx[rows], want, tol + half(BF) * (want.abs() + tol), "grad_x")
    gd = y[:, cols].double()
    want = gd.T @ x.double()
    tol = (n + 2) * 2 * U * (gd.abs().T @ x.double().abs())
    near(gw[cols], want, tol + half(BF) * (want.abs() + tol), "grad_weight")
    want = gd.sum(0)
    tol = (n + 2) * U * gd.abs().sum(0)
    near(gb[cols], want, tol + half(BF) * (want.abs() + tol), "grad_bias")
    del y, gx, gw
    k, m = 16384, 140000                                 # a weight of 2.3e9 elements
    w = torch.empty((m, k), dtype=BF, device=DEV)
    for part in w.split(20000):
        part.copy_(randn(g, *part.shape, dtype=BF, scale=k ** -0.5))
    cols = torch.tensor([0, 65535, 131072, 131073, m - 1], device=DEV)
    for n in (3, 40, 300):
        x = randn(g, n, k, dtype=BF)
        _, _, want, dy = linear_oracle(x, w[cols], None, "none", None)
        near(vpa.head_linear(x, w)[:, cols], want, dy + half(BF) * (want.abs() + dy), f"{n} rows")


def test_norm_offsets_past_32_bits():
    n, c = 540000, 4096                                  # 2.2e9 elements, 4.4 GB
    g = gen(22)
    x = torch.zeros((n, c), dtype=BF, device=DEV)
    rows = torch.tensor([0, 524287, 524288, n - 1], device=DEV)
    vals = randn(g, 4, c, dtype=BF)
    x[rows] = vals
    w, b = randn(g, c), randn(g, c)
    y, mean, rstd = vpa.layer_norm(x, w, b, with_stats=True)
    want = vpa.layer_norm(vals, w, b, with_stats=True)
    for got, exp in ((y, want[0]), (mean, want[1]), (rstd, want[2])):
        assert torch.equal(got[rows], exp)
    gx, gw, gb = vpa.layer_norm_backward(x, x, mean, rstd, w)
    sx, sw, sb = vpa.layer_norm_backward(vals, vals, want[1], want[2], w)
    assert torch.equal(gx[rows], sx)
    # the other rows' gradients are 0, so the column sums are of the 4 rows
    near(gw, sw.double(), 8 * U * (vals.double().abs() * ((vals.double() - want[1][:, None].double())
                                   * want[2][:, None].double()).abs()).sum(0), "grad_weight")
    near(gb, sb.double(), 8 * U * vals.double().abs().sum(0), "grad_bias")
