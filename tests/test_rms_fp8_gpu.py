"""GPU tests of the root-mean-square norm, its 8-bit form, the quantiser and the
8-bit product against plain 64-bit forms, with derived tolerances (see
test_head_gpu.py)."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import ACT, BF, DEV, F32, NEG, U, gen, half, near, randn, strided

pytestmark = pytest.mark.gpu

EPS = 1e-6
F8_MAX = 448.0
BLOCK = vpa.SCALE_BLOCK
LEAST = 2.0 ** -100


def blocks_of(t, rows=1):
    """The largest |t| of each block of `rows` x 128, in t's type."""
    r, c = t.shape
    pad = torch.nn.functional.pad(t.abs(), (0, -c % BLOCK, 0, -r % rows))
    return pad.view(pad.shape[0] // rows, rows, -1, BLOCK).amax((1, 3))


def spread(scale, rows, shape):
    return scale.repeat_interleave(rows, 0)[:shape[0]].repeat_interleave(BLOCK, 1)[:, :shape[1]]


def e4m3_tolerance(v):
    """Half a step of e4m3 at v: 2^-4 relative, at least half the spacing of subnormals (2^-9)."""
    return torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

NORM_CASES = [(1, 1), (1, 2), (3, 7), (2, 63), (5, 64), (4, 257), (33, 1000), (7, 1601), (2, 512),
              (32, 4096), (3, 8192), (2, 12289), (2, 16384), (1, 70001), (700, 520), (2100, 96),
              (5000, 3)]


def depth(c):
    """Terms of a row that one of its sums adds up in a row, and the tree above them."""
    return min(c, 70) + c / 64 + 16


def norm_oracle(s, w):
    d = s.double()
    rstd = 1 / (d.square().mean(1, keepdim=True) + EPS).sqrt()
    return d, rstd, d * rstd * (1.0 if w is None else w.double())


def make(seed, n, c, dtype, wdtype, residual):
    g = gen(seed)
    x = randn(g, n, c, dtype=dtype, scale=1.5)
    r = randn(g, n, c, dtype=dtype, scale=2.0) if residual else None
    w = None if wdtype is None else (1 + randn(g, c, scale=0.2)).to(wdtype)
    s = x if r is None else (x.float() + r.float()).to(dtype)
    return g, x, r, w, s


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (BF, None)])
@pytest.mark.parametrize("n,c", NORM_CASES)
def test_rms_norm(n, c, dtype, wdtype, residual):
    g, x, r, w, s = make(n * c, n, c, dtype, wdtype, residual)
    _, rstd, want = norm_oracle(s, w)
    # the mean of squares is off by depth u relative, its root by half of that; two products
    rel = (depth(c) / 2 + 6) * U
    tol = rel * want.abs()
    tol = tol + half(dtype) * (want.abs() + tol)
    got = vpa.rms_norm(x, w, r, EPS, with_rstd=True)
    near(got.y, want, tol, "y")
    near(got.rstd, rstd[:, 0], rel * rstd[:, 0], "rstd")
    assert torch.equal(got.summed, s) and (residual or got.summed is x)
    # other strides, outputs in the inputs' places
    xs, rs = strided(x, 3, 1), None if r is None else strided(r, 5, 2)
    again = vpa.rms_norm(xs, w, rs, EPS)
    assert torch.equal(again.y, got.y) and torch.equal(again.summed, s) and again.rstd is None
    a, b = x.clone(), None if r is None else r.clone()
    if residual:
        done = vpa.rms_norm(a, w, b, EPS, out=a, summed=b)
        assert torch.equal(a, got.y) and torch.equal(b, s) and done.summed is b
        a, b = x.clone(), r.clone()
        vpa.rms_norm(a, w, b, EPS, out=b, summed=a)
        assert torch.equal(b, got.y) and torch.equal(a, s)
    else:
        vpa.rms_norm(a, w, None, EPS, out=a)
        assert torch.equal(a, got.y)
    out = strided(torch.zeros_like(x), 7, 3)
    wide = out.as_strided((n, out.stride(0)), (out.stride(0), 1))
    vpa.rms_norm(x, w, r, EPS, out=out)
    assert torch.equal(out, got.y) and (n == 1 or bool(wide[:-1, c:].isnan().all()))


@pytest.mark.parametrize("with_sum", [False, True])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, None)])
@pytest.mark.parametrize("n,c", NORM_CASES)
def test_rms_norm_backward(n, c, dtype, wdtype, with_sum):
    g, x, _, w, s = make(n * c + 1, n, c, dtype, wdtype, False)
    gr = randn(g, n, c, dtype=dtype)
    gs = randn(g, n, c, dtype=dtype) if with_sum else None
    rstd = vpa.rms_norm(x, w, None, EPS, with_rstd=True).rstd
    d, r, _ = norm_oracle(s, w)
    xh, gd = d * r, gr.double()
    u = gd if w is None else gd * w.double()
    mean = (u * xh).mean(1, keepdim=True)
    want = r * (u - xh * mean)
    if gs is not None:
        want = want + gs.double()
    rel = (depth(c) + 12) * U
    t_mean = rel * (u * xh).abs().mean(1, keepdim=True)
    tol = r * (rel * u.abs() + xh.abs() * (t_mean + rel * mean.abs())) + 2 * U * want.abs()
    gx, gw = vpa.rms_norm_backward(gr, x, rstd, w, gs)
    near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
    ww = (gd * xh).sum(0)
    wt = dtype if wdtype is None else wdtype
    tol = (depth(c) / 2 + 8 + n) * U * (gd * xh).abs().sum(0)
    near(gw, ww, tol + half(wt) * (ww.abs() + tol), "grad_weight")
    assert gw.dtype is wt
    # strides, single outputs, outputs in the inputs' places
    gx2, gw2 = vpa.rms_norm_backward(strided(gr, 3, 1), strided(x, 5, 2), rstd, w,
                                     None if gs is None else strided(gs, 1, 1))
    assert torch.equal(gx2, gx) and torch.equal(gw2, gw)
    a = gr.clone()
    only, none = vpa.rms_norm_backward(a, x, rstd, w, gs, need_weight=False, out=a)
    assert none is None and torch.equal(a, gx) and only is a
    none, only = vpa.rms_norm_backward(gr, x, rstd, w, gs, need_x=False)
    assert none is None and torch.equal(only, gw)
    if gs is not None:
        a = gs.clone()
        vpa.rms_norm_backward(gr, x, rstd, w, a, out=a)
        assert torch.equal(a, gx)


def test_rms_norm_gradient_against_differences():
    g = gen(3)
    x, r, w = randn(g, 3, 9), randn(g, 3, 9), randn(g, 9)
    gr, gs = randn(g, 3, 9), randn(g, 3, 9)
    got = vpa.rms_norm(x, w, r, EPS, with_rstd=True)
    gx, gw = vpa.rms_norm_backward(gr, got.summed, got.rstd, w, gs)
    h = 2.0 ** -7

    def loss(dx, dr, dw):
        y, s, _ = vpa.rms_norm(x + dx, w + dw, r + dr, EPS)
        return (y.double() * gr).sum() + (s.double() * gs).sum()
    size = float((gr * w).abs().sum() + gs.abs().sum()) * 30
    tol = size * (h * h + 16 * U / h)
    z = torch.zeros_like(x)
    for i, j in ((0, 0), (2, 8), (1, 4)):
        e = z.clone()
        e[i, j] = h
        near(gx[i, j], (loss(e, z, 0) - loss(-e, z, 0)) / (2 * h), tol, "by x")
        near(gx[i, j], (loss(z, e, 0) - loss(z, -e, 0)) / (2 * h), tol, "by the residual")
        f = torch.zeros(9, device=DEV)
        f[j] = h
        near(gw[j], (loss(z, z, f) - loss(z, z, -f)) / (2 * h), tol, "by the weight")


@pytest.mark.parametrize("c", [5, 700, 20000])
def test_special_rows(c):
    """Rows of 0, of large and small values, with infinities and NaN: their own rows only."""
    x = randn(gen(4), 6, c)
    x[0] = 0.0
    x[1] *= 1e15
    x[2] *= 1e-20
    x[3, c // 2] = math.inf
    x[4, 0] = math.nan
    y, _, rstd = vpa.rms_norm(x, None, None, EPS, with_rstd=True)
    assert bool((y[0] == 0).all()) and abs(float(rstd[0]) - 1e3) < 1e-3
    for i in (1, 2, 5):
        _, _, want = norm_oracle(x[i:i + 1], None)
        near(y[i:i + 1], want, (depth(c) + 10) * U * want.abs(), f"row {i}")
    assert bool(y[3, c // 2].isnan()) and bool(y[4].isnan().all())
    q, scale, _ = vpa.rms_norm_fp8(x, None, None, EPS)
    assert bool((q[0].float() == 0).all()) and float(scale[0, 0]) == float(torch.tensor(LEAST / F8_MAX))
    assert bool(scale[4].isnan().all()) and bool(scale[3, c // 2 // BLOCK].isnan())
    assert bool(torch.isfinite(scale[[0, 1, 2, 5]]).all())


# ---------------------------------------------------------------------------
# 8-bit outputs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (BF, None)])
@pytest.mark.parametrize("n,c", NORM_CASES)
def test_rms_norm_fp8(n, c, dtype, wdtype, residual):
    g, x, r, w, s = make(n * c + 2, n, c, dtype, wdtype, residual)
    _, _, want = norm_oracle(s, w)
    y, scale, summed = vpa.rms_norm_fp8(x, w, r, EPS)
    assert torch.equal(summed, s) and y.dtype is vpa.FP8 and y.shape == (n, c)
    assert y.data_ptr() % 16 == 0 and (n == 1 or y.stride(0) % 16 == 0)
    rel = (depth(c) / 2 + 6) * U
    ws = blocks_of(want).clamp(min=LEAST) / F8_MAX
    near(scale, ws, (rel + 2 * U) * ws, "scale")
    v = want / spread(ws, 1, want.shape)
    # y / scale before its rounding is off by the norm's and the scale's error
    near(y, v, e4m3_tolerance(v) * (1 + 2.0 ** -12) + (2 * rel + 8 * U) * v.abs(), "y")
    # the same values as the norm's own, where that is not rounded before
    if dtype is F32:
        f = vpa.rms_norm(x, w, r, EPS).y
        q, sc = vpa.quantize_fp8(f)
        assert torch.equal(sc, scale) and torch.equal(q.view(torch.uint8), y.view(torch.uint8))
    xs = strided(x, 3, 1)
    y2, scale2, _ = vpa.rms_norm_fp8(xs, w, None if r is None else strided(r, 5, 2), EPS)
    assert torch.equal(scale2, scale) and torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
    if residual:
        a, b = x.clone(), r.clone()
        got = vpa.rms_norm_fp8(a, w, b, EPS, summed=a)
        assert torch.equal(a, s) and torch.equal(got.y.view(torch.uint8), y.view(torch.uint8))


QUANT_CASES = [(1, 1), (3, 5), (1, 128), (2, 129), (130, 127), (128, 128), (129, 300), (257, 1000),
               (64, 4096), (1000, 96)]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,c", QUANT_CASES)
def test_quantize_fp8(n, c, dtype, rows):
    x = randn(gen(n * c), n, c, dtype=dtype, scale=3.0)
    x[0, 0] = 1e4
    if n > 2 and c > 2:
        x[2] = 0.0
    y, scale = vpa.quantize_fp8(x, rows)
    # the scale is one rounded division of the block's own value (torch divides by a number as
    # by a product with its rounded inverse; in 64 bits and rounded again it is the division's)
    want = (blocks_of(x.float(), rows).clamp(min=LEAST).double() / F8_MAX).float()
    assert torch.equal(scale, want)
    v = x.double() / spread(want.double(), rows, x.shape)
    near(y, v, e4m3_tolerance(v) * (1 + 4 * U) + 4 * U * v.abs(), "y")
    assert float(y.float().abs().max()) <= F8_MAX
    y2, scale2 = vpa.quantize_fp8(strided(x, 3, 1), rows)
    assert torch.equal(scale2, scale) and torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
    assert y.data_ptr() % 16 == 0 and (n == 1 or y.stride(0) % 16 == 0)


def test_quantize_special_blocks():
    x = randn(gen(5), 4, 400)
    x[0, 130] = math.nan
    x[1, 7] = NEG
    x[2, :128] = 1e-38
    x[3, 256:384] = 3e38
    y, scale = vpa.quantize_fp8(x)
    bad = scale.isnan()
    assert bad.tolist() == [[False, True, False, False], [True, False, False, False],
                            [False] * 4, [False] * 4]
    back = y.float() * spread(scale, 1, x.shape)
    assert bool(back[0, 128:256].isnan().all()) and bool(back[1, :128].isnan().all())
    near(back[3, 256:384], x[3, 256:384].double(), x[3, 256:384].double().abs() * 2.0 ** -4, "large")
    # below 2^-100 the scale stays
    assert float(scale[2, 0]) == float(torch.tensor(LEAST / F8_MAX))
    near(back[2, :128], x[2, :128].double(),
         e4m3_tolerance(x[2, :128].double() / float(scale[2, 0])) * float(scale[2, 0]), "small")


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------

def operands(seed, n, k, m, wild=False):
    """8-bit operands with scales that differ from block to block by up to 2^8, in padded rows
    whose padding holds NaN."""
    g = gen(seed)

    def one(r, c, rows):
        ld = (c + 15) // 16 * 16
        buf = torch.full((r, ld + 16), 0x7F, dtype=torch.uint8, device=DEV).view(vpa.FP8)
        t = buf[:, :c]
        t.copy_((randn(g, r, c) * (100 if wild else 1)).clamp(-F8_MAX, F8_MAX).to(vpa.FP8))
        sr, sc = -(-r // rows), -(-c // BLOCK)
        s = torch.exp2(randn(g, sr, sc) * (2 if wild else 0.5)) * 0.01
        return t, s
    x, xs = one(n, k, 1)
    w, ws = one(m, k, BLOCK)
    return g, x, xs, w, ws


def product(x, xs, w, ws):
    """(x W^T, the bound of its error, sum |x| |W|) in 64 bits: a block's 128 products are exact
    and added in fp32 (2 u a step: the matrix cores may drop what is below the last bit), its sum
    is multiplied by a rounded product of scales and added, another 3 u of the running sum a block."""
    a = x.double() * spread(xs.double(), 1, x.shape)
    b = w.double() * spread(ws.double(), BLOCK, w.shape)
    z = a @ b.T
    blocks = -(-x.shape[1] // BLOCK)
    mag = a.abs() @ b.abs().T
    return z, (min(x.shape[1], 128) * 2 + 3 * blocks + 8) * U * mag, mag


# bf16 results of more rows come from the matrix cores' 8-bit instruction: of a group of 8 products
# it cuts what lies below 2^-13 of the largest, so that 7 of them lose up to 2^-13 of it each
FEW_ROWS = 64
CUT = 7 * 2.0 ** -13


FP8_CASES = [  # rows, inner, outer
    (1, 1, 1), (1, 16, 16), (2, 17, 33), (1, 128, 128), (3, 129, 127), (5, 1000, 300),
    (16, 4096, 1000), (17, 256, 129), (32, 2048, 1111), (33, 640, 500), (63, 1601, 515),
    (64, 384, 4097), (65, 130, 260), (100, 785, 1000), (128, 1024, 384), (200, 4096, 777),
    (257, 512, 513), (300, 2047, 1025), (1000, 96, 640), (1, 8192, 4096), (8, 1024, 40000),
    (31, 2048, 33000), (520, 1280, 2050),
]


@pytest.mark.parametrize("n,k,m", FP8_CASES)
def test_head_linear_fp8(n, k, m):
    g, x, xs, w, ws = operands(n * k + m, n, k, m, wild=(n + k) % 2 == 1)
    z, dz, mag = product(x, xs, w, ws)
    near(vpa.head_linear_fp8(x, xs, w, ws, out_dtype=F32), z, dz + U * z.abs(), "fp32")
    plain = vpa.head_linear_fp8(x, xs, w, ws)
    d16 = dz + (CUT * mag if n > FEW_ROWS else 0)
    near(plain, z, d16 + half(BF) * (z.abs() + d16), "bf16")
    # random operands: 1.4e-5 in the 2-norm for the instruction's cut, 2^-9 for the result's
    # rounding, of which its 2-norm over evenly spread values is 1 / sqrt(3) and less
    assert float((plain.double() - z).norm() / z.norm()) < half(BF) * 0.7 + 1e-4 or n * m < 100
    b, r = randn(g, m, dtype=BF, scale=0.5), randn(g, n, m, dtype=BF)
    for act in ACT:
        t = z + b.double()
        want = ACT[act](t) + r.double()
        # slopes are at most 1.13; the functions are good to 4 u of their value and 1
        more = 8 * U * (1 + t.abs()) + 2 * U * want.abs()
        tol = 1.13 * (dz + U * t.abs()) + more
        near(vpa.head_linear_fp8(x, xs, w, ws, b, act, r, out_dtype=F32), want, tol, act)
        tol = 1.13 * (d16 + U * t.abs()) + more
        y = vpa.head_linear_fp8(x, xs, w, ws, b, act, r)
        near(y, want, tol + half(BF) * (want.abs() + tol), act + " bf16")
    a = r.clone()
    assert vpa.head_linear_fp8(x, xs, w, ws, b, "silu", a, out=a) is a
    assert torch.equal(a, vpa.head_linear_fp8(x, xs, w, ws, b, "silu", r))
    # results in a shard's columns of a wider tensor, scales of other strides
    wide = torch.full((n, m + 9), math.nan, dtype=BF, device=DEV)
    vpa.head_linear_fp8(x, strided(xs, 2, 1), w, strided(ws, 3), out=wide[:, 5:5 + m])
    assert torch.equal(wide[:, 5:5 + m], plain)
    assert bool(wide[:, :5].isnan().all()) and bool(wide[:, 5 + m:].isnan().all())


def test_head_linear_fp8_carries_infinities_and_nan():
    """Of scales and operands: their own rows, columns and blocks only."""
    for n, k, m in ((3, 300, 200), (40, 300, 300), (200, 300, 400)):
        _, x, xs, w, ws = operands(n, n, k, m)
        x[1, 5] = math.nan
        y = vpa.head_linear_fp8(x, xs, w, ws)
        assert bool(y[1].isnan().all()) and not bool(y[[0, 2]].isnan().any())
        x[1, 5] = 1.0
        xs[2, 1] = math.nan
        y = vpa.head_linear_fp8(x, xs, w, ws)
        assert bool(y[2].isnan().all()) and not bool(y[:2].isnan().any())
        xs[2, 1] = 1.0
        ws[1, 2] = math.nan
        y = vpa.head_linear_fp8(x, xs, w, ws)
        assert bool(y[:, 128:256].isnan().all()) and not bool(y[:, :128].isnan().any())
        assert not bool(y[:, 256:].isnan().any())


def test_8_bit_head_end_to_end():
    """Norm, product, norm, vocabulary product, tokens: each step is near the one in full width."""
    g = gen(9)
    n, h, v = 40, 512, 3000
    x, res = randn(g, n, h, dtype=BF), randn(g, n, h, dtype=BF)
    w1 = (1 + randn(g, h, scale=0.1)).to(BF)
    block, vocab = randn(g, h, h, dtype=BF, scale=h ** -0.5), randn(g, v, h, dtype=BF, scale=0.2)
    b8, bs = vpa.quantize_fp8(block, BLOCK)
    v8, vs = vpa.quantize_fp8(vocab, BLOCK)
    y8, ys, s = vpa.rms_norm_fp8(x, w1, res)
    t = vpa.head_linear_fp8(y8, ys, b8, bs, None, "silu", s)
    z8, zs, s2 = vpa.rms_norm_fp8(t, w1, s)
    logits = vpa.head_linear_fp8(z8, zs, v8, vs)
    want_s = (x.float() + res.float()).to(BF)
    assert torch.equal(s, want_s)
    a = y8.double() * spread(ys.double(), 1, y8.shape)
    b = b8.double() * spread(bs.double(), BLOCK, b8.shape)
    near(a, norm_oracle(s, w1)[2], norm_oracle(s, w1)[2].abs() * (2.0 ** -4 + 2.0 ** -10) +
         spread(ys.double(), 1, y8.shape) * 2.0 ** -10, "norm in 8 bits")
    zt = a @ b.T
    near(t, ACT["silu"](zt) + s.double(), 2 * half(BF) * (zt.abs() + s.double().abs() + 1), "block")
    ids, _ = vpa.top_tokens(logits, v, v, 1)
    assert torch.equal(ids.long(), logits.float().argmax(1)) or bool(
        (logits.float().gather(1, ids.long()[:, None])[:, 0] == logits.float().amax(1)).all())
    k = 3
    reqs = n // (k + 1)
    drafts = ids.view(reqs, k + 1)[:, :k].contiguous()
    out, sampled, rejected = vpa.sampled_verify(
        logits, v, v, 1, drafts, torch.rand((reqs, k), generator=g, device=DEV),
        torch.rand(reqs, generator=g, device=DEV, dtype=torch.float64),
        temperature=torch.zeros(reqs, device=DEV))
    assert torch.equal(out.view(-1), ids) and bool((sampled == k + 1).all())
    r = vpa.token_logprobs(logits, v, v, 1, n_top=8)
    loss, grad = vpa.distill_loss_and_grad(logits, v, v, 1, r.top_ids, r.top_logprobs,
                                           torch.ones(n, device=DEV), tail=True)
    # the teacher is the student: nothing to learn, to the digits of its log probabilities
    near(loss, torch.zeros(n, dtype=torch.float64, device=DEV), 400 * U, "loss")
    near(grad, torch.zeros_like(grad, dtype=torch.float64), 400 * U, "gradient")


@pytest.mark.parametrize("n,k,m", [(1, 512, 600), (30, 4096, 1000), (300, 1024, 700)])
def test_repeats_streams_graphs_and_workspaces(n, k, m):
    g, x, xs, w, ws = operands(7, n, k, m)
    h, r = randn(g, n, k, dtype=BF), randn(g, n, k, dtype=BF)
    wt = randn(g, k, dtype=BF)

    def step(h, **kw):
        y8, ys, s = vpa.rms_norm_fp8(h, wt, r)
        y, _, rstd = vpa.rms_norm(h, wt, r, with_rstd=True)
        gx, gw = vpa.rms_norm_backward(y, s, rstd, wt, y)
        return (y8.view(torch.uint8) if y8.is_contiguous() else y8.float(), ys, s, y, rstd, gx, gw,
                vpa.head_linear_fp8(y8, ys, w, ws, **kw))
    want = step(h)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(step(h), want))
    need = vpa.draft_lib().vpa_head_linear_fp8_workspace(n, m, k)
    buf = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(step(h, workspace=buf[:need]), want))
    assert bool((buf[need:] == 0x5A).all())
    if need:
        with pytest.raises(vpa.VpaError, match="workspace"):
            step(h, workspace=buf[:need - 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = vpa.head_linear_fp8(x, xs, w, ws, stream=side)
    q = vpa.rms_norm_fp8(h, wt, r, stream=side)
    side.synchronize()
    assert torch.equal(y, vpa.head_linear_fp8(x, xs, w, ws)) and torch.equal(q.scale, want[1])
    h2 = h.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(h2)
    for turn in range(3):
        h2.copy_(h if turn != 1 else h.flip(0) * 2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(h2))), turn


def test_empty_batches():
    x = torch.zeros((0, 256), dtype=BF, device=DEV)
    y, s, rstd = vpa.rms_norm(x, None, x, with_rstd=True)
    assert y.shape == s.shape == (0, 256) and rstd.shape == (0,)
    y8, scale, _ = vpa.rms_norm_fp8(x)
    assert y8.shape == (0, 256) and scale.shape == (0, 2)
    gx, gw = vpa.rms_norm_backward(x, x, rstd)
    assert gx.shape == (0, 256) and bool((gw == 0).all()) and gw.shape == (256,)
    q, qs = vpa.quantize_fp8(x, 128)
    assert q.shape == (0, 256) and qs.shape == (0, 2)
    w, ws = vpa.quantize_fp8(torch.ones((130, 256), device=DEV), 128)
    assert vpa.head_linear_fp8(y8, scale, w, ws).shape == (0, 130)


def test_refusals():
    g, x, xs, w, ws = operands(8, 4, 300, 200)
    f = vpa.head_linear_fp8
    f(x, xs, w, ws)
    res = torch.zeros((4, 200), dtype=BF, device=DEV)
    for args, kw, err in (
            ((x, xs[:, :2], w, ws), {}, ValueError), ((x, xs, w, ws[:1]), {}, ValueError),
            ((x[:, :299], xs, w, ws), {}, ValueError), ((x.float(), xs, w, ws), {}, TypeError),
            ((x, xs, w.float(), ws), {}, TypeError), ((x, xs.double(), w, ws), {}, TypeError),
            ((x.cpu(), xs, w, ws), {}, ValueError), ((x, xs, w.cpu(), ws), {}, ValueError),
            ((x[:, 1:], xs, w[:, 1:], ws), {}, ValueError),            # rows not at 16 bytes
            ((x.contiguous(), xs, w, ws), {}, ValueError),             # 300 is no multiple of 16
            ((x, xs, w, ws), dict(bias=torch.zeros(199, dtype=BF, device=DEV)), ValueError),
            ((x, xs, w, ws), dict(bias=torch.zeros(200, device=DEV)), ValueError),
            ((x, xs, w, ws), dict(residual=res.float()), TypeError),
            ((x, xs, w, ws), dict(activation="tanh"), ValueError),
            ((x, xs, w, ws), dict(out_dtype=torch.float16), TypeError),
            ((x, xs, w, ws), dict(out=res, out_dtype=F32), TypeError),
            ((x, xs, w, ws), dict(out=res[:3]), ValueError)):
        with pytest.raises(err):
            f(*args, **kw)
    h = torch.zeros((4, 300), dtype=BF, device=DEV)
    with pytest.raises(vpa.VpaError):
        vpa.rms_norm(h, eps=-1.0)
    with pytest.raises(vpa.VpaError):
        vpa.rms_norm(h, eps=math.nan)
    with pytest.raises(ValueError):
        vpa.rms_norm(h, summed=h)
    with pytest.raises(vpa.VpaError):
        vpa.rms_norm(h, None, h.clone(), out=h, summed=h)
    with pytest.raises(ValueError):
        vpa.rms_norm(h, residual=h[:, :299])
    with pytest.raises(TypeError):
        vpa.rms_norm(h, residual=h.float())
    with pytest.raises((ValueError, TypeError)):
        vpa.rms_norm(h, torch.zeros(300, dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError):
        vpa.rms_norm(h.half())
    with pytest.raises(ValueError):
        vpa.rms_norm(h.t())
    rstd = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError):
        vpa.rms_norm_backward(h, h, rstd[:3])
    with pytest.raises(vpa.VpaError):
        a = h.clone()
        vpa.rms_norm_backward(a, h, rstd, out=a)                       # grad is read for the weight
    with pytest.raises(vpa.VpaError):
        vpa.rms_norm_backward(h.clone(), h, rstd, out=h)
    with pytest.raises(ValueError):
        vpa.rms_norm_backward(h, h, rstd, need_x=False, out=h.clone())
    with pytest.raises(ValueError):
        vpa.quantize_fp8(h, 64)
    with pytest.raises(TypeError):
        vpa.quantize_fp8(h.half())


def test_offsets_past_32_bits():
    n, c = 1100000, 4096                                 # 4.5e9 elements of 8 bits
    x = torch.zeros((n, c), dtype=BF, device=DEV)
    rows = torch.tensor([0, 524287, 1048576, n - 1], device=DEV)
    vals = randn(gen(10), 4, c, dtype=BF)
    x[rows] = vals
    want = vpa.rms_norm_fp8(vals)
    y, scale, _ = vpa.rms_norm_fp8(x)
    assert torch.equal(scale[rows], want.scale)
    assert torch.equal(y.view(torch.uint8)[rows], want.y.view(torch.uint8))
    w, ws = vpa.quantize_fp8(randn(gen(11), 130, c), BLOCK)
    del x
    out = vpa.head_linear_fp8(y, scale, w, ws)
    assert torch.equal(out[rows], vpa.head_linear_fp8(y[rows], want.scale, w, ws)) or bool(
        ((out[rows].float() - vpa.head_linear_fp8(y[rows], want.scale, w, ws).float()).abs()
         <= 2.0 ** -6 * out[rows].float().abs() + 1e-3).all())
    del y, out
    m, k = 560000, 8192                                  # a weight of 4.6e9 elements
    w8 = torch.zeros((m, k), dtype=torch.uint8, device=DEV).view(vpa.FP8)
    ws = torch.ones((m // BLOCK, k // BLOCK), device=DEV)
    at = torch.tensor([0, 262143, 262144, 524288, m - 1], device=DEV)
    some = randn(gen(12), 5, k).to(vpa.FP8)
    w8.view(torch.uint8)[at] = some.view(torch.uint8)
    for n in (1, 20, 70):
        xx = randn(gen(13), n, k).to(vpa.FP8)
        got = vpa.head_linear_fp8(xx, torch.ones((n, k // BLOCK), device=DEV), w8, ws)
        z = xx.double() @ some.double().T
        dz = xx.double().abs() @ some.double().abs().T
        dz *= (256 + 3 * 64 + 8) * U + (CUT if n > FEW_ROWS else 0)
        near(got[:, at], z, dz + half(BF) * (z.abs() + dz), f"{n} rows")
