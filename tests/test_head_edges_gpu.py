"""GPU tests of the head's operators where a size, a mask or a range of values
ends: thin operands, state carried from chunk to chunk of a long row, very
confident rows, many short rows.  Tolerances as in test_head_gpu.py: half(t) is
half a step of type t, U is fp32's, a sum of n terms is off by n U sum |terms|,
2 U a term on the matrix cores."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import (BF, DEV, F32, NEG, SUM, U, check_logprobs, gen, grad_oracle, half,
                           linear_oracle, logprob_oracle, near, randn, slope)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("n,m,k", [  # rows, outer, inner
    (40, 50257, 1), (64, 32000, 1), (17, 2000, 2), (1, 513, 1), (40, 1, 5025), (300, 1, 1),
    (33, 3, 3), (64, 2, 4097), (129, 513, 1)])
def test_products_of_thin_operands(n, m, k, act, dtype):
    """Forward and backward within a workspace that ends where it has to."""
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=dtype), randn(g, m, k, dtype=dtype, scale=k ** -0.5)
    b, gr = randn(g, m, dtype=dtype), randn(g, n, m, dtype=dtype)
    z, dz, y, dy = linear_oracle(x, w, b, act, gr)
    got, pre = vpa.head_linear(x, w, b, act, gr, with_pre=True)
    near(got, y, dy + half(dtype) * (y.abs() + dy), "y")
    d = gr.double() * slope(act, pre.double())
    off = 0 * d if act == "none" else gr.double().abs() * 16 * U * (1 + pre.double().abs())
    rounded = off if act == "none" else off + half(dtype) * (d.abs() + off)
    code = vpa.VPA_BF16 if dtype is BF else vpa.VPA_F32
    need = vpa.head_lib().vpa_head_linear_backward_workspace(code, n, m, k)
    buf = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    gx, gw, gb = vpa.head_linear_backward(gr, x, w, pre, act, workspace=buf[:need])
    assert bool((buf[need:] == 0xA5).all()), "written past the workspace"
    want = d @ w.double()
    tol = rounded @ w.double().abs() + (m + 2) * 2 * U * (d.abs() @ w.double().abs())
    near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
    want = d.T @ x.double()
    tol = rounded.T @ x.double().abs() + (n + 2) * 2 * U * (d.T.abs() @ x.double().abs())
    near(gw, want, tol + half(dtype) * (want.abs() + tol), "grad_weight")
    want = d.sum(0)
    tol = off.sum(0) + (n + 2) * U * d.abs().sum(0)
    near(gb, want, tol + half(dtype) * (want.abs() + tol), "grad_bias")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_norm_of_many_short_rows(dtype):
    """More rows than a dispatch has workgroups of 1024 threads: every row and
    the sums over all of them, the last rows among them."""
    n, c = (1 << 22) + 5, 9
    g = gen(n)
    x, gr = randn(g, n, c, dtype=dtype), randn(g, n, c, dtype=dtype)
    w, b = randn(g, c, dtype=dtype), randn(g, c, dtype=dtype)
    xd, gd, wd = x.double(), gr.double(), w.double()
    mu = xd.mean(1, keepdim=True)
    var = (xd - mu).square().mean(1, keepdim=True)
    rs = 1 / (var + 1e-5).sqrt()
    k = 33 * U                                           # one term a thread, then the tree
    dmu = k * xd.abs().mean(1, keepdim=True)
    drs = k + 0.5 * (dmu * dmu + 2 * U * dmu * rs.reciprocal()) / (var + 1e-5)
    want = (xd - mu) * rs * wd + b.double()
    part = ((xd - mu) * rs * wd).abs()
    tol = rs * dmu * wd.abs() + part * (drs + 4 * U) + U * want.abs()
    y, mean, rstd = vpa.layer_norm(x, w, b, with_stats=True)
    near(y, want, tol + half(dtype) * (want.abs() + tol), "y")
    rs = rstd.double()[:, None]
    xh = (xd - mean.double()[:, None]) * rs
    u = gd * wd
    m1, m2 = u.mean(1, keepdim=True), (u * xh).mean(1, keepdim=True)
    a1, a2 = u.abs().mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
    want = rs * (u - m1 - xh * m2)
    tol = rs * (8 * U * (u.abs() + a1 + xh.abs() * a2) + k * (a1 + xh.abs() * a2))
    gx, gw, gb = vpa.layer_norm_backward(gr, x, mean, rstd, w)
    near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
    # a thread's share of the rows one after the other, then a few sums of sums
    terms = n // 2048 + 64
    for got, t, what in ((gw, gd * xh, "grad_weight"), (gb, gd, "grad_bias")):
        tol = (terms + 6) * U * t.abs().sum(0)
        near(got, t.sum(0), tol + half(dtype) * (t.sum(0).abs() + tol), what)


# ---------------------------------------------------------------------------
# log probabilities: what a row carries from chunk to chunk
# ---------------------------------------------------------------------------

# rows, vocab, 16-byte vectors of a thread and chunk (bf16, fp32): a workgroup of
# 256 threads reads a row in several chunks
CHUNKED = [(1500, 20000, 8, 8), (1500, 40000, 8, 8), (3, 1200000, 2, 2), (60, 151936, 2, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v", [c[:2] for c in CHUNKED])
def test_finite_rows_far_apart(n, v, dtype):
    """Sums of many columns beside one that is further away than fp32 can
    multiply them by: the row is that one token."""
    x = torch.zeros((n, v), dtype=dtype, device=DEV)
    x[:, v // 3:] = 39.0
    x[:, v - 1] = 3.0e38
    if n > 1:
        x[1, v - 1] = 39.0
        x[1, 0] = 1.0e30
        x[1, v // 2] = -3.0e38
    tok = torch.full((n,), v - 1, dtype=torch.int32, device=DEV)
    ge = torch.ones(n, device=DEV)
    r = vpa.token_logprobs(x, v, v, 1, tok, 2)
    check_logprobs(r, x, v, tok, 2, "far apart")
    assert bool((r.entropy == 0).all())
    w = -(-v // 3)
    wide = torch.full((n, 3 * w), float("nan"), dtype=dtype, device=DEV)
    wide[:, :v] = x
    rec = vpa.logprob_stats(wide, v, w, 3, tok, 2)
    check_logprobs(vpa.combine_logprobs(rec, v, w, tok, 2), x, v, tok, 2, "far apart, sharded")
    got = vpa.token_logprobs_backward(x, v, v, 1, tok, r.row_stats, ge, ge)
    want, tol = grad_oracle(x[:3], v, tok[:3], ge[:3], ge[:3], r.row_stats[:3])
    near(got[:3], want, tol + half(dtype) * want.abs() + torch.finfo(F32).tiny, "gradient")


def late_rows(x, dtype, chunk):
    """Rows that go wrong, if they do, in a later chunk than the first."""
    n, v = x.shape
    last = (v - 1) // chunk * chunk                      # the first column of the last chunk
    x[0, :chunk] = NEG                                   # a first chunk of masked columns
    x[1, :last] = NEG
    x[2, :chunk] = torch.finfo(dtype).min
    x[3, last:] = NEG                                    # a last chunk of masked ones
    x[4, v - 2] = float("nan")
    x[5, v - 1] = float("inf")
    x[6, v - 3] = float("nan")
    x[6, 5] = float("inf")
    x[7, :chunk] -= 100.0                                # the rest is far above
    x[8] = torch.linspace(-60, 60, v, device=DEV).to(dtype)      # ascending, with ties in bf16
    x[9, chunk:] = 6.5                                   # thousands of ties, after the first chunk
    x[10, :chunk] = 6.5                                  # and before
    x[11] = torch.where(torch.arange(v, device=DEV) % 2 == 0, -0.0, 0.0).to(dtype)
    x[12] = NEG                                          # 3 tokens, all late
    x[12, last:last + 3] = torch.tensor([1.0, 3.0, 3.0], device=DEV).to(dtype)
    x[13, chunk:] += 41.0                                # rises past any lag of the maximum
    x[14, chunk:] += 0.9
    x[15, last] = 3.0e38
    x[16, last] = -3.0e38
    x[17] = x[17] * 1e30
    x[18, 1::2] = NEG
    x[19, last:] = float("nan")
    return x


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v,vecs_bf16,vecs_f32", CHUNKED)
@pytest.mark.parametrize("top", [0, 3, 64])
def test_rows_of_several_chunks(n, v, vecs_bf16, vecs_f32, top, dtype):
    g = gen(v + top)
    chunk = 256 * (8 * vecs_bf16 if dtype is BF else 4 * vecs_f32)
    kinds = late_rows(randn(g, 20, v, dtype=dtype, scale=2.0), dtype, chunk)
    # of a call of 3 rows the kinds come 3 at a time
    batches = [kinds[i:i + n] for i in range(0, 20, n)] if n < 20 else [kinds]
    for some in batches:
        x = torch.cat([some, randn(g, max(0, n - len(some)), v, dtype=dtype, scale=2.0)])
        tok = torch.randint(0, v, (x.shape[0], 3), generator=g, device=DEV, dtype=torch.int32)
        tok[:, 1], tok[:, 2] = v - 1, -1
        r = vpa.token_logprobs(x, v, v, 1, tok, top)
        few = len(some)
        check_logprobs(cut_rows(r, few), some, v, tok[:few], top, "chunks")
        if n > 20:
            near(r.lse[few:40], x[few:40].double().logsumexp(1), SUM * 16, "the others")
        w = -(-v // 2)
        wide = torch.full((x.shape[0], 2 * w), float("nan"), dtype=dtype, device=DEV)
        wide[:, :v] = x
        rec = vpa.logprob_stats(wide, v, w, 2, tok, top)
        check_logprobs(cut_rows(vpa.combine_logprobs(rec, v, w, tok, top), few), some, v, tok[:few],
                       top, "chunks, sharded")


class cut_rows:
    """The first n rows of a TokenLogprobs."""

    def __init__(self, r, n):
        for name in ("logprobs", "lse", "entropy", "top_ids", "top_logprobs"):
            t = getattr(r, name)
            setattr(self, name, t if t is None else t[:n])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v", [(1500, 50257), (1500, 20000), (1, 50257), (33, 151936), (3, 1200000)])
def test_confident_rows_keep_their_digits(n, v, dtype):
    """A trained model is sure of most tokens: the log probability of the sure
    one and the entropy are far below 1, and their error is too, wherever in
    the row the token stands."""
    g = gen(v + n)
    x = -4.0 * torch.rand((n, v), generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    at = (v - 1 - (i * 7919) % v) if n > 1 else torch.tensor([v - 5], device=DEV)
    gap = 24.0 + (i % 16) if n > 1 else torch.tensor([36.0], device=DEV)
    x[i, at] = gap.float()
    x = x.to(dtype)
    tok = at.to(torch.int32)
    lp, lse, ent, _, _ = logprob_oracle(x[:64], v, tok[:64], 0)
    gap = gap[:64].double()
    # What may be lost: terms of at most e^-gap each that a lane adds to the 1
    # of the sure token, v / 256 and a few of them, and some steps at 1 in 2^z,
    # the sum's logarithm and the distance from M.  Of u = sum z 2^z nothing
    # is lost but a relative (64 + 32) U, M's own term being 0.
    lost = (v / 256 + 64) * (-gap).exp() + 8 * U
    r = vpa.token_logprobs(x, v, v, 1, tok)
    near(r.logprobs[:64], lp, lost, "log probability of the sure token")
    near(r.entropy[:64], ent, lost + SUM * ent, "entropy")
    rec = vpa.logprob_stats(x, v, v, 1, tok)
    r = vpa.combine_logprobs(rec, v, v, tok)
    near(r.logprobs[:64], lp, lost, "log probability of the sure token, of records")
    near(r.entropy[:64], ent, lost + SUM * ent, "entropy, of records")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,v", [(1500, 50257), (33, 151936)])
def test_confident_rows_with_a_rival(n, v, dtype):
    """Two tokens carry a row, the later one ahead by any distance: what the sum
    loses to the distance between them has a bound that does not grow with it."""
    i = torch.arange(n, device=DEV)
    x = torch.full((n, v), -60.0, device=DEV)
    x[:, 7] = 0.0
    at = v - 1 - (i * 7919) % (v // 3)
    x[i, at] = 0.25 * (i % 160).float()
    x = x.to(dtype)
    tok = torch.stack([at, torch.full_like(at, 7)], 1).to(torch.int32)
    lp, lse, ent, _, _ = logprob_oracle(x, v, tok, 0)
    r = vpa.token_logprobs(x, v, v, 1, tok)
    # M is at most 4 behind: x - M is off by half a step there, 4 U, and a step
    # at 4 log2(e) < 8 is 8 U: log2 s has one of them, z half of one, which 2^z
    # and the logarithm carry on; 2^z, its scale and the sum of the two add 6 U.
    # The rest's v terms of e^-60 are nothing.
    tol = 24 * U + 2 * U * lp.abs()
    near(r.logprobs, lp, tol, "log probabilities")
    # u's terms are z 2^z, each 2^z off by the 10 U of before, z below 6
    near(r.entropy, ent, 24 * U + 2 * 6 * 10 * U * ent.clamp(max=1), "entropy")


# ---------------------------------------------------------------------------
# the gradient of fp32 results of bf16 operands
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["none", "silu", "relu"])
@pytest.mark.parametrize("n,k,m", [(1, 1, 1), (1, 129, 70), (3, 65, 129), (64, 256, 320),
                                   (100, 130, 1031), (513, 96, 2049), (1030, 520, 2904)])
def test_backward_for_an_fp32_gradient(n, k, m, act):
    g = gen(n + 31 * k + 7 * m)
    x, w = randn(g, n, k, dtype=BF), randn(g, m, k, dtype=BF, scale=k ** -0.5)
    b, gr = randn(g, m, dtype=BF), randn(g, n, m)
    y, pre = vpa.head_linear(x, w, b, act, out_dtype=F32, with_pre=True)
    assert y.dtype is F32 and pre.dtype is BF
    z = pre.double()
    dz = gr.double() * slope(act, z)
    off = 0 * dz if act == "none" else gr.double().abs() * 16 * U * (1 + z.abs())
    rounded = off + half(BF) * (dz.abs() + off)          # the products' operand is bf16
    wide = torch.full((n, m + 3), float("nan"), device=DEV)
    wide[:, 1:m + 1] = gr                                # rows that are not aligned
    for gg in (gr, wide[:, 1:m + 1]):
        gx, gw, gb = vpa.head_linear_backward(gg, x, w, pre, act)
        assert gx.dtype is gw.dtype is gb.dtype is BF
        want = dz @ w.double()
        tol = rounded @ w.double().abs() + (m + 2) * 2 * U * (dz.abs() @ w.double().abs())
        near(gx, want, tol + half(BF) * (want.abs() + tol), "grad_x")
        want = dz.T @ x.double()
        tol = rounded.T @ x.double().abs() + (n + 2) * 2 * U * (dz.T.abs() @ x.double().abs())
        near(gw, want, tol + half(BF) * (want.abs() + tol), "grad_weight")
        want = dz.sum(0)                                 # of the fp32 values, not of rounded ones
        tol = off.sum(0) + (n + 2) * U * dz.abs().sum(0)
        near(gb, want, tol + half(BF) * (want.abs() + tol), "grad_bias")
    only = vpa.head_linear_backward(gr, x, w, pre, act, need_weight=False, need_x=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], gb)


def test_fp32_logits_of_bf16_operands_train():
    """LM head with fp32 logits, their log probabilities and the way back."""
    n, k, v = 40, 96, 3001
    g = gen(12)
    x, w = randn(g, n, k, dtype=BF), randn(g, v, k, dtype=BF, scale=k ** -0.5)
    tok = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    logits = vpa.head_linear(x, w, out_dtype=F32)
    r = vpa.token_logprobs(logits, v, v, 1, tok)
    gl = torch.full((n,), -1.0 / n, device=DEV)
    d = vpa.token_logprobs_backward(logits, v, v, 1, tok, r.row_stats, gl)
    gx, gw, _ = vpa.head_linear_backward(d, x, w, need_bias=False)
    dd = d.double()
    want = dd @ w.double()
    tol = (half(BF) + (v + 2) * 2 * U) * (dd.abs() @ w.double().abs())
    near(gx, want, tol + half(BF) * (want.abs() + tol), "grad_x")
    want = dd.T @ x.double()
    tol = (half(BF) + (n + 2) * 2 * U) * (dd.T.abs() @ x.double().abs())
    near(gw, want, tol + half(BF) * (want.abs() + tol), "grad_weight")
    empty = vpa.head_linear_backward(d[:0], x[:0], w)
    assert empty[0].shape == (0, k) and bool((empty[1] == 0).all()) and bool((empty[2] == 0).all())
    with pytest.raises(TypeError):
        vpa.head_linear_backward(d.to(BF), x.float(), w.float())
    with pytest.raises(TypeError):
        vpa.head_linear_backward(d.half(), x, w)


def test_backward_takes_no_memory_for_what_it_does_not_do():
    """An aligned gradient without an activation is read in place: no dz."""
    n, k, v = 1024, 64, 65536
    g = gen(31)
    x, w = randn(g, n, k, dtype=BF), randn(g, v, k, dtype=BF, scale=k ** -0.5)
    gr = randn(g, n, v, dtype=BF)

    def peak(call):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        return torch.cuda.max_memory_allocated() - before
    vpa.head_linear_backward(gr, x, w)
    results = 2 * (n * k + v * k + v) + (1 << 20)        # and the allocator's rounding
    dz = 2 * n * v
    lean = peak(lambda: vpa.head_linear_backward(gr, x, w, need_x=False, need_bias=False))
    code = vpa.VPA_BF16
    slices = vpa.head_lib().vpa_head_linear_backward_need(code, n, v, k, 0, 0, 1, 0)
    assert lean <= results + slices and slices < dz / 2
    assert peak(lambda: vpa.head_linear_backward(gr, x, w, gr, "silu")) >= dz


# ---------------------------------------------------------------------------
# layer norm at the ends of the range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [1, 5, 9, 63, 100])
def test_layer_norm_backward_of_constant_rows_far_from_0(c, dtype):
    """mean * rstd is past fp32's range, (x - mean) * rstd is 0: the lanes past
    the row's end have no part in its sums."""
    g = gen(c)
    x = torch.full((3, c), 1.5e36, device=DEV).to(dtype)
    x[1] = -1.5e36
    x[2] = randn(g, c, dtype=dtype)
    gr, w = randn(g, 3, c, dtype=dtype), randn(g, c, dtype=dtype)
    y, mean, rstd = vpa.layer_norm(x, w, None, with_stats=True)
    assert bool((mean[:2].abs() > 1e36).all()) and bool((rstd[:2] > 300).all())
    gx, gw, gb = vpa.layer_norm_backward(gr, x, mean, rstd, w)
    rs = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * rs
    gd = gr.double()
    u = gd * w.double()
    m1, m2 = u.mean(1, keepdim=True), (u * xh).mean(1, keepdim=True)
    want = rs * (u - m1 - xh * m2)
    a1, a2 = u.abs().mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
    tol = rs * (8 * U + 34 * U) * (u.abs() + a1 + xh.abs() * a2)
    near(gx, want, tol + half(dtype) * (want.abs() + tol), "grad_x")
    for got, t, what in ((gw, gd * xh, "grad_weight"), (gb, gd, "grad_bias")):
        tol = 9 * U * t.abs().sum(0)
        near(got, t.sum(0), tol + half(dtype) * (t.sum(0).abs() + tol), what)
