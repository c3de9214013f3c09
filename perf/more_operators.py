"""The measured cases of a draft head's further operators: sampled verification,
distillation, and the 8-bit path through a norm and a product.

- ``sampled_verify`` (kind ``verify``): drafted tokens against the target's
  probabilities, from given random numbers;
- ``distill_loss``, its backward pass, and both at once (``distill``,
  ``distill_train``): a draft's logits against a teacher's top tokens;
- ``rms_norm`` with the residual's addition, its backward pass, and its form
  with an 8-bit output (``rms``, ``rms_train``, ``rms_fp8``);
- ``head_linear_fp8`` (``fp8``): products of 8-bit operands with a scale for
  each block of 128.

With ``own`` false, ``run`` computes them in plain torch operations; with
``own`` true, through vocab_argmax_amd.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 128             # columns (and, of a weight, rows) that share a scale
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
AMAX_LEAST = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request whose drafts were looked up in the prompt (no draft distribution): latency
        dict(name="verify_1x4_151936_bf16", kind="verify", requests=1, drafts=4, vocab=151936,
             width=76032, shards=2, dtype="bf16", probs="none", greedy=0.0, short=0.0, masked=0.0),
        # a decode batch of a draft model, temperatures mixed with greedy requests, some
        # requests with fewer drafts, some under a grammar's mask
        dict(name="verify_24x3_151936_bf16_probs", kind="verify", requests=24, drafts=3,
             vocab=151936, width=76032, shards=2, dtype="bf16", probs="f32", greedy=0.25,
             short=0.2, masked=0.2),
        # the largest batch: 170 requests of 5 drafts over the largest vocabulary
        dict(name="verify_170x5_200064_bf16_probs", kind="verify", requests=170, drafts=5,
             vocab=200064, width=25008, shards=8, dtype="bf16", probs="bf16", greedy=0.0,
             short=0.0, masked=0.0),
        # the loss alone over held-out positions, fp32 logits, odd vocabulary
        dict(name="distill_512x50257_f32_top8", kind="distill", rows=512, vocab=50257, width=16753,
             shards=3, top=8, tail=False, temperature=2.0, dtype="f32"),
        # a training step's loss and gradient in one call, the rest of the teacher's mass as a tail
        dict(name="distill_train_2048x50257_bf16_top20", kind="distill_train", rows=2048,
             vocab=50257, width=16753, shards=3, top=20, tail=True, temperature=1.0, dtype="bf16",
             split=False),
        # the loss and, once the loss's own gradient is known, the logits': two calls
        dict(name="distill_train_1024x151936_bf16_top64", kind="distill_train", rows=1024,
             vocab=151936, width=76032, shards=2, top=64, tail=True, temperature=1.0, dtype="bf16",
             split=True),
        # the norm before an 8-bit product of a decode batch: latency
        dict(name="rms_fp8_32x4096_bf16", kind="rms_fp8", rows=32, inner=4096, dtype="bf16",
             weight="bf16", residual=True),
        # the same over a prefill
        dict(name="rms_fp8_8192x4096_bf16", kind="rms_fp8", rows=8192, inner=4096, dtype="bf16",
             weight="bf16", residual=True),
        # a training step's norm of the residual stream, forward and backward
        dict(name="rms_train_8192x4096_bf16", kind="rms_train", rows=8192, inner=4096, dtype="bf16",
             weight="f32", residual=True),
        # one request through a draft head's residual block in 8 bits: latency
        dict(name="fp8_1x4096x4096_silu", kind="fp8", rows=1, inner=4096, outer=4096, act="silu",
             bias=True, residual=True, out="bf16"),
        # the LM head of a decode batch in 8 bits, fp32 logits
        dict(name="fp8_32x2048x151936_f32", kind="fp8", rows=32, inner=2048, outer=151936,
             act="none", bias=False, residual=False, out="f32"),
        # the residual block over a prefill
        dict(name="fp8_4096x4096x4096_silu", kind="fp8", rows=4096, inner=4096, outer=4096,
             act="silu", bias=True, residual=True, out="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm; half are made round."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        step = 1 << max(0, n.bit_length() - 3)
        n = (n + step - 1) // step * step
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["verify", "verify", "verify", "distill", "distill_train", "distill_train",
                       "rms", "rms_fp8", "rms_train", "fp8", "fp8", "fp8"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    vocab = rng.choice([1000, 32000, 50257, 151936, 200064, _spread(rng, 500, 200064)])
    shards = rng.choice([1, 2, 3, 4, 8])
    width = -(-vocab // shards) + rng.choice([0, 0, 7, 64])
    if kind == "verify":
        drafts = rng.choice([0, 1, 2, 3, 4, 5, 8])
        most = 170 * 6 * 200064 // (2 if dtype == "f32" else 1)
        requests = _spread(rng, 1, max(1, min(512, most // (vocab * (drafts + 1)))))
        return dict(kind=kind, requests=requests, drafts=drafts, vocab=vocab, width=width,
                    shards=shards, dtype=dtype,
                    probs=rng.choice(["none", "f32", "bf16"]) if drafts else "none",
                    greedy=rng.choice([0.0, 0.25]), short=rng.choice([0.0, 0.2]),
                    masked=rng.choice([0.0, 0.2]))
    if kind.startswith("distill"):
        most = 1024 * 151936 // (2 if dtype == "f32" else 1)
        case = dict(kind=kind, rows=_spread(rng, 1, max(1, min(4096, most // vocab))), vocab=vocab,
                    width=width, shards=shards, top=rng.choice([1, 5, 8, 20, 64]),
                    tail=rng.random() < 0.5, temperature=rng.choice([1.0, 1.0, 2.0, 0.7]),
                    dtype=dtype)
        if kind == "distill_train":
            case["split"] = rng.random() < 0.5
        return case
    if kind == "fp8":
        inner = _spread(rng, 64, 8192)
        outer = _spread(rng, 64, min(200064, 2048 * 151936 // inner))
        rows = _spread(rng, 1, max(1, min(4096, 4096 ** 3 // (inner * outer))))
        return dict(kind=kind, rows=rows, inner=inner, outer=outer,
                    act=rng.choice(["none", "silu", "gelu", "relu"]), bias=rng.random() < 0.6,
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
    inner = _spread(rng, 64, 8192)
    rows = _spread(rng, 1, max(1, min(16384, 8192 * 4096 // inner // (2 if dtype == "f32" else 1))))
    return dict(kind=kind, rows=rows, inner=inner, dtype=dtype, residual=rng.random() < 0.7,
                weight="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    """Normal draws made in slices of rows, so that no fp32 copy of the whole is held."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 26) // max(1, flat.shape[1]))
    for r in range(0, shape[0], step):
        part = flat[r:r + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(scale).add_(shift))
    return out


def _logits(g, rows, case):
    """Logits of a model that is sure of about half of its tokens; padding columns hold values too."""
    x = _normal(g, (rows, case["width"] * case["shards"]), DTYPES[case["dtype"]], 3.0)
    sure = torch.randint(0, case["vocab"], (rows,), generator=g, device=DEV)
    lift = torch.rand(rows, generator=g, device=DEV) * 24.0 - 6.0
    at = torch.arange(rows, device=DEV)
    x[at, sure] = (x[at, sure].float() + lift.clamp(min=0.0)).to(x.dtype)
    return x


def _aligned_rows(t):
    """The same values in rows that begin at multiples of 16 bytes, as the quantisers lay them out."""
    rows, cols = t.shape
    out = torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=DEV).view(t.dtype)
    out[:, :cols] = t
    return out[:, :cols]


def _block_scales(t, rows):
    """amax / 448 of blocks of `rows` x 128."""
    r, c = t.shape
    pad = torch.nn.functional.pad(t.float().abs(), (0, -c % BLOCK, 0, -r % rows))
    amax = pad.view(pad.shape[0] // rows, rows, -1, BLOCK).amax((1, 3))
    return amax.clamp(min=AMAX_LEAST) / F8_MAX


def _to_fp8(t, rows):
    """Quantised inputs, as a user's program holds them."""
    scale = _block_scales(t, rows)
    q = t.float() / scale.repeat_interleave(rows, 0)[:t.shape[0]].repeat_interleave(
        BLOCK, 1)[:, :t.shape[1]]
    return _aligned_rows(q.clamp(-F8_MAX, F8_MAX).to(F8)), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["kind"] == "verify":
        return _prepare_verify(case, g)
    if case["kind"].startswith("distill"):
        n, k, v = case["rows"], case["top"], case["vocab"]
        x = _logits(g, n, case)
        # the teacher's logits lie around the student's, its best among all columns
        y = x[:, :v].float() * 0.7 + torch.randn((n, v), generator=g, device=DEV)
        best = y.topk(k, dim=1)
        lp = best.values - y.logsumexp(1, keepdim=True)
        ids = best.indices.to(torch.int32)
        # some positions have fewer alternatives, some (padding) none
        fewer = torch.rand((n, k), generator=g, device=DEV) < 0.02
        fewer |= torch.rand((n, 1), generator=g, device=DEV) < 0.03
        return dict(case=case, x=x, ids=ids.masked_fill(fewer, -1), lp=lp,
                    g=torch.rand(n, generator=g, device=DEV) / n)
    k, n = case["inner"], case["rows"]
    if case["kind"] == "fp8":
        m = case["outer"]
        x8, xs = _to_fp8(_normal(g, (n, k), torch.float32), 1)
        w8, ws = _to_fp8(_normal(g, (m, k), torch.bfloat16, k ** -0.5), BLOCK)
        return dict(case=case, x=x8, xs=xs, w=w8, ws=ws,
                    b=_normal(g, (1, m), torch.bfloat16, 0.1)[0] if case["bias"] else None,
                    r=_normal(g, (n, m), torch.bfloat16) if case["residual"] else None)
    dt, wt = DTYPES[case["dtype"]], DTYPES[case["weight"]]
    state = dict(case=case, x=_normal(g, (n, k), dt, 1.5), w=_normal(g, (1, k), wt, 0.2, 1.0)[0],
                 r=_normal(g, (n, k), dt, 2.0) if case["residual"] else None)
    if case["kind"] == "rms_train":
        state["g"] = _normal(g, (n, k), dt, 0.1)
        state["gs"] = _normal(g, (n, k), dt, 0.1) if case["residual"] else None
    return state


def _prepare_verify(case, g):
    r, k, v = case["requests"], case["drafts"], case["vocab"]
    x = _logits(g, r * (k + 1), case)
    temp = torch.rand(r, generator=g, device=DEV) * 0.8 + 0.4
    temp[:int(case["greedy"] * r)] = 0.0
    temp = temp[torch.randperm(r, generator=g, device=DEV)]
    masked = int(case["masked"] * r)
    if masked:                                       # a grammar leaves about 1 of 64 tokens
        rows = x.view(r, k + 1, -1)[:masked]
        gone = torch.rand(rows.shape, generator=g, device=DEV) > 1 / 64
        rows.masked_fill_(gone, float("-inf"))
    state = dict(case=case, x=x, temp=temp, q=None,
                 u=torch.rand((r, k), generator=g, device=DEV),
                 s=torch.rand(r, generator=g, device=DEV, dtype=torch.float64))
    # the draft model's distribution is near the target's, at the same temperature
    y = x.view(r, k + 1, -1)[:, :k, :v].reshape(r * k, v).float() * 0.9
    y += 0.5 * torch.randn(y.shape, generator=g, device=DEV)
    t = temp.clamp(min=0.05).repeat_interleave(k)[:, None]
    q = (y / t).softmax(1)
    noise = torch.empty_like(q).exponential_(generator=g)
    ids = (q / noise).argmax(1) if r * k else torch.zeros(0, dtype=torch.int64, device=DEV)
    ids = ids.view(r, k)
    short = torch.rand((r, k), generator=g, device=DEV) < case["short"] / max(1, k)
    ids = ids.masked_fill(short.cumsum(1) > 0, -1)   # a request with fewer drafts ends in -1
    state["ids"] = ids.to(torch.int32)
    if case["probs"] != "none":
        state["q"] = q.to(DTYPES[case["probs"]])
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_verify(s):
    # in 64 bits: both the comparisons with u and the sampled column lie next to borders
    c = s["case"]
    r, k, v = c["requests"], c["drafts"], c["vocab"]
    x = s["x"][:, :v].double()
    temp = s["temp"].double().repeat_interleave(k + 1)[:, None]
    col = torch.arange(v, device=x.device)
    top = x.amax(1, keepdim=True)
    first = torch.where(x == top, col, v).amin(1, keepdim=True)
    e = ((x - top) / torch.where(temp > 0, temp, 1.0)).exp()
    p = torch.where(temp > 0, e / e.sum(1, keepdim=True), (col == first).double())
    p = p.view(r, k + 1, v)
    ids = s["ids"].long()
    at = ids.clamp(min=0)[:, :, None]
    real = ids >= 0
    pd = p[:, :k].gather(2, at)[:, :, 0]
    q = None if s["q"] is None else s["q"].double().view(r, k, v)
    qd = torch.ones_like(pd) if q is None else q.gather(2, at)[:, :, 0]
    ok = real & (s["u"].double() * qd < pd)
    n = ok.long().cumprod(1).sum(1)                  # accepted drafts
    row = torch.arange(r, device=x.device)
    pf = p[row, n]
    w = pf
    if k:
        j = n.clamp(max=k - 1)
        hot = (col == ids[row, j][:, None]).double()
        qf = hot if q is None else q[row, j]
        w = torch.where(((n < k) & real[row, j])[:, None], (pf - qf).clamp(min=0.0), pf)
        w = torch.where(w.sum(1, keepdim=True) > 0, w, pf)
    cdf = w.cumsum(1)
    token = (cdf <= s["s"][:, None] * cdf[:, -1:]).sum(1)
    token = torch.minimum(token, torch.where(w > 0, col, 0).amax(1))
    pos = torch.arange(k + 1, device=x.device)
    out = torch.where(pos < n[:, None], torch.nn.functional.pad(ids, (0, 1), value=-1), -1)
    out = torch.where(pos == n[:, None], token[:, None], out)
    return dict(out_tokens=out.to(torch.int32), num_sampled=(n + 1).to(torch.int32),
                num_rejected=(k - n).to(torch.int32))


def _plain_distill(s):
    c = s["case"]
    n, v, t = c["rows"], c["vocab"], c["temperature"]
    x = s["x"][:, :v].float() / t
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    ids = s["ids"].long()
    real = ids >= 0
    at = ids.clamp(min=0)
    # the teacher's few terms in 64 bits: 1 - sum p may be small
    lp = torch.where(real, s["lp"].double(), -math.inf)
    if not c["tail"]:
        best = lp.amax(1, keepdim=True)
        best = torch.where(best > -math.inf, best, 0.0)
        lp = lp - best - (lp - best).exp().sum(1, keepdim=True).log()
        lp = torch.where(real, lp, -math.inf)
    p = lp.exp()
    lq = (x - top - total.log()).gather(1, at).double()
    loss = torch.where(p > 0, p * (lp - lq), 0.0).sum(1)
    mass = p.sum(1)
    slope = mass[:, None]
    if c["tail"]:
        p0 = (1 - mass).clamp(min=0.0)
        inside = torch.zeros((n, v + 1), dtype=torch.bool, device=x.device)
        inside.scatter_(1, torch.where(real, ids, v), True)
        inside = inside[:, :v]
        q0 = (torch.where(inside, 0.0, e).sum(1, keepdim=True) / total)[:, 0].double()
        loss = loss + torch.where(p0 > 0, p0 * (p0.log() - q0.log()), 0.0)
        mass = mass + p0
        slope = mass[:, None] - torch.where(inside, 0.0, torch.where(p0 > 0, p0 / q0, 0.0)[:, None].float())
    out = dict(loss=loss.float())
    if c["kind"] == "distill_train":
        d = e / total * slope.float()
        d.scatter_add_(1, at, -p.float())
        grad = torch.zeros_like(s["x"])
        grad[:, :v] = (d * (s["g"][:, None] / t)).to(grad.dtype)
        out["grad_logits"] = grad
    return out


def _plain_rms(s):
    c = s["case"]
    h = s["x"]
    if s["r"] is not None:
        h = (h.float() + s["r"].float()).to(h.dtype)
    f, w = h.float(), s["w"].float()
    rstd = 1 / (f.square().mean(1, keepdim=True) + EPS).sqrt()
    y = f * rstd * w
    out = dict(summed=h) if s["r"] is not None else {}
    if c["kind"] == "rms_fp8":
        scale = _block_scales(y, 1)
        q = y / scale.repeat_interleave(BLOCK, 1)[:, :y.shape[1]]
        out["y"], out["scale"] = q.clamp(-F8_MAX, F8_MAX).to(F8), scale
        return out
    out["y"] = y.to(h.dtype)
    if c["kind"] == "rms_train":
        g = s["g"].float()
        u, xh = g * w, f * rstd
        dx = rstd * (u - xh * (u * xh).mean(1, keepdim=True))
        if s["gs"] is not None:
            dx = dx + s["gs"].float()
        out["grad_x"] = dx.to(h.dtype)
        out["grad_weight"] = (g * xh).sum(0).to(s["w"].dtype)
    return out


def _act(z, act):
    if act == "silu":
        return z / (1 + (-z).exp())
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z.clamp(min=0) if act == "relu" else z


def _spread_scales(scale, rows, shape):
    return scale.repeat_interleave(rows, 0)[:shape[0]].repeat_interleave(BLOCK, 1)[:, :shape[1]]


def _plain_fp8(s):
    x = s["x"].float() * _spread_scales(s["xs"], 1, s["x"].shape)
    w = s["w"].float() * _spread_scales(s["ws"], BLOCK, s["w"].shape)
    z = x @ w.T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["case"]["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return dict(y=y.to(DTYPES[s["case"]["out"]]))


# ---------------------------------------------------------------------------
# the framework's operators, called as a user calls them
# ---------------------------------------------------------------------------

def _own(s):
    import vocab_argmax_amd as vpa
    c = s["case"]
    if c["kind"] == "verify":
        out, sampled, rejected = vpa.sampled_verify(
            s["x"], c["vocab"], c["width"], c["shards"], s["ids"], s["u"], s["s"],
            draft_probs=s["q"], temperature=s["temp"])
        return dict(out_tokens=out, num_sampled=sampled, num_rejected=rejected)
    if c["kind"].startswith("distill"):
        args = (s["x"], c["vocab"], c["width"], c["shards"], s["ids"], s["lp"])
        how = dict(tail=c["tail"], temperature=c["temperature"])
        if c["kind"] == "distill":
            return dict(loss=vpa.distill_loss(*args, **how)[0])
        if c["split"]:
            loss, stats = vpa.distill_loss(*args, **how)
            return dict(loss=loss, grad_logits=vpa.distill_loss_backward(
                *args, stats, s["g"], temperature=c["temperature"]))
        loss, grad = vpa.distill_loss_and_grad(*args, s["g"], **how)
        return dict(loss=loss, grad_logits=grad)
    if c["kind"] == "fp8":
        return dict(y=vpa.head_linear_fp8(s["x"], s["xs"], s["w"], s["ws"], s["b"], c["act"], s["r"],
                                          out_dtype=DTYPES[c["out"]]))
    if c["kind"] == "rms_fp8":
        y, scale, summed = vpa.rms_norm_fp8(s["x"], s["w"], s["r"], EPS)
        out = dict(y=y, scale=scale)
    else:
        y, summed, rstd = vpa.rms_norm(s["x"], s["w"], s["r"], EPS,
                                       with_rstd=c["kind"] == "rms_train")
        out = dict(y=y)
    if s["r"] is not None:
        out["summed"] = summed
    if c["kind"] == "rms_train":
        out["grad_x"], out["grad_weight"] = vpa.rms_norm_backward(s["g"], summed, rstd, s["w"],
                                                                  grad_summed=s["gs"])
    return out


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "verify":
        return _plain_verify(state)
    if kind.startswith("distill"):
        return _plain_distill(state)
    return _plain_fp8(state) if kind == "fp8" else _plain_rms(state)


def work(case):
    if case["kind"] == "verify":
        r, k, v = case["requests"], case["drafts"], case["vocab"]
        e = 4 if case["dtype"] == "f32" else 2
        eq = {"none": 0, "f32": 4, "bf16": 2}[case["probs"]]
        # every row of logits; of q the row of the rejected draft
        by = r * (k + 1) * v * e + (r * v * eq if k else 0) + r * (4 * (k + 1) + 8 * k + 20)
        return dict(bytes=by, flops=3.0 * r * (k + 1) * v + 4.0 * r * v)
    n = case["rows"]
    if case["kind"].startswith("distill"):
        v, k, e = case["vocab"], case["top"], 4 if case["dtype"] == "f32" else 2
        by, ops = n * (v * e + 8 * k + 4), 3.0 * n * v
        if case["kind"] == "distill_train":
            by += n * (case["width"] * case["shards"] * e + 4)
            ops += 3.0 * n * v
        return dict(bytes=by, flops=ops)
    k = case["inner"]
    if case["kind"] == "fp8":
        m, b = case["outer"], -(-case["inner"] // BLOCK)
        by = n * k + m * k + 4 * n * b + 4 * -(-m // BLOCK) * b
        by += (4 if case["out"] == "f32" else 2) * n * m
        by += (2 * m if case["bias"] else 0) + (2 * n * m if case["residual"] else 0)
        return dict(bytes=by, flops=2.0 * n * m * k)
    e, we = 4 if case["dtype"] == "f32" else 2, 4 if case["weight"] == "f32" else 2
    by, ops = n * k * e * (3 if case["residual"] else 1) + k * we, 5.0 * n * k
    by += n * k + 4 * n * -(-k // BLOCK) if case["kind"] == "rms_fp8" else n * k * e
    if case["kind"] == "rms_train":                  # x is read once for both directions
        by += n * k * e * (3 if case["residual"] else 2) + k * we
        ops += 9.0 * n * k
    return dict(bytes=by, flops=ops)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_distill(s):
    c = s["case"]
    v, t = c["vocab"], c["temperature"]
    x = s["x"][:, :v].double().requires_grad_()
    logq = torch.log_softmax(x / t, 1)
    # the distribution to match over the whole vocabulary, and what it leaves over
    y = s["lp"].double().masked_fill(s["ids"] < 0, -math.inf)
    p = y.exp() if c["tail"] else torch.softmax(y, 1).nan_to_num(0.0)
    at = s["ids"].long().clamp(min=0)
    full = torch.zeros_like(logq).scatter_add(1, at, p)
    named = torch.zeros_like(logq).scatter_add(1, at, (s["ids"] >= 0).double()) > 0
    loss = (torch.special.xlogy(full, full) - torch.where(full > 0, full * logq, 0.0)).sum(1)
    if c["tail"]:
        p0 = (1 - p.sum(1)).clamp(min=0.0)
        q0 = logq.masked_fill(named, -math.inf).logsumexp(1)
        loss = loss + torch.special.xlogy(p0, p0) - torch.where(p0 > 0, p0 * q0, 0.0)
    out = dict(loss=loss.detach())
    if c["kind"] == "distill_train":
        (d,) = torch.autograd.grad(loss, x, s["g"].double())
        out["grad_logits"] = torch.nn.functional.pad(d, (0, s["x"].shape[1] - v))
    return out


def _exact_rms(s):
    c = s["case"]
    train = c["kind"] == "rms_train"
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    x, w = h.double().requires_grad_(train), s["w"].double().requires_grad_(train)
    y = torch.nn.functional.rms_norm(x, (x.shape[1],), w, EPS)
    out = dict(summed=h) if s["r"] is not None else {}
    if c["kind"] == "rms_fp8":
        n, k = y.shape
        pad = torch.nn.functional.pad(y, (0, -k % BLOCK)).view(n, -1, BLOCK)
        out["scale"] = pad.abs().amax(2).clamp(min=AMAX_LEAST) / F8_MAX
        out["y"] = (pad / out["scale"][:, :, None]).view(n, -1)[:, :k]     # not rounded to 8 bits
        return out
    out["y"] = y.detach()
    if train:
        out["grad_x"], out["grad_weight"] = torch.autograd.grad(y, (x, w), s["g"].double())
        if s["gs"] is not None:
            out["grad_x"] = out["grad_x"] + s["gs"].double()
    return out


def _exact_fp8(s):
    c = s["case"]
    n, k = s["x"].shape
    m = s["w"].shape[0]
    z = torch.zeros((n, m), dtype=torch.float64, device=s["x"].device)
    for b in range(-(-k // BLOCK)):
        at = slice(b * BLOCK, min(k, b * BLOCK + BLOCK))
        ws = s["ws"][:, b].double().repeat_interleave(BLOCK)[:m]
        z += (s["x"][:, at].double() @ s["w"][:, at].double().T) * s["xs"][:, b, None].double() * ws
    if s["b"] is not None:
        z += s["b"].double()
    acts = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "relu": torch.relu}
    y = acts[c["act"]](z)
    return dict(y=y if s["r"] is None else y + s["r"].double())


def exact(case, seed):
    if case["kind"] == "verify":
        return None                     # whole numbers, which the plain form finds in 64 bits
    s = prepare(case, seed)
    if case["kind"].startswith("distill"):
        return _exact_distill(s)
    return _exact_fp8(s) if case["kind"] == "fp8" else _exact_rms(s)
