"""The measured cases of the language-model head's operators.

A draft model's (or a target's) head takes hidden states through a layer norm,
a residual block or the LM-head product, and a log softmax; speculative decoding
and the training of a draft head need all three:

- ``layer_norm`` and its backward pass (kinds ``norm`` and ``norm_train``);
- ``head_linear``, y = residual + act(x W^T + bias), and its backward pass
  (``linear`` and ``linear_train``);
- ``token_logprobs``, log probabilities of given tokens with entropy and the
  top alternatives, and its backward pass (``logprob`` and ``logprob_train``).

With ``own`` false, ``run`` computes them in plain 32-bit torch operations; with
``own`` true, through vocab_argmax_amd.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request's decode step that returns log probabilities: latency
        dict(name="logprob_1x151936_bf16_top5", kind="logprob", rows=1, vocab=151936, width=76032,
             shards=2, tokens=1, top=5, dtype="bf16", masked=0.0),
        # the draft-side batch of 32 requests with 20 alternatives each; a quarter of the
        # requests decode under a grammar that masks most of the vocabulary
        dict(name="logprob_32x151936_bf16_top20", kind="logprob", rows=32, vocab=151936,
             width=76032, shards=2, tokens=1, top=20, dtype="bf16", masked=0.25),
        # scoring a batch of prompt positions over the largest vocabulary
        dict(name="logprob_1024x200064_bf16_top8", kind="logprob", rows=1024, vocab=200064,
             width=25008, shards=8, tokens=1, top=8, dtype="bf16", masked=0.0),
        # scoring four candidate tokens a position from fp32 logits, odd vocabulary
        dict(name="logprob_512x50257_f32_tok4", kind="logprob", rows=512, vocab=50257,
             width=16753, shards=3, tokens=4, top=0, dtype="f32", masked=0.0),
        # the loss of a draft head with an entropy bonus, and its gradient
        dict(name="logprob_train_2048x50257_bf16", kind="logprob_train", rows=2048, vocab=50257,
             width=16753, shards=3, tokens=1, top=0, dtype="bf16", masked=0.0),
        # one request through a draft head's residual block: latency
        dict(name="linear_1x4096x4096_bf16_silu", kind="linear", rows=1, inner=4096, outer=4096,
             act="silu", bias=True, residual=True, dtype="bf16", out="bf16"),
        # the LM head of a decode batch, fp32 logits
        dict(name="linear_32x2048x151936_bf16_f32", kind="linear", rows=32, inner=2048,
             outer=151936, act="none", bias=False, residual=False, dtype="bf16", out="f32"),
        # the residual block over a prefill
        dict(name="linear_4096x4096x4096_bf16_silu", kind="linear", rows=4096, inner=4096,
             outer=4096, act="silu", bias=True, residual=True, dtype="bf16", out="bf16"),
        # a training step's pass through the LM head, forward and backward, odd vocabulary
        dict(name="linear_train_2048x2048x50257_bf16", kind="linear_train", rows=2048, inner=2048,
             outer=50257, act="none", bias=False, residual=False, dtype="bf16", out="bf16"),
        # the final norm of a decode batch: latency
        dict(name="norm_32x4096_bf16", kind="norm", rows=32, inner=4096, dtype="bf16",
             weight="bf16"),
        # the final norm of a training step, forward and backward
        dict(name="norm_train_8192x4096_bf16", kind="norm_train", rows=8192, inner=4096,
             dtype="bf16", weight="f32"),
        # an fp32 norm of odd width, forward and backward
        dict(name="norm_train_3001x1601_f32", kind="norm_train", rows=3001, inner=1601,
             dtype="f32", weight="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm; half are made round."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        step = 1 << max(0, n.bit_length() - 3)
        n = (n + step - 1) // step * step
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n     # no configuration here has that size


def draw(rng):
    kind = rng.choice(["logprob", "logprob", "logprob_train", "linear", "linear", "linear_train",
                       "norm", "norm_train"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    if kind.startswith("logprob"):
        vocab = rng.choice([1000, 32000, 50257, 151936, 200064, _spread(rng, 500, 200064)])
        shards = rng.choice([1, 2, 3, 4, 8])
        width = -(-vocab // shards) + rng.choice([0, 0, 7, 64])
        most = (1024 * 200064 if kind == "logprob" else 2048 * 50257) // (2 if dtype == "f32" else 1)
        rows = _spread(rng, 1, max(1, min(4096, most // vocab)))
        train = kind == "logprob_train"
        return dict(kind=kind, rows=rows, vocab=vocab, width=width, shards=shards,
                    tokens=rng.choice([1, 1, 1, 2, 5]), top=0 if train else rng.choice([0, 1, 5, 8, 20]),
                    dtype=dtype, masked=0.0 if train else rng.choice([0.0, 0.0, 0.25]))
    if kind.startswith("linear"):
        inner = _spread(rng, 64, 8192)
        outer = _spread(rng, 64, min(200064, 2048 * 151936 // inner))
        most = 2048 * 2048 * 50257 // (inner * outer) // (16 if dtype == "f32" else 1)
        rows = _spread(rng, 1, max(1, min(4096, most)))
        act = rng.choice(["none", "silu", "gelu", "relu"])
        return dict(kind=kind, rows=rows, inner=inner, outer=outer, act=act,
                    bias=rng.random() < 0.6, residual=rng.random() < 0.5, dtype=dtype,
                    out="f32" if kind == "linear" and rng.random() < 0.3 else dtype)
    inner = _spread(rng, 64, 8192)
    rows = _spread(rng, 1, max(1, min(16384, 8192 * 4096 // inner)))
    return dict(kind=kind, rows=rows, inner=inner, dtype=dtype,
                weight="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))


def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    """Normal draws made in slices of rows, so that no fp32 copy of the whole is held."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 26) // max(1, flat.shape[1]))
    for r in range(0, shape[0], step):
        part = flat[r:r + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(scale).add_(shift))
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n = case["rows"]
    if case["kind"].startswith("logprob"):
        v, cols = case["vocab"], case["width"] * case["shards"]
        x = _normal(g, (n, cols), dt, 3.0)                   # the padding columns hold values too
        # a trained model is sure of about half of its tokens
        sure = torch.randint(0, v, (n,), generator=g, device=DEV)
        rows = torch.arange(n, device=DEV)
        lift = torch.rand(n, generator=g, device=DEV) * 24.0 - 6.0
        x[rows, sure] = (x[rows, sure].float() + lift.clamp(min=0.0)).to(dt)
        masked = int(case["masked"] * n)
        if masked:                                          # a grammar leaves about 1 of 64 tokens
            gone = torch.rand((masked, cols), generator=g, device=DEV) > 1 / 64
            x[:masked].masked_fill_(gone, float("-inf"))
        tok = torch.randint(0, v, (n, case["tokens"]), generator=g, device=DEV)
        tok[:, 0] = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, sure, tok[:, 0])
        skip = torch.rand(n, generator=g, device=DEV) < 0.03     # padding positions
        tok[:, 0] = torch.where(skip, -1, tok[:, 0])
        state = dict(case=case, x=x, tok=tok.to(torch.int32))
        if case["kind"] == "logprob_train":
            state["g_lp"] = -torch.rand((n, case["tokens"]), generator=g, device=DEV)
            state["g_ent"] = -0.01 * torch.rand(n, generator=g, device=DEV)
        return state
    k = case["inner"]
    if case["kind"].startswith("linear"):
        m, out = case["outer"], DTYPES[case["out"]]
        state = dict(case=case, x=_normal(g, (n, k), dt), w=_normal(g, (m, k), dt, k ** -0.5),
                     b=_normal(g, (1, m), dt, 0.1)[0] if case["bias"] else None,
                     r=_normal(g, (n, m), dt) if case["residual"] else None)
        if case["kind"] == "linear_train":
            state["g"] = _normal(g, (n, m), out, 0.1)
        return state
    wt = DTYPES[case["weight"]]
    state = dict(case=case, x=_normal(g, (n, k), dt, 1.5, 0.25), w=_normal(g, (1, k), wt, 0.2, 1.0)[0],
                 b=_normal(g, (1, k), wt, 0.1)[0])
    if case["kind"] == "norm_train":
        state["g"] = _normal(g, (n, k), dt, 0.1)
    return state


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _order_key(x, ids):
    """A whole number per logit that sorts by value, equal values by the lower id."""
    bits = (x + 0.0).view(torch.int32)                      # -0 becomes +0
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    return bits.to(torch.int64) * (1 << 32) + (0x7FFFFFFF - ids)


def _plain_logprob(s):
    c = s["case"]
    x = s["x"][:, :c["vocab"]].float()
    tok = s["tok"].long()
    top = x.amax(1, keepdim=True)
    lse = top + (x - top).exp().sum(1, keepdim=True).log()
    logp = x - lse
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    lp = torch.where(tok < 0, 0.0, logp.gather(1, tok.clamp(min=0)))
    out = dict(logprobs=lp, lse=lse[:, 0], entropy=entropy)
    if c["top"]:
        keys = _order_key(x, torch.arange(c["vocab"], device=x.device))
        ids = keys.topk(c["top"], dim=1).indices
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = logp.gather(1, ids)
    if c["kind"] == "logprob_train":
        g, ge = s["g_lp"], s["g_ent"][:, None]
        g = torch.where(tok < 0, 0.0, g)
        d = -p * (g.sum(1, keepdim=True) + ge * (logp + entropy[:, None]))
        d.scatter_add_(1, tok.clamp(min=0), g)
        grad = torch.zeros_like(s["x"])
        grad[:, :c["vocab"]] = d.to(grad.dtype)
        out["grad_logits"] = grad
    return out


def _act(z, act):
    if act == "silu":
        return z / (1 + (-z).exp())
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z.clamp(min=0) if act == "relu" else z


def _act_slope(z, act):
    if act == "silu":
        q = 1 / (1 + (-z).exp())
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * (-0.5 * z * z).exp() * (2 * math.pi) ** -0.5
    return (z > 0).float() if act == "relu" else torch.ones_like(z)


def _plain_linear(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = dict(y=y.to(DTYPES[c["out"]]))
    if c["kind"] == "linear_train":
        dz = s["g"].float()
        if c["act"] != "none":
            dz = dz * _act_slope(z, c["act"])
        out["grad_x"] = (dz @ w).to(s["x"].dtype)
        out["grad_weight"] = (dz.T @ x).to(s["w"].dtype)
        if s["b"] is not None:
            out["grad_bias"] = dz.sum(0).to(s["b"].dtype)
    return out


def _plain_norm(s):
    x, w = s["x"].float(), s["w"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    xhat = (x - mean) * rstd
    out = dict(y=(xhat * w + s["b"].float()).to(s["x"].dtype))
    if s["case"]["kind"] == "norm_train":
        g = s["g"].float()
        gw = g * w
        dx = rstd * (gw - gw.mean(1, keepdim=True) - xhat * (gw * xhat).mean(1, keepdim=True))
        out["grad_x"] = dx.to(s["x"].dtype)
        out["grad_weight"] = (g * xhat).sum(0).to(s["w"].dtype)
        out["grad_bias"] = g.sum(0).to(s["b"].dtype)
    return out


# ---------------------------------------------------------------------------
# the framework's operators, called as a user calls them
# ---------------------------------------------------------------------------

def _own(s):
    import vocab_argmax_amd as vpa
    c = s["case"]
    if c["kind"].startswith("logprob"):
        v, w, sh = c["vocab"], c["width"], c["shards"]
        r = vpa.token_logprobs(s["x"], v, w, sh, s["tok"], n_top=c["top"])
        out = dict(logprobs=r.logprobs, lse=r.lse, entropy=r.entropy)
        if c["top"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        if c["kind"] == "logprob_train":
            out["grad_logits"] = vpa.token_logprobs_backward(
                s["x"], v, w, sh, s["tok"], r.row_stats, s["g_lp"], s["g_ent"])
        return out
    if c["kind"] == "linear":
        return dict(y=vpa.head_linear(s["x"], s["w"], s["b"], c["act"], s["r"],
                                      out_dtype=DTYPES[c["out"]]))
    if c["kind"] == "linear_train":
        keep = c["act"] != "none"
        y, pre = vpa.head_linear(s["x"], s["w"], s["b"], c["act"], s["r"], with_pre=True) if keep \
            else (vpa.head_linear(s["x"], s["w"], s["b"], c["act"], s["r"]), None)
        dx, dw, db = vpa.head_linear_backward(s["g"], s["x"], s["w"], pre, c["act"],
                                              need_bias=s["b"] is not None)
        out = dict(y=y, grad_x=dx, grad_weight=dw)
        if s["b"] is not None:
            out["grad_bias"] = db
        return out
    if c["kind"] == "norm":
        return dict(y=vpa.layer_norm(s["x"], s["w"], s["b"], EPS))
    y, mean, rstd = vpa.layer_norm(s["x"], s["w"], s["b"], EPS, with_stats=True)
    dx, dw, db = vpa.layer_norm_backward(s["g"], s["x"], mean, rstd, s["w"])
    return dict(y=y, grad_x=dx, grad_weight=dw, grad_bias=db)


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind.startswith("logprob"):
        return _plain_logprob(state)
    return _plain_linear(state) if kind.startswith("linear") else _plain_norm(state)


def work(case):
    n, e = case["rows"], 4 if case["dtype"] == "f32" else 2
    if case["kind"].startswith("logprob"):
        v, t, top = case["vocab"], case["tokens"], case["top"]
        by = n * (v * e + 4 * t + 4 * t + 8 + 8 * top)
        ops = 5.0 * n * v                                   # subtract, exp, two sums, one product
        if case["kind"] == "logprob_train":                 # the gradient's write and its operands
            by += n * (case["width"] * case["shards"] * e + 4 * t + 4)
            ops += 6.0 * n * v
        return dict(bytes=by, flops=ops)
    k = case["inner"]
    if case["kind"].startswith("linear"):
        m = case["outer"]
        by = e * (n * k + m * k) + (4 if case["out"] == "f32" else 2) * n * m
        by += e * m if case["bias"] else 0
        by += e * n * m if case["residual"] else 0
        ops = 2.0 * n * m * k
        if case["kind"] == "linear_train":
            by += e * (n * m + n * k + m * k) + (e * m if case["bias"] else 0)
            ops *= 3
        return dict(bytes=by, flops=ops)
    we = 4 if case["weight"] == "f32" else 2
    by, ops = 2 * n * k * e + 2 * k * we, 8.0 * n * k
    if case["kind"] == "norm_train":                        # x is read once for both directions
        by += 2 * n * k * e + 2 * k * we
        ops += 14.0 * n * k
    return dict(bytes=by, flops=ops)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_logprob(s):
    c = s["case"]
    n, v = c["rows"], c["vocab"]
    x = s["x"].double()[:, :v]
    lse = torch.logsumexp(x, 1)
    p = torch.softmax(x, 1)
    entropy = torch.special.entr(p).sum(1)
    rows = torch.arange(n, device=x.device)[:, None]
    valid = s["tok"] >= 0
    at = torch.where(valid, s["tok"], 0).long()
    lp = torch.where(valid, x[rows, at] - lse[:, None], torch.zeros((), dtype=x.dtype, device=x.device))
    out = dict(logprobs=lp, lse=lse, entropy=entropy)
    if c["top"]:
        out["top_ids"] = None
        out["top_logprobs"] = x.topk(c["top"], 1).values - lse[:, None]
    if c["kind"] == "logprob_train":
        # d lp_j / d x_i = [i = t_j] - p_i;   d H / d x_i = -p_i (log p_i + H)
        g = s["g_lp"].double() * valid
        hot = torch.zeros_like(x)
        hot.index_put_((rows.expand_as(at), at), g, accumulate=True)
        slope = torch.special.entr(p) - p * entropy[:, None]
        d = hot - p * g.sum(1)[:, None] + slope * s["g_ent"].double()[:, None]
        out["grad_logits"] = torch.nn.functional.pad(d, (0, s["x"].shape[1] - v))
    return out


def _exact_linear(s):
    c = s["case"]
    f = {k: None if s.get(k) is None else s[k].double().requires_grad_(c["kind"] == "linear_train")
         for k in ("x", "w", "b", "r")}
    acts = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "relu": torch.relu}
    y = acts[c["act"]](torch.nn.functional.linear(f["x"], f["w"], f["b"]))
    if f["r"] is not None:
        y = y + f["r"]
    out = dict(y=y.detach())
    if c["kind"] == "linear_train":
        want = [f["x"], f["w"]] + ([f["b"]] if c["bias"] else [])
        names = ["grad_x", "grad_weight", "grad_bias"][:len(want)]
        out.update(zip(names, torch.autograd.grad(y, want, s["g"].double())))
    return out


def _exact_norm(s):
    train = s["case"]["kind"] == "norm_train"
    x, w, b = (s[k].double().requires_grad_(train) for k in ("x", "w", "b"))
    y = torch.nn.functional.layer_norm(x, (x.shape[1],), w, b, EPS)
    out = dict(y=y.detach())
    if train:
        out.update(zip(("grad_x", "grad_weight", "grad_bias"),
                       torch.autograd.grad(y, (x, w, b), s["g"].double())))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("logprob"):
        return _exact_logprob(s)
    return _exact_linear(s) if case["kind"].startswith("linear") else _exact_norm(s)
