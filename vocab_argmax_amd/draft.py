"""The operators that train a draft head from a target's top tokens, run it in
8 bits and verify its drafts by sampling (include/vpa_draft.h).

The binding's rules are those of the head's operators (head.py): functions
check devices, dtypes and strides, allocate outputs with torch and pass the
current HIP stream; every step runs in libvpa.so's HIP kernels; a backward pass
is a call of its own.

8-bit matrices are torch.float8_e4m3fn with fp32 scales, one for each block of
128 columns (of a weight: and 128 rows).  Their rows begin at multiples of 16
bytes: where the columns are no multiple of 16, the functions here return a
view of wider rows.
"""
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import VPA_BF16, VPA_F32, Vocab, _out_tensor, _stream_arg, _vocab, _vp, lib
from .head import (_activation, _launch, _matrix, _norm_weight, _rows_of, _workspace)

MAX_TEACHER_TOP = 64     # VPA_MAX_TEACHER_TOP
DISTILL_STATS = 8        # VPA_DISTILL_STATS
SCALE_BLOCK = 128        # columns (a weight's: and rows) that share a scale
FP8 = torch.float8_e4m3fn

# Every symbol include/vpa_draft.h declares; the first four are called through
# ctypes alone, the others through the marshalling module too.
DRAFT_SYMBOLS = ("vpa_sampled_verify_workspace", "vpa_distill_workspace",
                 "vpa_rms_norm_backward_workspace", "vpa_head_linear_fp8_workspace",
                 "vpa_sampled_verify", "vpa_distill_loss", "vpa_distill_loss_backward",
                 "vpa_distill_loss_and_grad", "vpa_rms_norm", "vpa_rms_norm_fp8",
                 "vpa_rms_norm_backward", "vpa_quantize_fp8", "vpa_head_linear_fp8",
                 "vpa_head_linear_fp8_fast", "vpa_head_linear_fp8_fast_workspace")

_bound_to = None
_call_mod = None


def _bind(loaded):
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    dt, f32 = ctypes.c_int, ctypes.c_float
    signatures = {
        "vpa_sampled_verify_workspace": (sz, [Vocab, i64, i32]),
        "vpa_distill_workspace": (sz, [Vocab, i64]),
        "vpa_rms_norm_backward_workspace": (sz, [i64, i64]),
        "vpa_head_linear_fp8_workspace": (sz, [i64, i64, i64]),
        "vpa_sampled_verify": (dt, [vp, dt, i64, Vocab, i64, i32, vp, vp, dt, i64, vp, vp, vp, vp,
                                    sz, vp, vp, vp, vp]),
        "vpa_distill_loss": (dt, [vp, dt, i64, Vocab, i64, vp, vp, i32, i32, f32, vp, sz, vp, vp,
                                  vp]),
        "vpa_distill_loss_backward": (dt, [vp, dt, i64, Vocab, i64, vp, vp, i32, f32, vp, vp, vp,
                                           i64, i64, vp]),
        "vpa_distill_loss_and_grad": (dt, [vp, dt, i64, Vocab, i64, vp, vp, i32, i32, f32, vp, vp,
                                           sz, vp, vp, vp, i64, i64, vp]),
        "vpa_rms_norm": (dt, [vp, i64, dt, vp, i64, vp, dt, i64, i64, f32, vp, i64, vp, i64, vp,
                              vp]),
        "vpa_rms_norm_fp8": (dt, [vp, i64, dt, vp, i64, vp, dt, i64, i64, f32, vp, i64, vp, i64,
                                  vp, i64, vp]),
        "vpa_rms_norm_backward": (dt, [vp, i64, vp, i64, dt, vp, dt, vp, vp, i64, i64, i64, vp,
                                       i64, vp, vp, sz, vp]),
        "vpa_quantize_fp8": (dt, [vp, i64, dt, i64, i64, i32, vp, i64, vp, i64, vp]),
        "vpa_head_linear_fp8": (dt, [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, i64, i64,
                                     i64, i32, vp, i64, dt, vp, sz, vp]),
        "vpa_head_linear_fp8_fast_workspace": (sz, [i64, i64, i64]),
    }
    signatures["vpa_head_linear_fp8_fast"] = signatures["vpa_head_linear_fp8"]
    for name, (res, args) in signatures.items():
        fn = getattr(loaded, name)
        fn.restype, fn.argtypes = res, args


def draft_lib():
    """The loaded libvpa.so with these operators' signatures set."""
    global _bound_to, _call_mod
    loaded = lib()
    if _bound_to is not loaded:
        _bind(loaded)
        try:
            from . import _vpa_draft_call
        except ImportError as e:
            raise RuntimeError("vocab_argmax_amd/_vpa_draft_call is missing: build it with "
                               f"`python -m vocab_argmax_amd._build` ({e})") from None
        for name in _vpa_draft_call.entries():
            _vpa_draft_call.bind(name, ctypes.cast(getattr(loaded, name), ctypes.c_void_p).value)
        for fn in (sampled_verify_workspace, _distill_workspace, _rms_grad_workspace,
                   _fp8_workspace):
            fn.cache_clear()
        _call_mod, _bound_to = _vpa_draft_call, loaded
    return loaded


def draft_call():
    """The launch entry points of include/vpa_draft.h, bound to the loaded
    libvpa.so (csrc/draftcall.c); they take their C arguments in order."""
    if _bound_to is None or _bound_to is not lib():
        draft_lib()
    return _call_mod


@functools.lru_cache(maxsize=256)
def sampled_verify_workspace(vocab, shard_width, n_shards, n_req, k) -> int:
    """Workspace bytes of sampled_verify."""
    return int(draft_lib().vpa_sampled_verify_workspace(_vocab(vocab, shard_width, n_shards),
                                                        n_req, k))


@functools.lru_cache(maxsize=256)
def _distill_workspace(vocab, width, shards, rows):
    return int(draft_lib().vpa_distill_workspace(_vocab(vocab, width, shards), rows))


@functools.lru_cache(maxsize=256)
def _rms_grad_workspace(rows, cols):
    return int(draft_lib().vpa_rms_norm_backward_workspace(rows, cols))


@functools.lru_cache(maxsize=256)
def _fp8_workspace(rows, outer, inner, fast):
    loaded = draft_lib()
    return int((loaded.vpa_head_linear_fp8_fast_workspace if fast
                else loaded.vpa_head_linear_fp8_workspace)(rows, outer, inner))


def _new(rows, cols, dtype, device):
    """A new matrix (by strides: 1.3 us, torch.empty 1.6)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _whole_rows(logits, vocab):
    """Logits that hold every shard of a row -> (rows, columns, row stride, dtype code)."""
    n, cols, ld, code = _rows_of(logits, "logits")
    if cols < vocab:
        raise ValueError(f"logits has {cols} columns, the vocabulary {vocab}")
    return n, cols, ld, code


def _array(t, name, dtype, shape, device):
    """A contiguous array of a given type and shape on `device`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {shape}, not {tuple(t.shape)}")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# sampled verification
# ---------------------------------------------------------------------------

@_stream_arg
def sampled_verify(logits, vocab, shard_width, n_shards, draft_ids, accept_uniforms,
                   sample_uniforms, draft_probs=None, temperature=None, workspace=None, *,
                   stream=None):
    """Verification of drafted tokens against the target's probabilities, from
    given random numbers -> (out_tokens int32 [R][K+1], num_sampled [R],
    num_rejected [R]), as greedy_verify returns them.

    logits [>= R*(K+1), ld], bf16 or fp32, holds the S shards side by side (ld
    >= vocab); request r owns rows r*(K+1) .. r*(K+1)+K.  draft_ids: int32
    [R][K], K >= 0; -1 where a request has fewer drafts.  draft_probs: the
    distributions q that the drafts were drawn from, [R*K, >= vocab], fp32 or
    bf16, or None for drafts that no model drew.  temperature: float32 [R]
    (None: 1); 0 makes a request greedy.

    Draft j is accepted iff accept_uniforms[r][j] * q_j(draft) < p_j(draft)
    (float32 [R][K] in [0, 1)).  The first position that is not draws from
    max(p - q, 0), position K from p: the least column whose running sum passes
    sample_uniforms[r] of the total (float64 [R] in [0, 1): float32 has too few
    digits for the columns of a vocabulary).  workspace: optional device tensor
    of at least sampled_verify_workspace() bytes."""
    n, cols, ld, code = _whole_rows(logits, vocab)
    dev = logits.device
    if draft_ids.dim() != 2:
        raise ValueError("draft_ids must be [requests][drafts]")
    r, k = draft_ids.shape
    if n < r * (k + 1):
        raise ValueError(f"logits has {n} rows, need {r * (k + 1)}")
    ids = _array(draft_ids, "draft_ids", torch.int32, (r, k), dev)
    accept = _array(accept_uniforms, "accept_uniforms", torch.float32, (r, k), dev)
    sample = _array(sample_uniforms, "sample_uniforms", torch.float64, (r,), dev)
    temp = None if temperature is None else _array(temperature, "temperature", torch.float32,
                                                   (r,), dev)
    q, q_code, ldq = None, VPA_F32, 0
    if draft_probs is not None and k:
        qn, q_cols, ldq, q_code = _rows_of(draft_probs, "draft_probs")
        if draft_probs.device != dev:
            raise ValueError(f"draft_probs is on {draft_probs.device}, logits on {dev}")
        if qn != r * k or q_cols < vocab:
            raise ValueError(f"draft_probs has shape {(qn, q_cols)}, expected {r * k} rows of at "
                             f"least {vocab} columns")
        q = draft_probs.data_ptr()
    fn = draft_call().vpa_sampled_verify
    per = r * (k + 1)
    words = (per + 2 * r + 63) // 64 * 64
    if workspace is None:
        # one allocation: the workspace after the outputs, at 256 bytes
        need = sampled_verify_workspace(vocab, shard_width, n_shards, r, k)
        buf = torch.empty(words + (need + 3) // 4, dtype=torch.int32, device=dev)
        ws = buf.data_ptr() + 4 * words
    else:
        _, ws, need = _workspace(workspace, 0, dev)
        buf = torch.empty(words, dtype=torch.int32, device=dev)
    base = buf.data_ptr()
    _launch(fn, stream, dev, logits.data_ptr(), code, ld, vocab, shard_width, n_shards, r, k,
            ids if k else None, q, q_code, ldq, accept if k else None, sample, temp, ws, need, base,
            base + 4 * per, base + 4 * (per + r))
    return (buf.as_strided((r, k + 1), (k + 1, 1), 0), buf.as_strided((r,), (1,), per),
            buf.as_strided((r,), (1,), per + r))


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def _teacher(ids, logprobs, n, device):
    """The teacher's ids int32 [N, k] and log probabilities float32 [N, k]
    -> (addresses, k)."""
    if ids.dim() != 2:
        raise ValueError("teacher_ids must be [rows][tokens]")
    shape = (n, ids.shape[1])
    return (_array(ids, "teacher_ids", torch.int32, shape, device),
            _array(logprobs, "teacher_logprobs", torch.float32, shape, device), shape[1])


def _grad_tensor(out, logits, n, cols, ld):
    """The gradient's tensor -> (tensor, row stride)."""
    if out is None:
        return _new(n, cols, logits.dtype, logits.device), cols
    if out is logits:
        return out, ld
    return out, _matrix(out, "out", logits.device, logits.dtype, n, cols)


@_stream_arg
def distill_loss(logits, vocab, shard_width, n_shards, teacher_ids, teacher_logprobs, tail=False,
                 temperature=1.0, workspace=None, *, stream=None):
    """Loss of each row of a student's logits against a teacher's top tokens
    -> (loss float32 [N], row_stats float32 [N, DISTILL_STATS] for the backward
    pass).

    logits [N, ld], bf16 or fp32, all shards side by side.  teacher_ids int32
    [N, k] and teacher_logprobs float32 [N, k], k <= MAX_TEACHER_TOP, are what
    token_logprobs gives as top_ids and top_logprobs; -1 names nothing, and a
    row that names nothing has loss 0.  With q = softmax(logits / temperature)
    the loss is sum p (log p - log q), p the teacher's probabilities made to
    sum to 1 over its tokens; with `tail` p is as given and what it leaves of 1
    is compared with q's sum over all other columns.

    The temperature is the student's alone.  To soften the teacher by it too,
    give token_logprobs of its logits / temperature (without a tail
    teacher_logprobs / temperature says the same)."""
    n, _, ld, code = _whole_rows(logits, vocab)
    dev = logits.device
    ids, lp, k = _teacher(teacher_ids, teacher_logprobs, n, dev)
    fn = draft_call().vpa_distill_loss
    _ws, ws, ws_bytes = _workspace(workspace, _distill_workspace(vocab, shard_width, n_shards, n),
                                   dev)
    buf = torch.empty(n * (1 + DISTILL_STATS), dtype=torch.float32, device=dev)
    base = buf.data_ptr()
    _launch(fn, stream, dev, logits.data_ptr(), code, ld, vocab, shard_width, n_shards, n, ids, lp,
            k, 1 if tail else 0, temperature, ws, ws_bytes, base + 4 * DISTILL_STATS * n, base)
    return (buf.as_strided((n,), (1,), DISTILL_STATS * n),
            buf.as_strided((n, DISTILL_STATS), (DISTILL_STATS, 1), 0))


def distill_workspace(vocab, shard_width, n_shards, n_rows) -> int:
    """Workspace bytes of distill_loss and distill_loss_and_grad."""
    return _distill_workspace(vocab, shard_width, n_shards, n_rows)


@_stream_arg
def distill_loss_backward(logits, vocab, shard_width, n_shards, teacher_ids, teacher_logprobs,
                          row_stats, grad_loss, temperature=1.0, out=None, *, stream=None):
    """Gradient by the logits, of their type and shape, for the gradient of each
    row's loss (float32 [N]).  row_stats and the other arguments: the forward
    call's (which holds whether there was a tail).  Columns past the vocabulary
    get 0.  out: the gradient's tensor; it may be the logits themselves, which
    are then replaced."""
    n, cols, ld, code = _whole_rows(logits, vocab)
    dev = logits.device
    ids, lp, k = _teacher(teacher_ids, teacher_logprobs, n, dev)
    stats = _array(row_stats, "row_stats", torch.float32, (n, DISTILL_STATS), dev)
    g = _array(grad_loss, "grad_loss", torch.float32, (n,), dev)
    out, gld = _grad_tensor(out, logits, n, cols, ld)
    _launch(draft_call().vpa_distill_loss_backward, stream, dev, logits.data_ptr(), code, ld, vocab,
            shard_width, n_shards, n, ids, lp, k, temperature, stats, g, out.data_ptr(), gld, cols)
    return out


@_stream_arg
def distill_loss_and_grad(logits, vocab, shard_width, n_shards, teacher_ids, teacher_logprobs,
                          grad_loss, tail=False, temperature=1.0, out=None, workspace=None, *,
                          stream=None):
    """distill_loss and distill_loss_backward at once, for a step that knows the
    rows' weights grad_loss (float32 [N]) beforehand -> (loss, grad_logits)."""
    n, cols, ld, code = _whole_rows(logits, vocab)
    dev = logits.device
    ids, lp, k = _teacher(teacher_ids, teacher_logprobs, n, dev)
    g = _array(grad_loss, "grad_loss", torch.float32, (n,), dev)
    fn = draft_call().vpa_distill_loss_and_grad
    out, gld = _grad_tensor(out, logits, n, cols, ld)
    _ws, ws, ws_bytes = _workspace(workspace, _distill_workspace(vocab, shard_width, n_shards, n),
                                   dev)
    buf = torch.empty(n * (1 + DISTILL_STATS), dtype=torch.float32, device=dev)
    base = buf.data_ptr()
    _launch(fn, stream, dev, logits.data_ptr(), code, ld, vocab, shard_width, n_shards, n, ids, lp,
            k, 1 if tail else 0, temperature, g, ws, ws_bytes, base + 4 * DISTILL_STATS * n, base,
            out.data_ptr(), gld, cols)
    return buf.as_strided((n,), (1,), DISTILL_STATS * n), out


# ---------------------------------------------------------------------------
# root-mean-square norm and 8-bit matrices
# ---------------------------------------------------------------------------

class RmsNorm(NamedTuple):
    """Results of rms_norm: y; summed, x + residual (x itself without one); rstd
    float32 [rows] (None unless asked for)."""
    y: torch.Tensor
    summed: torch.Tensor
    rstd: Optional[torch.Tensor]


class RmsNormFp8(NamedTuple):
    """Results of rms_norm_fp8: y in 8 bits, its scales float32
    [rows, ceil(cols / 128)]; summed as rms_norm's."""
    y: torch.Tensor
    scale: torch.Tensor
    summed: torch.Tensor


def _summed_tensor(x, residual, summed, rows, cols, device):
    """(address of residual, row stride, tensor of the sum, row stride)."""
    if residual is None:
        if summed is not None:
            raise ValueError("summed goes with a residual")
        return None, 0, None, 0
    ldr = _matrix(residual, "residual", device, x.dtype, rows, cols)
    if summed is None:
        return residual.data_ptr(), ldr, _new(rows, cols, x.dtype, device), cols
    return residual.data_ptr(), ldr, summed, _matrix(summed, "summed", device, x.dtype, rows, cols)


def _fp8_rows(rows, cols, device):
    """A new 8-bit matrix whose rows begin at multiples of 16 bytes -> (tensor, row stride)."""
    ld = (cols + 15) // 16 * 16
    if ld == cols:
        return _new(rows, cols, FP8, device), ld
    return _new(rows, ld, FP8, device).as_strided((rows, cols), (ld, 1)), ld


@_stream_arg
def rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, summed=None, with_rstd=False, *,
             stream=None):
    """y = s / sqrt(mean of s^2 + eps) * weight over each row of s = x + residual
    (rounded to x's dtype) -> RmsNorm(y, summed, rstd).  x, residual [rows,
    cols], bf16 or fp32; weight [cols]: x's dtype or float32.  out: y's tensor,
    which may be x or residual.  summed: the sum's tensor, which may be x or
    residual too (not out)."""
    rows, cols, ldx, code = _rows_of(x, "x")
    dev, dtype = x.device, x.dtype
    wdt = _norm_weight(weight, "weight", dtype, dev, None, cols)
    res, ldr, s, lds = _summed_tensor(x, residual, summed, rows, cols, dev)
    if out is None:
        out = _new(rows, cols, dtype, dev)
        ldy = cols
    else:
        ldy = _matrix(out, "out", dev, dtype, rows, cols)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if with_rstd else None
    _launch(draft_call().vpa_rms_norm, stream, dev, x.data_ptr(), ldx, code, res, ldr, _vp(weight),
            VPA_F32 if wdt is torch.float32 else code, rows, cols, eps, _vp(s), lds,
            out.data_ptr(), ldy, _vp(rstd))
    return RmsNorm(out, x if s is None else s, rstd)


@_stream_arg
def rms_norm_fp8(x, weight=None, residual=None, eps=1e-6, summed=None, *, stream=None):
    """rms_norm with y in 8 bits, as head_linear_fp8 takes it -> RmsNormFp8(y,
    scale, summed).  Each block of 128 columns of a row has the scale amax /
    448, amax its largest |y|, and y / scale is rounded to nearest even."""
    rows, cols, ldx, code = _rows_of(x, "x")
    dev, dtype = x.device, x.dtype
    wdt = _norm_weight(weight, "weight", dtype, dev, None, cols)
    res, ldr, s, lds = _summed_tensor(x, residual, summed, rows, cols, dev)
    y, ldy = _fp8_rows(rows, cols, dev)
    blocks = (cols + SCALE_BLOCK - 1) // SCALE_BLOCK
    scale = _new(rows, blocks, torch.float32, dev)
    _launch(draft_call().vpa_rms_norm_fp8, stream, dev, x.data_ptr(), ldx, code, res, ldr,
            _vp(weight), VPA_F32 if wdt is torch.float32 else code, rows, cols, eps, _vp(s), lds,
            y.data_ptr(), ldy, scale.data_ptr(), blocks)
    return RmsNormFp8(y, scale, x if s is None else s)


@_stream_arg
def rms_norm_backward(grad, summed, rstd, weight=None, grad_summed=None, need_x=True,
                      need_weight=True, out=None, workspace=None, *, stream=None):
    """(grad_x, grad_weight) of rms_norm for the gradient of y, each None where
    not needed.  summed and rstd: the forward call's.  grad_summed: the gradient
    that comes back along the residual, added to grad_x; grad_x is the gradient
    of x and of the residual.  grad_weight has weight's dtype (x's where weight
    is None).  out: grad_x's tensor, which may be grad_summed, or grad where
    grad_weight is not needed."""
    rows, cols, ldg, code = _rows_of(grad, "grad")
    dev, dt = grad.device, grad.dtype
    lds = _matrix(summed, "summed", dev, dt, rows, cols)
    wdt = _norm_weight(weight, "weight", dt, dev, None, cols) or dt
    _out_tensor(rstd, "rstd", torch.float32, rows, dev)
    ldgs = 0 if grad_summed is None else _matrix(grad_summed, "grad_summed", dev, dt, rows, cols)
    if out is not None and not need_x:
        raise ValueError("out is grad_x's tensor: it goes with need_x")
    gx, ldgx = None, 0
    if need_x:
        gx, ldgx = ((_new(rows, cols, dt, dev), cols) if out is None
                    else (out, _matrix(out, "out", dev, dt, rows, cols)))
    gw = torch.empty(cols, dtype=wdt, device=dev) if need_weight else None
    fn = draft_call().vpa_rms_norm_backward
    _ws, ws, ws_bytes = _workspace(workspace, _rms_grad_workspace(rows, cols) if need_weight else 0,
                                   dev)
    _launch(fn, stream, dev, grad.data_ptr(), ldg, summed.data_ptr(), lds, code, _vp(weight),
            VPA_F32 if wdt is torch.float32 else code, rstd.data_ptr(), _vp(grad_summed), ldgs,
            rows, cols, _vp(gx), ldgx, _vp(gw), ws, ws_bytes)
    return gx, gw


@_stream_arg
def quantize_fp8(x, block_rows=1, *, stream=None):
    """A bf16 or fp32 matrix [rows, cols] in 8 bits -> (e4m3 [rows, cols], scales
    float32 [ceil(rows / block_rows), ceil(cols / 128)]).  block_rows: 1 for
    activations, 128 for weights.  A block's scale is amax / 448."""
    rows, cols, ldx, code = _rows_of(x, "x")
    if block_rows not in (1, SCALE_BLOCK):
        raise ValueError(f"block_rows must be 1 or {SCALE_BLOCK}, not {block_rows}")
    dev = x.device
    y, ldy = _fp8_rows(rows, cols, dev)
    blocks = (cols + SCALE_BLOCK - 1) // SCALE_BLOCK
    scale = _new((rows + block_rows - 1) // block_rows, blocks, torch.float32, dev)
    _launch(draft_call().vpa_quantize_fp8, stream, dev, x.data_ptr(), ldx, code, rows, cols,
            block_rows, y.data_ptr(), ldy, scale.data_ptr(), blocks)
    return y, scale


def _fp8_operand(t, name, device, rows, cols):
    """An 8-bit operand -> its row stride; rows begin at multiples of 16 bytes."""
    ld = _matrix(t, name, device, FP8, rows, cols)
    if rows <= 1:
        ld = (cols + 15) // 16 * 16      # of one row: never stepped over
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}'s rows must begin at multiples of 16 bytes (quantize_fp8 and "
                         "rms_norm_fp8 lay them out so)")
    return ld


@_stream_arg
def head_linear_fp8(x, x_scale, weight, weight_scale, bias=None, activation="none", residual=None,
                    out=None, out_dtype=None, workspace=None, fast=False, *, stream=None):
    """y = residual + activation(x weight^T + bias) of 8-bit operands -> y [rows,
    outer], bf16 or (out_dtype) float32.  Products are exact and summed in fp32.

    x e4m3 [rows, inner] with x_scale float32 [rows, ceil(inner / 128)], weight
    e4m3 [outer, inner] with weight_scale float32 [ceil(outer / 128),
    ceil(inner / 128)], as rms_norm_fp8 and quantize_fp8 make them.  bias
    [outer] and residual [rows, outer] are bf16.  out may be the residual
    itself, or one shard's columns of a wider logits tensor.

    fast: bf16 results of more than 64 rows come from the matrix cores' 8-bit
    instruction, at up to twice the rate; it cuts in every group of 8 products
    what lies below 2^-13 of the largest, so a sum is off by up to 7 * 2^-13 of
    sum |x w| (random normal operands: 1.4e-5 of the result), which is much
    where large products cancel.  Other results are the same."""
    if not x.is_cuda or x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x and weight must be 2-D device tensors")
    dev = x.device
    rows, inner = x.shape
    outer = weight.shape[0]
    blocks = (inner + SCALE_BLOCK - 1) // SCALE_BLOCK
    ldx = _fp8_operand(x, "x", dev, rows, inner)
    ldw = _fp8_operand(weight, "weight", dev, outer, inner)
    ldxs = _matrix(x_scale, "x_scale", dev, torch.float32, rows, blocks)
    ldws = _matrix(weight_scale, "weight_scale", dev, torch.float32,
                   (outer + SCALE_BLOCK - 1) // SCALE_BLOCK, blocks)
    if bias is not None:
        _out_tensor(bias, "bias", torch.bfloat16, outer, dev)
    ldr = 0 if residual is None else _matrix(residual, "residual", dev, torch.bfloat16, rows, outer)
    if out is None:
        out = _new(rows, outer, out_dtype or torch.bfloat16, dev)
        ldy = outer
    else:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        ldy = _matrix(out, "out", dev, out.dtype, rows, outer)
    if out.dtype is torch.bfloat16:
        code = VPA_BF16
    elif out.dtype is torch.float32:
        code = VPA_F32
    else:
        raise TypeError(f"the output must be bfloat16 or float32, not {out.dtype}")
    calls = draft_call()
    fn = calls.vpa_head_linear_fp8_fast if fast else calls.vpa_head_linear_fp8
    _ws, ws, ws_bytes = _workspace(workspace, _fp8_workspace(rows, outer, inner, bool(fast)), dev)
    _launch(fn, stream, dev, x.data_ptr(), ldx, x_scale.data_ptr(), ldxs, weight.data_ptr(), ldw,
            weight_scale.data_ptr(), ldws, _vp(bias), _vp(residual), ldr, rows, outer, inner,
            _activation(activation), out.data_ptr(), ldy, code, ws, ws_bytes)
    return out
