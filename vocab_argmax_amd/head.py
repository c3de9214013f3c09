"""The language-model head's operators: layer norm, the head's products and
token log probabilities, each with its backward pass (include/vpa_head.h).

The same thin binding as the package's greedy path, whose names re-export
these: functions check devices, dtypes and strides, allocate outputs with
torch, pass addresses and the current HIP stream, and every step of the
computation runs in libvpa.so's HIP kernels.  Matrices are 2-D with
contiguous columns and any row stride.

The functions take part in no autograd graph: a backward pass is a call of
its own, with the forward call's saved tensors as arguments (see
examples/draft_head.py for a training step).
"""
import ctypes
import functools

import torch

from . import (VPA_BF16, VPA_F32, VPA_OK, Vocab, VpaError, _out_tensor, _raw_stream, _stream_arg,
               _vocab, _vp, last_error, lib)

MAX_TOP = 64             # VPA_MAX_TOP
MAX_ROW_TOKENS = 64      # VPA_MAX_ROW_TOKENS
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}   # vpa_act

# Every symbol include/vpa_head.h declares; the first five are called through
# ctypes alone, the others through the marshalling module too.
HEAD_SYMBOLS = ("vpa_logprobs_workspace", "vpa_logprob_words", "vpa_head_linear_workspace",
                "vpa_head_linear_backward_workspace", "vpa_layer_norm_backward_workspace",
                "vpa_logprob_stats", "vpa_combine_logprobs", "vpa_token_logprobs",
                "vpa_token_logprobs_backward", "vpa_head_linear", "vpa_head_linear_backward",
                "vpa_head_linear_backward_typed", "vpa_head_linear_backward_need",
                "vpa_layer_norm", "vpa_layer_norm_backward")

_bound_to = None
_call_mod = None


def _bind(loaded):
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    dt, f32 = ctypes.c_int, ctypes.c_float
    signatures = {
        "vpa_logprobs_workspace": (sz, [Vocab, i32, i64, i32]),
        "vpa_logprob_words": (i32, [i32, i32]),
        "vpa_head_linear_workspace": (sz, [dt, i64, i64, i64]),
        "vpa_head_linear_backward_workspace": (sz, [dt, i64, i64, i64]),
        "vpa_layer_norm_backward_workspace": (sz, [i64, i64]),
        "vpa_logprob_stats": (dt, [vp, dt, i64, Vocab, i32, i32, i64, vp, i32, i32, vp, sz, vp, vp]),
        "vpa_combine_logprobs": (dt, [vp, Vocab, i64, vp, i32, i32, vp, vp, vp, vp, vp, vp]),
        "vpa_token_logprobs": (dt, [vp, dt, i64, Vocab, i64, vp, i32, i32, vp, sz, vp, vp, vp, vp,
                                    vp, vp]),
        "vpa_token_logprobs_backward": (dt, [vp, dt, i64, Vocab, i32, i32, i64, vp, i32, vp, vp,
                                             vp, vp, i64, i64, vp]),
        "vpa_head_linear": (dt, [vp, i64, vp, i64, vp, vp, i64, dt, i64, i64, i64, i32, vp, i64,
                                 dt, vp, i64, vp, sz, vp]),
        "vpa_head_linear_backward": (dt, [vp, i64, vp, i64, vp, i64, vp, i64, dt, i64, i64, i64,
                                          i32, vp, i64, vp, i64, vp, vp, sz, vp]),
        "vpa_head_linear_backward_typed": (dt, [vp, i64, dt, vp, i64, vp, i64, vp, i64, dt, i64,
                                                i64, i64, i32, vp, i64, vp, i64, vp, vp, sz, vp]),
        "vpa_head_linear_backward_need": (sz, [dt, i64, i64, i64, i32, i32, i32, i32]),
        "vpa_layer_norm": (dt, [vp, i64, dt, vp, vp, dt, i64, i64, f32, vp, i64, vp, vp, vp]),
        "vpa_layer_norm_backward": (dt, [vp, i64, vp, i64, dt, vp, dt, vp, vp, i64, i64, vp, i64,
                                         vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in signatures.items():
        fn = getattr(loaded, name)
        fn.restype, fn.argtypes = res, args


def head_lib():
    """The loaded libvpa.so with the head operators' signatures set."""
    global _bound_to, _call_mod
    loaded = lib()
    if _bound_to is not loaded:
        _bind(loaded)
        try:
            from . import _vpa_head_call
        except ImportError as e:
            raise RuntimeError("vocab_argmax_amd/_vpa_head_call is missing: build it with "
                               f"`python -m vocab_argmax_amd._build` ({e})") from None
        for name in _vpa_head_call.entries():
            _vpa_head_call.bind(name, ctypes.cast(getattr(loaded, name), ctypes.c_void_p).value)
        for fn in (_logprobs_workspace, _linear_workspace, _linear_grad_workspace,
                   _linear_grad_need, _norm_grad_workspace):
            fn.cache_clear()
        _call_mod, _bound_to = _vpa_head_call, loaded
    return loaded


def head_call():
    """The launch entry points of include/vpa_head.h, bound to the loaded
    libvpa.so (csrc/headcall.c); they take their C arguments in order."""
    if _bound_to is None or _bound_to is not lib():
        head_lib()
    return _call_mod


@functools.lru_cache(maxsize=256)
def _logprobs_workspace(vocab, width, shards, n_local, rows, n_top):
    return int(head_lib().vpa_logprobs_workspace(_vocab(vocab, width, shards), n_local, rows,
                                                 n_top))


@functools.lru_cache(maxsize=256)
def _linear_workspace(code, rows, outer, inner):
    return int(head_lib().vpa_head_linear_workspace(code, rows, outer, inner))


@functools.lru_cache(maxsize=256)
def _linear_grad_workspace(code, rows, outer, inner):
    return int(head_lib().vpa_head_linear_backward_workspace(code, rows, outer, inner))


@functools.lru_cache(maxsize=256)
def _linear_grad_need(code, rows, outer, inner, dz, need_x, need_weight, need_bias):
    return int(head_lib().vpa_head_linear_backward_need(code, rows, outer, inner, dz, need_x,
                                                        need_weight, need_bias))


@functools.lru_cache(maxsize=256)
def _norm_grad_workspace(rows, cols):
    return int(head_lib().vpa_layer_norm_backward_workspace(rows, cols))


# The checks below are on the path of calls that take a few microseconds on the
# GPU, so each attribute of a tensor is read once and views are made when they
# are asked for.

def _workspace(workspace, need, device):
    """A caller's workspace (a contiguous device tensor) or a new one of
    `need` bytes, None if that is 0 -> (tensor kept alive, address, bytes)."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _matrix(t, name, device, dtype, rows, cols):
    """A 2-D operand with contiguous columns -> its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {(rows, cols)}")
    stride = t.stride()
    if cols > 1 and stride[1] != 1:
        raise ValueError(f"{name}'s columns must be contiguous (stride 1)")
    return stride[0] if rows > 1 else cols


def _rows_of(t, name):
    """The 2-D first operand of a call -> (rows, cols, row stride, dtype code)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    dtype = t.dtype
    if dtype is torch.bfloat16:
        code = VPA_BF16
    elif dtype is torch.float32:
        code = VPA_F32
    else:
        raise TypeError(f"{name} must be bfloat16 or float32, not {dtype}")
    rows, cols = shape
    stride = t.stride()
    if cols > 1 and stride[1] != 1:
        raise ValueError(f"{name}'s columns must be contiguous (stride 1)")
    return rows, cols, stride[0] if rows > 1 else cols, code


def _columns(cols, vocab, shard_width, first_shard, n_local):
    """Refuses logits narrower than what the shards hold of the vocabulary
    (their row stride may be wide enough, and the last row not)."""
    need = min(n_local * shard_width, vocab - first_shard * shard_width)
    if cols < need:
        raise ValueError(f"logits has {cols} columns, the shards hold {need}")


def _launch(fn, stream, device, *args):
    """Calls the entry point with `device` current, on the given stream or the
    device's current one, and raises what it reports."""
    index = device.index
    if stream is None:
        handle = _raw_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    else:
        handle = stream.cuda_stream
    if index is None or torch._C._cuda_getDevice() == index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != VPA_OK:
        raise VpaError(status, last_error())


# ---------------------------------------------------------------------------
# token log probabilities
# ---------------------------------------------------------------------------

class TokenLogprobs:
    """Results of token_logprobs / combine_logprobs for N rows, as views of one
    allocation that are made when first asked for:

    logprobs      float32, the shape of token_ids (None without tokens)
    lse           float32 [N]: log sum exp of the row
    entropy       float32 [N], in nats (a column of row_stats)
    top_ids       int32 [N, n_top] (None for n_top = 0)
    top_logprobs  float32 [N, n_top] (None for n_top = 0)
    row_stats     float32 [N, 3], what the backward pass takes: a logit near the
                  maximum, the log of the sum scaled by it, the entropy
    """
    __slots__ = ("_buf", "_n", "_tokens", "_top", "_made")

    def __init__(self, buf, n, token_shape, n_top):
        self._buf, self._n, self._tokens, self._top, self._made = buf, n, token_shape, n_top, {}

    def _view(self, name, shape, strides, at, dtype=None):
        v = self._made.get(name)
        if v is None:
            v = (self._buf if dtype is None else self._buf.view(dtype)).as_strided(
                shape, strides, at)
            self._made[name] = v
        return v

    # the buffer: row_stats, lse, logprobs, top_ids, top_logprobs
    @property
    def row_stats(self):
        return self._view("row_stats", (self._n, 3), (3, 1), 0)

    @property
    def entropy(self):
        return self._view("entropy", (self._n,), (3,), 2)

    @property
    def lse(self):
        return self._view("lse", (self._n,), (1,), 3 * self._n)

    @property
    def logprobs(self):
        shape = self._tokens
        if shape is None:
            return None
        return self._view("logprobs", shape, (1,) if len(shape) == 1 else (shape[1], 1),
                          4 * self._n)

    def _tops_at(self):
        shape = self._tokens
        count = 0 if shape is None else 1 if len(shape) == 1 else shape[1]
        return (4 + count) * self._n

    @property
    def top_ids(self):
        return self._view("top_ids", (self._n, self._top), (self._top, 1), self._tops_at(),
                          torch.int32) if self._top else None

    @property
    def top_logprobs(self):
        return self._view("top_logprobs", (self._n, self._top), (self._top, 1),
                          self._tops_at() + self._n * self._top) if self._top else None


def _tokens(token_ids, n, device):
    """token_ids int32 [N] or [N, T] -> (T, shape): (0, None) for None or T = 0."""
    if token_ids is None:
        return 0, None
    if token_ids.dtype is not torch.int32 or not token_ids.is_contiguous():
        raise ValueError("token_ids must be a contiguous int32 tensor")
    if token_ids.device != device:
        raise ValueError(f"token_ids is on {token_ids.device}, logits on {device}")
    shape = token_ids.shape
    if len(shape) not in (1, 2) or shape[0] != n:
        raise ValueError(f"token_ids has shape {tuple(shape)}, expected ({n},) or ({n}, tokens)")
    count = 1 if len(shape) == 1 else shape[1]
    return count, shape if count else None


def _output_addresses(base, n, n_tokens, n_top):
    """logprobs, lse, row_stats, top_ids, top_logprobs in a buffer at `base`."""
    tops = base + 4 * n * (4 + n_tokens)
    return (base + 16 * n if n_tokens else None, base + 12 * n, base, tops if n_top else None,
            tops + 4 * n * n_top if n_top else None)


@_stream_arg
def token_logprobs(logits, vocab, shard_width, n_shards, token_ids=None, n_top=0,
                   workspace=None, *, stream=None):
    """Log probabilities of given tokens, entropy and the n_top most likely
    tokens of each row, over all shards -> TokenLogprobs.

    logits [N, ld], bf16 or fp32, holds the S shards side by side (ld >=
    vocab).  token_ids: int32 [N] or [N, T], T <= MAX_ROW_TOKENS; -1 is a
    placeholder with log probability 0, another id outside the vocabulary
    gives NaN.  Alternatives come by value, the lower id first among equals.
    Masked columns hold -inf.  workspace: optional device tensor of at least
    logprobs_workspace() bytes."""
    n, cols, ld, code = _rows_of(logits, "logits")
    if cols < vocab:
        raise ValueError(f"logits has {cols} columns, the vocabulary {vocab}")
    dev = logits.device
    n_tokens, shape = _tokens(token_ids, n, dev)
    fn = head_call().vpa_token_logprobs
    words = n * (4 + n_tokens + 2 * max(n_top, 0))
    if workspace is None:
        # one allocation: the workspace after the outputs, at 256 bytes
        need = _logprobs_workspace(vocab, shard_width, n_shards, n_shards, n, n_top)
        words = (words + 63) // 64 * 64
        buf = torch.empty(words + need // 4, dtype=torch.float32, device=dev)
        base = buf.data_ptr()
        ws = base + 4 * words
    else:
        _, ws, need = _workspace(workspace, 0, dev)
        buf = torch.empty(words, dtype=torch.float32, device=dev)
        base = buf.data_ptr()
    _launch(fn, stream, dev, logits.data_ptr(), code, ld, vocab, shard_width, n_shards, n,
            token_ids.data_ptr() if n_tokens else None, n_tokens, n_top, ws, need,
            *_output_addresses(base, n, n_tokens, n_top))
    return TokenLogprobs(buf, n, shape, n_top)


def logprobs_workspace(vocab, shard_width, n_shards, n_rows, n_top=0, n_local=None) -> int:
    """Workspace bytes of token_logprobs (n_local None) or logprob_stats."""
    return _logprobs_workspace(vocab, shard_width, n_shards,
                               n_shards if n_local is None else n_local, n_rows, n_top)


@_stream_arg
def logprob_stats(logits, vocab, shard_width, n_shards, token_ids=None, n_top=0, first_shard=0,
                  n_local=None, workspace=None, *, stream=None):
    """Records of shards first_shard..first_shard+n_local-1 for a job whose
    ranks hold one shard each: int32 [n_local][N][words].  Gathered in rank
    order along dim 0 they go to combine_logprobs.  logits [N, ld]: column 0
    is global column first_shard * W; token_ids are global."""
    n, cols, ld, code = _rows_of(logits, "logits")
    dev = logits.device
    if n_local is None:
        n_local = n_shards - first_shard
    _columns(cols, vocab, shard_width, first_shard, n_local)
    n_tokens, _ = _tokens(token_ids, n, dev)
    words = head_lib().vpa_logprob_words(n_tokens, n_top)
    if words < 0:
        raise ValueError(f"at most {MAX_ROW_TOKENS} tokens and {MAX_TOP} alternatives a row")
    _ws, ws, ws_bytes = _workspace(workspace, _logprobs_workspace(vocab, shard_width, n_shards,
                                                                  n_local, n, n_top), dev)
    out = torch.empty((max(n_local, 0), n, words), dtype=torch.int32, device=dev)
    _launch(head_call().vpa_logprob_stats, stream, dev, logits.data_ptr(), code, ld, vocab,
            shard_width, n_shards, first_shard, n_local, n,
            token_ids.data_ptr() if n_tokens else None, n_tokens, n_top, ws, ws_bytes,
            out.data_ptr())
    return out


@_stream_arg
def combine_logprobs(stats, vocab, shard_width, token_ids=None, n_top=0, *, stream=None):
    """All shards' records int32 [S][N][words] -> TokenLogprobs."""
    if stats.dtype is not torch.int32 or stats.dim() != 3 or not stats.is_contiguous():
        raise ValueError("stats must be a contiguous int32 [shards][rows][words] tensor")
    if not stats.is_cuda:
        raise ValueError("stats must be a device tensor")
    s, n, words = stats.shape
    dev = stats.device
    n_tokens, shape = _tokens(token_ids, n, dev)
    if words != head_lib().vpa_logprob_words(n_tokens, n_top):
        raise ValueError(f"records of {words} words do not hold {n_tokens} tokens and {n_top} "
                         "alternatives")
    buf = torch.empty(n * (4 + n_tokens + 2 * n_top), dtype=torch.float32, device=dev)
    _launch(head_call().vpa_combine_logprobs, stream, dev, stats.data_ptr(), vocab, shard_width, s,
            n, token_ids.data_ptr() if n_tokens else None, n_tokens, n_top,
            *_output_addresses(buf.data_ptr(), n, n_tokens, n_top))
    return TokenLogprobs(buf, n, shape, n_top)


@_stream_arg
def token_logprobs_backward(logits, vocab, shard_width, n_shards, token_ids, row_stats,
                            grad_logprobs, grad_entropy=None, first_shard=0, n_local=None,
                            out=None, *, stream=None):
    """Gradient by the logits, of their type and shape, for the gradients of
    logprobs (float32, the shape of token_ids) and, optionally, of the
    entropy (float32 [N]).  row_stats: the forward call's.  Columns past the
    vocabulary get 0.  out: the gradient's tensor; it may be the logits
    themselves, which are then replaced."""
    n, cols, ld, code = _rows_of(logits, "logits")
    dev = logits.device
    if n_local is None:
        n_local = n_shards - first_shard
    _columns(cols, vocab, shard_width, first_shard, n_local)
    n_tokens, _ = _tokens(token_ids, n, dev)
    if (grad_logprobs is None) != (token_ids is None):
        raise ValueError("grad_logprobs goes with token_ids")
    for name, t, count in (("grad_logprobs", grad_logprobs, n * n_tokens),
                           ("grad_entropy", grad_entropy, n), ("row_stats", row_stats, 3 * n)):
        if t is not None:
            _out_tensor(t, name, torch.float32, count, dev)
    if out is None:
        out = torch.empty((n, cols), dtype=logits.dtype, device=dev)
        gld = cols
    else:
        gld = _matrix(out, "out", dev, logits.dtype, n, cols)
    _launch(head_call().vpa_token_logprobs_backward, stream, dev, logits.data_ptr(), code, ld,
            vocab, shard_width, n_shards, first_shard, n_local, n,
            token_ids.data_ptr() if n_tokens else None, n_tokens, row_stats.data_ptr(),
            grad_logprobs.data_ptr() if n_tokens else None, _vp(grad_entropy), out.data_ptr(), gld,
            cols)
    return out


# ---------------------------------------------------------------------------
# the head's products
# ---------------------------------------------------------------------------

def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {name!r}") \
            from None


@_stream_arg
def head_linear(x, weight, bias=None, activation="none", residual=None, out=None, out_dtype=None,
                with_pre=False, workspace=None, *, stream=None):
    """y = residual + activation(x weight^T + bias) -> y [rows, outer], or
    (y, pre) with_pre, pre = x weight^T + bias for the backward pass.

    x [rows, inner], weight [outer, inner], bias [outer], residual [rows,
    outer], all of x's dtype (bf16 or fp32).  activation: "none", "relu",
    "gelu" (erf) or "silu".  out / out_dtype: y's tensor or type (x's dtype or
    float32); out may be the residual itself, or one shard's columns of a
    wider logits tensor."""
    rows, inner, ldx, code = _rows_of(x, "x")
    dev, dtype = x.device, x.dtype
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D [outer, inner]")
    outer = weight.shape[0]
    ldw = _matrix(weight, "weight", dev, dtype, outer, inner)
    if bias is not None:
        _out_tensor(bias, "bias", dtype, outer, dev)
    ldr = 0 if residual is None else _matrix(residual, "residual", dev, dtype, rows, outer)
    if out is None:
        out = torch.empty((rows, outer), dtype=out_dtype or dtype, device=dev)
        ldy = outer
    else:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        ldy = _matrix(out, "out", dev, out.dtype, rows, outer)
    out_type = out.dtype
    if out_type is dtype:
        out_code = code
    elif out_type is torch.float32:
        out_code = VPA_F32
    else:
        raise TypeError(f"the output must be {dtype} or float32, not {out_type}")
    pre = torch.empty((rows, outer), dtype=dtype, device=dev) if with_pre else None
    fn = head_call().vpa_head_linear
    _ws, ws, ws_bytes = _workspace(workspace, _linear_workspace(code, rows, outer, inner), dev)
    _launch(fn, stream, dev, x.data_ptr(), ldx, weight.data_ptr(), ldw, _vp(bias), _vp(residual),
            ldr, code, rows, outer, inner, _activation(activation), out.data_ptr(), ldy, out_code,
            _vp(pre), outer, ws, ws_bytes)
    return (out, pre) if with_pre else out


@_stream_arg
def head_linear_backward(grad, x, weight, pre=None, activation="none", need_x=True,
                         need_weight=True, need_bias=True, workspace=None, *, stream=None):
    """(grad_x, grad_weight, grad_bias) of head_linear for the gradient of y
    [rows, outer], each None where not needed; the residual's gradient is
    `grad` itself.  grad has y's dtype: x's, or float32 (fp32 logits of bf16
    operands); the results have x's.  pre: head_linear's, required with an
    activation."""
    rows, outer, ldg, grad_code = _rows_of(grad, "grad")
    dev, dt = grad.device, x.dtype
    act = _activation(activation)
    if dt is grad.dtype:
        code = grad_code
    elif dt is torch.bfloat16:
        code = VPA_BF16
    else:
        raise TypeError(f"x must be {grad.dtype}, not {dt}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, inner]")
    inner = x.shape[1]
    ldx = _matrix(x, "x", dev, dt, rows, inner)
    ldw = _matrix(weight, "weight", dev, dt, outer, inner)
    if act and pre is None:
        raise ValueError(f"the backward pass of {activation} needs pre")
    ldp = _matrix(pre, "pre", dev, dt, rows, outer) if act else 0
    gx = torch.empty((rows, inner), dtype=dt, device=dev) if need_x else None
    gw = torch.empty((outer, inner), dtype=dt, device=dev) if need_weight else None
    gb = torch.empty(outer, dtype=dt, device=dev) if need_bias else None
    fn = head_call().vpa_head_linear_backward_typed
    at = grad.data_ptr()
    # the products read an aligned gradient itself: no place for dz then
    dz = bool(act or code != grad_code or at % 16 or ldg % (4 if code == VPA_F32 else 8))
    _ws, ws, ws_bytes = _workspace(workspace, _linear_grad_need(code, rows, outer, inner, dz,
                                                                bool(need_x), bool(need_weight),
                                                                bool(need_bias)),
                                   dev)
    _launch(fn, stream, dev, at, ldg, grad_code, x.data_ptr(), ldx, weight.data_ptr(),
            ldw, _vp(pre) if act else None, ldp, code, rows, outer, inner, act, _vp(gx), inner,
            _vp(gw), inner, _vp(gb), ws, ws_bytes)
    return gx, gw, gb


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def _norm_weight(t, name, dtype, device, wdtype, cols):
    """Checks weight or bias -> its dtype (wdtype, the other's, for None)."""
    if t is None:
        return wdtype
    td = t.dtype
    if td is not dtype and td is not torch.float32:
        raise TypeError(f"{name} must be {dtype} or float32, not {td}")
    if wdtype is not None and td is not wdtype:
        raise TypeError(f"weight and bias must have one dtype, not {wdtype} and {td}")
    _out_tensor(t, name, td, cols, device)
    return td


@_stream_arg
def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, with_stats=False, *, stream=None):
    """y = (x - mean) / sqrt(variance + eps) * weight + bias over each row of
    x [rows, cols] -> y, or (y, mean, rstd) with_stats (float32 [rows], for
    the backward pass).  weight, bias [cols]: x's dtype or float32.  out may
    be x itself."""
    rows, cols, ldx, code = _rows_of(x, "x")
    dev, dtype = x.device, x.dtype
    wdt = _norm_weight(bias, "bias", dtype, dev,
                       _norm_weight(weight, "weight", dtype, dev, None, cols), cols)
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
        ldy = cols
    else:
        ldy = _matrix(out, "out", dev, dtype, rows, cols)
    mean = rstd = None
    if with_stats:
        mean = torch.empty(rows, dtype=torch.float32, device=dev)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    _launch(head_call().vpa_layer_norm, stream, dev, x.data_ptr(), ldx, code, _vp(weight),
            _vp(bias), VPA_F32 if wdt is torch.float32 else code, rows, cols, eps, out.data_ptr(),
            ldy, _vp(mean), _vp(rstd))
    return (out, mean, rstd) if with_stats else out


@_stream_arg
def layer_norm_backward(grad, x, mean, rstd, weight=None, need_x=True, need_weight=True,
                        need_bias=True, workspace=None, *, stream=None):
    """(grad_x, grad_weight, grad_bias) of layer_norm for the gradient of y,
    each None where not needed.  mean, rstd: the forward call's.  grad_weight
    and grad_bias have weight's dtype (x's where weight is None)."""
    rows, cols, ldg, code = _rows_of(grad, "grad")
    dev, dt = grad.device, grad.dtype
    ldx = _matrix(x, "x", dev, dt, rows, cols)
    wdt = _norm_weight(weight, "weight", dt, dev, None, cols) or dt
    _out_tensor(mean, "mean", torch.float32, rows, dev)
    _out_tensor(rstd, "rstd", torch.float32, rows, dev)
    gx = torch.empty((rows, cols), dtype=dt, device=dev) if need_x else None
    gw = torch.empty(cols, dtype=wdt, device=dev) if need_weight else None
    gb = torch.empty(cols, dtype=wdt, device=dev) if need_bias else None
    fn = head_call().vpa_layer_norm_backward
    need = _norm_grad_workspace(rows, cols) if need_weight or need_bias else 0
    _ws, ws, ws_bytes = _workspace(workspace, need, dev)
    _launch(fn, stream, dev, grad.data_ptr(), ldg, x.data_ptr(), ldx, code, _vp(weight),
            VPA_F32 if wdt is torch.float32 else code, mean.data_ptr(), rstd.data_ptr(), rows,
            cols, _vp(gx), cols, _vp(gw), _vp(gb), ws, ws_bytes)
    return gx, gw, gb
