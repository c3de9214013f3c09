"""The head operators' C ABI on the CPU (include/vpa_head.h): every declared
symbol is exported, invalid arguments are rejected before any HIP call, empty
batches are no-ops, and the binding refuses what the kernels cannot take.
Pointers passed here are never dereferenced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import vocab_argmax_amd as vpa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "vpa_head.h")
P = 0x7F0000010000          # aligned, never dereferenced
ODD = P + 1
F32, BF16 = vpa.VPA_F32, vpa.VPA_BF16
INVALID, UNSUPPORTED, OK = vpa.VPA_ERR_INVALID, vpa.VPA_ERR_UNSUPPORTED, vpa.VPA_OK
HUGE = 1 << 50


class Calls:
    """Each launch entry point through ctypes and through the marshalling
    module; both must answer alike."""

    def __getattr__(self, name):
        through_ctypes = getattr(vpa.head_lib(), name)
        through_module = getattr(vpa.head_call(), name)

        def both(*args):
            flat = [a for arg in args
                    for a in ([arg.vocab, arg.shard_width, arg.n_shards]
                              if isinstance(arg, vpa.Vocab) else [arg])]
            st = through_ctypes(*args)
            msg = vpa.last_error() if st else ""
            st2 = through_module(*flat)
            assert (st2, vpa.last_error() if st2 else "") == (st, msg), name
            return st
        return both


lib = Calls()


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(vpa_[a-z_]+)\s*\(", text))
    assert names == set(vpa.HEAD_SYMBOLS)
    for name in names:
        assert hasattr(vpa.head_lib(), name)
    assert set(vpa.head_call().entries()) == set(vpa.HEAD_SYMBOLS[5:])


def test_header_is_plain_c_and_cxx(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "vpa_head.h"\nint main(void) { return 0; }\n')
    for cc, std in (("gcc", ["-std=c99"]), ("g++", ["-std=c++11", "-x", "c++"])):
        if not shutil.which(cc):
            pytest.skip(f"{cc} not available")
        subprocess.run([cc, *std, "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.dirname(HEADER), "-fsyntax-only", str(src)], check=True)


def V(v=1000, w=250, s=4):
    return vpa.Vocab(v, w, s)


def logprobs(**kw):
    a = dict(logits=P, dt=BF16, ld=1000, v=V(), n=4, tok=P, t=1, top=5, ws=P, wsb=HUGE, lp=P,
             lse=P, stats=P, ids=P, tops=P)
    a.update(kw)
    return lib.vpa_token_logprobs(a["logits"], a["dt"], a["ld"], a["v"], a["n"], a["tok"], a["t"],
                                  a["top"], a["ws"], a["wsb"], a["lp"], a["lse"], a["stats"],
                                  a["ids"], a["tops"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=9), UNSUPPORTED), (dict(v=V(0)), INVALID), (dict(v=V(1 << 24, 1 << 24, 1)), INVALID),
    (dict(v=V(1001)), INVALID), (dict(ld=999), INVALID), (dict(n=-1), INVALID),
    (dict(n=1 << 31), INVALID), (dict(logits=None), INVALID), (dict(logits=ODD), INVALID),
    (dict(dt=F32, logits=P + 2), INVALID), (dict(t=65), INVALID), (dict(t=-1), INVALID),
    (dict(top=65), INVALID), (dict(top=-1), INVALID), (dict(v=V(3, 3, 1), top=4), INVALID),
    (dict(tok=None), INVALID), (dict(tok=ODD), INVALID), (dict(lp=None), INVALID),
    (dict(t=0), INVALID),                                # log probabilities of no tokens
    (dict(stats=None), INVALID), (dict(stats=ODD), INVALID), (dict(lse=ODD), INVALID),
    (dict(ids=None), INVALID), (dict(tops=None), INVALID), (dict(top=0), INVALID),
    (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID), (dict(wsb=16), INVALID),
    (dict(n=(1 << 31) - 1, v=V(200064, 200064, 1), ld=200064), INVALID),   # beyond one dispatch
    (dict(n=0, logits=None, ws=None, stats=None), OK),
])
def test_token_logprobs_rejects(kw, status):
    assert logprobs(**kw) == status
    assert status == OK or vpa.last_error() != ""


def test_logprob_workspace_and_words():
    need = vpa.head_lib().vpa_logprobs_workspace(V(), 4, 4, 5)
    assert need > 0
    for bad in ((V(0), 1, 4, 5), (V(), 5, 4, 5), (V(), 0, 4, 5), (V(), 4, 0, 5), (V(), 4, -1, 5),
                (V(), 4, 4, 65), (V(), 4, 1 << 31, 5)):
        assert vpa.head_lib().vpa_logprobs_workspace(*bad) == 0
    assert vpa.head_lib().vpa_logprob_words(2, 5) == 15
    assert vpa.head_lib().vpa_logprob_words(65, 0) == -1
    assert vpa.head_lib().vpa_logprob_words(0, -1) == -1


def test_logprob_stats_and_combine_reject():
    def stats(first=0, nloc=1, ld=250, out=P, n=4, t=1, tok=P, ws=P, wsb=HUGE, top=3):
        return lib.vpa_logprob_stats(P, BF16, ld, V(), first, nloc, n, tok, t, top, ws, wsb, out,
                                     None)
    for kw in (dict(first=-1), dict(first=4), dict(nloc=0), dict(first=3, nloc=2), dict(ld=249),
               dict(out=None), dict(out=ODD), dict(tok=None), dict(ws=None), dict(wsb=0),
               dict(n=-2), dict(t=99), dict(top=99)):
        assert stats(**kw) == INVALID, kw
    assert stats(n=0, out=None, ws=None) == OK

    def combine(st=P, n=4, tok=P, t=1, top=3, lp=P, stats=P, ids=P, tops=P, v=None):
        return lib.vpa_combine_logprobs(st, v or V(), n, tok, t, top, lp, None, stats, ids, tops,
                                        None)
    for kw in (dict(st=None), dict(st=ODD), dict(n=-1), dict(tok=None), dict(t=70), dict(top=70),
               dict(lp=None), dict(stats=None), dict(ids=None), dict(tops=ODD),
               dict(n=1 << 27), dict(v=V(1 << 24, 1 << 24, 1))):
        assert combine(**kw) == INVALID, kw
    assert combine(n=0, st=None) == OK


def test_logprobs_backward_rejects():
    def back(x=P, dt=BF16, ld=1000, v=None, first=0, nloc=4, n=4, tok=P, t=1, stats=P, g=P, ge=P,
             out=P + (1 << 30), gld=1000, gcols=1000):
        return lib.vpa_token_logprobs_backward(x, dt, ld, v or V(), first, nloc, n, tok, t, stats,
                                               g, ge, out, gld, gcols, None)
    for kw in (dict(x=None), dict(x=ODD), dict(ld=999), dict(first=2), dict(n=-1), dict(tok=None),
               dict(t=65), dict(stats=None), dict(stats=ODD), dict(g=None), dict(g=ODD),
               dict(ge=ODD), dict(t=0), dict(out=None), dict(out=ODD), dict(gcols=999),
               dict(gld=999), dict(gcols=1 << 31, gld=1 << 31), dict(out=P, gld=1008),
               dict(n=1 << 28)):
        assert back(**kw) == INVALID, kw
    assert back(dt=5) == UNSUPPORTED
    assert back(n=0, x=None) == OK


def linear(**kw):
    a = dict(x=P, ldx=64, w=P, ldw=64, b=P, r=P, ldr=96, dt=BF16, rows=8, outer=96, inner=64,
             act=3, y=P, ldy=96, odt=BF16, pre=None, ldp=0, ws=P, wsb=HUGE)
    a.update(kw)
    return lib.vpa_head_linear(a["x"], a["ldx"], a["w"], a["ldw"], a["b"], a["r"], a["ldr"],
                               a["dt"], a["rows"], a["outer"], a["inner"], a["act"], a["y"],
                               a["ldy"], a["odt"], a["pre"], a["ldp"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), UNSUPPORTED), (dict(odt=7), UNSUPPORTED), (dict(act=4), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(dt=F32), UNSUPPORTED),          # bf16 from fp32 operands
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(outer=0), INVALID),
    (dict(inner=0), INVALID), (dict(outer=1 << 31), INVALID), (dict(x=None), INVALID),
    (dict(x=ODD), INVALID), (dict(w=None), INVALID), (dict(w=ODD), INVALID),
    (dict(b=ODD), INVALID), (dict(r=ODD), INVALID), (dict(y=None), INVALID),
    (dict(y=ODD), INVALID), (dict(pre=ODD, ldp=96), INVALID), (dict(pre=P, ldp=95), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(ldr=95), INVALID),
    (dict(ldy=95), INVALID), (dict(ldy=104, y=P, r=P), INVALID),       # in place, other stride
    (dict(odt=F32), INVALID),                                          # in place, other type
    (dict(rows=(1 << 31) - 1, outer=(1 << 31) - 1, ldr=1 << 31, ldy=1 << 31), INVALID),
    (dict(rows=0, x=None, w=None, y=None), OK),
])
def test_head_linear_rejects(kw, status):
    assert linear(**kw) == status
    assert status == OK or vpa.last_error() != ""


def test_head_linear_backward_rejects():
    def back(g=P, ldg=96, x=P, ldx=64, w=P, ldw=64, pre=P, ldp=96, dt=BF16, rows=8, outer=96,
             inner=64, act=3, gx=P, ldgx=64, gw=P, ldgw=64, gb=P, ws=P, wsb=HUGE):
        return lib.vpa_head_linear_backward(g, ldg, x, ldx, w, ldw, pre, ldp, dt, rows, outer,
                                            inner, act, gx, ldgx, gw, ldgw, gb, ws, wsb, None)
    for kw in (dict(g=None), dict(g=ODD), dict(ldg=95), dict(x=None), dict(ldx=63), dict(w=None),
               dict(ldw=63), dict(pre=None), dict(ldp=95), dict(rows=-1), dict(outer=0),
               dict(inner=1 << 31), dict(gx=ODD), dict(ldgx=63), dict(gw=ODD), dict(ldgw=63),
               dict(gb=ODD), dict(ws=None), dict(ws=P + 4), dict(wsb=0)):
        assert back(**kw) == INVALID, kw
    assert back(dt=3) == UNSUPPORTED and back(act=9) == UNSUPPORTED
    need = vpa.head_lib().vpa_head_linear_backward_workspace(BF16, 8, 96, 64)
    assert need >= 8 * 96 * 2 and back(wsb=8 * 96) == INVALID
    assert vpa.head_lib().vpa_head_linear_backward_workspace(BF16, -1, 96, 64) == 0
    assert vpa.head_lib().vpa_head_linear_workspace(7, 8, 96, 64) == 0
    # nothing asked for, nothing enqueued
    assert back(rows=0, gx=None, gw=None, gb=None, ws=None) == OK


def test_layer_norm_rejects():
    def norm(x=P, ldx=64, dt=BF16, w=P, b=P, wdt=F32, rows=4, cols=64, eps=1e-5, y=P, ldy=64,
             mean=P, rstd=P):
        return lib.vpa_layer_norm(x, ldx, dt, w, b, wdt, rows, cols, eps, y, ldy, mean, rstd, None)
    for kw in (dict(x=None), dict(x=ODD), dict(ldx=63), dict(w=ODD), dict(b=ODD), dict(rows=-1),
               dict(cols=0), dict(cols=1 << 31), dict(eps=-1e-5), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(y=None), dict(ldy=63), dict(ldy=72), dict(mean=ODD),
               dict(rstd=ODD), dict(rows=(1 << 31) - 1, cols=1 << 20, ldx=1 << 20, ldy=1 << 20)):
        assert norm(**kw) == INVALID, kw
    assert norm(dt=4) == UNSUPPORTED and norm(wdt=4) == UNSUPPORTED
    assert norm(dt=F32, wdt=BF16) == UNSUPPORTED
    assert norm(rows=0, x=None, y=None) == OK

    def back(g=P, ldg=64, x=P, ldx=64, dt=BF16, w=P, wdt=F32, mean=P, rstd=P, rows=4, cols=64,
             gx=P + 4096, ldgx=64, gw=P, gb=P, ws=P, wsb=HUGE):
        return lib.vpa_layer_norm_backward(g, ldg, x, ldx, dt, w, wdt, mean, rstd, rows, cols, gx,
                                           ldgx, gw, gb, ws, wsb, None)
    for kw in (dict(g=None), dict(ldg=63), dict(x=ODD), dict(ldx=63), dict(w=ODD),
               dict(mean=None), dict(rstd=None), dict(rows=-1), dict(cols=0), dict(gx=ODD),
               dict(ldgx=63), dict(gw=ODD), dict(gb=ODD), dict(ws=None), dict(wsb=0),
               dict(gx=P), dict(gx=P, gw=None, gb=None, ldgx=72)):
        assert back(**kw) == INVALID, kw
    assert back(dt=4) == UNSUPPORTED and back(dt=F32, wdt=BF16) == UNSUPPORTED
    assert vpa.head_lib().vpa_layer_norm_backward_workspace(4, 0) == 0
    assert vpa.head_lib().vpa_layer_norm_backward_workspace(-1, 8) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        vpa.token_logprobs(x, 8, 8, 1)
    with pytest.raises(ValueError):
        vpa.layer_norm(x)
    with pytest.raises(ValueError):
        vpa.head_linear(x, x)
    with pytest.raises(ValueError):
        vpa.head_linear_backward(x, x, x)
    with pytest.raises(ValueError):
        vpa.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError):
        vpa.combine_logprobs(torch.zeros(1, 4, 3, dtype=torch.int32), 8, 8)
    with pytest.raises(ValueError):
        vpa.combine_logprobs(torch.zeros(4, 3, dtype=torch.int32), 8, 8)


def test_module_rejects_bad_python_arguments():
    c = vpa.head_call()
    ok = (P, 64, BF16, P, P, F32, 0, 64, 1e-5, P, 64, None, None, None)
    assert c.vpa_layer_norm(*ok) == OK                       # zero rows
    with pytest.raises(TypeError, match="takes 14 arguments"):
        c.vpa_layer_norm(*ok[:-1])
    with pytest.raises(TypeError):
        c.vpa_layer_norm(*ok[:8], "x", *ok[9:])
    with pytest.raises(OverflowError):
        c.vpa_layer_norm(-1, *ok[1:])
    with pytest.raises(KeyError):
        c.bind("vpa_no_such_entry", 0x10000)
