"""The draft operators' C ABI on the CPU (include/vpa_draft.h): every declared
symbol is exported, invalid arguments are rejected before any HIP call, empty
batches are no-ops.  Pointers passed here are never dereferenced."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import vocab_argmax_amd as vpa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "vpa_draft.h")
P = 0x7F0000010000          # aligned, never dereferenced
P2, P3, P4 = P + (1 << 20), P + (2 << 20), P + (3 << 20)
ODD = P + 1
F32, BF16 = vpa.VPA_F32, vpa.VPA_BF16
INVALID, UNSUPPORTED, OK = vpa.VPA_ERR_INVALID, vpa.VPA_ERR_UNSUPPORTED, vpa.VPA_OK
HUGE = 1 << 50


class Calls:
    """Each launch entry point through ctypes and through the marshalling
    module; both must answer alike."""

    def __getattr__(self, name):
        through_ctypes = getattr(vpa.draft_lib(), name)
        through_module = getattr(vpa.draft_call(), name)

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


def V(v=1000, w=250, s=4):
    return vpa.Vocab(v, w, s)


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(vpa_[a-z0-9_]+)\s*\(", text))
    assert names == set(vpa.DRAFT_SYMBOLS)
    for name in names:
        assert hasattr(vpa.draft_lib(), name)
    assert set(vpa.draft_call().entries()) == set(vpa.DRAFT_SYMBOLS[4:])


def test_header_is_plain_c_and_cxx(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "vpa_draft.h"\nint main(void) { return 0; }\n')
    for cc, std in (("gcc", ["-std=c99"]), ("g++", ["-std=c++11", "-x", "c++"])):
        if not shutil.which(cc):
            pytest.skip(f"{cc} not available")
        subprocess.run([cc, *std, "-pedantic", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.dirname(HEADER), "-fsyntax-only", str(src)], check=True)


def refused(status, want):
    assert status == want
    assert want == OK or vpa.last_error() != ""


def sampled(**kw):
    a = dict(x=P, dt=BF16, ld=1000, v=V(), r=4, k=3, ids=P, q=P, qdt=F32, ldq=1000, u=P, s=P, t=P,
             ws=P, wsb=HUGE, out=P, ns=P, nr=P)
    a.update(kw)
    return lib.vpa_sampled_verify(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), UNSUPPORTED), (dict(qdt=7), UNSUPPORTED), (dict(v=V(0)), INVALID),
    (dict(v=V(1001)), INVALID), (dict(v=V(1 << 24, 1 << 24, 1), ld=1 << 24), INVALID),
    (dict(ld=999), INVALID), (dict(ld=(1 << 40) + 1), INVALID), (dict(ldq=999), INVALID),
    (dict(r=-1), INVALID), (dict(r=1 << 31), INVALID), (dict(r=(1 << 31) // 4), INVALID),
    (dict(k=-1), INVALID), (dict(k=4097), INVALID), (dict(k=0), INVALID),   # q of no drafts
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(dt=F32, x=P + 2), INVALID),
    (dict(ids=None), INVALID), (dict(ids=P + 2), INVALID), (dict(q=ODD), INVALID),
    (dict(u=None), INVALID), (dict(u=ODD), INVALID), (dict(s=None), INVALID),
    (dict(s=P + 4), INVALID), (dict(t=ODD), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 8), INVALID), (dict(wsb=8), INVALID), (dict(out=None), INVALID),
    (dict(out=ODD), INVALID), (dict(ns=None), INVALID), (dict(nr=None), INVALID),
    (dict(r=100_000_000, k=20, v=V(200000, 200000, 1), ld=200000, ldq=200000), INVALID),
    (dict(r=0, x=None, ws=None, s=None, out=None), OK),
])
def test_sampled_verify_rejects(kw, status):
    refused(sampled(**kw), status)


def test_workspaces():
    w = vpa.draft_lib().vpa_sampled_verify_workspace
    assert w(V(), 4, 3) > 0 and w(V(), 4, 0) > 0
    for bad in ((V(0), 4, 3), (V(), 0, 3), (V(), -1, 3), (V(), 4, -1), (V(), 4, 4097),
                (V(), 1 << 31, 3), (V(), 1 << 30, 3)):
        assert w(*bad) == 0
    d = vpa.draft_lib().vpa_distill_workspace
    for bad in ((V(0), 4), (V(), 0), (V(), -1), (V(), 1 << 31)):
        assert d(*bad) == 0
    n = vpa.draft_lib().vpa_rms_norm_backward_workspace
    assert n(4, 100) >= 400
    for bad in ((0, 4), (-1, 4), (1 << 31, 4), (4, 0), (4, 1 << 31)):
        assert n(*bad) == 0
    f = vpa.draft_lib().vpa_head_linear_fp8_workspace
    for bad in ((0, 4, 4), (-1, 4, 4), (4, 0, 4), (4, 4, 0), (1 << 31, 4, 4), (4, 1 << 31, 4)):
        assert f(*bad) == 0


def distill(**kw):
    a = dict(x=P, dt=BF16, ld=1000, v=V(), n=4, ids=P, lp=P, k=5, tail=1, t=1.0, ws=P, wsb=HUGE,
             loss=P, st=P)
    a.update(kw)
    return lib.vpa_distill_loss(*a.values(), None)


def backward(**kw):
    a = dict(x=P, dt=BF16, ld=1000, v=V(), n=4, ids=P, lp=P, k=5, t=1.0, st=P, g=P, d=P2,
             gld=1000, gc=1000)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.vpa_distill_loss_backward(*a.values(), None)


def at_once(**kw):
    a = dict(x=P, dt=BF16, ld=1000, v=V(), n=4, ids=P, lp=P, k=5, tail=1, t=1.0, g=P, ws=P,
             wsb=HUGE, loss=P, st=P, d=P2, gld=1000, gc=1000)
    a.update(kw)
    return lib.vpa_distill_loss_and_grad(*a.values(), None)


BOTH = [
    (dict(dt=7), UNSUPPORTED), (dict(v=V(0)), INVALID), (dict(ld=999), INVALID),
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(k=0), INVALID),
    (dict(k=65), INVALID), (dict(t=0.0), INVALID), (dict(t=-1.0), INVALID),
    (dict(t=float("inf")), INVALID), (dict(t=float("nan")), INVALID), (dict(t=1e39), INVALID),
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(ids=None), INVALID),
    (dict(ids=P + 2), INVALID), (dict(lp=None), INVALID), (dict(lp=ODD), INVALID),
    (dict(st=None), INVALID), (dict(st=ODD), INVALID),
    (dict(n=0, x=None, ids=None, lp=None, st=None), OK),
]
LOSS = [(dict(loss=None), INVALID), (dict(loss=ODD), INVALID)]
GRAD = [(dict(g=None), INVALID), (dict(g=ODD), INVALID), (dict(d=None), INVALID),
        (dict(d=ODD), INVALID), (dict(gc=999), INVALID), (dict(gld=999), INVALID),
        (dict(gc=1001), INVALID), (dict(d=P, gld=1008), INVALID)]


@pytest.mark.parametrize("kw,status", BOTH + LOSS)
def test_distill_loss_rejects(kw, status):
    refused(distill(**kw), status)


@pytest.mark.parametrize("kw,status", BOTH + GRAD)
def test_distill_backward_rejects(kw, status):
    refused(backward(**kw), status)


@pytest.mark.parametrize("kw,status", BOTH + LOSS + GRAD)
def test_distill_at_once_rejects(kw, status):
    refused(at_once(**kw), status)


def rms(fp8=False, **kw):
    a = dict(x=P, ldx=300, dt=BF16, r=P2, ldr=300, w=P, wdt=F32, n=4, c=300, eps=1e-6, s=P3,
             lds=300, y=P4, ldy=300)
    a.update({k: v for k, v in kw.items() if k in a})
    rest = [kw.get("sc", P), kw.get("ldsc", 3)] if fp8 else [kw.get("rstd", P)]
    return (lib.vpa_rms_norm_fp8 if fp8 else lib.vpa_rms_norm)(*a.values(), *rest, None)


RMS = [
    (dict(dt=7), UNSUPPORTED), (dict(wdt=7), UNSUPPORTED), (dict(dt=F32, wdt=BF16), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(c=0), INVALID),
    (dict(c=1 << 31), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(x=ODD), INVALID),
    (dict(ldx=299), INVALID), (dict(ldr=299), INVALID), (dict(r=ODD), INVALID),
    (dict(r=None), INVALID), (dict(s=None), INVALID), (dict(s=ODD), INVALID),
    (dict(lds=299), INVALID), (dict(y=None), INVALID), (dict(ldy=299), INVALID),
    (dict(w=P + 2), INVALID), (dict(y=P3), INVALID), (dict(s=P, lds=301), INVALID),
    (dict(s=P2, lds=301), INVALID), (dict(y=P, ldy=301), INVALID), (dict(y=P2, ldy=301), INVALID),
    (dict(n=1 << 30, c=40000, ldx=40000, ldr=40000, lds=40000, ldy=40000, ldsc=400), INVALID),
    (dict(n=0, x=None, y=None, r=None, s=None), OK),
]


@pytest.mark.parametrize("kw,status", RMS + [(dict(rstd=ODD), INVALID), (dict(y=ODD), INVALID)])
def test_rms_norm_rejects(kw, status):
    refused(rms(**kw), status)


@pytest.mark.parametrize("kw,status", RMS + [
    (dict(sc=None), INVALID), (dict(sc=ODD), INVALID), (dict(ldsc=2), INVALID),
    (dict(y=P), INVALID), (dict(y=P2), INVALID)])
def test_rms_norm_fp8_rejects(kw, status):
    refused(rms(True, **kw), status)


def rms_backward(**kw):
    a = dict(g=P, ldg=300, s=P2, lds=300, dt=BF16, w=P, wdt=F32, rstd=P, gs=P3, ldgs=300, n=4,
             c=300, gx=P4, ldgx=300, gw=P, ws=P, wsb=HUGE)
    a.update(kw)
    return lib.vpa_rms_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), UNSUPPORTED), (dict(wdt=7), UNSUPPORTED), (dict(dt=F32, wdt=BF16), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(c=0), INVALID),
    (dict(g=None), INVALID), (dict(g=ODD), INVALID), (dict(ldg=299), INVALID),
    (dict(s=None), INVALID), (dict(s=ODD), INVALID), (dict(lds=299), INVALID),
    (dict(rstd=None), INVALID), (dict(rstd=ODD), INVALID), (dict(gs=ODD), INVALID),
    (dict(ldgs=299), INVALID), (dict(gx=ODD), INVALID), (dict(ldgx=299), INVALID),
    (dict(gw=P + 2), INVALID), (dict(w=P + 2), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 4), INVALID), (dict(wsb=16), INVALID), (dict(gx=P), INVALID),
    (dict(gx=P, gw=None, ldgx=301), INVALID), (dict(gx=P3, ldgx=301), INVALID),
    (dict(gx=P2), INVALID), (dict(gx=None, gw=None), OK), (dict(n=0, gw=None, g=None), OK),
])
def test_rms_norm_backward_rejects(kw, status):
    refused(rms_backward(**kw), status)


def quant(**kw):
    a = dict(x=P, ldx=300, dt=BF16, n=4, c=300, rows=1, y=P2, ldy=304, sc=P, ldsc=3)
    a.update(kw)
    return lib.vpa_quantize_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), UNSUPPORTED), (dict(n=-1), INVALID), (dict(c=0), INVALID), (dict(rows=0), INVALID),
    (dict(rows=64), INVALID), (dict(rows=-1), INVALID), (dict(x=None), INVALID),
    (dict(x=ODD), INVALID), (dict(ldx=299), INVALID), (dict(y=None), INVALID),
    (dict(ldy=299), INVALID), (dict(sc=None), INVALID), (dict(sc=ODD), INVALID),
    (dict(ldsc=2), INVALID), (dict(n=(1 << 31) - 1), INVALID), (dict(n=0, x=None), OK),
])
def test_quantize_rejects(kw, status):
    refused(quant(**kw), status)


def linear(**kw):
    a = dict(x=P, ldx=304, xs=P, ldxs=3, w=P, ldw=304, ws_=P, ldws=3, b=P, r=P2, ldr=200, n=4, m=200,
             k=300, act=0, y=P3, ldy=200, odt=BF16, ws=P, wsb=HUGE)
    a.update(kw)
    return lib.vpa_head_linear_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(odt=7), UNSUPPORTED), (dict(act=9), UNSUPPORTED), (dict(act=-1), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(m=0), INVALID), (dict(k=0), INVALID),
    (dict(m=1 << 31), INVALID), (dict(k=1 << 31), INVALID), (dict(x=None), INVALID),
    (dict(x=P + 8), INVALID), (dict(ldx=300), INVALID), (dict(ldx=288), INVALID),
    (dict(w=None), INVALID), (dict(w=P + 4), INVALID), (dict(ldw=308), INVALID),
    (dict(ldx=(1 << 21) + 16), INVALID), (dict(ldw=(1 << 21) + 16), INVALID),
    (dict(xs=None), INVALID), (dict(xs=ODD), INVALID), (dict(ldxs=2), INVALID),
    (dict(ws_=None), INVALID), (dict(ws_=ODD), INVALID), (dict(ldws=2), INVALID),
    (dict(b=ODD), INVALID), (dict(r=ODD), INVALID), (dict(ldr=199), INVALID),
    (dict(y=None), INVALID), (dict(y=ODD), INVALID), (dict(ldy=199), INVALID),
    (dict(y=P2, ldy=208), INVALID), (dict(y=P2, odt=F32), INVALID),
    (dict(n=0, x=None, w=None, y=None), OK),
])
def test_head_linear_fp8_rejects(kw, status):
    refused(linear(**kw), status)


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="device"):
        vpa.rms_norm(x)
    with pytest.raises(ValueError, match="device"):
        vpa.quantize_fp8(x)
    with pytest.raises(ValueError, match="device"):
        vpa.sampled_verify(x, 64, 64, 1, torch.zeros((4, 0), dtype=torch.int32), x, x)
    with pytest.raises(ValueError, match="device"):
        vpa.distill_loss(x, 64, 64, 1, x, x)
    with pytest.raises(ValueError, match="device"):
        vpa.head_linear_fp8(x.to(vpa.FP8), x, x.to(vpa.FP8), x)
