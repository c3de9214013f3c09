"""Refusals of the head's operators on the CPU that test_head_cpu.py does not
have.  Pointers passed here are never dereferenced."""
import pytest

import vocab_argmax_amd as vpa
from test_head_cpu import BF16, F32, HUGE, INVALID, ODD, OK, P, UNSUPPORTED, lib


def typed(g=P, ldg=96, gdt=F32, x=P, ldx=64, w=P, ldw=64, pre=P, ldp=96, dt=BF16, rows=8, outer=96,
          inner=64, act=3, gx=P, ldgx=64, gw=P, ldgw=64, gb=P, ws=P, wsb=HUGE):
    return lib.vpa_head_linear_backward_typed(g, ldg, gdt, x, ldx, w, ldw, pre, ldp, dt, rows,
                                              outer, inner, act, gx, ldgx, gw, ldgw, gb, ws, wsb,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(gdt=7), UNSUPPORTED), (dict(dt=7), UNSUPPORTED), (dict(act=4), UNSUPPORTED),
    (dict(gdt=BF16, dt=F32), UNSUPPORTED),               # a gradient in fewer bits
    (dict(g=None), INVALID), (dict(g=ODD), INVALID), (dict(g=P + 2), INVALID),
    (dict(ldg=95), INVALID), (dict(x=None), INVALID), (dict(w=ODD), INVALID),
    (dict(pre=None), INVALID), (dict(outer=0), INVALID), (dict(rows=-1), INVALID),
    (dict(gx=ODD), INVALID), (dict(ldgw=63), INVALID), (dict(gb=ODD), INVALID),
    (dict(wsb=0), INVALID), (dict(ws=None), INVALID),
    (dict(act=0, pre=None, ws=None, wsb=0), INVALID),    # the copy of grad needs its place
    (dict(rows=0, g=None, gx=None, gw=None, gb=None, ws=None), OK),
])
def test_backward_for_another_type_of_gradient_rejects(kw, status):
    assert typed(**kw) == status
    assert status == OK or vpa.last_error() != ""
