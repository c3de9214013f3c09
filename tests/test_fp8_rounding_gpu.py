"""8-bit elements bit for bit: y / scale, one division rounded to fp32, then to the
nearest e4m3 value, ties to the even one.  The division is the CPU's."""
import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, gen, randn

pytestmark = pytest.mark.gpu

F8_MAX = 448.0


def rounded(y, scale, rows=1):
    """y (fp32, CPU) over its blocks' scales in 8 bits."""
    s = scale.cpu().repeat_interleave(rows, 0)[:y.shape[0]].repeat_interleave(128, 1)[:, :y.shape[1]]
    return (y / s).clamp(-F8_MAX, F8_MAX).to(vpa.FP8).float()


def check(x, rows=1):
    y, scale = vpa.quantize_fp8(x.to(DEV), rows)
    got, want = y.cpu().float(), rounded(x.float(), scale, rows)
    off = (got != want).nonzero()
    assert len(off) == 0, (f"{len(off)} of {got.numel()} differ, the first at {off[0].tolist()}: "
                           f"{got[tuple(off[0])]} for {want[tuple(off[0])]}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bf16_values_of_every_mantissa(dtype):
    """All bf16 mantissas of a largest value against all of an element at up to 11 binades below
    it: many quotients are ties of e4m3.  Blocks of 128 columns, the first of each the largest."""
    mantissa = torch.arange(128, dtype=torch.float32) / 128 + 1
    elements = torch.cat([mantissa * 2.0 ** -e for e in range(1, 12)])
    elements = torch.nn.functional.pad(elements, (0, -len(elements) % 127))
    blocks = elements.view(-1, 127)
    x = torch.cat([torch.cat([amax.expand(len(blocks), 1), blocks], 1).view(1, -1)
                   for amax in mantissa])
    for x in (x, -x, x * 2.0 ** 90, x * 2.0 ** -80):
        check(x.to(dtype))
    wide = x[:, :128 * 3].repeat_interleave(128, 0)[:2000].contiguous()      # 128 x 128, one amax
    check(wide.to(dtype), 128)


@pytest.mark.parametrize("rows", [1, 128])
def test_ties_and_their_neighbours(rows):
    """scale = s exactly (s of 18 bits, 448 s the largest value), elements t s for every border t
    between two e4m3 values, and the fp32 numbers next to those."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(vpa.FP8).float()
    t = (grid[1:] + grid[:-1]) / 2                       # 126 borders, exact
    g = torch.Generator().manual_seed(1)
    s = (torch.randint(2 ** 17, 2 ** 18, (256,), generator=g).float() *
         torch.exp2(torch.randint(-60, 60, (256,), generator=g).float()))
    if rows > 1:
        s = s[:2].repeat_interleave(rows)
    tie = t * s[:, None]
    inf = torch.full((), float("inf"))
    for x in (tie, torch.nextafter(tie, inf), torch.nextafter(tie, -inf)):
        x = torch.cat([F8_MAX * s[:, None], x, -x[:, :1]], 1).contiguous()
        check(x, rows)


@pytest.mark.parametrize("n", [1000, 1600, 2048])
def test_random_values(n):
    check(torch.randn(500, n, generator=torch.Generator().manual_seed(n)))


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("n,c", [(300, 64), (200, 513), (500, 2048), (50, 16384), (6, 20000)])
def test_rms_norm_fp8(n, c, dtype, wdtype):
    """y is (s rstd) w with two fp32 roundings and the rstd that rms_norm gives."""
    g = gen(n + c)
    x, r = randn(g, n, c, dtype=dtype), randn(g, n, c, dtype=dtype)
    w = (1 + randn(g, c, scale=0.2)).to(wdtype)
    full = vpa.rms_norm(x, w, r, with_rstd=True)
    q = vpa.rms_norm_fp8(x, w, r)
    y = full.summed.cpu().float() * full.rstd.cpu()[:, None] * w.cpu().float()
    amax = torch.nn.functional.pad(y.abs(), (0, -c % 128)).view(n, -1, 128).amax(2)
    assert torch.equal(q.scale.cpu(), (amax.double() / F8_MAX).float())
    assert torch.equal(q.y.cpu().float(), rounded(y, q.scale))
