"""The sums of an 8-bit product keep every digit of fp32, whatever the rows: large
products that cancel beside small ones.  All partial sums are whole numbers below
2^24, so any order of fp32 additions gives them exactly."""
import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, gen

pytestmark = pytest.mark.gpu


def operands(seed, n, k, m):
    """Blocks of k that hold 448 * 448 and its negative a few times, in places of their own in
    every row, beside products of 1, 0 and -1; scales are 1."""
    g = gen(seed)
    w = torch.randint(-1, 2, (m, k), generator=g, device=DEV).float()
    x = torch.randint(-1, 2, (n, k), generator=g, device=DEV).float()
    at = torch.arange(0, k - k % 16, 16, device=DEV)
    a = at + torch.randint(0, 8, at.shape, generator=g, device=DEV)
    b = at + 8 * torch.randint(0, 2, at.shape, generator=g, device=DEV)
    b = torch.where(b == at, at + (a - at + 1) % 8, b)   # in the same eight, or in the next
    w[:, a] = w[:, b] = 448.0
    x[:, a], x[:, b] = 448.0, -448.0

    def rows(t):
        out = torch.zeros((t.shape[0], (k + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
        out.view(vpa.FP8)[:, :k] = t.to(vpa.FP8)
        return out.view(vpa.FP8)[:, :k]
    blocks = -(-k // 128)
    return (rows(x), torch.ones((n, blocks), device=DEV), rows(w),
            torch.ones((-(-m // 128), blocks), device=DEV), x.double() @ w.double().T)


SIZES = [  # rows, inner, outer: each kernel's tiles, whole and with ends
    (1, 4096, 300), (16, 1000, 300), (20, 2048, 1000), (64, 130, 515), (65, 256, 130),
    (128, 4096, 2048), (200, 2047, 777), (300, 512, 16500), (512, 4200, 4096), (1000, 200, 4090),
    (2048, 384, 4096), (4096, 1024, 4100),
]


@pytest.mark.parametrize("n,k,m", SIZES)
def test_sums_are_exact(n, k, m):
    x, xs, w, ws, z = operands(n + k + m, n, k, m)
    assert torch.equal(vpa.head_linear_fp8(x, xs, w, ws, out_dtype=F32).double(), z), "fp32"
    assert torch.equal(vpa.head_linear_fp8(x, xs, w, ws), z.to(BF)), "bf16"


def test_a_row_does_not_depend_on_the_batch():
    """The first rows of products of 64 and more rows, to bf16, are alike."""
    x, xs, w, ws, _ = operands(5, 700, 1024, 4096)
    want = vpa.head_linear_fp8(x[:64], xs[:64], w, ws)
    for n in (65, 128, 300, 700):
        assert torch.equal(vpa.head_linear_fp8(x[:n], xs[:n], w, ws)[:64], want), n
