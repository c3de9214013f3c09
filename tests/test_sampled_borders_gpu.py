"""Acceptances of the sampled verification next to their borders: p is within 2^-36 of its
value, so u q that is 2^-34 and more below it is accepted, and above it is not."""
import math

import numpy as np
import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, gen, randn
from test_row_sums_gpu import logits, row_sum

pytestmark = pytest.mark.gpu

F64 = torch.float64


def pair(p, side, rng):
    """(u, q), fp32, with u q between 2^-34 and 2^-30 of p below (side < 0) or above it, u < 1."""
    q = (p * (1.05 + rng.random(60000))).astype("float32")
    q = q[q < 1] if (q < 1).any() else (p + (1 - p) * rng.random(60000)).astype("float32")
    u = (p / q.astype("float64")).astype("float32")
    off = u.astype("float64") * q.astype("float64") / p - 1
    ok = (u < 1) & (off * side > 2.0 ** -34) & (off * side < 2.0 ** -30)
    i = ok.nonzero()[0][0]
    return float(u[i]), float(q[i])


def late_peaks(seed, rows, v, dtype):
    """Rows whose first columns are far below a token that comes late, and others of many sizes."""
    g = gen(seed)
    x = randn(g, rows, v, scale=2.0)
    lift = 10 + 25 * torch.rand(rows, generator=g, device=DEV)
    at = v // 2 + torch.randint(0, v // 2, (rows,), generator=g, device=DEV)
    row = torch.arange(rows, device=DEV)
    x[row, at] += lift
    x[row, at - 1000] = x[row, at] - 0.2 - 1.3 * torch.rand(rows, generator=g, device=DEV)
    x[row, 100] += 8
    return x.to(dtype), at


def borders(x, ids, temp, sides, seed):
    """(u, q at the drafts) of one draft a request, each within 2^-30 of its border."""
    rng = np.random.default_rng(seed)
    out = []
    for i, side in enumerate(sides):
        z = x[i].double().cpu() / (1.0 if temp is None else float(temp[i]))
        p = float((z - z.max()).exp()[ids[i]] / (z - z.max()).exp().sum())
        out.append(pair(p, side, rng))
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,v", [(3, 151936), (40, 32000), (300, 40000)])
def test_acceptances_next_to_their_border(r, v, dtype):
    x, at = late_peaks(r, 2 * r, v, dtype)
    g = gen(r + 1)
    temp = (0.4 + 0.8 * torch.rand(r, generator=g, device=DEV))
    sides = [-1 if i % 2 else 1 for i in range(r)]
    ids = at[0::2]
    uq = borders(x[0::2], ids, temp, sides, r)
    q = torch.zeros((r, v), device=DEV)
    q[torch.arange(r, device=DEV), ids] = torch.tensor([b for _, b in uq], device=DEV)
    u = torch.tensor([[a] for a, _ in uq], device=DEV)
    s = torch.rand(r, generator=g, device=DEV, dtype=F64)
    args = (x, v, v, 1, ids.int().view(r, 1), u, s)
    out, n, rejected = vpa.sampled_verify(*args, draft_probs=q, temperature=temp)
    want = [2 if side < 0 else 1 for side in sides]
    assert n.tolist() == want and rejected.tolist() == [2 - i for i in want]
    again = vpa.sampled_verify(*args, draft_probs=q, temperature=temp)
    assert all(torch.equal(a, b) for a, b in zip(again, (out, n, rejected)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,v", [(512, 2 ** 20), (5, 2 ** 23)])
def test_acceptances_over_long_rows(r, v, dtype):
    """Drafts next to their border: below it accepted, above it not."""
    rng = np.random.default_rng(v)
    c = -2.5
    x = logits(2 * r, v, c, dtype)
    p = 1 / row_sum(v, c)
    side = [-1 if i % 2 else 1 for i in range(r)]
    uq = [pair(p, s, rng) for s in side]
    q = torch.zeros((r, v), device=DEV)
    at = torch.tensor([256 * (i % 7) for i in range(r)], device=DEV)
    q[torch.arange(r, device=DEV), at] = torch.tensor([b for _, b in uq], device=DEV)
    u = torch.tensor([[a] for a, _ in uq], device=DEV)
    _, n, _ = vpa.sampled_verify(x, v, v, 1, at.int().view(r, 1), u,
                                 torch.full((r,), 0.5, dtype=torch.float64, device=DEV), draft_probs=q)
    assert n.tolist() == [2 if s < 0 else 1 for s in side]


@pytest.mark.parametrize("k", [3, 4, 9])
def test_several_in_one_request(k):
    """Positions one after another at their borders, the last of them on the far side, for each
    length: those before it are accepted."""
    v, r = 20000, k + 1
    x, at = late_peaks(k, r * (k + 1), v, BF)
    ids = at.view(r, k + 1)[:, :k].contiguous()
    q = torch.zeros((r * k, v), device=DEV)
    u = torch.zeros((r, k), device=DEV)
    for i in range(r):
        sides = [1 if j == i else -1 for j in range(k)]
        uq = borders(x.view(r, k + 1, v)[i, :k], ids[i], None, sides, i)
        u[i] = torch.tensor([a for a, _ in uq])
        q[torch.arange(i * k, i * k + k, device=DEV), ids[i]] = torch.tensor([b for _, b in uq],
                                                                            device=DEV)
    s = torch.rand(r, generator=gen(k), device=DEV, dtype=F64)
    out, n, _ = vpa.sampled_verify(x, v, v, 1, ids.int(), u, s, draft_probs=q)
    assert n.tolist() == [i + 1 for i in range(r)]
    for i in range(r):
        assert out[i, :i].tolist() == ids[i, :i].tolist()
        assert bool((out[i, i + 1:] == -1).all())


def test_borders_that_are_exact():
    """Equal logits: p = 1 / n exactly, and u = p is not below it."""
    for v in (2, 8, 1024, 65536):
        x = torch.full((4, v), 3.25, device=DEV)
        ids = torch.tensor([[0], [v - 1]], dtype=torch.int32, device=DEV)
        s = torch.full((2,), 0.75, dtype=F64, device=DEV)
        for u, want in ((1 / v, 1), (np.nextafter(np.float32(1 / v), np.float32(0)), 2)):
            _, n, _ = vpa.sampled_verify(x, v, v, 1, ids, torch.full((2, 1), float(u), device=DEV), s)
            assert n.tolist() == [want, want], (v, u)
