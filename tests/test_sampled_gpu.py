"""GPU tests of the sampled verification against its definition in 64 bits.

The oracle says how near each of its comparisons was: a draft's acceptance to
its border, relatively, and the drawn column's border, of the whole sum.  A
case whose margins are below what the header promises (2^-20 for p, 64-bit sums
for the draw) would say nothing, so the tests assert that they are not."""
import math

import pytest
import torch

import vocab_argmax_amd as vpa
from test_head_gpu import BF, DEV, F32, NEG, gen, randn, strided

pytestmark = pytest.mark.gpu

F64 = torch.float64


def argmax_id(row):
    """vpa.h's order: NaN first, then by value, the lower id first."""
    nan = row.isnan().nonzero()
    if len(nan):
        return int(nan[0])
    return int((row == row.max()).nonzero()[0])


def probabilities(row, temp):
    """p of a row (64 bits, CPU) at a temperature (a float), and p times its sum of exponentials:
    the same draw, with sums of equal columns that are exact."""
    has = not bool(row.isnan().any()) and bool((row > NEG).any()) and not bool((row == math.inf).any())
    if not has or not (2.0 ** -100 <= temp < math.inf):
        p = torch.zeros_like(row)
        p[argmax_id(row)] = 1.0
        return p, p
    e = ((row - row.max()) / temp).exp()
    return e / e.sum(), e


def draw(w, u):
    """(the least column whose running sum passes u of the whole, margin)."""
    c = w.cumsum(0)
    target = (u if u > 0 else 0.0) * c[-1]
    hit = (c > target).nonzero()
    token = int(hit[0]) if len(hit) else int((w > 0).nonzero()[-1])
    sure = bool((c == c[-1]).sum() == len(c) - int((w > 0).nonzero()[0])) or u <= 0 or u >= 1
    near = 1.0 if sure else float(((c - target).abs() / c[-1]).min())
    return token, near


def oracle(x, vocab, ids, u, s, q, temp):
    """(out_tokens, num_sampled, num_rejected, margin of the acceptances, of the draws)."""
    r, k = ids.shape
    x, ids = x.cpu().double()[:, :vocab], ids.cpu()
    u, s = u.cpu().double(), s.cpu()
    q = None if q is None else q.cpu().double()[:, :vocab]
    out = torch.full((r, k + 1), -1, dtype=torch.int32)
    sampled = torch.zeros(r, dtype=torch.int32)
    m_accept = m_draw = 1.0
    for i in range(r):
        t = 1.0 if temp is None else float(temp[i])
        for j in range(k + 1):
            p, e = probabilities(x[i * (k + 1) + j], t)
            w = e
            d = int(ids[i, j]) if j < k else -1
            if 0 <= d < vocab:
                hot = torch.zeros_like(p)
                hot[d] = 1.0
                qj = hot if q is None else q[i * k + j]
                left, right = float(u[i, j] * qj[d]), float(p[d])
                if max(left, right) > 0 and 0 < right < 1:
                    m_accept = min(m_accept, abs(left - right) / max(left, right))
                if left < right:
                    out[i, j] = d
                    continue
                w = (p - qj).clamp(min=0.0)
                if q is None:
                    w = torch.where(hot > 0, 0.0, e)
                if not float(w.sum()) > 0:
                    w = e
            out[i, j], near = draw(w, float(s[i]))
            m_draw = min(m_draw, near)
            sampled[i] = j + 1
            break
    return out, sampled, k + 1 - sampled, m_accept, m_draw


def check(x, v, w, shards, ids, u, s, q=None, temp=None, margins=True, what=""):
    want = oracle(x, v, ids, u, s, q, temp)
    if margins:
        assert want[3] > 2.0 ** -19 and want[4] > 1e-12, f"{what}: inputs next to a border {want[3:]}"
    got = vpa.sampled_verify(x, v, w, shards, ids, u, s, draft_probs=q, temperature=temp)
    for name, a, b in zip(("out_tokens", "num_sampled", "num_rejected"), got, want):
        a = a.cpu()
        assert torch.equal(a, b), f"{what} {name}: got {a.tolist()}, want {b.tolist()}"
    return got


def batch(seed, r, k, v, width, shards, dtype, probs, temps=True, short=0.1):
    """Logits, drafts drawn from a draft distribution near the target's, random numbers."""
    g = gen(seed)
    x = randn(g, r * (k + 1), width * shards, scale=2.0)
    sure = torch.randint(0, v, (r * (k + 1),), generator=g, device=DEV)
    x[torch.arange(r * (k + 1), device=DEV), sure] += 12 * torch.rand(r * (k + 1), generator=g,
                                                                     device=DEV)
    x = x.to(dtype)
    temp = None
    if temps:
        temp = 0.3 + torch.rand(r, generator=g, device=DEV)
        temp[::5] = 0.0
    y = x.view(r, k + 1, -1)[:, :k, :v].reshape(r * k, v).float() + 0.5 * randn(g, r * k, v)
    q = y.softmax(1)
    ids = (q / torch.empty_like(q).exponential_(generator=g)).argmax(1).view(r, k) if k else \
        torch.zeros((r, 0), dtype=torch.int64, device=DEV)
    ids = ids.masked_fill(torch.rand((r, k), generator=g, device=DEV) < short, -1).to(torch.int32)
    x[:, v:] = float("nan")                              # padding is never read
    u = torch.rand((r, k), generator=g, device=DEV)
    s = torch.rand(r, generator=g, device=DEV, dtype=F64)
    return x, ids, u, s, q.to(probs) if probs is not None and k else None, temp


CASES = [  # requests, drafts, vocab, width, shards
    (1, 0, 1, 1, 1), (1, 1, 1, 1, 1), (2, 1, 2, 1, 2), (3, 2, 7, 3, 3), (5, 3, 64, 64, 1),
    (4, 1, 257, 300, 1), (7, 4, 1000, 125, 8), (33, 0, 1000, 1000, 1), (2, 9, 4097, 4097, 1),
    (3, 2, 8191, 4100, 2), (2, 3, 16385, 5462, 3), (9, 3, 50257, 16753, 3), (2, 4, 151936, 76032, 2),
    (3, 5, 200064, 25008, 8), (300, 2, 500, 500, 1), (1, 70, 130, 130, 1),
]


@pytest.mark.parametrize("probs", [None, F32, BF])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,k,v,w,s", CASES)
def test_sampled_verify(r, k, v, w, s, dtype, probs):
    x, ids, u, su, q, temp = batch(r * v + k, r, k, v, w, s, dtype, probs)
    check(x, v, w, s, ids, u, su, q, temp, what="whole rows")
    # odd strides, rows that are not aligned
    xs = strided(x[:, :v], 3, 1)
    qs = None if q is None else strided(q, 5, 1)
    got = vpa.sampled_verify(xs, v, w, s, ids, u, su, draft_probs=qs, temperature=temp)
    for a, b in zip(got, vpa.sampled_verify(x, v, w, s, ids, u, su, draft_probs=q,
                                            temperature=temp)):
        assert torch.equal(a, b)


def test_no_temperature_is_1():
    x, ids, u, s, q, _ = batch(3, 6, 2, 1000, 1000, 1, BF, F32, temps=False)
    a = check(x, 1000, 1000, 1, ids, u, s, q)
    b = vpa.sampled_verify(x, 1000, 1000, 1, ids, u, s, draft_probs=q,
                           temperature=torch.ones(6, device=DEV))
    assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_without_a_distribution(dtype):
    """All -inf, NaN, +inf, the type's lowest value, one column left; and temperatures that are
    none: the argmax stands."""
    v, k = 3000, 2
    low = torch.finfo(dtype).min
    rows = []
    g = gen(4)
    for fill in ("inf", "nan", "empty", "low", "one", "two", "nan_inf", "plain"):
        x = randn(g, v, scale=2.0)
        if fill == "inf":
            x[[2500, 700]] = math.inf
        elif fill == "nan":
            x[[2999, 1200]] = math.nan
        elif fill == "empty":
            x[:] = NEG
        elif fill == "low":
            x[:] = low
        elif fill == "one":
            x[:] = NEG
            x[1777] = -5.0
        elif fill == "two":
            x[:] = NEG
            x[[5, 2990]] = low
        elif fill == "nan_inf":
            x[3], x[9] = math.inf, math.nan
        rows.append(x)
    n = len(rows)
    x = torch.stack(rows).to(dtype)
    x = x.repeat_interleave(k + 1, 0)
    for j in range(n):                               # the second row of a request is another kind
        x[j * (k + 1) + 1] = x[((j + 3) % n) * (k + 1)]
    first = [argmax_id(x[j * (k + 1)].double().cpu()) for j in range(n)]
    u = torch.full((n, k), 0.25, device=DEV)
    for s in (0.0, 0.4, 0.99):
        su = torch.full((n,), s, device=DEV, dtype=F64)
        for ids in (torch.tensor([[f, 1777] for f in first]), torch.full((n, k), 1777),
                    torch.full((n, k), -1), torch.tensor([[f, -1] for f in first])):
            ids = ids.to(torch.int32).to(DEV)
            check(x, v, v, 1, ids, u, su, margins=False, what=f"s {s}")
            q = torch.full((n * k, v), 1.0 / v, device=DEV)
            check(x, v, v, 1, ids, u, su, q=q, margins=False, what=f"q, s {s}")


def test_temperatures():
    v = 2000
    x = randn(gen(5), 10, v, scale=3.0)
    temp = torch.tensor([0.0, -1.0, math.nan, math.inf, 2.0 ** -101, 2.0 ** -100, 1e-3, 1.0, 50.0,
                         1e30], device=DEV)
    s = torch.rand(10, generator=gen(6), device=DEV, dtype=F64)
    empty = torch.zeros((10, 0), device=DEV)
    check(x, v, v, 1, empty.to(torch.int32), empty, s, temp=temp, what="temperatures")


def test_draws_cover_the_distribution():
    """Evenly spaced random numbers draw every column as often as its probability says."""
    n, v = 4096, 40
    row = randn(gen(7), 1, v, scale=1.5)
    row[0, [3, 17]] = NEG
    x = row.expand(n, v).contiguous()
    s = (torch.arange(n, device=DEV, dtype=F64) + 0.5) / n
    none = torch.zeros((n, 0), device=DEV)
    out, sampled, _ = vpa.sampled_verify(x, v, v, 1, none.to(torch.int32), none, s)
    count = torch.bincount(out[:, 0].long(), minlength=v).double()
    p = row[0].double().softmax(0)
    assert bool(((count - p * n).abs() <= 1).all()) and bool((sampled == 1).all())
    assert bool((out[1:, 0] >= out[:-1, 0]).all())


def test_emitted_tokens_have_the_targets_distribution():
    """Over a grid of drafts and random numbers the emitted token has p's probability, whatever q."""
    v, nu, ns = 7, 200, 50
    g = gen(8)
    p_row, q_row = randn(g, 1, v, scale=1.0), randn(g, 1, v, scale=1.0).softmax(1)
    grid = [(d, (a + 0.5) / nu, (b + 0.5) / ns) for d in range(v) for a in range(nu)
            for b in range(ns)]
    t = torch.tensor(grid, dtype=F64, device=DEV)
    n = len(grid)
    x = p_row.expand(2 * n, v).contiguous()
    out, sampled, _ = vpa.sampled_verify(
        x, v, v, 1, t[:, :1].to(torch.int32).contiguous(), t[:, 1:2].float().contiguous(),
        t[:, 2].contiguous(), draft_probs=q_row.expand(n, v).contiguous())
    weight = q_row[0].double()[t[:, 0].long()] / (nu * ns)
    first = torch.zeros(v, dtype=F64, device=DEV).scatter_add_(0, out[:, 0].long(), weight)
    # a grid of nu acceptances is off by half a step a draft, one of ns draws by one
    tol = 1.0 / nu + 1.0 / ns
    assert bool(((first - p_row[0].double().softmax(0)).abs() <= tol).all())


def test_random_numbers_at_the_ends():
    v = 1000
    x = randn(gen(9), 2, v)
    x[:, :20] = NEG
    x[:, 980:] = NEG
    none = torch.zeros((2, 0), device=DEV)
    for s, want in ((0.0, 20), (-3.0, 20), (math.nan, 20), (1.0 - 2.0 ** -53, 979), (1.0, 979),
                    (7.0, 979), (math.inf, 979)):
        out, _, _ = vpa.sampled_verify(x, v, v, 1, none.to(torch.int32), none,
                                       torch.full((2,), s, device=DEV, dtype=F64))
        assert out[:, 0].tolist() == [want, want], s
    # accepted at 0 unless p is 0; rejected from 1 on where q is not above p
    ids = torch.tensor([[50], [5]], dtype=torch.int32, device=DEV)
    xx = torch.cat([x, x])
    s = torch.full((2,), 0.5, device=DEV, dtype=F64)
    _, sampled, _ = vpa.sampled_verify(xx, v, v, 1, ids, torch.zeros((2, 1), device=DEV), s)
    assert sampled.tolist() == [2, 1]


def test_draft_distributions_of_any_kind():
    """q above p everywhere draws from p; q equal to p accepts; q of 0 at the draft accepts."""
    v = 600
    x = randn(gen(10), 4, v, scale=1.0)
    p = x[::2].double().softmax(1).float()
    ids = torch.tensor([[3], [599]], dtype=torch.int32, device=DEV)
    s = torch.tensor([0.3, 0.8], device=DEV, dtype=F64)
    u = torch.full((2, 1), 0.999, device=DEV)
    check(x, v, v, 1, ids, u, s, q=p * 3, what="above")
    check(x, v, v, 1, ids, u, s, q=p, what="equal")
    check(x, v, v, 1, ids, u, s, q=p * 1.5, what="some above")
    zero = p.clone()
    zero[torch.arange(2), ids[:, 0].long()] = 0.0
    check(x, v, v, 1, ids, u, s, q=zero, what="zero")
    other = torch.zeros_like(p)
    other[:, 100] = 1.0
    check(x, v, v, 1, torch.full_like(ids, 100), u, s, q=other, what="one column")


def test_ids_that_are_no_drafts():
    v = 300
    x = randn(gen(11), 12, v)
    ids = torch.tensor([[v, 1], [-7, 2], [2 ** 31 - 1, 3], [-2 ** 31, 4]], dtype=torch.int32,
                       device=DEV)
    u = torch.zeros((4, 2), device=DEV)
    s = torch.rand(4, generator=gen(12), device=DEV, dtype=F64)
    out = check(x, v, v, 1, ids, u, s)
    assert out[1].tolist() == [1, 1, 1, 1]


def test_rows_after_a_placeholder_are_not_needed():
    v = 5000
    x, ids, u, s, q, temp = batch(13, 4, 3, v, v, 1, BF, F32, short=0.0)
    ids[:, 1] = -1
    a = check(x, v, v, 1, ids, u, s, q, temp)
    x.view(4, 4, v)[:, 2:] = float("nan")
    b = vpa.sampled_verify(x, v, v, 1, ids, u, s, draft_probs=q, temperature=temp)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("r,k,v", [(3, 2, 1000), (24, 3, 151936)])
def test_repeats_streams_graphs_and_workspaces(r, k, v):
    x, ids, u, s, q, temp = batch(14, r, k, v, v, 1, BF, BF)
    args, kw = (x, v, v, 1, ids, u, s), dict(draft_probs=q, temperature=temp)
    want = [t.clone() for t in vpa.sampled_verify(*args, **kw)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(vpa.sampled_verify(*args, **kw), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vpa.sampled_verify(*args, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    need = vpa.sampled_verify_workspace(v, v, 1, r, k)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    got = vpa.sampled_verify(*args, workspace=ws[:need], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((ws[need:] == 0x5A).all())
    with pytest.raises(vpa.VpaError, match="workspace"):
        vpa.sampled_verify(*args, workspace=ws[:need - 1], **kw)
    # replays, the inputs changed in place between them
    graph = torch.cuda.CUDAGraph()
    x2, u2 = x.clone(), u.clone()
    with torch.cuda.graph(graph):
        out = vpa.sampled_verify(x2, *args[1:5], u2, s, **kw)
    for turn in range(4):
        x2.copy_(x if turn % 2 == 0 else x.flip(0))
        u2.copy_(u if turn < 2 else u.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        fresh = vpa.sampled_verify(x2, *args[1:5], u2, s, **kw)
        assert all(torch.equal(a, b) for a, b in zip(out, fresh)), turn


def test_empty_batch():
    x = torch.zeros((0, 100), dtype=BF, device=DEV)
    out, a, b = vpa.sampled_verify(x, 100, 100, 1, torch.zeros((0, 3), dtype=torch.int32, device=DEV),
                                   torch.zeros((0, 3), device=DEV),
                                   torch.zeros(0, dtype=F64, device=DEV))
    assert out.shape == (0, 4) and a.shape == b.shape == (0,)


def test_refusals():
    x, ids, u, s, q, temp = batch(15, 2, 2, 100, 100, 1, BF, F32, temps=True)
    ok = dict(draft_probs=q, temperature=temp)
    vpa.sampled_verify(x, 100, 100, 1, ids, u, s, **ok)
    for bad, err in (
            ((x[:5], 100, 100, 1, ids, u, s), ValueError), ((x[:, :99], 100, 100, 1, ids, u, s), ValueError),
            ((x, 100, 100, 1, ids.long(), u, s), TypeError), ((x, 100, 100, 1, ids, u.double(), s), TypeError),
            ((x, 100, 100, 1, ids, u, s.float()), TypeError), ((x, 100, 100, 1, ids, u, s[:1]), ValueError),
            ((x, 100, 100, 1, ids.cpu(), u, s), ValueError), ((x.cpu(), 100, 100, 1, ids, u, s), ValueError),
            ((x.half(), 100, 100, 1, ids, u, s), TypeError), ((x, 100, 40, 2, ids, u, s), vpa.VpaError),
            ((x, 100, 100, 1, ids[0], u, s), ValueError), ((x, 100, 100, 1, ids.T, u, s), ValueError)):
        with pytest.raises(err):
            vpa.sampled_verify(*bad, **ok)
    for kw in (dict(draft_probs=q[:3]), dict(draft_probs=q[:, :99]), dict(temperature=temp[:1]),
               dict(temperature=temp.double()), dict(draft_probs=q.half()),
               dict(draft_probs=q.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            vpa.sampled_verify(x, 100, 100, 1, ids, u, s, **kw)


def test_offsets_past_32_bits():
    """Rows of logits and of q that lie past 2^32 bytes and 2^31 elements."""
    v, k, r = 200064, 7, 1400                            # 2.2e9 elements of logits
    x = torch.zeros((r * (k + 1), v), dtype=BF, device=DEV)
    g = gen(16)
    at = [0, r - 1]
    for i in at:
        x[i * (k + 1):(i + 1) * (k + 1)] = randn(g, k + 1, v, dtype=BF, scale=3.0)
    q = torch.zeros((r * k, v), dtype=BF, device=DEV)
    ids = torch.full((r, k), -1, dtype=torch.int32, device=DEV)
    for i in at:
        q[i * k:(i + 1) * k] = x[i * (k + 1):(i + 1) * (k + 1) - 1].float().softmax(1).to(BF)
        ids[i] = q[i * k:(i + 1) * k].argmax(1)
    u = torch.rand((r, k), generator=g, device=DEV)
    s = torch.rand(r, generator=g, device=DEV, dtype=F64)
    out, sampled, rejected = vpa.sampled_verify(x, v, v, 1, ids, u, s, draft_probs=q)
    for i in at:
        want = oracle(x[i * (k + 1):(i + 1) * (k + 1)], v, ids[i:i + 1], u[i:i + 1], s[i:i + 1],
                      q[i * k:(i + 1) * k], None)
        assert torch.equal(out[i:i + 1].cpu(), want[0]) and int(sampled[i]) == int(want[1])
    # a row of equal logits draws column floor(u V)
    mid = (s[1:-1].cpu() * v).floor().long()
    assert torch.equal(out[1:-1, 0].cpu().long(), mid)
