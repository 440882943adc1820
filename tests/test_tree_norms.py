"""csa_tree_attn and csa_paged_attn against fp64 in 2-norms, per query and per request.

A bound on each element by the largest |v| leaves room for much where many rows average out: V rows that are left out, or
a piece's output taken for another's, while the softmax's sum and lse are right.  With u = 2^-8 (bf16, half a step) and
A = sum_r p_r^2 |v_r|^2 of a query:
  - a weight's rounding is off by at most u relative (f16's less), so the error of out is |sum_r d_r p_r v_r| with |d_r| <= u,
    independent of one another: for up to four rows at most u 2 sqrt(A) by Cauchy and Schwarz, for more its mean square is
    u^2 A / 3 at most, of which 2 sqrt(3) roots are out of reach of a sum of many.  The output's rounding adds u |out|.
    Per query, then, u (2 sqrt(A) + |out|).
  - over a request of 64 rows and more, thousands of roundings: 1.3 u / sqrt(3) sqrt(sum A + sum |out|^2).
The scores' fp32 sums move weights by up to LSE_TOL (see test_paged_attn.py): as much of sqrt(A) + |out| on top of either.
"""
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import csa
from test_paged_attn import LSE_TOL, _pool
from test_tree_attn import DEV, _gpu, _sees, _tree

U = 2.0 ** -8


def definition(q, k, v, lens, counts, sees, pos, table, block, win):
    """out, lse and A in fp64."""
    b, s, h, d = q.shape
    out = torch.zeros(b, s, h, d, dtype=torch.float64)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64)
    spread = torch.zeros(b, s, h, dtype=torch.float64)
    for i, (n, c) in enumerate(zip(lens, counts)):
        if n <= 0 or c <= 0:
            continue
        r = torch.arange(n)
        rows = table[i].long()[r // block] * block + r % block
        kk, vv = (x[rows].repeat_interleave(h // k.shape[1], 1) for x in (k, v))
        seen = (r < n - c).expand(c, n).clone()
        if win:
            seen &= r > pos[i, :c, None] - win
        seen[:, max(n - c, 0):] = sees[i, :c, max(c - n, 0):c]
        sc = torch.einsum("shd,lhd->shl", q[i, :c].double(), kk) * d ** -0.5
        sc = torch.where(seen[:, None], sc, -math.inf)
        top = sc.amax(2, keepdim=True).clamp_min(-1e300)
        p = torch.exp(sc - top)
        total = p.sum(2, keepdim=True)
        p = p / total.clamp_min(1e-300)
        lse[i, :c] = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
        out[i, :c] = torch.einsum("shl,lhd->shd", p, vv)
        spread[i, :c] = torch.einsum("shl,lh->sh", p * p, (vv * vv).sum(2))
    return out, lse, spread


def faults(got, lse_got, want, lens):
    """What is wrong with out and lse, as texts."""
    out, lse, spread = want
    found = []
    if not torch.equal(torch.isinf(lse_got), torch.isinf(lse)):
        found.append("lse: queries without a row")
    elif ((lse_got - lse)[~torch.isinf(lse)].abs() > LSE_TOL).any():
        found.append("lse")
    err, size = (got - out).norm(dim=3), out.norm(dim=3)
    extra = LSE_TOL * (spread.sqrt() + size)
    if (err > U * (2 * spread.sqrt() + size) + extra).any():
        found.append("a query's output")
    for i, n in enumerate(lens):
        if n >= 64:
            most = 1.3 * U / math.sqrt(3) * math.sqrt(float(spread[i].sum() + (size[i] ** 2).sum())) + float(extra[i].norm())
            if float(err[i].norm()) > most:
                found.append(f"request {i}'s output, {float(err[i].norm()) / most:.2f} times the bound")
    return found


def _case(lens, s, h, hk, d, block, fp8, seed, counts=None, win=0, chain=False):
    pool, k, v = _pool(lens, hk, d, block, seed, fp8)
    b = len(lens)
    q = torch.randn(b, s, h, d, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    masks = csa.tree_masks((torch.arange(s) - 1).repeat(b, 1), win) if chain else _tree(b, s, seed + 2)
    sees = _sees(masks, s)
    counts = [s] * b if counts is None else counts
    depth = torch.arange(s).expand(b, s) if chain else sees.sum(2) - 1
    pos = ((torch.tensor(lens) - torch.tensor(counts))[:, None] + depth).int()
    want = definition(q, k, v, lens, counts, sees, pos, pool["table"].cpu(), block, win)
    return pool, q, masks, pos, counts, want


# ---------------------------------------------------------------------------
# CPU: the bounds see what they are for

@pytest.fixture(scope="module")
def sample():
    """Four drafts of two heads over 6000 rows, in fp64: the rows' parts of out, and what the checks take."""
    g = torch.Generator().manual_seed(3)
    n, s, h, d = 6000, 4, 2, 128
    sc = torch.randn(s, h, n, generator=g).double()
    v = torch.randn(n, h, d, generator=g).double()
    p = torch.softmax(sc, 2)
    want = (torch.einsum("shl,lhd->shd", p, v)[None], torch.logsumexp(sc, 2)[None],
            torch.einsum("shl,lh->sh", p * p, (v * v).sum(2))[None])
    return p, v, want


def _rounded(p, v):
    top = p.amax(2, keepdim=True)
    return torch.einsum("shl,lhd->shd", (p / top).bfloat16().double() * top, v)[None].bfloat16().double()


def test_roundings_are_within_the_bounds(sample):
    p, v, want = sample
    assert faults(_rounded(p, v), want[1], want, [6000]) == []


@pytest.mark.parametrize("mistake", ["tenth of the rows left out", "one tile of V left out", "a piece's output twice",
                                     "two heads' pieces exchanged", "one percent", "one query's weights in 4 bits"])
def test_planted_mistakes_are_found(sample, mistake):
    p, v, want = sample
    p2, v2 = p.clone(), v.clone()
    if mistake == "tenth of the rows left out":
        v2[::10] = 0
    elif mistake == "one tile of V left out":
        v2[1280:1408] = 0
    elif mistake == "a piece's output twice":
        v2[3000:3400] *= 2
    elif mistake == "two heads' pieces exchanged":
        v2[4000:4500] = v[4000:4500].flip(1)
    elif mistake == "one percent":
        v2 *= 0.99
    else:
        p2[1, 0] = torch.round(torch.log2(p2[1, 0]) * 8).div(8).exp2()
    assert faults(_rounded(p2, v2), want[1], want, [6000])


# ---------------------------------------------------------------------------
# GPU

LONG = [[20011], [9000, 200, 101, 12001, 640], [177] * 40]
MANY = [(130 + 37 * i) % 700 + 70 for i in range(650)]     # more requests than a block has threads
SHAPES = [(8, 8, 2, 128, False), (6, 4, 1, 256, False), (64, 4, 1, 128, False), (30, 16, 2, 64, False), (64, 8, 2, 128, True),
          (16, 8, 1, 128, True), (9, 4, 2, 128, True)]


def _tree_faults(lens, s, h, hk, d, fp8, block, max_len, seed, counts=None, win=0, chain=False):
    _gpu()
    pool, q, masks, pos, counts, want = _case(lens, s, h, hk, d, block, fp8, seed, counts, win, chain)
    kk, vv = pool.pop("k"), pool.pop("v")
    dev = lambda t: t.to(DEV)
    got = csa.TreeAttention(dev(q), kk, vv, dev(torch.tensor(lens, dtype=torch.int32)), dev(masks),
                            count=dev(torch.tensor(counts, dtype=torch.int32)), pos=dev(pos) if win else None, win=win,
                            max_len=max_len, **pool)()
    torch.cuda.synchronize()
    return faults(got["out"].cpu().double(), got["lse"].cpu().double(), want, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
@pytest.mark.parametrize("lens", LONG)
@pytest.mark.parametrize("max_len", [None, 1 << 20])
def test_long_requests_that_are_split_and_joined(lens, s, h, hk, d, fp8, max_len):
    assert _tree_faults(lens, s, h, hk, d, fp8, 128, max_len, d) == []


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 1, 128, False), (64, 1, 1, 64, False), (40, 2, 1, 128, True), (3, 2, 1, 128, True)])
@pytest.mark.parametrize("max_len", [None, 1 << 20])
def test_many_requests(s, h, hk, d, fp8, max_len):
    counts = [s if i % 5 else i % (s + 1) for i in range(len(MANY))]
    assert _tree_faults(MANY, s, h, hk, d, fp8, 64, max_len, 13, counts) == []


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
@pytest.mark.parametrize("block", [1, 3, 17, 40])
@pytest.mark.parametrize("win", [0, 150])
def test_pages_of_odd_sizes_windows_and_counts(s, h, hk, d, fp8, block, win):
    # pages of one row to forty: copies of one row, and of eight
    lens = [700, 64 + s, 129 + s, 400]
    assert _tree_faults(lens, s, h, hk, d, fp8, block, 1 << 20, block + win, [s, max(1, s // 2), s, 1], win) == []


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
@pytest.mark.parametrize("win", [0, 21, 500])
@pytest.mark.parametrize("max_len", [None, 1 << 20])
def test_a_chain_in_both_attentions(s, h, hk, d, fp8, win, max_len):
    lens = [s, 300, 1111, 5000]
    assert _tree_faults(lens, s, h, hk, d, fp8, 64, max_len, 4, None, win, True) == []
    if max_len is None:
        pool, q, _, _, _, want = _case(lens, s, h, hk, d, 64, fp8, 4, None, win, True)
        got = csa.PagedAttention(q.to(DEV), pool.pop("k"), pool.pop("v"), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 win=win, **pool)()
        torch.cuda.synchronize()
        assert faults(got["out"].cpu().double(), got["lse"].cpu().double(), want, lens) == []


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8,lens", [(1, 32, 8, 128, False, [1023]), (1, 64, 8, 128, True, [30000, 17, 2000]),
                                               (4, 16, 8, 64, False, [9000, 8, 100]), (16, 8, 8, 256, False, [4100, 700])])
def test_the_causal_attention(s, h, hk, d, fp8, lens):
    _gpu()
    pool, q, _, _, _, want = _case(lens, s, h, hk, d, 64, fp8, 9, None, 0, True)
    got = csa.PagedAttention(q.to(DEV), pool.pop("k"), pool.pop("v"), torch.tensor(lens, dtype=torch.int32, device=DEV), **pool)()
    torch.cuda.synchronize()
    assert faults(got["out"].cpu().double(), got["lse"].cpu().double(), want, lens) == []
