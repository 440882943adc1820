"""Attention over E4M3 pools whose V scales lie next to fp32's ends, where a weight with its row's scale, or the
softmax's sum without it, leaves a format's range.

Tolerance, in 2-norms over all outputs.  The weights are rounded to bf16 or f16 and the output to bf16: each rounding is
off by at most u = 2^-8 relative, in the mean square by u / sqrt(3) where a mantissa is at its lowest.  Roundings of
different weights are independent, so with A = sum_r p_r^2 |v_r|^2 of a query the error's norm is about
u / sqrt(3) sqrt(A + |out|^2); the tests allow 1.3 of it, summed over the queries, for the sample and the fp32 scores.

The warps' kernel forms its weights w_r = p_r |v_scale_r| in f16, 2^-25 off at most where the largest W of a query's is
2^7 or more: by 2^-32 W (csa.h says so), whatever row W is of, one of zeros too.  That is up to 2^-32 W sum_r |code_r| in
the output's norm, which says little where the scales of a request lie 2^32 apart, and is nothing where they are alike.
"""
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa
from test_paged_attn import LSE_TOL, _pool
from test_tree_attn import DEV, _gpu, _sees, _tree

U = 2.0 ** -8


def definition(q, k, codes, vs, lens, sees, table, block, scale=128 ** -0.5):
    """out, lse and A in fp64, and what the warps' kernel may add; sees [B, S, S]: among the drafts."""
    b, s, h, d = q.shape
    v = codes * vs[..., None]
    out = torch.zeros(b, s, h, d, dtype=torch.float64)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64)
    spread, apart = torch.zeros(2, b, s, h, dtype=torch.float64)
    for i, n in enumerate(lens):
        if n <= 0:
            continue
        r = torch.arange(n)
        rows = table[i].long()[r // block] * block + r % block
        kk, vv, cc, ss = (x[rows].repeat_interleave(h // k.shape[1], 1) for x in (k, v, codes, vs.abs()))
        seen = torch.ones(s, n, dtype=torch.bool)
        seen[:, n - s:] = sees[i]
        sc = torch.einsum("shd,lhd->shl", q[i].double(), kk) * scale
        sc = torch.where(seen[:, None], sc, -math.inf)
        p = torch.softmax(sc, 2)
        lse[i] = torch.logsumexp(sc, 2)
        out[i] = torch.einsum("shl,lhd->shd", p, vv)
        unit = float(ss.max())
        spread[i] = torch.einsum("shl,lh->sh", p * p, ((vv / unit) ** 2).sum(2)).sqrt() * unit
        apart[i] = 2.0 ** -32 * (p * ss.t()).amax(2) * (cc.norm(dim=2)[None].transpose(1, 2) * seen[:, None]).sum(2)
    return out, lse, spread, apart


def check(got, want, unit=1.0, warps=False):
    """unit: a power of two that the values are near (their squares stay in fp64's range)."""
    out, lse, spread, apart = want
    assert (got["lse"].cpu().double() - lse).abs().max() <= LSE_TOL
    err = float(((got["out"].cpu().double() - out) / unit).norm())
    most = 1.3 * U / math.sqrt(3) * math.sqrt(float(((spread / unit) ** 2).sum() + ((out / unit) ** 2).sum()))
    if warps:
        most += float((apart / unit).norm())
    assert err <= most, err / most


# drafts, heads, kv heads, the bound on the lengths: few query rows and short requests go to the warps' kernel
SHAPES = [(5, 8, 2, None), (16, 8, 1, None), (16, 8, 1, 1 << 20), (64, 8, 2, 1 << 20)]


def _rows(lens, s, h, hk, seed, qstd):
    pool, k, v = _pool(lens, hk, 128, 64, seed, True)
    scale = pool.pop("v_scale").cpu().double()
    codes = torch.where(torch.isfinite(v), v / scale[..., None], 0.0)
    q = (torch.randn(len(lens), s, h, 128, generator=torch.Generator().manual_seed(seed + 1)) * qstd).bfloat16()
    r = torch.full((scale.shape[0],), -1)             # a pool row's place in its request
    table = pool["table"].cpu().long()
    for i, n in enumerate(lens):
        at = torch.arange(n)
        r[table[i][at // 64] * 64 + at % 64] = at
    return pool, k, codes, q, r


def _attend(pool, codes, vs, q, lens, masks, **kw):
    return csa.TreeAttention(q.to(DEV), pool["k"], codes.to(torch.float8_e4m3fn).to(DEV),
                             torch.tensor(lens, dtype=torch.int32, device=DEV), masks.to(DEV), table=pool["table"], block=64,
                             k_scale=pool["k_scale"], v_scale=vs.float().to(DEV), **kw)()


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", SHAPES)
@pytest.mark.parametrize("power", [-126, -118, -100, -88, -60, 60, 70, 80])
@pytest.mark.parametrize("qstd", [0.1, 1.0, 4.0])
def test_all_scales_of_one_size(s, h, hk, max_len, power, qstd):
    _gpu()
    lens = [1500, s + 100, 700]
    pool, k, codes, q, _ = _rows(lens, s, h, hk, 31, qstd)
    masks, unit = _tree(3, s, 2), 2.0 ** power
    vs = torch.full((codes.shape[0], hk), unit, dtype=torch.float64)
    vs[::3] *= -1
    got = _attend(pool, codes, vs, q, lens, masks, max_len=max_len)
    torch.cuda.synchronize()
    check(got, definition(q, k, codes, vs, lens, _sees(masks, s), pool["table"].cpu(), 64), unit, max_len is None)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", SHAPES)
@pytest.mark.parametrize("power,other", [(-126, 1.0), (-126, 0.0), (0, 2.0 ** 70), (0, 2.0 ** -126), (-126, 2.0 ** 70), (-30, 2.0 ** 30)])
@pytest.mark.parametrize("late", [False, True])
def test_rows_of_zeros_with_another_scale(s, h, hk, max_len, power, other, late):
    # rows whose codes are all zero, as csa_kv_append writes them with scale 1, before or behind the others
    _gpu()
    lens = [1500, s + 400, 700]
    pool, k, codes, q, r = _rows(lens, s, h, hk, 37, 1.0)
    masks, unit = _tree(3, s, 2), 2.0 ** power
    zero = (r >= 200) if late else (r < 200)
    codes[zero] = 0
    vs = torch.where(zero, other, unit).double()[:, None].expand(-1, hk).contiguous()
    got = _attend(pool, codes, vs, q, lens, masks, max_len=max_len)
    torch.cuda.synchronize()
    check(got, definition(q, k, codes, vs, lens, _sees(masks, s), pool["table"].cpu(), 64), unit, max_len is None)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", SHAPES)
@pytest.mark.parametrize("first", [2.0 ** -126, 2.0 ** 80])
def test_ordinary_rows_beside_extreme_ones(s, h, hk, max_len, first):
    # the larger scales' rows are what the output is made of
    _gpu()
    lens = [1500, s + 400, 700]
    pool, k, codes, q, r = _rows(lens, s, h, hk, 41, 1.0)
    masks = _tree(3, s, 2)
    vs = torch.where(r < 150, first, 2.0 ** -7).double()[:, None].expand(-1, hk).contiguous()
    got = _attend(pool, codes, vs, q, lens, masks, max_len=max_len)
    torch.cuda.synchronize()
    check(got, definition(q, k, codes, vs, lens, _sees(masks, s), pool["table"].cpu(), 64), max(first, 2.0 ** -7),
          max_len is None)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,lens", [(1, 8, 2, [6000, 40, 130]), (4, 8, 8, [300, 2000, 5]), (7, 16, 2, [20000])])
@pytest.mark.parametrize("power", [-126, -110, -95, -89, 100])
def test_causal_attention(s, h, hk, lens, power):
    # csa_paged_attn over the same rows; long requests are cut between blocks and joined
    _gpu()
    pool, k, codes, q, _ = _rows(lens, s, h, hk, 43, 1.0)
    vs = torch.full((codes.shape[0], hk), 2.0 ** power, dtype=torch.float64)
    got = csa.PagedAttention(q.to(DEV), pool["k"], codes.to(torch.float8_e4m3fn).to(DEV),
                             torch.tensor(lens, dtype=torch.int32, device=DEV), table=pool["table"], block=64,
                             k_scale=pool["k_scale"], v_scale=vs.float().to(DEV))()
    torch.cuda.synchronize()
    chain = torch.ones(s, s, dtype=torch.bool).tril().expand(len(lens), s, s)
    check(got, definition(q, k, codes, vs, lens, chain, pool["table"].cpu(), 64), 2.0 ** power, True)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", SHAPES)
@pytest.mark.parametrize("at", [0, 3, 700, 1499])
def test_a_nan_key_beside_the_smallest_scales(s, h, hk, max_len, at):
    # it reaches out and lse, whether the rows that take the sum to fp32's end come before or behind it (enough
    # requests for a block to have several tiles of one)
    _gpu()
    lens = [1500 + s] * 80
    pool, k, codes, q, r = _rows(lens, s, h, hk, 47, 1.0)
    masks = _tree(len(lens), s, 2)
    vs = torch.where((r < at) == (at > 100), 2.0 ** -126, 1.0).double()[:, None].expand(-1, hk).contiguous()
    row = pool["table"][::2, at // 64].long() * 64 + at % 64
    pool["k_scale"][row] = float("nan")
    got = _attend(pool, codes, vs, q, lens, masks, max_len=max_len)
    torch.cuda.synchronize()
    for x in ("out", "lse"):
        assert got[x][::2].isnan().all() and got[x][1::2].isfinite().all(), x


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", SHAPES)
def test_tiny_values_from_append_to_attention(s, h, hk, max_len):
    """Keys and values as csa_kv_append writes them: values whose scale is the smallest that it writes."""
    _gpu()
    n, block = 600 + s, 64
    g = torch.Generator().manual_seed(3)
    pools = [torch.zeros(1024, hk, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros(1024, hk, device=DEV) for _ in range(2)]
    k, v = torch.randn(1, n, hk, 128, generator=g), torch.randn(1, n, hk, 128, generator=g) * 2.0 ** -119
    v[:, ::9] = 0.0
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    table = torch.randperm(16, generator=g).int()[None].to(DEV)
    csa.KvAppend(k.to(DEV), v.to(DEV), *pools, *scales, ctx_len=lens, table=table, block=block, rope_dim=0)()
    q = torch.randn(1, s, h, 128, generator=g).bfloat16()
    masks = _tree(1, s, 2)
    got = csa.TreeAttention(q.to(DEV), *pools, lens, masks.to(DEV), table=table, block=block, k_scale=scales[0],
                            v_scale=scales[1], max_len=max_len)()
    torch.cuda.synchronize()
    kk, codes = (p.cpu().view(torch.float8_e4m3fn).double() for p in pools)
    kk, vs = kk * scales[0].cpu().double()[..., None], scales[1].cpu().double()
    assert float(scales[1][scales[1] > 0].min()) == 2.0 ** -126
    check(got, definition(q, kk, codes, vs, [n], _sees(masks, s), table.cpu(), block), 2.0 ** -119, max_len is None)
