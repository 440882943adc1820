"""csa_tree_attn: attention of trees of drafted tokens over (paged) K / V pools, against a plain fp64 implementation.

Tolerances as derived in test_paged_attn.py: lse within LSE_TOL for normal inputs, out within u max |v| over the rows
that a draft sees (the rounding of the weights to bf16 or f16, u = 2^-8) and its own rounding u |out|.
"""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa
from test_paged_attn import _check, _pool

DEV = "cuda:0"


# ---------------------------------------------------------------------------
# CPU: refusals and masks

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, tree=0x10000, count=None, pos=None, **kw):
    a = 0x10000
    base = dict(B=2, S=5, heads=8, kv_heads=2, dim=128, kv_dtype=csa.CSA_DTYPE_BF16, win=0, max_len=1000,
                softmax_scale=0.0, block=64, table_stride=16, ctx_len=a, q=a, q_stride=1024, k=a, v=a, k_stride=256,
                v_stride=256, rows=100, k_scale=None, v_scale=None, scale_stride=0, off=None, table=a, out=a,
                out_stride=1024, lse=None, status=None, workspace=a, workspace_bytes=1 << 40)
    base.update(kw)
    return L.csa_tree_attn(ctypes.byref(csa.CTree(base=csa.CPaged(**base), tree=tree, count=count, pos=pos)), None)


def test_empty_batch_is_a_no_op(L):
    assert _call(L, B=0) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(tree=None), csa.CSA_ERR_INVALID_ARG),
    (dict(tree=0x10004), csa.CSA_ERR_INVALID_ARG),
    (dict(count=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(win=9), csa.CSA_ERR_INVALID_ARG),                   # no positions
    (dict(win=9, pos=0x10001), csa.CSA_ERR_INVALID_ARG),
    (dict(S=1025, heads=2, q_stride=256, out_stride=256), csa.CSA_ERR_UNSUPPORTED),
    (dict(S=0), csa.CSA_ERR_INVALID_ARG),
    (dict(dim=96), csa.CSA_ERR_UNSUPPORTED),
    (dict(heads=7), csa.CSA_ERR_INVALID_ARG),
    (dict(q=None), csa.CSA_ERR_INVALID_ARG),
    (dict(q_stride=1028), csa.CSA_ERR_INVALID_ARG),
    (dict(v_stride=260), csa.CSA_ERR_INVALID_ARG),
    (dict(table=None), csa.CSA_ERR_INVALID_ARG),
    (dict(softmax_scale=math.nan), csa.CSA_ERR_INVALID_ARG),
    (dict(kv_dtype=csa.CSA_DTYPE_FP8_E4M3), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_tree_attn(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    bf = torch.bfloat16
    q, k = torch.zeros(2, 5, 8, 128, dtype=bf), torch.zeros(100, 2, 128, dtype=bf)
    n, t, m = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 5, 1, dtype=torch.int64)
    good = dict(table=t, block=16)
    for args, kw in (((q, k, k, n, m.int()), good), ((q, k, k, n, m[:, :4]), good), ((q, k, k, n, m[:, :, 0]), good),
                     ((q, k, k, n, m), dict(good, win=4)), ((q, k, k, n, m), dict(good, count=n.long())),
                     ((q, k, k, n, m), dict(good, win=4, pos=n)), ((q.float(), k, k, n, m), good), ((q, k, k, n, m), {})):
        with pytest.raises(csa.CsaError):
            csa.TreeAttention(*args, **kw)


def _sees(masks, s):
    """bool [B, S, S] of packed masks."""
    t = torch.arange(s)
    return ((masks[:, :, t // 64] >> (t % 64)) & 1).bool()


def test_masks_of_parents():
    chain = torch.arange(70)[None] - 1
    assert torch.equal(_sees(csa.tree_masks(chain), 70)[0], torch.ones(70, 70).tril().bool())
    star = torch.full((1, 66), -1)
    assert torch.equal(_sees(csa.tree_masks(star), 66)[0], torch.eye(66).bool())
    p = torch.tensor([[-1, 0, 0, 2, 1, -1]], dtype=torch.int32)
    want = [[0], [0, 1], [0, 2], [0, 2, 3], [0, 1, 4], [5]]
    got = _sees(csa.tree_masks(p), 6)[0]
    assert [torch.nonzero(r)[:, 0].tolist() for r in got] == want
    for bad in (torch.tensor([[0, 0]]), torch.tensor([[-1, 1]]), torch.tensor([-1, 0]), torch.tensor([[-1.0]])):
        with pytest.raises(csa.CsaError):
            csa.tree_masks(bad)


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _tree(b, s, seed):
    g = torch.Generator().manual_seed(seed)
    parent = ((torch.rand(b, s, generator=g).sqrt() * (torch.arange(s) + 1)).long() - 1)
    return csa.tree_masks(torch.minimum(parent, torch.arange(s) - 1))


def _exact(q, k, v, lens, counts, sees, pos, table, block, win, scale):
    b, s, h, d = q.shape
    hk = k.shape[1]
    out = torch.zeros(b, s, h, d, dtype=torch.float64)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64)
    big = torch.zeros(b, s, h, 1, dtype=torch.float64)
    for i, n in enumerate(lens):
        m = s if counts is None else counts[i]
        if n <= 0 or m <= 0:
            continue
        r = torch.arange(n)
        rows = table[i].long()[r // block] * block + r % block
        first = n - m
        kk, vv = k[rows].repeat_interleave(h // hk, 1), v[rows].repeat_interleave(h // hk, 1)
        for t in range(m):
            at = min(max(int(pos[i, t]), first), n - 1) if win else 0
            keep = (r < first) & (r > at - win) if win else r < first
            own = sees[i, t, :m] if first >= 0 else sees[i, t, -first:m]
            keep[max(first, 0):] = own
            if not keep.any():
                continue
            sc = torch.einsum("hd,lhd->hl", q[i, t].double(), kk[keep]) * scale
            lse[i, t] = torch.logsumexp(sc, 1)
            out[i, t] = torch.einsum("hl,lhd->hd", torch.softmax(sc, 1), vv[keep])
            big[i, t] = vv[keep].abs().amax((0, 2))[:, None]
    return out, lse, big


def _run(lens, s, h, hk, d, block, win=0, fp8=False, seed=0, counts=None, masks=None, qstd=1.0, **kw):
    pool, k, v = _pool(lens, hk, d, block, seed, fp8)
    b = len(lens)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(b, s, h, d, generator=g) * qstd).bfloat16()
    masks = _tree(b, s, seed + 2) if masks is None else masks
    sees = _sees(masks, s)
    m = torch.tensor([s] * b if counts is None else counts)
    pos = ((torch.tensor(lens) - m)[:, None] + (sees.sum(2) - 1)).int()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = lambda t: t.to(DEV)
    want = _exact(q, k, v, lens, counts, sees, pos, pool["table"].cpu(), block, win, d ** -0.5)
    kk, vv = pool.pop("k"), pool.pop("v")
    for max_len in LONGEST:
        op = csa.TreeAttention(dev(q), kk, vv, torch.tensor(lens, dtype=torch.int32, device=DEV), dev(masks),
                               count=None if counts is None else dev(m.int()), pos=dev(pos) if win else None, win=win,
                               status=status, max_len=max_len, **pool, **kw)
        got = op()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        _check(got, want, (lens, s, h, hk, d, block, win, fp8, max_len))
    return op, want


# The bound on the lengths goes into the choice of the kernel: few and short requests, and what might be long ones.
LONGEST = (None, 1 << 20)

SHAPES = [  # drafts, heads, kv heads, dim, E4M3
    (1, 8, 8, 64, False), (5, 8, 8, 64, False), (8, 8, 2, 128, False), (3, 4, 1, 256, False), (7, 14, 2, 128, True),
    (16, 8, 1, 64, False), (33, 2, 2, 128, False), (21, 12, 2, 128, False), (9, 16, 2, 128, True), (64, 4, 1, 128, False),
    (64, 8, 2, 128, True), (70, 6, 2, 64, False), (40, 8, 1, 256, False), (17, 64, 4, 128, False), (100, 3, 1, 128, True),
    (130, 4, 2, 128, False), (200, 2, 1, 64, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
@pytest.mark.parametrize("block", [16, 48])
def test_trees_over_edge_lengths(s, h, hk, d, fp8, block):
    _gpu()
    _run([s, s + 1, s + 127, s + 128, 128, 129 + s, 256 + s, 300 + s, 0, 1000 + s, 255 + s, s + 2], s, h, hk, d, block, fp8=fp8,
         seed=s + d)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
def test_fewer_drafts_than_places(s, h, hk, d, fp8):
    # counts from none to all of them, and lengths below the count (drafts before the first row)
    _gpu()
    lens = [300, 40, 0, 129, 700, 5, 2, 130, 128]
    counts = [max(0, min(s, c)) for c in (s, 1, s, s // 2, 0, 5, s, 2, s - 1)]
    _run(lens, s, h, hk, d, 64, fp8=fp8, seed=s, counts=counts)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
@pytest.mark.parametrize("win", [1, 37, 200])
def test_windows(s, h, hk, d, fp8, win):
    _gpu()
    _run([s, 40 + s, 130 + s, 257 + s, 700], s, h, hk, d, 64, win=win, fp8=fp8, seed=s + win,
         counts=[s, max(1, s // 2), s, 1, s])


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 2, 128, False), (6, 4, 1, 256, False), (64, 4, 1, 128, False), (30, 16, 2, 64, False),
                                          (64, 8, 2, 128, True), (100, 8, 1, 128, True), (9, 4, 2, 128, True)])
@pytest.mark.parametrize("lens", [[20011], [9000, 200, 101, 12001, 640], [177] * 160])
def test_long_requests_are_split_and_joined(lens, s, h, hk, d, fp8):
    _gpu()
    if len(lens) > 5 and s * h > 300:
        lens = lens[:40]
    _run(lens, s, h, hk, d, 128, fp8=fp8, seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(16, 16, 2, 128, False), (33, 2, 2, 64, False), (40, 4, 2, 128, True), (64, 8, 2, 128, False),
                                          (21, 28, 4, 128, True), (37, 14, 2, 64, False)])
@pytest.mark.parametrize("block", [64, 24, 2])
def test_many_tiles_per_block_of_threads(s, h, hk, d, fp8, block):
    # every CTA takes several tiles of one request after another, and several requests
    _gpu()
    lens = [2200 - 61 * i for i in range(30)] + [130] * 10
    _run(lens, s, h, hk, d, block, fp8=fp8, seed=s, counts=[s if i % 3 else max(1, s // 2) for i in range(40)])


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", SHAPES)
def test_masks_that_leave_rows_empty_or_full(s, h, hk, d, fp8):
    # no bits, every bit (those of drafts behind the count too), and only another draft's
    _gpu()
    words = -(-s // 64)
    masks = torch.zeros(6, s, words, dtype=torch.int64)
    masks[1] = masks[4] = -1
    masks[2, :, 0] = masks[5, :, 0] = 1
    masks[3, 0] = -1
    _run([s, s, s + 3, s, 140 + s, 300 + s], s, h, hk, d, 16, fp8=fp8, counts=[s, s, s, max(1, s - 2), max(1, s // 2), s], masks=masks)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 2, 128, False), (64, 4, 1, 128, False), (64, 8, 2, 128, True), (40, 4, 2, 64, False)])
@pytest.mark.parametrize("qstd", [0.0, 16.0])
def test_flat_and_peaked_weights(s, h, hk, d, fp8, qstd):
    _gpu()
    _run([2000, 700, 129], s, h, hk, d, 64, qstd=qstd, fp8=fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 2, 128, False), (64, 4, 1, 128, False), (8, 8, 2, 128, True), (64, 8, 2, 128, True)])
@pytest.mark.parametrize("max_len", LONGEST)
def test_a_chain_is_the_causal_attention(s, h, hk, d, fp8, max_len):
    _gpu()
    lens = [s, 300, 1111]
    pool, _, _ = _pool(lens, hk, d, 64, 4, fp8)
    q = torch.randn(3, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    k, v = pool.pop("k"), pool.pop("v")
    chain = csa.tree_masks((torch.arange(s) - 1).repeat(3, 1)).to(DEV)
    got = csa.TreeAttention(q, k, v, n, chain, max_len=max_len, **pool)()
    ref = csa.PagedAttention(q, k, v, n, **pool)()
    torch.cuda.synchronize()
    big = 6.0   # normal values
    _check(got, (ref["out"].cpu().double(), ref["lse"].cpu().double(), torch.full((3, s, h, 1), 2 * big)))


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(6, 8, 2, 128, False), (64, 4, 2, 128, False), (6, 8, 2, 128, True), (64, 8, 2, 128, True),
                                          (40, 4, 1, 64, False), (12, 8, 1, 256, False), (64, 8, 2, 128, False),
                                          (80, 8, 2, 64, False)])
@pytest.mark.parametrize("what", ["nan", "inf", "key"])
@pytest.mark.parametrize("max_len", LONGEST)
def test_nan_in_a_row_reaches_only_the_drafts_that_see_it(s, h, hk, d, fp8, what, max_len):
    """Drafts' rows (seen by their descendants) and a row at the window's edge hold NaN or infinity: the others' outputs
    do not change by a bit."""
    _gpu()
    lens, win, block = [100 + s, 37 + s, 300 + s], 33, 16
    pool, _, _ = _pool(lens, hk, d, block, 11, fp8)
    q = torch.randn(3, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    masks = _tree(3, s, 5)
    sees = _sees(masks, s)
    pos = ((torch.tensor(lens) - s)[:, None] + sees.sum(2) - 1).int()
    op = csa.TreeAttention(q, pool["k"], pool["v"], n, masks.to(DEV), pos=pos.to(DEV), win=win, table=pool["table"], block=block,
                           k_scale=pool.get("k_scale"), v_scale=pool.get("v_scale"), max_len=max_len)
    clean = {x: t.clone() for x, t in op().items()}
    torch.cuda.synchronize()
    touched = torch.zeros(3, s, dtype=torch.bool)
    for i, length in enumerate(lens):
        first = length - s
        for r in (length - 1, length - s // 2, first - win + 2):
            row = int(pool["table"][i, r // block]) * block + r % block
            if fp8:
                if what == "key":
                    pool["k_scale"][row] = float("nan")
                elif what == "nan":
                    pool["v"][row, :, 3::7] = 0x7f
                else:
                    pool["v_scale"][row] = float("inf")
            else:
                (pool["k"] if what == "key" else pool["v"])[row, :, 3::7] = float("inf" if what == "inf" else "nan")
            touched[i] |= sees[i, :, r - first] if r >= first else r > pos[i] - win
    got = op()
    torch.cuda.synchronize()
    # A V scale outside 2^-24 .. 2^24 near a row changes how the softmax's sum is formed: exp2(s - ref) in place of
    # exp2(s + lv - ref) 2^-lv with lv = log2 of the row's scale.  For |s| + |lv| + |ref| <= 64 each exponent is off by two
    # roundings of 2^-24 64 (2^-17 log2 units, 5.3e-6 relative), ex2 by 2^-22 and the product by 2^-24: lse by less than
    # 2 (5.3e-6 + 3e-7) < 1.2e-5, and out's quotient as much, one step of bf16 (2^-7) once it is rounded.
    apart = fp8 and what == "inf"
    for x, tol in (("out", 2.0 ** -7), ("lse", 1.2e-5)):
        a, b = got[x].cpu()[~touched].double(), clean[x].cpu()[~touched].double()
        assert torch.equal(a, b) or (apart and ((a - b).abs() <= tol * (b.abs() if x == "out" else 1)).all()), x
    hit = got["out"].cpu()[touched]
    if what == "key" or (fp8 and what == "inf"):
        assert hit.isnan().all()
    else:
        assert not torch.isfinite(hit[..., 3::7]).any()
        rest = torch.ones(d, dtype=torch.bool)
        rest[3::7] = False
        assert torch.equal(hit[..., rest], clean["out"].cpu()[touched][..., rest])
        assert torch.equal(got["lse"].cpu(), clean["lse"].cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(6, 8, 2, 128, False), (64, 4, 2, 128, False), (64, 8, 2, 128, True)])
@pytest.mark.parametrize("long", [False, True])
def test_bad_lengths_counts_and_pages(s, h, hk, d, fp8, long):
    _gpu()
    lens, block = [100 + s, 300 + s, 200 + s, 50 + s], 16
    pool, k, v = _pool(lens, hk, d, block, 5, fp8)
    q = torch.randn(4, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    masks = _tree(4, s, 5)
    sees = _sees(masks, s)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    max_len = LONGEST[1] if long else 300 + s

    def run(n, c, table):
        status.zero_()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        got = csa.TreeAttention(q.to(DEV), pool["k"], pool["v"], i32(n), masks.to(DEV), count=i32(c), table=table, block=block,
                                k_scale=pool.get("k_scale"), v_scale=pool.get("v_scale"), status=status, max_len=max_len)()
        torch.cuda.synchronize()
        return got, int(status.item())

    def exact(n, c, kk=k, vv=v):
        return _exact(q, kk, vv, n, c, sees, None, pool["table"].cpu(), block, 0, d ** -0.5)

    c = [s] * 4
    got, st = run([100 + s, max_len + 1, -1, 50 + s], c, pool["table"])
    assert st == 1
    _check(got, exact([100 + s, 0, 0, 50 + s], c))
    got, st = run(lens, [s + 1, -1, s, 0], pool["table"])
    assert st == 1
    _check(got, exact(lens, [0, 0, s, 0]))
    # an unmapped and an outside block: their rows weigh as zeros
    table = pool["table"].clone()
    kk, vv = k.clone(), v.clone()
    for i, j, bad in ((1, 3, -1), (2, 2, 1 << 26)):
        row = int(table[i, j]) * block
        kk[row:row + block] = vv[row:row + block] = 0
        table[i, j] = bad
    got, st = run(lens, c, table)
    assert st == 1
    _check(got, exact(lens, c, kk, vv))


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", [(5, 8, 2, 600), (64, 8, 2, 600), (64, 8, 2, 1 << 20)])
def test_offsets_strides_and_outside_columns(s, h, hk, max_len):
    _gpu()
    lens, d = [200, 64 + s, 517], 128
    g = torch.Generator().manual_seed(3)
    pool = torch.full((900 + s, 2 * hk + 1, d), float("nan"))
    off = torch.tensor([5, 230, 320 + s])
    for b, n in enumerate(lens):
        pool[off[b]:off[b] + n, :2 * hk] = torch.randn(n, 2 * hk, d, generator=g)
    pool = pool.bfloat16().to(DEV)
    wide = torch.randn(3, s, h + 4, d, generator=g).bfloat16().to(DEV)
    outw = torch.full((3, s, h + 4, d), 7.0, dtype=torch.bfloat16, device=DEV)
    masks = _tree(3, s, 6)
    got = csa.TreeAttention(wide[:, :, 2:2 + h], pool[:, :hk], pool[:, hk:2 * hk],
                            torch.tensor(lens, dtype=torch.int32, device=DEV), masks.to(DEV), off=off.to(DEV), max_len=max_len,
                            out=outw[:, :, 4:], scale=0.05)()
    torch.cuda.synchronize()
    table = torch.arange(900 + s, dtype=torch.int32)[None] + off[:, None].int()
    want = _exact(wide[:, :, 2:2 + h].cpu(), pool[:, :hk].cpu().double(), pool[:, hk:2 * hk].cpu().double(), lens, None,
                  _sees(masks, s), None, table, 1, 0, 0.05)
    _check(got, want)
    assert (outw[:, :, :4] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,max_len", [(4, 4, 2, None), (48, 4, 2, 1 << 20)])
def test_rows_far_into_a_large_pool(s, h, hk, max_len):
    """Rows beyond 2^32 bytes and 2^31 elements of the pool."""
    _gpu()
    d, block, rows = 128, 64, 64 * 140000
    k = torch.empty(rows, hk, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    lens = [150 + s, 90 + s]
    table = torch.tensor([[139999, 1, 139000, 70000, 3], [139997, 131073, 5, 0, 2]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    used = table.view(-1).long()[:, None] * block + torch.arange(block)
    ck, cv = (torch.randn(used.numel(), hk, d, generator=g).bfloat16() for _ in range(2))
    k[used.view(-1).to(DEV)], v[used.view(-1).to(DEV)] = ck.to(DEV), cv.to(DEV)
    q = torch.randn(2, s, h, d, generator=g).bfloat16()
    masks = _tree(2, s, 6)
    got = csa.TreeAttention(q.to(DEV), k, v, torch.tensor(lens, dtype=torch.int32, device=DEV), masks.to(DEV),
                            table=table.to(DEV), block=block, max_len=max_len)()
    torch.cuda.synchronize()
    local = torch.arange(10, dtype=torch.int32).view(2, 5)
    _check(got, _exact(q, ck.double(), cv.double(), lens, None, _sees(masks, s), None, local, block, 0, d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 2, 128, False), (64, 8, 2, 128, False), (64, 8, 2, 128, True)])
@pytest.mark.parametrize("max_len", LONGEST)
def test_captured_replays_follow_the_device_and_repeat_exactly(s, h, hk, d, fp8, max_len):
    _gpu()
    lens = [700, 300, 2000, 64 + s]
    pool, k, v = _pool(lens, hk, d, 64, 8, fp8)
    q = torch.randn(4, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    masks = _tree(4, s, 5)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c = torch.full((4,), s, dtype=torch.int32, device=DEV)
    dm = masks.to(DEV)
    kk, vv = pool.pop("k"), pool.pop("v")
    op = csa.TreeAttention(q.to(DEV), kk, vv, n, dm, count=c, max_len=max_len, **pool)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        op()
    lens2, counts2, masks2 = [500, 0, 1999, 64], [s, s, 3, s - 1], _tree(4, s, 77)
    for ln, cn, mk in ((lens, [s] * 4, masks), (lens2, counts2, masks2), (lens, [s] * 4, masks)):
        n.copy_(torch.tensor(ln))
        c.copy_(torch.tensor(cn))
        dm.copy_(mk)
        g.replay()
        torch.cuda.synchronize()
        first = {x: t.clone() for x, t in op._out.items()}
        _check(first, _exact(q, k, v, ln, cn, _sees(mk, s), None, pool["table"].cpu(), 64, 0, d ** -0.5))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(first[x], op._out[x]) for x in first)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,s,h,hk,d,fp8", [([1500, 1024, 1023], 1024, 2, 1, 64, False), ([1300], 1023, 4, 4, 128, True),
                                               ([700, 90], 3, 128, 1, 128, False), ([700, 90], 2, 127, 1, 64, False),
                                               ([300, 90], 2, 130, 1, 128, False), ([300, 90], 5, 77, 1, 128, True)])
def test_the_most_drafts_and_heads_per_row(lens, s, h, hk, d, fp8):
    _gpu()
    _run(lens, s, h, hk, d, 64, fp8=fp8, seed=s + h, counts=[min(s, n) for n in lens])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_two_calls_at_once(fp8):
    """Calls on two streams with workspaces of their own, many times over each other: as each alone."""
    _gpu()
    ops, alone, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, (s, h, hk) in enumerate(((64, 8, 2), (16, 32, 4))):
        lens = [2000 - 300 * i, 700, 64 + s, 1200]
        pool, _, _ = _pool(lens, hk, 128, 64, 20 + i, fp8)
        q = torch.randn(4, s, h, 128, generator=torch.Generator().manual_seed(i)).bfloat16().to(DEV)
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        op = csa.TreeAttention(q, pool.pop("k"), pool.pop("v"), n, _tree(4, s, i).to(DEV), max_len=1 << 20, **pool)
        alone.append({x: t.clone() for x, t in op().items()})
        ops.append(op)
    torch.cuda.synchronize()
    for _ in range(20):
        for op, st in zip(ops, streams):
            with torch.cuda.stream(st):
                op()
    torch.cuda.synchronize()
    for op, want in zip(ops, alone):
        assert all(torch.equal(op._out[x], want[x]) for x in want)


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", LONGEST)
@pytest.mark.parametrize("scale", [2.0 ** 80, 2.0 ** -80])
@pytest.mark.parametrize("s,h,hk", [(64, 8, 2), (5, 8, 2)])
def test_scales_of_any_size(s, h, hk, scale, max_len):
    """E4M3 rows whose V scales are all huge or small (flat weights add up), or a few huge among ordinary ones."""
    _gpu()
    lens, block = [3000, s + 100, 700], 64
    pool, k, v = _pool(lens, hk, 128, block, 31, True)
    q = (torch.randn(3, s, h, 128, generator=torch.Generator().manual_seed(1)) * 0.1).bfloat16()
    masks = _tree(3, s, 2)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kk, vv = pool.pop("k"), pool.pop("v")
    base = pool.pop("v_scale")
    for mix in (False, True):
        rows = torch.zeros(base.shape[0], dtype=torch.bool)
        rows[::7 if mix else 1] = True
        factor = torch.where(rows, scale, 1.0).double()
        op = csa.TreeAttention(q.to(DEV), kk, vv, n, masks.to(DEV), max_len=max_len,
                               v_scale=base * factor.float().to(DEV)[:, None], **pool)
        got = op()
        torch.cuda.synchronize()
        want = _exact(q, k, v * factor[:, None, None], lens, None, _sees(masks, s), None, pool["table"].cpu(), block, 0, 128 ** -0.5)
        _check(got, want, (s, scale, mix, max_len))
