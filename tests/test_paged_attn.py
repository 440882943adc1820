"""csa_paged_attn: dense causal attention of each request's newest tokens over (paged) K / V pools, against a
plain fp64 implementation.

Tolerances.  Scores are fp32 sums of exact bf16 products: with |scale q . k| terms adding up to A they are off
by at most (dim + 4) 2^-23 A, so lse is too, plus 2^-22 for exp2 and n 2^-24 for the sum of n weights (lse is a
convex function of the scores with gradient 1) and 2^-23 |lse| for its rounding; the tests' scores have A below
64 for dim up to 256, so 64 (260) 2^-23 = 2e-3 would be the worst case and 2e-4 holds with a wide margin
for the random inputs here, whose rounding errors add up like a random walk (sqrt(dim) 2^-24 A < 4e-5 each).
A weight is rounded to bf16 (u = 2^-8) before the product with v: |out - exact| <= u max_r |v| over the visible
rows (a convex combination of rows, each weight off by u relative), plus the output's own u |out|; with the
E4M3 pools the weight times the row's scale is what is rounded, the same bound.
"""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa

DEV = "cuda:0"
U = 2.0 ** -8
LSE_TOL = 2e-4


# ---------------------------------------------------------------------------
# CPU: refusals

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, **kw):
    a = 0x10000
    base = dict(B=2, S=1, heads=8, kv_heads=2, dim=128, kv_dtype=csa.CSA_DTYPE_BF16, win=0, max_len=1000,
                softmax_scale=0.0, block=64, table_stride=16, ctx_len=a, q=a, q_stride=1024, k=a, v=a, k_stride=256,
                v_stride=256, rows=100, k_scale=None, v_scale=None, scale_stride=0, off=None, table=a, out=a,
                out_stride=1024, lse=None, status=None, workspace=a, workspace_bytes=1 << 40)
    base.update(kw)
    return L.csa_paged_attn(ctypes.byref(csa.CPaged(**base)), None)


FP8 = dict(kv_dtype=csa.CSA_DTYPE_FP8_E4M3, k_scale=0x10000, v_scale=0x10000, scale_stride=2)


def test_empty_batch_is_a_no_op(L):
    assert _call(L, B=0) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(kv_dtype=7), csa.CSA_ERR_UNSUPPORTED),
    (dict(dim=96), csa.CSA_ERR_UNSUPPORTED),
    (dict(FP8, dim=64), csa.CSA_ERR_UNSUPPORTED),
    (dict(B=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(S=0), csa.CSA_ERR_INVALID_ARG),
    (dict(heads=7), csa.CSA_ERR_INVALID_ARG),                # not a multiple of kv_heads
    (dict(kv_heads=0), csa.CSA_ERR_INVALID_ARG),
    (dict(win=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(max_len=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(max_len=(1 << 30) + 1), csa.CSA_ERR_UNSUPPORTED),
    (dict(q=None), csa.CSA_ERR_INVALID_ARG),
    (dict(q=0x10008), csa.CSA_ERR_INVALID_ARG),
    (dict(q_stride=1023), csa.CSA_ERR_INVALID_ARG),
    (dict(q_stride=1028), csa.CSA_ERR_INVALID_ARG),
    (dict(out=None), csa.CSA_ERR_INVALID_ARG),
    (dict(out_stride=1000), csa.CSA_ERR_INVALID_ARG),
    (dict(k=None), csa.CSA_ERR_INVALID_ARG),
    (dict(v=0x10004), csa.CSA_ERR_INVALID_ARG),
    (dict(k_stride=255), csa.CSA_ERR_INVALID_ARG),
    (dict(v_stride=260), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, v_stride=264), csa.CSA_ERR_INVALID_ARG),      # 264 bytes
    (dict(FP8, k_scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, scale_stride=1), csa.CSA_ERR_INVALID_ARG),
    (dict(rows=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(rows=1 << 31), csa.CSA_ERR_INVALID_ARG),
    (dict(ctx_len=None), csa.CSA_ERR_INVALID_ARG),
    (dict(table=None), csa.CSA_ERR_INVALID_ARG),             # neither table nor off
    (dict(block=0), csa.CSA_ERR_INVALID_ARG),
    (dict(table_stride=0), csa.CSA_ERR_INVALID_ARG),
    (dict(off=0x10004, table=None), csa.CSA_ERR_INVALID_ARG),
    (dict(lse=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(workspace=0x10008), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_paged_attn(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    bf = torch.bfloat16
    q, k = torch.zeros(2, 1, 8, 128, dtype=bf), torch.zeros(100, 2, 128, dtype=bf)
    n, t = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    good = dict(table=t, block=16)
    for args, kw in (((q.float(), k, k, n), good), ((q, k, k.float(), n), good), ((q, k, k[:50], n), good),
                     ((q, k, k, n.long()), good), ((q, k, k, n), {}), ((q, k, k, n), dict(good, off=n.long())),
                     ((q, k, k, n), dict(table=t.long(), block=16)), ((q, k, k, n), dict(off=n.long())),
                     ((q, k.byte(), k.byte(), n), good), ((q, k, k, n), dict(good, k_scale=torch.zeros(100, 2))),
                     ((q, k, k, n), dict(good, lse=torch.zeros(2, 8))),
                     ((q, k, k, n), dict(good, out=torch.zeros(2, 1, 8, 64, dtype=bf))),
                     ((torch.zeros(2, 1, 8, 256, dtype=bf)[..., ::2], k, k, n), good)):
        with pytest.raises(csa.CsaError):
            csa.PagedAttention(*args, **kw)


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _pool(lens, hk, d, block, seed, fp8=False, spare=3):
    """K and V pools with each request's rows in shuffled blocks; every other row is NaN.
    Returns a dict of device tensors and the dense fp64 rows."""
    g = torch.Generator().manual_seed(seed)
    nblk = [-(-n // block) for n in lens]
    total = sum(nblk) + spare
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(1, max(nblk))), -1, dtype=torch.int32)
    at = 0
    k, v = (torch.full((total * block, hk, d), float("nan")) for _ in range(2))
    for b, n in enumerate(lens):
        table[b, :nblk[b]] = perm[at:at + nblk[b]].int()
        at += nblk[b]
        if n:
            r = torch.arange(n)
            rows = table[b].long()[r // block] * block + r % block
            k[rows] = torch.randn(n, hk, d, generator=g)
            v[rows] = torch.randn(n, hk, d, generator=g)
    out = dict(table=table.to(DEV), block=block)
    if fp8:
        for name, t in (("k", k), ("v", v)):
            amax = t.abs().amax(2)
            scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            codes = (t / scale[..., None]).to(torch.float8_e4m3fn)
            out[name], out[name + "_scale"] = codes.view(torch.uint8).to(DEV), scale.to(DEV)
        k, v = (out[x].cpu().view(torch.float8_e4m3fn).double() * out[x + "_scale"].cpu().double()[..., None]
                for x in ("k", "v"))
    else:
        out["k"], out["v"] = k.bfloat16().to(DEV), v.bfloat16().to(DEV)
        k, v = out["k"].cpu().double(), out["v"].cpu().double()
    return out, k, v


def _exact(q, k, v, lens, table, block, win, scale):
    b, s, h, d = q.shape
    hk = k.shape[1]
    out = torch.zeros(b, s, h, d, dtype=torch.float64)
    lse = torch.full((b, s, h), -math.inf, dtype=torch.float64)
    big = torch.zeros(b, s, h, 1, dtype=torch.float64)
    for i, n in enumerate(lens):
        r = torch.arange(max(n, 0))
        rows = table[i].long()[r // block] * block + r % block if n > 0 else r
        for t in range(s):
            pos = n - s + t
            if pos < 0:
                continue
            at = rows[max(0, pos - win + 1) if win else 0:pos + 1]
            kk, vv = k[at].repeat_interleave(h // hk, 1), v[at].repeat_interleave(h // hk, 1)
            sc = torch.einsum("hd,lhd->hl", q[i, t].double(), kk) * scale
            lse[i, t] = torch.logsumexp(sc, 1)
            out[i, t] = torch.einsum("hl,lhd->hd", torch.softmax(sc, 1), vv)
            big[i, t] = vv.abs().amax((0, 2))[:, None]
    return out, lse, big


def _check(got, want, what=""):
    out, lse, big = want
    o, l = got["out"].cpu().double(), got["lse"].cpu().double()
    empty = torch.isinf(lse)
    assert (l[empty] == -math.inf).all() and (o[empty] == 0).all(), what
    err = (l - lse)[~empty].abs()
    assert err.numel() == 0 or err.max() <= LSE_TOL, (what, float(err.max()))
    tol = 1.01 * U * (big + out.abs()) + 1e-5 * big
    assert ((o - out).abs() <= tol).all(), (what, float(((o - out).abs() / tol.clamp_min(1e-30)).max()))


def _run(lens, s, h, hk, d, block, win=0, fp8=False, seed=0, qstd=1.0, **kw):
    pool, k, v = _pool(lens, hk, d, block, seed, fp8)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), s, h, d, generator=g) * qstd).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    op = csa.PagedAttention(q.to(DEV), pool.pop("k"), pool.pop("v"), n, win=win, status=status, **pool, **kw)
    got = op()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = _exact(q, k, v, lens, pool["table"].cpu(), block, win, d ** -0.5)
    _check(got, want, (lens, s, h, hk, d, block, win, fp8))
    return op, want


EDGE = [1, 2, 15, 16, 17, 127, 128, 129, 0, 255, 256, 300, 1, 0, 1000, 63]


@pytest.mark.gpu
@pytest.mark.parametrize("h,hk,d,fp8", [(8, 8, 64, False), (8, 2, 128, False), (4, 1, 256, False), (6, 2, 128, True),
                                        (48, 2, 128, False), (34, 2, 64, False), (40, 1, 256, False), (64, 2, 128, True)])
@pytest.mark.parametrize("block", [16, 48])
def test_single_tokens_over_edge_lengths(h, hk, d, fp8, block):
    _gpu()
    _run(EDGE, 1, h, hk, d, block, fp8=fp8, seed=h + d)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(2, 8, 8, 64, False), (4, 8, 2, 128, False), (3, 4, 1, 256, False),
                                          (5, 14, 2, 128, True), (7, 12, 2, 128, False), (8, 16, 1, 64, False),
                                          (20, 4, 4, 128, True)])
@pytest.mark.parametrize("win", [0, 1, 37, 200])
def test_several_tokens_and_windows(s, h, hk, d, fp8, win):
    # lengths below S leave the first tokens without a row
    _gpu()
    _run([0, 1, 2, 5, 16, 40, 130, 257, 700], s, h, hk, d, 64, win=win, fp8=fp8, seed=s + win)


@pytest.mark.gpu
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (256, False), (128, True)])
@pytest.mark.parametrize("lens", [[20011], [1], [9000, 3, 1, 12001, 640], [77] * 300, [5, 0, 130] * 150])
def test_long_requests_are_split_and_joined(lens, d, fp8):
    _gpu()
    _run(lens, 1, 4, 2, d, 128, fp8=fp8, seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_a_window_of_a_long_request(fp8):
    _gpu()
    _run([20011, 5000, 100], 2, 4, 1, 128, 64, win=4097, fp8=fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("qstd", [0.0, 16.0])
def test_flat_and_peaked_weights(qstd):
    # peaked: a few weights dominate and the reference maximum moves often; scores have |q . k| scale up to
    # about 16 x 5, A (see above) up to 16 x 9: LSE_TOL still covers 128 random roundings of 2^-24 of A
    _gpu()
    _run([3000, 700, 129], 1, 8, 2, 128, 64, qstd=qstd)


@pytest.mark.gpu
def test_offsets_strides_and_one_pool_for_both():
    # contiguous rows by offset, K and V interleaved in one pool with extra columns, q and out slices of wider
    # rows; nothing outside out's columns is written
    _gpu()
    lens, h, hk, d = [200, 64, 517], 8, 2, 128
    g = torch.Generator().manual_seed(3)
    pool = torch.full((900, 2 * hk + 1, d), float("nan"))
    off = torch.tensor([5, 230, 310])
    for b, n in enumerate(lens):
        pool[off[b]:off[b] + n, :2 * hk] = torch.randn(n, 2 * hk, d, generator=g)
    pool = pool.bfloat16().to(DEV)
    wide = torch.randn(3, 1, h + 4, d, generator=g).bfloat16().to(DEV)
    outw = torch.full((3, 1, h + 4, d), 7.0, dtype=torch.bfloat16, device=DEV)
    op = csa.PagedAttention(wide[:, :, 2:2 + h], pool[:, :hk], pool[:, hk:2 * hk],
                            torch.tensor(lens, dtype=torch.int32, device=DEV), off=off.to(DEV), max_len=600,
                            out=outw[:, :, 4:], scale=0.05)
    got = op()
    torch.cuda.synchronize()
    k, v = pool[:, :hk].cpu().double(), pool[:, hk:2 * hk].cpu().double()
    out, lse, big = (torch.zeros(3, 1, h, d, dtype=torch.float64), torch.zeros(3, 1, h, dtype=torch.float64),
                     torch.zeros(3, 1, h, 1, dtype=torch.float64))
    for i, n in enumerate(lens):
        rows = torch.arange(n) + off[i]
        kk, vv = k[rows].repeat_interleave(4, 1), v[rows].repeat_interleave(4, 1)
        sc = torch.einsum("hd,lhd->hl", wide[i, 0, 2:2 + h].cpu().double(), kk) * 0.05
        lse[i, 0], out[i, 0] = torch.logsumexp(sc, 1), torch.einsum("hl,lhd->hd", torch.softmax(sc, 1), vv)
        big[i, 0] = vv.abs().amax((0, 2))[:, None]
    _check(got, (out, lse, big))
    assert (outw[:, :, :4] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("win", [0, 20])
def test_nan_in_a_row_reaches_only_the_tokens_that_see_it(fp8, win):
    # the last rows (seen by the last tokens only) and, with a window, the first rows (seen by the first tokens
    # only) hold NaN and infinity: the other tokens' outputs do not change by a bit
    _gpu()
    lens, s, h, hk, d, block = [100, 37], 4, 8, 2, 128, 16
    pool, _, _ = _pool(lens, hk, d, block, 11, fp8)
    q = torch.randn(2, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    op = csa.PagedAttention(q, pool["k"], pool["v"], n, table=pool["table"], block=block, win=win,
                            k_scale=pool.get("k_scale"), v_scale=pool.get("v_scale"))
    clean = {x: t.clone() for x, t in op().items()}
    torch.cuda.synchronize()
    for i, length in enumerate(lens):
        for r in [length - 1] + ([length - s - win + 1] if win else []):
            row = int(pool["table"][i, r // block]) * block + r % block
            if fp8:
                pool["k_scale"][row], pool["v_scale"][row] = float("nan"), float("inf")
            else:
                pool["k"][row], pool["v"][row] = float("nan"), float("inf")
    got = op()
    torch.cuda.synchronize()
    sees = [3] + ([0] if win else [])
    for t in range(s):
        if t in sees:
            assert torch.isnan(got["out"][:, t]).all() and torch.isnan(got["lse"][:, t]).all()
        else:
            assert torch.equal(got["out"][:, t], clean["out"][:, t]) and torch.equal(got["lse"][:, t], clean["lse"][:, t])


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported_and_leave_the_others_alone():
    _gpu()
    lens, h, hk, d, block = [100, 300, 200, 50], 4, 2, 128, 16
    pool, k, v = _pool(lens, hk, d, block, 5)
    q = torch.randn(4, 1, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    want = _exact(q, k, v, lens, pool["table"].cpu(), block, 0, d ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(n, table):
        status.zero_()
        got = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], torch.tensor(n, dtype=torch.int32, device=DEV),
                                 table=table, block=block, status=status, max_len=304)()
        torch.cuda.synchronize()
        return got, int(status.item())

    got, st = run([100, 305, -1, 50], pool["table"])        # above max_len, negative
    assert st == 1
    assert (got["out"][1:3] == 0).all() and (got["lse"][1:3] == -math.inf).all()
    keep = torch.tensor([0, 3])
    _check({x: t.cpu()[keep] for x, t in got.items()}, tuple(t[keep] for t in want))
    for bad in (-1, 1 << 20):                               # unmapped, outside the pool
        t = pool["table"].clone()
        t[1, 3] = bad
        got, st = run(lens, t)
        assert st == 1 and torch.isfinite(got["out"]).all()
        keep = torch.tensor([0, 2, 3])
        _check({x: y.cpu()[keep] for x, y in got.items()}, tuple(y[keep] for y in want))
    got, st = run(lens, pool["table"])
    assert st == 0
    _check(got, want)


@pytest.mark.gpu
def test_a_graph_follows_the_lengths_and_repeats_bit_for_bit():
    _gpu()
    lens, h, hk, d, block = [4000, 100, 2500, 0], 8, 2, 128, 64
    pool, k, v = _pool(lens, hk, d, block, 6)
    q = torch.randn(4, 1, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    op = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], n, table=pool["table"], block=block)
    first = {x: t.clone() for x, t in op().items()}
    for _ in range(10):
        again = op()
    torch.cuda.synchronize()
    assert all(torch.equal(again[x], first[x]) for x in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op()
    for now in ([1, 100, 2500, 0], lens, [3999, 0, 1, 0]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        _check(op._out, _exact(q, k, v, now, pool["table"].cpu(), block, 0, d ** -0.5), now)
    n.copy_(torch.tensor(lens, dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], n, table=pool["table"], block=block)
    side.wait_stream(torch.cuda.current_stream())
    other(stream=side)                                      # its own workspace: beside a call on this stream
    op()
    torch.cuda.synchronize()
    assert all(torch.equal(other._out[x], first[x]) and torch.equal(op._out[x], first[x]) for x in first)


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    # a pool of more than 2^31 elements: the request's last blocks lie behind it
    _gpu()
    rows, hk, d, block = 2_200_000, 8, 128, 64
    k = torch.zeros(rows, hk, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(rows, hk, d, dtype=torch.bfloat16, device=DEV)
    n = 300
    last = rows // block - 1
    table = torch.tensor([[last, 3, last - 7, 1, last - 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    r = torch.arange(n)
    at = table[0].long()[r // block] * block + r % block
    kk, vv = torch.randn(n, hk, d, generator=g).bfloat16(), torch.randn(n, hk, d, generator=g).bfloat16()
    k[at.to(DEV)], v[at.to(DEV)] = kk.to(DEV), vv.to(DEV)
    q = torch.randn(1, 1, 16, d, generator=g).bfloat16()
    got = csa.PagedAttention(q.to(DEV), k, v, torch.tensor([n], dtype=torch.int32, device=DEV), table=table.to(DEV),
                             block=block)()
    torch.cuda.synchronize()
    dense = torch.arange(5, dtype=torch.int32)[None]
    pad = torch.zeros(20, hk, d).double()
    _check(got, _exact(q, torch.cat([kk.double(), pad]), torch.cat([vv.double(), pad]), [n], dense, block, 0, d ** -0.5))


@pytest.mark.gpu
def test_a_window_over_everything_is_none_and_no_lse():
    _gpu()
    lens, h, hk, d, block = [3000, 40], 4, 2, 128, 64
    pool, _, _ = _pool(lens, hk, d, block, 8)
    q = torch.randn(2, 1, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    args = (q, pool["k"], pool["v"], n)
    kw = dict(table=pool["table"], block=block)
    base = csa.PagedAttention(*args, **kw)()["out"].clone()
    for win in (3008, 5000, (1 << 31) - 1):
        got = csa.PagedAttention(*args, win=win, lse=False, **kw)()
        assert list(got) == ["out"] and torch.equal(got["out"], base)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_many_tokens_of_one_request(fp8):
    # a prompt's chunk: more query rows than one unit holds
    _gpu()
    _run([70, 64, 200], 64, 4, 2, 128, 16, fp8=fp8, seed=4)


@pytest.mark.gpu
def test_e4m3_scales_far_apart_zero_and_negative():
    # the weights take the V rows' scales in: rows with scales from 1e-12 to 1e12, zero and negative ones
    _gpu()
    lens, h, hk, d, block = [700], 6, 2, 128, 64
    pool, _, _ = _pool(lens, hk, d, block, 9, True)
    rows = pool["v_scale"].shape[0]
    g = torch.Generator().manual_seed(3)
    f = 10.0 ** torch.randint(-12, 13, (rows, 1), generator=g).float()
    f[::5] = 0.0
    f[1::5] *= -1
    pool["v_scale"] = (pool["v_scale"] * f.to(DEV)).contiguous()
    q = (torch.randn(1, 1, h, d, generator=g) * 3).bfloat16()
    got = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                             table=pool["table"], block=block, k_scale=pool["k_scale"], v_scale=pool["v_scale"])()
    torch.cuda.synchronize()
    k, v = (pool[x].cpu().view(torch.float8_e4m3fn).double() * pool[x + "_scale"].cpu().double()[..., None] for x in "kv")
    want = _exact(q, k, v, lens, pool["table"].cpu(), block, 0, d ** -0.5)
    _check(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_e4m3_queries_of_any_size(scale):
    # a query row is scaled to f16's range by a power of two: rows far outside it, keys scaled back
    _gpu()
    lens, h, hk, d, block = [300, 20], 4, 2, 128, 64
    pool, _, _ = _pool(lens, hk, d, block, 9, True)
    pool["k_scale"] = (pool["k_scale"] / scale).contiguous()
    q = (torch.randn(2, 1, h, d, generator=torch.Generator().manual_seed(5)) * scale).bfloat16()
    got = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                             table=pool["table"], block=block, k_scale=pool["k_scale"], v_scale=pool["v_scale"])()
    torch.cuda.synchronize()
    k, v = (pool[x].cpu().view(torch.float8_e4m3fn).double() * pool[x + "_scale"].cpu().double()[..., None] for x in "kv")
    _check(got, _exact(q, k, v, lens, pool["table"].cpu(), block, 0, d ** -0.5))


def _by_row(lens, h, hk, factor, seed, win=0):
    """A run over E4M3 pools whose V scales take the factor of their row in the request (a tensor)."""
    d, block = 128, 64
    pool, _, _ = _pool(lens, hk, d, block, seed, True)
    for i, n in enumerate(lens):
        r = torch.arange(n)
        rows = (pool["table"][i].cpu().long()[r // block] * block + r % block).to(DEV)
        pool["v_scale"][rows] *= factor[:n, None].to(DEV)
    q = torch.randn(len(lens), 1, h, d, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    got = csa.PagedAttention(q.to(DEV), pool["k"], pool["v"], torch.tensor(lens, dtype=torch.int32, device=DEV), win=win,
                             table=pool["table"], block=block, k_scale=pool["k_scale"], v_scale=pool["v_scale"])()
    torch.cuda.synchronize()
    k, v = (pool[x].cpu().view(torch.float8_e4m3fn).double() * pool[x + "_scale"].cpu().double()[..., None] for x in "kv")
    _check(got, _exact(q, k, v, lens, pool["table"].cpu(), block, win, d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("h", [6, 64])
@pytest.mark.parametrize("few,many", [(0.0, 2.0 ** 40), (0.0, 2.0 ** 100), (2.0 ** -40, 2.0 ** 95), (2.0 ** -29, 2.0 ** 100)])
@pytest.mark.parametrize("run", [32, 768, 5000])
@pytest.mark.parametrize("first", [0, 1])
def test_e4m3_scales_far_apart_between_warps_tiles_and_ctas(run, few, many, h, first):
    # rows of tiny or zero V scales beside rows of huge ones, in runs that a warp, a tile or a CTA has to itself, in
    # both orders: the softmax's sum keeps the part of either, whatever the V scales
    _gpu()
    r = torch.arange(10000)
    _by_row([10000, 1500], h, 2, torch.where((r // run + first) % 2 == 0, few, many).float(), run)


@pytest.mark.gpu
def test_e4m3_one_huge_scale_among_ordinary_ones():
    # a single row raises the reference: the rows after it, ordinary by themselves, stay in the sum
    _gpu()
    for at in (0, 40, 399):
        for rest in (1.0, 2.0 ** -30):
            f = torch.full((3000,), rest)
            f[at] = 2.0 ** 100
            _by_row([3000, 500], 6, 2, f, at)


@pytest.mark.gpu
def test_e4m3_many_rows_far_below_a_peak():
    # a peak in every warp's first rows, whose V rows are zeros, and 2^23 rows that weigh 2^-25.25 of it: together 1.7 %
    # of the output's weight.  A weight is an f16 number; one below 2^-25 of the largest must not vanish from the
    # output while the softmax's sum counts it.  (Pages are shared: one page of tail rows, read over and over.)
    _gpu()
    hk, d, block, pages = 8, 128, 1024, 1 << 13
    b = max(1, torch.cuda.get_device_properties(0).multi_processor_count // hk)
    n = (pages + 1) * block
    k = torch.zeros(2 * block, hk, d, dtype=torch.uint8, device=DEV)
    k[0:384:32, :, 0] = 0x38                                 # 1.0
    v = torch.randn(1, hk, d, generator=torch.Generator().manual_seed(1)).to(torch.float8_e4m3fn).view(torch.uint8)
    v = v.to(DEV).expand(2 * block, hk, d).contiguous()
    v[0:384:32] = 0
    one = torch.ones(2 * block, hk, device=DEV)
    q = torch.zeros(b, 1, hk, d, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    scale = 25.25 * math.log(2)
    table = torch.ones(b, pages + 1, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    got = csa.PagedAttention(q, k, v, torch.full((b,), n, dtype=torch.int32, device=DEV), table=table, block=block,
                             k_scale=one, v_scale=one, scale=scale)()
    torch.cuda.synchronize()
    tail = (n - 12) * 2.0 ** -25.25
    row = v[1].view(torch.float8_e4m3fn).double().cpu()
    want = (row * tail / (12 + tail)).expand(b, 1, hk, d)
    # A thread adds the weights of a quarter of its warp's rows, one after the other, to an fp32 sum: n / 48 terms with
    # twelve warps, each addition off by 2^-24 of the sum at most, so the sum is within `most` of its value, lse too,
    # and the output by that part of itself more than the rounded weights make it
    most = n / 48 * 2.0 ** -24
    assert ((got["lse"].cpu().double() - scale - math.log(12 + tail)).abs() <= most + LSE_TOL).all()
    big = row.abs().amax(1)[:, None]
    assert ((got["out"].cpu().double() - want).abs() <= 1.01 * U * (big + want.abs()) + 1.01 * most * want.abs()).all()
    # and the tail is there (its weights, 2^-18.25 in f16, are off by 2^-6.75 of themselves at most): without it the
    # output is zero
    assert ((got["out"].cpu().double() - want).abs() <= 0.1 * want.abs() + 1e-4).all()


def test_sizes_that_do_not_fit_32_bits_are_refused():
    # (the C struct's fields have 32 bits: 2^32 + 64 would arrive as 64)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(64, 2, 128, dtype=torch.bfloat16)
    n, t = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    for kw in (dict(table=t, block=2 ** 32 + 64, max_len=64), dict(table=t, block=64, win=2 ** 32 + 1),
               dict(table=t, block=64, max_len=2 ** 32 + 64),
               dict(table=torch.zeros(1, 1 << 20, dtype=torch.int32), block=4096)):    # what the table holds: 2^32
        with pytest.raises(csa.CsaError, match="32 bits"):
            csa.PagedAttention(q, k, k, n, **kw)
    b = 2 ** 32 + 1
    many = [torch.empty(s, dtype=d, device="meta") for s, d in (((b, 1, 4, 128), torch.bfloat16), ((64, 2, 128), torch.bfloat16),
                                                                ((b,), torch.int32), ((b, 1), torch.int32))]
    with pytest.raises(csa.CsaError, match="32 bits"):
        csa.PagedAttention(many[0], many[1], many[1], many[2], table=many[3], block=64)


@pytest.mark.gpu
def test_e4m3_queries_at_the_end_of_the_range():
    # |q| from 2^127 on: the power of two taken out of the row is 2^127
    _gpu()
    n, h, hk, d, block = 200, 4, 2, 128, 64
    g = torch.Generator().manual_seed(5)
    k = torch.randn(256, hk, d, generator=g) * 2.0 ** -6
    k, v = (t.to(torch.float8_e4m3fn) for t in (k, torch.randn(256, hk, d, generator=g)))
    ks, vs = torch.full((256, hk), 2.0 ** -115), torch.ones(256, hk)
    q = torch.zeros(1, 1, h, d)
    q[..., 0] = torch.tensor([1.8e38, 2.5e38, -3e38, 3.38e38])
    q = q.bfloat16()
    table = torch.arange(4, dtype=torch.int32)[None]
    got = csa.PagedAttention(q.to(DEV), k.view(torch.uint8).to(DEV), v.view(torch.uint8).to(DEV),
                             torch.tensor([n], dtype=torch.int32, device=DEV), table=table.to(DEV), block=block,
                             k_scale=ks.to(DEV), v_scale=vs.to(DEV))()
    torch.cuda.synchronize()
    _check(got, _exact(q, k.double() * 2.0 ** -115, v.double(), [n], table, block, 0, d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_rows_in_a_long_chunk_cost_passes_for_the_tokens_of_one_product_only(fp8):
    # a NaN among the V rows of a tile that tokens see in part: a pass for each token whose queries are in the product
    # (32 at most, some 32 times a tile's time), not for each of the chunk's 4096
    _gpu()
    s, h, d, block = 4096, 2, 128, 64
    pool, _, _ = _pool([s], 2, d, block, 12, fp8)
    q = torch.randn(1, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    n = torch.tensor([s], dtype=torch.int32, device=DEV)
    op = csa.PagedAttention(q, pool["k"], pool["v"], n, table=pool["table"], block=block, k_scale=pool.get("k_scale"),
                            v_scale=pool.get("v_scale"))

    def timed():
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        op()
        t1.record()
        torch.cuda.synchronize()
        return t0.elapsed_time(t1)

    timed()
    clean, base = {x: t.clone() for x, t in op().items()}, max(timed(), timed())
    for r in range(s - 64, s, 16):                       # one in each 16 rows at the end: most tokens do not see them
        row = int(pool["table"][0, r // block]) * block + r % block
        pool["v"].view(torch.uint8 if fp8 else torch.int16)[row] = 0x7F if fp8 else 0x7FC0
    got, took = op(), timed()
    assert torch.equal(got["out"][:, :s - 64], clean["out"][:, :s - 64]) and torch.equal(got["lse"], clean["lse"])
    assert torch.isnan(got["out"][:, s - 64:]).all()
    assert took <= 60 * base + 1, (took, base)


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_a_softmax_scale_that_is_no_number_is_refused(L, scale):
    # (a NaN would be taken for "not given", 1 / sqrt(dim))
    assert _call(L, softmax_scale=scale) == csa.CSA_ERR_INVALID_ARG
    assert "softmax_scale" in csa.last_error()


def test_a_workspace_that_is_no_plain_memory_is_refused():
    # its size is taken from its elements: with gaps or repeated ones that is not the memory behind it
    q, k = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(64, 2, 128, dtype=torch.bfloat16)
    n, t = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 24), torch.empty(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(csa.CsaError, match="workspace"):
            csa.PagedAttention(q, k, k, n, table=t, block=64, workspace=ws)
    csa.PagedAttention(q, k, k, n, table=t, block=64, workspace=torch.empty(1 << 12, dtype=torch.uint8))
