"""csa_kv_append: new tokens' keys and values into (paged) pools, against the formulas in fp64.

Tolerances: before they are rounded to their type keys and queries are off by 40 u (|a| + |b|) as in
test_qk_rope.py (u = 2^-24); values are copied (bf16, fp32 pools: exactly).  E4M3: the scale is max|y| / 448
with a y that is off by that much, and 2 u for the quotient; a code's value is off by half a step, 2^-4
relative or 2^-10 below E4M3's normal range, of the exact quotient, whose own error is the key's and the scale's.
"""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa
from test_qk_rope import U32, check, exact

DEV = "cuda:0"
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# CPU: refusals

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, **kw):
    a = 0x10000
    base = dict(B=2, S=3, q_heads=4, kv_heads=2, dim=64, dtype=csa.CSA_DTYPE_BF16, kv_dtype=csa.CSA_DTYPE_BF16, norm=0,
                eps=0.0, rope_dim=64, rope_at=0, halves=0, base=10000.0, freq=None, pos=None, ctx_len=a, count=None,
                slot=None, off=None, table=a, block=16, table_stride=4, rows=100, q=a, q_stride=256, q_weight=None, q_out=a,
                q_out_stride=256, k=a, k_stride=128, k_weight=None, v=a, v_stride=128, k_pool=a, k_pool_stride=128,
                v_pool=a, v_pool_stride=128, k_scale=None, v_scale=None, scale_stride=0, status=None)
    base.update(kw)
    return L.csa_kv_append(ctypes.byref(csa.CAppend(**base)), None)


FP8 = dict(kv_dtype=csa.CSA_DTYPE_FP8_E4M3, k_scale=0x10000, v_scale=0x10000, scale_stride=2)
SLOT = dict(table=None, slot=0x10000)


def test_empty_batch_is_a_no_op(L):
    assert _call(L, B=0) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(S=0), csa.CSA_ERR_INVALID_ARG),
    (dict(q_heads=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(kv_heads=0), csa.CSA_ERR_INVALID_ARG),
    (dict(kv_heads=5000), csa.CSA_ERR_UNSUPPORTED),
    (dict(dtype=2), csa.CSA_ERR_UNSUPPORTED),
    (dict(dtype=csa.CSA_DTYPE_F32), csa.CSA_ERR_UNSUPPORTED),   # a bf16 pool for fp32 rows
    (dict(kv_dtype=3), csa.CSA_ERR_UNSUPPORTED),
    (dict(dim=36), csa.CSA_ERR_UNSUPPORTED),
    (dict(rope_dim=65), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_at=4), csa.CSA_ERR_INVALID_ARG),
    (dict(base=0.0), csa.CSA_ERR_INVALID_ARG),
    (dict(norm=1, eps=-1.0), csa.CSA_ERR_INVALID_ARG),
    (dict(k_weight=0x10000), csa.CSA_ERR_INVALID_ARG),          # a weight without the norm
    (dict(q=None), csa.CSA_ERR_INVALID_ARG),
    (dict(q_out=None), csa.CSA_ERR_INVALID_ARG),
    (dict(k=None), csa.CSA_ERR_INVALID_ARG),
    (dict(k=0x10008), csa.CSA_ERR_INVALID_ARG),
    (dict(k_stride=120), csa.CSA_ERR_INVALID_ARG),
    (dict(k_pool=None), csa.CSA_ERR_INVALID_ARG),
    (dict(k_pool_stride=127), csa.CSA_ERR_INVALID_ARG),
    (dict(v=None), csa.CSA_ERR_INVALID_ARG),                    # v_pool without v
    (dict(v_pool=None), csa.CSA_ERR_INVALID_ARG),
    (dict(v_pool_stride=132), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, k_scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, v_scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, scale_stride=1), csa.CSA_ERR_INVALID_ARG),
    (dict(FP8, k_pool_stride=136), csa.CSA_ERR_INVALID_ARG),    # 136 bytes
    (dict(rows=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(ctx_len=None), csa.CSA_ERR_INVALID_ARG),
    (dict(table=None), csa.CSA_ERR_INVALID_ARG),
    (dict(block=0), csa.CSA_ERR_INVALID_ARG),
    (dict(table_stride=0), csa.CSA_ERR_INVALID_ARG),
    (dict(slot=0x10000), csa.CSA_ERR_INVALID_ARG),              # and a table
    (dict(SLOT, ctx_len=None), csa.CSA_ERR_INVALID_ARG),        # no positions
    (dict(SLOT, slot=0x10004), csa.CSA_ERR_INVALID_ARG),
    (dict(count=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(status=0x10002), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_kv_append(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    bf, i32 = torch.bfloat16, torch.int32
    k, pool = torch.zeros(2, 3, 2, 64, dtype=bf), torch.zeros(100, 2, 64, dtype=bf)
    n, t = torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    good = dict(ctx_len=n, table=t, block=16)
    f8 = pool.to(torch.float8_e4m3fn)
    for args, kw in (((k, k, pool, None), good), ((k, None, pool, pool), good), ((k, k, pool, pool.float()), good),
                     ((k, k, pool, pool[:50]), good), ((k, k.float(), pool, pool), good), ((k, k, pool, pool), dict(ctx_len=n)),
                     ((k, k, pool, pool), dict(good, off=n.long())), ((k, k, pool, pool), dict(table=t, block=16)),
                     ((k, k, pool, pool), dict(good, ctx_len=n.long())), ((k, k, pool, pool), dict(good, count=n[:1])),
                     ((k, k, pool, pool), dict(slot=torch.zeros(6, dtype=torch.int64))),
                     ((k, k, pool, pool), dict(slot=torch.zeros(5, dtype=torch.int64), ctx_len=n)),
                     ((k, k, f8, f8), good), ((k, k, f8, f8), dict(good, k_scale=torch.zeros(100, 2))),
                     ((k, k, f8, pool), dict(good, k_scale=torch.zeros(100, 2), v_scale=torch.zeros(100, 2))),
                     ((k, k, pool, pool), dict(good, k_scale=torch.zeros(100, 2))),
                     ((k, k, pool, pool), dict(good, q=k[:, :2])), ((k, k, pool, pool), dict(good, q_out=k)),
                     ((k, k, pool, pool), dict(good, k_weight=torch.ones(64, dtype=bf)))):
        with pytest.raises(csa.CsaError):
            csa.KvAppend(*args, **kw)


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


class Case:
    """Inputs on the host, pools filled with a pattern, and the exact rows that a call has to leave."""

    def __init__(self, lens, s, hk, dim, seed, dt=torch.bfloat16, fp8=False, hq=0, v=True, norm=False, rope=None, at=0,
                 halves=True, counts=None, block=16, place="table", spare=2):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *shape: torch.randn(*shape, generator=g)
        self.lens, self.s, self.hk, self.dim, self.dt, self.fp8, self.place = lens, s, hk, dim, dt, fp8, place
        self.rope, self.at, self.halves, self.norm, self.block = dim - at if rope is None else rope, at, halves, norm, block
        b = len(lens)
        self.counts = counts
        self.k, self.v = rn(b, s, hk, dim).to(dt), rn(b, s, hk, dim).to(dt) if v else None
        self.q = rn(b, s, hq, dim).to(dt) if hq else None
        self.kw = (1 + 0.2 * rn(dim)).to(dt) if norm else None
        self.qw = (1 + 0.2 * rn(dim)).to(dt) if norm and hq else None
        nblk = [max(0, -(-x // block)) for x in lens]
        total = sum(nblk) + spare
        perm = torch.randperm(total, generator=g)
        self.table = torch.full((b, max(1, max(nblk))), -1, dtype=torch.int32)
        a = 0
        for i, n in enumerate(nblk):
            self.table[i, :n] = perm[a:a + n].int()
            a += n
        self.rows = total * block
        # where each token goes (-1: nowhere) and its position
        self.to, self.pos = torch.full((b, s), -1, dtype=torch.int64), torch.zeros(b, s, dtype=torch.int32)
        for i, length in enumerate(lens):
            n = s if counts is None else counts[i]
            for t in range(s):
                r = length - n + t
                self.pos[i, t] = r
                if t < n and r >= 0:
                    self.to[i, t] = int(self.table[i, r // block]) * block + r % block

    def pools(self):
        fill = lambda: torch.full((self.rows, self.hk, self.dim), 3.0, dtype=self.dt)
        d = dict(k_pool=fill(), v_pool=fill() if self.v is not None else None)
        if self.fp8:
            for x in ("k", "v"):
                if d[x + "_pool"] is not None:
                    d[x + "_pool"] = d[x + "_pool"].to(torch.float8_e4m3fn)
                    d[x + "_scale"] = torch.full((self.rows, self.hk), 5.0)
        return {n: None if t is None else t.to(DEV) for n, t in d.items()}

    def op(self, pools, **kw):
        dev = lambda t: None if t is None else t.to(DEV)
        how = dict(ctx_len=torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                   count=None if self.counts is None else torch.tensor(self.counts, dtype=torch.int32, device=DEV))
        if self.place == "table":
            how.update(table=dev(self.table), block=self.block)
        elif self.place == "slot":
            how = dict(slot=dev(self.to), pos=dev(self.pos))
        self.q_out = None if self.q is None else torch.full(self.q.shape, 9.0, dtype=self.dt, device=DEV)
        how.update(kw)
        return csa.KvAppend(dev(self.k), dev(self.v), pools["k_pool"], pools["v_pool"], k_scale=pools.get("k_scale"),
                            v_scale=pools.get("v_scale"), q=dev(self.q), q_out=self.q_out, q_weight=dev(self.qw),
                            k_weight=dev(self.kw), norm=self.norm, rope_dim=self.rope, rope_at=self.at,
                            halves=self.halves, **how)

    def check(self, pools):
        real = (self.to >= 0).view(-1)
        to, pos = self.to.view(-1)[real], self.pos.view(-1)[real]
        still = torch.ones(self.rows, dtype=torch.bool)
        still[to] = False
        flat = lambda t: t.reshape(-1, *t.shape[2:])
        for name, x in (("k", self.k), ("v", self.v)):
            if x is None:
                continue
            x = flat(x)[real]
            if name == "k":
                want, size = exact(x, self.kw, pos, self.norm, 1e-6, self.rope, self.at, self.halves)
            else:
                want, size = x.double(), x.double().abs()
            pool = pools[name + "_pool"].cpu()
            if not self.fp8:
                assert (pool[still] == 3.0).all()
                if name == "v":
                    assert torch.equal(pool[to], x)
                else:
                    check(pool[to], want, size, self.dt, name)
                continue
            pool, scale = pool.float(), pools[name + "_scale"].cpu()
            assert (pool[still] == 3.0).all() and (scale[still] == 5.0).all()
            got_s = scale[to].double()
            most = want.abs().amax(2)
            off = 40 * U32 * size
            ws = torch.where(most > 0, (most / E4M3_MAX).clamp_min(2.0 ** -126), 1.0)
            assert ((got_s - ws).abs() <= off.amax(2) / E4M3_MAX + 2 * U32 * ws + 2.0 ** -149).all(), name
            val = pool[to].double() * got_s[:, :, None]
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 * got_s[:, :, None] + 2 * off + off.amax(2, keepdim=True)
            assert ((val - want).abs() <= tol).all(), name
        if self.q is not None:
            got = flat(self.q_out.cpu())
            assert (got[~real] == 9.0).all()
            want, size = exact(flat(self.q)[real], self.qw, pos, self.norm, 1e-6, self.rope, self.at, self.halves)
            check(got[real], want, size, self.dt, "q")


KINDS = [dict(dt=torch.bfloat16), dict(dt=torch.float32), dict(dt=torch.bfloat16, fp8=True), dict(dt=torch.float32, fp8=True)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "f32", "bf16-e4m3", "f32-e4m3"])
@pytest.mark.parametrize("shape", [
    dict(dim=128), dict(dim=128, hq=8, norm=True), dict(dim=64, rope=32, at=32, halves=False, hq=2), dict(dim=80, rope=20, hq=4),
    dict(dim=576, rope=64, at=512, halves=False, v=False, hk=1, hq=3), dict(dim=256, hq=2, norm=True),
    dict(dim=128, rope=0, norm=True), dict(dim=16, rope=6, at=5, norm=True), dict(dim=1024, rope=256, hk=1)])
@pytest.mark.parametrize("place", ["table", "slot"])
def test_rows(kind, shape, place):
    _gpu()
    shape = dict(dict(hk=2), **shape)
    for lens, s, counts in (([1], 1, None), ([40, 0, 17, 3], 3, None), ([33, 5, 64, 1, 0], 5, [2, 5, 1, 0, 0])):
        c = Case(lens, s, seed=sum(lens) + shape["dim"], counts=counts, place=place, **kind, **shape)
        pools = c.pools()
        c.op(pools)()
        c.check(pools)


@pytest.mark.gpu
def test_many_tokens_of_one_head():
    """Indexer keys of a long prompt: the FP8 key pool's rows and scales."""
    _gpu()
    c = Case([9001], 9001, 1, 128, 3, fp8=True, v=False, norm=True, rope=64, at=64, halves=False, block=128, place="slot")
    pools = c.pools()
    c.op(pools)()
    c.check(pools)


@pytest.mark.gpu
def test_offsets_and_positions_apart_from_rows():
    """Rows through off; drafted tokens whose positions are their depths."""
    _gpu()
    c = Case([20, 9], 4, 2, 64, 5, block=64, spare=0)
    c.table = torch.tensor([[0], [1]], dtype=torch.int32)
    c.to = torch.tensor([[16, 17, 18, 19], [64 + 5, 64 + 6, 64 + 7, 64 + 8]])
    c.pos = torch.tensor([[16, 17, 17, 18], [5, 6, 6, 6]], dtype=torch.int32)
    c.place = "off"
    pools = c.pools()
    c.op(pools, off=torch.tensor([0, 64], device=DEV), pos=c.pos.to(DEV))()
    c.check(pools)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_bad_rows_are_skipped_and_recorded(fp8):
    _gpu()
    c = Case([10, 40, 12, 30], 2, 2, 64, 7, fp8=fp8, hq=2)
    c.table[1, 2] = -1                                       # rows 38, 39: an unmapped block
    c.table[3, 1] = 1 << 27                                  # rows 28, 29: a block outside the pool
    keep = c.to.clone()
    c.to[1] = c.to[3] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pools = c.pools()
    c.op(pools, status=status)()
    assert int(status) == 1
    q, c.q = c.q, None
    c.check(pools)
    # the queries of those tokens are made all the same
    c.q, c.to = q, keep
    want, size = exact(q.view(8, 2, 64), None, c.pos.view(-1), False, 0, 64, 0, True)
    check(c.q_out.view(8, 2, 64), want, size, c.dt)


@pytest.mark.gpu
def test_bad_lengths_counts_and_slots():
    _gpu()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for kw, lens in ((dict(count=torch.tensor([3, 1], dtype=torch.int32)), [8, 8]), (dict(count=torch.tensor([-1, 1], dtype=torch.int32)), [8, 8]),
                     ({}, [-5, 8]), ({}, [-2 ** 31, 8])):
        c = Case([max(0, x) for x in lens], 2, 1, 64, 9, counts=[0, 1] if kw else None)
        c.lens = lens
        status.zero_()
        pools = c.pools()
        c.op(pools, status=status, **{n: t.to(DEV) for n, t in kw.items()})()
        assert int(status) == 1
        c.check(pools)
    c = Case([8, 8], 2, 1, 64, 9, place="slot")
    bad = c.to.clone()
    bad[0, 1] = c.rows
    bad[1, 0] = 2 ** 40
    c.to[0, 1] = c.to[1, 0] = -1
    status.zero_()
    pools = c.pools()
    c.op(pools, status=status, slot=bad.to(DEV))()
    assert int(status) == 1
    c.check(pools)


@pytest.mark.gpu
def test_row_sizes_of_e4m3():
    """All-zero, tiny, huge, infinite and NaN heads."""
    _gpu()
    c = Case([6], 6, 1, 64, 11, dt=torch.float32, fp8=True, rope=0)
    c.k[0, 0] = 0
    c.k[0, 1] *= 1e-38
    c.k[0, 2] *= 1e36
    c.k[0, 3] *= 1e-42
    c.k[0, 4, 0, 3] = math.inf
    c.k[0, 5, 0, 7] = math.nan
    pools = c.pools()
    c.op(pools)()
    kp, ks = pools["k_pool"].cpu().float(), pools["k_scale"].cpu()
    to = c.to[0]
    assert (kp[to[0]] == 0).all() and ks[to[0], 0] == 1
    for i in (1, 2):
        want = c.k[0, i].double()
        val = kp[to[i]].double() * ks[to[i]].double()
        assert ((val - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * float(ks[to[i], 0])).all()
    assert ks[to[3], 0] == 2.0 ** -126
    assert math.isinf(ks[to[4], 0]) and kp[to[4], 0, 3].isnan() and (kp[to[4], 0, :3] == 0).all()
    row = kp[to[5], 0]
    assert row[7].isnan() and torch.isfinite(torch.cat([row[:7], row[8:]])).all() and math.isfinite(ks[to[5], 0])


@pytest.mark.gpu
def test_captured_lengths_follow_the_device():
    """A captured call takes the lengths, counts and inputs that the buffers hold when it is replayed."""
    _gpu()
    c = Case([20, 33], 3, 2, 128, 13, hq=2, norm=True, counts=[3, 2])
    pools = c.pools()
    lens, counts = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([20, 33], [3, 2]))
    op = c.op(pools, ctx_len=lens, count=counts)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        op()
    torch.cuda.synchronize()
    d = Case([18, 31], 3, 2, 128, 13, hq=2, norm=True, counts=[1, 3])
    d.table, d.q_out = c.table, c.q_out
    for i, (n, m) in enumerate(((18, 1), (31, 3))):
        for t in range(3):
            r = n - m + t
            d.pos[i, t] = r
            d.to[i, t] = int(c.table[i, r // 16]) * 16 + r % 16 if t < m else -1
    d.rows, d.k, d.v, d.q, d.kw, d.qw = c.rows, c.k, c.v, c.q, c.kw, c.qw
    lens.copy_(torch.tensor([18, 31]))
    counts.copy_(torch.tensor([1, 3]))
    g.replay()
    torch.cuda.synchronize()
    d.check(pools)
