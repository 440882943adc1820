"""csa_qk_rope: norm and rotation of query and key heads, against the formulas in fp64.

Tolerance.  With u = 2^-24: a head's sum of squares is off by at most 40 u relative (chains of at most 32
products per lane and 5 shuffles), its inverse root by half of that, 2 ulp of rsqrtf and two products: y by 30 u.
The cosine and sine: the fraction of a turn is rounded to fp32 (2^-25 half turns, 9.4e-8 in the angle) and
sincospif adds 2 ulp: below 4 u together; the rotation's products and sum add 3 u.  So an element is off by at most
40 u (|a| + |b|) of its pair before it is rounded to the output's type (2^-8 relative for bf16, u for fp32).
"""
import ctypes
import math

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa

DEV = "cuda:0"
U32 = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def exact(x, weight, pos, norm, eps, rope, at, halves, base=10000.0, freq=None):
    """Heads [n, heads, dim] in fp64, and the bound |a| + |b| of each element."""
    y = x.double()
    d = y.shape[2]
    if norm:
        y = y / torch.sqrt((y * y).sum(2, keepdim=True) / d + eps)
        if weight is not None:
            y = y * weight.double()
    i = torch.arange(rope // 2, dtype=torch.float64)
    theta = base ** (-2 * i / rope) if freq is None else freq.double()
    ang = pos.double()[:, None] * theta
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    j = torch.arange(rope // 2)
    fa = at + (j if halves else 2 * j)
    fb = fa + (rope // 2 if halves else 1)
    a, b = y[:, :, fa], y[:, :, fb]
    out, size = y.clone(), y.abs()
    out[:, :, fa], out[:, :, fb] = a * c - b * s, a * s + b * c
    size[:, :, fa] = size[:, :, fb] = a.abs() + b.abs()
    return out, size


def check(got, want, size, dt, what=""):
    got = got.cpu().double()
    err = (got - want).abs()
    tol = ROUND[dt] * want.abs() + 40 * U32 * size * (1 + ROUND[dt])
    assert torch.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3e} above, worst error {float(err.max()):.3e}"


# ---------------------------------------------------------------------------
# CPU: refusals

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, **kw):
    a = 0x10000
    base = dict(n=4, q_heads=2, k_heads=1, dim=64, dtype=csa.CSA_DTYPE_BF16, norm=1, eps=1e-6, rope_dim=64, rope_at=0,
                halves=1, base=10000.0, freq=None, pos=a, q=a, q_stride=128, q_weight=a, q_out=a, q_out_stride=128, k=a,
                k_stride=64, k_weight=None, k_out=a, k_out_stride=64)
    base.update(kw)
    return L.csa_qk_rope(ctypes.byref(csa.CRope(**base)), None)


def test_no_tokens_is_a_no_op(L):
    assert _call(L, n=0) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(q_heads=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(q_heads=0, k_heads=0), csa.CSA_ERR_INVALID_ARG),
    (dict(q_heads=4096, k_heads=1), csa.CSA_ERR_UNSUPPORTED),
    (dict(q_heads=2147483647, k_heads=2147483647), csa.CSA_ERR_UNSUPPORTED),
    (dict(dtype=2), csa.CSA_ERR_UNSUPPORTED),
    (dict(dim=0), csa.CSA_ERR_INVALID_ARG),
    (dict(dim=60), csa.CSA_ERR_UNSUPPORTED),
    (dict(dim=1032), csa.CSA_ERR_UNSUPPORTED),
    (dict(rope_dim=-2), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_dim=31), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_dim=66), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_at=2), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_at=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(rope_at=2147483647), csa.CSA_ERR_INVALID_ARG),
    (dict(dim=512, rope_dim=258, q_stride=1024, k_stride=512, q_out_stride=1024, k_out_stride=512), csa.CSA_ERR_UNSUPPORTED),
    (dict(norm=2), csa.CSA_ERR_INVALID_ARG),
    (dict(halves=2), csa.CSA_ERR_INVALID_ARG),
    (dict(norm=0), csa.CSA_ERR_INVALID_ARG),                  # a weight without the norm
    (dict(eps=-1.0), csa.CSA_ERR_INVALID_ARG),
    (dict(eps=math.nan), csa.CSA_ERR_INVALID_ARG),
    (dict(base=0.5), csa.CSA_ERR_INVALID_ARG),
    (dict(base=math.inf), csa.CSA_ERR_INVALID_ARG),
    (dict(base=math.nan), csa.CSA_ERR_INVALID_ARG),
    (dict(pos=None), csa.CSA_ERR_INVALID_ARG),
    (dict(pos=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(freq=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(q=None), csa.CSA_ERR_INVALID_ARG),
    (dict(q=0x10008), csa.CSA_ERR_INVALID_ARG),
    (dict(q_stride=120), csa.CSA_ERR_INVALID_ARG),
    (dict(q_stride=132), csa.CSA_ERR_INVALID_ARG),
    (dict(q_weight=0x10004), csa.CSA_ERR_INVALID_ARG),
    (dict(q_out=None), csa.CSA_ERR_INVALID_ARG),
    (dict(q_out_stride=64), csa.CSA_ERR_INVALID_ARG),
    (dict(k=None), csa.CSA_ERR_INVALID_ARG),
    (dict(k_out=0x10001), csa.CSA_ERR_INVALID_ARG),
    (dict(k_stride=56), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_qk_rope(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    bf = torch.bfloat16
    q, k, p = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, 1, 64, dtype=bf), torch.zeros(4, dtype=torch.int32)
    w = torch.ones(64, dtype=bf)
    for args, kw in (((None, None, p), {}), ((q, k), {}), ((q, k, p.long()), {}), ((q, k, p[:3]), {}), ((q, k[:3], p), {}),
                     ((q, k.float(), p), {}), ((q.half(), None, p), {}), ((q, k, p), dict(q_weight=w)),
                     ((q, k, p), dict(q_weight=w.float(), norm=True)), ((q, None, p), dict(k_weight=w, norm=True)),
                     ((q, k, p), dict(q_weight=w[:32], norm=True)), ((q, k, p), dict(freq=torch.zeros(31))),
                     ((q, k, p), dict(q_out=q.float())), ((q.transpose(0, 1), k, p), {}),
                     ((torch.zeros(4, 2, 128, dtype=bf)[..., ::2], None, p), {})):
        with pytest.raises(csa.CsaError):
            csa.QkRope(*args, **kw)


def test_object_on_the_cpu_does_not_launch(L):
    with pytest.raises(csa.CsaError):
        csa.QkRope(torch.zeros(4, 2, 64, dtype=torch.bfloat16), None, torch.zeros(4, dtype=torch.int32))()


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _case(n, hq, hk, d, dt, seed, norm=True, far=1 << 20):
    q = _randn(seed, n, hq, d).to(dt) if hq else None
    k = _randn(seed + 1, n, hk, d).to(dt) if hk else None
    qw, kw = ((1 + 0.3 * _randn(seed + i, d)).to(dt) if h and norm else None for i, h in ((2, hq), (3, hk)))
    pos = torch.randint(0, far, (n,), generator=torch.Generator().manual_seed(seed + 4), dtype=torch.int32)
    return q, k, qw, kw, pos


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _run(q, k, qw, kw, pos, norm, rope, at, halves, **kws):
    dq, dk, dqw, dkw, dpos = _dev(q, k, qw, kw, pos)
    return csa.QkRope(dq, dk, dpos, q_weight=dqw, k_weight=dkw, norm=norm, eps=1e-6, rope_dim=rope, rope_at=at, halves=halves,
                      **kws)()


SHAPES = [  # dim, rotated dims, first of them
    (8, 8, 0), (8, 2, 6), (16, 16, 0), (24, 16, 8), (64, 64, 0), (64, 32, 32), (80, 20, 0), (80, 20, 60), (96, 64, 3),
    (128, 128, 0), (128, 64, 64), (128, 48, 16), (128, 0, 0), (192, 64, 128), (256, 256, 0), (256, 128, 5), (576, 64, 512),
    (576, 256, 0), (1024, 256, 768), (1024, 30, 1), (1016, 32, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dim,rope,at", SHAPES)
def test_shapes(dim, rope, at, halves, dt):
    _gpu()
    for n, hq, hk, norm in ((1, 3, 1, True), (37, 5, 2, True), (19, 4, 0, False), (211, 0, 1, True)):
        q, k, qw, kw, pos = _case(n, hq, hk, dim, dt, 100 + dim + n, norm)
        got = _run(q, k, qw, kw, pos, norm, rope, at, halves)
        for name, x, w in (("q", q, qw), ("k", k, kw)):
            assert (x is not None) == (name in got)
            if x is not None:
                want, size = exact(x, w, pos, norm, 1e-6, rope, at, halves)
                check(got[name], want, size, dt, f"{name} n={n}")


@pytest.mark.gpu
@pytest.mark.parametrize("halves", [False, True])
def test_extreme_positions(halves):
    _gpu()
    q, _, _, _, _ = _case(8, 2, 0, 128, torch.float32, 5, False)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 123456789, -77777777], dtype=torch.int32)
    got = _run(q, None, None, None, pos, False, 128, 0, halves)
    want, size = exact(q, None, pos, False, 0, 128, 0, halves)
    # theta = 10000^(-2i/R) in fp64 on either side: off by 2^-51 |pos theta| at most, 1e-6 rad at 2^31
    err = (got["q"].cpu().double() - want).abs()
    assert (err <= (41 * U32 + 2.0 ** -20) * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dim,rope,at", [(128, 64, 64), (80, 20, 0)])
def test_given_frequencies(dim, rope, at):
    _gpu()
    q, k, qw, kw, pos = _case(50, 2, 1, dim, torch.float32, 9)
    for freq in ((8.0 * 10000.0 ** (-2 * torch.arange(rope // 2) / rope)).float(), torch.zeros(rope // 2),
                 -torch.rand(rope // 2, generator=torch.Generator().manual_seed(1)) * 3):
        got = _run(q, k, qw, kw, pos, True, rope, at, True, freq=freq.to(DEV))
        for name, x, w in (("q", q, qw), ("k", k, kw)):
            want, size = exact(x, w, pos, True, 1e-6, rope, at, True, freq=freq)
            check(got[name], want, size, torch.float32, name)


@pytest.mark.gpu
@pytest.mark.parametrize("base", [1.0, 500000.0, 3e38])
def test_bases(base):
    _gpu()
    q, _, _, _, pos = _case(33, 3, 0, 64, torch.float32, 12, False)
    got = _run(q, None, None, None, pos, False, 64, 0, True, base=base)
    base = float(torch.tensor(base, dtype=torch.float32))
    want, size = exact(q, None, pos, False, 0, 64, 0, True, base=base)
    check(got["q"], want, size, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,rope,at", [(128, 128, 0), (80, 20, 3)])
def test_in_place_within_a_fused_projection(dim, rope, at):
    """Queries and keys are slices of one [n, (Hq + 2 Hk) dim] buffer and stay there; the values keep what they hold."""
    _gpu()
    n, hq, hk, dt = 77, 6, 2, torch.bfloat16
    q, k, qw, kw, pos = _case(n, hq, hk, dim, dt, 21)
    v = _randn(25, n, hk, dim).to(dt)
    fused = torch.cat([q, k, v], 1).to(DEV)
    dq, dk = fused[:, :hq], fused[:, hq:hq + hk]
    op = csa.QkRope(dq, dk, pos.to(DEV), q_weight=qw.to(DEV), k_weight=kw.to(DEV), norm=True, rope_dim=rope, rope_at=at,
                    halves=True, q_out=dq, k_out=dk)
    op()
    for x, w, got in ((q, qw, fused[:, :hq]), (k, kw, fused[:, hq:hq + hk])):
        want, size = exact(x, w, pos, True, 1e-6, rope, at, True)
        check(got, want, size, dt)
    assert torch.equal(fused[:, hq + hk:].cpu(), v)


@pytest.mark.gpu
def test_batches_of_tokens_and_padded_strides():
    _gpu()
    b, s, h, d = 3, 5, 4, 64
    wide = _randn(31, b, s, h * d + 24).to(torch.bfloat16).to(DEV)
    q = wide[:, :, :h * d].unflatten(2, (h, d))
    pos = torch.arange(b * s, dtype=torch.int32).view(b, s)
    out = torch.full((b, s, h * d + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    csa.QkRope(q, None, pos.to(DEV), halves=True, q_out=out[:, :, :h * d].unflatten(2, (h, d)))()
    want, size = exact(q.cpu().reshape(b * s, h, d), None, pos.view(-1), False, 0, d, 0, True)
    check(out[:, :, :h * d].reshape(b * s, h, d), want, size, torch.bfloat16)
    assert (out[:, :, h * d:] == 7.0).all()


@pytest.mark.gpu
def test_values_stay_within_their_head():
    """Zeros with eps = 0 aside, what a head holds reaches no other head: NaN, infinities, zeros, tiny and large rows."""
    _gpu()
    q, _, qw, _, pos = _case(40, 4, 0, 128, torch.float32, 41)
    clean = _run(q, None, qw, None, pos, True, 64, 32, False)["q"].cpu()
    x = q.clone()
    x[3, 1, 5], x[7, 0, 100], x[9, 2] = math.nan, math.inf, 0.0
    got = _run(x, None, qw, None, pos, True, 64, 32, False)["q"].cpu()
    assert got[3, 1].isnan().all() and not torch.isfinite(got[7, 0, 100]) and (got[9, 2] == 0).all()
    same = torch.ones(40, 4, dtype=torch.bool)
    same[3, 1] = same[7, 0] = same[9, 2] = False
    assert torch.equal(got[same], clean[same])
    for size in (1e-15, 1e15):
        got = _run(q * size, None, qw, None, pos, True, 64, 32, False)["q"]
        want, bound = exact(q * size, qw, pos, True, 1e-6, 64, 32, False)
        check(got, want, bound, torch.float32)


@pytest.mark.gpu
def test_many_tokens_and_heads():
    _gpu()
    for n, hq, hk, d, dt in ((5003, 32, 8, 128, torch.bfloat16), (20011, 1, 0, 8, torch.float32), (3, 700, 60, 64, torch.bfloat16)):
        q, k, qw, kw, pos = _case(n, hq, hk, d, dt, 51)
        got = _run(q, k, qw, kw, pos, True, d, 0, True)
        for name, x, w in (("q", q, qw), ("k", k, kw)):
            if x is not None:
                want, size = exact(x, w, pos, True, 1e-6, d, 0, True)
                check(got[name], want, size, dt, name)


@pytest.mark.gpu
def test_captured_on_another_stream():
    _gpu()
    q, k, qw, kw, pos = _case(64, 4, 2, 64, torch.bfloat16, 61)
    dq, dk, dqw, dkw, dpos = _dev(q, k, qw, kw, pos)
    op = csa.QkRope(dq, dk, dpos, q_weight=dqw, k_weight=dkw, norm=True, halves=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        op()
        with torch.cuda.graph(g, stream=st):
            op()
    torch.cuda.synchronize()
    q2, k2, _, _, pos2 = _case(64, 4, 2, 64, torch.bfloat16, 71)
    for a, b in ((dq, q2), (dk, k2), (dpos, pos2)):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    for name, x, w in (("q", q2, qw), ("k", k2, kw)):
        want, size = exact(x, w, pos2, True, 1e-6, 64, 0, True)
        check(op._out[name], want, size, torch.bfloat16, name)
