"""csa_fp8_matmul: E4M3 codes with a scale per (row, 128) of a and per (128, 128) of b, against a plain fp64
product of the values the codes stand for.

Tolerance.  A product of two E4M3 values is exact in fp32.  Within a block the tensor core adds 128 of them,
then the scaled block sums are added in fp32: at most 128 + ceil(K / 128) additions, each off by at most one
unit in the last place of a partial sum (2^-23 of sum |a b| scale, whichever way it rounds), and three products
with or of scales (2^-24 each).  So |out - exact| <= (128 + ceil(K / 128) + 3) 2^-23 sum |a b| scale, and
u(t) |exact| more (bf16 2^-8) for the output's one rounding.
"""
import ctypes

import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa

DEV = "cuda:0"


# ---------------------------------------------------------------------------
# CPU: refusals

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, **kw):
    base = dict(M=4, N=256, K=300, out_dtype=csa.CSA_DTYPE_BF16, a=0x10000, a_stride=304, a_scale=0x10000,
                a_scale_stride=3, b=0x10000, b_stride=304, b_scale=0x10000, b_scale_stride=3, out=0x10000,
                out_stride=256, status=None)
    base.update(kw)
    return L.csa_fp8_matmul(ctypes.byref(csa.CFp8Mm(**base)), None)


def test_empty_calls_are_no_ops(L):
    assert _call(L, M=0) == csa.CSA_OK
    assert _call(L, N=0) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(N=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(K=0), csa.CSA_ERR_INVALID_ARG),
    (dict(M=(1 << 30) + 1), csa.CSA_ERR_UNSUPPORTED),
    (dict(N=(1 << 31) - 1), csa.CSA_ERR_UNSUPPORTED),
    (dict(K=(1 << 31) - 1), csa.CSA_ERR_UNSUPPORTED),
    (dict(out_dtype=csa.CSA_DTYPE_FP8_E4M3), csa.CSA_ERR_UNSUPPORTED),
    (dict(a=None), csa.CSA_ERR_INVALID_ARG),
    (dict(a=0x10008), csa.CSA_ERR_INVALID_ARG),
    (dict(a_stride=300), csa.CSA_ERR_INVALID_ARG),          # rows off the 16-byte boundary
    (dict(a_stride=288), csa.CSA_ERR_INVALID_ARG),          # below the width
    (dict(b=None), csa.CSA_ERR_INVALID_ARG),
    (dict(b_stride=302), csa.CSA_ERR_INVALID_ARG),
    (dict(a_scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(a_scale=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(a_scale_stride=2), csa.CSA_ERR_INVALID_ARG),
    (dict(b_scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(b_scale_stride=2), csa.CSA_ERR_INVALID_ARG),
    (dict(out=None), csa.CSA_ERR_INVALID_ARG),
    (dict(out=0x10001), csa.CSA_ERR_INVALID_ARG),
    (dict(out_dtype=csa.CSA_DTYPE_F32, out=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(out_stride=255), csa.CSA_ERR_INVALID_ARG),
    (dict(status=0x10002), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_fp8_matmul(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    a, b = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(200, 256, dtype=torch.uint8)
    sa, sb = torch.ones(4, 2), torch.ones(2, 2)
    for args, kw in (((a.float(), sa, b, sb), {}), ((a, sa, b[:, :128], sb), {}), ((a, sa[:, :1], b, sb), {}),
                     ((a, sa, b, sb[:1]), {}), ((a, sa.double(), b, sb), {}), ((a, sa, b, sb), dict(out=torch.zeros(4, 199))),
                     ((a, sa, b, sb), dict(out=torch.zeros(4, 200).half())),
                     ((a, sa, b, sb), dict(out=torch.zeros(4, 200), out_dtype=torch.bfloat16)),
                     ((a, sa, b, sb), dict(status=torch.zeros(2, dtype=torch.int32))),
                     ((a.t(), sa, b, sb), {})):
        with pytest.raises(csa.CsaError):
            csa.Fp8Matmul(*args, **kw)
    with pytest.raises(csa.CsaError, match="not on a CUDA device"):
        csa.Fp8Matmul(a, sa, b, sb)()


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _codes(rows, k, gen, pitch=None):
    """Random finite codes [rows, k] in rows of `pitch` bytes; what is behind k is the NaN code."""
    pitch = pitch or -(-k // 16) * 16
    c = torch.randint(0, 256, (rows, pitch), generator=gen, device=DEV, dtype=torch.uint8)
    c[(c & 0x7F) == 0x7F] = 0x3A
    c[:, k:] = 0x7F
    return c[:, :k]


def _scales(rows, cols, gen):
    return torch.exp(torch.randn(rows, cols, generator=gen, device=DEV) - 8)


def _exact(a, sa, b, sb):
    """out and sum |a b| scale in fp64, by blocks of k."""
    (m, k), n = a.shape, b.shape[0]
    out = torch.zeros(m, n, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    rb = torch.arange(n, device=DEV) // 128
    for kb in range(-(-k // 128)):
        pa = a[:, 128 * kb:128 * kb + 128].contiguous().view(torch.float8_e4m3fn).double() * sa[:, kb:kb + 1].double()
        pb = b[:, 128 * kb:128 * kb + 128].contiguous().view(torch.float8_e4m3fn).double() * sb[rb, kb][:, None].double()
        out += pa @ pb.t()
        size += pa.abs() @ pb.abs().t()
    return out, size


def _check(got, a, sa, b, sb, what=""):
    out, size = _exact(a, sa, b, sb)
    k = a.shape[1]
    tol = (128 + -(-k // 128) + 3) * 2.0 ** -23 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * out.abs()
    err = (got.double() - out).abs()
    assert (err <= tol).all(), (what, float((err / tol.clamp_min(1e-300)).max()))


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 8192, 1536), (2, 130, 17), (3, 257, 129), (15, 1000, 640), (16, 64, 4096),
          (17, 129, 1000), (32, 4096, 512), (33, 300, 2048), (63, 576, 1280), (64, 2304, 1536), (65, 129, 300),
          (100, 77, 7168), (128, 128, 128), (129, 513, 384), (200, 4100, 1000), (331, 1100, 7000), (1000, 1111, 333),
          (1, 100000, 256), (2048, 2176, 512), (700, 300, 16384), (5, 40, 65536),
          (2500, 2300, 700), (4000, 1290, 1), (2300, 2650, 1500),
          (20000, 257, 300), (300, 20000, 130)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matches_the_definition(m, n, k, dtype):
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(m * 31 + n * 7 + k)
    a, b = _codes(m, k, g), _codes(n, k, g)
    kb = -(-k // 128)
    sa, sb = _scales(m, kb, g), _scales(-(-n // 128), kb, g)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = csa.Fp8Matmul(a, sa, b, sb, out_dtype=dtype, status=status)()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check(got, a, sa, b, sb, (m, n, k))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [7, 90, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_what_stays_untouched(m, dtype):
    # every matrix inside a wider one; out with an odd pitch (element alignment alone), rows and columns
    # behind it keep their values; NaN codes behind k and NaN scales behind the used ones are not read
    _gpu()
    n, k = 261, 700
    g = torch.Generator(device=DEV).manual_seed(m)
    a, b = _codes(m, k, g, 800), _codes(n, k, g, 1024)
    sa = torch.full((m, 9), float("nan"), device=DEV)
    sb = torch.full((4, 7), float("nan"), device=DEV)
    sa[:, :6], sb[:3, :6] = _scales(m, 6, g), _scales(3, 6, g)
    ob = torch.full((m + 2, 2 * n + 1), 5.0, dtype=dtype, device=DEV)
    for first in (0, 1, 3):                               # also outputs off the 16-byte boundary
        out = ob[:m, first:first + n]
        csa.Fp8Matmul(a, sa[:, :6], b, sb[:3, :6], out=out)()
        torch.cuda.synchronize()
        _check(out, a, sa[:, :6], b, sb[:3, :6], first)
        assert (ob[m:] == 5).all() and (ob[:, first + n:] == 5).all() and (ob[:, :first] == 5).all()
        ob.fill_(5.0)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40, 200])
def test_scales_of_any_size_and_sign(m):
    # negative, zero and far-apart scales: every block is scaled on its own, in fp32
    _gpu()
    n, k = 300, 1024
    g = torch.Generator(device=DEV).manual_seed(m)
    a, b = _codes(m, k, g), _codes(n, k, g)
    sa, sb = _scales(m, 8, g), _scales(3, 8, g)
    sa[:, 1] *= -1
    sa[:, 2] = 0
    sa[:, 3] *= 1e12
    sb[:, 4] *= 1e-12
    sb[1, 5] = -sb[1, 5]
    got = csa.Fp8Matmul(a, sa, b, sb, out_dtype=torch.float32)()
    torch.cuda.synchronize()
    _check(got, a, sa, b, sb)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 1024, 4096), (70, 1024, 4096), (1100, 1024, 640)])
def test_nan_codes_stay_in_their_row_and_column(m, n, k):
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(5)
    a, b = _codes(m, k, g), _codes(n, k, g)
    sa, sb = _scales(m, k // 128, g), _scales(n // 128, k // 128, g)
    clean = csa.Fp8Matmul(a, sa, b, sb, out_dtype=torch.float32)().clone()
    a[m - 1, 300] = 0x7F
    b[77, 5] = 0xFF
    got = csa.Fp8Matmul(a, sa, b, sb, out_dtype=torch.float32)()
    torch.cuda.synchronize()
    bad = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    bad[m - 1], bad[:, 77] = True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 8192, 1536), (64, 5000, 1536), (130, 1000, 4096), (3000, 2100, 1000)])
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(m, n, k):
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(9)
    a, b = _codes(m, k, g), _codes(n, k, g)
    kb = -(-k // 128)
    sa, sb = _scales(m, kb, g), _scales(-(-n // 128), kb, g)
    op = csa.Fp8Matmul(a, sa, b, sb)
    first = op().clone()
    for _ in range(20):
        op()
    assert torch.equal(op(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = csa.Fp8Matmul(a, sa, b, sb)
    other(stream=side)
    op()                                                   # both at once, on two streams
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    graphed = csa.Fp8Matmul(a, sa, b, sb)
    with torch.cuda.graph(graph):
        graphed()
        graphed()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(other._out, first) and torch.equal(graphed._out, first) and torch.equal(op._out, first)


@pytest.mark.gpu
def test_empty_matrices():
    _gpu()
    b, sb = torch.zeros(200, 256, dtype=torch.uint8, device=DEV), torch.ones(2, 2, device=DEV)
    a, sa = torch.zeros(3, 256, dtype=torch.uint8, device=DEV), torch.ones(3, 2, device=DEV)
    assert csa.Fp8Matmul(a[:0], sa[:0], b, sb)().shape == (0, 200)
    assert csa.Fp8Matmul(a, sa, b[:0], sb[:0])().shape == (3, 0)


@pytest.mark.gpu
def test_two_products_at_once_on_two_streams():
    # kernels with tensor memory of their own beside each other, of different shapes
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(1)
    ops, firsts = [], []
    for m, n, k in ((1, 8192, 1536), (60, 4096, 2048), (300, 1000, 2048), (2600, 2600, 512)):
        a, b = _codes(m, k, g), _codes(n, k, g)
        ops.append(csa.Fp8Matmul(a, _scales(m, k // 128, g), b, _scales(-(-n // 128), k // 128, g)))
        firsts.append(ops[-1]().clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(50):
        for op, st in zip(ops, streams):
            op(stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(op._out, f) for op, f in zip(ops, firsts))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(5, 77, 300), (200, 333, 700), (700, 8191, 130), (3000, 2047, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_the_default_buffer_and_contiguous_ones(m, n, k, dtype):
    # by default rows start on 32-byte boundaries (vector stores); a contiguous output of an odd
    # number of columns is stored element by element: the same bits
    _gpu()
    gen = torch.Generator(device=DEV).manual_seed(m + n)
    kb = -(-k // 128)
    a, b = _codes(m, k, gen), _codes(n, k, gen)
    sa, sb = torch.rand(m, kb, generator=gen, device=DEV), torch.rand(-(-n // 128), kb, generator=gen, device=DEV)
    got = csa.Fp8Matmul(a, sa, b, sb, out_dtype=dtype)()
    assert got.shape == (m, n) and got.stride(0) * got.element_size() % 32 == 0 and got.stride(1) == 1
    flat = torch.full((m * n + 3,), 7.0, dtype=dtype, device=DEV)
    csa.Fp8Matmul(a, sa, b, sb, out=flat[:m * n].view(m, n))()
    torch.cuda.synchronize()
    assert torch.equal(flat[:m * n].view(m, n), got) and (flat[m * n:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1100, 4000, 1300), (1990, 4801, 2500), (130, 19900, 2100), (2200, 2321, 1700)])
def test_tiles_in_one_turn_of_the_sms_and_in_several(m, n, k, dtype):
    _gpu()
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    a, b = _codes(m, k, g), _codes(n, k, g)
    kb = -(-k // 128)
    sa, sb = _scales(m, kb, g), _scales(-(-n // 128), kb, g)
    got = csa.Fp8Matmul(a, sa, b, sb, out=torch.empty(m, n, dtype=dtype, device=DEV))()
    _check(got, a, sa, b, sb, (m, n, k))
    padded = csa.Fp8Matmul(a, sa, b, sb, out_dtype=dtype)()
    torch.cuda.synchronize()
    assert torch.equal(got, padded)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 40, 200])
@pytest.mark.parametrize("ea,eb", [(-63, -63), (-100, -26), (-26, -100), (60, 40), (100, 0), (-20, 120)])
def test_scales_at_the_ends_of_the_range(m, ea, eb):
    # the product of a block's two scales at the lowest normal number, and so large that the sums (up to
    # 448^2 x 1024 < 2^28) just stay numbers.  At the low end a block's sum is about 2^13 and its bound above 2^-130,
    # far above fp32's last place there (2^-149)
    _gpu()
    n, k = 300, 1024
    g = torch.Generator(device=DEV).manual_seed(m)
    a, b = _codes(m, k, g), _codes(n, k, g)
    sign = lambda *s: torch.randint(0, 2, s, generator=g, device=DEV).float() * 2 - 1
    sa, sb = sign(m, 8) * 2.0 ** ea, sign(3, 8) * 2.0 ** eb
    sa[:, 2], sb[1, 3] = 0, 0
    got = csa.Fp8Matmul(a, sa, b, sb, out_dtype=torch.float32)()
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    _check(got, a, sa, b, sb, (m, ea, eb))


def test_sizes_that_do_not_fit_32_bits_are_refused():
    # (the C struct's fields have 32 bits: 2^32 + 16 rows would arrive as 16)
    big = 2 ** 32 + 128
    t = lambda *s, d=torch.uint8: torch.empty(s, dtype=d, device="meta")
    for m, n, k in ((big, 128, 128), (128, big, 128), (128, 128, big)):
        kb = -(-k // 128)
        with pytest.raises(csa.CsaError, match="32 bits"):
            csa.Fp8Matmul(t(m, k), t(m, kb, d=torch.float32), t(n, k), t(-(-n // 128), kb, d=torch.float32))
