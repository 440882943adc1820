"""csa_norm_rows: residual addition, RMS norm, output in the layer's type and / or E4M3 codes with one
scale per 128 elements, against a plain fp64 implementation.

Tolerances.  u(t) = finfo(t).eps / 2 is half a rounding step (bf16 2^-8, fp32 2^-24).  s = x + residual is
one fp32 rounding.  The sum of squares is at most 64 sequential additions per thread and 9 + 5 tree levels,
each 2^-24, the mean, rsqrtf (2 ulp = 2^-22) and two products add less than 16 x 2^-24: the square root halves
the sum's error, so y is within (78 / 2 + 16) 2^-24 < 2^-18 of its value.  An output in type t adds u(t), a
scale 2^-24 more (the division), a code half an E4M3 step: 2^-4 of its value, or 2^-10 among the subnormals.
"""
import ctypes

import numpy as np
import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import build as csa_build
from compressed_sparse_attention_indexer_gb300 import csa

DEV = "cuda:0"
Y_TOL = 2.0 ** -18


def reference(x, residual, weight, norm, eps):
    """s and y in fp64."""
    s = x.double()
    if residual is not None:
        s = s + residual.double()
    y = s
    if norm:
        y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    return s, y


def check(got, x, residual, weight, norm, eps, what=""):
    s, y = reference(x, residual, weight, norm, eps)
    u = torch.finfo(x.dtype).eps / 2
    y_tol = Y_TOL if norm else 2.0 ** -23
    if residual is not None:
        r = got["residual"].cpu().double()
        assert ((r - s).abs() <= (u + 2.0 ** -23) * s.abs()).all(), what
    if "out" in got:
        o = got["out"].cpu().double()
        assert ((o - y).abs() <= (u + y_tol) * y.abs() + 1e-42).all(), what
    if "codes" in got:
        n, width = x.shape
        v = got["codes"].cpu().float().double()
        scale = got["scale"].cpu().double()
        for j in range(scale.shape[1]):
            part, code = y[:, 128 * j:128 * j + 128], v[:, 128 * j:128 * j + 128]
            most = part.abs().amax(1)
            want = torch.where(most > 0, (most / 448).clamp_min(2.0 ** -126), torch.ones_like(most))
            assert ((scale[:, j] - want).abs() <= (y_tol + 2.0 ** -23) * want).all(), what
            z = part / scale[:, j:j + 1]
            tol = torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10)) + 2.0 ** -17 * z.abs()
            assert ((code - z).abs() <= tol).all(), what


# ---------------------------------------------------------------------------
# CPU: refusals

@pytest.fixture(scope="module")
def L():
    csa_build.build()
    return csa.lib()


def _call(L, **kw):
    base = dict(n=4, width=256, dtype=csa.CSA_DTYPE_BF16, norm=1, eps=1e-6, x=0x10000, x_stride=256,
                residual=0x10000, residual_stride=256, residual_out=0x10000, residual_out_stride=256,
                weight=0x10000, out=0x10000, out_stride=256, codes=0x10000, codes_stride=256, scale=0x10000,
                scale_stride=2)
    base.update(kw)
    return L.csa_norm_rows(ctypes.byref(csa.CNorm(**base)), None)


def test_empty_call_is_a_no_op(L):
    assert _call(L, n=0) == csa.CSA_OK
    assert _call(L, n=0, x=None, out=None, codes=None, scale=None) == csa.CSA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), csa.CSA_ERR_INVALID_ARG),
    (dict(width=0), csa.CSA_ERR_INVALID_ARG),
    (dict(width=32769, x_stride=40000), csa.CSA_ERR_UNSUPPORTED),
    (dict(width=16385, dtype=csa.CSA_DTYPE_F32), csa.CSA_ERR_UNSUPPORTED),
    (dict(dtype=csa.CSA_DTYPE_FP8_E4M3), csa.CSA_ERR_UNSUPPORTED),
    (dict(norm=2), csa.CSA_ERR_INVALID_ARG),
    (dict(norm=0), csa.CSA_ERR_INVALID_ARG),                       # weight without a norm
    (dict(eps=-1.0), csa.CSA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), csa.CSA_ERR_INVALID_ARG),
    (dict(x=None), csa.CSA_ERR_INVALID_ARG),
    (dict(x=0x10008), csa.CSA_ERR_INVALID_ARG),                    # not 16-byte aligned
    (dict(x_stride=255), csa.CSA_ERR_INVALID_ARG),                 # below the width
    (dict(x_stride=260), csa.CSA_ERR_INVALID_ARG),                 # rows off the 16-byte boundary
    (dict(residual_out=None), csa.CSA_ERR_INVALID_ARG),
    (dict(residual=None), csa.CSA_ERR_INVALID_ARG),
    (dict(weight=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(out=None, codes=None, scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(scale=None), csa.CSA_ERR_INVALID_ARG),
    (dict(codes=None), csa.CSA_ERR_INVALID_ARG),
    (dict(codes_stride=264), csa.CSA_ERR_INVALID_ARG),
    (dict(scale=0x10002), csa.CSA_ERR_INVALID_ARG),
    (dict(scale_stride=1), csa.CSA_ERR_INVALID_ARG),
])
def test_refusals(L, kw, code):
    assert _call(L, **kw) == code
    assert csa.last_error()


def test_null_args(L):
    assert L.csa_norm_rows(None, None) == csa.CSA_ERR_INVALID_ARG


def test_object_refusals(L):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for kw in (dict(weight=torch.ones(255, dtype=torch.bfloat16)), dict(weight=torch.ones(256)),
               dict(residual=torch.zeros(4, 256)), dict(residual=torch.zeros(3, 256, dtype=torch.bfloat16)),
               dict(residual_out=x), dict(out=torch.zeros(4, 128, dtype=torch.bfloat16)),
               dict(codes=torch.zeros(4, 256, dtype=torch.int8)), dict(codes=False, out=True, scale=torch.zeros(4, 2))):
        with pytest.raises(csa.CsaError):
            csa.NormRows(x, **kw)
    with pytest.raises(csa.CsaError):
        csa.NormRows(x, weight=torch.ones(256, dtype=torch.bfloat16), norm=False)
    assert csa.NormRows(x, norm=False, out=True, codes=False)()["out"] is x      # nothing is asked of the rows
    with pytest.raises(csa.CsaError):
        csa.NormRows(x.half())
    with pytest.raises(csa.CsaError):
        csa.NormRows(torch.zeros(256, 4, dtype=torch.bfloat16).t())     # a row's elements apart
    with pytest.raises(csa.CsaError, match="not on a CUDA device"):
        csa.NormRows(x)()                                               # no CPU path


# ---------------------------------------------------------------------------
# GPU

def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    csa_build.build()
    torch.cuda.set_device(0)


def _rows(n, width, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    return (torch.randn(n, -(-width // unit) * unit, generator=g) * std).to(dtype)[:, :width]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,width", [(1, 1), (3, 7), (33, 128), (70, 129), (5, 255), (9, 256), (4, 257), (64, 576),
                                     (2, 1000), (1, 4096), (300, 4100), (17, 7168), (400, 8200), (3, 16384)])
@pytest.mark.parametrize("norm,residual", [(True, True), (True, False), (False, True), (False, False)])
def test_matches_the_definition(n, width, dtype, norm, residual):
    _gpu()
    x = _rows(n, width, dtype, n * 13 + width, 3.0)
    r = _rows(n, width, dtype, n + width * 7) if residual else None
    w = (1 + 0.2 * _rows(1, width, torch.float32, width)[0]).to(dtype).contiguous() if norm else None
    d = lambda t: None if t is None else t.to(DEV)
    # .to() keeps the padded rows' strides only for dense tensors: rebuild them on the device
    def dev(t):
        if t is None:
            return None
        unit = 16 // t.element_size()
        b = torch.zeros(n, -(-width // unit) * unit, dtype=t.dtype, device=DEV)
        b[:, :width] = t.to(DEV)
        return b[:, :width]
    op = csa.NormRows(dev(x), d(w), dev(r), norm=norm, eps=1e-5, out=True, codes=True)
    got = op()
    torch.cuda.synchronize()
    check(got, x, r, w, norm, 1e-5, (n, width, dtype, norm, residual))
    for alone in (dict(out=True, codes=False), dict(out=False, codes=True)):   # one output gives the same bits
        one = csa.NormRows(dev(x), d(w), dev(r), norm=norm, eps=1e-5, **alone)()
        torch.cuda.synchronize()
        for k, t in one.items():
            assert torch.equal(t.contiguous().view(torch.uint8), got[k].contiguous().view(torch.uint8)), k


@pytest.mark.gpu
def test_widest_rows():
    _gpu()
    for dtype, width in ((torch.bfloat16, 32768), (torch.bfloat16, 32761), (torch.float32, 16384)):
        x = _rows(160, width, dtype, width)
        b = torch.zeros(160, 32768, dtype=dtype, device=DEV)
        b[:, :width] = x.to(DEV)
        w = torch.full((width,), 0.5, dtype=dtype)
        got = csa.NormRows(b[:, :width], w.to(DEV), out=True)()
        torch.cuda.synchronize()
        check(got, x, None, w, True, 1e-6, width)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_in_place_and_what_stays_untouched(dtype):
    # rows inside wider buffers: columns behind the width and rows behind the last keep their bytes;
    # residual_out is the residual, out is x
    _gpu()
    n, width, pitch = 37, 201, 256
    x, r = _rows(n, width, dtype, 1), _rows(n, width, dtype, 2)
    xb = torch.full((n + 2, pitch), 7.0, dtype=dtype, device=DEV)
    rb = torch.full((n + 2, pitch), 9.0, dtype=dtype, device=DEV)
    cb = torch.full((n + 2, pitch), 0x55, dtype=torch.uint8, device=DEV)
    sb = torch.full((n + 2, 5), 11.0, device=DEV)
    xb[:n, :width], rb[:n, :width] = x.to(DEV), r.to(DEV)
    got = csa.NormRows(xb[:n, :width], None, rb[:n, :width], eps=0.0, out=xb[:n, :width], codes=cb[:n, :width],
                       scale=sb[:n, :2], residual_out=rb[:n, :width])()
    torch.cuda.synchronize()
    check(got, x, r, None, True, 0.0)
    assert got["out"].data_ptr() == xb.data_ptr() and got["residual"].data_ptr() == rb.data_ptr()
    for t, v in ((xb, 7.0), (rb, 9.0), (cb, 0x55)):
        assert (t[:, width:] == v).all() and (t[n:] == v).all()
    assert (sb[:, 2:] == 11.0).all() and (sb[n:] == 11.0).all()


@pytest.mark.gpu
def test_zero_tiny_infinite_and_nan_rows():
    _gpu()
    x = torch.zeros(7, 256)
    x[1] = 1e-41                       # subnormal: the scale stays at the smallest normal number
    x[2, 5] = 3.0                      # one block all zero
    x[3, 130] = float("inf")
    x[4, 130] = float("nan")
    x[5] = -448.0
    x[6] = torch.linspace(-1e-4, 300, 256)
    got = csa.NormRows(x.to(DEV), norm=False, out=False)()
    torch.cuda.synchronize()
    scale, code = got["scale"].cpu(), got["codes"].cpu().float()
    fine = [0, 1, 2, 5, 6]
    check({"codes": got["codes"][fine], "scale": got["scale"][fine]}, x[fine], None, None, False, 0.0)
    assert (scale[0] == 1).all() and (code[0] == 0).all()
    assert (scale[1] == 2.0 ** -126).all()
    assert scale[2, 1] == 1 and scale[5, 0] == 1
    assert torch.isinf(scale[3, 1]) and torch.isnan(code[3, 130]) and (code[3, 131:] == 0).all() and scale[3, 0] == 1
    assert torch.isnan(code[4, 130]) and (code[4, 131:] == 0).all() and scale[4, 1] == 1
    # a norm of a row of zeros is zero, whatever eps > 0; a row with a NaN or an infinity is NaN throughout
    got = csa.NormRows(x.to(DEV), out=True, codes=True)()
    torch.cuda.synchronize()
    assert (got["out"][0] == 0).all() and torch.isnan(got["out"][4]).all() and torch.isnan(got["out"][3, 130])


@pytest.mark.gpu
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    _gpu()
    n, width = 300, 4100
    xb = torch.randn(n, 4104, device=DEV).bfloat16()
    op = csa.NormRows(xb[:, :width], out=True)
    first = {k: t.clone() for k, t in op().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = csa.NormRows(xb[:, :width], out=True)
    again(stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        third = csa.NormRows(xb[:, :width], out=True)()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    graphed = csa.NormRows(xb[:, :width], out=True)
    graphed()
    with torch.cuda.graph(g):
        graphed()
    for t in graphed._out.values():
        t.view(torch.uint8).zero_()
    g.replay()
    torch.cuda.synchronize()
    for other in (again._out, third, graphed._out):
        for k, t in first.items():
            assert torch.equal(t.view(torch.uint8), other[k].contiguous().view(torch.uint8)), k


@pytest.mark.gpu
def test_width_128_makes_the_fp8_indexer_key_pool():
    # normalised keys quantised on the device, written into the key pool by slot, and scored: the scores are
    # those of the pool's own values, so the codes and scales are what the indexer reads
    _gpu()
    import oracle
    from compressed_sparse_attention_indexer_gb300.workloads import BF16_CFG, Workload, make_batch, to_device
    from dataclasses import replace
    cfg = replace(BF16_CFG, idx_dtype="fp8")
    hb = make_batch(Workload("keys", cfg, B=2, S=1, L=1, seed=31), lens=[2600, 3001])
    db = to_device(hb, DEV)
    rows = int(hb["idx_k"].shape[0])
    keys = torch.randn(rows, 128, device=DEV).bfloat16()
    got = csa.NormRows(keys, torch.full((128,), 1.25, device=DEV).bfloat16())()
    slot = torch.randperm(rows, device=DEV)
    back = torch.empty_like(slot)
    back[slot] = torch.arange(rows, device=DEV)
    pool = torch.zeros_like(db["idx_k"])
    scales = torch.zeros_like(db["idx_scale"])
    csa.cache_writeback(got["codes"], slot, pool)
    csa.cache_writeback(got["scale"], slot, scales.view(-1, 1))
    db["idx_k"], db["idx_scale"] = pool, scales
    torch.cuda.synchronize()
    assert torch.equal(pool, got["codes"].view(torch.uint8)[back]) and torch.equal(scales, got["scale"][back, 0])
    dec = csa.Decoder(cfg, 2, 1, 4096)
    out = torch.zeros(2, 1024, device=DEV)
    dec.indexer_scores(csa.make_batch_struct(db), out)
    assert dec.status() == csa.CSA_OK
    values = (pool.view(torch.float8_e4m3fn).float() * scales[:, None]).double().cpu().numpy()
    for b, length in enumerate([2600, 3001]):
        off, vis = int(hb["idx_off"][b]), length // 4
        want = oracle.index_scores(hb["q_idx"][b, 0].double().numpy(), hb["w"][b, 0].double().numpy(),
                                   values[off:off + vis])
        err = np.abs(out[b, :vis].cpu().numpy() - want)
        assert err.max() <= 2e-5 * np.abs(want).max()


@pytest.mark.gpu
def test_no_rows():
    _gpu()
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    got = csa.NormRows(x, residual=x, out=True)()
    assert got["out"].shape == (0, 256) and got["codes"].shape == (0, 256) and got["scale"].shape == (0, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_of_rows_as_they_are_are_the_nearest(dtype):
    # norm = 0: the quotient y / scale decides the code; off a border by less than its own rounding it may take
    # either neighbour, elsewhere it is the fp64 quotient's
    _gpu()
    x = _rows(3000, 384, dtype, 8)
    got = csa.NormRows(x.to(DEV), norm=False)()
    torch.cuda.synchronize()
    z = x.double().view(3000, 3, 128) / got["scale"].cpu().double()[..., None]
    want = z.float().to(torch.float8_e4m3fn).double()
    code = got["codes"].cpu().double().view(3000, 3, 128)
    off = code != want
    # next to a border: half an E4M3 step from the code, to within 2^-22 of the value
    _, e = torch.frexp(z.abs().clamp_min(2.0 ** -9))
    half = torch.ldexp(torch.ones_like(z), (e - 1).clamp_min(-6) - 4)
    assert (((z - want).abs() - half).abs()[off] <= 2.0 ** -22 * z.abs()[off]).all()
    assert off.double().mean() < 1e-5


@pytest.mark.gpu
def test_rows_copied_as_they_are():
    # nothing but a tensor to fill: a copy
    _gpu()
    x = torch.randn(50, 200, device=DEV)
    out = torch.zeros(50, 208, device=DEV)
    csa.NormRows(x, norm=False, out=out[:, :200], codes=False)()
    torch.cuda.synchronize()
    assert torch.equal(out[:, :200], x) and (out[:, 200:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [130, 257, 300, 761, 768, 1497, 2048, 4092, 6001])
@pytest.mark.parametrize("residual", [False, True])
def test_many_rows_per_block(width, dtype, residual):
    # more rows than the device holds at once: the rows in flight wrap around; in place, rows' padding left alone
    _gpu()
    n = 9001 if width < 1000 else 3001
    g = torch.Generator().manual_seed(width)
    stride = -(-width // 16) * 16 + 16
    x, res = (torch.randn(n, stride, generator=g).to(dtype) for _ in range(2))
    weight = (1 + 0.1 * torch.randn(width, generator=g)).to(dtype)
    xd, rd = x.to(DEV), res.to(DEV)
    kw = dict(residual=rd[:, :width], residual_out=rd[:, :width]) if residual else {}
    got = csa.NormRows(xd[:, :width], weight=weight.to(DEV), out=xd[:, :width], codes=True, **kw)()
    torch.cuda.synchronize()
    check(got, x[:, :width], res[:, :width] if residual else None, weight, True, 1e-6, f"{width} {dtype}")
    assert torch.equal(xd[:, width:].cpu(), x[:, width:]) and torch.equal(rd[:, width:].cpu(), res[:, width:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [128, 200, 1003, 4096])
def test_out_without_the_norm_is_the_sum(width, dtype):
    # no second copy of the sum: "out" is the tensor under "residual" (codes or not); a tensor to fill is filled
    _gpu()
    g = torch.Generator().manual_seed(width)
    pad = -(-width // 16) * 16
    x, res = (torch.randn(70, pad, generator=g).to(dtype)[:, :width] for _ in range(2))
    xd, rd = x.to(DEV), res.to(DEV)
    xd, rd = (torch.nn.functional.pad(t, (0, pad - width))[:, :width] for t in (xd, rd))
    own = torch.zeros(70, pad, dtype=dtype, device=DEV)[:, :width]
    for codes in (False, True):
        got = csa.NormRows(xd, residual=rd, norm=False, out=True, codes=codes)()
        assert got["out"] is got["residual"]
        filled = csa.NormRows(xd, residual=rd, norm=False, out=own, codes=codes)()
        torch.cuda.synchronize()
        check(got, x, res, None, False, 1e-6)
        assert filled["out"] is own and torch.equal(own, got["out"])
        same = csa.NormRows(xd, norm=False, out=True, codes=codes)()
        assert same["out"] is xd
        if codes:
            check(same, x, None, None, False, 1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [128, 512])
@pytest.mark.parametrize("size", [1e-36, 1e-30, 1.0, 1e17])
def test_codes_of_rows_near_the_ends_of_the_range(width, size):
    # the scale's lower bound among them; the mean square stays inside fp32's range (eps carries the smallest
    # rows, whose squares vanish)
    _gpu()
    g = torch.Generator().manual_seed(width)
    x = torch.randn(40, width, generator=g) * size
    x[3] = 0
    x[4, :128] = 0
    weight = (1 + 0.1 * torch.randn(width, generator=g))
    got = csa.NormRows(x.to(DEV), weight=weight.to(DEV), eps=1e-6, out=True, codes=True)()
    torch.cuda.synchronize()
    check(got, x, None, weight, True, 1e-6, f"{width} {size}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width,residual", [(128, False), (100, True), (512, False), (512, True), (1003, False)])
@pytest.mark.parametrize("size", [1e-36, 3e-37, 1e-37, 1e-39])
def test_codes_of_tiny_blocks(width, residual, dtype, size):
    # blocks so small that norm factor / scale is no fp32 number: whole rows, and one block of an ordinary row
    # (where the scale is at its lower bound), zeros among their elements.  A value that is subnormal before the
    # division is off by 2^-150 at most, which is 2^-24 of the smallest scale (2^-23 allowed)
    _gpu()
    g = torch.Generator().manual_seed(width)
    unit = 16 // torch.empty(0, dtype=dtype).element_size()
    x = torch.randn(60, -(-width // unit) * unit, generator=g)
    x[:30] *= size
    x[30:, :128] *= size
    x[::7, 3::5] = 0
    if width == 128 or width == 100:
        x[30:, 0] = 0.1                                    # one block: an ordinary maximum over tiny elements
    x = x.to(dtype)
    res = torch.zeros_like(x) if residual else None
    r = None if res is None else res.to(DEV)[:, :width]
    got = csa.NormRows(x.to(DEV)[:, :width], torch.full((width,), 0.5, dtype=dtype, device=DEV), r, eps=1e-6)()
    torch.cuda.synchronize()
    s, y = reference(x[:, :width], None, torch.full((width,), 0.5, dtype=dtype), True, 1e-6)
    code, scale = got["codes"].cpu().double(), got["scale"].cpu().double()
    assert torch.isfinite(code).all()
    for j in range(scale.shape[1]):
        part = y[:, 128 * j:128 * j + 128]
        most = part.abs().amax(1)
        want = torch.where(most > 0, (most / 448).clamp_min(2.0 ** -126), torch.ones_like(most))
        assert ((scale[:, j] - want).abs() <= (Y_TOL + 2.0 ** -23) * want).all()
        z = part / scale[:, j:j + 1]
        tol = torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10)) + 2.0 ** -17 * z.abs() + 2.0 ** -23
        assert ((code[:, 128 * j:128 * j + 128] - z).abs() <= tol).all()


def test_sizes_that_do_not_fit_32_bits_are_refused():
    # (the C struct's fields have 32 bits: 2^32 + 4 rows would arrive as 4)
    for shape in ((2 ** 32 + 4, 256), (4, 2 ** 32 + 256)):
        with pytest.raises(csa.CsaError, match="32 bits"):
            csa.NormRows(torch.empty(shape, dtype=torch.bfloat16, device="meta"))
