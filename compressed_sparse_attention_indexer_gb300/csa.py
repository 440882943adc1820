"""ctypes binding of libcsa (include/csa.h): argument marshalling only.

Every step of the decode path runs in the CUDA library; this module turns
torch device tensors into the C structs and pointers the entry points take,
and raises on a non-zero return code.  If the library has not been built,
the first call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

CSA_OK, CSA_ERR_INVALID_ARG, CSA_ERR_UNSUPPORTED, CSA_ERR_WORKSPACE = 0, 1, 2, 3
CSA_ERR_CUDA, CSA_ERR_BAD_INDEX, CSA_ERR_TIMEOUT = 4, 5, 6
CSA_DTYPE_F32, CSA_DTYPE_BF16, CSA_DTYPE_FP8_E4M3 = 0, 1, 2
ERROR_NAMES = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_WORKSPACE",
               4: "CSA_ERR_CUDA", 5: "CSA_ERR_BAD_INDEX", 6: "CSA_ERR_TIMEOUT"}

EXPORTS = ("csa_decode_create", "csa_decode_destroy", "csa_indexer_topk", "csa_sparse_attn",
           "csa_decode_step", "csa_indexer_scores", "csa_topk_select", "csa_check_batch",
           "csa_get_status", "csa_last_error", "csa_last_launch_count", "csa_abi_version",
           "csa_profile_enable", "csa_profile_read", "csa_indexer_topk_static", "csa_cache_writeback",
           "csa_debug_set_wait_polls", "csa_norm_rows", "csa_fp8_matmul",
           "csa_paged_attn", "csa_paged_attn_workspace", "csa_qk_rope", "csa_kv_append",
           "csa_tree_attn", "csa_tree_attn_workspace")
STAGES = ("plan", "indexer", "topk", "attention")


class CsaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


class CConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("heads", "row_dim", "v_dim", "idx_heads", "idx_dim", "ratio", "topk", "win",
                 "hca_ratio", "dtype")] + [
        ("softmax_scale", ctypes.c_float), ("rope_base", ctypes.c_float),
        ("max_batch", ctypes.c_int32), ("max_queries_per_req", ctypes.c_int32),
        ("max_context", ctypes.c_int32), ("idx_dtype", ctypes.c_int32)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64


class CBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("S", ctypes.c_int32), ("ctx_len", _P), ("ctx_len_host", _P),
                ("q", _P), ("q_idx", _P), ("w", _P),
                ("raw_kv", _P), ("raw_off", _P), ("raw_stride", _I64), ("raw_rows", _I64),
                ("cmp_kv", _P), ("cmp_off", _P), ("cmp_stride", _I64), ("cmp_rows", _I64),
                ("idx_k", _P), ("idx_off", _P), ("idx_stride", _I64), ("idx_rows", _I64),
                ("hca_kv", _P), ("hca_off", _P), ("hca_stride", _I64), ("hca_rows", _I64),
                ("idx_scale", _P),
                ("raw_table", _P), ("cmp_table", _P), ("idx_table", _P), ("hca_table", _P),
                ("raw_block", ctypes.c_int32), ("cmp_block", ctypes.c_int32),
                ("idx_block", ctypes.c_int32), ("hca_block", ctypes.c_int32),
                ("table_stride", ctypes.c_int32)]


class CNorm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "width", "dtype", "norm")] + [
        ("eps", ctypes.c_float), ("x", _P), ("x_stride", _I64), ("residual", _P), ("residual_stride", _I64),
        ("residual_out", _P), ("residual_out_stride", _I64), ("weight", _P), ("out", _P), ("out_stride", _I64),
        ("codes", _P), ("codes_stride", _I64), ("scale", _P), ("scale_stride", _I64)]


class CFp8Mm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "out_dtype")] + [
        ("a", _P), ("a_stride", _I64), ("a_scale", _P), ("a_scale_stride", _I64),
        ("b", _P), ("b_stride", _I64), ("b_scale", _P), ("b_scale_stride", _I64),
        ("out", _P), ("out_stride", _I64), ("status", _P)]


class CPaged(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "S", "heads", "kv_heads", "dim", "kv_dtype", "win", "max_len")] + [
        ("softmax_scale", ctypes.c_float), ("block", ctypes.c_int32), ("table_stride", ctypes.c_int32),
        ("ctx_len", _P), ("q", _P), ("q_stride", _I64), ("k", _P), ("v", _P), ("k_stride", _I64), ("v_stride", _I64),
        ("rows", _I64), ("k_scale", _P), ("v_scale", _P), ("scale_stride", _I64), ("off", _P), ("table", _P),
        ("out", _P), ("out_stride", _I64), ("lse", _P), ("status", _P), ("workspace", _P), ("workspace_bytes", _I64)]


class CTree(ctypes.Structure):
    _fields_ = [("base", CPaged), ("tree", _P), ("count", _P), ("pos", _P)]


class CRope(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "q_heads", "k_heads", "dim", "dtype", "norm")] + [
        ("eps", ctypes.c_float), ("rope_dim", ctypes.c_int32), ("rope_at", ctypes.c_int32), ("halves", ctypes.c_int32),
        ("base", ctypes.c_float), ("freq", _P), ("pos", _P), ("q", _P), ("q_stride", _I64), ("q_weight", _P),
        ("q_out", _P), ("q_out_stride", _I64), ("k", _P), ("k_stride", _I64), ("k_weight", _P), ("k_out", _P),
        ("k_out_stride", _I64)]


class CAppend(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "S", "q_heads", "kv_heads", "dim", "dtype", "kv_dtype", "norm")] + [
        ("eps", ctypes.c_float), ("rope_dim", ctypes.c_int32), ("rope_at", ctypes.c_int32), ("halves", ctypes.c_int32),
        ("base", ctypes.c_float), ("freq", _P), ("pos", _P), ("ctx_len", _P), ("count", _P), ("slot", _P), ("off", _P),
        ("table", _P), ("block", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("rows", _I64),
        ("q", _P), ("q_stride", _I64), ("q_weight", _P), ("q_out", _P), ("q_out_stride", _I64),
        ("k", _P), ("k_stride", _I64), ("k_weight", _P), ("v", _P), ("v_stride", _I64),
        ("k_pool", _P), ("k_pool_stride", _I64), ("v_pool", _P), ("v_pool_stride", _I64),
        ("k_scale", _P), ("v_scale", _P), ("scale_stride", _I64), ("status", _P)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def lib(path: str | None = None):
    """Loads libcsa; raises if it has not been built (no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or os.environ.get("CSA_LIB") or _build.LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"libcsa is not built ({p} missing): run "
                                   "compressed_sparse_attention_indexer_gb300.build.build()")
            L = ctypes.CDLL(p)
            i32, vp = ctypes.c_int32, ctypes.c_void_p
            H = ctypes.c_void_p
            L.csa_decode_create.argtypes = [ctypes.POINTER(CConfig), ctypes.POINTER(H)]
            L.csa_decode_destroy.argtypes = [H]
            L.csa_decode_destroy.restype = None
            L.csa_indexer_topk.argtypes = [H, ctypes.POINTER(CBatch), vp, vp, vp]
            L.csa_sparse_attn.argtypes = [H, ctypes.POINTER(CBatch), vp, vp, vp, vp, vp]
            L.csa_decode_step.argtypes = [H, ctypes.POINTER(CBatch), vp, vp, vp, vp, vp]
            L.csa_indexer_scores.argtypes = [H, ctypes.POINTER(CBatch), vp, ctypes.c_int64, i32, vp]
            L.csa_topk_select.argtypes = [H, i32, vp, ctypes.c_int64, vp, vp, vp, vp]
            L.csa_check_batch.argtypes = [ctypes.POINTER(CConfig), ctypes.POINTER(CBatch)]
            L.csa_get_status.argtypes = [H, vp]
            L.csa_last_error.restype = ctypes.c_char_p
            L.csa_last_launch_count.argtypes = [H]
            L.csa_last_launch_count.restype = i32
            L.csa_abi_version.restype = i32
            L.csa_profile_enable.argtypes = [H, i32]
            L.csa_profile_read.argtypes = [H, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32)]
            L.csa_debug_set_wait_polls.argtypes = [H, i32]
            L.csa_indexer_topk_static.argtypes = [ctypes.POINTER(CConfig), ctypes.POINTER(CBatch), vp,
                                                  vp, vp, vp]
            L.csa_cache_writeback.argtypes = [vp, ctypes.c_int64, vp, i32, vp, ctypes.c_int64,
                                              ctypes.c_int64, ctypes.c_int64, vp, vp]
            L.csa_norm_rows.argtypes = [ctypes.POINTER(CNorm), vp]
            L.csa_fp8_matmul.argtypes = [ctypes.POINTER(CFp8Mm), vp]
            L.csa_paged_attn.argtypes = [ctypes.POINTER(CPaged), vp]
            L.csa_qk_rope.argtypes = [ctypes.POINTER(CRope), vp]
            L.csa_kv_append.argtypes = [ctypes.POINTER(CAppend), vp]
            L.csa_tree_attn.argtypes = [ctypes.POINTER(CTree), vp]
            L.csa_tree_attn_workspace.argtypes = [i32]
            L.csa_tree_attn_workspace.restype = ctypes.c_int64
            L.csa_paged_attn_workspace.argtypes = [i32]
            L.csa_paged_attn_workspace.restype = ctypes.c_int64
            for name in ("csa_decode_create", "csa_indexer_topk", "csa_sparse_attn", "csa_decode_step",
                         "csa_indexer_scores", "csa_topk_select", "csa_check_batch", "csa_get_status",
                         "csa_profile_enable", "csa_profile_read", "csa_indexer_topk_static",
                         "csa_cache_writeback", "csa_debug_set_wait_polls", "csa_norm_rows",
                         "csa_fp8_matmul", "csa_paged_attn", "csa_qk_rope", "csa_kv_append",
                         "csa_tree_attn"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def last_error() -> str:
    return lib().csa_last_error().decode()


def _check(rc: int):
    if rc != CSA_OK:
        raise CsaError(rc, last_error())


def make_config(cfg, max_batch: int, max_queries: int, max_context: int) -> CConfig:
    """C config from a workloads.CsaConfig."""
    return CConfig(heads=cfg.H, row_dim=cfg.D, v_dim=cfg.V, idx_heads=cfg.Hi, idx_dim=cfg.Di,
                   ratio=cfg.ratio, topk=cfg.topk, win=cfg.win, hca_ratio=cfg.hca_ratio,
                   dtype=CSA_DTYPE_BF16 if cfg.dtype == "bf16" else CSA_DTYPE_F32,
                   softmax_scale=cfg.softmax_scale, rope_base=cfg.rope_base,
                   max_batch=max_batch, max_queries_per_req=max_queries, max_context=max_context,
                   idx_dtype=CSA_DTYPE_FP8_E4M3 if getattr(cfg, "idx_dtype", "") == "fp8" else 0)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def make_batch_struct(batch: dict, ctx_len_host=None) -> CBatch:
    """C batch from a dict of device tensors (see workloads.make_batch/to_device).

    ctx_len_host: optional int32 CPU tensor with the same lengths (kept alive by
    the caller while the struct is in use)."""
    def rows(t):
        return 0 if t is None else int(t.shape[0])
    return CBatch(
        B=int(batch["B"]), S=int(batch["S"]), ctx_len=_ptr(batch["ctx_len"]),
        ctx_len_host=_ptr(ctx_len_host),
        q=_ptr(batch["q"]), q_idx=_ptr(batch["q_idx"]), w=_ptr(batch["w"]),
        raw_kv=_ptr(batch["raw_kv"]), raw_off=_ptr(batch.get("raw_off")),
        raw_stride=int(batch["raw_stride"]), raw_rows=rows(batch["raw_kv"]),
        cmp_kv=_ptr(batch["cmp_kv"]), cmp_off=_ptr(batch.get("cmp_off")),
        cmp_stride=int(batch["cmp_stride"]), cmp_rows=rows(batch["cmp_kv"]),
        idx_k=_ptr(batch["idx_k"]), idx_off=_ptr(batch.get("idx_off")),
        idx_stride=int(batch["idx_stride"]), idx_rows=rows(batch["idx_k"]),
        hca_kv=_ptr(batch.get("hca_kv")), hca_off=_ptr(batch.get("hca_off")),
        hca_stride=int(batch.get("hca_stride") or 0), hca_rows=rows(batch.get("hca_kv")),
        idx_scale=_ptr(batch.get("idx_scale")),
        raw_table=_ptr(batch.get("raw_table")), cmp_table=_ptr(batch.get("cmp_table")),
        idx_table=_ptr(batch.get("idx_table")), hca_table=_ptr(batch.get("hca_table")),
        raw_block=int(batch.get("raw_block") or 0), cmp_block=int(batch.get("cmp_block") or 0),
        idx_block=int(batch.get("idx_block") or 0), hca_block=int(batch.get("hca_block") or 0),
        table_stride=int(batch.get("table_stride") or 0))


def check_batch(cconfig: CConfig, cbatch: CBatch) -> int:
    """Host-side validation only (no GPU); returns the C return code."""
    return lib().csa_check_batch(ctypes.byref(cconfig), ctypes.byref(cbatch))


def indexer_topk_static(cconfig: CConfig, cb: CBatch, topk_idx, topk_cnt, status=None, stream=None):
    """Steps (a)+(b) without a handle or any device allocation (scratch in the
    library's static device array; see csa_indexer_topk_static in csa.h)."""
    _check(lib().csa_indexer_topk_static(ctypes.byref(cconfig), ctypes.byref(cb), _ptr(topk_idx),
                                         _ptr(topk_cnt), _ptr(status), _stream(stream)))


def cache_writeback(rows, slot, pool, status=None, stream=None):
    """pool[slot[t]] = rows[t] on the device (see csa_cache_writeback in csa.h).

    rows [n, ...] and pool [pool_rows, ...]: device tensors whose rows are
    contiguous and of the same byte size; slot [n] int64 (negative = skip)."""
    n = int(rows.shape[0])
    row_bytes = rows[0].numel() * rows.element_size() if n else 0
    assert n == 0 or pool[0].numel() * pool.element_size() == row_bytes, "row sizes differ"
    _check(lib().csa_cache_writeback(_ptr(rows), int(rows.stride(0)) * rows.element_size(), _ptr(slot),
                                     n, _ptr(pool), int(pool.stride(0)) * pool.element_size(),
                                     int(pool.shape[0]), int(row_bytes), _ptr(status), _stream(stream)))


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(stream) if not hasattr(stream, "cuda_stream") else stream.cuda_stream


class Decoder:
    """One csa_handle: a fixed layer shape plus its device workspace."""

    def __init__(self, cfg, max_batch: int, max_queries: int, max_context: int):
        self.cfg = cfg
        self.cconfig = make_config(cfg, max_batch, max_queries, max_context)
        h = ctypes.c_void_p()
        _check(lib().csa_decode_create(ctypes.byref(self.cconfig), ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            lib().csa_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- entry points (tensors must be on the current device) --------------
    def decode_step(self, cb: CBatch, out, lse=None, topk_idx=None, topk_cnt=None, stream=None):
        _check(lib().csa_decode_step(self.handle, ctypes.byref(cb), _ptr(out), _ptr(lse),
                                     _ptr(topk_idx), _ptr(topk_cnt), _stream(stream)))

    def indexer_topk(self, cb: CBatch, topk_idx, topk_cnt, stream=None):
        _check(lib().csa_indexer_topk(self.handle, ctypes.byref(cb), _ptr(topk_idx), _ptr(topk_cnt),
                                      _stream(stream)))

    def sparse_attn(self, cb: CBatch, topk_idx, topk_cnt, out, lse=None, stream=None):
        _check(lib().csa_sparse_attn(self.handle, ctypes.byref(cb), _ptr(topk_idx), _ptr(topk_cnt),
                                     _ptr(out), _ptr(lse), _stream(stream)))

    def indexer_scores(self, cb: CBatch, scores, score_all: bool = True, stream=None):
        _check(lib().csa_indexer_scores(self.handle, ctypes.byref(cb), _ptr(scores),
                                        int(scores.stride(0)), 1 if score_all else 0, _stream(stream)))

    def topk_select(self, scores, n, topk_idx, topk_cnt, stream=None):
        _check(lib().csa_topk_select(self.handle, int(scores.shape[0]), _ptr(scores),
                                     int(scores.stride(0)), _ptr(n), _ptr(topk_idx), _ptr(topk_cnt),
                                     _stream(stream)))

    def status(self, stream=None) -> int:
        """Synchronises and returns (and clears) the device status code."""
        return lib().csa_get_status(self.handle, _stream(stream))

    def last_launch_count(self) -> int:
        return lib().csa_last_launch_count(self.handle)

    def debug_wait_polls(self, polls: int):
        """Test hook: the attention tile kernel's consumer waits give up after
        `polls` polls (0: at once); negative restores the default."""
        _check(lib().csa_debug_set_wait_polls(self.handle, int(polls)))

    def profile(self, enable: bool):
        _check(lib().csa_profile_enable(self.handle, 1 if enable else 0))

    def profile_read(self) -> dict:
        """{stage: (milliseconds, launches)} since the last read."""
        ms = (ctypes.c_float * 4)()
        n = (ctypes.c_int32 * 4)()
        _check(lib().csa_profile_read(self.handle, ms, n))
        return {STAGES[i]: (float(ms[i]), int(n[i])) for i in range(4)}


# -- operators around the step ------------------------------------------------
# Each object keeps one call's arguments (the C struct), its output buffers and
# references to the tensors it points at, and launches when called; a serving
# loop builds it once and calls it every step on the same buffers.  Like a
# handle, an object belongs to the device of its tensors and is used with that
# device current; its calls share its output buffers, so they must be ordered.

_CTYPE = {"torch.bfloat16": CSA_DTYPE_BF16, "torch.float32": CSA_DTYPE_F32}


def _dtype_code(t) -> int:
    c = _CTYPE.get(str(t.dtype))
    if c is None:
        raise CsaError(CSA_ERR_UNSUPPORTED, f"dtype must be bfloat16 or float32, got {t.dtype}")
    return c


def _bad(msg: str):
    raise CsaError(CSA_ERR_INVALID_ARG, msg)


def _int32(**sizes):
    """Refuses sizes that the C structs' 32-bit fields would silently cut."""
    for name, v in sizes.items():
        if not -2 ** 31 <= int(v) < 2 ** 31:
            raise CsaError(CSA_ERR_UNSUPPORTED, f"{name} = {v} does not fit 32 bits")


def _rows2d(name: str, t, n: int, width: int, dtype=None):
    """A matrix [n, width] whose rows are contiguous (any row stride)."""
    if t.dim() != 2 or tuple(t.shape) != (n, width):
        _bad(f"{name} must have shape ({n}, {width}), got {tuple(t.shape)}")
    if width > 1 and t.stride(1) != 1:
        _bad(f"{name}: the elements of a row must be contiguous")
    if dtype is not None and t.dtype != dtype:
        _bad(f"{name} must be {dtype}, got {t.dtype}")


def _row_stride(t, unit: int = 1) -> int:
    """Row stride of [n, width]; a single row's stride is never used and given as a valid one."""
    return int(t.stride(0)) if t.shape[0] > 1 else -(-int(t.shape[1]) // unit) * unit


def _empty_rows(like, n: int, width: int, dtype, align: int = 16):
    """[n, width] whose rows start on boundaries of `align` bytes."""
    import torch
    unit = align // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(n, -(-width // unit) * unit, dtype=dtype, device=like.device)[:, :width]


class _Operator:
    """What the operators' objects share: the tensors kept alive, the device and the launch."""

    def _bind(self, entry, struct, tensors):
        self._entry, self.struct, self._arg = entry, struct, ctypes.byref(struct)
        self._keep = [t for t in tensors if t is not None]
        devs = {t.device for t in self._keep}
        if len(devs) != 1:
            _bad(f"tensors on different devices: {sorted(map(str, devs))}")
        dev = devs.pop()
        self.device = dev.index if dev.type == "cuda" else None

    def _launch(self, stream):
        import torch
        if self.device is None:
            _bad("the tensors are not on a CUDA device")
        if torch.cuda.current_device() != self.device:
            _bad(f"the tensors are on cuda:{self.device}, which is not the current device")
        _check(self._entry(self._arg, torch._C._cuda_getCurrentRawStream(self.device) if stream is None
                           else _stream(stream)))


class NormRows(_Operator):
    """csa_norm_rows: residual addition, RMS norm, output in x's dtype and / or E4M3 codes with scales.

    x [n, width] bf16 or fp32, residual [n, width] (residual_out: where the sum goes, a buffer of the
    object by default, `residual` itself for in place), weight [width] or None (ones).  norm=False:
    the rows as they are.  out / codes: which outputs to make, or the tensors to fill (codes uint8 or
    float8_e4m3fn [n, width], scale fp32 [n, ceil(width / 128)]).  Calling the object returns
    {"residual", "out", "codes", "scale"} as far as they are made.  out=True without the norm is no copy:
    out is x itself, or with a residual the sum (the tensor under "residual")."""

    def __init__(self, x, weight=None, residual=None, norm: bool = True, eps: float = 1e-6, out=False,
                 codes=True, scale=None, residual_out=None):
        import torch
        dt = _dtype_code(x)
        if x.dim() != 2:
            _bad("x must have two dimensions")
        n, width = (int(v) for v in x.shape)
        _int32(n=n, width=width)
        _rows2d("x", x, n, width)
        if residual is not None:
            _rows2d("residual", residual, n, width, x.dtype)
            if residual_out is None:
                residual_out = _empty_rows(x, n, width, x.dtype)
            _rows2d("residual_out", residual_out, n, width, x.dtype)
        elif residual_out is not None:
            _bad("residual_out given without residual")
        if weight is not None and (tuple(weight.shape) != (width,) or weight.dtype != x.dtype or
                                   not weight.is_contiguous()):
            _bad(f"weight must be contiguous {x.dtype} of shape ({width},)")
        if weight is not None and not norm:
            _bad("weight given with norm=False")
        given = out is True and not norm               # the rows asked for are there already
        if out is True:
            out = _empty_rows(x, n, width, x.dtype) if norm else x if residual is None else residual_out
        if codes is True:
            codes = _empty_rows(x, n, width, torch.uint8)
        out, codes = (None if t is False else t for t in (out, codes))
        if out is not None:
            _rows2d("out", out, n, width, x.dtype)
        if codes is not None:
            if codes.dtype not in (torch.uint8, torch.float8_e4m3fn):
                _bad(f"codes must be uint8 or float8_e4m3fn, got {codes.dtype}")
            _rows2d("codes", codes, n, width)
            if scale is None:
                scale = torch.empty(n, -(-width // 128), dtype=torch.float32, device=x.device)
            _rows2d("scale", scale, n, -(-width // 128), torch.float32)
        elif scale is not None:
            _bad("scale given without codes")
        unit = 8 if dt == CSA_DTYPE_BF16 else 4
        st = CNorm(n=n, width=width, dtype=dt, norm=1 if norm else 0, eps=eps, x=_ptr(x), x_stride=_row_stride(x, unit),
                   weight=_ptr(weight))
        self._idle = given and residual is None and codes is None
        written = out if not given or codes is None else None
        for name, t, u in (("residual", residual, unit), ("residual_out", residual_out, unit), ("out", written, unit),
                           ("codes", codes, 16), ("scale", scale, 1)):
            if t is not None:
                setattr(st, name, _ptr(t))
                setattr(st, name + "_stride", _row_stride(t, u))
        self._bind(lib().csa_norm_rows, st, (x, weight, residual, residual_out, out, codes, scale))
        self._out = {}
        if residual is not None:
            self._out["residual"] = residual_out
        if out is not None:
            self._out["out"] = out
        if codes is not None:
            self._out["codes"], self._out["scale"] = codes.view(torch.float8_e4m3fn), scale

    def __call__(self, stream=None) -> dict:
        if not self._idle:
            self._launch(stream)
        return self._out


_E4M3_DTYPES = ("torch.uint8", "torch.float8_e4m3fn")


def _status_word(status):
    if status is not None and (str(status.dtype) != "torch.int32" or status.numel() != 1):
        _bad("status must be one int32")


class Fp8Matmul(_Operator):
    """csa_fp8_matmul: out [M, N] = a [M, K] times b [N, K] transposed, both E4M3 codes (uint8 or
    float8_e4m3fn) with fp32 scales a_scale [M, ceil(K / 128)] and b_scale [ceil(N / 128), ceil(K / 128)].

    out: the tensor to fill (bf16 or fp32), by default a buffer of the object in out_dtype whose rows
    start on 32-byte boundaries (a view of a wider buffer where N * its size is no multiple of 32).
    status: an int32 on the device that records a wait that gave up.  Calling the object returns out."""

    def __init__(self, a, a_scale, b, b_scale, out=None, out_dtype=None, status=None):
        import torch
        for name, t in (("a", a), ("b", b)):
            if t.dim() != 2 or str(t.dtype) not in _E4M3_DTYPES:
                _bad(f"{name} must be a matrix of uint8 or float8_e4m3fn")
        (m, k), n = (int(v) for v in a.shape), int(b.shape[0])
        _int32(M=m, N=n, K=k)
        kb = -(-k // 128)
        _rows2d("a", a, m, k)
        _rows2d("b", b, n, k)
        _rows2d("a_scale", a_scale, m, kb, torch.float32)
        _rows2d("b_scale", b_scale, -(-n // 128), kb, torch.float32)
        if out is None:
            out = _empty_rows(a, m, n, out_dtype or torch.bfloat16, 32)
        elif out_dtype is not None and out.dtype != out_dtype:
            _bad(f"out is {out.dtype}, not {out_dtype}")
        _rows2d("out", out, m, n)
        _status_word(status)
        st = CFp8Mm(M=m, N=n, K=k, out_dtype=_dtype_code(out), status=_ptr(status))
        for name, t, u in (("a", a, 16), ("a_scale", a_scale, 1), ("b", b, 16), ("b_scale", b_scale, 1), ("out", out, 1)):
            setattr(st, name, _ptr(t))
            setattr(st, name + "_stride", _row_stride(t, u))
        self._bind(lib().csa_fp8_matmul, st, (a, a_scale, b, b_scale, out, status))
        self._out = out

    def __call__(self, stream=None):
        self._launch(stream)
        return self._out


def paged_attn_workspace(dim: int) -> int:
    """Bytes of workspace csa_paged_attn needs on the current device (dim: 64, 128 or 256)."""
    return int(lib().csa_paged_attn_workspace(int(dim)))


class PagedAttention(_Operator):
    """csa_paged_attn: dense causal attention of each request's S newest tokens over its cache.

    q [B, S, heads, dim] bf16; k, v [rows, kv_heads, dim] bf16, or E4M3 codes (uint8 or float8_e4m3fn) with
    k_scale, v_scale fp32 [rows, kv_heads]; ctx_len [B] int32 including the S new tokens; the rows of a
    request through table [B, blocks] int32 and block, or off [B] int64.  max_len bounds every length
    (default with a table: what the table can hold).  win: sliding window (0: none).  scale <= 0:
    1/sqrt(dim).  out (bf16, like q), lse (fp32 [B, S, heads]; False: not made), workspace (uint8, at
    least paged_attn_workspace(dim) bytes) are buffers of the object by default.  Calling the object
    returns {"out", "lse"}."""

    def __init__(self, q, k, v, ctx_len, table=None, block: int = 0, off=None, k_scale=None, v_scale=None,
                 win: int = 0, scale: float = 0.0, max_len: int | None = None, out=None, lse=True, status=None,
                 workspace=None):
        st, tensors, self._out = self._paged(q, k, v, ctx_len, table, block, off, k_scale, v_scale, win, scale, max_len, out,
                                             lse, status, workspace, paged_attn_workspace)
        self._bind(lib().csa_paged_attn, st, tensors)

    def _paged(self, q, k, v, ctx_len, table, block, off, k_scale, v_scale, win, scale, max_len, out, lse, status, workspace,
               workspace_bytes):
        """The C struct, the tensors it points at and what the call returns."""
        import torch
        if q.dim() != 4 or k.dim() != 3:
            _bad("q must be [B, S, heads, dim] and k, v [rows, kv_heads, dim]")
        b, s, heads, dim = (int(x) for x in q.shape)
        rows, kv_heads = int(k.shape[0]), int(k.shape[1])
        _int32(B=b, S=s, heads=heads, kv_heads=kv_heads, dim=dim, win=win, block=block)
        if out is None:
            out = torch.empty(b, s, heads, dim, dtype=q.dtype, device=q.device)
        strides = []
        for name, t in (("q", q), ("out", out)):
            if tuple(t.shape) != (b, s, heads, dim) or t.dtype != torch.bfloat16:
                _bad(f"{name} must be bfloat16 of shape ({b}, {s}, {heads}, {dim})")
            if (dim > 1 and t.stride(3) != 1) or (heads > 1 and t.stride(2) != dim):
                _bad(f"{name}: a token's heads must be contiguous")
            step = t.stride(1) if s > 1 else t.stride(0) if b > 1 else heads * dim
            if b > 1 and s > 1 and t.stride(0) != s * step:
                _bad(f"{name}: the tokens must be evenly spaced")
            strides.append(int(step))
        fp8 = str(k.dtype) in _E4M3_DTYPES
        for name, t in (("k", k), ("v", v)):
            if tuple(t.shape) != (rows, kv_heads, dim) or (str(t.dtype) not in _E4M3_DTYPES if fp8
                                                           else t.dtype != torch.bfloat16):
                _bad(f"{name} must be bfloat16 or E4M3 codes, like k, of shape ({rows}, {kv_heads}, {dim})")
            if (dim > 1 and t.stride(2) != 1) or (kv_heads > 1 and t.stride(1) != dim):
                _bad(f"{name}: the heads of a row must be contiguous")
        if fp8:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is None:
                    _bad(f"{name} is needed with E4M3 codes")
                _rows2d(name, t, rows, kv_heads, torch.float32)
            if rows > 1 and k_scale.stride(0) != v_scale.stride(0):
                _bad("k_scale and v_scale must have the same row stride")
        elif k_scale is not None or v_scale is not None:
            _bad("scales given with a bfloat16 pool")
        if tuple(ctx_len.shape) != (b,) or ctx_len.dtype != torch.int32 or not ctx_len.is_contiguous():
            _bad(f"ctx_len must be contiguous int32 of shape ({b},)")
        if (table is None) == (off is None):
            _bad("give either table and block, or off")
        if table is not None:
            if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != b or not table.is_contiguous():
                _bad(f"table must be contiguous int32 of shape ({b}, blocks)")
            if max_len is None:
                max_len = int(table.shape[1]) * int(block)
        else:
            if off.dtype != torch.int64 or tuple(off.shape) != (b,) or not off.is_contiguous():
                _bad(f"off must be contiguous int64 of shape ({b},)")
            if max_len is None:
                _bad("max_len is needed with off")
        _int32(max_len=max_len, table_stride=0 if table is None else table.shape[1])
        if lse is True:
            lse = torch.empty(b, s, heads, dtype=torch.float32, device=q.device)
        elif lse is False:
            lse = None
        if lse is not None and (tuple(lse.shape) != (b, s, heads) or lse.dtype != torch.float32 or
                                not lse.is_contiguous()):
            _bad(f"lse must be contiguous float32 of shape ({b}, {s}, {heads})")
        _status_word(status)
        if workspace is not None and not workspace.is_contiguous():
            _bad("workspace must be contiguous")
        if workspace is None and q.is_cuda:
            with torch.cuda.device(q.device):
                workspace = torch.empty(workspace_bytes(dim), dtype=torch.uint8, device=q.device)
        st = CPaged(B=b, S=s, heads=heads, kv_heads=kv_heads, dim=dim,
                    kv_dtype=CSA_DTYPE_FP8_E4M3 if fp8 else CSA_DTYPE_BF16, win=win, max_len=max_len,
                    softmax_scale=scale, block=block, table_stride=0 if table is None else int(table.shape[1]),
                    ctx_len=_ptr(ctx_len), q=_ptr(q), q_stride=strides[0], k=_ptr(k), v=_ptr(v),
                    k_stride=int(k.stride(0)) if rows > 1 else kv_heads * dim,
                    v_stride=int(v.stride(0)) if rows > 1 else kv_heads * dim, rows=rows,
                    k_scale=_ptr(k_scale), v_scale=_ptr(v_scale),
                    scale_stride=0 if not fp8 else int(k_scale.stride(0)) if rows > 1 else kv_heads,
                    off=_ptr(off), table=_ptr(table), out=_ptr(out), out_stride=strides[1], lse=_ptr(lse),
                    status=_ptr(status), workspace=_ptr(workspace),
                    workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size())
        return st, (q, k, v, ctx_len, table, off, k_scale, v_scale, out, lse, status, workspace), \
            {"out": out} if lse is None else {"out": out, "lse": lse}

    def __call__(self, stream=None) -> dict:
        self._launch(stream)
        return self._out


def tree_attn_workspace(dim: int) -> int:
    """Bytes of workspace csa_tree_attn needs on the current device (dim: 64, 128 or 256)."""
    return int(lib().csa_tree_attn_workspace(int(dim)))


def tree_masks(parent, win: int = 0):
    """The masks csa_tree_attn takes, int64 [B, S, ceil(S / 64)], of trees given by each draft's parent: parent [B, S],
    an earlier draft of the request, or negative for a draft that follows the context's last token.  win: the sliding
    window (0: none), which the attention applies to the rows before the drafts alone: ancestors `win` and more
    tokens back are left out."""
    import torch
    if parent.dim() != 2 or parent.dtype not in (torch.int32, torch.int64):
        _bad("parent must be int32 or int64 of shape (B, S)")
    if win < 0:
        _bad("win must be >= 0")
    b, s = parent.shape
    if bool((parent >= torch.arange(s, device=parent.device)).any()):
        _bad("a draft's parent must come before it")
    masks = torch.zeros(b, s, -(-s // 64), dtype=torch.int64, device=parent.device)
    depth = torch.zeros(b, s, dtype=torch.int64, device=parent.device)
    at = torch.arange(b, device=parent.device)
    for t in range(s):
        p = parent[:, t].long()
        seen = torch.where((p >= 0)[:, None], masks[at, p.clamp_min(0)], 0)
        depth[:, t] = torch.where(p >= 0, depth[at, p.clamp_min(0)] + 1, 0)
        if win > 0 and t > 0:
            near = torch.zeros(b, masks.shape[2] * 64, dtype=torch.int64, device=parent.device)
            near[:, :t] = depth[:, :t] > depth[:, t:t + 1] - win
            bits = near.view(b, -1, 64) << torch.arange(64, device=parent.device)
            seen = seen & bits.sum(2)
        masks[:, t] = seen
        masks[:, t, t // 64] |= -2 ** 63 if t % 64 == 63 else 1 << (t % 64)
    return masks


class TreeAttention(PagedAttention):
    """csa_tree_attn: attention of a tree of S drafted tokens per request over its cache.

    tree [B, S, ceil(S / 64)] int64: bit t % 64 of word t / 64 set where a draft sees draft t, itself included
    (tree_masks makes them of parents; with a window give it that too: here it hides rows before the drafts only).
    count [B] int32: the real drafts of each request, the first of its S (None: all S); they lie in the last rows of
    its context.  pos [B, S] int32: the drafts' positions, needed with a window.
    workspace: at least tree_attn_workspace(dim) bytes.  The rest is as in PagedAttention."""

    def __init__(self, q, k, v, ctx_len, tree, count=None, pos=None, table=None, block: int = 0, off=None, k_scale=None,
                 v_scale=None, win: int = 0, scale: float = 0.0, max_len: int | None = None, out=None, lse=True,
                 status=None, workspace=None):
        import torch
        base, tensors, self._out = self._paged(q, k, v, ctx_len, table, block, off, k_scale, v_scale, win, scale, max_len,
                                               out, lse, status, workspace, tree_attn_workspace)
        b, s = int(q.shape[0]), int(q.shape[1])
        _flat("tree", tree, torch.int64, (b, s, -(-s // 64)))
        _flat("count", count, torch.int32, (b,))
        _flat("pos", pos, torch.int32, [(b, s), (b * s,)])
        if win > 0 and pos is None:
            _bad("pos is needed with a window")
        st = CTree(base=base, tree=_ptr(tree), count=_ptr(count), pos=_ptr(pos))
        self._bind(lib().csa_tree_attn, st, (*tensors, tree, count, pos))


def _tokens(name: str, t, lead, heads: int, dim: int, dtype):
    """Heads of tokens [*lead, heads, dim]: a token's heads together, the tokens evenly spaced.
    Returns the elements from one token to the next."""
    shape = (*lead, heads, dim)
    if tuple(t.shape) != shape or t.dtype != dtype:
        _bad(f"{name} must be {dtype} of shape {shape}, got {t.dtype} {tuple(t.shape)}")
    if (dim > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != dim):
        _bad(f"{name}: a token's heads must be contiguous")
    step, width = None, 1
    for size, stride in zip(reversed(lead), reversed(t.stride()[:len(lead)])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != width * step:
            _bad(f"{name}: the tokens must be evenly spaced")
        width *= size
    return heads * dim if step is None else int(step)


def _head_weight(name: str, weight, like, dim: int, norm: bool):
    if weight is not None and not norm:
        _bad(f"{name} given with norm=False")
    if weight is not None and (tuple(weight.shape) != (dim,) or weight.dtype != like.dtype or not weight.is_contiguous()):
        _bad(f"{name} must be contiguous {like.dtype} of shape ({dim},)")


def _flat(name: str, t, dtype, shape):
    if t is not None and (t.dtype != dtype or tuple(t.shape) not in (shape if isinstance(shape, list) else [shape]) or
                          not t.is_contiguous()):
        _bad(f"{name} must be contiguous {dtype} of shape {shape}, got {t.dtype} {tuple(t.shape)}")


class QkRope(_Operator):
    """csa_qk_rope: each query and key head normed (norm=True: RMS over its dims, times q_weight / k_weight [dim],
    None: ones) and rotated by its token's position.

    q [n, q_heads, dim] and / or k [n, k_heads, dim], bf16 or fp32 (or [B, S, heads, dim], the tokens evenly
    spaced), pos [n] (or [B, S]) int32.  rope_dim dims from rope_at on are rotated (None: all of them; 0: none),
    as pairs (2i, 2i + 1) or with halves=True (i, i + rope_dim / 2), by pos * base^(-2i / rope_dim) or pos * freq[i]
    (fp32 [rope_dim / 2]).  q_out, k_out: buffers of the object by default, the input itself for in place.
    Calling the object returns {"q", "k"} as far as they are given."""

    def __init__(self, q=None, k=None, pos=None, q_weight=None, k_weight=None, norm: bool = False, eps: float = 1e-6,
                 rope_dim: int | None = None, rope_at: int = 0, halves: bool = False, base: float = 10000.0, freq=None,
                 q_out=None, k_out=None):
        import torch
        x = k if q is None else q
        if x is None or x.dim() < 3:
            _bad("give q or k, [n, heads, dim] or [B, S, heads, dim]")
        lead, dim, dt = tuple(int(v) for v in x.shape[:-2]), int(x.shape[-1]), _dtype_code(x)
        rope_dim = dim - rope_at if rope_dim is None else rope_dim
        n = 1
        for v in lead:
            n *= v
        _int32(n=n, dim=dim, rope_dim=rope_dim, rope_at=rope_at)
        st = CRope(n=n, dim=dim, dtype=dt, norm=1 if norm else 0, eps=eps, rope_dim=rope_dim, rope_at=rope_at,
                   halves=1 if halves else 0, base=base, freq=_ptr(freq), pos=_ptr(pos))
        if pos is None and rope_dim > 0:
            _bad("pos is needed for the rotation")
        _flat("pos", pos, torch.int32, [lead, (n,)])
        _flat("freq", freq, torch.float32, (rope_dim // 2,))
        self._out = {}
        for name, t, w, out in (("q", q, q_weight, q_out), ("k", k, k_weight, k_out)):
            if t is None:
                if w is not None or out is not None:
                    _bad(f"{name}_weight or {name}_out given without {name}")
                continue
            heads = int(t.shape[-2]) if t.dim() >= 2 else 0
            _int32(heads=heads)
            stride = _tokens(name, t, lead, heads, dim, x.dtype)
            _head_weight(name + "_weight", w, x, dim, norm)
            if out is None:
                out = torch.empty(t.shape, dtype=t.dtype, device=t.device)
            setattr(st, name + "_heads", heads)
            setattr(st, name, _ptr(t))
            setattr(st, name + "_stride", stride)
            setattr(st, name + "_weight", _ptr(w))
            setattr(st, name + "_out", _ptr(out))
            setattr(st, name + "_out_stride", _tokens(name + "_out", out, lead, heads, dim, x.dtype))
            self._out[name] = out
        self._bind(lib().csa_qk_rope, st, (q, k, pos, q_weight, k_weight, freq, *self._out.values()))

    def __call__(self, stream=None) -> dict:
        self._launch(stream)
        return self._out


class KvAppend(_Operator):
    """csa_kv_append: the keys (normed and rotated as QkRope does it) and values of new tokens into the pools of a
    cache, their queries normed and rotated beside them.

    k, v [B, S, kv_heads, dim] bf16 or fp32 (v None: keys only); k_pool, v_pool [rows, kv_heads, dim] in the same
    type, or E4M3 codes (uint8 or float8_e4m3fn) with k_scale, v_scale fp32 [rows, kv_heads].  The tokens' rows: through
    ctx_len [B] int32 (the new tokens included) with table [B, blocks] int32 and block, or with off [B] int64; or by
    slot int64 [B * S] (negative: padding).  count [B] int32: the real tokens of each request, the first of its S
    (None: all S).  pos int32 [B * S]: positions, by default the tokens' rows in their request.  q [B, S, q_heads, dim]
    with q_out (a buffer of the object by default; padding tokens' rows are left as they are), weights, norm and rotation
    as in QkRope.  status: an int32 on the device that records bad rows.  Calling the object returns the pools and
    what else it writes: {"k", "v", "k_scale", "v_scale", "q"} as far as they are given."""

    def __init__(self, k, v, k_pool, v_pool, k_scale=None, v_scale=None, ctx_len=None, count=None, table=None,
                 block: int = 0, off=None, slot=None, pos=None, q=None, q_out=None, q_weight=None, k_weight=None,
                 norm: bool = False, eps: float = 1e-6, rope_dim: int | None = None, rope_at: int = 0,
                 halves: bool = False, base: float = 10000.0, freq=None, status=None):
        import torch
        if k.dim() != 4 or k_pool.dim() != 3:
            _bad("k, v must be [B, S, kv_heads, dim] and the pools [rows, kv_heads, dim]")
        b, s, heads, dim = (int(x) for x in k.shape)
        rows, dt = int(k_pool.shape[0]), _dtype_code(k)
        rope_dim = dim - rope_at if rope_dim is None else rope_dim
        _int32(B=b, S=s, kv_heads=heads, dim=dim, rope_dim=rope_dim, rope_at=rope_at, block=block)
        fp8 = str(k_pool.dtype) in _E4M3_DTYPES
        st = CAppend(B=b, S=s, kv_heads=heads, dim=dim, dtype=dt, kv_dtype=CSA_DTYPE_FP8_E4M3 if fp8 else dt,
                     norm=1 if norm else 0, eps=eps, rope_dim=rope_dim, rope_at=rope_at, halves=1 if halves else 0,
                     base=base, freq=_ptr(freq), pos=_ptr(pos), ctx_len=_ptr(ctx_len), count=_ptr(count),
                     slot=_ptr(slot), off=_ptr(off), table=_ptr(table), block=block, rows=rows, status=_ptr(status))
        if (v is None) != (v_pool is None):
            _bad("v and v_pool go together")
        self._out = {}
        for name, t, pool, scale in (("k", k, k_pool, k_scale), ("v", v, v_pool, v_scale)):
            if t is None:
                if scale is not None:
                    _bad(f"{name}_scale given without {name}")
                continue
            setattr(st, name, _ptr(t))
            setattr(st, name + "_stride", _tokens(name, t, (b, s), heads, dim, k.dtype))
            if tuple(pool.shape) != (rows, heads, dim) or (str(pool.dtype) not in _E4M3_DTYPES if fp8
                                                           else pool.dtype != k.dtype):
                _bad(f"{name}_pool must be {k.dtype} or E4M3 codes, both alike, of shape ({rows}, {heads}, {dim})")
            if (dim > 1 and pool.stride(2) != 1) or (heads > 1 and pool.stride(1) != dim):
                _bad(f"{name}_pool: the heads of a row must be contiguous")
            setattr(st, name + "_pool", _ptr(pool))
            setattr(st, name + "_pool_stride", int(pool.stride(0)) if rows > 1 else -(-heads * dim // 16) * 16)
            if fp8:
                if scale is None:
                    _bad(f"{name}_scale is needed with E4M3 codes")
                _rows2d(name + "_scale", scale, rows, heads, torch.float32)
                step = int(scale.stride(0)) if rows > 1 else heads
                if name == "v" and st.scale_stride != step:
                    _bad("k_scale and v_scale must have the same row stride")
                st.scale_stride = step
                setattr(st, name + "_scale", _ptr(scale))
                self._out[name + "_scale"] = scale
            elif scale is not None:
                _bad("scales given with a pool that is not of E4M3 codes")
            self._out[name] = pool.view(torch.float8_e4m3fn) if fp8 else pool
            w = k_weight if name == "k" else None
            _head_weight("k_weight", w, k, dim, norm)
        st.k_weight = _ptr(k_weight)
        if q is not None:
            if q.dim() != 4:
                _bad("q must be [B, S, q_heads, dim]")
            q_heads = int(q.shape[2])
            _int32(q_heads=q_heads)
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            _head_weight("q_weight", q_weight, k, dim, norm)
            st.q_heads, st.q, st.q_weight, st.q_out = q_heads, _ptr(q), _ptr(q_weight), _ptr(q_out)
            st.q_stride = _tokens("q", q, (b, s), q_heads, dim, k.dtype)
            st.q_out_stride = _tokens("q_out", q_out, (b, s), q_heads, dim, k.dtype)
            self._out["q"] = q_out
        elif q_out is not None or q_weight is not None:
            _bad("q_out or q_weight given without q")
        if (table is not None) + (off is not None) + (slot is not None) != 1:
            _bad("give one of table (with block), off and slot")
        if slot is None and ctx_len is None:
            _bad("ctx_len is needed without slot")
        if rope_dim > 0 and pos is None and ctx_len is None:
            _bad("pos or ctx_len is needed for the rotation")
        if table is not None:
            if table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != b or not table.is_contiguous():
                _bad(f"table must be contiguous int32 of shape ({b}, blocks)")
            _int32(table_stride=table.shape[1])
            st.table_stride = int(table.shape[1])
        _flat("ctx_len", ctx_len, torch.int32, (b,))
        _flat("count", count, torch.int32, (b,))
        _flat("off", off, torch.int64, (b,))
        _flat("slot", slot, torch.int64, [(b * s,), (b, s)])
        _flat("pos", pos, torch.int32, [(b * s,), (b, s)])
        _flat("freq", freq, torch.float32, (rope_dim // 2,))
        _status_word(status)
        self._bind(lib().csa_kv_append, st, (k, v, k_pool, v_pool, k_scale, v_scale, ctx_len, count, table, off, slot, pos,
                                             q, q_out, q_weight, k_weight, freq, status))

    def __call__(self, stream=None) -> dict:
        self._launch(stream)
        return self._out
