"""Python binding of the lossless BF16 weight compression library (libuw.so).

Every function here only marshals arguments into the C ABI declared in
include/uw.h and has the same name without the ``uw_`` prefix.  All compute
runs in the library's CUDA kernels (and its host compressor); PyTorch
tensors merely provide device memory and the current CUDA stream.  There is
no fallback: if libuw.so is missing, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libuw.so")

UW_OK = 0
UW_ERR_INVALID_ARG = 1
UW_ERR_SHAPE = 2
UW_ERR_BUFFER_TOO_SMALL = 3
STATUS_NAMES = {0: "UW_OK", 1: "UW_ERR_INVALID_ARG", 2: "UW_ERR_SHAPE", 3: "UW_ERR_BUFFER_TOO_SMALL",
                4: "UW_ERR_CORRUPT", 5: "UW_ERR_CUDA", 6: "UW_ERR_TIMEOUT", 7: "UW_ERR_UNSUPPORTED",
                8: "UW_ERR_INTERNAL"}
STRATEGY_DEFAULT, STRATEGY_DECOMPRESS_GEMM, STRATEGY_FUSED, STRATEGY_PALETTE4, STRATEGY_EXPONENT = -1, 0, 1, 2, 3


class UwError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (%d)" % (what, STATUS_NAMES.get(status, "?"), status))
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("blob_bytes", ctypes.c_uint64), ("code_bits", ctypes.c_uint64),
        ("n_groups", ctypes.c_uint64), ("n_escaped", ctypes.c_uint64), ("n_tiles", ctypes.c_uint64),
        ("n_palette", ctypes.c_int32), ("lmax", ctypes.c_int32),
        ("palette", ctypes.c_uint8 * 16), ("code_len", ctypes.c_uint8 * 16),
        ("off_sm", ctypes.c_uint64), ("off_glen", ctypes.c_uint64), ("off_tcode", ctypes.c_uint64),
        ("off_tesc", ctypes.c_uint64), ("off_code", ctypes.c_uint64), ("off_esc", ctypes.c_uint64),
        ("max_tile_bytes", ctypes.c_uint64),
    ]


class Plan(ctypes.Structure):
    _fields_ = [("strategy", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("us", ctypes.c_float)]

    def __repr__(self):
        return "Plan(strategy=%d, variant=%d, batch=%d, us=%.2f)" % (
            self.strategy, self.variant, self.batch, self.us)


class MlpMatrix(ctypes.Structure):
    """One weight matrix of an MLP chain (uw_mlp_matrix)."""
    _fields_ = [("desc", ctypes.POINTER(Desc)), ("blob_dev", ctypes.c_void_p), ("form_dev", ctypes.c_void_p),
                ("plan", Plan)]


class Schedule(ctypes.Structure):
    """Preprocess slots and SM split of an MLP chain (uw_schedule)."""
    _fields_ = [("slots", ctypes.c_int32), ("dec_ctas", ctypes.c_int32)]

    def __repr__(self):
        return "Schedule(slots=%d, dec_ctas=%d)" % (self.slots, self.dec_ctas)


class Kv4CacheDesc(ctypes.Structure):
    """The 4-bit paged cache of keys and values of one layer (uw_kv4_cache)."""
    _fields_ = [("pages_dev", ctypes.c_void_p), ("table_dev", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class Kv4Rows(ctypes.Structure):
    """BF16 rows [tokens, heads, head_dim] with their strides in elements (uw_kv4_rows)."""
    _fields_ = [("dev", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Block(ctypes.Structure):
    """The norm after a block, its gate and scales (uw_block)."""
    _fields_ = [("post_weight_dev", ctypes.c_void_p), ("gate_dev", ctypes.c_void_p), ("gate_stride", ctypes.c_int64),
                ("weight_offset", ctypes.c_float), ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("eps", ctypes.c_float)]


class Rope(ctypes.Structure):
    """Positions on several axes and the tables they turn by (uw_rope)."""
    _fields_ = [("pos_dev", ctypes.c_void_p), ("axis_stride", ctypes.c_int64), ("n_axes", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("pair_axis", ctypes.c_char_p), ("cos_dev", ctypes.c_void_p),
                ("sin_dev", ctypes.c_void_p), ("rope_len", ctypes.c_int64), ("interleaved", ctypes.c_int32)]


_lib = None

# (name, restype, argtypes) of every symbol in include/uw.h
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_F32, _CACHE, _ROWS = ctypes.c_float, ctypes.POINTER(Kv4CacheDesc), ctypes.POINTER(Kv4Rows)
_BLOCK, _ROPE = ctypes.POINTER(Block), ctypes.POINTER(Rope)
SIGNATURES = [
    ("uw_compress", ctypes.c_int, [_P, _I64, _I64, _P, ctypes.POINTER(_SZ)]),
    ("uw_blob_info", ctypes.c_int, [_P, _SZ, ctypes.POINTER(Desc)]),
    ("uw_workspace_size", ctypes.c_int, [ctypes.POINTER(Desc), _I64, ctypes.POINTER(Plan), ctypes.POINTER(_SZ)]),
    ("uw_workspace_size_bf16", ctypes.c_int, [_I64, _I64, _I64, _I32, ctypes.POINTER(_SZ)]),
    ("uw_workspace_init", ctypes.c_int, [_P, _SZ, _P]),
    ("uw_decompress", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _P, _SZ, _P]),
    ("uw_matmul", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _I64, _P, ctypes.POINTER(Plan), _P, _SZ, _P]),
    ("uw_matmul_bf16", ctypes.c_int, [_P, _I64, _I64, _P, _I64, _P, _I32, _P, _SZ, _P]),
    ("uw_autotune", ctypes.c_int, [ctypes.POINTER(Desc), _P, ctypes.POINTER(_I64), _I32, ctypes.POINTER(Plan),
                                   _P, _SZ, _P]),
    ("uw_autotune_workspace_size", ctypes.c_int, [ctypes.POINTER(Desc), ctypes.POINTER(_I64), _I32,
                                                  ctypes.POINTER(_SZ)]),
    ("uw_matmul_noalloc", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _I64, _P, _P]),
    ("uw_swiglu", ctypes.c_int, [_P, _P, _P, _I64, _P]),
    ("uw_palette4_bytes", ctypes.c_int, [ctypes.POINTER(Desc), ctypes.POINTER(_SZ)]),
    ("uw_transcode_palette4", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _P, _SZ, _P]),
    ("uw_matmul_palette4", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _P, _I64, _P, _I32, _P, _SZ, _P]),
    ("uw_exponent_bytes", ctypes.c_int, [ctypes.POINTER(Desc), ctypes.POINTER(_SZ)]),
    ("uw_decode_exponents", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _P, _SZ, _P]),
    ("uw_matmul_exponents", ctypes.c_int, [ctypes.POINTER(Desc), _P, _P, _P, _I64, _P, _I32, _P, _SZ, _P]),
    ("uw_mlp_workspace_size", ctypes.c_int, [ctypes.POINTER(MlpMatrix), _I32, _I64, ctypes.POINTER(Schedule),
                                             ctypes.POINTER(_SZ)]),
    ("uw_mlp_forward", ctypes.c_int, [ctypes.POINTER(MlpMatrix), _I32, _P, _I64, _P, ctypes.POINTER(Schedule),
                                      _P, _SZ, _P, _P]),
    ("uw_mlp_autotune", ctypes.c_int, [ctypes.POINTER(MlpMatrix), _I32, _P, _I64, _P, _I32, ctypes.POINTER(Plan),
                                       ctypes.POINTER(Schedule), _P, _SZ, _P, _P]),
    ("uw_mlp_autotune_workspace_size", ctypes.c_int, [ctypes.POINTER(MlpMatrix), _I32, _I64,
                                                      ctypes.POINTER(_SZ)]),
    ("uw_rmsnorm", ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _F32, _P, _I64, _P]),
    ("uw_rmsnorm_e4m3", ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _F32, _P, _I64, _P, _P]),
    ("uw_block_norm", ctypes.c_int, [_BLOCK, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _P]),
    ("uw_block_norm_e4m3", ctypes.c_int, [_BLOCK, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _P, _P]),
    ("uw_rope_axes", ctypes.c_int, [_ROPE, _I64, _ROWS, _I32, _ROWS, _ROWS, _I32, _ROWS, _I32, _P, _SZ, _P]),
    ("uw_kv4_append_axes", ctypes.c_int, [_CACHE, _P, _P, _I64, _ROPE, _ROWS, _I32, _ROWS, _ROWS, _ROWS, _ROWS, _P,
                                          _SZ, _P]),
    ("uw_kv4_page_bytes", ctypes.c_int, [_I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    ("uw_kv4_workspace_size", ctypes.c_int, [_CACHE, _I32, ctypes.POINTER(_SZ)]),
    ("uw_kv4_append", ctypes.c_int, [_CACHE, _P, _P, _I64, _ROWS, _I32, _ROWS, _ROWS, _ROWS, _P, _P, _I64, _I32,
                                     _I32, _P, _SZ, _P]),
    ("uw_kv4_read", ctypes.c_int, [_CACHE, _P, _P, _I64, _ROWS, _ROWS, _P, _SZ, _P]),
    ("uw_kv4_attention", ctypes.c_int, [_CACHE, _P, _P, _I64, _ROWS, _I32, _ROWS, _P, _I64, _I64, _F32, _I32, _I32,
                                        _P, _SZ, _P]),
    ("uw_attention_workspace_size", ctypes.c_int, [_I32, ctypes.POINTER(_SZ)]),
    ("uw_attention", ctypes.c_int, [_P, _P, _I32, _I64, _I64, _ROWS, _I32, _ROWS, _ROWS, _I32, _I32, _ROWS, _P, _F32,
                                    _I32, _I32, _P, _SZ, _P]),
    ("uw_selftest_attention_wait", ctypes.c_int, [_P, _SZ, ctypes.c_uint32, _P]),
    ("uw_check_status", ctypes.c_int, [_P, _P]),
    ("uw_selftest_bounded_wait", ctypes.c_int, [_P, _SZ, ctypes.c_uint32, _P]),
    ("uw_variant_name", ctypes.c_char_p, [_I32, _I32]),
    ("uw_variant_count", ctypes.c_int32, [_I32]),
    ("uw_status_string", ctypes.c_char_p, [ctypes.c_int]),
]


def build(force: bool = False) -> str:
    from .build import build as _build
    return _build(force=force)


def load():
    """Load libuw.so (built beforehand by build()).  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libuw.so is not built (run lossless_bf16_weight_gb300.build())")
        lib = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int, what: str):
    if status != UW_OK:
        raise UwError(status, what)


def _ptr(t) -> int:
    """Device or host address of a torch tensor or numpy array."""
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    """The address of the CUDA stream to pass; None: the current one of the current device."""
    if stream is None:
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _current_stream() -> int:
    """torch.cuda.current_stream().cuda_stream without building the Stream
    object (2.9 us a call against 0.2 us, of 3 us for a launch)."""
    global _current_stream
    import torch
    raw, device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is not None and device is not None:
        torch.cuda.current_device()  # (initialises CUDA)
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream()


def _plan_ptr(plan):
    return None if plan is None else ctypes.byref(plan)


def _nbytes(t) -> int:
    return t.nbytes


def _contiguous(t) -> bool:
    return t.flags.c_contiguous if isinstance(t, np.ndarray) else t.is_contiguous()


def _short(*bufs) -> str | None:
    """The C ABI sees plain pointers, so a buffer smaller than what a call
    reads or writes would make a kernel run past its end.  Each argument is
    (buffer, bytes the call touches, name); returns why the first one that
    is not contiguous or too small is refused, or None."""
    for t, need, name in bufs:
        if not _contiguous(t):
            return "%s is not contiguous" % name
        if _nbytes(t) < need:
            return "%s holds %d bytes, the call needs %d" % (name, _nbytes(t), need)
    return None


def _refuse(why: str | None, what: str):
    if why is not None:
        raise UwError(UW_ERR_BUFFER_TOO_SMALL, "%s (%s)" % (what, why))


def _batch(x) -> int:
    return x.shape[0] if x.dim() == 2 else 1


def _form_bytes(desc) -> int:
    """Weights of a blob's stored width (rows extended to whole 64-column
    groups): the exponent form's bytes, twice the palette-4 form's."""
    return desc.rows * (-(-desc.cols // 64) * 64)


def _mm_bufs(desc, blob_dev, x, y):
    b = _batch(x)
    return [(blob_dev, desc.blob_bytes, "blob_dev"), (x, 2 * b * desc.cols, "x"), (y, 2 * b * desc.rows, "y")]


# ---------------------------------------------------------------- host side
def compress(w: np.ndarray) -> np.ndarray:
    """uw_compress: BF16 weight matrix (uint16 bits, [rows, cols]) -> blob bytes (uint8)."""
    w = np.ascontiguousarray(w)
    if w.dtype != np.uint16 or w.ndim != 2:
        raise TypeError("w must be a 2-D uint16 array of BF16 bit patterns")
    L = load()
    size = ctypes.c_size_t(0)
    s = L.uw_compress(w.ctypes.data, w.shape[0], w.shape[1], None, ctypes.byref(size))
    if s != 3:  # UW_ERR_BUFFER_TOO_SMALL answers the size query
        _check(s, "uw_compress")
    blob = np.empty(size.value, np.uint8)
    _check(L.uw_compress(w.ctypes.data, w.shape[0], w.shape[1], blob.ctypes.data, ctypes.byref(size)),
           "uw_compress")
    return blob


def blob_info(blob) -> Desc:
    """uw_blob_info on a host copy of the blob (numpy uint8 or bytes)."""
    b = np.frombuffer(blob, np.uint8) if isinstance(blob, (bytes, bytearray)) else np.ascontiguousarray(blob)
    d = Desc()
    _check(load().uw_blob_info(b.ctypes.data, b.size, ctypes.byref(d)), "uw_blob_info")
    return d


def blob_info_status(blob) -> int:
    b = np.frombuffer(blob, np.uint8) if isinstance(blob, (bytes, bytearray)) else np.ascontiguousarray(blob)
    d = Desc()
    return int(load().uw_blob_info(b.ctypes.data, b.size, ctypes.byref(d)))


def workspace_size(desc: Desc, batch: int = 0, plan: Plan | None = None) -> int:
    n = ctypes.c_size_t(0)
    _check(load().uw_workspace_size(ctypes.byref(desc), batch, _plan_ptr(plan), ctypes.byref(n)),
           "uw_workspace_size")
    return n.value


def workspace_size_bf16(rows: int, cols: int, batch: int = 1, variant: int = -1) -> int:
    """Workspace bytes of matmul_bf16 for this shape, batch and variant."""
    n = ctypes.c_size_t(0)
    _check(load().uw_workspace_size_bf16(rows, cols, batch, variant, ctypes.byref(n)), "uw_workspace_size_bf16")
    return n.value


def autotune_workspace_size(desc: Desc, batches) -> int:
    arr = (ctypes.c_int64 * len(batches))(*batches)
    n = ctypes.c_size_t(0)
    _check(load().uw_autotune_workspace_size(ctypes.byref(desc), arr, len(batches), ctypes.byref(n)),
           "uw_autotune_workspace_size")
    return n.value


def variant_count(strategy: int) -> int:
    return int(load().uw_variant_count(strategy))


def variant_name(strategy: int, variant: int) -> str | None:
    r = load().uw_variant_name(strategy, variant)
    return None if r is None else r.decode()


def status_string(status: int) -> str:
    return load().uw_status_string(status).decode()


# ---------------------------------------------------------------- device side
def workspace_init(ws, stream=None):
    _check(load().uw_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "uw_workspace_init")


def decompress(desc: Desc, blob_dev, w_out, ws, stream=None):
    _refuse(_short((blob_dev, desc.blob_bytes, "blob_dev"), (w_out, 2 * desc.rows * desc.cols, "w_out")),
            "uw_decompress")
    _check(load().uw_decompress(ctypes.byref(desc), _ptr(blob_dev), _ptr(w_out), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "uw_decompress")


def matmul(desc: Desc, blob_dev, x, y, ws, plan: Plan | None = None, stream=None):
    """y[batch, rows] = x[batch, cols] W^T with W compressed in blob_dev."""
    _refuse(_short(*_mm_bufs(desc, blob_dev, x, y)), "uw_matmul")
    batch = _batch(x)
    _check(load().uw_matmul(ctypes.byref(desc), _ptr(blob_dev), _ptr(x), batch, _ptr(y), _plan_ptr(plan),
                            _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "uw_matmul")


def matmul_status(desc: Desc, blob_dev, x, y, ws, plan: Plan | None = None, stream=None) -> int:
    if _short(*_mm_bufs(desc, blob_dev, x, y)):
        return UW_ERR_BUFFER_TOO_SMALL
    batch = _batch(x)
    return int(load().uw_matmul(ctypes.byref(desc), _ptr(blob_dev), _ptr(x), batch, _ptr(y), _plan_ptr(plan),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def matmul_noalloc(desc: Desc, blob_dev, x, y, stream=None) -> int:
    """uw_matmul_noalloc: fused matmul with library-held scratch; returns the status."""
    if _short(*_mm_bufs(desc, blob_dev, x, y)):
        return UW_ERR_BUFFER_TOO_SMALL
    batch = _batch(x)
    return int(load().uw_matmul_noalloc(ctypes.byref(desc), _ptr(blob_dev), _ptr(x), batch, _ptr(y),
                                        _stream(stream)))


def matmul_bf16(w, x, y, ws, variant: int = -1, stream=None):
    rows, cols = w.shape
    batch = _batch(x)
    _refuse(_short((w, 2 * rows * cols, "w"), (x, 2 * batch * cols, "x"), (y, 2 * batch * rows, "y")),
            "uw_matmul_bf16")
    _check(load().uw_matmul_bf16(_ptr(w), rows, cols, _ptr(x), batch, _ptr(y), variant, _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "uw_matmul_bf16")


def autotune(desc: Desc, blob_dev, batches, ws, stream=None) -> list[Plan]:
    arr = (ctypes.c_int64 * len(batches))(*batches)
    plans = (Plan * len(batches))()
    _check(load().uw_autotune(ctypes.byref(desc), _ptr(blob_dev), arr, len(batches), plans, _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "uw_autotune")
    return list(plans)


def palette4_bytes(desc: Desc) -> int:
    n = _SZ(0)
    _check(load().uw_palette4_bytes(ctypes.byref(desc), ctypes.byref(n)), "uw_palette4_bytes")
    return int(n.value)


def transcode_palette4(desc: Desc, blob_dev, p4_out, ws, stream=None):
    """uw_transcode_palette4: the 4-bit palette index of every weight into p4_out."""
    _refuse(_short((blob_dev, desc.blob_bytes, "blob_dev"), (p4_out, _form_bytes(desc) // 2, "p4_out")),
            "uw_transcode_palette4")
    _check(load().uw_transcode_palette4(ctypes.byref(desc), _ptr(blob_dev), _ptr(p4_out), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)), "uw_transcode_palette4")


def matmul_palette4_status(desc: Desc, blob_dev, p4, x, y, ws, variant: int = -1, stream=None) -> int:
    if _short(*_mm_bufs(desc, blob_dev, x, y), (p4, _form_bytes(desc) // 2, "p4")):
        return UW_ERR_BUFFER_TOO_SMALL
    batch = _batch(x)
    return int(load().uw_matmul_palette4(ctypes.byref(desc), _ptr(blob_dev), _ptr(p4), _ptr(x), batch, _ptr(y),
                                         variant, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def matmul_palette4(desc: Desc, blob_dev, p4, x, y, ws, variant: int = -1, stream=None):
    """y[batch, rows] = x W^T from the palette-4 form p4 (plus the blob)."""
    _check(matmul_palette4_status(desc, blob_dev, p4, x, y, ws, variant, stream), "uw_matmul_palette4")


def exponent_bytes(desc: Desc) -> int:
    n = _SZ(0)
    _check(load().uw_exponent_bytes(ctypes.byref(desc), ctypes.byref(n)), "uw_exponent_bytes")
    return int(n.value)


def decode_exponents(desc: Desc, blob_dev, e_out, ws, stream=None):
    """uw_decode_exponents: the exponent byte of every weight into e_out."""
    _refuse(_short((blob_dev, desc.blob_bytes, "blob_dev"), (e_out, _form_bytes(desc), "e_out")),
            "uw_decode_exponents")
    _check(load().uw_decode_exponents(ctypes.byref(desc), _ptr(blob_dev), _ptr(e_out), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "uw_decode_exponents")


def matmul_exponents_status(desc: Desc, blob_dev, e, x, y, ws, variant: int = -1, stream=None) -> int:
    if _short(*_mm_bufs(desc, blob_dev, x, y), (e, _form_bytes(desc), "e")):
        return UW_ERR_BUFFER_TOO_SMALL
    batch = _batch(x)
    return int(load().uw_matmul_exponents(ctypes.byref(desc), _ptr(blob_dev), _ptr(e), _ptr(x), batch, _ptr(y),
                                          variant, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def matmul_exponents(desc: Desc, blob_dev, e, x, y, ws, variant: int = -1, stream=None):
    """y[batch, rows] = x W^T from the exponent form e (plus the blob)."""
    _check(matmul_exponents_status(desc, blob_dev, e, x, y, ws, variant, stream), "uw_matmul_exponents")


def swiglu(g, u, h, stream=None):
    n = g.numel()
    _refuse(_short((g, 2 * n, "g"), (u, 2 * n, "u"), (h, 2 * n, "h")), "uw_swiglu")
    _check(load().uw_swiglu(_ptr(g), _ptr(u), _ptr(h), g.numel(), _stream(stream)), "uw_swiglu")


# ---------------------------------------------------------------- MLP chain
def mlp_matrices(entries) -> ctypes.Array:
    """uw_mlp_matrix array from (desc, blob_dev, form_dev or None, plan or None)
    entries, three per layer (gate, up, down).  Keep `entries` alive while
    the array is used."""
    arr = (MlpMatrix * len(entries))()
    for i, (d, blob, form, plan) in enumerate(entries):
        _refuse(_short((blob, d.blob_bytes, "blob_dev")), "uw_mlp_matrix %d" % i)
        arr[i].desc = ctypes.pointer(d)
        arr[i].blob_dev = _ptr(blob)
        arr[i].form_dev = None if form is None else _ptr(form)
        arr[i].plan = plan if plan is not None else Plan(STRATEGY_DEFAULT, -1, 0, 0.0)
    return arr


def _side(stream):
    if stream is None:
        return None
    return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)


def _sched_ptr(sched):
    return None if sched is None else ctypes.byref(sched)


def mlp_workspace_size(mats, batch: int, sched: Schedule | None = None) -> int:
    n = _SZ(0)
    _check(load().uw_mlp_workspace_size(mats, len(mats) // 3, batch, _sched_ptr(sched), ctypes.byref(n)),
           "uw_mlp_workspace_size")
    return int(n.value)


def _chain_short(mats, x, y) -> str | None:
    if len(mats) < 3:
        return None  # the library refuses an empty chain itself
    dim_in, dim_out = mats[0].desc.contents.cols, mats[len(mats) // 3 * 3 - 1].desc.contents.rows
    return _short((x, 2 * x.shape[0] * dim_in, "x"), (y, 2 * x.shape[0] * dim_out, "y"))


def mlp_forward_status(mats, x, y, ws, sched: Schedule | None = None, stream=None, side_stream=None) -> int:
    """uw_mlp_forward: y = the chain of len(mats)//3 SwiGLU MLP layers applied to x."""
    if _chain_short(mats, x, y):
        return UW_ERR_BUFFER_TOO_SMALL
    return int(load().uw_mlp_forward(mats, len(mats) // 3, _ptr(x), x.shape[0], _ptr(y), _sched_ptr(sched),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream),
                                     _side(side_stream)))


def mlp_forward(mats, x, y, ws, sched: Schedule | None = None, stream=None, side_stream=None):
    _check(mlp_forward_status(mats, x, y, ws, sched, stream, side_stream), "uw_mlp_forward")


def mlp_autotune_workspace_size(mats, batch: int) -> int:
    n = _SZ(0)
    _check(load().uw_mlp_autotune_workspace_size(mats, len(mats) // 3, batch, ctypes.byref(n)),
           "uw_mlp_autotune_workspace_size")
    return int(n.value)


def mlp_autotune(mats, x, y, ws, passes: int = 2, stream=None, side_stream=None):
    """uw_mlp_autotune: (6 plans: gate, up, down without a form, then with
    one; Schedule) by coordinate descent."""
    _refuse(_chain_short(mats, x, y), "uw_mlp_autotune")
    plans = (Plan * 6)()
    sched = Schedule()
    _check(load().uw_mlp_autotune(mats, len(mats) // 3, _ptr(x), x.shape[0], _ptr(y), passes, plans,
                                  ctypes.byref(sched), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream),
                                  _side(side_stream)), "uw_mlp_autotune")
    return list(plans), sched


# ---------------------------------------------------------------- around the matmuls of a decoder layer
def _types():
    """The tensor types that hold BF16 values, e4m3 values, int32 and fp32 (the first two also as plain bits)."""
    global _types
    import torch
    found = (frozenset((torch.bfloat16, torch.int16, torch.uint16)),
             frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8)), torch.int32, torch.float32)
    _types = lambda: found  # noqa: E731
    return found


def _row_stride(t, shape, kinds, name: str, what: str) -> int:
    """Row stride in elements of a [n, d] (or, for one row, [d]) tensor of one
    of the types `kinds` whose rows are contiguous; `shape` is one or the other."""
    if t.shape == shape and t.dtype in kinds and t.is_contiguous():
        return shape[-1]
    d, n = shape[-1], shape[0] if len(shape) == 2 else 1
    if t.dtype not in kinds or t.shape[-1] != d or t.numel() != n * d or t.dim() > 2:
        raise UwError(UW_ERR_SHAPE, "%s (%s is %s of %s)" % (what, name, tuple(t.shape), t.dtype))
    if t.is_contiguous():
        return d
    if d > 1 and t.stride(-1) != 1:
        raise UwError(UW_ERR_INVALID_ARG, "%s (%s has rows that are not contiguous)" % (what, name))
    return t.stride(0) if t.dim() == 2 and n > 1 else d


def rmsnorm(x, weight, y, eps: float = 1e-5, residual=None, residual_out=None, scale=None, stream=None):
    """uw_rmsnorm: h = bf16(x + residual) into residual_out (if given), y = h / rms(h) * weight in BF16.
    With `scale` (fp32, one for each row): uw_rmsnorm_e4m3, y holds e4m3 bytes (torch.float8_e4m3fn or uint8).
    Tensors are [n, d], whose rows may be strided, or [d]; more dimensions are for the caller to flatten."""
    what = "uw_rmsnorm" if scale is None else "uw_rmsnorm_e4m3"
    shape = x.shape
    if not 1 <= len(shape) <= 2:
        raise UwError(UW_ERR_SHAPE, "%s (x is %s, neither [n, d] nor [d])" % (what, tuple(shape)))
    d, n = shape[-1], shape[0] if len(shape) == 2 else 1
    bf16, e4m3, _, fp32 = _types()
    xs = _row_stride(x, shape, bf16, "x", what)
    ys = _row_stride(y, shape, bf16 if scale is None else e4m3, "y", what)
    rp = hp = None
    rs = hs = 0
    if residual is not None:
        rp, rs = residual.data_ptr(), _row_stride(residual, shape, bf16, "residual", what)
    if residual_out is not None:
        hp, hs = residual_out.data_ptr(), _row_stride(residual_out, shape, bf16, "residual_out", what)
    if weight.dtype not in bf16 or (scale is not None and scale.dtype is not fp32):
        raise UwError(UW_ERR_SHAPE, "%s (weight is not BF16, or scale not fp32)" % what)
    _refuse(_short((weight, 2 * d, "weight")), what)
    if scale is None:
        _check(load().uw_rmsnorm(x.data_ptr(), xs, rp, rs, hp, hs, weight.data_ptr(), n, d, eps, y.data_ptr(), ys,
                                 _stream(stream)), what)
    else:
        _refuse(_short((scale, 4 * n, "scale")), what)
        _check(load().uw_rmsnorm_e4m3(x.data_ptr(), xs, rp, rs, hp, hs, weight.data_ptr(), n, d, eps, y.data_ptr(),
                                      ys, scale.data_ptr(), _stream(stream)), what)


def _here(what: str, *tensors):
    """Refuses tensors that are not on the current CUDA device, whose stream the call would be made on."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            device = -1
    if device < 0 or device != _current_device():
        raise UwError(UW_ERR_INVALID_ARG, "%s (tensors are not all on the current CUDA device)" % what)


def _current_device() -> int:
    """torch.cuda.current_device() without the check that CUDA is initialised (it is, once there are tensors)."""
    global _current_device
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def block_norm(x, residual, weight, residual_out, y, eps: float = 1e-5, post_weight=None, gate=None,
               residual_scale: float = 1.0, block_scale: float = 1.0, weight_offset: float = 0.0, scale=None,
               stream=None):
    """uw_block_norm: z = x, with post_weight its norm times post_weight + weight_offset; h = bf16(residual_scale *
    residual + block_scale * gate * z) into residual_out (or None); y = the norm of h times weight + weight_offset in BF16
    (weight and y None: only h).  With `scale` (fp32, one for each row): uw_block_norm_e4m3, y holds e4m3 bytes.
    Tensors are [n, d], whose rows may be strided, or [d]; gate is [d] for all rows, or like x."""
    what = "uw_block_norm" if scale is None else "uw_block_norm_e4m3"
    shape = x.shape
    if not 1 <= len(shape) <= 2:
        raise UwError(UW_ERR_SHAPE, "%s (x is %s, neither [n, d] nor [d])" % (what, tuple(shape)))
    d, n = shape[-1], shape[0] if len(shape) == 2 else 1
    bf16, e4m3, _, fp32 = _types()
    xs, rs = _row_stride(x, shape, bf16, "x", what), _row_stride(residual, shape, bf16, "residual", what)
    hp = yp = wp = gp = pp = None
    hs = ys = gs = 0
    if residual_out is not None:
        hp, hs = residual_out.data_ptr(), _row_stride(residual_out, shape, bf16, "residual_out", what)
    if (weight is None) != (y is None):
        raise UwError(UW_ERR_INVALID_ARG, "%s (weight and y: both or neither)" % what)
    if y is not None:
        yp, ys = y.data_ptr(), _row_stride(y, shape, bf16 if scale is None else e4m3, "y", what)
    if gate is not None:
        gp = gate.data_ptr()
        if gate.dim() == 2:
            gs = _row_stride(gate, shape, bf16, "gate", what)
        elif gate.dim() != 1 or gate.dtype not in bf16:
            raise UwError(UW_ERR_SHAPE, "%s (gate is %s of %s)" % (what, tuple(gate.shape), gate.dtype))
        else:
            _refuse(_short((gate, 2 * d, "gate")), what)
    for t, name in ((weight, "weight"), (post_weight, "post_weight")):
        if t is not None:
            if t.dtype not in bf16:
                raise UwError(UW_ERR_SHAPE, "%s (%s is not BF16)" % (what, name))
            _refuse(_short((t, 2 * d, name)), what)
    if weight is not None:
        wp = weight.data_ptr()
    if post_weight is not None:
        pp = post_weight.data_ptr()
    b = Block(pp, gp, gs, weight_offset, residual_scale, block_scale, eps)
    if scale is not None:
        if scale.dtype is not fp32:
            raise UwError(UW_ERR_SHAPE, "%s (scale is not fp32)" % what)
        _refuse(_short((scale, 4 * n, "scale")), what)
    _here(what, x, residual, weight, residual_out, y, post_weight, gate, scale)
    if scale is None:
        _check(load().uw_block_norm(b, x.data_ptr(), xs, residual.data_ptr(), rs, hp, hs, wp, n, d, yp, ys,
                                    _stream(stream)), what)
    else:
        _check(load().uw_block_norm_e4m3(b, x.data_ptr(), xs, residual.data_ptr(), rs, hp, hs, wp, n, d, yp, ys,
                                         scale.data_ptr(), _stream(stream)), what)


class Kv4Cache:
    """A layer's cache: its descriptor with the tensors behind it (made by kv4_cache)."""

    def __init__(self, desc, pages, table):
        self.desc, self.pages, self.table, self.ref = desc, pages, table, ctypes.byref(desc)
        self.n_seqs, self.kv_heads, self.head_dim = desc.n_seqs, desc.kv_heads, desc.head_dim


def kv4_page_bytes(kv_heads: int, head_dim: int, page_size: int) -> int:
    n = _SZ(0)
    _check(load().uw_kv4_page_bytes(kv_heads, head_dim, page_size, ctypes.byref(n)), "uw_kv4_page_bytes")
    return int(n.value)


def kv4_cache(pages, table, kv_heads: int, head_dim: int, page_size: int) -> Kv4Cache:
    """The cache in `pages` (bytes of whole pages, contiguous) with the page table
    `table` (int32 [sequences, pages of the longest])."""
    size = kv4_page_bytes(kv_heads, head_dim, page_size)
    if not pages.is_contiguous() or _nbytes(pages) % size:
        raise UwError(UW_ERR_SHAPE, "uw_kv4_cache (pages are not whole pages of %d bytes)" % size)
    if table.dim() != 2 or table.dtype is not _types()[2] or (table.shape[1] > 1 and table.stride(1) != 1):
        raise UwError(UW_ERR_SHAPE, "uw_kv4_cache (table is not int32 [sequences, pages])")
    stride = table.stride(0) if table.shape[0] > 1 else table.shape[1]
    d = Kv4CacheDesc(pages.data_ptr(), table.data_ptr(), _nbytes(pages) // size, stride, table.shape[1],
                     table.shape[0], kv_heads, head_dim, page_size)
    return Kv4Cache(d, pages, table)


def kv4_workspace_size(cache: Kv4Cache, q_heads: int) -> int:
    n = _SZ(0)
    _check(load().uw_kv4_workspace_size(cache.ref, q_heads, ctypes.byref(n)), "uw_kv4_workspace_size")
    return int(n.value)


def _kv4_rows(t, n: int, heads: int, dim: int, name: str, what: str) -> Kv4Rows:
    if t.shape != (n, heads, dim) or t.dtype not in _types()[0]:
        raise UwError(UW_ERR_SHAPE, "%s (%s is %s of %s, not BF16 [%d, %d, %d])" % (what, name, tuple(t.shape),
                                                                                  t.dtype, n, heads, dim))
    ts, hs, ds = t.stride() if n else (0, 0, 1)
    if ds != 1:
        raise UwError(UW_ERR_INVALID_ARG, "%s (%s: a head's values are not contiguous)" % (what, name))
    return Kv4Rows(t.data_ptr(), ts if n > 1 else 0, hs if heads > 1 else 0)


def _kv4_seqs(cache, start, length, what):
    """start and length are int32 [sequences + 1] and [sequences] at least."""
    n, int32 = cache.n_seqs, _types()[2]
    if not (start.is_contiguous() and length.is_contiguous() and start.dtype is int32 and length.dtype is int32
            and start.numel() > n and length.numel() >= n):
        _refuse("start and length are not int32 of %d and %d values" % (n + 1, n), what)


def kv4_append(cache: Kv4Cache, start, length, q, k, v, q_out, cos, sin, ws, interleaved: bool = False, stream=None):
    """uw_kv4_append: rotate q (into q_out; both may be None) and k, and append k and v.  Tensors
    [tokens, heads, head_dim], strided if need be; cos and sin fp32 [positions, rotated pairs], or None."""
    what, d = "uw_kv4_append", cache
    n = k.shape[0]
    _kv4_seqs(cache, start, length, what)
    kr = _kv4_rows(k, n, d.kv_heads, d.head_dim, "k", what)
    vr = _kv4_rows(v, n, d.kv_heads, d.head_dim, "v", what)
    if (q is None) != (q_out is None) or (cos is None) != (sin is None):
        raise UwError(UW_ERR_INVALID_ARG, "%s (q and q_out, cos and sin: both or neither)" % what)
    heads = 0 if q is None else q.shape[1] if q.dim() == 3 else -1
    qr = orow = None
    if q is not None:
        qr = _kv4_rows(q, n, heads, d.head_dim, "q", what)
        orow = _kv4_rows(q_out, n, heads, d.head_dim, "q_out", what)
    rope_len = rot = 0
    if cos is not None:
        rope = cos.shape
        fp32 = _types()[3]
        if len(rope) != 2 or rope != sin.shape or cos.dtype is not fp32 or sin.dtype is not fp32:
            raise UwError(UW_ERR_SHAPE, "%s (cos and sin are not fp32 [positions, pairs])" % what)
        if not (cos.is_contiguous() and sin.is_contiguous()):
            raise UwError(UW_ERR_INVALID_ARG, "%s (cos and sin are not contiguous)" % what)
        rope_len, rot = rope[0], 2 * rope[1]
    _check(load().uw_kv4_append(cache.ref, start.data_ptr(), length.data_ptr(), n, qr, heads, orow, kr, vr,
                                cos.data_ptr() if rot else None, sin.data_ptr() if rot else None, rope_len, rot,
                                interleaved, ws.data_ptr(), _nbytes(ws), _stream(stream)), what)


def _rope(pos, pair_axis, cos, sin, n: int, interleaved: bool, what: str) -> Rope:
    _, _, int32, fp32 = _types()
    if not pair_axis and (cos is None or cos.dim() == 2 and cos.shape[1] == 0) and (cos is None) == (sin is None):
        return Rope(None, 0, 0, 0, None, None, None, 0, interleaved)    # nothing turns
    if pos is None or cos is None or sin is None:
        raise UwError(UW_ERR_SHAPE, "%s (pos, cos and sin: all of them where pairs turn)" % what)
    if pos.dim() != 2 or pos.shape[1] != n or pos.dtype is not int32 or (n > 1 and pos.stride(1) != 1):
        raise UwError(UW_ERR_SHAPE, "%s (pos is not int32 [axes, %d])" % (what, n))
    rope = cos.shape
    if len(rope) != 2 or rope != sin.shape or cos.dtype is not fp32 or sin.dtype is not fp32 or rope[1] != len(pair_axis):
        raise UwError(UW_ERR_SHAPE, "%s (cos and sin are not fp32 [positions, pairs])" % what)
    if not (cos.is_contiguous() and sin.is_contiguous()):
        raise UwError(UW_ERR_INVALID_ARG, "%s (cos and sin are not contiguous)" % what)
    return Rope(pos.data_ptr(), pos.stride(0) if pos.shape[0] > 1 else n, pos.shape[0], 2 * rope[1], pair_axis,
                cos.data_ptr(), sin.data_ptr(), rope[0], interleaved)


def _head_rows(t, n: int, dim: int, name: str, what: str):
    """Heads and rows of [n, heads, dim]; (0, None) for None."""
    if t is None:
        return 0, None
    heads = t.shape[1] if t.dim() == 3 else -1
    return heads, _kv4_rows(t, n, heads, dim, name, what)


def rope_axes(q, k, pos, pair_axis: bytes, q_out, k_out, cos, sin, ws, interleaved: bool = False, stream=None):
    """uw_rope_axes: rotate q and k [tokens, heads, head_dim] (either may be None) into q_out and k_out by the positions
    pos, int32 [axes, tokens]; pair i turns by axis pair_axis[i].  cos and sin fp32 [positions, pairs]."""
    what = "uw_rope_axes"
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise UwError(UW_ERR_INVALID_ARG, "%s (q and q_out, k and k_out: both or neither)" % what)
    some = k if q is None else q
    if some is None or some.dim() != 3:
        raise UwError(UW_ERR_SHAPE, "%s (q and k are not [tokens, heads, head_dim])" % what)
    n, d = some.shape[0], some.shape[2]
    hq, qr = _head_rows(q, n, d, "q", what)
    hk, kr = _head_rows(k, n, d, "k", what)
    qo = None if q is None else _kv4_rows(q_out, n, hq, d, "q_out", what)
    ko = None if k is None else _kv4_rows(k_out, n, hk, d, "k_out", what)
    r = _rope(pos, pair_axis, cos, sin, n, interleaved, what)
    _here(what, some, q, k, q_out, k_out, pos, cos, sin, ws)
    _check(load().uw_rope_axes(r, n, qr, hq, qo, kr, hk, ko, d, ws.data_ptr(), _nbytes(ws), _stream(stream)), what)


def kv4_append_axes(cache: Kv4Cache, start, length, pos, pair_axis: bytes, q, k, v, q_out, cos, sin, ws, k_out=None,
                    interleaved: bool = False, stream=None):
    """uw_kv4_append_axes: kv4_append with positions on several axes (pos and pair_axis as for rope_axes); k_out, if
    given, takes the rotated k.  With no pairs (pair_axis b"") nothing turns; pos, cos and sin may be None."""
    what, d = "uw_kv4_append_axes", cache
    n = k.shape[0]
    _kv4_seqs(cache, start, length, what)
    kr = _kv4_rows(k, n, d.kv_heads, d.head_dim, "k", what)
    vr = _kv4_rows(v, n, d.kv_heads, d.head_dim, "v", what)
    if (q is None) != (q_out is None):
        raise UwError(UW_ERR_INVALID_ARG, "%s (q and q_out: both or neither)" % what)
    hq, qr = _head_rows(q, n, d.head_dim, "q", what)
    qo = None if q is None else _kv4_rows(q_out, n, hq, d.head_dim, "q_out", what)
    ko = None if k_out is None else _kv4_rows(k_out, n, d.kv_heads, d.head_dim, "k_out", what)
    r = _rope(pos, pair_axis, cos, sin, n, interleaved, what)
    _here(what, cache.pages, cache.table, start, length, pos, q, k, v, q_out, k_out, cos, sin, ws)
    _check(load().uw_kv4_append_axes(cache.ref, start.data_ptr(), length.data_ptr(), n, r, qr, hq, qo, kr, vr, ko,
                                     ws.data_ptr(), _nbytes(ws), _stream(stream)), what)


def kv4_read(cache: Kv4Cache, start, length, k, v, ws, stream=None):
    """uw_kv4_read: the new tokens' entries as BF16 into k and v [tokens, kv heads, head_dim]."""
    what, d = "uw_kv4_read", cache
    n = k.shape[0]
    _kv4_seqs(cache, start, length, what)
    kr = _kv4_rows(k, n, d.kv_heads, d.head_dim, "k", what)
    vr = _kv4_rows(v, n, d.kv_heads, d.head_dim, "v", what)
    _check(load().uw_kv4_read(cache.ref, start.data_ptr(), length.data_ptr(), n, kr, vr, ws.data_ptr(), _nbytes(ws),
                              _stream(stream)), what)


def kv4_attention(cache: Kv4Cache, start, length, q, out, ws, max_new: int = 0, max_len: int = 0,
                  scale: float = 0.0, causal: bool = True, window: int = 0, lse=None, stream=None):
    """uw_kv4_attention: attention of the new tokens' q [tokens, q heads, head_dim] over the cache into out."""
    what, d = "uw_kv4_attention", cache
    n, heads = q.shape[0], q.shape[1] if q.dim() == 3 else -1
    _kv4_seqs(cache, start, length, what)
    qr = _kv4_rows(q, n, heads, d.head_dim, "q", what)
    orow = _kv4_rows(out, n, heads, d.head_dim, "out", what)
    if lse is not None:
        if lse.dtype is not _types()[3]:
            raise UwError(UW_ERR_SHAPE, "%s (lse is not fp32)" % what)
        _refuse(_short((lse, 4 * n * heads, "lse")), what)
    _check(load().uw_kv4_attention(cache.ref, start.data_ptr(), length.data_ptr(), n, qr, heads, orow,
                                   None if lse is None else lse.data_ptr(), max_new, max_len, scale, causal, window,
                                   ws.data_ptr(), _nbytes(ws), _stream(stream)), what)


def attention_workspace_size(head_dim: int) -> int:
    n = _SZ(0)
    _check(load().uw_attention_workspace_size(head_dim, ctypes.byref(n)), "uw_attention_workspace_size")
    return int(n.value)


def attention(q, k, v, out, start, ws, kv_start=None, scale: float = 0.0, causal: bool = True, window: int = 0, lse=None,
              stream=None):
    """uw_attention: attention of q [tokens, q heads, head_dim] over k and v [keys, kv heads, head_dim] into out;
    sequence s has the tokens start[s] .. start[s + 1] - 1 (int32) and the same keys, or those of kv_start.  lse: fp32
    [tokens, q heads], or None."""
    what, int32 = "uw_attention", _types()[2]
    if q.dim() != 3 or k.dim() != 3:
        raise UwError(UW_ERR_SHAPE, "%s (q and k are not [tokens, heads, head_dim])" % what)
    (n, hq, d), (m, hk, _) = q.shape, k.shape
    qr, orow = _kv4_rows(q, n, hq, d, "q", what), _kv4_rows(out, n, hq, d, "out", what)
    kr, vr = _kv4_rows(k, m, hk, d, "k", what), _kv4_rows(v, m, hk, d, "v", what)
    seqs = start.numel() - 1
    for t in (start, start if kv_start is None else kv_start):
        if t.dtype is not int32 or t.dim() != 1 or t.numel() != seqs + 1 or seqs < 0 or not t.is_contiguous():
            raise UwError(UW_ERR_SHAPE, "%s (start and kv_start are not int32 [sequences + 1])" % what)
    if lse is not None:
        if lse.dtype is not _types()[3]:
            raise UwError(UW_ERR_SHAPE, "%s (lse is not fp32)" % what)
        _refuse(_short((lse, 4 * n * hq, "lse")), what)
        if lse.dim() > 1 and lse.shape[-1] != hq and min(n, hq) > 1:
            raise UwError(UW_ERR_SHAPE, "%s (lse is %s, its rows are not of %d heads)" % (what, tuple(lse.shape), hq))
    _here(what, q, k, v, out, start, kv_start, lse, ws)
    _check(load().uw_attention(start.data_ptr(), None if kv_start is None else kv_start.data_ptr(), seqs, n, m, qr, hq, kr,
                               vr, hk, d, orow, None if lse is None else lse.data_ptr(), scale, causal, window,
                               ws.data_ptr(), _nbytes(ws), _stream(stream)), what)


def selftest_attention_wait(ws, tries: int, stream=None) -> None:
    """uw_selftest_attention_wait: the waits of uw_attention run out; read the result with check_status."""
    _check(load().uw_selftest_attention_wait(_ptr(ws), ws.numel() * ws.element_size(), int(tries), _stream(stream)),
           "uw_selftest_attention_wait")


def selftest_bounded_wait(ws, tries: int, stream=None) -> None:
    """uw_selftest_bounded_wait: a kernel whose bounded wait runs out; read
    the result with check_status."""
    _check(load().uw_selftest_bounded_wait(_ptr(ws), ws.numel() * ws.element_size(), int(tries), _stream(stream)),
           "uw_selftest_bounded_wait")


def check_status(ws, stream=None) -> int:
    """uw_check_status: synchronises and returns the device error status (0 = ok)."""
    return int(load().uw_check_status(_ptr(ws), _stream(stream)))
