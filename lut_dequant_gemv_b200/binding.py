"""Python binding of ``libsqz.so`` (C ABI in ``include/sqz.h``).

Argument marshalling only: every step of the computation runs in the CUDA
library.  Functions keep the C names.  Device arrays are torch CUDA tensors
(fp16 data may be passed as ``torch.float16`` or as its ``torch.int16`` bit
pattern); streams default to torch's current stream.  A non-OK status raises
:class:`SqzError` carrying the library's message.  If ``libsqz.so`` is
missing the first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsqz.so")

SQZ_OK = 0
SQZ_ERR_INVALID_ARG = 1
SQZ_ERR_UNSUPPORTED = 2
SQZ_ERR_CUDA = 3
SQZ_ERR_OOM = 4
SQZ_ERR_TIMEOUT = 5
SQZ_MAX_BATCH = 16
SQZ_MAC_TENSOR_CORES = 0
SQZ_MAC_CUDA_CORES = 1
SQZ_MAC_MIXED = 2
SQZ_CSR_BALANCED = 0
SQZ_CSR_ROWWISE = 1
SQZ_FP8_E4M3 = 0
SQZ_FP8_E5M2 = 1
SQZ_TYPE_F16 = 0
SQZ_TYPE_BF16 = 1
SQZ_TYPE_F32 = 2
SQZ_MOE_MAX_TOKENS = 32
SQZ_MOE_MAX_EXPERTS = 1024
SQZ_MOE_MAX_TOP_K = 16

STATUS_NAMES = {0: "SQZ_OK", 1: "SQZ_ERR_INVALID_ARG", 2: "SQZ_ERR_UNSUPPORTED", 3: "SQZ_ERR_CUDA",
                4: "SQZ_ERR_OOM", 5: "SQZ_ERR_TIMEOUT"}

# Every entry point include/sqz.h declares.
EXPORTED = ("sqz_create_layer", "sqz_gemv", "sqz_gemv_host", "sqz_debug_dequant", "sqz_layer_info",
            "sqz_destroy", "sqz_fp16_gemv", "sqz_last_error", "sqz_version", "sqz_check_csr_static",
            "sqz_layer_set_mac", "sqz_layer_set_csr_mode", "sqz_layer_status", "sqz_encode",
            "sqz_encode_outliers", "sqz_plan_query", "sqz_layer_set_predecode", "sqz_tile_split_query",
            "sqz_fp8_quantize", "sqz_fp8_gemm", "sqz_fp8_status", "sqz_fp8_plan_query", "sqz_create_moe",
            "sqz_moe_workspace_bytes", "sqz_moe_forward", "sqz_moe_status", "sqz_destroy_moe")


class SqzError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class sqz_plan_info(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "fused", "columns_per_launch", "launches", "grid", "threads", "ctas_per_sm", "smem_bytes", "passes",
        "ring_stages", "csr_stage_entries", "predecode")]


class sqz_layer_desc(ctypes.Structure):
    _fields_ = [
        ("n_out", ctypes.c_int32),
        ("k_in", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("codes", ctypes.c_void_p),
        ("lut", ctypes.c_void_p),
        ("nnz", ctypes.c_int64),
        ("rowptr", ctypes.c_void_p),
        ("col", ctypes.c_void_p),
        ("val", ctypes.c_void_p),
    ]


class sqz_fp8_matrix(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("ld", ctypes.c_int64),
        ("scale", ctypes.c_void_p),
        ("ld_scale", ctypes.c_int64),
        ("format", ctypes.c_int32),
    ]


class sqz_fp8_plan_info(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("many_rows", "tile_rows", "tile_cols", "splits")]


class sqz_moe_desc(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("experts", "top_k", "hidden", "inter", "x_type", "renormalize")] + [
        ("router", ctypes.c_void_p),
        ("ld_router", ctypes.c_int64),
        ("w13", ctypes.c_void_p),
        ("w13_scale", ctypes.c_void_p),
        ("w2", ctypes.c_void_p),
        ("w2_scale", ctypes.c_void_p),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libsqz.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m lut_dequant_gemv_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.sqz_create_layer.argtypes = [ctypes.POINTER(sqz_layer_desc), P, ctypes.POINTER(P)]
        L.sqz_gemv.argtypes = [P, P, i32, i64, P, i64, P]
        L.sqz_gemv_host.argtypes = [P, P, i32, i64, P, i64, P]
        L.sqz_debug_dequant.argtypes = [P, P, P]
        L.sqz_layer_info.argtypes = [P, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32),
                                     ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.sqz_destroy.argtypes = [P]
        L.sqz_fp16_gemv.argtypes = [P, i32, i32, i64, P, i32, i64, P, i64, P]
        for name in ("sqz_create_layer", "sqz_gemv", "sqz_gemv_host", "sqz_debug_dequant", "sqz_layer_info",
                     "sqz_destroy", "sqz_fp16_gemv"):
            getattr(L, name).restype = ctypes.c_int
        L.sqz_layer_set_mac.argtypes = [P, i32]
        L.sqz_layer_set_mac.restype = ctypes.c_int
        L.sqz_layer_set_csr_mode.argtypes = [P, i32]
        L.sqz_layer_set_csr_mode.restype = ctypes.c_int
        L.sqz_layer_set_predecode.argtypes = [P, i32]
        L.sqz_layer_set_predecode.restype = ctypes.c_int
        L.sqz_layer_status.argtypes = [P, P, ctypes.POINTER(i32)]
        L.sqz_layer_status.restype = ctypes.c_int
        L.sqz_check_csr_static.argtypes = [P, P, i32, i32, i64, P, ctypes.POINTER(i32)]
        L.sqz_check_csr_static.restype = ctypes.c_int
        L.sqz_encode.argtypes = [P, i32, i32, i32, ctypes.c_double, i32, P, P, P, P, P, i64,
                                 ctypes.POINTER(i64), P, P]
        L.sqz_encode.restype = ctypes.c_int
        L.sqz_plan_query.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(sqz_plan_info)]
        L.sqz_plan_query.restype = ctypes.c_int
        L.sqz_tile_split_query.argtypes = [P, i32, i32, i32, i32, P, ctypes.POINTER(i32)]
        L.sqz_tile_split_query.restype = ctypes.c_int
        L.sqz_fp8_quantize.argtypes = [P, i32, i64, i32, i32, i64, i32, i32, P, i64, P, i64, P]
        L.sqz_fp8_quantize.restype = ctypes.c_int
        M = ctypes.POINTER(sqz_fp8_matrix)
        L.sqz_fp8_gemm.argtypes = [M, M, i32, i32, i32, P, i64, i32, P]
        L.sqz_fp8_gemm.restype = ctypes.c_int
        L.sqz_fp8_status.argtypes = [P, ctypes.POINTER(i32)]
        L.sqz_fp8_status.restype = ctypes.c_int
        L.sqz_fp8_plan_query.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sqz_fp8_plan_info)]
        L.sqz_fp8_plan_query.restype = ctypes.c_int
        L.sqz_create_moe.argtypes = [ctypes.POINTER(sqz_moe_desc), ctypes.POINTER(P)]
        L.sqz_moe_workspace_bytes.argtypes = [P, i32, ctypes.POINTER(i64)]
        L.sqz_moe_forward.argtypes = [P, P, i32, i64, P, i64, P, P, P, i64, P]
        L.sqz_moe_status.argtypes = [P, P, ctypes.POINTER(i32)]
        L.sqz_destroy_moe.argtypes = [P]
        for name in ("sqz_create_moe", "sqz_moe_workspace_bytes", "sqz_moe_forward", "sqz_moe_status",
                     "sqz_destroy_moe"):
            getattr(L, name).restype = ctypes.c_int
        L.sqz_encode_outliers.argtypes = [i64, ctypes.c_double]
        L.sqz_encode_outliers.restype = i64
        L.sqz_last_error.argtypes = []
        L.sqz_last_error.restype = ctypes.c_char_p
        L.sqz_version.argtypes = []
        L.sqz_version.restype = ctypes.c_int32
        _lib = L
    return _lib


def sqz_last_error() -> str:
    return lib().sqz_last_error().decode("utf-8", "replace")


def sqz_version() -> int:
    return int(lib().sqz_version())


def _check(status: int, where: str) -> None:
    if status != SQZ_OK:
        raise SqzError(status, where, sqz_last_error())


def _dptr(t: Optional[torch.Tensor], name: str, dtypes) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() else None


def _hptr(t: torch.Tensor, name: str) -> Optional[int]:
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype not in (torch.float16, torch.int16):
        raise TypeError(f"{name} must hold fp16 data")
    return t.data_ptr() if t.numel() else None


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


_H16 = (torch.float16, torch.int16)


def _lead(t: torch.Tensor, name: str) -> int:
    """Rows of a 2-D (or 1-D = one row) row-major tensor and its leading dimension."""
    if t.dim() == 1:
        return t.shape[0]
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 1-D or a 2-D row-major matrix")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class Layer:
    """Owning handle for an ``sqz_layer_t`` (destroyed on garbage collection)."""

    def __init__(self, handle: int, n_out: int, k_in: int, bits: int, nnz: int):
        self.handle = ctypes.c_void_p(handle)
        self.n_out, self.k_in, self.bits, self.nnz = n_out, k_in, bits, nnz

    def close(self) -> None:
        if self.handle is not None and self.handle.value:
            sqz_destroy(self)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def _as_parameter_(self):
        if self.handle is None:
            raise ValueError("layer has been destroyed")
        return self.handle


def sqz_create_layer(n_out: int, k_in: int, bits: int, codes: torch.Tensor, lut: torch.Tensor,
                     rowptr: Optional[torch.Tensor] = None, col: Optional[torch.Tensor] = None,
                     val: Optional[torch.Tensor] = None, stream=None) -> Layer:
    """Create a layer from canonical device arrays (see ``include/sqz.h``)."""
    nnz = 0 if col is None else int(col.numel())
    d = sqz_layer_desc(
        n_out=n_out, k_in=k_in, bits=bits,
        codes=_dptr(codes, "codes", (torch.int32, torch.uint32)),
        lut=_dptr(lut, "lut", _H16),
        nnz=nnz,
        rowptr=_dptr(rowptr, "rowptr", (torch.int32,)),
        col=_dptr(col, "col", (torch.int32,)),
        val=_dptr(val, "val", _H16),
    )
    out = ctypes.c_void_p()
    _check(lib().sqz_create_layer(ctypes.byref(d), _stream(stream), ctypes.byref(out)), "sqz_create_layer")
    return Layer(out.value, n_out, k_in, bits, nnz)


def _check_shapes(layer: Layer, x: torch.Tensor, y: torch.Tensor, batch: int) -> None:
    rows_x = x.shape[0] if x.dim() == 2 else 1
    rows_y = y.shape[0] if y.dim() == 2 else 1
    if x.shape[-1] < layer.k_in or y.shape[-1] < layer.n_out:
        raise ValueError(f"x needs >= {layer.k_in} columns and y >= {layer.n_out} (got {tuple(x.shape)}, "
                         f"{tuple(y.shape)})")
    if batch > rows_x or batch > rows_y:
        raise ValueError(f"batch {batch} exceeds the rows of x {tuple(x.shape)} or y {tuple(y.shape)}")


def sqz_gemv(layer: Layer, x: torch.Tensor, y: torch.Tensor, batch: Optional[int] = None, stream=None) -> None:
    """y[b, :N] = (Q + S) x[b, :K] for b < batch (device tensors, fp16)."""
    batch = (x.shape[0] if x.dim() == 2 else 1) if batch is None else batch
    _check_shapes(layer, x, y, batch)
    _check(lib().sqz_gemv(layer, _dptr_any(x, "x"), batch, _lead(x, "x"), _dptr_any(y, "y"), _lead(y, "y"),
                          _stream(stream)), "sqz_gemv")


def _dptr_any(t: torch.Tensor, name: str) -> Optional[int]:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _H16:
        raise TypeError(f"{name} must hold fp16 data")
    return t.data_ptr() if t.numel() else None


def sqz_gemv_host(layer: Layer, x: torch.Tensor, y: torch.Tensor, batch: Optional[int] = None, stream=None) -> None:
    """Host-memory variant: x and y are CPU tensors (pinned for async copies)."""
    batch = (x.shape[0] if x.dim() == 2 else 1) if batch is None else batch
    _check_shapes(layer, x, y, batch)
    _check(lib().sqz_gemv_host(layer, _hptr(x, "x"), batch, _lead(x, "x"), _hptr(y, "y"), _lead(y, "y"),
                               _stream(stream)), "sqz_gemv_host")


def sqz_debug_dequant(layer: Layer, w_out: torch.Tensor, stream=None) -> None:
    _check(lib().sqz_debug_dequant(layer, _dptr(w_out, "w_out", _H16), _stream(stream)), "sqz_debug_dequant")


def sqz_layer_info(layer: Layer) -> dict:
    n, k, b = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    nnz, nbytes = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().sqz_layer_info(layer, ctypes.byref(n), ctypes.byref(k), ctypes.byref(b), ctypes.byref(nnz),
                                ctypes.byref(nbytes)), "sqz_layer_info")
    return dict(n_out=n.value, k_in=k.value, bits=b.value, nnz=nnz.value, device_bytes=nbytes.value)


def sqz_destroy(layer: Layer) -> None:
    h = layer.handle if isinstance(layer, Layer) else layer
    _check(lib().sqz_destroy(h), "sqz_destroy")
    if isinstance(layer, Layer):
        layer.handle = None


def sqz_fp16_gemv(w: torch.Tensor, x: torch.Tensor, y: torch.Tensor, batch: Optional[int] = None,
                  stream=None) -> None:
    """Dense fp16 yardstick: y = W x, W [N][ldw] fp16 on the device."""
    batch = (x.shape[0] if x.dim() == 2 else 1) if batch is None else batch
    n_out, k_in = w.shape
    _check(lib().sqz_fp16_gemv(_dptr_any(w, "w"), n_out, k_in, _lead(w, "w"), _dptr_any(x, "x"), batch,
                               _lead(x, "x"), _dptr_any(y, "y"), _lead(y, "y"), _stream(stream)), "sqz_fp16_gemv")


def create_layer_from_numpy(n_out: int, k_in: int, bits: int, codes, lut, rowptr=None, col=None, val=None,
                            device=None, stream=None) -> Layer:
    """Copy host (numpy) arrays in canonical storage to the device and create a layer."""
    import numpy as np

    dev = torch.device("cuda") if device is None else torch.device(device)

    def up(a, dt):
        if a is None:
            return None
        return torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(dev)

    nnz = 0 if col is None else len(col)
    t_codes = up(codes, np.int32)
    t_lut = up(lut, np.int16)
    t_rp = up(rowptr, np.int32) if nnz else None
    t_col = up(col, np.int32) if nnz else None
    t_val = up(val, np.int16) if nnz else None
    layer = sqz_create_layer(n_out, k_in, bits, t_codes, t_lut, t_rp, t_col, t_val, stream=stream)
    torch.cuda.current_stream(dev).synchronize()
    return layer


def sqz_check_csr_static(rowptr: Optional[torch.Tensor], col: Optional[torch.Tensor], n_out: int, k_in: int,
                         stream=None) -> int:
    """CSR check without device allocation; returns the flag word (0 = well formed)."""
    nnz = 0 if col is None else int(col.numel())
    flags = ctypes.c_int32(-1)
    _check(lib().sqz_check_csr_static(_dptr(rowptr, "rowptr", (torch.int32,)), _dptr(col, "col", (torch.int32,)),
                                      n_out, k_in, nnz, _stream(stream), ctypes.byref(flags)),
           "sqz_check_csr_static")
    return int(flags.value)


B200_DEVICE = {"sm_count": 148, "smem_per_sm": 233472, "smem_optin": 232448}


def sqz_plan_query(n_out: int, k_in: int, bits: int, batch: int, sm_count: int = 148, smem_per_sm: int = 233472,
                   smem_optin: int = 232448, predecode: int = 0) -> dict:
    """The launch plan sqz_gemv would use (host computation; defaults: B200)."""
    info = sqz_plan_info()
    _check(lib().sqz_plan_query(n_out, k_in, bits, batch, sm_count, smem_per_sm, smem_optin, int(predecode),
                                ctypes.byref(info)), "sqz_plan_query")
    return {name: int(getattr(info, name)) for name, _ in sqz_plan_info._fields_}


def sqz_tile_split_query(rowptr, n_out: int, k_in: int, bits: int, sm_count: int = 148):
    """The CTA -> tile split sqz_create_layer would use for this host rowptr
    (host computation): (first tile of every CTA plus the tile count as an
    int32 array of grid + 1 entries, True when the split by weight is used)."""
    rp = np.ascontiguousarray(rowptr, dtype=np.int32)
    if rp.shape != (n_out + 1,):
        raise ValueError(f"rowptr must have n_out + 1 = {n_out + 1} entries")
    ntiles = (max(n_out, 0) + 15) // 16
    first = np.zeros(max(1, min(sm_count, ntiles)) + 1, dtype=np.int32)
    weighted = ctypes.c_int32(0)
    _check(lib().sqz_tile_split_query(rp.ctypes.data, n_out, k_in, bits, sm_count, first.ctypes.data,
                                      ctypes.byref(weighted)), "sqz_tile_split_query")
    return first, bool(weighted.value)


def sqz_encode_outliers(n_weights: int, outlier_fraction: float) -> int:
    return int(lib().sqz_encode_outliers(int(n_weights), float(outlier_fraction)))


def sqz_encode(w: torch.Tensor, bits: int, outlier_fraction: float, max_iters: int, stream=None,
               want_iters: bool = False):
    """Quantize fp16 weights [n_out, k_in] (CUDA) into (codes, lut, rowptr, col,
    val[, iters]) device tensors in the layout sqz_create_layer takes."""
    if w.dim() != 2 or not w.is_contiguous():
        raise ValueError("w must be a contiguous [n_out, k_in] tensor")
    n_out, k_in = (int(d) for d in w.shape)
    dev = w.device
    nnz = sqz_encode_outliers(n_out * k_in, outlier_fraction)
    wpr = k_in * bits // 32 if bits in (3, 4) else 0
    codes = torch.empty((n_out, max(wpr, 1)), dtype=torch.int32, device=dev)
    lut = torch.empty((n_out, 1 << bits if bits in (3, 4) else 1), dtype=torch.int16, device=dev)
    rowptr = torch.empty(n_out + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
    val = torch.empty(max(nnz, 1), dtype=torch.int16, device=dev)
    iters = torch.empty(n_out, dtype=torch.int32, device=dev) if want_iters else None
    got = ctypes.c_int64(0)
    _check(lib().sqz_encode(_dptr_any(w, "w"), n_out, k_in, int(bits), float(outlier_fraction), int(max_iters),
                            codes.data_ptr(), lut.data_ptr(), rowptr.data_ptr(), col.data_ptr(), val.data_ptr(),
                            max(nnz, 1), ctypes.byref(got), None if iters is None else iters.data_ptr(),
                            _stream(stream)), "sqz_encode")
    n = int(got.value)
    out = (codes[:, :wpr], lut, rowptr, col[:n], val[:n])
    return out + (iters,) if want_iters else out


def sqz_layer_set_mac(layer: Layer, mac: int) -> None:
    _check(lib().sqz_layer_set_mac(layer, int(mac)), "sqz_layer_set_mac")


def sqz_layer_set_csr_mode(layer: Layer, mode: int) -> None:
    _check(lib().sqz_layer_set_csr_mode(layer, int(mode)), "sqz_layer_set_csr_mode")


def sqz_layer_set_predecode(layer: Layer, enable: int) -> None:
    _check(lib().sqz_layer_set_predecode(layer, int(enable)), "sqz_layer_set_predecode")


def sqz_layer_status(layer: Layer, stream=None) -> int:
    st = ctypes.c_int32(-1)
    _check(lib().sqz_layer_status(layer, _stream(stream), ctypes.byref(st)), "sqz_layer_status")
    return int(st.value)


# ------------------------------------------------ 8-bit floating point, block scales
_FP8_FORMATS = {torch.float8_e4m3fn: SQZ_FP8_E4M3, torch.float8_e5m2: SQZ_FP8_E5M2}
_H16_TYPES = (torch.float16, torch.bfloat16)
_TYPES = {torch.float16: SQZ_TYPE_F16, torch.bfloat16: SQZ_TYPE_BF16, torch.float32: SQZ_TYPE_F32}


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _on_current_device(t: torch.Tensor, name: str) -> int:
    """The tensor's device, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")
    return dev


def _raw_stream(stream, device: int) -> Optional[int]:
    """As _stream; torch's current stream of the device without making an object of it (these calls take a
    few microseconds on the GPU)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device) or None
    return _stream(stream)


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory that a call on `stream` writes: it belongs to that stream (what the current stream has freed may still
    be in use there)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _pitch(t: torch.Tensor, name: str) -> int:
    """Elements from one row to the next of a tensor whose rows are contiguous and, beyond two
    dimensions, evenly spaced; for a single row, its length rounded up to 16."""
    shape, strides = t.shape, t.stride()
    if len(shape) < 2:
        raise ValueError(f"{name} must have at least two dimensions")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be row-major")
    if len(shape) == 2:
        return strides[0] if shape[0] > 1 else (shape[1] + 15) // 16 * 16
    rows, ld = 1, None
    for d in range(len(shape) - 2, -1, -1):
        if shape[d] != 1:
            if ld is None:
                ld = strides[d] // rows if strides[d] % rows == 0 else -1
            if strides[d] != rows * ld:
                raise ValueError(f"{name} must have evenly spaced rows")
        rows *= shape[d]
    if ld is None:  # a single row
        ld = (shape[-1] + 15) // 16 * 16
    return ld


def sqz_fp8_quantize(x: torch.Tensor, block_rows: int = 1, dtype: torch.dtype = torch.float8_e4m3fn,
                     q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """Quantize fp16/bf16 x [rows, cols] or [batch, rows, cols] (CUDA) to 8-bit codes with one fp32 scale per block of
    block_rows (1 or 128) x 128; returns (q, scale).  q has x's shape and an fp8 dtype on a 16-byte row pitch;
    scale is [(batch,) ceil(rows / block_rows), ceil(cols / 128)].  Both are allocated (on `stream`) unless given (q's
    dtype then names the format)."""
    shape, dev = x.shape, _on_current_device(x, "x")
    if len(shape) not in (2, 3):
        raise ValueError("x must be [rows, cols] or [batch, rows, cols]")
    if x.dtype not in _H16_TYPES:
        raise TypeError(f"x has dtype {x.dtype}, expected fp16 or bf16")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    rows, cols = shape[-2], shape[-1]
    if q is None:
        if dtype not in _FP8_FORMATS:
            raise TypeError(f"dtype {dtype} is not an 8-bit floating-point type")
        q = _empty((*shape[:-1], (cols + 15) // 16 * 16), dtype, x.device, stream)[..., :cols]
    elif q.get_device() != dev or q.dtype not in _FP8_FORMATS or q.shape != shape:
        raise ValueError(f"q must have shape {tuple(shape)} and an fp8 dtype, on x's device")
    s_shape = (*shape[:-2], -(-rows // block_rows), -(-cols // 128))
    if scale is None:
        scale = _empty(s_shape, torch.float32, x.device, stream)
    elif scale.get_device() != dev or scale.dtype is not torch.float32 or scale.shape != s_shape:
        raise ValueError(f"scale must be fp32 of shape {s_shape}, on x's device")
    if rows and cols and (len(shape) == 2 or shape[0]):
        status = (_lib or lib()).sqz_fp8_quantize(
            x.data_ptr(), _TYPES[x.dtype], shape[0] if len(shape) == 3 else 1, rows, cols, _pitch(x, "x"), block_rows,
            _FP8_FORMATS[q.dtype], q.data_ptr(), _pitch(q, "q"), scale.data_ptr(), _pitch(scale, "scale"),
            _raw_stream(stream, dev))
        if status:
            _check(status, "sqz_fp8_quantize")
    return q, scale


def _fp8_matrix(q: torch.Tensor, scale: torch.Tensor, name: str, block_rows: int, dev: int) -> sqz_fp8_matrix:
    fmt = _FP8_FORMATS.get(q.dtype)
    if fmt is None:
        raise TypeError(f"{name} has dtype {q.dtype}, expected float8_e4m3fn or float8_e5m2")
    if q.get_device() != dev or scale.get_device() != dev:
        raise ValueError(f"{name} and its scales must be on y's device")
    if q.dim() != 2 or scale.dim() != 2 or scale.dtype is not torch.float32:
        raise ValueError(f"{name} must be [rows, k] with 2-D fp32 scales")
    (rows, k), (srows, blocks), (ld, inner), (lds, sinner) = q.shape, scale.shape, q.stride(), scale.stride()
    if srows != -(-rows // block_rows) or blocks != -(-k // 128):
        raise ValueError(f"{name} {tuple(q.shape)} needs scales [ceil(rows / {block_rows}), ceil(k / 128)], got "
                         f"{tuple(scale.shape)}")
    if (inner != 1 and k > 1) or (sinner != 1 and blocks > 1):
        raise ValueError(f"{name} and its scales must be row-major")
    return sqz_fp8_matrix(q.data_ptr(), ld if rows > 1 else (k + 15) // 16 * 16, scale.data_ptr(),
                          lds if srows > 1 else blocks, fmt)


def sqz_fp8_gemm(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, y: torch.Tensor,
                 stream=None) -> None:
    """y [m, n] (fp16, bf16 or fp32) = A W^T of 8-bit matrices a [m, k] (scales [m, ceil(k/128)]) and w [n, k]
    (scales [ceil(n/128), ceil(k/128)])."""
    dev, y_type = _on_current_device(y, "y"), _TYPES.get(y.dtype)
    A, W = _fp8_matrix(a, a_scale, "a", 1, dev), _fp8_matrix(w, w_scale, "w", 128, dev)
    (m, k), (n, kw) = a.shape, w.shape
    if kw != k or y.shape != (m, n):
        raise ValueError(f"a {tuple(a.shape)}, w {tuple(w.shape)} and y {tuple(y.shape)} do not fit together")
    if y_type is None:
        raise TypeError(f"y has dtype {y.dtype}, expected fp16, bf16 or fp32")
    ldy, inner = y.stride()
    if inner != 1 and n > 1:
        raise ValueError("y must be row-major")
    status = (_lib or lib()).sqz_fp8_gemm(A, W, m, n, k, y.data_ptr(), ldy if m > 1 else n, y_type,
                                          _raw_stream(stream, dev))
    if status:
        _check(status, "sqz_fp8_gemm")


def sqz_fp8_status(stream=None) -> int:
    st = ctypes.c_int32(-1)
    _check(lib().sqz_fp8_status(_stream(stream), ctypes.byref(st)), "sqz_fp8_status")
    return int(st.value)


def sqz_fp8_plan_query(m: int, n: int, k: int, sm_count: int = 148) -> dict:
    """How sqz_fp8_gemm would cut a product (host computation; default: B200)."""
    info = sqz_fp8_plan_info()
    _check(lib().sqz_fp8_plan_query(m, n, k, sm_count, ctypes.byref(info)), "sqz_fp8_plan_query")
    return {name: int(getattr(info, name)) for name, _ in sqz_fp8_plan_info._fields_}


# ------------------------------------------------ mixture of experts
class Moe:
    """Owning handle for an ``sqz_moe_t`` (destroyed on garbage collection); keeps the borrowed weights alive."""

    def __init__(self, handle: int, desc: sqz_moe_desc, dtype: torch.dtype, tensors):
        self.handle = ctypes.c_void_p(handle)
        self.experts, self.top_k, self.hidden, self.inter = desc.experts, desc.top_k, desc.hidden, desc.inter
        self.dtype, self._tensors = dtype, tensors

    def close(self) -> None:
        if self.handle is not None and self.handle.value:
            sqz_destroy_moe(self)
        self.handle = self._tensors = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def _as_parameter_(self):
        if self.handle is None:
            raise ValueError("moe has been destroyed")
        return self.handle


def sqz_create_moe(router: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                   w2_scale: torch.Tensor, top_k: int, renormalize: bool = True) -> Moe:
    """A mixture-of-experts layer: router [experts, hidden] (fp16 or bf16, also x's and y's type), w13
    [experts, 2 * inter, hidden] (gate rows, then up rows) and w2 [experts, hidden, inter] float8_e4m3fn, their fp32
    scales [experts, 2, ceil(inter/128), ceil(hidden/128)] and [experts, ceil(hidden/128), ceil(inter/128)].  The
    tensors are borrowed."""
    for name, t in (("router", router), ("w13", w13), ("w13_scale", w13_scale), ("w2", w2), ("w2_scale", w2_scale)):
        _on_current_device(t, name)
        if name != "router" and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if router.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("router must be 2-D, w13 and w2 3-D")
    if router.dtype not in _H16_TYPES:
        raise TypeError(f"router has dtype {router.dtype}, expected fp16 or bf16")
    if w13.dtype != torch.float8_e4m3fn or w2.dtype != torch.float8_e4m3fn:
        raise TypeError("w13 and w2 must be float8_e4m3fn")
    if w13_scale.dtype != torch.float32 or w2_scale.dtype != torch.float32:
        raise TypeError("the scales must be fp32")
    (experts, hidden), inter = router.shape, w2.shape[2]
    bi, bh = -(-inter // 128), -(-hidden // 128)
    if w13.shape != (experts, 2 * inter, hidden) or w2.shape != (experts, hidden, inter) or \
            w13_scale.shape != (experts, 2, bi, bh) or w2_scale.shape != (experts, bh, bi):
        raise ValueError(f"shapes do not fit together: router {tuple(router.shape)}, w13 {tuple(w13.shape)}, w13_scale "
                         f"{tuple(w13_scale.shape)}, w2 {tuple(w2.shape)}, w2_scale {tuple(w2_scale.shape)}")
    if router.stride(1) != 1:
        raise ValueError("router must be row-major")
    d = sqz_moe_desc(experts=experts, top_k=top_k, hidden=hidden, inter=inter, x_type=_TYPES[router.dtype],
                     renormalize=int(renormalize), router=router.data_ptr(),
                     ld_router=router.stride(0) if experts > 1 else hidden, w13=w13.data_ptr(),
                     w13_scale=w13_scale.data_ptr(), w2=w2.data_ptr(), w2_scale=w2_scale.data_ptr())
    out = ctypes.c_void_p()
    _check(lib().sqz_create_moe(ctypes.byref(d), ctypes.byref(out)), "sqz_create_moe")
    return Moe(out.value, d, router.dtype, (router, w13, w13_scale, w2, w2_scale))


def sqz_moe_workspace_bytes(moe: Moe, tokens: int) -> int:
    n = ctypes.c_int64(0)
    _check(lib().sqz_moe_workspace_bytes(moe, int(tokens), ctypes.byref(n)), "sqz_moe_workspace_bytes")
    return int(n.value)


def sqz_moe_workspace(moe: Moe, tokens: int) -> torch.Tensor:
    """A workspace for calls of up to `tokens` tokens with this handle, on the current device, zeroed on the current
    stream."""
    return torch.zeros(sqz_moe_workspace_bytes(moe, tokens), dtype=torch.uint8, device="cuda")


def sqz_moe_forward(moe: Moe, x: torch.Tensor, y: torch.Tensor, ids: Optional[torch.Tensor] = None,
                    weights: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """y [tokens, hidden] = the layer applied to x; ids (int32) and weights (fp32) [tokens, top_k] receive the routing.
    workspace: from sqz_moe_workspace, not shared with a call that may overlap."""
    if workspace is None:
        raise ValueError("workspace is required (sqz_moe_workspace)")
    tokens, hidden = x.shape[0], moe.hidden
    for name, t in (("x", x), ("y", y)):
        dev = _on_current_device(t, name)
        if t.dtype != moe.dtype or t.shape != (tokens, hidden) or t.stride(1) != 1:
            raise ValueError(f"{name} must be a row-major [{tokens}, {hidden}] tensor of {moe.dtype}")
    for name, t, dt in (("ids", ids, torch.int32), ("weights", weights, torch.float32)):
        if t is not None:
            _on_current_device(t, name)
            if t.dtype != dt or t.shape != (tokens, moe.top_k) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [{tokens}, {moe.top_k}] tensor of {dt}")
    _on_current_device(workspace, "workspace")
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    one = tokens <= 1
    _check((_lib or lib()).sqz_moe_forward(
        moe, x.data_ptr(), tokens, hidden if one else x.stride(0), y.data_ptr(), hidden if one else y.stride(0),
        None if ids is None else ids.data_ptr(), None if weights is None else weights.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _raw_stream(stream, dev)), "sqz_moe_forward")


def sqz_moe_status(workspace: torch.Tensor, stream=None) -> int:
    _on_current_device(workspace, "workspace")
    st = ctypes.c_int32(-1)
    _check(lib().sqz_moe_status(workspace.data_ptr(), _stream(stream), ctypes.byref(st)), "sqz_moe_status")
    return int(st.value)


def sqz_destroy_moe(moe) -> None:
    _check(lib().sqz_destroy_moe(moe.handle if isinstance(moe, Moe) else moe), "sqz_destroy_moe")
    if isinstance(moe, Moe):
        moe.handle = None
