"""Python binding of libbakron.so (ctypes): argument marshalling only.

The functions named like the C ABI (``bakron_ldl``, ``bakron_round``,
``bakron_round_stochastic``, ``bakron_round_ex``, ``bakron_proxy_loss``, ``bakron_damped_gram``,
``bakron_sketch_b``, ``bakron_rht``, ``bakron_row_scales``, ``bakron_pack4``, ``bakron_unpack4``,
``bakron_matvec4``, ``bakron_rms_norm_q8``, ``bakron_distill``, ``bakron_read_status``,
``bakron_status_string`` and the ``*_workspace_bytes`` queries) take torch CUDA tensors, pass
their device pointers and the current CUDA stream to the library and return its status code.
``ldl``, ``round_weights``, ``proxy_loss``, ``damped_gram``, ``sketch_b``, ``rht``,
``row_scales``, ``pack4``, ``unpack4``, ``matvec4``, ``rms_norm_q8``, ``distill`` and ``solve``
additionally allocate outputs and workspaces with torch and raise on any error. ``PackedLayer``
keeps a rounded layer in 4 bits.

Every step of the computation runs in the library's CUDA kernels; there is no CPU path. If
the shared library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbakron.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "bakron.h")

BAKRON_OK = 0
BAKRON_ERR_INVALID_ARG = -1
BAKRON_ERR_NOT_PD = -2
BAKRON_ERR_CUDA = -3
BAKRON_ERR_TIMEOUT = -4
BAKRON_ERR_WORKSPACE = -5
BAKRON_ERR_NONFINITE = -6
BAKRON_ERR_CAPTURE = -7

# bakron_dtype
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3, torch.int32: 4,
           torch.int64: 5}

_c_size_t, _c_int, _vp = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p
_i64 = ctypes.c_int64
_SIGNATURES = {
    "bakron_ldl_workspace_bytes": (_c_size_t, [_c_int]),
    "bakron_ldl": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _c_size_t, _vp, _vp]),
    "bakron_round_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "bakron_round": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp, _vp, _vp,
                              _c_size_t, _vp, _vp]),
    "bakron_round_stochastic": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _c_int,
                                         ctypes.c_uint64, _vp, _vp, _vp, _c_size_t, _vp, _vp]),
    "bakron_round_ex": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _c_int, _vp, _c_int, _vp,
                                 _vp, _vp, _c_size_t, _vp, _vp]),
    "bakron_proxy_loss_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "bakron_proxy_loss": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size_t, _vp]),
    "bakron_damped_gram_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "bakron_damped_gram": (_c_int, [_vp, _c_int, _c_int, ctypes.c_float, _vp, _vp, _c_size_t,
                                    _vp, _vp]),
    "bakron_sketch_b_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int]),
    "bakron_sketch_b": (_c_int, [_vp, _c_int, _c_int, _c_int, ctypes.c_float, _vp, _vp, _vp,
                                 _c_size_t, _vp, _vp]),
    "bakron_rht_supported": (_c_int, [_c_int]),
    "bakron_rht_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "bakron_rht": (_c_int, [_vp, _c_int, _c_int, ctypes.c_uint64, ctypes.c_uint64, _c_int, _vp,
                            _vp, _c_size_t, _vp]),
    "bakron_row_scales": (_c_int, [_vp, _c_int, _c_int, _c_int, ctypes.c_float, _vp, _vp]),
    "bakron_pack4_bytes": (_c_size_t, [_c_int, _c_int, _c_int]),
    "bakron_pack4": (_c_int, [_vp, _i64, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "bakron_unpack4": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _i64, _vp, _vp]),
    "bakron_matvec4": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _c_int, _i64, _vp,
                                _c_int, _c_int, _vp, _c_int, _i64, _vp]),
    "bakron_rms_norm_q8": (_c_int, [_vp, _i64, _vp, _i64, _c_int, _vp, _c_int, _c_int, _c_int,
                                    ctypes.c_float, _c_int, _vp, _vp, _vp, _i64, _vp, _vp]),
    "bakron_distill": (_c_int, [_vp, _c_int, _c_int, _c_int, _i64, _vp, _c_int, _vp, _c_int,
                                _c_int, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _i64, _vp, _vp]),
    "bakron_read_status": (_c_int, [_vp, _vp]),
    "bakron_status_string": (ctypes.c_char_p, [_c_int]),
    "bakron_version": (_c_int, []),
    "bakron_kernel_launches": (ctypes.c_ulonglong, []),
    "bakron_ldl_noalloc": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp]),
    "bakron_ldl_noalloc_max_n": (_c_int, []),
    # test hooks (include/bakron_internal.h)
    "bakron_internal_gemm3x_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int]),
    "bakron_internal_gemm3x": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _c_int, _c_int, _vp,
                                        _c_int, _vp, _c_size_t, _vp, _vp]),
    "bakron_internal_proxy_loss_simt_workspace_bytes": (_c_size_t, [_c_int, _c_int]),
    "bakron_internal_hadamard28": (None, [_vp]),
    "bakron_internal_matvec4_plan": (_c_int, [_c_int] * 9 + [_vp]),
    "bakron_internal_proxy_loss_simt": (_c_int, [_vp, _c_int, _c_int, _vp, _vp, _vp, _vp,
                                                 _c_size_t, _vp]),
}

_lib: Optional[ctypes.CDLL] = None


class BakronError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} ({code})")
        self.code = code


def header_functions(path: str = HEADER_PATH) -> list[str]:
    """Names of the functions that a header (default include/bakron.h) declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bakron_\w+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """Loads libbakron.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m two_sided_adaptive_bakron_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().bakron_status_string(int(code)).decode()


bakron_status_string = status_string


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check_cuda(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")


# ----------------------------------------------------------------------------- C-ABI mirrors
def bakron_ldl_workspace_bytes(n: int) -> int:
    return int(lib().bakron_ldl_workspace_bytes(int(n)))


def bakron_round_workspace_bytes(m: int, n: int) -> int:
    return int(lib().bakron_round_workspace_bytes(int(m), int(n)))


def bakron_proxy_loss_workspace_bytes(m: int, n: int) -> int:
    return int(lib().bakron_proxy_loss_workspace_bytes(int(m), int(n)))


def bakron_ldl(H, L, D, ws, dev_status, stream=None) -> int:
    n = H.shape[0]
    _check_cuda(H, torch.float32, (n, n), "H")
    _check_cuda(L, torch.float32, (n, n), "L")
    _check_cuda(D, torch.float32, (n,), "D")
    return lib().bakron_ldl(_ptr(H), n, _ptr(L), _ptr(D), _ptr(ws), ws.numel() * ws.element_size(),
                            _ptr(dev_status), _stream(stream))


def bakron_round(Wstar, L_O, L_I, scales, bits, codes, W, ws, dev_status, stream=None) -> int:
    m, n = Wstar.shape
    _check_cuda(Wstar, torch.float32, (m, n), "Wstar")
    _check_cuda(L_O, torch.float32, (m, m), "L_O")
    _check_cuda(L_I, torch.float32, (n, n), "L_I")
    _check_cuda(scales, torch.float32, (m,), "scales")
    _check_cuda(codes, torch.int8, (m, n), "codes")
    _check_cuda(W, torch.float32, (m, n), "W")
    return lib().bakron_round(_ptr(Wstar), m, n, _ptr(L_O), _ptr(L_I), _ptr(scales), int(bits),
                              _ptr(codes), _ptr(W), _ptr(ws), ws.numel() * ws.element_size(),
                              _ptr(dev_status), _stream(stream))


def bakron_round_stochastic(Wstar, L_O, L_I, scales, bits, seed, codes, W, ws, dev_status,
                            stream=None) -> int:
    m, n = Wstar.shape
    _check_cuda(Wstar, torch.float32, (m, n), "Wstar")
    _check_cuda(L_O, torch.float32, (m, m), "L_O")
    _check_cuda(L_I, torch.float32, (n, n), "L_I")
    _check_cuda(scales, torch.float32, (m,), "scales")
    _check_cuda(codes, torch.int8, (m, n), "codes")
    _check_cuda(W, torch.float32, (m, n), "W")
    return lib().bakron_round_stochastic(_ptr(Wstar), m, n, _ptr(L_O), _ptr(L_I), _ptr(scales),
                                         int(bits), int(seed) & ((1 << 64) - 1), _ptr(codes),
                                         _ptr(W), _ptr(ws), ws.numel() * ws.element_size(),
                                         _ptr(dev_status), _stream(stream))


def bakron_round_ex(Wstar, L_O, L_I, scales, group_size, codebook, bits, codes, W, ws,
                    dev_status, stream=None) -> int:
    """``scales``: m x G device tensor (G = ceil(n / group_size)); ``codebook``: None or a
    host sequence of 2^bits increasing floats (copied by the call)."""
    m, n = Wstar.shape
    _check_cuda(Wstar, torch.float32, (m, n), "Wstar")
    _check_cuda(L_O, torch.float32, (m, m), "L_O")
    _check_cuda(L_I, torch.float32, (n, n), "L_I")
    gs = min(int(group_size), n)
    _check_cuda(scales, torch.float32, (m, (n + gs - 1) // gs), "scales")
    _check_cuda(codes, torch.int8, (m, n), "codes")
    _check_cuda(W, torch.float32, (m, n), "W")
    cb = None
    if codebook is not None:
        vals = [float(v) for v in codebook]
        cb = (ctypes.c_float * len(vals))(*vals)
    return lib().bakron_round_ex(_ptr(Wstar), m, n, _ptr(L_O), _ptr(L_I), _ptr(scales),
                                 int(group_size), cb, int(bits), _ptr(codes), _ptr(W), _ptr(ws),
                                 ws.numel() * ws.element_size(), _ptr(dev_status),
                                 _stream(stream))


def bakron_proxy_loss(dW, H_O, H_I, loss, ws, stream=None) -> int:
    m, n = dW.shape
    _check_cuda(dW, torch.float32, (m, n), "dW")
    _check_cuda(H_O, torch.float32, (m, m), "H_O")
    _check_cuda(H_I, torch.float32, (n, n), "H_I")
    _check_cuda(loss, torch.float64, (1,), "loss")
    return lib().bakron_proxy_loss(_ptr(dW), m, n, _ptr(H_O), _ptr(H_I), _ptr(loss), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream))


def bakron_damped_gram_workspace_bytes(N: int, d: int) -> int:
    return int(lib().bakron_damped_gram_workspace_bytes(int(N), int(d)))


def bakron_sketch_b_workspace_bytes(S: int, m: int, n: int) -> int:
    return int(lib().bakron_sketch_b_workspace_bytes(int(S), int(m), int(n)))


def bakron_damped_gram(X, damp, H, ws, dev_status, stream=None) -> int:
    N, d = X.shape
    _check_cuda(X, torch.float32, (N, d), "X")
    _check_cuda(H, torch.float32, (d, d), "H")
    return lib().bakron_damped_gram(_ptr(X), N, d, float(damp), _ptr(H), _ptr(ws),
                                    ws.numel() * ws.element_size(), _ptr(dev_status),
                                    _stream(stream))


def bakron_sketch_b(G, damp, H_O, H_I, ws, dev_status, stream=None) -> int:
    S, m, n = G.shape
    _check_cuda(G, torch.float32, (S, m, n), "G")
    _check_cuda(H_O, torch.float32, (m, m), "H_O")
    _check_cuda(H_I, torch.float32, (n, n), "H_I")
    return lib().bakron_sketch_b(_ptr(G), S, m, n, float(damp), _ptr(H_O), _ptr(H_I), _ptr(ws),
                                 ws.numel() * ws.element_size(), _ptr(dev_status),
                                 _stream(stream))


def bakron_rht_supported(d: int) -> bool:
    return bool(lib().bakron_rht_supported(int(d)))


def bakron_rht_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().bakron_rht_workspace_bytes(int(rows), int(cols)))


def bakron_rht(X, seed_rows, seed_cols, inverse, Y, ws, stream=None) -> int:
    r, c = X.shape
    _check_cuda(X, torch.float32, (r, c), "X")
    _check_cuda(Y, torch.float32, (r, c), "Y")
    m64 = (1 << 64) - 1
    return lib().bakron_rht(_ptr(X), r, c, int(seed_rows) & m64, int(seed_cols) & m64,
                            int(bool(inverse)), _ptr(Y), _ptr(ws), ws.numel() * ws.element_size(),
                            _stream(stream))


def bakron_row_scales(W, group_size, divisor, scales, stream=None) -> int:
    m, n = W.shape
    _check_cuda(W, torch.float32, (m, n), "W")
    g = min(int(group_size), n)
    _check_cuda(scales, torch.float32, (m, (n + g - 1) // g), "scales")
    return lib().bakron_row_scales(_ptr(W), m, n, int(group_size), float(divisor), _ptr(scales),
                                   _stream(stream))


# The entry points below are called once a layer and token, so their binding is kept short: sizes
# and strides are read once, the library checks them, and only what it cannot see (device, type,
# a strided last dimension, the length of a buffer) is checked here.
def _rows(t: torch.Tensor, name: str, device: int):
    """(rows, columns, row stride) of a 1-D or 2-D tensor on ``device`` whose last stride is 1."""
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{device}" if device >= 0
                                                            else ""))
    dim = t.dim()
    if dim == 2:
        r, c = t.shape
        ld, inner = t.stride()
        if r <= 1:
            ld = c
        if (c > 1 and inner != 1) or ld < c:
            raise ValueError(f"{name}: expected rows of stride-1 elements that do not overlap, got "
                             f"strides {tuple(t.stride())}")
        return r, c, ld
    if dim != 1:
        raise ValueError(f"{name}: expected one or two dimensions, got {tuple(t.shape)}")
    c = t.shape[0]
    if c > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: expected stride-1 elements, got {tuple(t.stride())}")
    return 1, c, c


def _flat(t, dtype, numel: int, name: str, device: int) -> int:
    """Data pointer of a contiguous tensor of a given type and length on ``device``."""
    if t.dtype != dtype or t.numel() != numel or t.get_device() != device or \
            not t.is_contiguous():
        raise ValueError(f"{name}: expected {numel} contiguous {dtype} on cuda:{device}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} on "
                         f"{t.device}")
    return t.data_ptr()


def _grid(t, dtype, rows: int, cols: int, name: str, device: int) -> int:
    """The same for rows x cols elements: neither a transposed tensor nor rows cut otherwise."""
    if t.dim() > 1 and rows > 1 and cols > 1 and t.shape[0] != rows and t.shape[-1] != cols:
        raise ValueError(f"{name}: expected {rows} x {cols}, got {tuple(t.shape)}")
    return _flat(t, dtype, rows * cols, name, device)


def _dtype(t: torch.Tensor, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name}: unsupported type {t.dtype}")
    return d


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _empty(rows, cols: int, dtype, device) -> torch.Tensor:
    """A new rows x cols tensor, or cols without rows (the shortest way torch has to one)."""
    if rows is None:
        return torch.empty_strided((cols,), (1,), dtype=dtype, device=device)
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _call(fn, device: int, stream, *args) -> int:
    """fn(*args, stream) with ``device`` current: the library launches on the current device."""
    if device == torch.cuda.current_device():
        return fn(*args, _raw_stream(device) if stream is None else _stream(stream))
    with torch.cuda.device(device):
        return fn(*args, _raw_stream(device) if stream is None else _stream(stream))


def _steps(n: int, group_size) -> tuple[int, int]:
    """(columns per step, steps per row); None is one step per row."""
    if group_size is None:
        return n, 1
    g = int(group_size)
    if g < 1:
        raise ValueError(f"group_size must be positive, got {group_size}")
    return g, (1 if g >= n else -(-n // g))


def _packed_bytes(m: int, n: int, G: int) -> int:
    """bakron_pack4_bytes for G steps a row, without a call (and without its refusals)."""
    mt = (m + 15) // 16
    return mt * ((n + 63) // 64) * 512 + mt * G * 64


def _codebook(codebook):
    """(ctypes array or None, bits) of a host codebook of 2, 4, 8 or 16 entries."""
    if codebook is None:
        return None, 0
    if not isinstance(codebook, ctypes.Array):
        codebook = (ctypes.c_float * len(codebook))(*codebook)
    bits = len(codebook).bit_length() - 1
    if len(codebook) != 1 << bits or not 1 <= bits <= 4:
        raise ValueError(f"a codebook has 2, 4, 8 or 16 entries, got {len(codebook)}")
    return codebook, bits


def bakron_pack4_bytes(m: int, n: int, group_size: int) -> int:
    return int(lib().bakron_pack4_bytes(int(m), int(n), int(group_size)))


def bakron_pack4(codes, scales, group_size, unsigned_codes, packed, dev_status,
                 stream=None) -> int:
    dev = codes.get_device()
    m, n, ldc = _rows(codes, "codes", dev)
    if codes.dtype != torch.int8:
        raise ValueError(f"codes: expected torch.int8, got {codes.dtype}")
    g, G = _steps(n, group_size)
    return _call(lib().bakron_pack4, dev, stream, codes.data_ptr(), ldc,
                 _grid(scales, torch.float32, m, G, "scales", dev), m, n, g,
                 int(bool(unsigned_codes)),
                 _flat(packed, torch.uint8, _packed_bytes(m, n, G), "packed", dev),
                 _flat(dev_status, torch.int32, 1, "dev_status", dev))


def bakron_unpack4(packed, group_size, unsigned_codes, codes, scales, stream=None) -> int:
    dev = codes.get_device()
    m, n, ldc = _rows(codes, "codes", dev)
    if codes.dtype != torch.int8:
        raise ValueError(f"codes: expected torch.int8, got {codes.dtype}")
    g, G = _steps(n, group_size)
    return _call(lib().bakron_unpack4, dev, stream,
                 _flat(packed, torch.uint8, _packed_bytes(m, n, G), "packed", dev), m, n, g,
                 int(bool(unsigned_codes)), codes.data_ptr(), ldc,
                 _grid(scales, torch.float32, m, G, "scales", dev))


def bakron_matvec4(packed, group_size, codebook, x, x_scales, x_group_size, y,
                   stream=None) -> int:
    """``x``: tokens x n (or n), ``y``: tokens x m (or m); ``codebook``: None, a sequence or a
    ctypes float array."""
    dev = x.get_device()
    rows, m, ldy = _rows(y, "y", dev)
    if rows != (1 if x.dim() == 1 else x.shape[0]):
        raise ValueError(f"y: expected the rows of x, got {tuple(y.shape)}")
    return _matvec4(packed, m, group_size, codebook, x, x_scales, x_group_size, y, ldy, dev, stream)


def _matvec4(packed, m, group_size, codebook, x, x_scales, x_group_size, y, ldy, dev, stream):
    """bakron_matvec4 for a y that is known to have the rows of x, m columns and stride ldy."""
    tokens, n, ldx = _rows(x, "x", dev)
    g, G = _steps(n, group_size)
    cb, bits = (None, 0) if codebook is None else _codebook(codebook)
    gx, xs = n, None
    if x_scales is not None:
        gx, Gx = _steps(n, x_group_size)
        xs = _grid(x_scales, torch.float32, tokens, Gx, "x_scales", dev)
    return _call(lib().bakron_matvec4, dev, stream,
                 _flat(packed, torch.uint8, _packed_bytes(m, n, G), "packed", dev), m, n, g, cb,
                 bits, x.data_ptr(), _dtype(x, "x"), ldx, xs, gx, tokens, y.data_ptr(),
                 _dtype(y, "y"), ldy)


def bakron_rms_norm_q8(x, residual, weight, eps, group_size, q, scales, sum_out=None,
                       dev_status=None, stream=None) -> int:
    dev = x.get_device()
    rows, n, _ = _rows(x, "x", dev)
    _, G = _steps(n, group_size)
    lds = 0
    if sum_out is not None:
        sr, sn, lds = _rows(sum_out, "sum_out", dev)
        if sr != rows or sn != n or sum_out.dtype != x.dtype:
            raise ValueError("sum_out: expected the shape and type of x")
    _grid(q, torch.int8, rows, n, "q", dev)
    _grid(scales, torch.float32, rows, G, "scales", dev)
    return _rms_norm_q8(x, residual, weight, eps, group_size, q, scales, sum_out, lds, dev_status,
                        dev, stream)


def _rms_norm_q8(x, residual, weight, eps, group_size, q, scales, sum_out, lds, dev_status, dev,
                 stream):
    """bakron_rms_norm_q8 for outputs that are known to fit."""
    rows, n, ldx = _rows(x, "x", dev)
    dt = x.dtype
    ldr = wd = 0
    rp = wp = None
    if residual is not None:
        rr, rn, ldr = _rows(residual, "residual", dev)
        if rr != rows or rn != n or residual.dtype != dt:
            raise ValueError("residual: expected the shape and type of x")
        rp = residual.data_ptr()
    if weight is not None:
        wd = _dtype(weight, "weight")
        wp = _flat(weight, weight.dtype, n, "weight", dev)
    return _call(lib().bakron_rms_norm_q8, dev, stream, x.data_ptr(), ldx, rp, ldr,
                 _dtype(x, "x"), wp, wd, rows, n, eps, n if group_size is None else group_size,
                 q.data_ptr(), scales.data_ptr(),
                 None if sum_out is None else sum_out.data_ptr(), lds,
                 None if dev_status is None else
                 _flat(dev_status, torch.int32, 1, "dev_status", dev))


def bakron_distill(logits, top_idx, top_logits, teacher_lse, row_weights, temperature, loss, lse,
                   dlogits, dev_status, stream=None) -> int:
    dev = logits.get_device()
    rows, V, _ = _rows(logits, "logits", dev)
    ldd = 0
    if dlogits is not None:
        dr, dv, ldd = _rows(dlogits, "dlogits", dev)
        if dr != rows or dv != V or dlogits.dtype != logits.dtype:
            raise ValueError("dlogits: expected the shape and type of logits")
    _flat(loss, torch.float32, rows, "loss", dev)
    _flat(lse, torch.float32, rows, "lse", dev)
    return _distill(logits, top_idx, top_logits, teacher_lse, row_weights, temperature, loss, lse,
                    dlogits, ldd, dev_status, dev, stream)


def _distill(logits, top_idx, top_logits, teacher_lse, row_weights, temperature, loss, lse, dlogits,
             ldd, dev_status, dev, stream):
    """bakron_distill for outputs that are known to fit."""
    rows, V, ld = _rows(logits, "logits", dev)
    k = top_idx.shape[-1]
    return _call(lib().bakron_distill, dev, stream, logits.data_ptr(), _dtype(logits, "logits"),
                 rows, V, ld, _grid(top_idx, top_idx.dtype, rows, k, "top_idx", dev),
                 _dtype(top_idx, "top_idx"),
                 _grid(top_logits, top_logits.dtype, rows, k, "top_logits", dev),
                 _dtype(top_logits, "top_logits"), k,
                 None if teacher_lse is None else
                 _flat(teacher_lse, torch.float32, rows, "teacher_lse", dev),
                 None if row_weights is None else
                 _flat(row_weights, torch.float32, rows, "row_weights", dev),
                 temperature, loss.data_ptr(), lse.data_ptr(),
                 None if dlogits is None else dlogits.data_ptr(), ldd,
                 _flat(dev_status, torch.int32, 1, "dev_status", dev))


def internal_matvec4_plan(m, n, x_dtype, group_size=None, x_group_size=None, out_dtype=None,
                          book=False, tokens=1, sms=148):
    """How bakron_matvec4 cuts a call on a GPU of ``sms`` SMs (host only), as a dict; None where it
    refuses one."""
    out = (ctypes.c_int64 * 8)()
    g, _ = _steps(n, group_size)
    gx, _ = _steps(n, x_group_size)
    if out_dtype is None:
        out_dtype = torch.float32 if x_dtype == torch.int8 else x_dtype
    if lib().bakron_internal_matvec4_plan(m, n, g, _DTYPES[x_dtype], gx, _DTYPES[out_dtype],
                                          int(book), tokens, sms, out):
        return None
    return dict(zip(("smem", "cluster", "slice", "chunk", "clusters", "max_tiles", "product_tiles",
                     "warps"), out))


def internal_hadamard28():
    """The order-28 Hadamard matrix the library's transform uses (host construction)."""
    import numpy as np
    buf = (ctypes.c_byte * 784)()
    lib().bakron_internal_hadamard28(buf)
    return np.frombuffer(bytes(buf), dtype=np.int8).reshape(28, 28).copy()


def bakron_ldl_noalloc(H, L, D, dev_status, stream=None) -> int:
    """bakron_ldl with the library's own fixed scratch (no workspace argument)."""
    n = H.shape[0]
    _check_cuda(H, torch.float32, (n, n), "H")
    _check_cuda(L, torch.float32, (n, n), "L")
    _check_cuda(D, torch.float32, (n,), "D")
    return lib().bakron_ldl_noalloc(_ptr(H), n, _ptr(L), _ptr(D), _ptr(dev_status),
                                    _stream(stream))


def bakron_ldl_noalloc_max_n() -> int:
    return int(lib().bakron_ldl_noalloc_max_n())


def bakron_read_status(dev_status, stream=None) -> int:
    return int(lib().bakron_read_status(_ptr(dev_status), _stream(stream)))


def bakron_kernel_launches() -> int:
    return int(lib().bakron_kernel_launches())


def bakron_version() -> int:
    return int(lib().bakron_version())


def internal_gemm3x(A: torch.Tensor, B: torch.Tensor, stream=None) -> torch.Tensor:
    """C = A B^T through the 3xTF32 tensor-core engine (test hook)."""
    M, K = A.shape
    N = B.shape[0]
    C = torch.empty((M, N), dtype=torch.float32, device=A.device)
    ws = workspace(int(lib().bakron_internal_gemm3x_workspace_bytes(M, N, K)), A.device)
    st = new_status(A.device)
    _raise(lib().bakron_internal_gemm3x(_ptr(A), M, K, A.stride(0), _ptr(B), N, B.stride(0),
                                        _ptr(C), N, _ptr(ws), ws.numel(), _ptr(st),
                                        _stream(stream)), "bakron_internal_gemm3x")
    _raise(bakron_read_status(st, stream), "bakron_internal_gemm3x (device)")
    return C


def internal_proxy_loss_simt(dW, H_O, H_I, stream=None) -> torch.Tensor:
    """The CUDA-core proxy loss (test hook, cross-check of bakron_proxy_loss)."""
    m, n = dW.shape
    loss = torch.empty((1,), dtype=torch.float64, device=dW.device)
    ws = workspace(int(lib().bakron_internal_proxy_loss_simt_workspace_bytes(m, n)), dW.device)
    _raise(lib().bakron_internal_proxy_loss_simt(_ptr(dW), m, n, _ptr(H_O), _ptr(H_I),
                                                 _ptr(loss), _ptr(ws), ws.numel(),
                                                 _stream(stream)), "proxy_loss_simt")
    return loss


# ----------------------------------------------------------------------------- conveniences
def workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte aligned byte buffer (torch's caching allocator aligns to 512 bytes)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def new_status(device) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def _raise(code: int, where: str):
    if code != BAKRON_OK:
        raise BakronError(code, where)


def ldl(H: torch.Tensor, stream=None, check: bool = True):
    """(L, D) with H = (I + L) diag(D) (I + L)^T, L strictly upper."""
    n = H.shape[0]
    L = torch.empty((n, n), dtype=torch.float32, device=H.device)
    D = torch.empty((n,), dtype=torch.float32, device=H.device)
    ws = workspace(bakron_ldl_workspace_bytes(n), H.device)
    st = new_status(H.device)
    _raise(bakron_ldl(H, L, D, ws, st, stream), "bakron_ldl")
    if check:
        _raise(bakron_read_status(st, stream), "bakron_ldl (device)")
    return L, D


def round_weights(Wstar, L_O, L_I, scales, bits, stream=None, check: bool = True, seed=None,
                  group_size=None, codebook=None):
    """(codes int8, W fp32) of the BaKron solve; a seed selects stochastic Q, a group size
    (with m x G scales) and/or a host codebook select the base quantizer of bakron_round_ex."""
    m, n = Wstar.shape
    codes = torch.empty((m, n), dtype=torch.int8, device=Wstar.device)
    W = torch.empty((m, n), dtype=torch.float32, device=Wstar.device)
    ws = workspace(bakron_round_workspace_bytes(m, n), Wstar.device)
    st = new_status(Wstar.device)
    if group_size is not None or codebook is not None:
        if seed is not None:
            raise ValueError("stochastic Q takes the per-row integer grid")
        _raise(bakron_round_ex(Wstar, L_O, L_I, scales, n if group_size is None else group_size,
                               codebook, bits, codes, W, ws, st, stream), "bakron_round_ex")
    elif seed is None:
        _raise(bakron_round(Wstar, L_O, L_I, scales, bits, codes, W, ws, st, stream),
               "bakron_round")
    else:
        _raise(bakron_round_stochastic(Wstar, L_O, L_I, scales, bits, seed, codes, W, ws, st,
                                       stream), "bakron_round_stochastic")
    if check:
        _raise(bakron_read_status(st, stream), "bakron_round (device)")
    return codes, W


def damped_gram(X, damp: float = 0.01, stream=None, check: bool = True) -> torch.Tensor:
    """X^T X / N + damp * mean(diag) * I for samples X (N x d) on the device."""
    N, d = X.shape
    H = torch.empty((d, d), dtype=torch.float32, device=X.device)
    ws = workspace(bakron_damped_gram_workspace_bytes(N, d), X.device)
    st = new_status(X.device)
    _raise(bakron_damped_gram(X, damp, H, ws, st, stream), "bakron_damped_gram")
    if check:
        _raise(bakron_read_status(st, stream), "bakron_damped_gram (device)")
    return H


def sketch_b(G, damp: float = 0.01, stream=None, check: bool = True):
    """(H_O, H_I) of Sketch B from per-sequence gradients G (S x m x n) on the device."""
    S, m, n = G.shape
    H_O = torch.empty((m, m), dtype=torch.float32, device=G.device)
    H_I = torch.empty((n, n), dtype=torch.float32, device=G.device)
    ws = workspace(bakron_sketch_b_workspace_bytes(S, m, n), G.device)
    st = new_status(G.device)
    _raise(bakron_sketch_b(G, damp, H_O, H_I, ws, st, stream), "bakron_sketch_b")
    if check:
        _raise(bakron_read_status(st, stream), "bakron_sketch_b (device)")
    return H_O, H_I


def rht(X, seed_rows: int, seed_cols: int, inverse: bool = False, stream=None) -> torch.Tensor:
    """T_rows X T_cols^T (inverse: T_rows^T X T_cols) on the device (a new tensor)."""
    Y = torch.empty_like(X)
    ws = workspace(bakron_rht_workspace_bytes(*X.shape), X.device)
    _raise(bakron_rht(X, seed_rows, seed_cols, inverse, Y, ws, stream), "bakron_rht")
    return Y


def row_scales(W, divisor: float, group_size=None, stream=None) -> torch.Tensor:
    """max |W| over each row (and group of columns) / divisor, on the device."""
    m, n = W.shape
    g = n if group_size is None else min(int(group_size), n)
    out = torch.empty((m, (n + g - 1) // g), dtype=torch.float32, device=W.device)
    _raise(bakron_row_scales(W, g, divisor, out, stream), "bakron_row_scales")
    return out if group_size is not None else out.view(m)


def proxy_loss(dW, H_O, H_I, stream=None) -> torch.Tensor:
    """tr(H_O dW H_I dW^T) as a one-element float64 CUDA tensor."""
    m, n = dW.shape
    loss = torch.empty((1,), dtype=torch.float64, device=dW.device)
    ws = workspace(bakron_proxy_loss_workspace_bytes(m, n), dW.device)
    _raise(bakron_proxy_loss(dW, H_O, H_I, loss, ws, stream), "bakron_proxy_loss")
    return loss


def _stream_on(stream, device):
    """The torch stream of ``device`` that a Stream object or an integer handle names."""
    if hasattr(stream, "cuda_stream"):
        if device.type == "cuda" and stream.device != device:
            raise ValueError(f"stream: expected one of {device}, got one of {stream.device}")
        return stream
    if int(stream):
        return torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.default_stream(device)


def _on_stream(f):
    """Runs a call that is given a ``stream`` with that stream current: what it allocates then
    belongs to the stream that writes it, and nothing the current stream still uses is reused. A
    handle is one of the device that the call's first tensor is on."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        first = next((t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if first is None:
            raise ValueError("expected tensors")
        with torch.cuda.stream(_stream_on(stream, first.device)):
            return f(*args, **kw)
    return call


def _no_gradient(where: str):
    """The library has no gradient of these calls: an input that needs one is refused, where a result
    without history would drop it in silence."""
    if torch.is_grad_enabled():
        raise ValueError(f"{where}: an input requires a gradient, which this call does not pass on; call "
                         "it under torch.no_grad() or with detached inputs")


def _status_of(status, device, check: bool):
    """(status word, whether to read it): the caller's own word is left to the caller."""
    if status is not None:
        return status, False
    return new_status(device), check


@_on_stream
def pack4(codes, scales, group_size=None, unsigned: bool = False, check: bool = True,
          status=None) -> torch.Tensor:
    """The 4-bit layout of a layer's codes (m x n int8) and grid steps (m, or m x G with a
    group size); ``unsigned`` for codebook indices. With the caller's own ``status`` word the
    call does not wait for the device."""
    m, n = codes.shape
    _, G = _steps(n, group_size)
    device = codes.device
    packed = _empty(None, _packed_bytes(m, n, G), torch.uint8, device)
    st, read = _status_of(status, device, check)
    _raise(bakron_pack4(codes, scales, group_size, unsigned, packed, st), "bakron_pack4")
    if read:
        _raise(bakron_read_status(st, torch.cuda.current_stream(device)),
               "bakron_pack4 (device)")
    return packed


@_on_stream
def unpack4(packed, m: int, n: int, group_size=None, unsigned: bool = False):
    """(codes, scales) of a layer in the 4-bit layout; scales m, or m x G with a group size."""
    _, G = _steps(n, group_size)
    device = packed.device
    codes = _empty(m, n, torch.int8, device)
    scales = _empty(None if group_size is None else m, m if group_size is None else G, torch.float32,
                    device)
    _raise(bakron_unpack4(packed, group_size, unsigned, codes, scales), "bakron_unpack4")
    return codes, scales


@_on_stream
def matvec4(packed, m: int, n: int, x, group_size=None, codebook=None, x_scales=None,
            x_group_size=None, out_dtype=None) -> torch.Tensor:
    """y = x W^T for a layer (m x n) in the 4-bit layout and x of one token (n) or a few (tokens x
    n); y has x's type (float32 for int8 x) unless ``out_dtype`` names another. It has no gradient:
    an x that requires one is refused while gradients are recorded."""
    if x.requires_grad or (x_scales is not None and x_scales.requires_grad):
        _no_gradient("matvec4")
    shape = x.shape
    if shape[-1] != n:
        raise ValueError(f"x: expected {n} columns, got {tuple(shape)}")
    if out_dtype is None:
        out_dtype = torch.float32 if x.dtype == torch.int8 else x.dtype
    y = _empty(shape[0] if len(shape) == 2 else None, m, out_dtype, x.device)
    code = _matvec4(packed, m, group_size, codebook, x, x_scales, x_group_size, y, m,
                    x.get_device(), None)
    if code:
        raise BakronError(code, "bakron_matvec4")
    return y


@_on_stream
def rms_norm_q8(x, weight=None, eps: float = 1e-6, residual=None, group_size=None, sum_out=None,
                status=None):
    """(q int8, scales, sum): the norm of x + residual in 8 bits, and the sum in x's type (None
    without a residual, unless ``sum_out`` asks for it). Scales: one per row, or rows x G with a
    group size. Rows that are not finite give NaN scales and, where the caller gives a ``status``
    word, BAKRON_ERR_NONFINITE in it. It has no gradient: an x or residual that requires one is
    refused while gradients are recorded (``weight`` is taken as a constant)."""
    if x.requires_grad or (residual is not None and residual.requires_grad):
        _no_gradient("rms_norm_q8")
    shape = x.shape
    n = shape[-1]
    _, G = _steps(n, group_size)
    rows, device = shape[0] if len(shape) == 2 else None, x.device
    q = _empty(rows, n, torch.int8, device)
    scales = _empty(rows, G, torch.float32, device)
    if sum_out is not None:
        code = bakron_rms_norm_q8(x, residual, weight, eps, group_size, q, scales, sum_out, status)
    else:
        if residual is not None:
            sum_out = _empty(rows, n, x.dtype, device)
        code = _rms_norm_q8(x, residual, weight, eps, group_size, q, scales, sum_out, n,
                            status, x.get_device(), None)
    if code:
        raise BakronError(code, "bakron_rms_norm_q8")
    return q, scales, sum_out


@_on_stream
def distill(logits, top_idx, top_logits, temperature: float = 1.0, teacher_lse=None,
            row_weights=None, grad: bool = True, dlogits=None, check: bool = True, status=None):
    """(loss, lse, dlogits) of the distillation from a teacher's top logits: per-row weighted KL,
    the student's log-sum-exp of logits / temperature, and the gradient of the summed loss (None
    unless ``grad``; ``dlogits`` names its buffer, which may be ``logits``). With the caller's own
    ``status`` word the call does not wait for the device."""
    shape = logits.shape
    rows, device = 1 if len(shape) == 1 else shape[0], logits.device
    loss = _empty(None, rows, torch.float32, device)
    lse = _empty(None, rows, torch.float32, device)
    st, read = _status_of(status, device, check)
    if grad and dlogits is not None:
        code = bakron_distill(logits, top_idx, top_logits, teacher_lse, row_weights, temperature,
                              loss, lse, dlogits, st)
    else:
        dlogits = None
        if grad:
            dlogits = _empty(None if len(shape) == 1 else rows, shape[-1], logits.dtype, device)
        code = _distill(logits, top_idx, top_logits, teacher_lse, row_weights, temperature, loss,
                        lse, dlogits, shape[-1], st, logits.get_device(), None)
    if code:
        raise BakronError(code, "bakron_distill")
    if read:
        _raise(bakron_read_status(st, torch.cuda.current_stream(device)),
               "bakron_distill (device)")
    return loss, lse, dlogits


class PackedLayer:
    """A rounded layer kept in 4 bits: what ``Solver.run`` or ``round_weights`` left in ``codes``,
    with its grid steps and, where the round took one, its codebook.

        layer = bk.PackedLayer(codes, scales, group_size=128)
        y = layer.matvec(x)                           # x: n, or tokens x n
        y = layer.matvec(q, x_scales=s)               # the int8 output of rms_norm_q8
    """

    def __init__(self, codes, scales, group_size=None, codebook=None, stream=None):
        self.m, self.n = codes.shape
        self.group_size = group_size
        self.codebook, _ = _codebook(codebook)
        self.packed = pack4(codes, scales, group_size, codebook is not None, stream=stream)

    def matvec(self, x, x_scales=None, x_group_size=None, out_dtype=None, stream=None):
        return matvec4(self.packed, self.m, self.n, x, self.group_size, self.codebook, x_scales,
                       x_group_size, out_dtype, stream=stream)

    def unpack(self, stream=None):
        """(codes, scales) as they were given."""
        return unpack4(self.packed, self.m, self.n, self.group_size, self.codebook is not None,
                       stream=stream)


class Solver:
    """Reusable buffers for the whole path: ldl(H_O), ldl(H_I), round, proxy loss.

    The round workspace keeps E = W* - W at its start (see bakron.h), which is the dW handed
    to the proxy loss.
    """

    def __init__(self, m: int, n: int, device="cuda"):
        self.m, self.n, self.device = m, n, torch.device(device)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.L_O = torch.empty((m, m), **f32)
        self.D_O = torch.empty((m,), **f32)
        self.L_I = torch.empty((n, n), **f32)
        self.D_I = torch.empty((n,), **f32)
        self.codes = torch.empty((m, n), dtype=torch.int8, device=self.device)
        self.W = torch.empty((m, n), **f32)
        self.loss = torch.empty((1,), dtype=torch.float64, device=self.device)
        self.ws_round = workspace(bakron_round_workspace_bytes(m, n), self.device)
        self.ws_O = workspace(bakron_ldl_workspace_bytes(m), self.device)
        self.ws = workspace(max(bakron_ldl_workspace_bytes(n),
                                bakron_proxy_loss_workspace_bytes(m, n)), self.device)
        self.E = self.ws_round[: 4 * m * n].view(torch.float32).view(m, n)
        self._rot = None     # incoherence buffers, made on first use
        self._steps = None   # (scales, group_size, codebook) of the last run
        self.status = new_status(self.device)
        # the two factorisations are independent: ldl(H_O) runs on a side stream while
        # ldl(H_I) runs on the caller's stream
        self.side = torch.cuda.Stream(device=self.device)
        self._fork = torch.cuda.Event()
        self._join = torch.cuda.Event()

    def _rotated(self):
        if self._rot is None:
            m, n, dev = self.m, self.n, self.device
            f32 = dict(dtype=torch.float32, device=dev)
            self._rot = dict(W=torch.empty((m, n), **f32), HO=torch.empty((m, m), **f32),
                             HI=torch.empty((n, n), **f32), s=torch.empty((m, 1), **f32),
                             W_orig=torch.empty((m, n), **f32),
                             ws=workspace(max(bakron_rht_workspace_bytes(m, n),
                                              bakron_rht_workspace_bytes(m, m),
                                              bakron_rht_workspace_bytes(n, n)), dev))
        return self._rot

    def run(self, Wstar, H_O, H_I, scales, bits, stream=None, with_loss=True, timing=None,
            seed=None, group_size=None, codebook=None, incoherence=None):
        """Enqueues the whole path (reads: self.codes, self.W, self.E, self.loss); a seed
        selects stochastic Q for the round, a group size (with m x G scales) and/or a host
        codebook the base quantizer of bakron_round_ex.

        incoherence=(seed_o, seed_i) runs the path on the rotated layer (bakron_rht):
        W~ = T_m W* T_n^T, H_O~ = T_m H_O T_m^T, H_I~ = T_n H_I T_n^T, per-row grid steps of
        W~ (``scales`` is then ignored), and writes self.W_orig = T_m^T W~_q T_n. self.codes,
        self.W and self.E stay in the rotated basis, where the proxy loss is the same.

        timing: optional {name: (start_event, end_event)} for any of "ldl_O", "ldl_I", "round",
        "loss"; each pair is recorded around its call on the stream that runs it.
        """
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        timing = timing or {}
        if incoherence is not None:
            if group_size is not None or codebook is not None:
                raise ValueError("incoherence processing takes per-row integer-grid steps")
            so, si = incoherence
            R = self._rotated()
            ev = timing.get("rotate")
            if ev is not None:
                ev[0].record(stream)
            for X, Y, a, b in ((Wstar, R["W"], so, si), (H_O, R["HO"], so, so),
                               (H_I, R["HI"], si, si)):
                _raise(bakron_rht(X, a, b, False, Y, R["ws"], stream), "bakron_rht")
            _raise(bakron_row_scales(R["W"], self.n, (1 << (bits - 1)) - 0.5, R["s"], stream),
                   "bakron_row_scales")
            if ev is not None:
                ev[1].record(stream)
            Wstar, H_O, H_I, scales = R["W"], R["HO"], R["HI"], R["s"].view(self.m)

        def call(name, st, fn, *a):
            ev = timing.get(name)
            if ev is not None:
                ev[0].record(st)
            _raise(fn(*a, st), "bakron " + name)
            if ev is not None:
                ev[1].record(st)

        self._fork.record(stream)
        self.side.wait_event(self._fork)
        call("ldl_O", self.side, bakron_ldl, H_O, self.L_O, self.D_O, self.ws_O, self.status)
        call("ldl_I", stream, bakron_ldl, H_I, self.L_I, self.D_I, self.ws, self.status)
        self._join.record(self.side)
        stream.wait_event(self._join)
        if group_size is not None or codebook is not None:
            call("round", stream, bakron_round_ex, Wstar, self.L_O, self.L_I, scales,
                 self.n if group_size is None else group_size, codebook, bits, self.codes,
                 self.W, self.ws_round, self.status)
        elif seed is None:
            call("round", stream, bakron_round, Wstar, self.L_O, self.L_I, scales, bits,
                 self.codes, self.W, self.ws_round, self.status)
        else:
            call("round", stream, bakron_round_stochastic, Wstar, self.L_O, self.L_I, scales,
                 bits, seed, self.codes, self.W, self.ws_round, self.status)
        self._steps = (scales, group_size, codebook)
        if with_loss:
            call("loss", stream, bakron_proxy_loss, self.E, H_O, H_I, self.loss, self.ws)
        if incoherence is not None:
            R = self._rotated()
            ev = timing.get("unrotate")
            if ev is not None:
                ev[0].record(stream)
            _raise(bakron_rht(self.W, so, si, True, R["W_orig"], R["ws"], stream), "bakron_rht")
            if ev is not None:
                ev[1].record(stream)
            self.W_orig = R["W_orig"]

    def check(self, stream=None):
        _raise(bakron_read_status(self.status, stream), "bakron (device)")

    def packed(self, stream=None) -> PackedLayer:
        """The layer that the last ``run`` rounded, in 4 bits (for bits <= 4), with the grid steps,
        group size and codebook of that run (the tensors that it was given, as they are now). After a
        run with ``incoherence`` it is the rotated layer W~."""
        if self._steps is None:
            raise ValueError("no layer was rounded yet")
        return PackedLayer(self.codes, *self._steps, stream)


def solve(Wstar, H_O, H_I, scales, bits, stream=None, seed=None):
    """Whole path on device tensors: returns (codes, W, loss, (L_O, D_O), (L_I, D_I)); a seed
    selects stochastic Q."""
    s = Solver(Wstar.shape[0], Wstar.shape[1], Wstar.device)
    s.run(Wstar, H_O, H_I, scales, bits, stream, seed=seed)
    s.check(stream)
    return s.codes, s.W, s.loss, (s.L_O, s.D_O), (s.L_I, s.D_I)
