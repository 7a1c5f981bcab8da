"""Binding of the serving entry points (``include/gptq_serve.h``): the 8-bit block product and the
quantized cache.

Argument marshalling only, like the rest of the package, whose ``__init__`` exports these names. A
decode step makes these calls once per layer, so the checks are kept to what the C ABI cannot see
(types, shapes, devices); sizes, alignments and options are refused by the library itself.
"""
from __future__ import annotations

import ctypes

import torch

from . import GPTQ_BF16, GPTQ_F32, GptqError, _lib

GPTQ_F16 = 2
GPTQ_FP8_BLOCK = 128
GPTQ_CACHE_INT4, GPTQ_CACHE_INT8, GPTQ_CACHE_E4M3 = 0, 1, 2
GPTQ_CACHE_UNCLAIMED = 512
GPTQ_CACHE_CLEAR = 16

EXPORTED_SERVE = ("gptq_fp8_quantize", "gptq_fp8_matmul", "gptq_cache_write", "gptq_cache_read")

_DTYPES = {torch.bfloat16: GPTQ_BF16, torch.float32: GPTQ_F32, torch.float16: GPTQ_F16}
_E4M3, _F32, _U8 = torch.float8_e4m3fn, torch.float32, torch.uint8


def _bind():
    i, i64, p = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "gptq_fp8_quantize": [p, i, i64, i64, i64, i, p, i64, p, p],
        "gptq_fp8_matmul": [p, i64, p, p, i64, p, i64, i64, i64, p, i, i64, p],
        "gptq_cache_write": [p, i64, i64, p, i64, i64, i, i64, i, i, p, i64, i, i, p, p, p, p, p, p,
                             p, p],
        "gptq_cache_read": [p, i64, i64, i, i, i, i, p, p, p, p, p, p, p, i64, i64, p, i64, i64, i,
                            p],
    }
    out = []
    for name in EXPORTED_SERVE:
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = i, sig[name]
        out.append(fn)
    return out


_fp8_quantize, _fp8_matmul, _cache_write, _cache_read = _bind()


# The functions behind torch.cuda.current_device and current_stream, without the objects these make;
# a torch built without CUDA has neither, and no tensor there reaches them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream_of(stream, dev: int) -> int:
    """The handle of the stream to run on, for tensors of device ``dev`` (which the library takes to
    be the current one)."""
    if dev < 0 or dev != _current_device():
        raise ValueError(f"the tensors must be on the current device (a CUDA one), not on device {dev}")
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _devices_differ():
    raise ValueError("the tensors must all be on the current device")


def _want(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _code(t: torch.Tensor) -> int:
    c = _DTYPES.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return c


def _pitch(t: torch.Tensor, name: str) -> int:
    """Distance of the rows of a matrix whose columns are contiguous, in elements."""
    r, c = t.shape
    s, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError(f"{name}: the columns must be contiguous")
    if s < c:
        if r > 1:
            raise ValueError(f"{name}: the rows must not overlap")
        return c
    return s


def gptq_fp8_quantize(X: torch.Tensor, block_rows: int, codes: torch.Tensor, scales: torch.Tensor,
                      stream=None):
    """codes (e4m3, as X), scales (fp32) = X (rows x cols, bf16 / fp16 / fp32, any row pitch) in
    8-bit floating point with one scale per block of ``block_rows`` (1 or 128) x 128."""
    rows, cols = X.shape
    if codes.dtype is not _E4M3:
        raise TypeError(f"codes must be {_E4M3}, got {codes.dtype}")
    if scales.dtype is not _F32:
        raise TypeError(f"scales must be {_F32}, got {scales.dtype}")
    if codes.shape != (rows, cols):
        raise ValueError("codes must have the shape of X")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    if scales.shape != (-(-rows // block_rows), (cols + 127) >> 7) or not scales.is_contiguous():
        raise ValueError("scales must be contiguous, ceil(rows / block_rows) x ceil(cols / 128)")
    dev = X.get_device()
    if codes.get_device() != dev or scales.get_device() != dev:
        _devices_differ()
    st = _fp8_quantize(X.data_ptr(), _code(X), rows, cols, _pitch(X, "X"), block_rows,
                       codes.data_ptr(), _pitch(codes, "codes"), scales.data_ptr(),
                       _stream_of(stream, dev))
    if st:
        raise GptqError(st, "gptq_fp8_quantize")


def fp8_quantize(X: torch.Tensor, *, block_rows: int = 1):
    """``gptq_fp8_quantize`` with fresh outputs: (codes, scales). The rows of the codes start on
    16-byte boundaries, as ``gptq_fp8_matmul`` wants them."""
    rows, cols = X.shape
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    dtype, ldx, stream = _code(X), _pitch(X, "X"), _stream_of(None, X.get_device())
    dev = X.device
    pitch = (cols + 15) & -16
    kb = (cols + 127) >> 7
    codes = torch.empty_strided((rows, cols), (pitch, 1), dtype=_E4M3, device=dev)
    scales = torch.empty_strided((-(-rows // block_rows), kb), (kb, 1), dtype=_F32, device=dev)
    st = _fp8_quantize(X.data_ptr(), dtype, rows, cols, ldx, block_rows, codes.data_ptr(), pitch,
                       scales.data_ptr(), stream)
    if st:
        raise GptqError(st, "gptq_fp8_quantize")
    return codes, scales


def _bad_operands(A, sA, B, sB):
    """Raises for the first thing that is wrong with the operands of a product."""
    (m, k), (n, kn) = A.shape, B.shape
    kb = (k + 127) >> 7
    if A.dtype is not _E4M3 or B.dtype is not _E4M3:
        raise TypeError(f"A and B must be {_E4M3}")
    if sA.dtype is not _F32 or sB.dtype is not _F32:
        raise TypeError(f"sA and sB must be {_F32}")
    if kn != k:
        raise ValueError("A and B must have the same number of columns")
    if sA.shape != (m, kb) or not sA.is_contiguous():
        raise ValueError("sA must be contiguous, m x ceil(k / 128)")
    raise ValueError("sB must be contiguous, ceil(n / 128) x ceil(k / 128)")


def gptq_fp8_matmul(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                    Y: torch.Tensor, stream=None):
    """Y (m x n, bf16 / fp16 / fp32) = A B^T for e4m3 codes A (m x k, scales m x ceil(k / 128))
    and B (n x k, scales ceil(n / 128) x ceil(k / 128))."""
    m, k = A.shape
    n, kn = B.shape
    kb = (k + 127) >> 7
    if (A.dtype is not _E4M3 or B.dtype is not _E4M3 or sA.dtype is not _F32 or sB.dtype is not _F32
            or kn != k or sA.shape != (m, kb) or sB.shape != ((n + 127) >> 7, kb)
            or not sA.is_contiguous() or not sB.is_contiguous()):
        _bad_operands(A, sA, B, sB)
    if Y.shape != (m, n):
        raise ValueError("Y must be m x n")
    dev = A.get_device()
    if (sA.get_device() != dev or B.get_device() != dev or sB.get_device() != dev
            or Y.get_device() != dev):
        _devices_differ()
    st = _fp8_matmul(A.data_ptr(), _pitch(A, "A"), sA.data_ptr(), B.data_ptr(), _pitch(B, "B"),
                     sB.data_ptr(), m, n, k, Y.data_ptr(), _code(Y), _pitch(Y, "Y"),
                     _stream_of(stream, dev))
    if st:
        raise GptqError(st, "gptq_fp8_matmul")


def fp8_matmul(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, *,
               out_dtype=torch.bfloat16) -> torch.Tensor:
    """``gptq_fp8_matmul`` into a fresh m x n tensor of ``out_dtype``."""
    if out_dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {out_dtype}")
    m, n = A.shape[0], B.shape[0]
    Y = torch.empty_strided((m, n), (n, 1), dtype=out_dtype, device=A.device)
    gptq_fp8_matmul(A, sA, B, sB, Y)
    return Y


def _row_bytes(fmt: int, head_dim: int) -> int:
    return head_dim // 2 if fmt == GPTQ_CACHE_INT4 else head_dim


def _cache_plane(shape, meta, grid, dev, codes, scales, zeros):
    """Addresses of the codes, scales and zero-points of K or V, checked against the cache: `shape`
    of the codes and `meta` of the others."""
    if codes is None or scales is None or (grid and zeros is None):
        raise ValueError("the cache lacks an array for these rows")
    if codes.dtype is not _U8 or scales.dtype is not _F32:
        raise TypeError("codes must be uint8 and scales float32")
    if codes.shape != shape or not codes.is_contiguous():
        raise ValueError("codes must be contiguous, n_slots x heads x bytes of a head")
    if scales.shape != meta or not scales.is_contiguous():
        raise ValueError("scales must be contiguous, n_slots x heads x groups")
    if codes.get_device() != dev or scales.get_device() != dev:
        _devices_differ()
    if not grid:
        return codes.data_ptr(), scales.data_ptr(), None
    if zeros.dtype is not _U8:
        raise TypeError("zeros must be uint8")
    if zeros.shape != meta or not zeros.is_contiguous():
        raise ValueError("zeros must be contiguous and have the shape of scales")
    if zeros.get_device() != dev:
        _devices_differ()
    return codes.data_ptr(), scales.data_ptr(), zeros.data_ptr()


_NO_PLANE = (None, None, None)


def _cache_args(K, V, slots, fmt, group_size, codes_k, scales_k, zeros_k, codes_v, scales_v, zeros_v):
    """Checks what both cache calls take. Returns (device, slots of the cache, (tokens, heads,
    head_dim), address and strides of K, of V, addresses of the cache's arrays)."""
    t, h, d = K.shape
    if slots.dtype is not torch.int64:
        raise TypeError(f"slots must be {torch.int64}, got {slots.dtype}")
    if slots.shape != (t,) or not slots.is_contiguous():
        raise ValueError("slots must be one number per token")
    kt, kh, one = K.stride()
    if one != 1 and d > 1:
        raise ValueError("K: the values of a head must be contiguous")
    if codes_k is None:
        raise ValueError("the cache lacks an array for these rows")
    n = codes_k.shape[0]
    if group_size < 0 or (group_size and d % group_size):
        raise ValueError("group_size must divide head_dim")
    shape = (n, h, d >> 1 if fmt == GPTQ_CACHE_INT4 else d)
    meta = (n, h, d // group_size if group_size else 1)
    grid = fmt != GPTQ_CACHE_E4M3
    dev = K.get_device()
    if slots.get_device() != dev:
        _devices_differ()
    pk = _cache_plane(shape, meta, grid, dev, codes_k, scales_k, zeros_k)
    if V is None:
        return dev, n, (t, h, d), (K.data_ptr(), kt, kh), (None, 0, 0), pk + _NO_PLANE
    if V.shape != (t, h, d):
        raise ValueError("V must have the shape of K")
    if V.dtype is not K.dtype:
        raise TypeError(f"V must be {K.dtype}, got {V.dtype}")
    vt, vh, one = V.stride()
    if one != 1 and d > 1:
        raise ValueError("V: the values of a head must be contiguous")
    if V.get_device() != dev:
        _devices_differ()
    pv = _cache_plane(shape, meta, grid, dev, codes_v, scales_v, zeros_v)
    return dev, n, (t, h, d), (K.data_ptr(), kt, kh), (V.data_ptr(), vt, vh), pk + pv


def gptq_cache_write(K: torch.Tensor, V: torch.Tensor | None, slots: torch.Tensor, fmt: int,
                     group_size: int, codes_k: torch.Tensor, scales_k: torch.Tensor,
                     zeros_k: torch.Tensor | None, codes_v: torch.Tensor | None,
                     scales_v: torch.Tensor | None, zeros_v: torch.Tensor | None,
                     claims: torch.Tensor | None, stream=None):
    """Quantize rows of K and V (tokens x heads x head_dim) into ``slots`` of a cache. Negative
    slots skip their token; of tokens with the same slot the last one stays."""
    dev, n, thd, k, v, planes = _cache_args(K, V, slots, fmt, group_size, codes_k, scales_k, zeros_k,
                                            codes_v, scales_v, zeros_v)
    cp = None
    if claims is not None:
        if claims.dtype is not torch.int32:
            raise TypeError(f"claims must be {torch.int32}, got {claims.dtype}")
        if claims.shape != (n,) or not claims.is_contiguous():
            raise ValueError("claims must be one number per slot")
        if claims.get_device() != dev:
            _devices_differ()
        cp = claims.data_ptr()
    st = _cache_write(*k, *v, _code(K), *thd, slots.data_ptr(), n, fmt, group_size, *planes, cp,
                      _stream_of(stream, dev))
    if st:
        raise GptqError(st, "gptq_cache_write")


def gptq_cache_read(slots: torch.Tensor, fmt: int, group_size: int, codes_k: torch.Tensor,
                    scales_k: torch.Tensor, zeros_k: torch.Tensor | None,
                    codes_v: torch.Tensor | None, scales_v: torch.Tensor | None,
                    zeros_v: torch.Tensor | None, K: torch.Tensor, V: torch.Tensor | None,
                    stream=None):
    """K, V (tokens x heads x head_dim, written) = the values of the cache's ``slots``. Rows of
    negative slots are left as they are, or zero with ``fmt + GPTQ_CACHE_CLEAR``."""
    dev, n, (t, h, d), k, v, planes = _cache_args(K, V, slots, fmt & ~GPTQ_CACHE_CLEAR, group_size,
                                                  codes_k, scales_k, zeros_k, codes_v, scales_v,
                                                  zeros_v)
    st = _cache_read(slots.data_ptr(), t, n, h, d, fmt, group_size, *planes, *k, *v, _code(K),
                     _stream_of(stream, dev))
    if st:
        raise GptqError(st, "gptq_cache_read")


def kv_cache(n_slots: int, heads: int, head_dim: int, *, fmt: int = GPTQ_CACHE_INT8,
             group_size: int = 0, values: bool = True, device=None) -> dict:
    """An empty cache of keys and, with ``values``, of values: the arrays that ``cache_write`` and
    ``cache_read`` work on. Slot i of a paged cache is entry i % page of page i // page."""
    _want(fmt in (GPTQ_CACHE_INT4, GPTQ_CACHE_INT8, GPTQ_CACHE_E4M3), f"unknown format {fmt}")
    group = group_size or head_dim
    _want(head_dim > 0 and head_dim % 8 == 0 and 0 < group <= 1024 and group % 8 == 0
          and head_dim % group == 0, "head_dim and group_size must be multiples of 8, and groups "
                                     "of at most 1024 fill a head")
    _want(heads > 0 and heads * head_dim <= 65536, "heads must be positive and heads * head_dim at "
                                                   "most 65536")
    dev = "cuda" if device is None else device
    c = dict(fmt=fmt, group_size=group_size,
             claims=torch.zeros(n_slots, dtype=torch.int32, device=dev))
    for p in ("k", "v"):
        on = p == "k" or values
        c["codes_" + p] = torch.zeros(n_slots, heads, _row_bytes(fmt, head_dim), dtype=torch.uint8,
                                      device=dev) if on else None
        c["scales_" + p] = torch.zeros(n_slots, heads, head_dim // group, dtype=_F32,
                                       device=dev) if on else None
        c["zeros_" + p] = (torch.zeros(n_slots, heads, head_dim // group, dtype=torch.uint8,
                                       device=dev) if on and fmt != GPTQ_CACHE_E4M3 else None)
    return c


def cache_write(cache: dict, K: torch.Tensor, V: torch.Tensor | None, slots: torch.Tensor):
    """Quantize rows of K and V into ``slots`` of a ``kv_cache``."""
    c = cache
    gptq_cache_write(K, V, slots, c["fmt"], c["group_size"], c["codes_k"], c["scales_k"],
                     c["zeros_k"], c["codes_v"], c["scales_v"], c["zeros_v"], c["claims"])


def cache_read(cache: dict, slots: torch.Tensor, *, dtype=torch.bfloat16, out=None):
    """(K, V) of ``slots`` of a ``kv_cache`` (V None for a cache of keys only): in fresh tensors of
    ``dtype``, rows of negative slots zero, or in the two of ``out``, those rows left as they are."""
    c = cache
    fmt = c["fmt"]
    if out is None:
        if c["codes_k"] is None:
            raise ValueError("the cache lacks an array for these rows")
        n, heads, nbytes = c["codes_k"].shape
        dim = nbytes * 2 if fmt == GPTQ_CACHE_INT4 else nbytes
        out = [torch.empty((slots.shape[0], heads, dim), dtype=dtype, device=slots.device)
               if c["codes_" + p] is not None else None for p in ("k", "v")]
        fmt += GPTQ_CACHE_CLEAR
    K, V = out
    gptq_cache_read(slots, fmt, c["group_size"], c["codes_k"], c["scales_k"], c["zeros_k"],
                    c["codes_v"], c["scales_v"], c["zeros_v"], K, V)
    return K, V
