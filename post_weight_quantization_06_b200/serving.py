"""Binding of the serving entry points (``include/gptq_serve.h``): the 8-bit block product and the
quantized cache.

Argument marshalling only, like the rest of the package, whose ``__init__`` exports these names. A
decode step makes these calls once per layer, so the checks are kept to what the C ABI cannot see
(types, shapes, devices); sizes, alignments and options are refused by the library itself.
"""
from __future__ import annotations

import ctypes

import torch

from . import GPTQ_BF16, GPTQ_F32, GPTQ_OK, GptqError, _lib

GPTQ_F16 = 2
GPTQ_FP8_BLOCK = 128
GPTQ_CACHE_INT4, GPTQ_CACHE_INT8, GPTQ_CACHE_E4M3 = 0, 1, 2
GPTQ_CACHE_UNCLAIMED = 512

EXPORTED_SERVE = ("gptq_fp8_quantize", "gptq_fp8_matmul", "gptq_cache_write", "gptq_cache_read")

_DTYPES = {torch.bfloat16: GPTQ_BF16, torch.float32: GPTQ_F32, torch.float16: GPTQ_F16}
_E4M3 = torch.float8_e4m3fn


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


def _stream_of(stream, tensors) -> int:
    """The stream's handle; every tensor has to be on the current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}: the current device is cuda:{dev}")
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _want(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _typed(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _code(t: torch.Tensor) -> int:
    c = _DTYPES.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return c


def _check(st: int, where: str):
    if st != GPTQ_OK:
        raise GptqError(st, where)


def _rows(t: torch.Tensor, name: str) -> int:
    """Distance of the rows of a matrix whose columns are contiguous, in elements."""
    r, c = t.shape
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns must be contiguous")
    s = t.stride(0)
    if r > 1 and s < c:
        raise ValueError(f"{name}: the rows must not overlap")
    return s if s > c else c


def gptq_fp8_quantize(X: torch.Tensor, block_rows: int, codes: torch.Tensor, scales: torch.Tensor,
                      stream=None):
    """codes (e4m3, as X), scales (fp32) = X (rows x cols, bf16 / fp16 / fp32, any row pitch) in
    8-bit floating point with one scale per block of ``block_rows`` (1 or 128) x 128."""
    rows, cols = X.shape
    _typed(codes, _E4M3, "codes")
    _typed(scales, torch.float32, "scales")
    _want(codes.shape == X.shape, "codes must have the shape of X")
    _want(block_rows in (1, 128), "block_rows must be 1 or 128")
    _want(scales.shape == (-(-rows // block_rows), -(-cols // 128)) and scales.is_contiguous(),
          "scales must be contiguous, ceil(rows / block_rows) x ceil(cols / 128)")
    st = _stream_of(stream, (X, codes, scales))
    _check(_fp8_quantize(X.data_ptr(), _code(X), rows, cols, _rows(X, "X"), block_rows,
                         codes.data_ptr(), _rows(codes, "codes"), scales.data_ptr(), st),
           "gptq_fp8_quantize")


def fp8_quantize(X: torch.Tensor, *, block_rows: int = 1):
    """``gptq_fp8_quantize`` with fresh outputs: (codes, scales). The rows of the codes start on
    16-byte boundaries, as ``gptq_fp8_matmul`` wants them."""
    rows, cols = X.shape
    _want(block_rows in (1, 128), "block_rows must be 1 or 128")
    pitch = -(-cols // 16) * 16
    codes = torch.empty((rows, pitch), dtype=_E4M3, device=X.device)
    if pitch != cols:
        codes = codes[:, :cols]
    scales = torch.empty((-(-rows // block_rows), -(-cols // 128)), dtype=torch.float32,
                         device=X.device)
    gptq_fp8_quantize(X, block_rows, codes, scales)
    return codes, scales


def gptq_fp8_matmul(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                    Y: torch.Tensor, stream=None):
    """Y (m x n, bf16 / fp16 / fp32) = A B^T for e4m3 codes A (m x k, scales m x ceil(k / 128))
    and B (n x k, scales ceil(n / 128) x ceil(k / 128))."""
    m, k = A.shape
    n = B.shape[0]
    kb = -(-k // 128)
    _typed(A, _E4M3, "A")
    _typed(B, _E4M3, "B")
    _typed(sA, torch.float32, "sA")
    _typed(sB, torch.float32, "sB")
    _want(B.shape[1] == k, "A and B must have the same number of columns")
    _want(sA.shape == (m, kb) and sA.is_contiguous(), "sA must be contiguous, m x ceil(k / 128)")
    _want(sB.shape == (-(-n // 128), kb) and sB.is_contiguous(),
          "sB must be contiguous, ceil(n / 128) x ceil(k / 128)")
    _want(Y.shape == (m, n), "Y must be m x n")
    st = _stream_of(stream, (A, sA, B, sB, Y))
    _check(_fp8_matmul(A.data_ptr(), _rows(A, "A"), sA.data_ptr(), B.data_ptr(), _rows(B, "B"),
                       sB.data_ptr(), m, n, k, Y.data_ptr(), _code(Y), _rows(Y, "Y"), st),
           "gptq_fp8_matmul")


def fp8_matmul(A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor, *,
               out_dtype=torch.bfloat16) -> torch.Tensor:
    """``gptq_fp8_matmul`` into a fresh m x n tensor of ``out_dtype``."""
    Y = torch.empty((A.shape[0], B.shape[0]), dtype=out_dtype, device=A.device)
    gptq_fp8_matmul(A, sA, B, sB, Y)
    return Y


def _row_bytes(fmt: int, head_dim: int) -> int:
    return head_dim // 2 if fmt == GPTQ_CACHE_INT4 else head_dim


def _cache_arrays(n_slots, heads, head_dim, fmt, group_size, arrays, two):
    """Addresses of (codes, scales, zeros) of K and V, checked against the cache's shape."""
    _want(group_size >= 0 and head_dim % (group_size or 1) == 0, "group_size must divide head_dim")
    groups = head_dim // group_size if group_size else 1
    ptrs = []
    for i, (codes, scales, zeros) in enumerate((arrays[:3], arrays[3:])):
        if i == 1 and not two:
            ptrs += [None, None, None]
            continue
        _typed(codes, torch.uint8, "codes")
        _typed(scales, torch.float32, "scales")
        _want(codes.shape == (n_slots, heads, _row_bytes(fmt, head_dim)) and codes.is_contiguous(),
              "codes must be contiguous, n_slots x heads x bytes of a head")
        _want(scales.shape == (n_slots, heads, groups) and scales.is_contiguous(),
              "scales must be contiguous, n_slots x heads x groups")
        if fmt != GPTQ_CACHE_E4M3:
            _typed(zeros, torch.uint8, "zeros")
            _want(zeros.shape == scales.shape and zeros.is_contiguous(),
                  "zeros must be contiguous and have the shape of scales")
            ptrs += [codes.data_ptr(), scales.data_ptr(), zeros.data_ptr()]
        else:
            ptrs += [codes.data_ptr(), scales.data_ptr(), None]
    return ptrs


def _cache_values(K, V, slots):
    """(tokens, heads, head_dim) and the strides of K and V (tokens x heads x head_dim, the last
    axis contiguous)."""
    _typed(slots, torch.int64, "slots")
    t, h, d = K.shape
    _want(slots.shape == (t,) and slots.is_contiguous(), "slots must be one number per token")
    _want(d < 2 or K.stride(2) == 1, "K: the values of a head must be contiguous")
    if V is not None:
        _want(V.shape == K.shape, "V must have the shape of K")
        _typed(V, K.dtype, "V")
        _want(d < 2 or V.stride(2) == 1, "V: the values of a head must be contiguous")
        return t, h, d, K.stride(0), K.stride(1), V.data_ptr(), V.stride(0), V.stride(1)
    return t, h, d, K.stride(0), K.stride(1), None, 0, 0


def gptq_cache_write(K: torch.Tensor, V: torch.Tensor | None, slots: torch.Tensor, fmt: int,
                     group_size: int, codes_k: torch.Tensor, scales_k: torch.Tensor,
                     zeros_k: torch.Tensor | None, codes_v: torch.Tensor | None,
                     scales_v: torch.Tensor | None, zeros_v: torch.Tensor | None,
                     claims: torch.Tensor | None, stream=None):
    """Quantize rows of K and V (tokens x heads x head_dim) into ``slots`` of a cache. Negative
    slots skip their token; of tokens with the same slot the last one stays."""
    t, h, d, ks, kh, vp, vs, vh = _cache_values(K, V, slots)
    n = codes_k.shape[0]
    p = _cache_arrays(n, h, d, fmt, group_size, (codes_k, scales_k, zeros_k, codes_v, scales_v,
                                                 zeros_v), V is not None)
    if claims is not None:
        _typed(claims, torch.int32, "claims")
        _want(claims.shape == (n,) and claims.is_contiguous(), "claims must be one number per slot")
    on = [x for x in (K, V, slots, codes_k, scales_k, zeros_k, codes_v, scales_v, zeros_v, claims)
          if x is not None]
    st = _stream_of(stream, on)
    _check(_cache_write(K.data_ptr(), ks, kh, vp, vs, vh, _code(K), t, h, d, slots.data_ptr(), n, fmt,
                        group_size, *p, None if claims is None else claims.data_ptr(), st),
           "gptq_cache_write")


def gptq_cache_read(slots: torch.Tensor, fmt: int, group_size: int, codes_k: torch.Tensor,
                    scales_k: torch.Tensor, zeros_k: torch.Tensor | None,
                    codes_v: torch.Tensor | None, scales_v: torch.Tensor | None,
                    zeros_v: torch.Tensor | None, K: torch.Tensor, V: torch.Tensor | None,
                    stream=None):
    """K, V (tokens x heads x head_dim, written) = the values of the cache's ``slots``. Rows of
    negative slots are left as they are."""
    t, h, d, ks, kh, vp, vs, vh = _cache_values(K, V, slots)
    n = codes_k.shape[0]
    p = _cache_arrays(n, h, d, fmt, group_size, (codes_k, scales_k, zeros_k, codes_v, scales_v,
                                                 zeros_v), V is not None)
    on = [x for x in (K, V, slots, codes_k, scales_k, zeros_k, codes_v, scales_v, zeros_v)
          if x is not None]
    st = _stream_of(stream, on)
    _check(_cache_read(slots.data_ptr(), t, n, h, d, fmt, group_size, *p, K.data_ptr(), ks, kh, vp,
                       vs, vh, _code(K), st), "gptq_cache_read")


def kv_cache(n_slots: int, heads: int, head_dim: int, *, fmt: int = GPTQ_CACHE_INT8,
             group_size: int = 0, values: bool = True, device=None) -> dict:
    """An empty cache of keys and, with ``values``, of values: the arrays that ``cache_write`` and
    ``cache_read`` work on. Slot i of a paged cache is entry i % page of page i // page."""
    _want(fmt in (GPTQ_CACHE_INT4, GPTQ_CACHE_INT8, GPTQ_CACHE_E4M3), f"unknown format {fmt}")
    group = group_size or head_dim
    _want(head_dim > 0 and head_dim % 8 == 0 and 0 < group <= 1024 and group % 8 == 0
          and head_dim % group == 0, "head_dim and group_size must be multiples of 8, and groups "
                                     "of at most 1024 fill a head")
    dev = device or "cuda"
    c = dict(fmt=fmt, group_size=group_size,
             claims=torch.zeros(n_slots, dtype=torch.int32, device=dev))
    for p in ("k", "v"):
        on = p == "k" or values
        c["codes_" + p] = torch.zeros(n_slots, heads, _row_bytes(fmt, head_dim), dtype=torch.uint8,
                                      device=dev) if on else None
        c["scales_" + p] = torch.zeros(n_slots, heads, head_dim // group,
                                       device=dev) if on else None
        c["zeros_" + p] = (torch.zeros(n_slots, heads, head_dim // group, dtype=torch.uint8,
                                       device=dev) if on and fmt != GPTQ_CACHE_E4M3 else None)
    return c


def cache_write(cache: dict, K: torch.Tensor, V: torch.Tensor | None, slots: torch.Tensor):
    """Quantize rows of K and V into ``slots`` of a ``kv_cache``."""
    c = cache
    gptq_cache_write(K, V, slots, c["fmt"], c["group_size"], c["codes_k"], c["scales_k"],
                     c["zeros_k"], c["codes_v"], c["scales_v"], c["zeros_v"], c["claims"])


def cache_read(cache: dict, slots: torch.Tensor, *, dtype=torch.bfloat16):
    """(K, V) of ``slots`` of a ``kv_cache`` in fresh tensors (V None for a cache of keys only);
    rows of negative slots are zero."""
    c = cache
    n, heads, nbytes = c["codes_k"].shape
    dim = nbytes * 2 if c["fmt"] == GPTQ_CACHE_INT4 else nbytes
    out = [torch.zeros((slots.shape[0], heads, dim), dtype=dtype, device=slots.device)
           if c["codes_" + p] is not None else None for p in ("k", "v")]
    gptq_cache_read(slots, c["fmt"], c["group_size"], c["codes_k"], c["scales_k"], c["zeros_k"],
                    c["codes_v"], c["scales_v"], c["zeros_v"], *out)
    return tuple(out)
