"""Paged key/value cache: tensor-level calls (marshalling only).

    cache = KVCache.empty(num_pages, page_size, Hkv, d, torch.float8_e4m3fn)
    cache_write(cache, k_new, v_new, page_table, kv_lens, cu_q)      # each step's new rows
    out = sdpa_paged(q, cache, page_table, kv_lens, cu_q)            # their attention
    k, v = cache_read(cache, page_table, kv_lens, T=T)               # dense tensors for sdpa()

``page_table`` [B, max_pages], ``kv_lens`` [B] and ``cu_q`` [B + 1] are int32
CUDA tensors; the kernels read them in stream order, the host never does.
``kv_lens`` counts the new rows.  ``cu_q`` None means one new row per sequence.
``max_q`` bounds a sequence's new rows (default: all rows given); a bound close
to the truth lets ``sdpa_paged`` choose better.

Every step runs in the CUDA kernels behind ``include/sdpa.h``; see there for
the formats, the formulas and what the kernels check.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

from . import sdpa_strides_t

PAGED_AUTO, PAGED_EXACT, PAGED_DECODE, PAGED_TCGEN05 = 0, 1, 2, 3
PAGED_PATHS = {"auto": PAGED_AUTO, "exact": PAGED_EXACT, "decode": PAGED_DECODE, "tcgen05": PAGED_TCGEN05}
CACHE_F32, CACHE_BF16, CACHE_E4M3, CACHE_INT8 = 0, 1, 2, 3


_package = None


def _S():
    global _package
    if _package is None:
        import attention_sdpa_fwd_b200 as S
        _package = S
    return _package


class sdpa_rows_t(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class sdpa_cache_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("k_strides", sdpa_strides_t), ("v_strides", sdpa_strides_t),
                ("k_scale_strides", sdpa_strides_t), ("v_scale_strides", sdpa_strides_t)]


class sdpa_batch_t(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("kv_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("B", ctypes.c_int),
                ("total_q", ctypes.c_int), ("max_q", ctypes.c_int)]


_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


def bind(L) -> None:
    L.sdpa_cache_write.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp]
    L.sdpa_cache_read.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp]
    L.sdpa_fwd_paged.argtypes = [_vp] * 6 + [_i32, _i32, _f32, _i32, _f32, _vp, _vp, _i32, _vp, _i64, _vp]
    L.sdpa_fwd_paged_workspace.argtypes = [_vp] * 6 + [_i32] * 4
    for n in ("sdpa_cache_write", "sdpa_cache_read", "sdpa_fwd_paged"):
        getattr(L, n).restype = _i32
    L.sdpa_fwd_paged_workspace.restype = _i64


# ---------------------------------------------------------------------------
# Raw C-ABI calls (pointers are ints; cache, batch and strides are structures or None)
# ---------------------------------------------------------------------------
_byref = ctypes.byref


def _ref(x):
    return None if x is None else _byref(x)


def sdpa_cache_write(cache, batch, k, k_strides, v, v_strides, dtype, stream) -> int:
    return _S().lib().sdpa_cache_write(_ref(cache), _ref(batch), k, _ref(k_strides), v, _ref(v_strides), dtype, stream)


def sdpa_cache_read(cache, batch, k_out, k_strides, v_out, v_strides, dtype, T, stream) -> int:
    return _S().lib().sdpa_cache_read(_ref(cache), _ref(batch), k_out, _ref(k_strides), v_out, _ref(v_strides), dtype,
                                      T, stream)


def sdpa_fwd_paged(q, q_strides, cache, batch, out, out_strides, dtype, Hq, scale, window, softcap, slopes, lse, path,
                   workspace, workspace_bytes, stream) -> int:
    return _S().lib().sdpa_fwd_paged(q, _ref(q_strides), _ref(cache), _ref(batch), out, _ref(out_strides), dtype, Hq,
                                     scale, window, softcap, slopes, lse, path, workspace, workspace_bytes, stream)


def sdpa_fwd_paged_workspace(cache, batch, q, q_strides, out, out_strides, dtype, Hq, window, path) -> int:
    return _S().lib().sdpa_fwd_paged_workspace(_ref(cache), _ref(batch), q, _ref(q_strides), out, _ref(out_strides),
                                               dtype, Hq, window, path)


# ---------------------------------------------------------------------------
# Tensor level
# ---------------------------------------------------------------------------
def _cache_code(dtype) -> int:
    import torch
    codes = {torch.float32: CACHE_F32, torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3,
             torch.int8: CACHE_INT8}
    if dtype not in codes:
        raise TypeError(f"unsupported cache dtype {dtype}; use float32, bfloat16, float8_e4m3fn or int8")
    return codes[dtype]


class KVCache:
    """A pool of pages: ``k`` and ``v`` [num_pages, Hkv, page_size, d] CUDA
    tensors of one dtype with a contiguous last axis (any other strides: a pool
    laid out [num_pages, page_size, Hkv, d] is passed as its transpose(1, 2)).
    float8_e4m3fn and int8 pools also have float32 ``k_scale`` and ``v_scale``
    [num_pages, Hkv, page_size].  The tensors of a cache do not change."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        code = _cache_code(k.dtype)
        for t in (k, v):
            if t.dim() != 4 or t.shape != k.shape or t.dtype != k.dtype or t.device != k.device:
                raise ValueError("k and v must be [num_pages, Hkv, page_size, d] of one shape, dtype and device")
            if t.stride(3) != 1:
                raise ValueError("k and v must have a contiguous last axis")
        if code in (CACHE_E4M3, CACHE_INT8):
            for t in (k_scale, v_scale):
                if t is None or t.shape != k.shape[:3] or t.dtype != torch.float32 or t.device != k.device:
                    raise ValueError("an 8-bit cache needs float32 k_scale and v_scale [num_pages, Hkv, page_size]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only 8-bit caches have scales")
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self.Hkv, self.page_size, self.d = k.shape[1:]
        self.device = k.device
        c = sdpa_cache_t(k=k.data_ptr(), v=v.data_ptr(), dtype=code, num_pages=k.shape[0], Hkv=self.Hkv,
                         page_size=self.page_size, d=self.d, k_strides=_strides(k), v_strides=_strides(v))
        if k_scale is not None:
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.k_scale_strides, c.v_scale_strides = _strides(k_scale), _strides(v_scale)
        self._descriptor = c
        self._scratch = (None, 0)  # sizes of the last sdpa_paged and the bytes of scratch it asked for

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hkv: int, d: int, dtype, device="cuda") -> "KVCache":
        """A cache with uninitialised pages."""
        import torch
        new = lambda *shape, dt: torch.empty(shape, dtype=dt, device=device)
        k, v = (new(num_pages, Hkv, page_size, d, dt=dtype) for _ in range(2))
        if _cache_code(dtype) in (CACHE_E4M3, CACHE_INT8):
            return cls(k, v, *(new(num_pages, Hkv, page_size, dt=torch.float32) for _ in range(2)))
        return cls(k, v)

    def descriptor(self) -> sdpa_cache_t:
        """The C structure of the pool."""
        return self._descriptor


def _strides(t) -> sdpa_strides_t:
    """Of the first three axes; an axis of one element is never stepped, so it
    may carry any stride."""
    return sdpa_strides_t(*(max(1, s) if n == 1 else s for s, n in zip(t.stride()[:3], t.shape[:3])))


def _batch(cache: KVCache, page_table, kv_lens, cu_q, total_q: int, max_q: Optional[int]) -> sdpa_batch_t:
    import torch
    dev, i32 = cache.device, torch.int32
    for t, dim, name in ((page_table, 2, "page_table"), (kv_lens, 1, "kv_lens"), (cu_q, 1, "cu_q")):
        if t is None and name == "cu_q":
            continue
        if t.dtype != i32 or t.dim() != dim or t.device != dev:
            raise ValueError(f"{name} must be a {dim}-D int32 tensor on the cache's device")
        if not t.is_contiguous() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a contiguous last axis")
    B, width = kv_lens.shape[0], page_table.shape[1]
    if page_table.shape[0] != B or (cu_q is not None and cu_q.shape[0] != B + 1):
        raise ValueError("page_table must be [B, max_pages], kv_lens [B], cu_q [B + 1]")
    if cu_q is None and total_q != B:
        raise ValueError("without cu_q there is one new row per sequence")
    if max_q is None:
        max_q = total_q
    elif max_q < 0:
        raise ValueError("max_q must not be negative")
    return sdpa_batch_t(page_table.data_ptr(), page_table.stride(0) if B > 1 else width, width, kv_lens.data_ptr(),
                        None if cu_q is None else cu_q.data_ptr(), B, total_q, min(int(max_q), 0x7fffffff))


def _rows(t, heads: int, cache: KVCache, name: str) -> Optional[sdpa_rows_t]:
    """Strides of packed rows (None: dense), checked."""
    if t.device != cache.device or not t.is_cuda:
        raise ValueError(f"{name} must be on the cache's CUDA device (no CPU fallback)")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != cache.d:
        raise ValueError(f"{name} must be [tokens, {heads}, {cache.d}]")
    if t.is_contiguous():
        return None
    n, h, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return sdpa_rows_t(n if t.shape[0] > 1 else max(1, n), h if heads > 1 else max(1, h))


def _on(device, stream, call):
    """``call(handle)`` with the tensors' device, and the stream asked for,
    current: what a call allocates belongs to the stream its kernels run on.
    (By the current stream's handle where nothing has to change: the Stream
    object alone would cost more than a call's checks.)"""
    import torch
    if stream is None and torch.cuda.current_device() == device.index:
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return call((stream or torch.cuda.current_stream(device)).cuda_stream)


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise _S().SdpaError(rc, what)


def _need_cuda(cache: KVCache) -> None:
    if cache.device.type != "cuda":
        raise ValueError("the cache must be on a CUDA device (no CPU fallback)")


def cache_write(cache: KVCache, k, v, page_table, kv_lens, cu_q=None, *, max_q: Optional[int] = None,
                stream=None) -> KVCache:
    """Put new rows ``k``, ``v`` [total_q, Hkv, d] (float32 or bfloat16, any
    token / head strides) into their pages (sdpa_cache_write): the last rows of
    every sequence.  8-bit caches quantise them, one scale per row."""
    S = _S()
    _need_cuda(cache)
    ks, vs = _rows(k, cache.Hkv, cache, "k"), _rows(v, cache.Hkv, cache, "v")
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    batch = _batch(cache, page_table, kv_lens, cu_q, k.shape[0], max_q)
    _check(_on(cache.device, stream, lambda st: sdpa_cache_write(
        cache.descriptor(), batch, k.data_ptr(), ks, v.data_ptr(), vs, S._dtype_code(k), st)), "sdpa_cache_write")
    return cache


def cache_read(cache: KVCache, page_table, kv_lens, k_out=None, v_out=None, *, T: Optional[int] = None, dtype=None,
               stream=None):
    """Tokens 0 .. min(kv_lens[b], T) - 1 of every sequence as dense tensors
    [B, Hkv, T, d] (sdpa_cache_read), for ``sdpa``.  Outputs given are written
    in place, any strides, and keep their other rows; outputs made here (T
    required, bfloat16 unless the cache is float32) have zeros there."""
    import torch
    S = _S()
    _need_cuda(cache)
    B, Hkv, d = kv_lens.shape[0], cache.Hkv, cache.d
    if (k_out is None) != (v_out is None):
        raise ValueError("give both outputs or none")
    batch = _batch(cache, page_table, kv_lens, None, B, None)

    def call(st):
        nonlocal k_out, v_out, dtype
        if k_out is None:
            if T is None:
                raise ValueError("cache_read needs T or outputs")
            dtype = dtype or (torch.float32 if cache.k.dtype == torch.float32 else torch.bfloat16)
            k_out, v_out = (torch.zeros(B, Hkv, T, d, dtype=dtype, device=cache.device) for _ in range(2))
        for t in (k_out, v_out):
            if t.dim() != 4 or t.shape != k_out.shape or t.shape[0] != B or t.shape[1] != Hkv or t.shape[3] != d or \
                    t.stride(3) != 1 or t.dtype != k_out.dtype or t.device != cache.device:
                raise ValueError("outputs must be [B, Hkv, T, d] of one dtype with a contiguous last axis, on the cache's device")
        if T is not None and T != k_out.shape[2]:
            raise ValueError("T differs from the outputs given")
        if dtype is not None and dtype != k_out.dtype:
            raise ValueError("dtype differs from the outputs given")
        ks, vs = (None if t.is_contiguous() else _strides(t) for t in (k_out, v_out))
        return sdpa_cache_read(cache.descriptor(), batch, k_out.data_ptr(), ks, v_out.data_ptr(), vs,
                               S._dtype_code(k_out), k_out.shape[2], st)
    _check(_on(cache.device, stream, call), "sdpa_cache_read")
    return k_out, v_out


def sdpa_paged(q, cache: KVCache, page_table, kv_lens, cu_q=None, scale: Optional[float] = None, *,
               max_q: Optional[int] = None, window: int = 0, softcap: float = 0.0, slopes=None, out=None, lse=None,
               path: str = "auto", stream=None):
    """Attention of every sequence's new rows over its cache (sdpa_fwd_paged).

    ``q`` [total_q, Hq, d], float32 or bfloat16, any token / head strides;
    ``scale`` defaults to 1/sqrt(d).  A row sees its own token and those before
    it, ``window`` of them if positive.  ``softcap`` c caps scores to
    c tanh(x / c); ``slopes`` (float32 [Hq]) add slope (j - pos).  ``lse``, a
    float32 [total_q, Hq] tensor, receives the log-sum-exp.  Returns ``out``."""
    import torch
    S = _S()
    _need_cuda(cache)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, Hq, d]")
    T, Hq, d = q.shape
    qs = _rows(q, Hq, cache, "q")
    batch = _batch(cache, page_table, kv_lens, cu_q, T, max_q)
    dev = cache.device
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (Hq,) or not slopes.is_contiguous()
                               or slopes.device != dev):
        raise ValueError("slopes must be a contiguous float32 [Hq] tensor on the cache's device")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()
                            or lse.device != dev):
        raise ValueError("lse must be a contiguous float32 [tokens, Hq] tensor on the cache's device")
    desc, code, way = cache.descriptor(), S._dtype_code(q), PAGED_PATHS[path]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if window != 0:  # to the C int's range (ctypes would keep the low bits only); one past every cache is none there too
        window = min(max(int(window), -1), 0x7fffffff)
    sizes = (batch.B, T, batch.max_q, batch.max_pages, Hq, window, way)  # what scratch goes by, beside layouts

    def call(st):
        nonlocal out
        os_ = None
        if out is None:
            out = torch.empty_like(q) if qs is None else torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
        else:
            if out.shape != q.shape or out.dtype != q.dtype:
                raise ValueError("out must have q's shape and dtype")
            os_ = _rows(out, Hq, cache, "out")
        qp, op = q.data_ptr(), out.data_ptr()
        last, have = cache._scratch
        if last != sizes:
            have = 0
        while True:
            ws = torch.empty(have, dtype=torch.uint8, device=dev) if have else None
            rc = sdpa_fwd_paged(qp, qs, desc, batch, op, os_, code, Hq, scale, window, float(softcap),
                                None if slopes is None else slopes.data_ptr(), None if lse is None else lse.data_ptr(),
                                way, None if ws is None else ws.data_ptr(), have, st)
            if rc != -6:
                cache._scratch = (sizes, have)
                return rc
            ws = None
            need = sdpa_fwd_paged_workspace(desc, batch, qp, qs, op, os_, code, Hq, window, way)
            if need <= have:
                return int(min(need, -6))
            have = need
    _check(_on(dev, stream, call), "sdpa_fwd_paged")
    return out
