"""Python binding of the serving operators around the recurrent-state layers of a hybrid
language model (C ABI: ``include/wbserve.h``): the paged key-value cache of its
full-attention layers and the norm with an 8-bit output.

Argument marshalling only, as for the write-back calls: tensors are checked for type,
shape, device and layout (ValueError), then pointers and the stream are forwarded.
Outputs are tensors of the caller, calls are asynchronous on the tensors' device (on
``stream``, or that device's current stream), nothing is kept between calls and every
call can be captured into a graph.

A key-value cache is two tensors ``[pages, H, page, D]`` (bfloat16, float16 or
float8_e4m3fn; D 64, 128 or 256; page a power of two from 8 to 4096) and, for
float8_e4m3fn, their scales ``[pages, H, page]`` (float32): a stored value stands for
``code * scale``. Slot ``s`` is place ``s % page`` of page ``s // page``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("pages", ctypes.c_int64),
                ("page", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_C = ctypes.POINTER(KVCacheDesc)
SERVE_SIGNATURES = {
    "kv_plan_pages": (_I, [_P, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "kv_plan_work": (_I, [_I, _I64]),
    "kv_release_pages": (_I, [_P, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P]),
    "kv_append": (_I, [_C, _P, _P, _I64, _I64, _I, _P, _I, _P]),
    "kv_attend": (_I, [_C, _P, _I64, _I64, _I, _I, _I, _P, _I, _P, _F, _I, _P, _P, _P, _SZ, _P]),
    "kv_attend_work": (_I, [_C, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "norm_quant": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I, _I, _I, _F, _I, _P, _I64, _P, _P]),
}

# element types (values of include/wbserve.h)
BF16, F16, F32, E4M3 = 0, 1, 2, 3
_fns = None
_codes = None


def _lib():
    """The library's serving functions, and the element codes of the torch types."""
    global _fns, _codes
    if _fns is None:
        import torch

        from . import lib
        h = lib()
        for name, (res, args) in SERVE_SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _codes = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.float8_e4m3fn: E4M3}
        _fns = h
    return _fns


def _check(status: int, what: str) -> None:
    if status:
        from . import check
        check(status, what)


def _device(t, name) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: expected a tensor on the GPU, got device={t.device}")
    return d


def _ptr(t, name, dtype, shape, device) -> int:
    """Address of a contiguous tensor of this type and shape on this device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{device}, got {t.dtype} "
                         f"{tuple(t.shape)} device={t.device} contiguous={t.is_contiguous()}")
    return t.data_ptr()


def _rows(t, name, dtype, shape, device):
    """Address and row stride of a tensor whose rows are contiguous each."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t[:1].is_contiguous():
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{device} with contiguous rows, got {t.dtype} "
                         f"{tuple(t.shape)} strides={t.stride()} device={t.device}")
    row = 1
    for n in shape[1:]:
        row *= n
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else row


class _on:
    """The tensors' device made current (a launch needs it to be its stream's), and the
    stream: the given one, or the device's current one."""
    __slots__ = ("device", "stream", "inner")

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        import torch
        self.inner = None
        if torch.cuda.current_device() != self.device:
            self.inner = torch.cuda.device(self.device)
            self.inner.__enter__()
        if self.stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        if self.stream.device.index != self.device:
            if self.inner is not None:
                self.inner.__exit__(None, None, None)
            raise ValueError(f"stream: on {self.stream.device}, the tensors on cuda:{self.device}")
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def _workspace(n, dtype, device, stream):
    """Memory for one call, taken from the allocator on the call's stream: it is given to
    another call only behind this one."""
    import torch
    with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
        return torch.empty(n, dtype=dtype, device=f"cuda:{device}")


def _cache(k_cache, v_cache, k_scale, v_scale):
    """The cache's descriptor, its device and its shape."""
    import torch
    _lib()
    dev = _device(k_cache, "k_cache")
    if k_cache.dim() != 4 or _codes.get(k_cache.dtype) not in (BF16, F16, E4M3):
        raise ValueError(f"k_cache: expected bfloat16, float16 or float8_e4m3fn [pages, H, page, D], got {k_cache.dtype} "
                         f"{tuple(k_cache.shape)}")
    shape = k_cache.shape
    k, v = _ptr(k_cache, "k_cache", k_cache.dtype, shape, dev), _ptr(v_cache, "v_cache", k_cache.dtype, shape, dev)
    ks = vs = None
    if k_cache.dtype is torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("k_scale, v_scale: a float8_e4m3fn cache needs the scales [pages, H, page]")
        ks = _ptr(k_scale, "k_scale", torch.float32, shape[:3], dev)
        vs = _ptr(v_scale, "v_scale", torch.float32, shape[:3], dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale, v_scale: only a float8_e4m3fn cache has scales")
    if max(shape[1:]) > 0x7FFFFFFF:
        raise ValueError(f"k_cache: {tuple(shape)} is too large")
    return KVCacheDesc(k, v, ks, vs, shape[0], shape[2], shape[1], shape[3], _codes[k_cache.dtype]), dev, shape


def plan_pages(lens, more, table, free, n_free, page: int, slots, starts, status, lens_out=None, n_free_out=None,
               stream=None):
    """Places ``more[r]`` new tokens behind the ``lens[r]`` stored ones of each request:
    pages are popped off the stack ``free[:n_free]`` (topmost first, request by request)
    into ``table`` (int32 [R, width]), ``slots`` (int64 [n]) gets each new token's slot in
    request order and -1 behind the last, ``starts`` (int32 [R + 1]) each request's first
    new token. ``lens_out`` and ``n_free_out`` get the new lengths and number of free pages
    (default: in place). int32 [R]: lens, more; int32 [1]: n_free, status. All or nothing:
    ``status`` becomes 0, or 1 (a negative count, ``n_free`` out of range), 2 (more pages
    than ``table`` is wide), 3 (more new tokens than ``slots``), 4 (not enough free pages),
    and then nothing is placed and every slot is -1."""
    import torch
    fns = _lib()
    dev = _device(lens, "lens")
    i32 = torch.int32
    if table.dim() != 2 or free.dim() != 1 or slots.dim() != 1:
        raise ValueError(f"table, free, slots: expected 2, 1 and 1 dimensions, got {table.dim()}, {free.dim()}, {slots.dim()}")
    R, width = table.shape
    lens_out = lens if lens_out is None else lens_out
    n_free_out = n_free if n_free_out is None else n_free_out
    n = slots.shape[0]
    args = [_ptr(lens, "lens", i32, (R,), dev), _ptr(more, "more", i32, (R,), dev), R,
            _ptr(table, "table", i32, (R, width), dev), width, _ptr(free, "free", i32, free.shape, dev), free.shape[0],
            _ptr(n_free, "n_free", i32, (1,), dev), page, _ptr(slots, "slots", torch.int64, (n,), dev), n,
            _ptr(starts, "starts", i32, (R + 1,), dev), _ptr(lens_out, "lens_out", i32, (R,), dev),
            _ptr(n_free_out, "n_free_out", i32, (1,), dev), _ptr(status, "status", i32, (1,), dev)]
    with _on(dev, stream) as s:
        work = fns.kv_plan_work(R, n)
        held = _workspace(work, i32, dev, stream) if work else None
        _check(fns.kv_plan_pages(*args, held.data_ptr() if work else None, s), "kv_plan_pages")


def release_pages(ended, lens, table, free, n_free, page: int, status, stream=None):
    """Requests with ``ended[r]`` (bool or uint8 [R]) give their pages back to the stack
    ``free[:n_free]``; their lengths become 0 and ``n_free`` grows, in place. ``status``
    (int32 [1]) as for ``plan_pages`` (4: more pages than ``free`` holds)."""
    import torch
    fns = _lib()
    dev = _device(lens, "lens")
    i32 = torch.int32
    if table.dim() != 2 or free.dim() != 1:
        raise ValueError(f"table, free: expected 2 and 1 dimensions, got {table.dim()}, {free.dim()}")
    R, width = table.shape
    kind = torch.bool if ended.dtype is torch.bool else torch.uint8
    args = [_ptr(ended, "ended", kind, (R,), dev), _ptr(lens, "lens", i32, (R,), dev), R,
            _ptr(table, "table", i32, (R, width), dev), width, _ptr(free, "free", i32, free.shape, dev), free.shape[0],
            _ptr(n_free, "n_free", i32, (1,), dev), page, _ptr(status, "status", i32, (1,), dev)]
    with _on(dev, stream) as s:
        _check(fns.kv_release_pages(*args, s), "kv_release_pages")


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, stream=None):
    """Writes keys and values of new tokens, ``k``, ``v`` [N, H, D] (rows may be strided), at
    ``slots`` (int64 [N]) of the cache; tokens with a slot outside the cache (-1: padding)
    are not stored. They are of the cache's type or float32, for a float8_e4m3fn cache also
    bfloat16 or float16: each vector is then stored as max|x| / 448 and the nearest codes."""
    import torch
    c, dev, shape = _cache(k_cache, v_cache, k_scale, v_scale)
    want = (slots.shape[0] if slots.dim() == 1 else -1, shape[1], shape[3])
    kp, k_row = _rows(k, "k", k.dtype, want, dev)
    vp, v_row = _rows(v, "v", k.dtype, want, dev)
    if k.dtype not in _codes:
        raise ValueError(f"k: {k.dtype} is not supported")
    sp = _ptr(slots, "slots", torch.int64, want[:1], dev)
    with _on(dev, stream) as s:
        _check(_fns.kv_append(c, kp, vp, k_row, v_row, _codes[k.dtype], sp, want[0], s), "kv_append")


def kv_attend(q, k_cache, v_cache, table, lens, o, scale=None, window: int = 0, lse=None, k_scale=None, v_scale=None,
              stream=None):
    """Attention of one new token per request over its stored tokens (the last ``window``
    of them; 0: all): ``o`` [R, Hq, D] = softmax(scale q k^T) v, ``lse`` (float32 [R, Hq],
    optional) the log-sum-exp of its scores. ``q`` [R, Hq, D] is of the cache's type
    (bfloat16 or float16 for a float8_e4m3fn cache), requests and heads may be strided;
    query head h reads key-value head h // (Hq // H). ``table`` int32 [R, width], ``lens``
    int32 [R]: the stored tokens of each request, the new one's among them. ``scale``
    defaults to 1 / sqrt(D). A request without tokens has o = 0 and lse = -inf; one whose
    length or page ids are out of range has NaN."""
    import torch
    c, dev, shape = _cache(k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3 or table.dim() != 2 or q.dtype not in _codes:
        raise ValueError(f"q, table: expected [R, Hq, D] and [R, width], got {q.dtype} {tuple(q.shape)}, {tuple(table.shape)}")
    R, Hq, D = q.shape
    if q.get_device() != dev or D != shape[3] or q.stride(2) != 1:
        raise ValueError(f"q: expected [R, Hq, {shape[3]}] on cuda:{dev} with contiguous heads, got {tuple(q.shape)} "
                         f"strides={q.stride()} device={q.device}")
    width = table.shape[1]
    f32, i32 = torch.float32, torch.int32
    tp, lp = _ptr(table, "table", i32, (R, width), dev), _ptr(lens, "lens", i32, (R,), dev)
    op = _ptr(o, "o", q.dtype, (R, Hq, D), dev)
    lsep = None if lse is None else _ptr(lse, "lse", f32, (R, Hq), dev)
    need = _SZ()
    _check(_fns.kv_attend_work(c, R, Hq, width, need), "kv_attend")
    n = need.value
    with _on(dev, stream) as s:
        held = _workspace(n, torch.uint8, dev, stream) if n else None
        _check(_fns.kv_attend(c, q.data_ptr(), q.stride(0) if R > 1 else 0, q.stride(1) if Hq > 1 else 0, _codes[q.dtype],
                              R, Hq, tp, width, lp, 1.0 / math.sqrt(D) if scale is None else scale, window, op, lsep,
                              held.data_ptr() if n else None, n, s), "kv_attend")


def norm_quant(x, weight, codes, scales, eps: float = 1e-6, group: int = 0, residual=None, residual_out=None,
               stream=None):
    """Root-mean-square norm with an 8-bit output: with h = x + residual (float32, stored
    into ``residual_out``, by default in place) and y = h / sqrt(mean(h^2) + eps) * weight,
    ``scales`` (float32 [N, groups]) gets max|y| / 448 of each 128 columns (``group`` 128)
    or of each row (``group`` 0) and ``codes`` (float8_e4m3fn [N, D]) y / scale. ``x``,
    ``residual``, ``weight`` ([D], or None for 1) are of one type: bfloat16, float16 or
    float32; rows may be strided."""
    import torch
    fns = _lib()
    dev = _device(x, "x")
    if x.dim() != 2 or _codes.get(x.dtype) not in (BF16, F16, F32):
        raise ValueError(f"x: expected bfloat16, float16 or float32 [N, D], got {x.dtype} {tuple(x.shape)}")
    N, D = x.shape
    xp, x_row = _rows(x, "x", x.dtype, (N, D), dev)
    rp = rop = None
    r_row = ro_row = D
    if residual is not None:
        residual_out = residual if residual_out is None else residual_out
        rp, r_row = _rows(residual, "residual", x.dtype, (N, D), dev)
        rop, ro_row = _rows(residual_out, "residual_out", x.dtype, (N, D), dev)
    elif residual_out is not None:
        raise ValueError("residual_out: there is no residual")
    groups = -(-D // group) if group > 0 else 1
    wp = None if weight is None else _ptr(weight, "weight", x.dtype, (D,), dev)
    cp, c_row = _rows(codes, "codes", torch.float8_e4m3fn, (N, D), dev)
    sp = _ptr(scales, "scales", torch.float32, (N, groups), dev)
    with _on(dev, stream) as s:
        _check(fns.norm_quant(xp, x_row, rp, r_row, rop, ro_row, wp, _codes[x.dtype], N, D, eps, group, cp, c_row, sp, s),
               "norm_quant")
