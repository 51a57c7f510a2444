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

import ctypes
import functools
import struct

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
    "kv_plan_work": (_I, [_I, _I64, _I]),
    "kv_release_pages": (_I, [_P, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P]),
    "kv_append": (_I, [_C, _P, _P, _I64, _I64, _I, _P, _I, _P]),
    "kv_attend": (_I, [_C, _P, _I64, _I64, _I, _I, _I, _P, _I, _P, _F, _I, _P, _P, _P, _SZ, _P]),
    "kv_attend_work": (_I, [_C, _I, _I, _I, ctypes.POINTER(_SZ)]),
    "norm_quant": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I, _I, _I, _F, _I, _P, _I64, _P, _P]),
}

# element types (values of include/wbserve.h)
BF16, F16, F32, E4M3 = 0, 1, 2, 3

# Set by _load() at the first call. The small calls here are bound by the host (a launch is
# 3.5 us of the 7 us a call of one kernel takes), so checks are plain attribute reads, the
# cache's descriptor is packed into bytes rather than built as a ctypes structure, and
# functions take it as a plain address.
_torch = None
_fn = {}
_codes = {}
_desc = struct.Struct("PPPPqiiii")         # wb_kv_cache


def _load():
    global _torch
    import torch

    from . import lib
    h = lib()
    for name, (res, args) in SERVE_SIGNATURES.items():
        _fn[name] = ctypes.CFUNCTYPE(res, *(_P if a is _C else a for a in args))((name, h))
    _codes.update({torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32, torch.float8_e4m3fn: E4M3})
    _torch = torch


def _check(status: int, what: str) -> None:
    if status:
        from . import check
        check(status, what)


def _refuse(t, name, what, device):
    raise ValueError(f"{name}: expected {what} on cuda:{device}, got {t.dtype} {tuple(t.shape)} strides={t.stride()} "
                     f"device={t.device}")


def _device(t, name) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: expected a tensor on the GPU, got device={t.device}")
    return d


def _ptr(t, name, dtype, shape, device) -> int:
    """Address of a contiguous tensor of this type and shape on this device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(t, name, f"contiguous {dtype} {tuple(shape)}", device)
    return t.data_ptr()


def _rows(t, name, dtype, shape, device, row):
    """Address and row stride of a tensor of `row` contiguous elements a row."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _refuse(t, name, f"{dtype} {tuple(shape)}", device)
    if t.is_contiguous():
        return t.data_ptr(), row
    strides = t.stride()
    if strides[1:] != ((shape[2], 1) if len(shape) == 3 else (1,)) and not t[:1].is_contiguous():
        _refuse(t, name, f"{dtype} {tuple(shape)} with contiguous rows", device)
    return t.data_ptr(), strides[0]


def _stream_of(device, stream):
    """Handle of the given stream, or of the device's current one."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"stream: on {stream.device}, the tensors on cuda:{device}")
    return stream.cuda_stream


def _call(name, device, *args):
    """One library call with the tensors' device current (a launch needs its stream's)."""
    if _torch._C._cuda_getDevice() == device:
        status = _fn[name](*args)
    else:
        with _torch.cuda.device(device):
            status = _fn[name](*args)
    if status:
        _check(status, name)


def _workspace(n, dtype, device, stream):
    """Memory for one call, taken from the allocator on the call's stream: it is given to
    another call only behind this one."""
    if stream is None:
        return _torch.empty(n, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(n, dtype=dtype, device=device)


def _cache(k_cache, v_cache, k_scale, v_scale):
    """The cache's descriptor, its device, shape and element code."""
    if _torch is None:
        _load()
    kind, shape, dev = k_cache.dtype, k_cache.shape, k_cache.get_device()
    code = _codes.get(kind, F32)
    if not (dev >= 0 and code != F32 and len(shape) == 4 and v_cache.dtype is kind and v_cache.shape == shape
            and v_cache.get_device() == dev and k_cache.is_contiguous() and v_cache.is_contiguous()):
        dev = _device(k_cache, "k_cache")
        if code == F32 or len(shape) != 4:
            raise ValueError(f"k_cache: expected bfloat16, float16 or float8_e4m3fn [pages, H, page, D], got {kind} "
                             f"{tuple(shape)}")
        _ptr(k_cache, "k_cache", kind, shape, dev)
        _ptr(v_cache, "v_cache", kind, shape, dev)
    ks = vs = 0
    if code == E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("k_scale, v_scale: a float8_e4m3fn cache needs the scales [pages, H, page]")
        ks = _ptr(k_scale, "k_scale", _torch.float32, shape[:3], dev)
        vs = _ptr(v_scale, "v_scale", _torch.float32, shape[:3], dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale, v_scale: only a float8_e4m3fn cache has scales")
    pages, H, page, D = shape
    if H > _MAX or page > _MAX or D > _MAX:
        raise ValueError(f"k_cache: {tuple(shape)} is too large")
    return _desc.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, pages, page, H, D, code), dev, shape, code


_MAX = 0x7FFFFFFF


@functools.lru_cache(maxsize=1024)
def _plan_work(R, n, in_place):
    return _fn["kv_plan_work"](R, n, in_place)


@functools.lru_cache(maxsize=1024)
def _attend_work(code, pages, H, page, D, R, Hq, width):
    """Workspace bytes of kv_attend, which follow from the sizes alone."""
    fake, need = 16, _SZ()
    scale = fake if code == E4M3 else 0
    _check(_fn["kv_attend_work"](_desc.pack(fake, fake, scale, scale, pages, page, H, D, code), R, Hq, width,
                                 ctypes.byref(need)), "kv_attend")
    return need.value


def plan_pages(lens, more, table, free, n_free, page: int, slots, starts, status, lens_out=None, n_free_out=None,
               stream=None):
    """Places ``more[r]`` new tokens behind the ``lens[r]`` stored ones of each request:
    pages are popped off the stack ``free[:n_free]`` (topmost first, request by request)
    into ``table`` (int32 [R, width]), ``slots`` (int64 [n], 16-byte aligned) gets each new
    token's slot in request order and -1 behind the last, ``starts`` (int32 [R + 1]) each request's first
    new token. ``lens_out`` and ``n_free_out`` get the new lengths and number of free pages
    (default: in place). int32 [R]: lens, more; int32 [1]: n_free, status. All or nothing:
    ``status`` becomes 0, or 1 (a negative count, ``n_free`` out of range), 2 (more pages
    than ``table`` is wide), 3 (more new tokens than ``slots``), 4 (not enough free pages),
    and then nothing is placed and every slot is -1. Other outputs overlap no input."""
    if _torch is None:
        _load()
    if not -_MAX <= page <= _MAX:         # (ctypes would pass its lower 32 bits)
        raise ValueError(f"page: {page} is out of range")
    dev = _device(lens, "lens")
    i32 = _torch.int32
    if table.dim() != 2 or free.dim() != 1 or slots.dim() != 1:
        raise ValueError(f"table, free, slots: expected 2, 1 and 1 dimensions, got {table.dim()}, {free.dim()}, {slots.dim()}")
    R, width = table.shape
    lens_out = lens if lens_out is None else lens_out
    n_free_out = n_free if n_free_out is None else n_free_out
    n = slots.shape[0]
    size = free.shape[0]
    if R > _MAX or width > _MAX or size > _MAX:
        raise ValueError(f"table, free: {tuple(table.shape)}, {tuple(free.shape)} are too large")
    # (one expression for what _ptr checks of each: twelve calls are 2 us)
    rows, one = (R,), (1,)
    if not (lens.dtype is i32 and more.dtype is i32 and table.dtype is i32 and free.dtype is i32 and n_free.dtype is i32
            and starts.dtype is i32 and lens_out.dtype is i32 and n_free_out.dtype is i32 and status.dtype is i32
            and slots.dtype is _torch.int64 and lens.shape == rows and more.shape == rows and lens_out.shape == rows
            and n_free.shape == one and n_free_out.shape == one and status.shape == one and starts.shape == (R + 1,)
            and more.get_device() == table.get_device() == free.get_device() == n_free.get_device() == slots.get_device()
            == starts.get_device() == lens_out.get_device() == n_free_out.get_device() == status.get_device() == dev
            and lens.is_contiguous() and more.is_contiguous() and table.is_contiguous() and free.is_contiguous()
            and slots.is_contiguous() and starts.is_contiguous() and lens_out.is_contiguous()):
        for t, name, shape in ((lens, "lens", rows), (more, "more", rows), (table, "table", (R, width)), (free, "free", (size,)),
                               (n_free, "n_free", one), (starts, "starts", (R + 1,)), (lens_out, "lens_out", rows),
                               (n_free_out, "n_free_out", one), (status, "status", one)):
            _ptr(t, name, i32, shape, dev)
        _ptr(slots, "slots", _torch.int64, (n,), dev)
    lens_p, n_free_p, lens_out_p, n_free_out_p = lens.data_ptr(), n_free.data_ptr(), lens_out.data_ptr(), n_free_out.data_ptr()
    work = _plan_work(R, n, lens_out_p == lens_p or n_free_out_p == n_free_p)
    held = _workspace(work, i32, dev, stream) if work else None
    _call("kv_plan_pages", dev, lens_p, more.data_ptr(), R, table.data_ptr(), width, free.data_ptr(), size, n_free_p, page,
          slots.data_ptr(), n, starts.data_ptr(), lens_out_p, n_free_out_p, status.data_ptr(),
          held.data_ptr() if work else None, _stream_of(dev, stream))


def release_pages(ended, lens, table, free, n_free, page: int, status, stream=None):
    """Requests with ``ended[r]`` (bool or uint8 [R]) give their pages back to the stack
    ``free[:n_free]``; their lengths become 0 and ``n_free`` grows, in place. ``status``
    (int32 [1]) as for ``plan_pages`` (4: more pages than ``free`` holds)."""
    if _torch is None:
        _load()
    if not -_MAX <= page <= _MAX:
        raise ValueError(f"page: {page} is out of range")
    dev = _device(lens, "lens")
    i32 = _torch.int32
    if table.dim() != 2 or free.dim() != 1:
        raise ValueError(f"table, free: expected 2 and 1 dimensions, got {table.dim()}, {free.dim()}")
    R, width = table.shape
    if R > _MAX or width > _MAX or free.shape[0] > _MAX:
        raise ValueError(f"table, free: {tuple(table.shape)}, {tuple(free.shape)} are too large")
    kind = _torch.bool if ended.dtype is _torch.bool else _torch.uint8
    _call("kv_release_pages", dev, _ptr(ended, "ended", kind, (R,), dev), _ptr(lens, "lens", i32, (R,), dev), R,
          _ptr(table, "table", i32, (R, width), dev), width, _ptr(free, "free", i32, free.shape, dev), free.shape[0],
          _ptr(n_free, "n_free", i32, (1,), dev), page, _ptr(status, "status", i32, (1,), dev), _stream_of(dev, stream))


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, stream=None):
    """Writes keys and values of new tokens, ``k``, ``v`` [N, H, D] (rows may be strided, all
    16-byte aligned), at ``slots`` (int64 [N]) of the cache; tokens with a slot outside the cache (-1: padding)
    are not stored, and no slot is given twice. They are of the cache's type or float32, for a float8_e4m3fn cache also
    bfloat16 or float16: each vector is then stored as max|x| / 448 and the nearest codes."""
    c, dev, shape, _ = _cache(k_cache, v_cache, k_scale, v_scale)
    kind = k.dtype
    if kind not in _codes:
        raise ValueError(f"k: {kind} is not supported")
    if slots.dim() != 1:
        _refuse(slots, "slots", "torch.int64 [N]", dev)
    N, H, D = slots.shape[0], shape[1], shape[3]
    if N > _MAX:
        raise ValueError(f"slots: {N} are too many")
    rows = (N, H, D)
    if (v.dtype is kind and k.shape == rows and v.shape == rows and k.get_device() == v.get_device() == dev
            and k.is_contiguous() and v.is_contiguous()):
        kp, vp, k_row, v_row = k.data_ptr(), v.data_ptr(), H * D, H * D
    else:
        kp, k_row = _rows(k, "k", kind, rows, dev, H * D)
        vp, v_row = _rows(v, "v", kind, rows, dev, H * D)
    _call("kv_append", dev, c, kp, vp, k_row, v_row, _codes[kind], _ptr(slots, "slots", _torch.int64, (N,), dev), N,
          _stream_of(dev, stream))


def kv_attend(q, k_cache, v_cache, table, lens, o, scale=None, window: int = 0, lse=None, k_scale=None, v_scale=None,
              stream=None):
    """Attention of one new token per request over its stored tokens (the last ``window``
    of them; 0: all): ``o`` [R, Hq, D] = softmax(scale q k^T) v, ``lse`` (float32 [R, Hq],
    optional) the log-sum-exp of its scores. ``q`` [R, Hq, D] is of the cache's type
    (bfloat16 or float16 for a float8_e4m3fn cache), requests and heads may be strided (by
    multiples of 8; ``q`` and ``o`` are 16-byte aligned);
    query head h reads key-value head h // (Hq // H). ``table`` int32 [R, width], ``lens``
    int32 [R]: the stored tokens of each request, the new one's among them. ``scale``
    defaults to 1 / sqrt(D). A request without tokens has o = 0 and lse = -inf; one whose
    length or page ids are out of range has NaN. ``o`` is not ``q``: outputs overlap no input."""
    c, dev, shape, code = _cache(k_cache, v_cache, k_scale, v_scale)
    kind = q.dtype
    if q.dim() != 3 or table.dim() != 2 or kind not in _codes:
        raise ValueError(f"q, table: expected [R, Hq, D] and [R, width], got {kind} {tuple(q.shape)}, {tuple(table.shape)}")
    R, Hq, D = q.shape
    pages, H, page, d = shape
    q_row, q_head, q_col = q.stride()
    if q.get_device() != dev or D != d or q_col != 1:
        _refuse(q, "q", f"[R, Hq, {d}] with contiguous heads", dev)
    width = table.shape[1]
    if R > _MAX or Hq > _MAX or width > _MAX or not 0 <= window:
        raise ValueError(f"q, table, window: {tuple(q.shape)}, {tuple(table.shape)}, {window} are out of range")
    i32 = _torch.int32
    if not (table.dtype is i32 and lens.dtype is i32 and o.dtype is kind and table.shape[0] == R and lens.shape == (R,)
            and o.shape == (R, Hq, D) and table.get_device() == lens.get_device() == o.get_device() == dev
            and table.is_contiguous() and lens.is_contiguous() and o.is_contiguous()):
        _ptr(table, "table", i32, (R, width), dev)
        _ptr(lens, "lens", i32, (R,), dev)
        _ptr(o, "o", kind, (R, Hq, D), dev)
    lsep = None if lse is None else _ptr(lse, "lse", _torch.float32, (R, Hq), dev)
    n = _attend_work(code, pages, H, page, D, R, Hq, width)
    held = _workspace(n, _torch.uint8, dev, stream) if n else None
    _call("kv_attend", dev, c, q.data_ptr(), q_row if R > 1 else 0, q_head if Hq > 1 else 0, _codes[kind], R, Hq,
          table.data_ptr(), width, lens.data_ptr(), D ** -0.5 if scale is None else scale, window if window < _MAX else 0,
          o.data_ptr(), lsep, held.data_ptr() if n else None, n, _stream_of(dev, stream))


def norm_quant(x, weight, codes, scales, eps: float = 1e-6, group: int = 0, residual=None, residual_out=None,
               stream=None):
    """Root-mean-square norm with an 8-bit output: with h = x + residual (float32, stored
    into ``residual_out``, by default in place) and y = h / sqrt(mean(h^2) + eps) * weight,
    ``scales`` (float32 [N, groups]) gets max|y| / 448 of each 128 columns (``group`` 128)
    or of each row (``group`` 0) and ``codes`` (float8_e4m3fn [N, D]) y / scale. ``x``,
    ``residual``, ``weight`` ([D], or None for 1) are of one type: bfloat16, float16 or
    float32; rows may be strided. Other outputs overlap no input."""
    if _torch is None:
        _load()
    if not -_MAX <= group <= _MAX:        # (the library would take its lower 32 bits, and write their number of scales)
        raise ValueError(f"group: {group} is out of range")
    dev = _device(x, "x")
    kind = x.dtype
    code = _codes.get(kind, E4M3)
    if code == E4M3 or x.dim() != 2:
        raise ValueError(f"x: expected bfloat16, float16 or float32 [N, D], got {kind} {tuple(x.shape)}")
    shape = N, D = x.shape
    if N > _MAX or D > _MAX:
        raise ValueError(f"x: {tuple(shape)} is too large")
    groups = -(-D // group) if group > 0 else 1
    f8, f32 = _torch.float8_e4m3fn, _torch.float32
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out: there is no residual")
        r, out = x, x                     # (checked with x, not passed)
    else:
        r, out = residual, residual if residual_out is None else residual_out
    w = x if weight is None else weight
    if (r.dtype is kind and out.dtype is kind and w.dtype is kind and codes.dtype is f8 and scales.dtype is f32
            and r.shape == shape and out.shape == shape and codes.shape == shape and scales.shape == (N, groups)
            and (weight is None or w.shape == (D,))
            and r.get_device() == out.get_device() == w.get_device() == codes.get_device() == scales.get_device() == dev
            and x.is_contiguous() and r.is_contiguous() and out.is_contiguous() and w.is_contiguous()
            and codes.is_contiguous() and scales.is_contiguous()):
        x_row = r_row = ro_row = c_row = D
    else:
        x_row = _rows(x, "x", kind, shape, dev, D)[1]
        r_row = _rows(r, "residual", kind, shape, dev, D)[1]
        ro_row = _rows(out, "residual_out", kind, shape, dev, D)[1]
        c_row = _rows(codes, "codes", f8, shape, dev, D)[1]
        if weight is not None:
            _ptr(w, "weight", kind, (D,), dev)
        _ptr(scales, "scales", f32, (N, groups), dev)
    have = residual is not None
    _call("norm_quant", dev, x.data_ptr(), x_row, r.data_ptr() if have else None, r_row, out.data_ptr() if have else None,
          ro_row, None if weight is None else w.data_ptr(), code, N, D, eps, group, codes.data_ptr(), c_row,
          scales.data_ptr(), _stream_of(dev, stream))
