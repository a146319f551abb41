"""ctypes binding of libmqa's 8-bit K/V caches (include/mqa_q8.h).

Argument marshalling only, like ``binding``: shapes and dtypes are checked,
device pointers and the current CUDA stream are handed to the C ABI, and a
non-OK status becomes an ``MqaError``.

A cache is four tensors (``Cache``): e4m3 codes and one exponent byte per row
and K/V head, for keys and for values.  A row's values are
``code * 2**(exponent - 127)``.

    cache = q8.new_cache(b, m_max, g, d)
    q8.append(cache, k_new, v_new, pos)              # one row per sequence, or
    q8.append(cache, k_new, v_new, pos, cu_new=cu)   # packed rows, ragged counts
    o = q8.decode(q, cache, lens, scale)
    o = q8.decode_shared(q, prefix, prefix_len, cache, lens, scale)   # prefix: a Cache of b = 1
    k, v = q8.read(cache, cu_rows, total)

Every call has a plan (``AppendPlan``, ``ReadPlan``, ``DecodePlan``,
``SharedPlan``) that marshals its arguments once; ``run()`` is then one C call
on those buffers.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from .binding import (MQA_OK, PATHS, DecodeOptions, MqaError, _c_float, _c_int, _c_ptr, _c_size, _check_cuda,
                      _dtype_code, _ptr, _stream_handle)
from . import binding

# Every symbol include/mqa_q8.h declares, with its ctypes signature.
SIGNATURES = {
    "mqa_q8_append": (_c_int, [_c_ptr] * 8 + [_c_int] * 7 + [_c_ptr, _c_ptr]),
    "mqa_q8_read": (_c_int, [_c_ptr] * 8 + [_c_int] * 7 + [_c_ptr, _c_ptr]),
    "mqa_q8_decode_workspace_size": (_c_size, [_c_int] * 4),
    "mqa_q8_decode": (_c_int, [_c_ptr] * 7 + [_c_int] * 6 + [_c_float, _c_int, _c_ptr, _c_size, _c_ptr,
                                                             ctypes.POINTER(DecodeOptions), _c_ptr]),
    "mqa_q8_decode_shared_workspace_size": (_c_size, [_c_int] * 5),
    "mqa_q8_decode_shared": (_c_int, [_c_ptr] * 12 + [_c_int] * 6 + [_c_float, _c_int, _c_ptr, _c_size, _c_ptr, _c_ptr]),
}

_LIB = None


def lib():
    """libmqa.so with the 8-bit entry points' signatures declared."""
    global _LIB
    if _LIB is None:
        lib_ = binding.lib()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib_, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib_
    return _LIB


_UNTYPED = {}


def _untyped(name):
    """The entry point as a function object of its own without argument types."""
    if name not in _UNTYPED:
        fn = lib()[name]   # indexing makes a new function object
        fn.restype = SIGNATURES[name][0]
        _UNTYPED[name] = fn
    return _UNTYPED[name]


class Cache(NamedTuple):
    """K and V codes [b, m_max, g, d] (float8_e4m3fn) and exponents [b, g, m_max] (uint8)."""

    k: object
    k_exp: object
    v: object
    v_exp: object


def new_cache(b, m_max, g, d_k, d_v=None, device="cuda"):
    """An empty cache (zero codes and exponents: every row reads as zeros)."""
    import torch
    d_v = d_k if d_v is None else d_v

    def codes(d):
        return torch.zeros((b, m_max, g, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)

    def exps():
        return torch.zeros((b, g, m_max), dtype=torch.uint8, device=device)

    return Cache(codes(d_k), exps(), codes(d_v), exps())


def _cache_shape(cache, where):
    """(b, m_max, g, d_k, d_v) of a consistent cache."""
    import torch
    k, ke, v, ve = cache
    _check_cuda(k, ke, v, ve)
    if k.dtype != torch.float8_e4m3fn or v.dtype != torch.float8_e4m3fn or ke.dtype != torch.uint8 \
            or ve.dtype != torch.uint8:
        raise TypeError(f"{where}: a cache holds float8_e4m3fn codes and uint8 exponents")
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError(f"{where}: codes must be [b, m_max, g, d]")
    b, m_max, g, d_k = k.shape
    if tuple(v.shape[:3]) != (b, m_max, g) or tuple(ke.shape) != (b, g, m_max) or tuple(ve.shape) != (b, g, m_max):
        raise ValueError(f"{where}: inconsistent cache shapes")
    return b, m_max, g, d_k, v.shape[3]


def _check_i32(t, n, what):
    import torch
    if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n,)):
        raise ValueError(f"{what} must be int32 [{n}]")


def _same_device(first, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("libmqa needs all tensors of a call on one device")


def _on(stream):
    """Allocations made here belong to the stream that will use them: memory
    freed with a plan is then reused in that stream's order."""
    import contextlib
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _workspace(workspace, need, device, stream):
    import torch
    if workspace is None:
        with _on(stream):
            return torch.empty(max(256, need), dtype=torch.uint8, device=device)
    return workspace


class _Plan:
    """One C call with its arguments marshalled; tensors it points to are kept.
    ``stream`` None is the current stream of the tensors' device at each run.
    Like any tensor in use, a plan is kept until the work of its runs is done
    (and while a graph that captured a run may still be replayed); runs of one
    plan must be ordered on the GPU, as they share its workspace.

    The arguments are ctypes objects made once and handed to a function object
    without declared argument types, which skips their conversion at every call
    (about two thirds of a small call's host time)."""

    def _set(self, name, result, keep, args, stream):
        import torch
        self._name, self._result, self._keep, self._stream = name, result, keep, stream
        device = next(t.device for t in keep if t is not None)
        self._index = device.index if device.index is not None else torch.cuda.current_device()
        types = SIGNATURES[name][1]
        ready = (ctypes._SimpleCData, type(ctypes.byref(ctypes.c_int())))
        self._args = tuple(a if isinstance(a, ready) else t(a) for a, t in zip(args, types))
        self._fn = _untyped(name)
        self._current_stream, self._current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device

    def run(self):
        handle = _c_ptr(self._current_stream(self._index) if self._stream is None else self._stream.cuda_stream)
        if self._current_device() == self._index:
            st = self._fn(*self._args, handle)
        else:
            import torch
            with torch.cuda.device(self._index):
                st = self._fn(*self._args, handle)
        if st != MQA_OK:
            raise MqaError(st, self._name)
        return self._result


class AppendPlan(_Plan):
    """mqa_q8_append: quantise k_new / v_new [total, g, d] into ``cache``.

    Sequence s's rows are cu_new[s] .. cu_new[s+1]-1 (int32 [b+1]; without
    ``cu_new`` one row per sequence) and go to cache rows pos[s], pos[s]+1, ...
    (pos int32 [b]).  ``run()`` returns the cache."""

    def __init__(self, cache, k_new, v_new, pos, cu_new=None, status_flags=None, stream=None):
        cache = Cache(*cache)
        b, m_max, g, d_k, d_v = _cache_shape(cache, "append")
        _check_cuda(k_new, v_new, pos, cu_new, status_flags)
        _same_device(cache.k, *cache[1:], k_new, v_new, pos, cu_new, status_flags)
        total = k_new.shape[0]
        if tuple(k_new.shape) != (total, g, d_k) or tuple(v_new.shape) != (total, g, d_v):
            raise ValueError("append: k_new/v_new must be [total, g, d]")
        if cu_new is None and total != b:
            raise ValueError("append: without cu_new there is one new row per sequence")
        _check_i32(pos, b, "pos")
        _check_i32(cu_new, b + 1, "cu_new")
        dt = _dtype_code(k_new)
        if _dtype_code(v_new) != dt:
            raise TypeError("append: k_new and v_new must share one dtype")
        self._set("mqa_q8_append", cache, (*cache, k_new, v_new, pos, cu_new, status_flags),
                  tuple(_ptr(t) for t in (*cache, k_new, v_new, pos, cu_new)) +
                  (b, total, m_max, g, d_k, d_v, dt, _ptr(status_flags)), stream)


class ReadPlan(_Plan):
    """mqa_q8_read: cache rows start[s] .. of every sequence (start int32 [b],
    0 without it), packed by cu_rows (int32 [b+1]) into k_out / v_out
    [total, g, d] of ``dtype``.  ``run()`` returns (k_out, v_out); packed rows
    that belong to no cache row are left as they were (zeros, when the plan
    allocates the outputs)."""

    def __init__(self, cache, cu_rows, total, start=None, dtype=None, out=None, status_flags=None, stream=None):
        import torch
        cache = Cache(*cache)
        b, m_max, g, d_k, d_v = _cache_shape(cache, "read")
        total = int(total)
        if total < 0:
            raise ValueError("read: total must not be negative")
        if out is None:
            dtype = torch.bfloat16 if dtype is None else dtype
            with _on(stream):
                out = tuple(torch.zeros((total, g, d), dtype=dtype, device=cache.k.device) for d in (d_k, d_v))
        k_out, v_out = out
        _check_cuda(cu_rows, start, k_out, v_out, status_flags)
        _same_device(cache.k, *cache[1:], cu_rows, start, k_out, v_out, status_flags)
        if tuple(k_out.shape) != (total, g, d_k) or tuple(v_out.shape) != (total, g, d_v):
            raise ValueError("read: outputs must be [total, g, d]")
        _check_i32(cu_rows, b + 1, "cu_rows")
        _check_i32(start, b, "start")
        dt = _dtype_code(k_out)
        if _dtype_code(v_out) != dt or (dtype is not None and k_out.dtype != dtype):
            raise TypeError("read: outputs must share one dtype")
        self._set("mqa_q8_read", (k_out, v_out), (*cache, k_out, v_out, start, cu_rows, status_flags),
                  tuple(_ptr(t) for t in (k_out, v_out, *cache, start, cu_rows)) +
                  (b, total, m_max, g, d_k, d_v, dt, _ptr(status_flags)), stream)


def decode_workspace_size(b, h, g, d_v):
    return int(lib().mqa_q8_decode_workspace_size(b, h, g, d_v))


class DecodePlan(_Plan):
    """mqa_q8_decode: o [b, h, d_v] of q [b, h, d_k] over rows t < lens[b] of
    the cache (the newest ``window`` of them when window > 0).  ``run()``
    returns o, the plan's own buffer unless ``out`` is given.  A plan without
    ``workspace`` holds one of its own."""

    def __init__(self, q, cache, lens, scale, out=None, workspace=None, status_flags=None, path="auto", num_ctas=0,
                 window=0, stream=None):
        import torch
        cache = Cache(*cache)
        b, m_max, g, d_k, d_v = _cache_shape(cache, "decode")
        _check_cuda(q, lens, out, workspace, status_flags)
        _same_device(cache.k, *cache[1:], q, lens, out, workspace, status_flags)
        if q.dim() != 3 or q.shape[0] != b or q.shape[2] != d_k:
            raise ValueError("decode: q must be [b, h, d_k] of the cache's b and d_k")
        h = q.shape[1]
        _check_i32(lens, b, "lens")
        if out is None:
            with _on(stream):
                out = torch.empty((b, h, d_v), dtype=q.dtype, device=q.device)
        elif tuple(out.shape) != (b, h, d_v) or out.dtype != q.dtype:
            raise ValueError("decode: out must be [b, h, d_v] in q's dtype")
        ws = _workspace(workspace, decode_workspace_size(b, h, g, d_v), q.device, stream)
        self.out = out
        self._opts = DecodeOptions(PATHS[path], int(num_ctas), int(window))
        self._set("mqa_q8_decode", out, (q, *cache, lens, out, ws, status_flags),
                  tuple(_ptr(t) for t in (out, q, *cache, lens)) +
                  (b, h, g, m_max, d_k, d_v, float(scale), _dtype_code(q), _ptr(ws), ws.numel() * ws.element_size(),
                   _ptr(status_flags), ctypes.byref(self._opts)), stream)


class SharedPlan(_Plan):
    """mqa_q8_decode_shared: o [b, h, d] of q [b, h, d], every sequence over
    the first prefix_len[0] rows of ``prefix`` (a Cache of one sequence;
    prefix_len int32 [1]) and then its own first lens[b] rows of ``cache``.
    ``run()`` returns o."""

    def __init__(self, q, prefix, prefix_len, cache, lens, scale, out=None, workspace=None, status_flags=None,
                 stream=None):
        import torch
        prefix, cache = Cache(*prefix), Cache(*cache)
        b, m_s, g, d, d_v = _cache_shape(cache, "decode_shared")
        one, m_p, *rest = _cache_shape(prefix, "decode_shared")
        if one != 1 or rest != [g, d, d_v] or d != d_v:
            raise ValueError("decode_shared: the prefix must be one sequence of the caches' g and d")
        _check_cuda(q, prefix_len, lens, out, workspace, status_flags)
        _same_device(cache.k, *prefix, *cache[1:], q, prefix_len, lens, out, workspace, status_flags)
        if q.dim() != 3 or q.shape[0] != b or q.shape[2] != d:
            raise ValueError("decode_shared: q must be [b, h, d] of the cache's b and d")
        h = q.shape[1]
        _check_i32(prefix_len, 1, "prefix_len")
        _check_i32(lens, b, "lens")
        if out is None:
            with _on(stream):
                out = torch.empty((b, h, d), dtype=q.dtype, device=q.device)
        elif tuple(out.shape) != (b, h, d) or out.dtype != q.dtype:
            raise ValueError("decode_shared: out must be [b, h, d] in q's dtype")
        ws = _workspace(workspace, int(lib().mqa_q8_decode_shared_workspace_size(b, h, g, m_p, d)), q.device, stream)
        self.out = out
        self._set("mqa_q8_decode_shared", out, (q, *prefix, prefix_len, *cache, lens, out, ws, status_flags),
                  tuple(_ptr(t) for t in (out, q, *prefix, prefix_len, *cache, lens)) +
                  (b, h, g, m_p, m_s, d, float(scale), _dtype_code(q), _ptr(ws), ws.numel() * ws.element_size(),
                   _ptr(status_flags)), stream)


def append(cache, k_new, v_new, pos, cu_new=None, status_flags=None, stream=None):
    """Quantise new rows into the cache, in place (see ``AppendPlan``)."""
    return AppendPlan(cache, k_new, v_new, pos, cu_new, status_flags, stream).run()


def read(cache, cu_rows, total, start=None, dtype=None, out=None, status_flags=None, stream=None):
    """The values of cached rows, packed (see ``ReadPlan``)."""
    return ReadPlan(cache, cu_rows, total, start, dtype, out, status_flags, stream).run()


def decode(q, cache, lens, scale, out=None, workspace=None, status_flags=None, path="auto", num_ctas=0, window=0,
           stream=None):
    """One decode step's attention over the cache (see ``DecodePlan``)."""
    return DecodePlan(q, cache, lens, scale, out, workspace, status_flags, path, num_ctas, window, stream).run()


def decode_shared(q, prefix, prefix_len, cache, lens, scale, out=None, workspace=None, status_flags=None, stream=None):
    """One decode step of a batch behind one shared prefix (see ``SharedPlan``)."""
    return SharedPlan(q, prefix, prefix_len, cache, lens, scale, out, workspace, status_flags, stream).run()
