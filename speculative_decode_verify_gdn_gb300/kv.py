"""Python binding of the paged key/value cache's C ABI (include/gdn_kv.h): attention of verify
windows over the cache, commit, fork and compact.

Argument marshalling only, as in ``gdn``: each function checks the torch tensors' device, dtype,
shape and strides against ``dims`` and passes raw pointers and the CUDA stream to the library.
Errors are ``gdn.GdnError``; what only the device sees is reported by ``gdn.gdn_device_status``
with the DEVERR_* bits below.

The cache is a pair of tensors of logical shape [n_layers, n_pages, page_size, Hkv, D].  Any
strides will do that the header allows, so a cache kept as [.., Hkv, page_size, D], or keys and
values kept in one tensor, are passed as views; give one of them to ``make_kv_dims``.
"""
from __future__ import annotations

import ctypes

import torch

from . import gdn
from .gdn import _check

EXPORTED = ("gdn_attn_verify", "gdn_attn_workspace_size", "gdn_kv_commit", "gdn_kv_fork", "gdn_kv_compact",
            "gdn_kv_workspace_size")

DEVERR_KV_LEN, DEVERR_KV_PAGE, DEVERR_KV_SLOT, DEVERR_KV_FULL, DEVERR_KV_SHARED, DEVERR_KV_WINDOW = 32, 64, 128, 256, 512, 1024

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_TORCH = (torch.bfloat16, torch.float16)
_I32 = torch.int32


class KvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "K", "Hq", "Hkv", "D", "page_size", "n_pages", "max_pages",
                                              "n_slots", "slot0", "n_layers", "dtype")] + \
               [(n, ctypes.c_int64) for n in ("cache_layer_stride", "cache_page_stride", "cache_token_stride",
                                              "cache_head_stride", "q_token_stride", "win_token_stride",
                                              "win_layer_stride")]


def make_kv_dims(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_slots=None, slot0=0, n_layers=1,
                 dtype=torch.bfloat16, cache=None, q=None, win=None) -> KvDims:
    """Dims of the cache calls.  ``cache`` (k_cache or v_cache), ``q`` [B, K, Hq, D] and ``win``
    (k_win or v_win, [B, K, Hkv, D] or [n_layers, B, K, Hkv, D]) give the strides; contiguous
    [n_layers, n_pages, page_size, Hkv, D], q and windows otherwise."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
    row = Hkv * D
    cs = (n_pages * page_size * row, page_size * row, row, D) if cache is None else cache.stride()[:4]
    step = -3 if K > 1 else -4  # from token to token; a single one has none, whatever its stride says
    one = B * K == 1
    qs = Hq * D if q is None or one else q.stride(step)
    ws = row if win is None or one else win.stride(step)
    ls = B * K * row if win is None else win.stride(0) if win.dim() == 5 else 0
    return KvDims(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, B if n_slots is None else n_slots, slot0, n_layers,
                  _DTYPES[dtype], *cs, qs, ws, ls)


_lib = None


def load_library() -> ctypes.CDLL:
    """The library of ``gdn`` with this module's entry points declared."""
    global _lib
    if _lib is None:
        lib = gdn.load_library()
        P, D, U = ctypes.c_void_p, ctypes.POINTER(KvDims), ctypes.c_uint64
        lib.gdn_attn_verify.argtypes = [D, ctypes.c_int32] + [P] * 10 + [ctypes.c_float, P, P, P, U, P]
        lib.gdn_kv_commit.argtypes = [D] + [P] * 13 + [U, P]
        lib.gdn_kv_fork.argtypes = [D] + [P] * 10 + [U, P]
        lib.gdn_kv_compact.argtypes = [D] + [P] * 9 + [U, P]
        lib.gdn_attn_workspace_size.argtypes = [D, ctypes.POINTER(U)]
        lib.gdn_kv_workspace_size.argtypes = [D, ctypes.POINTER(U)]
        for f in EXPORTED:
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _tensor(t, name, dtype, shape, strides):
    """Address of a CUDA tensor of this dtype, shape and strides (those of single entries aside;
    None: contiguous)."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape and \
            (t.is_contiguous() if strides is None else t.stride() == strides):
        return t.data_ptr()
    return _explain(t, name, dtype, shape, strides)


def _explain(t, name, dtype, shape, strides):
    """What _tensor found amiss, if anything is."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if strides is None:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif any(n > 1 and have != want for n, have, want in zip(shape, t.stride(), strides)):
        raise ValueError(f"{name} has strides {t.stride()}, dims say {strides}")
    return t.data_ptr()


def _ints(t, name, shape, optional=False):
    if t is None and optional:
        return None
    return _tensor(t, name, _I32, shape, None)


def _stream(stream):
    """Handle of `stream`, or of the current one (straight from torch's runtime: building a Stream
    object for it takes 3 us, as long as a launch)."""
    return _current_stream(_current_device()) if stream is None else stream.cuda_stream


_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _cache(d, k_cache, v_cache):
    dt = _TORCH[d.dtype]
    shape = (d.n_layers, d.n_pages, d.page_size, d.Hkv, d.D)
    strides = (d.cache_layer_stride, d.cache_page_stride, d.cache_token_stride, d.cache_head_stride, 1)
    return _tensor(k_cache, "k_cache", dt, shape, strides), _tensor(v_cache, "v_cache", dt, shape, strides)


def _workspace(ws):
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _size(f, dims) -> int:
    n = ctypes.c_uint64(0)
    _check(f(ctypes.byref(dims), ctypes.byref(n)))
    return n.value


def gdn_attn_workspace_size(dims: KvDims) -> int:
    """Bytes of device scratch gdn_attn_verify needs for these dims."""
    return _size(load_library().gdn_attn_workspace_size, dims)


def gdn_kv_workspace_size(dims: KvDims) -> int:
    """Bytes of device scratch gdn_kv_commit, gdn_kv_fork and gdn_kv_compact need for these dims."""
    return _size(load_library().gdn_kv_workspace_size, dims)


def alloc_attn_workspace(dims: KvDims, device="cuda") -> torch.Tensor:
    return torch.empty(gdn_attn_workspace_size(dims), dtype=torch.uint8, device=device)


def alloc_kv_workspace(dims: KvDims, device="cuda") -> torch.Tensor:
    return torch.empty(gdn_kv_workspace_size(dims), dtype=torch.uint8, device=device)


def gdn_attn_verify(dims: KvDims, layer, q, k_win, v_win, k_cache, v_cache, page_table, seq_len, prefix_of, win_len,
                    parent, scale, out, lse, workspace, stream=None) -> None:
    """Attention of B windows of K tokens over the cache (see include/gdn_kv.h): q [B, K, Hq, D],
    k_win, v_win [B, K, Hkv, D]; page_table [n_slots, max_pages], seq_len [n_slots] int32;
    prefix_of, win_len [B] and parent [B, K] int32 or None; out [B, K, Hq, D], lse [B, K, Hq]
    f32 or None."""
    d = dims
    lib = load_library()
    B, K, Hq, Hkv, D = d.B, d.K, d.Hq, d.Hkv, d.D
    dt, qs, ws = _TORCH[d.dtype], d.q_token_stride, d.win_token_stride
    kc, vc = _cache(d, k_cache, v_cache)
    wp, wb = _workspace(workspace)
    win_shape, win_strides = (B, K, Hkv, D), (K * ws, ws, D, 1)
    _check(lib.gdn_attn_verify(
        ctypes.byref(d), layer, _tensor(q, "q", dt, (B, K, Hq, D), (K * qs, qs, D, 1)),
        _tensor(k_win, "k_win", dt, win_shape, win_strides), _tensor(v_win, "v_win", dt, win_shape, win_strides),
        kc, vc, _ints(page_table, "page_table", (d.n_slots, d.max_pages)), _ints(seq_len, "seq_len", (d.n_slots,)),
        _ints(prefix_of, "prefix_of", (B,), True), _ints(win_len, "win_len", (B,), True),
        _ints(parent, "parent", (B, K), True), scale, _tensor(out, "out", dt, (B, K, Hq, D), None),
        None if lse is None else _tensor(lse, "lse", torch.float32, (B, K, Hq), None), wp, wb, _stream(stream)))


def _books(d, table_in, table_out, len_in, len_out, ref_in, ref_out):
    table, slots, pages = (d.n_slots, d.max_pages), (d.n_slots,), (d.n_pages,)
    return (_ints(table_in, "table_in", table), _ints(table_out, "table_out", table), _ints(len_in, "len_in", slots),
            _ints(len_out, "len_out", slots), _ints(ref_in, "ref_in", pages), _ints(ref_out, "ref_out", pages))


def gdn_kv_commit(dims: KvDims, accept_len, parent, k_win, v_win, k_cache, v_cache, table_in, table_out, len_in,
                  len_out, ref_in, ref_out, workspace, stream=None) -> None:
    """Writes the accepted window tokens (accept_len [B]; with parent [B, K] the path to node
    accept_len - 1) of k_win, v_win [n_layers, B, K, Hkv, D] to pages, allocating them.  Each
    *_out may be its *_in."""
    d = dims
    lib = load_library()
    B, K = d.B, d.K
    dt, ws = _TORCH[d.dtype], d.win_token_stride
    kc, vc = _cache(d, k_cache, v_cache)
    wp, wb = _workspace(workspace)
    shape, strides = (d.n_layers, B, K, d.Hkv, d.D), (d.win_layer_stride, K * ws, ws, d.D, 1)
    _check(lib.gdn_kv_commit(
        ctypes.byref(d), _ints(accept_len, "accept_len", (B,)), _ints(parent, "parent", (B, K), True),
        _tensor(k_win, "k_win", dt, shape, strides), _tensor(v_win, "v_win", dt, shape, strides), kc, vc,
        *_books(d, table_in, table_out, len_in, len_out, ref_in, ref_out), wp, wb, _stream(stream)))


def gdn_kv_fork(dims: KvDims, src, k_cache, v_cache, table_in, table_out, len_in, len_out, ref_in, ref_out, workspace,
                stream=None) -> None:
    """Slot i takes the sequence of slot src[i] (src [n_slots] int32, -1: none); sequences that no
    slot takes are freed.  ref_out may be ref_in."""
    d = dims
    lib = load_library()
    kc, vc = _cache(d, k_cache, v_cache)
    wp, wb = _workspace(workspace)
    _check(lib.gdn_kv_fork(ctypes.byref(d), _ints(src, "src", (d.n_slots,)), kc, vc,
                           *_books(d, table_in, table_out, len_in, len_out, ref_in, ref_out), wp, wb, _stream(stream)))


def gdn_kv_compact(dims: KvDims, k_cache, v_cache, table_in, table_out, seq_len, ref_in, ref_out, n_live, workspace,
                   stream=None) -> None:
    """Moves the live pages to pages 0..n_live-1 (n_live [1] int32).  table_out may be table_in,
    ref_out ref_in."""
    d = dims
    lib = load_library()
    kc, vc = _cache(d, k_cache, v_cache)
    wp, wb = _workspace(workspace)
    table, pages = (d.n_slots, d.max_pages), (d.n_pages,)
    _check(lib.gdn_kv_compact(
        ctypes.byref(d), kc, vc, _ints(table_in, "table_in", table), _ints(table_out, "table_out", table),
        _ints(seq_len, "seq_len", (d.n_slots,)), _ints(ref_in, "ref_in", pages), _ints(ref_out, "ref_out", pages),
        _ints(n_live, "n_live", (1,)), wp, wb, _stream(stream)))
