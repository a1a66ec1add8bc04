"""Python binding of the paged key/value cache's C ABI (include/gdn_kv.h): attention of verify
windows over the cache, commit, fork and compact; norms and rotation of windows; reserve, append and
attention of packed tokens.

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
            "gdn_kv_workspace_size", "gdn_rope_turns", "gdn_attn_rope", "gdn_kv_reserve", "gdn_kv_append",
            "gdn_attn_prefill", "gdn_attn_prefill_workspace_size", "gdn_kv_reserve_marked", "gdn_kv_append_marked",
            "gdn_attn_prefill_marked")

MAX_BATCH = 65535  # sequences of a call

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


class GdnRope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("reserved", ctypes.c_int32)] + \
               [(n, ctypes.c_int64) for n in ("q_token_stride", "q_head_stride", "kv_token_stride", "kv_head_stride")]


def make_kv_dims(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_slots=None, slot0=0, n_layers=1,
                 dtype=torch.bfloat16, cache=None, q=None, win=None) -> KvDims:
    """Dims of the cache calls.  ``cache`` (k_cache or v_cache), ``q`` [B, K, Hq, D] and ``win``
    (k_win or v_win, [B, K, Hkv, D] or [n_layers, B, K, Hkv, D]) give the strides; contiguous
    [n_layers, n_pages, page_size, Hkv, D], q and windows otherwise.  q may also be packed tokens, [tokens, Hq, D]."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
    row = Hkv * D
    cs = (n_pages * page_size * row, page_size * row, row, D) if cache is None else cache.stride()[:4]
    step = -3 if K > 1 else -4  # from token to token; a single one has none, whatever its stride says
    one = B * K == 1
    if q is not None and q.dim() == 3:
        qs = q.stride(0) if q.shape[0] > 1 else Hq * D
    else:
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
        R, L, I = ctypes.POINTER(GdnRope), ctypes.c_int64, ctypes.c_int32
        lib.gdn_rope_turns.argtypes = [P, I, P]
        lib.gdn_attn_rope.argtypes = [D, R] + [P] * 15
        lib.gdn_kv_reserve.argtypes = [D] + [P] * 8 + [U, P]
        lib.gdn_kv_append.argtypes = [D, I, R, P, P, P, L] + [P] * 12
        lib.gdn_attn_prefill.argtypes = [D, I, L] + [P] * 7 + [I, ctypes.c_float, P, P, P, U, P]
        lib.gdn_kv_reserve_marked.argtypes = [D] + [P] * 9 + [U, P]
        lib.gdn_kv_append_marked.argtypes = [D, I, R, P, P, P, L] + [P] * 13
        lib.gdn_attn_prefill_marked.argtypes = [D, I, L] + [P] * 8 + [I, ctypes.c_float, P, P, P, U, P]
        lib.gdn_attn_prefill_workspace_size.argtypes = [D, L, ctypes.POINTER(U)]
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


def stream_state(stream):
    """Handle of `stream`, or of the current one, and whether work on it is being captured into a graph."""
    if stream is None:
        return _current_stream(_current_device()), torch.cuda.is_current_stream_capturing()
    return stream.cuda_stream, _capturing(stream)


def _capturing(stream):
    """Whether work on `stream` is being captured: a look with the stream as the current one, set by torch's runtime
    directly where it is on the current device (1 us, by a context 7)."""
    if stream.device_index != _current_device():
        with torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()
    was = torch._C._cuda_getCurrentStream(stream.device_index)
    torch._C._cuda_setStream(stream_id=stream.stream_id, device_index=stream.device_index, device_type=stream.device_type)
    try:
        return torch.cuda.is_current_stream_capturing()
    finally:
        torch._C._cuda_setStream(stream_id=was[0], device_index=was[1], device_type=was[2])


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
    """Bytes of device scratch gdn_kv_commit, gdn_kv_reserve, gdn_kv_fork and gdn_kv_compact need for these dims."""
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


# ---------------------------------------------------------------- norms and rotation; packed tokens
def rope_turns(radians) -> torch.Tensor:
    """Angles of one token (radians, float64: a tensor, an array or a list) as 64-bit fractions of a turn, the
    form in which the kernels read them: int64 on the CPU."""
    f = torch.as_tensor(radians, dtype=torch.float64).detach().cpu().contiguous()
    t = torch.empty(f.shape, dtype=torch.int64)
    _check(load_library().gdn_rope_turns(f.data_ptr(), f.numel(), t.data_ptr()))
    return t


class Rope:
    """What a layer keeps of its norms and its rotation: weights and turns on the device, and the C struct
    for each set of strides that it has met."""

    def __init__(self, D, turns, interleaved, magnitude, q_weight, k_weight, eps, weight_offset):
        self.D, self.turns, self.q_weight, self.k_weight = D, turns, q_weight, k_weight
        self._scalars = (2 * turns.numel(), int(interleaved), magnitude, eps, weight_offset, 0)
        self._device = turns.get_device()
        self._at = tuple(None if t is None or t.numel() == 0 else t.data_ptr() for t in (turns, q_weight, k_weight))
        self._structs = {}

    def _args(self, strides):
        r = self._structs.get(strides)
        if r is None:
            r = self._structs[strides] = ctypes.byref(GdnRope(*self._scalars, *strides))
        return r


def make_rope(D, radians=(), interleaved=False, magnitude=1.0, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0,
              device="cuda") -> Rope:
    """Norms and rotation of heads of D elements.  radians [rot_dim / 2] float64 holds each pair's angle of one token
    (``rope.frequencies``; empty: no rotation) and magnitude scales what is rotated; interleaved pairs
    elements 2i and 2i + 1 rather than i and i + rot_dim / 2.  q_weight, k_weight [D] are the norms' weights
    (None: no norm), to which weight_offset is added."""
    turns = rope_turns(radians).to(device)
    if turns.dim() != 1 or 2 * turns.numel() > D:
        raise ValueError(f"radians has shape {tuple(turns.shape)}: one angle per pair of at most {D} elements")

    def weight(w, name):
        if w is None:
            return None
        if w.shape != (D,):
            raise ValueError(f"{name} has shape {tuple(w.shape)}, expected ({D},)")
        return w.detach().to(device=turns.device, dtype=torch.float32).contiguous().clone()

    return Rope(D, turns, interleaved, magnitude, weight(q_weight, "q_weight"), weight(k_weight, "k_weight"), eps,
                weight_offset)


def _arg(t, name, dtype, shape, dev, optional=False):
    """Address of a contiguous tensor on the current device."""
    if t is None and optional:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    p = _explain(t, name, dtype, shape, None)
    _on_device(t, name, dev)
    return p


def _lengths(t, name, n_slots, dev):
    """Addresses of lengths and, where they are one of a pair, of the refused entries beside them."""
    if not isinstance(t, tuple):
        return _arg(t, name, _I32, (n_slots,), dev), None
    lens, refused = t
    return _arg(lens, name, _I32, (n_slots,), dev), _arg(refused, "refused", _I32, (n_slots,), dev)


def _on_device(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the current one is {dev}")


def _heads(t, name, dtype, shape, dev):
    """Address, and strides of tokens and heads, of rows [.., heads, D] whose tokens are evenly apart (0: a single one)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _explain(t, name, dtype, shape, t.stride() if isinstance(t, torch.Tensor) else None)
        _on_device(t, name, dev)
    s = t.stride()
    if len(s) == 3:
        step = s[0] if shape[0] > 1 else 0
        even = s[2] == 1
    else:
        n, k = shape[0], shape[1]
        step = s[1] if k > 1 else s[0] if n > 1 else 0
        even = s[3] == 1 and (n == 1 or k == 1 or s[0] == k * s[1])
    if not even:
        raise ValueError(f"{name} has strides {s}: elements of a head one after the other, tokens evenly apart")
    return t.data_ptr(), step, s[-2] if shape[-2] > 1 else shape[-1]


def _like(t, dtype, shape, other, dev):
    """Address of a tensor with the shape and strides of another that has been looked at, None of any other."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.stride() == other.stride() and t.get_device() == dev:
        return t.data_ptr()
    return None


def _beside(k, kt, kh, v, dtype, shape, dev):
    """Address of the values, and the strides that keys (kt and kh, if there are any) and values have alike."""
    if v is None:
        return None, kt, kh
    if k is not None:
        at = _like(v, dtype, shape, k, dev)
        if at is not None:
            return at, kt, kh
    vp, vt, vh = _heads(v, "v", dtype, shape, dev)
    if k is not None and (vt != kt or vh != kh):
        raise ValueError(f"k and v have different strides: {k.stride()} and {v.stride()}")
    return vp, vt, vh


def _out_rows(t, name, dtype, shape, stride, dev):
    """Address of rows [.., heads, D] with heads side by side and tokens `stride` apart."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _explain(t, name, dtype, shape, t.stride() if isinstance(t, torch.Tensor) else None)
        _on_device(t, name, dev)
    D = shape[-1]
    want = (stride, D, 1) if len(shape) == 3 else (shape[1] * stride, stride, D, 1)
    if t.stride() != want:
        _explain(t, name, dtype, shape, want)
    return t.data_ptr()


def _place(stream):
    """The current device and the stream's handle."""
    dev = _current_device()
    if stream is None:
        return dev, _current_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream is on device {stream.device.index}, the current one is {dev}")
    return dev, stream.cuda_stream


def _turning(rope, D, stream):
    """_place, with a rotation that has to fit."""
    if not isinstance(rope, Rope):
        raise TypeError("rope must be what make_rope returns")
    if rope.D != D:
        raise ValueError(f"rope is of heads of {rope.D} elements, dims say {D}")
    dev, st = _place(stream)
    if rope._device != dev:
        raise ValueError(f"rope is on device {rope._device}, the current one is {dev}")
    return dev, st


def gdn_attn_rope(dims: KvDims, rope: Rope, q, k, v, seq_len, prefix_of, win_len, parent, positions, q_out, k_win, v_win,
                  stream=None) -> None:
    """Norms and rotation of windows (see include/gdn_kv.h): q [B, K, Hq, D], k, v [B, K, Hkv, D], of any even
    strides (k and v alike), to q_out, k_win and v_win; each may be None with its output, and each may be its
    output.  Positions follow from seq_len, prefix_of and parent as in gdn_attn_verify, or are given [B, K]."""
    d = dims
    lib = load_library()
    B, K, Hq, Hkv, D = d.B, d.K, d.Hq, d.Hkv, d.D
    dev, st = _turning(rope, D, stream)
    dt, qs, ks = _TORCH[d.dtype], (B, K, Hq, D), (B, K, Hkv, D)
    qp, qt, qh = (None, 0, 0) if q is None else _heads(q, "q", dt, qs, dev)
    kp, kt, kh = (None, 0, 0) if k is None else _heads(k, "k", dt, ks, dev)
    vp, kt, kh = _beside(k, kt, kh, v, dt, ks, dev)
    q_to = None if q_out is None else _out_rows(q_out, "q_out", dt, qs, d.q_token_stride, dev)
    k_to = None if k_win is None else _out_rows(k_win, "k_win", dt, ks, d.win_token_stride, dev)
    v_to = None if v_win is None or k_win is None else _like(v_win, dt, ks, k_win, dev)
    if v_to is None and v_win is not None:
        v_to = _out_rows(v_win, "v_win", dt, ks, d.win_token_stride, dev)
    _check(lib.gdn_attn_rope(
        ctypes.byref(d), rope._args((qt, qh, kt, kh)), *rope._at, qp, kp, vp,
        _arg(seq_len, "seq_len", _I32, (d.n_slots,), dev, True), _arg(prefix_of, "prefix_of", _I32, (B,), dev, True),
        _arg(win_len, "win_len", _I32, (B,), dev, True), _arg(parent, "parent", _I32, (B, K), dev, True),
        _arg(positions, "positions", _I32, (B, K), dev, True), q_to, k_to, v_to, st))


def gdn_kv_reserve(dims: KvDims, n_new, table_in, table_out, len_in, len_out, ref_in, ref_out, workspace, stream=None) -> None:
    """Pages for n_new [B] more tokens of each sequence, whose lengths grow by them.  Each *_out may be its *_in.
    len_out may be a pair of the lengths and of refused [n_slots] int32, -1 to begin with, in which the call notes the
    sequences that it had no room for; as a pair with seq_len, gdn_kv_append and gdn_attn_prefill leave those out."""
    d = dims
    lib = load_library()
    dev, st = _place(stream)
    table, slots, pages = (d.n_slots, d.max_pages), (d.n_slots,), (d.n_pages,)
    wp, wb = _workspace(workspace)
    _on_device(workspace, "workspace", dev)
    lens, refused = _lengths(len_out, "len_out", d.n_slots, dev)
    _check(lib.gdn_kv_reserve_marked(
        ctypes.byref(d), _arg(n_new, "n_new", _I32, (d.B,), dev), _arg(table_in, "table_in", _I32, table, dev),
        _arg(table_out, "table_out", _I32, table, dev), _arg(len_in, "len_in", _I32, slots, dev),
        lens, _arg(ref_in, "ref_in", _I32, pages, dev), _arg(ref_out, "ref_out", _I32, pages, dev), refused, wp, wb, st))


def gdn_kv_append(dims: KvDims, layer, rope: Rope, cu_seqlens, q, k, v, positions, k_cache, v_cache, page_table, seq_len,
                  prefix_of, q_out, stream=None) -> None:
    """One layer's packed tokens into place (see include/gdn_kv.h): q [N, Hq, D] to q_out (or both None), k, v
    [N, Hkv, D] to the last tokens of the slots.  cu_seqlens [B + 1]; positions [N] int32 or None.  seq_len may be a
    pair with what reserve refused: without it every sequence has to have got its room."""
    d = dims
    lib = load_library()
    Hq, Hkv, D = d.Hq, d.Hkv, d.D
    dev, st = _turning(rope, D, stream)
    dt = _TORCH[d.dtype]
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a tensor [tokens, Hkv, D]")
    N = k.shape[0]
    kc, vc = _cache(d, k_cache, v_cache)
    _on_device(k_cache, "k_cache", dev)
    _on_device(v_cache, "v_cache", dev)
    qp, qt, qh = (None, 0, 0) if q is None else _heads(q, "q", dt, (N, Hq, D), dev)
    kp, kt, kh = _heads(k, "k", dt, (N, Hkv, D), dev)
    vp, kt, kh = _beside(k, kt, kh, v, dt, (N, Hkv, D), dev)
    q_to = None if q_out is None else _out_rows(q_out, "q_out", dt, (N, Hq, D), d.q_token_stride, dev)
    lens, refused = _lengths(seq_len, "seq_len", d.n_slots, dev)
    _check(lib.gdn_kv_append_marked(
        ctypes.byref(d), layer, rope._args((qt, qh, kt, kh)), *rope._at, N, _arg(cu_seqlens, "cu_seqlens", _I32, (d.B + 1,), dev),
        qp, kp, vp, _arg(positions, "positions", _I32, (N,), dev, True), kc, vc,
        _arg(page_table, "page_table", _I32, (d.n_slots, d.max_pages), dev), lens, refused,
        _arg(prefix_of, "prefix_of", _I32, (d.B,), dev, True), q_to, st))


def gdn_attn_prefill_workspace_size(dims: KvDims, n_tokens: int) -> int:
    """Bytes of device scratch gdn_attn_prefill needs for these dims and n_tokens rows."""
    n = ctypes.c_uint64(0)
    _check(load_library().gdn_attn_prefill_workspace_size(ctypes.byref(dims), n_tokens, ctypes.byref(n)))
    return n.value


def alloc_attn_prefill_workspace(dims: KvDims, n_tokens: int, device="cuda") -> torch.Tensor:
    return torch.empty(gdn_attn_prefill_workspace_size(dims, n_tokens), dtype=torch.uint8, device=device)


def gdn_attn_prefill(dims: KvDims, layer, cu_seqlens, q, k_cache, v_cache, page_table, seq_len, prefix_of, causal, scale,
                     out, lse, workspace, stream=None) -> None:
    """Attention of packed queries over the cache (see include/gdn_kv.h): q [N, Hq, D], out [N, Hq, D], lse [N, Hq]
    f32 or None; cu_seqlens [B + 1].  causal: a sequence's rows are its slot's last tokens; else every row
    sees the whole slot.  seq_len may be a pair with what reserve refused."""
    d = dims
    lib = load_library()
    Hq, D = d.Hq, d.D
    dev, st = _place(stream)
    dt = _TORCH[d.dtype]
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [tokens, Hq, D]")
    N = q.shape[0]
    kc, vc = _cache(d, k_cache, v_cache)
    wp, wb = _workspace(workspace)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache"), (workspace, "workspace")):
        _on_device(t, name, dev)
    lens, refused = _lengths(seq_len, "seq_len", d.n_slots, dev)
    _check(lib.gdn_attn_prefill_marked(
        ctypes.byref(d), layer, N, _arg(cu_seqlens, "cu_seqlens", _I32, (d.B + 1,), dev),
        _out_rows(q, "q", dt, (N, Hq, D), d.q_token_stride, dev), kc, vc,
        _arg(page_table, "page_table", _I32, (d.n_slots, d.max_pages), dev), lens, refused,
        _arg(prefix_of, "prefix_of", _I32, (d.B,), dev, True), 1 if causal else 0, scale,
        _arg(out, "out", dt, (N, Hq, D), dev), _arg(lse, "lse", torch.float32, (N, Hq), dev, True), wp, wb, st))
