"""Device-resident paged cache of a hybrid model's softmax-attention layers, and its part of the
verify round (rope -> attend -> commit, fork, compact) and of prompts (reserve, then layer by layer
append_layer -> attend_prefill).

Torch allocates the memory; every step runs through the C ABI (include/gdn_kv.h).  The slots are
the batch's sequences, 0..B-1, and behind them the shared prefixes.  Tables, lengths and
reference counts are updated in place except by a fork, which writes the other one of two sets.

Every method takes the stream that it runs on (None: the current one).  What it allocates for
itself belongs to that stream; the caller's tensors and the cache have to be ready there, as for the
C calls.  The two attentions only read the cache, and may run on several streams at once: each stream has a workspace for
them, made by its first call, and a captured call has one in its graph's own memory.  What changes the cache
runs alone.
"""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

from . import kv


@dataclass
class PagedCache:
    B: int
    K: int
    Hq: int
    Hkv: int
    D: int
    page_size: int
    n_pages: int
    max_pages: int
    n_prefixes: int
    n_layers: int
    dtype: torch.dtype
    k: torch.Tensor           # [n_layers, n_pages, page_size, Hkv, D]
    v: torch.Tensor
    tables: list              # two [n_slots, max_pages] int32
    lens: list                # two [n_slots] int32
    ref: torch.Tensor         # [n_pages] int32
    prefix_of: torch.Tensor   # [B] int32: slot of the sequence's prefix, -1 without
    n_live: torch.Tensor      # [1] int32, set by compact
    dims: kv.KvDims
    pool_workspace: torch.Tensor
    fork_scratch: tuple
    refused: torch.Tensor     # [n_slots] int32: length of a slot that reserve had no room for, else -1
    cur: int = 0
    reserved: bool = False    # some reserve has written refused
    workspaces: dict = field(default_factory=dict)  # of the attentions: (which, stream) -> tensor

    @classmethod
    def create(cls, B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_prefixes=0, n_layers=1, dtype=torch.bfloat16,
               device="cuda") -> "PagedCache":
        n_slots = B + n_prefixes
        dims = kv.make_kv_dims(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_slots, 0, n_layers, dtype)
        kv.gdn_attn_workspace_size(dims)  # (refuses here what the attention would refuse later)
        shape = (n_layers, n_pages, page_size, Hkv, D)

        def ints(*s, fill=0):
            return torch.full(s, fill, dtype=torch.int32, device=device)

        return cls(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_prefixes, n_layers, dtype,
                   torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   [ints(n_slots, max_pages, fill=-1) for _ in range(2)], [ints(n_slots) for _ in range(2)],
                   ints(n_pages), ints(B, fill=-1), ints(1), dims,
                   kv.alloc_kv_workspace(kv.make_kv_dims(min(n_slots, kv.MAX_BATCH), K, Hq, Hkv, D, page_size, n_pages, max_pages,
                                                         n_slots, 0, n_layers, dtype), device),  # (reserve takes any of the slots)
                   (ints(B), torch.empty(B, dtype=torch.bool, device=device), ints(B),
                    torch.arange(B, dtype=torch.int32, device=device), ints(n_slots, fill=-1)),
                   ints(n_slots, fill=-1))

    @property
    def table(self) -> torch.Tensor:
        return self.tables[self.cur]

    @property
    def seq_len(self) -> torch.Tensor:
        return self.lens[self.cur]

    def append(self, slot, k_new, v_new, stream=None) -> None:
        """Adds N tokens [n_layers, N, Hkv, D] to one slot: a prompt, or a shared prefix."""
        n = k_new.shape[1]
        d = kv.make_kv_dims(1, n, self.Hq, self.Hkv, self.D, self.page_size, self.n_pages, self.max_pages,
                            self.B + self.n_prefixes, slot, self.n_layers, self.dtype, win=k_new.unsqueeze(1))
        with torch.cuda.stream(stream):  # (what the call allocates belongs to the stream it runs on)
            all_of_it = torch.full((1,), n, dtype=torch.int32, device=k_new.device)
            kv.gdn_kv_commit(d, all_of_it, None, k_new.unsqueeze(1), v_new.unsqueeze(1), self.k, self.v, self.table,
                             self.table, self.seq_len, self.seq_len, self.ref, self.ref,
                             kv.alloc_kv_workspace(d, k_new.device), stream)

    def rope(self, rope, q, k, v, q_out, k_win, v_win, parent=None, win_len=None, positions=None, stream=None) -> None:
        """One layer's window [B, K, heads, D] ready for attend and commit: queries and keys normed and rotated
        (kv.make_rope) at their positions behind prefix and slot, values copied.  q, k, v may be parts of a
        projection's rows, and each output its input."""
        kv.gdn_attn_rope(self._dims(self.B, q=q_out, win=k_win if k_win is not None else v_win), rope, q, k, v, self.seq_len,
                         self._prefixes(0, self.B), win_len, parent, positions, q_out, k_win, v_win, stream)

    def reserve(self, n_new, slot0=0, stream=None) -> None:
        """Pages for n_new (int32) more tokens of the sequences from slot0 on, in all layers, which grow by them;
        append_layer fills them.  A sequence that there is no room for (gdn_device_status) stays as it is, and
        append_layer and causal attend_prefill leave it out until its slot has grown or has been asked for again."""
        self.reserved = True
        kv.gdn_kv_reserve(self._dims(n_new.shape[0], slot0), n_new, self.table, self.table, self.seq_len,
                          (self.seq_len, self.refused), self.ref, self.ref, self.pool_workspace, stream)

    def append_layer(self, layer, rope, cu_seqlens, q, k, v, q_out, slot0=0, positions=None, stream=None) -> None:
        """One layer's packed tokens of the sequences from slot0 on, with bounds cu_seqlens (int32), to the places
        that reserve made for them: q [N, Hq, D] normed and rotated to q_out (both may be None), k normed and
        rotated, and v, [N, Hkv, D], to the pages."""
        n = cu_seqlens.shape[0] - 1
        kv.gdn_kv_append(self._dims(n, slot0, q=q_out), layer, rope, cu_seqlens, q, k, v, positions, self.k, self.v, self.table,
                         (self.seq_len, self.refused), self._prefixes(slot0, n), q_out, stream)

    def attend_prefill(self, layer, cu_seqlens, q, out, lse=None, slot0=0, causal=True, scale=None, stream=None) -> None:
        """Packed queries [N, Hq, D] of the sequences from slot0 on attend to prefix and slot: causally, a
        sequence's queries being those of its last tokens, or to all of the slot (cross attention)."""
        n = cu_seqlens.shape[0] - 1
        kv.gdn_attn_prefill(self._dims(n, slot0, q=q), layer, cu_seqlens, q, self.k, self.v, self.table,
                            (self.seq_len, self.refused), self._prefixes(slot0, n), causal,
                            1.0 / math.sqrt(self.D) if scale is None else scale, out, lse,
                            self._workspace(kv.alloc_attn_prefill_workspace, 0, stream=stream), stream)

    def _workspace(self, alloc, *args, stream=None) -> torch.Tensor:
        """Scratch of an attention that runs on this stream.  Eager calls on one stream come one after the other and share
        theirs; graphs that were captured on one stream may be replayed on two at once, so each has its own."""
        if not self.k.is_cuda:
            return alloc(self.dims, *args, self.k.device)
        handle, captured = kv.stream_state(stream)
        ws = None if captured else self.workspaces.get((alloc.__name__, handle))
        if ws is None:
            with torch.cuda.stream(stream):
                ws = alloc(self.dims, *args, self.k.device)
            if not captured:
                self.workspaces[alloc.__name__, handle] = ws
        return ws

    def _dims(self, n, slot0=0, q=None, win=None) -> kv.KvDims:
        """The dims of a call on n sequences from slot0 on, with these queries' and windows' strides."""
        return kv.make_kv_dims(n, self.K, self.Hq, self.Hkv, self.D, self.page_size, self.n_pages, self.max_pages,
                               self.B + self.n_prefixes, slot0, self.n_layers, self.dtype, q=q, win=win)

    def _prefixes(self, slot0, n):
        """Prefixes of the sequences from slot0 on (the prefixes' own slots have none)."""
        if not self.n_prefixes or slot0 >= self.B:
            return None
        if slot0 + n > self.B:
            raise ValueError(f"slots {slot0}..{slot0 + n - 1} are sequences and prefixes (from {self.B} on): one call for each")
        return self.prefix_of[slot0:slot0 + n]

    def attend(self, layer, q, k_win, v_win, out, lse=None, parent=None, win_len=None, scale=None, stream=None) -> None:
        """The window's attention in one layer (a chain, or a token tree given by parent [B, K])."""
        kv.gdn_attn_verify(self.dims, layer, q, k_win, v_win, self.k, self.v, self.table, self.seq_len,
                           self.prefix_of if self.n_prefixes else None, win_len, parent,
                           1.0 / math.sqrt(self.D) if scale is None else scale, out, lse,
                           self._workspace(kv.alloc_attn_workspace, stream=stream), stream)

    def commit(self, accept_len, k_win, v_win, parent=None, stream=None) -> None:
        """Keeps each sequence's accepted window tokens, all layers: k_win, v_win [n_layers, B, K, Hkv, D]."""
        kv.gdn_kv_commit(self.dims, accept_len, parent, k_win, v_win, self.k, self.v, self.table, self.table,
                         self.seq_len, self.seq_len, self.ref, self.ref, self.pool_workspace, stream)

    def fork(self, src, stream=None) -> None:
        """Sequence i goes on from sequence src[i], behind that one's prefix (src [n_slots] int32; prefixes
        keep their slots by src[s] = s); -1 drops it and leaves its entry of prefix_of.  A sequence that
        goes on from a prefix's own slot has that as its tokens, and none behind them."""
        i, o = self.cur, 1 - self.cur
        kv.gdn_kv_fork(self.dims, src, self.k, self.v, self.tables[i], self.tables[o], self.lens[i], self.lens[o],
                       self.ref, self.ref, self.pool_workspace, stream)
        self.cur = o
        if self.reserved and stream is None and not self.n_prefixes:  # (without a context: 9 us of the host's for 13)
            self.refused.fill_(-1)
        elif self.n_prefixes or self.reserved:
            with torch.cuda.stream(stream):
                if self.reserved:
                    self.refused.fill_(-1)  # (the slots hold other sequences now)
                if self.n_prefixes:
                    self._take_prefixes(src[:self.B])

    def _take_prefixes(self, src) -> None:
        """prefix_of of the slots that src names.  Five small kernels into buffers of the cache: 80 us of the
        host's time (160 with every intermediate result a tensor of its own); nothing without prefixes."""
        in_range, known, at, own, rows = self.fork_scratch
        torch.clamp(src, 0, self.B + self.n_prefixes - 1, out=in_range)
        torch.eq(in_range, src, out=known)
        torch.where(known, src, own, out=at)        # (no slot: its own entry)
        rows[:self.B].copy_(self.prefix_of)         # (behind them, the prefixes' slots: -1)
        torch.index_select(rows, 0, at, out=self.prefix_of)

    def compact(self, stream=None) -> None:
        """Moves the live pages to the front of the pool; their number goes to n_live."""
        kv.gdn_kv_compact(self.dims, self.k, self.v, self.table, self.table, self.seq_len, self.ref, self.ref,
                          self.n_live, self.pool_workspace, stream)
