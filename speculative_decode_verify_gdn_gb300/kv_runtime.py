"""Device-resident paged cache of a hybrid model's softmax-attention layers, and its part of the
verify round (attend -> commit, fork, compact).

Torch allocates the memory; every step runs through the C ABI (include/gdn_kv.h).  The slots are
the batch's sequences, 0..B-1, and behind them the shared prefixes.  Tables, lengths and
reference counts are updated in place except by a fork, which writes the other one of two sets.

Every method takes the stream that it runs on (None: the current one).  What it allocates for
itself belongs to that stream; the caller's tensors and the cache have to be ready there, as for the
C calls.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

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
    attn_workspace: torch.Tensor
    pool_workspace: torch.Tensor
    fork_scratch: tuple
    cur: int = 0

    @classmethod
    def create(cls, B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_prefixes=0, n_layers=1, dtype=torch.bfloat16,
               device="cuda") -> "PagedCache":
        n_slots = B + n_prefixes
        dims = kv.make_kv_dims(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_slots, 0, n_layers, dtype)
        shape = (n_layers, n_pages, page_size, Hkv, D)

        def ints(*s, fill=0):
            return torch.full(s, fill, dtype=torch.int32, device=device)

        return cls(B, K, Hq, Hkv, D, page_size, n_pages, max_pages, n_prefixes, n_layers, dtype,
                   torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   [ints(n_slots, max_pages, fill=-1) for _ in range(2)], [ints(n_slots) for _ in range(2)],
                   ints(n_pages), ints(B, fill=-1), ints(1), dims, kv.alloc_attn_workspace(dims, device),
                   kv.alloc_kv_workspace(dims, device),
                   (ints(B), torch.empty(B, dtype=torch.bool, device=device), ints(B),
                    torch.arange(B, dtype=torch.int32, device=device), ints(n_slots, fill=-1)))

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

    def attend(self, layer, q, k_win, v_win, out, lse=None, parent=None, win_len=None, scale=None, stream=None) -> None:
        """The window's attention in one layer (a chain, or a token tree given by parent [B, K])."""
        kv.gdn_attn_verify(self.dims, layer, q, k_win, v_win, self.k, self.v, self.table, self.seq_len,
                           self.prefix_of if self.n_prefixes else None, win_len, parent,
                           1.0 / math.sqrt(self.D) if scale is None else scale, out, lse, self.attn_workspace, stream)

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
        if self.n_prefixes:
            with torch.cuda.stream(stream):
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
