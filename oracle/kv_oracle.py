"""Plain float64 CPU implementation of the paged key/value cache calls (test infrastructure only).

One sequence, one row, one key at a time from the definitions in include/gdn_kv.h; it shares no
code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np


def pages_of(n: int, page_size: int) -> int:
    return -(-n // page_size)


def gather(cache, table_row, n: int) -> np.ndarray:
    """The first n tokens [n, Hkv, D] of a slot; cache [n_pages, page_size, Hkv, D]."""
    ps = cache.shape[1]
    if n == 0:
        return np.zeros((0,) + cache.shape[2:])
    return np.concatenate([cache[table_row[c]] for c in range(pages_of(n, ps))])[:n]


def ancestors(parent, t: int) -> list:
    """Node t's path from the root down to t (parent None: a chain)."""
    path = []
    while t >= 0:
        path.append(t)
        t = t - 1 if parent is None else int(parent[t])
    return path[::-1]


def attention(q, k_win, v_win, k_cache, v_cache, table, seq_len, prefix_of, win_len, parent, scale, slot0=0):
    """out [B, K, Hq, D] and lse [B, K, Hq]; q [B, K, Hq, D], windows [B, K, Hkv, D], one layer's caches."""
    B, K, Hq, D = q.shape
    G = Hq // k_win.shape[2]
    out = np.zeros((B, K, Hq, D))
    lse = np.full((B, K, Hq), -math.inf)
    for b in range(B):
        s = slot0 + b
        keys, values = [], []
        if prefix_of is not None and prefix_of[b] >= 0:
            p = prefix_of[b]
            keys.append(gather(k_cache, table[p], seq_len[p]))
            values.append(gather(v_cache, table[p], seq_len[p]))
        keys.append(gather(k_cache, table[s], seq_len[s]))
        values.append(gather(v_cache, table[s], seq_len[s]))
        for t in range(K if win_len is None else win_len[b]):
            path = ancestors(None if parent is None else parent[b], t)
            k = np.concatenate(keys + [k_win[b, path]])
            v = np.concatenate(values + [v_win[b, path]])
            for h in range(Hq):
                x = scale * (k[:, h // G] @ q[b, t, h])
                m = x.max()
                e = np.exp(x - m)
                lse[b, t, h] = m + math.log(e.sum())
                out[b, t, h] = (e / e.sum()) @ v[:, h // G]
    return out, lse


def commit(accept_len, parent, k_win, v_win, k_cache, v_cache, table, seq_len, ref, page_size, slot0=0):
    """Copies of (k_cache, v_cache, table, seq_len, ref) after the commit; windows
    [n_layers, B, K, Hkv, D], caches [n_layers, n_pages, page_size, Hkv, D]."""
    k_cache, v_cache, table, seq_len = k_cache.copy(), v_cache.copy(), table.copy(), seq_len.copy()
    new_ref = ref.copy()
    free = [p for p in range(len(ref)) if ref[p] == 0]
    wanted = 0
    B, K = k_win.shape[1:3]
    for b in range(B):
        s = slot0 + b
        L, n = int(accept_len[b]), int(seq_len[s])
        if L < 1 or L > K:
            continue
        path = ancestors(None if parent is None else parent[b], L - 1)
        have, want = pages_of(n, page_size), pages_of(n + len(path), page_size)
        if n % page_size and ref[table[s, have - 1]] != 1:
            continue
        if want > table.shape[1]:
            continue
        first = wanted
        wanted += want - have
        if want > have and wanted > len(free):
            continue
        for i, c in enumerate(range(have, want)):
            table[s, c] = free[first + i]
            new_ref[free[first + i]] = 1
        for r, t in enumerate(path):
            at = n + r
            k_cache[:, table[s, at // page_size], at % page_size] = k_win[:, b, t]
            v_cache[:, table[s, at // page_size], at % page_size] = v_win[:, b, t]
        seq_len[s] = n + len(path)
    return k_cache, v_cache, table, seq_len, new_ref


def fork(src, k_cache, v_cache, table, seq_len, ref, page_size):
    """Copies of (k_cache, v_cache, table, seq_len, ref) after the fork."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    new_table, new_len, new_ref = np.full_like(table, -1), np.zeros_like(seq_len), ref.copy()
    free = [p for p in range(len(ref)) if ref[p] == 0]
    taken = set()
    for i, s in enumerate(src):
        if s < 0:
            continue
        n = int(seq_len[s])
        first = s not in taken
        taken.add(s)
        if first or n % page_size == 0:
            new_table[i], new_len[i] = table[s], n
            if not first:
                for c in range(n // page_size):
                    new_ref[table[s, c]] += 1
            continue
        if not free:
            continue
        new_table[i], new_len[i] = table[s], n
        for c in range(n // page_size):
            new_ref[table[s, c]] += 1
        page, old, fill = free.pop(0), table[s, n // page_size], n % page_size
        new_table[i, n // page_size] = page
        new_ref[page] = 1
        k_cache[:, page, :fill] = k_cache[:, old, :fill]
        v_cache[:, page, :fill] = v_cache[:, old, :fill]
    for s in range(len(seq_len)):
        if s not in taken:
            for c in range(pages_of(int(seq_len[s]), page_size)):
                new_ref[table[s, c]] -= 1
    return k_cache, v_cache, new_table, new_len, new_ref


def compact(k_cache, v_cache, table, seq_len, ref, page_size):
    """Copies of (k_cache, v_cache, table, ref) after compaction, and the number of live pages."""
    k_cache, v_cache, table, new_ref = k_cache.copy(), v_cache.copy(), table.copy(), ref.copy()
    live = int((ref > 0).sum())
    holes = [p for p in range(live) if ref[p] == 0]
    movers = [p for p in range(live, len(ref)) if ref[p] > 0]
    new = {}
    for a, b in zip(movers, holes):
        k_cache[:, b], v_cache[:, b] = k_cache[:, a], v_cache[:, a]
        new_ref[b], new_ref[a] = ref[a], 0
        new[a] = b
    for s in range(len(seq_len)):
        for c in range(pages_of(int(seq_len[s]), page_size)):
            table[s, c] = new.get(int(table[s, c]), table[s, c])
    return k_cache, v_cache, table, new_ref, live
