"""Plain float64 CPU implementation of the attention layers' prompt path (test infrastructure only): norms and
rotation, reserve, append, and attention of packed queries.

One token and one head at a time from the definitions in include/gdn_kv.h; it shares no code with the
CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .kv_oracle import ancestors, gather, pages_of


def turn(x, position, radians, interleaved=False, magnitude=1.0, weight=None, eps=0.0, weight_offset=0.0):
    """One head [D] at a position; radians [rot_dim / 2]."""
    y = np.array(x, dtype=np.float64)
    D, half = len(y), len(radians)
    if weight is not None:
        y = y / math.sqrt(sum(v * v for v in y) / D + eps) * (weight_offset + np.asarray(weight, dtype=np.float64))
    z = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # the angle modulo a turn, so that far positions lose nothing
        phi = math.fmod(float(position) * float(radians[i]), 2 * math.pi)
        c, s = math.cos(phi), math.sin(phi)
        z[a], z[b] = magnitude * (y[a] * c - y[b] * s), magnitude * (y[b] * c + y[a] * s)
    return z


def window_positions(seq_len, prefix_of, parent, B, K, slot0=0):
    pos = np.zeros((B, K), dtype=np.int64)
    for b in range(B):
        base = int(seq_len[slot0 + b]) + (int(seq_len[prefix_of[b]]) if prefix_of is not None and prefix_of[b] >= 0 else 0)
        for t in range(K):
            pos[b, t] = base + len(ancestors(None if parent is None else parent[b], t)) - 1
    return pos


def window(x, positions, win_len, weight, **how):
    """x [B, K, H, D] normed and rotated; 0 at padding tokens."""
    y = np.zeros(x.shape)
    for b in range(x.shape[0]):
        for t in range(x.shape[1] if win_len is None else int(win_len[b])):
            for h in range(x.shape[2]):
                y[b, t, h] = turn(x[b, t, h], positions[b, t], weight=weight, **how)
    return y


def reserve(n_new, table, seq_len, ref, page_size, slot0=0):
    """Copies of (table, seq_len, ref) with room for n_new tokens more."""
    table, seq_len, new_ref = table.copy(), seq_len.copy(), ref.copy()
    free = [p for p in range(len(ref)) if ref[p] == 0]
    wanted = 0
    for b, m in enumerate(n_new):
        s, n = slot0 + b, int(seq_len[slot0 + b])
        if m <= 0:
            continue
        have, want = pages_of(n, page_size), pages_of(n + int(m), page_size)
        if (n % page_size and ref[table[s, have - 1]] != 1) or want > table.shape[1]:
            continue
        first = wanted
        wanted += want - have
        if want > have and wanted > len(free):
            continue
        for i, c in enumerate(range(have, want)):
            table[s, c] = free[first + i]
            new_ref[free[first + i]] = 1
        seq_len[s] = n + int(m)
    return table, seq_len, new_ref


def append(cu, q, k, v, k_cache, v_cache, table, seq_len, prefix_of, q_out, positions, q_weight, k_weight, slot0=0, **how):
    """Copies of (q_out, k_cache, v_cache) of one layer, caches [n_pages, page_size, Hkv, D]."""
    q_out, k_cache, v_cache = q_out.copy(), k_cache.copy(), v_cache.copy()
    ps = k_cache.shape[1]
    for b in range(len(cu) - 1):
        s, lo, hi = slot0 + b, int(cu[b]), int(cu[b + 1])
        n = int(seq_len[s])
        if hi - lo > n:
            continue
        before = int(seq_len[prefix_of[b]]) if prefix_of is not None and prefix_of[b] >= 0 else 0
        for token in range(lo, hi):
            at = n - (hi - token)
            pos = at + before if positions is None else int(positions[token])
            page = table[s, at // ps]
            for h in range(q.shape[1]):
                q_out[token, h] = turn(q[token, h], pos, weight=q_weight, **how)
            for h in range(k.shape[1]):
                k_cache[page, at % ps, h] = turn(k[token, h], pos, weight=k_weight, **how)
                v_cache[page, at % ps, h] = v[token, h]
    return q_out, k_cache, v_cache


def attention(cu, q, k_cache, v_cache, table, seq_len, prefix_of, causal, scale, slot0=0):
    """out [N, Hq, D] and lse [N, Hq] of packed queries; NaN in rows that no sequence holds."""
    N, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    out, lse = np.full((N, Hq, D), math.nan), np.full((N, Hq), math.nan)
    for b in range(len(cu) - 1):
        s, lo, hi = slot0 + b, int(cu[b]), int(cu[b + 1])
        p = prefix_of[b] if prefix_of is not None else -1
        pre_k, pre_v = (gather(c, table[p], int(seq_len[p])) if p >= 0 else np.zeros((0,) + c.shape[2:]) for c in (k_cache, v_cache))
        own_k, own_v = (gather(c, table[s], int(seq_len[s])) for c in (k_cache, v_cache))
        for token in range(lo, hi):
            n = int(seq_len[s])
            if causal:
                n = max(0, n - (hi - token) + 1)
            k, v = np.concatenate([pre_k, own_k[:n]]), np.concatenate([pre_v, own_v[:n]])
            for h in range(Hq):
                if len(k) == 0:
                    out[token, h], lse[token, h] = 0.0, -math.inf
                    continue
                x = scale * (k[:, h // G] @ q[token, h])
                m = x.max()
                e = np.exp(x - m)
                lse[token, h] = m + math.log(e.sum())
                out[token, h] = (e / e.sum()) @ v[:, h // G]
    return out, lse
