"""fp64 CPU oracle for the cache calls: drafted-token attention over a cache,
appending accepted drafts, accumulated key weights, eviction.

TEST INFRASTRUCTURE ONLY, written as the plain definitions (no tiles, no
online softmax); it shares no code with the CUDA kernels.  Arrays are numpy:
16-bit inputs decoded exactly to float64, lengths and indices as integers.
"""

from __future__ import annotations

import numpy as np

LOG2E = 1.0 / np.log(2.0)


def chain_mask(B: int, T: int) -> np.ndarray:
    return np.broadcast_to(np.tril(np.ones((T, T), dtype=np.uint8)), (B, T, T))


def tree_forward(q, k, v, k_new, v_new, cache_len, tree_len, mask, scale):
    """O [B,Hq,T,D], base-2 lse [B,Hq,T], and A [B,Hq,T,D] = sum_j P_j |V_j|,
    the scale that rounding errors of P are measured on.  mask None: chain;
    tree_len None: T.  Rows past tree_len and rows that see nothing: O = 0,
    lse = +inf."""
    B, Hq, T, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    G = Hq // Hkv
    if mask is None:
        mask = chain_mask(B, T)
    o, mag = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T, D))
    lse = np.full((B, Hq, T), np.inf)
    for b in range(B):
        n = int(np.clip(cache_len[b], 0, Lk))
        m = T if tree_len is None else int(np.clip(tree_len[b], 0, T))
        for h in range(Hq):
            hk = h // G
            for t in range(m):
                seen = np.flatnonzero(mask[b, t, :m])
                keys = np.concatenate([k[b, hk, :n], k_new[b, hk, seen]])
                vals = np.concatenate([v[b, hk, :n], v_new[b, hk, seen]])
                if len(keys) == 0:
                    continue
                s = scale * (keys @ q[b, h, t])
                top = s.max()
                p = np.exp(s - top)
                tot = p.sum()
                o[b, h, t] = (p / tot) @ vals
                mag[b, h, t] = (p / tot) @ np.abs(vals)
                lse[b, h, t] = (top + np.log(tot)) * LOG2E
    return o, lse, mag


def key_weight(q, k, lse, scale, causal=False, limit=None):
    """[B,Hkv,Lk]: sum over the group's query heads and the rows that see key j of exp2(scale log2e q.k - lse)."""
    B, Hq, Lq, _ = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = np.zeros((B, Hkv, Lk))
    j = np.arange(Lk)[None, :]
    for b in range(B):
        if limit is not None:
            lim = np.clip(limit[b], 0, Lk)
        else:
            lim = np.arange(Lq) + (Lk - Lq) + 1 if causal else np.full(Lq, Lk)
        for h in range(Hq):
            x = scale * LOG2E * (q[b, h] @ k[b, h // G].T) - lse[b, h][:, None]
            out[b, h // G] += np.where(j < lim[:, None], np.exp2(np.where(j < lim[:, None], x, -np.inf)), 0.0).sum(0)
    return out


def append(k_new, v_new, k, v, cache_len, accept_len, path, seen, pos):
    """Copies of k, v, pos with the accepted drafts in, new lengths, new seen and the key limits [B,T]."""
    B, Hkv, T = k_new.shape[:3]
    Lk = k.shape[2]
    k, v, pos = k.copy(), v.copy(), pos.copy()
    new_len, new_seen = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    limit = np.zeros((B, T), dtype=np.int64)
    for b in range(B):
        at = int(np.clip(cache_len[b], 0, Lk))
        n = T if accept_len is None else int(np.clip(accept_len[b], 0, T))
        rows = []
        for i in range(min(n, Lk - at)):
            r = i if path is None else int(path[b, i])
            if not 0 <= r < T:
                break
            rows.append(r)
        for i, r in enumerate(rows):
            k[b, :, at + i], v[b, :, at + i] = k_new[b, :, r], v_new[b, :, r]
            pos[b, :, at + i] = seen[b] + i
            limit[b, r] = at + i + 1
        new_len[b], new_seen[b] = at + len(rows), seen[b] + len(rows)
    return k, v, pos, new_len, new_seen, limit


def evict(k, v, weight, pos, cache_len, seen, keep, recent):
    """Copies of k, v after the eviction, weight_out, pos_out, new lengths."""
    B, Hkv, Lk = weight.shape
    k, v = k.copy(), v.copy()
    w_out, p_out = np.zeros_like(weight), np.full_like(pos, -1)
    new_len = np.zeros(B, dtype=np.int64)
    for b in range(B):
        n = int(np.clip(cache_len[b], 0, Lk))
        new_len[b] = min(n, keep)
        for h in range(Hkv):
            slots = list(range(n))
            if n > keep:
                def order(j):
                    late = int(pos[b, h, j]) >= int(seen[b]) - recent
                    w = weight[b, h, j]
                    return (not late, 0.0 if late else (np.inf if np.isnan(w) else -w), np.isnan(w) and not late, j)

                stay = sorted(sorted(range(n), key=order)[:keep])
                inside = set(stay)
                free = [j for j in range(keep) if j not in inside]
                move = [j for j in stay if j >= keep]
                slots = list(range(keep))
                for f, m in zip(free, move):
                    slots[f] = m
                    k[b, h, f], v[b, h, f] = k[b, h, m], v[b, h, m]
            for s, j in enumerate(slots):
                w_out[b, h, s], p_out[b, h, s] = weight[b, h, j], pos[b, h, j]
    return k, v, w_out, p_out, new_len
