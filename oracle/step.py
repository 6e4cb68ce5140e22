"""fp64 CPU oracle for the calls around attention in a model step: norm and
rotation of queries and keys (forward and backward), the paged cache
(quantising, reading back, attention over it), verification of drafts.

TEST INFRASTRUCTURE ONLY, written as the plain definitions; it shares no code
with the CUDA kernels.  Arrays are numpy: 16-bit inputs decoded exactly to
float64, lengths, pages and tokens as integers.
"""

from __future__ import annotations

import numpy as np

EXP_MIN, EXP_MAX = -64, 120


# --- norm and rotation -------------------------------------------------------


def angles(pos, freq, axis):
    """[B, L, rot/2] from pos [axes, B, L], freq [rot/2], axis [rot/2] or None."""
    pos = np.asarray(pos, dtype=np.float64)
    a = np.zeros(len(freq), dtype=int) if axis is None else np.minimum(np.asarray(axis, dtype=int), len(pos) - 1)
    return np.stack([pos[a[i]] * float(freq[i]) for i in range(len(freq))], -1)


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, ang, interleaved):
    """Rows x [B, H, L, D] turned by ang [B, L, rot/2]."""
    one, two = _pairs(2 * ang.shape[-1], interleaved)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def pair_mag(x, rot, interleaved):
    """|a| + |b| of each element's pair (|x| where it has none): what a rotation's rounding errors are measured on."""
    one, two = _pairs(rot, interleaved)
    m = np.abs(x)
    m[..., one] = m[..., two] = np.abs(x[..., one]) + np.abs(x[..., two])
    return m


def norm_rope(x, w, eps, ang, interleaved):
    """The output, and the normed row."""
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(n, ang, interleaved), n


def norm_rope_bwd(x, w, eps, dy, ang, interleaved):
    """dx, dw (None without w) and the rounding-error measures: of dx, of dw, with `eg` a bound per element of g's own error factored out."""
    g = rotate(dy, -ang, interleaved)
    if w is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1, 2))
    t = g * w
    return r * (t - x * r * r * (t * x).mean(-1, keepdims=True)), dw


# --- the paged cache ---------------------------------------------------------


def quantise(x):
    """Codes (as values) and exponents of rows [..., D]."""
    fine = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = fine.max(-1)
    e = np.full(top.shape, EXP_MIN, dtype=np.int64)
    for i in np.ndindex(top.shape):
        while e[i] < EXP_MAX and top[i] > 448.0 * 2.0 ** float(e[i]):
            e[i] += 1
    y = np.where(np.isfinite(x), x, 0.0) / 2.0 ** e[..., None].astype(np.float64)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    c = np.round(y / step) * step  # ties to the even multiple
    return np.where(np.isfinite(x), np.clip(c, -448, 448), np.nan), e


def place(table, page_size, n_pages, b, j):
    """(page, row) of token j of sequence b, None for a hole."""
    p = int(table[b][j // page_size])
    return (p, j % page_size) if 0 <= p < n_pages else None


def tokens_of(pool, exp, table, page_size, b, n):
    """Values [Hkv, n, D] of the first n tokens and which of them are there [n]."""
    n_pages, H, _, D = pool.shape
    out, there = np.zeros((H, n, D)), np.zeros(n, dtype=bool)
    for j in range(n):
        at = place(table, page_size, n_pages, b, j)
        if at is None:
            continue
        there[j] = True
        out[:, j] = pool[at[0], :, at[1]]
        if exp is not None:
            out[:, j] *= 2.0 ** exp[at[0], :, at[1]].astype(np.float64)[:, None]
    return out, there


def paged_attention(q, k, v, ke, ve, table, page_size, cache_len, scale):
    """O, base-2 lse, and sum_j P_j |V_j| [B, Hq, T, D]."""
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    room = len(table[0]) * page_size
    o, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((B, Hq, T), np.inf)
    for b in range(B):
        n = int(np.clip(cache_len[b], 0, room))
        kk, there = tokens_of(k, ke, table, page_size, b, n)
        vv, _ = tokens_of(v, ve, table, page_size, b, n)
        for t in range(T):
            see = np.flatnonzero(there & (np.arange(n) <= n - T + t))
            if len(see) == 0:
                continue
            for h in range(Hq):
                hk = h * Hkv // Hq
                s = scale * (kk[hk, see] @ q[b, h, t])
                top = s.max()
                p = np.exp(s - top)
                o[b, h, t] = p @ vv[hk, see] / p.sum()
                mag[b, h, t] = p @ np.abs(vv[hk, see]) / p.sum()
                lse[b, h, t] = (top + np.log(p.sum())) / np.log(2.0)
    return o, lse, mag


# --- verification ------------------------------------------------------------


def fixed(x):
    """Probabilities as integers, the nearest multiples of 2^-45."""
    x = np.minimum(np.where(np.isnan(x) | (x < 0), 0.0, np.asarray(x, dtype=np.float64)), 1.0)
    return [int(v) for v in np.rint(x * 2.0 ** 45)]


def verify(target, draft, tokens, u, r, draft_len=None):
    """accept_len and token, exact."""
    B, T = tokens.shape
    V = target.shape[-1]
    accept, token = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in range(B):
        most = T if draft_len is None else int(np.clip(draft_len[b], 0, T))
        n = 0
        while n < most:
            x = int(tokens[b, n])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, n, x])
            if not float(u[b, n]) * q < float(target[b, n, x]):
                break
            n += 1
        w = p = fixed(target[b, n])
        if n < most:
            if draft is None:
                w = [0 if i == int(tokens[b, n]) else a for i, a in enumerate(p)]
            else:
                w = [max(a - c, 0) for a, c in zip(p, fixed(draft[b, n]))]
            w = w if sum(w) else p
        limit = int(min(max(float(r[b]), 0.0), 1.0) * 2.0 ** 64)
        limit = min(limit, 2 ** 64 - 1) * sum(w) >> 64
        accept[b], token[b] = n, -1
        run = 0
        for i, a in enumerate(w):
            run += a
            if run > limit:
                token[b] = i
                break
    return accept, token
