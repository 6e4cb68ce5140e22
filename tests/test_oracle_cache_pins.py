"""The cache oracle against the attention oracle and hand-made cases (CPU)."""

import numpy as np

import oracle.attention as A
import oracle.cache as C


def _qkv(rng, B, Hq, Hkv, T, L, D):
    return (rng.standard_normal((B, Hq, T, D)), rng.standard_normal((B, Hkv, L, D)),
            rng.standard_normal((B, Hkv, L, D)))


def test_chain_is_causal_attention():
    """Context + a chain of drafts is bottom-right causal attention over both."""
    rng = np.random.default_rng(0)
    B, Hq, Hkv, T, n, D = 2, 4, 2, 5, 7, 8
    q, kk, vv = _qkv(rng, B, Hq, Hkv, T, n + T, D)
    cache_k, cache_v = np.full((B, Hkv, n + 3, D), np.nan), np.full((B, Hkv, n + 3, D), np.nan)
    cache_k[:, :, :n], cache_v[:, :, :n] = kk[:, :, :n], vv[:, :, :n]
    o, lse, _ = C.tree_forward(q, cache_k, cache_v, kk[:, :, n:], vv[:, :, n:], [n] * B, None, None, 0.3)
    o_ref, lse_ref, _ = A.forward(q, kk, vv, 0.3, True)
    assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, lse_ref, atol=1e-12)


def test_weights_sum_to_rows():
    """Every row gives its keys a total weight of one."""
    rng = np.random.default_rng(1)
    B, Hq, Hkv, T, D = 1, 6, 2, 9, 4
    q, k, v = _qkv(rng, B, Hq, Hkv, T, T, D)
    _, lse, _ = A.forward(q, k, v, 0.5, True)
    w = C.key_weight(q, k, lse, 0.5, causal=True)
    assert np.allclose(w.sum(-1), (Hq // Hkv) * T)
    assert np.allclose(C.key_weight(q, k, lse, 0.5, limit=np.arange(1, T + 1)[None]), w)
    lse[:, :, 3] = np.inf
    assert np.allclose(C.key_weight(q, k, lse, 0.5, causal=True).sum(-1), (Hq // Hkv) * (T - 1))


def test_tree_rows_that_see_nothing():
    rng = np.random.default_rng(2)
    q, k, v = _qkv(rng, 1, 2, 1, 3, 3, 4)
    mask = np.array([[[0, 0, 0], [1, 1, 0], [0, 0, 1]]], dtype=np.uint8)
    o, lse, _ = C.tree_forward(q, k, v, k, v, [0], [2], mask, 1.0)
    assert np.isposinf(lse[:, :, 0]).all() and np.isposinf(lse[:, :, 2]).all() and (o[:, :, [0, 2]] == 0).all()
    assert np.isfinite(lse[:, :, 1]).all()


def test_append_and_evict_by_hand():
    k = np.arange(6.0).reshape(1, 1, 6, 1)
    pos = np.array([[[0, 1, 2, -1, -1, -1]]])
    new = np.array([10.0, 11.0, 12.0, 13.0]).reshape(1, 1, 4, 1)
    k2, _, pos2, n, seen, limit = C.append(new, new, k, k, [3], [3], np.array([[1, 3, 9, 0]]), [5], pos)
    assert k2.ravel().tolist() == [0, 1, 2, 11, 13, 5] and n.tolist() == [5] and seen.tolist() == [7]
    assert pos2.ravel().tolist() == [0, 1, 2, 5, 6, -1] and limit.tolist() == [[0, 4, 0, 5]]
    w = np.array([[[3.0, 1.0, 1.0, 0.5, 9.0, 0.0]]])
    pos3 = np.array([[[4, 0, 1, 2, 3, 5]]])
    # keep 4: the newest (pos 5, slot 5), then 9, 3 and the lower of the equal ones
    k3, _, wo, po, n3 = C.evict(k, k, w, pos3, [6], [6], 4, 1)
    assert k3.ravel().tolist() == [0, 1, 4, 5, 4, 5] and n3.tolist() == [4]
    assert po.ravel().tolist() == [4, 0, 3, 5, -1, -1] and wo.ravel().tolist() == [3, 1, 9, 0, 0, 0]
    w[0, 0, 1] = np.nan  # counts as the smallest
    assert C.evict(k, k, w, pos3, [6], [6], 4, 1)[3].ravel().tolist() == [4, 3, 1, 5, -1, -1]
