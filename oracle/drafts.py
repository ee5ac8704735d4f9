"""Drafted tokens over the paged cache: trees of guesses that one step checks.

Sequence s has m_s drafted tokens in rows cu_s .. of a batch, its length n_s with
them, ctx_s = n_s - m_s. Token i has slot ctx_s + i; its parent is the drafted token
parents[cu_s + i] of its sequence, or the last cached token (-1). Its ancestors are
what its parents lead to; with depth(i) of them its position is ctx_s + depth(i). It
attends to the ctx_s cached tokens, its ancestors and itself. Accepting a path puts
its i-th token into slot ctx_s + i.

Test infrastructure only.
"""
import numpy as np

from .serving import gather_cache, rope_rotate


def chain(m):
    return [i - 1 for i in range(m)]


def path(tree, i):
    """Token i and its ancestors, the oldest first."""
    out = []
    while i >= 0:
        out.append(i)
        i = tree[i]
    return out[::-1]


def visible(tree):
    """[m, m] whether token i sees token j."""
    m = len(tree)
    out = np.zeros((m, m), dtype=bool)
    for i in range(m):
        out[i, path(tree, i)] = True
    return out


def tree_attention(q, k_pool, v_pool, table, cu, lens, trees):
    """q [T, nq, d] -> o [T, nq, d], lse [T, nq] (NaN in rows of no sequence), and for
    error bounds sum p |v| and max_j sum |q k| / sqrt(d)."""
    T, nq, d = q.shape
    g = nq // k_pool.shape[2]
    o, lse = np.full((T, nq, d), np.nan), np.full((T, nq), np.nan)
    a, mx = np.zeros((T, nq, d)), np.zeros((T, nq))
    for s, n in enumerate(lens):
        m = cu[s + 1] - cu[s]
        if n == 0 or m == 0:
            continue
        seen = np.concatenate([np.ones((m, n - m), dtype=bool), visible(trees[s])], axis=1)
        k, v = gather_cache(k_pool, table[s], n), gather_cache(v_pool, table[s], n)
        for h in range(nq):
            x = q[cu[s]:cu[s + 1], h]
            kh, vh = k[:, h // g], v[:, h // g]
            sc = np.where(seen, x @ kh.T / np.sqrt(d), -np.inf)
            top = sc.max(axis=1, keepdims=True)
            e = np.exp(sc - top)
            p = e / e.sum(axis=1, keepdims=True)
            o[cu[s]:cu[s + 1], h] = p @ vh
            lse[cu[s]:cu[s + 1], h] = (top + np.log(e.sum(axis=1, keepdims=True)))[:, 0]
            a[cu[s]:cu[s + 1], h] = p @ np.abs(vh)
            mx[cu[s]:cu[s + 1], h] = (np.abs(x) @ np.abs(kh).T).max(axis=1) / np.sqrt(d)
    return o, lse, a, mx


def append_tree(q, k, v, cu, lens, trees, rope, interleaved, table, k_pool, v_pool):
    """As serving.kv_append, the rotation by depth."""
    q, k = np.array(q, dtype=np.float64), np.array(k, dtype=np.float64)
    k_pool, v_pool = np.array(k_pool, dtype=np.float64), np.array(v_pool, dtype=np.float64)
    page = k_pool.shape[1]
    for s, n in enumerate(lens):
        m = cu[s + 1] - cu[s]
        if n == 0:
            continue
        for i in range(m):
            t, pos, slot = cu[s] + i, n - m + len(path(trees[s], i)) - 1, n - m + i
            if rope is not None:
                q[t:t + 1] = rope_rotate(q[t:t + 1], rope[pos:pos + 1], interleaved)
                k[t:t + 1] = rope_rotate(k[t:t + 1], rope[pos:pos + 1], interleaved)
            k_pool[table[s][slot // page], slot % page] = k[t]
            v_pool[table[s][slot // page], slot % page] = v[t]
    return q, k, k_pool, v_pool


def accept(pools, table, cu, lens, trees, accepted):
    """Copies of the pools with the accepted paths in front, and the new lengths."""
    page = pools[0].shape[1]
    out = [np.array(x) for x in pools]
    new = []
    for s, n in enumerate(lens):
        m = cu[s + 1] - cu[s]
        if n == 0 or m == 0:
            new.append(n)
            continue
        keep = path(trees[s], accepted[s]) if accepted[s] >= 0 else []
        for i, a in enumerate(keep):
            src, dst = n - m + a, n - m + i
            for x, y in zip(out, pools):
                x[table[s][dst // page], dst % page] = y[table[s][src // page], src % page]
        new.append(n - m + len(keep))
    return out, new
