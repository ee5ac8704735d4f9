"""Serving on sequences of different lengths: rotary positions, the paged
key/value cache, attention over packed prompts and over the cache.

Rotation: a head's first `rot` elements in pairs (a, b) at position p,
    a' = a cos t_j - b sin t_j,  b' = a sin t_j + b cos t_j,
with (cos t_j, sin t_j) = rope[p, j]; pairs (x_j, x_{j + rot/2}), or (x_2j,
x_2j+1) when interleaved. Position of row t of sequence s with n_s new rows
and length len_s after the step: len_s - n_s + t - cu_s. Its key and value are
stored at slot p mod page_size of page table[s, p div page_size].

Attention is the layer's ("02 - How a whole Transformer block is split",
section 2) sequence by sequence; one query against a cached sequence for the
decode form. A sequence of length 0 gives o = 0, lse = -inf.

Test infrastructure only.
"""
import numpy as np

from .attention import attention_fwd
from .layer import _act, _lin
from .layernorm import ln_fwd


def rope_rotate(x, rows, interleaved=False):
    """x [T, heads, d], rows [T, rot/2, 2] -> x with its first rot elements rotated."""
    half = rows.shape[1]
    c, s = rows[:, None, :, 0], rows[:, None, :, 1]
    out = np.array(x, dtype=np.float64)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


def append_positions(cu, lens, tokens):
    """(sequence, position) of every row; (-1, -1) for rows of padding
    sequences (length 0) and behind the last sequence."""
    where = [(-1, -1)] * tokens
    for s, n in enumerate(lens):
        rows = cu[s + 1] - cu[s]
        for i in range(rows):
            if n > 0:
                where[cu[s] + i] = (s, n - rows + i)
    return where


def kv_append(q, k, v, cu, lens, rope, interleaved, table, k_pool, v_pool):
    """q [T, nq, d], k, v [T, nkv, d]; pools [pages, page_size, nkv, d]. Returns
    the rotated q and k and copies of the pools; rows without a position keep
    their input in the returned q and k."""
    q, k = np.array(q, dtype=np.float64), np.array(k, dtype=np.float64)
    k_pool, v_pool = np.array(k_pool, dtype=np.float64), np.array(v_pool, dtype=np.float64)
    page_size = k_pool.shape[1]
    for t, (s, p) in enumerate(append_positions(cu, lens, q.shape[0])):
        if s < 0:
            continue
        if rope is not None:
            q[t:t + 1] = rope_rotate(q[t:t + 1], rope[p:p + 1], interleaved)
            k[t:t + 1] = rope_rotate(k[t:t + 1], rope[p:p + 1], interleaved)
        page = table[s][p // page_size]
        k_pool[page, p % page_size] = k[t]
        v_pool[page, p % page_size] = v[t]
    return q, k, k_pool, v_pool


def packed_attention(q, k, v, cu, causal=True):
    """q [T, nq, d], k, v [T, nkv, d] -> (o [T, nq, d], lse [nq, T]); rows of no
    sequence are NaN."""
    o = np.full(q.shape, np.nan)
    lse = np.full((q.shape[1], q.shape[0]), np.nan)
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            x = [np.moveaxis(np.asarray(y[a:b], dtype=np.float64), 1, 0)[None] for y in (q, k, v)]
            os, ls = attention_fwd(*x, causal=causal)
            o[a:b] = np.moveaxis(os[0], 0, 1)
            lse[:, a:b] = ls[0]
    return o, lse


def gather_cache(pool, table_row, n):
    """The first n cached vectors of a sequence, [n, nkv, d]."""
    page_size = pool.shape[1]
    p = np.arange(n)
    return pool[np.asarray(table_row)[p // page_size], p % page_size]


def decode_attention(q, k_pool, v_pool, table, lens):
    """q [n, nq, d] -> (o [n, nq, d], lse [n, nq])."""
    n, nq, d = q.shape
    nkv = k_pool.shape[2]
    o = np.zeros((n, nq, d))
    lse = np.full((n, nq), -np.inf)
    for s in range(n):
        if lens[s] == 0:
            continue
        k, v = gather_cache(k_pool, table[s], lens[s]), gather_cache(v_pool, table[s], lens[s])
        for h in range(nq):
            g = h // (nq // nkv)
            x = (k[:, g] @ q[s, h]) / np.sqrt(d)
            m = x.max()
            e = np.exp(x - m)
            o[s, h] = (e / e.sum()) @ v[:, g]
            lse[s, h] = m + np.log(e.sum())
    return o, lse


def layer_fwd(cfg, w, x, rope=None, interleaved=False):
    """The layer (layer.block_fwd) on one whole sequence x [L, H] at positions
    0 .. L - 1, queries and keys rotated (rope [L or more, rot/2, 2])."""
    x = np.asarray(x, dtype=np.float64)
    L, nq, nkv, d, eps = x.shape[0], cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ln_eps
    pre = cfg.norm_pos == "pre"
    a = ln_fwd(x, w["ln1_g"], w["ln1_b"], eps)[0] if pre else x
    qkv = _lin(a, w["w_qkv"], w["b_qkv"]).reshape(L, nq + 2 * nkv, d)
    q, k, v = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    if rope is not None:
        q, k = (rope_rotate(z, rope[:L], interleaved) for z in (q, k))
    o, _ = packed_attention(q, k, v, [0, L], cfg.causal)
    h = x + _lin(o.reshape(L, nq * d), w["w_o"], w["b_o"])
    if not pre:
        h = ln_fwd(h, w["ln1_g"], w["ln1_b"], eps)[0]
    f = ln_fwd(h, w["ln2_g"], w["ln2_b"], eps)[0] if pre else h
    y = h + _lin(_act(_lin(f, w["w_1"], w["b_1"]), cfg), w["w_2"], w["b_2"])
    return y if pre else ln_fwd(y, w["ln2_g"], w["ln2_b"], eps)[0]
