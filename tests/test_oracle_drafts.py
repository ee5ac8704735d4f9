"""The float64 oracle of drafted tokens: trees, and its agreement with the oracle of
plain serving where the two say the same."""
import numpy as np

from oracle import drafts, serving

RNG = np.random.default_rng(1)


def _cache(lens, page=4, nkv=2, d=8):
    need = [(n + page - 1) // page for n in lens]
    pages = RNG.permutation(sum(need))
    table, at = [], 0
    for k in need:
        table.append(list(pages[at:at + k]))
        at += k
    shape = (sum(need), page, nkv, d)
    return RNG.standard_normal(shape), RNG.standard_normal(shape), table


def test_paths_and_masks():
    tree = [-1, 0, 0, 1, 3, -1, 5]
    assert drafts.path(tree, 4) == [0, 1, 3, 4] and drafts.path(tree, 6) == [5, 6]
    seen = drafts.visible(tree)
    assert seen.sum(1).tolist() == [1, 2, 2, 3, 4, 1, 2] and seen[4].tolist() == [1, 1, 0, 1, 1, 0, 0]
    assert (drafts.visible(drafts.chain(5)) == np.tril(np.ones((5, 5)))).all()


def test_a_chain_is_causal_attention_over_the_whole_sequence():
    n, m = 13, 6
    k, v, table = _cache([n])
    q = RNG.standard_normal((n, 4, 8))
    rows = [serving.gather_cache(x, table[0], n) for x in (k, v)]
    want, want_lse = serving.packed_attention(q, rows[0], rows[1], [0, n])
    o, lse, _, _ = drafts.tree_attention(q[n - m:], k, v, table, [0, m], [n], [drafts.chain(m)])
    assert np.allclose(o, want[n - m:]) and np.allclose(lse, want_lse[:, n - m:].T)


def test_a_leaf_sees_what_its_path_alone_would():
    ctx, tree = 9, [-1, 0, 0, 2, 1]
    k, v, table = _cache([ctx + 5])
    q = RNG.standard_normal((5, 4, 8))
    o, lse, _, _ = drafts.tree_attention(q, k, v, table, [0, 5], [ctx + 5], [tree])
    (ka, va), new = drafts.accept((k, v), table, [0, 5], [ctx + 5], [tree], [3])
    assert new == [ctx + 3]
    want, want_lse = serving.decode_attention(q[3:4], ka, va, table, new)
    assert np.allclose(o[3], want[0]) and np.allclose(lse[3], want_lse[0])


def test_an_accepted_path_is_what_appending_it_would_have_left():
    """Rotated by depth, the moved keys are those of the tokens in order."""
    ctx, tree = 3, [-1, 0, 0, 2]
    k, v, table = _cache([ctx + 4])
    th = RNG.standard_normal((12, 4))
    rows = np.stack([np.cos(th), np.sin(th)], axis=-1)
    q, kn, vn = (RNG.standard_normal((4, 2, 8)) for _ in range(3))
    _, _, ka, va = drafts.append_tree(q, kn, vn, [0, 4], [ctx + 4], [tree], rows, False, table, k, v)
    (ka, va), new = drafts.accept((ka, va), table, [0, 4], [ctx + 4], [tree], [3])
    keep = [0, 2, 3]
    _, _, kb, vb = serving.kv_append(q[keep], kn[keep], vn[keep], [0, 3], [ctx + 3], rows, False, table, k, v)
    for a, b in ((ka, kb), (va, vb)):
        assert np.allclose(serving.gather_cache(a, table[0], new[0]), serving.gather_cache(b, table[0], new[0]))
