"""GPU parity of mgb_attention_tree against the float64 oracle: trees and chains,
lengths around the unit's borders, row blocks, group sizes, page sizes and layouts,
splits over many CTAs, padding, rows behind the last sequence, poisoned unused slots,
repeats, graph replay, device-side index errors."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import TORCH, Cache, check_attention, dev, host, ints, values
from tests.util import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def check(got, lse, batch, c, q, d, dtype):
    """o [T, nq, d], lse [T, nq] of the batch's live rows."""
    ref, ref_lse, a, m = drafts.tree_attention(q, c.k, c.v, c.table, batch.cu, batch.lens, batch.trees)
    on = batch.live()
    n = np.zeros(batch.tokens)
    for s, x in enumerate(batch.lens):
        n[batch.cu[s]:batch.cu[s + 1]] = x
    check_attention(got[on], None if lse is None else lse[on], ref[on], ref_lse[on], a[on], m[on],
                    n[on][:, None] * np.ones(q.shape[1]), d, dtype)


def _run(seed, dtype, nq, nkv, d, page, seqs, head_major=False, tail=0, parents=True, scale=1.0):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, tail)
    c = Cache(rng, b.lens, page, nkv, d, dtype, head_major)
    T = b.tokens
    q = values(rng, (T, nq, d), dtype, scale)
    wide = dev(np.concatenate([q.reshape(T, -1), values(rng, (T, 16), dtype)], axis=1), dtype)
    g = Guarded()
    o = g.empty((T, nq * d + 32), TORCH[dtype], 3.0)
    lse = g.empty((T, nq), torch.float32, 5.0)
    plan = b.plan(nq, nkv, d, g, parents)
    first = None
    for _ in range(2):
        mgb.mgb_attention_tree(plan, c.desc, wide, nq * d + 16, o, nq * d + 32, lse)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        now = host(o), host(lse)
        if first is not None:
            assert (now[0] == first[0]).all() and (now[1] == first[1]).all()
        first = now
    g.check()
    on = b.live()
    assert (first[0][:, nq * d:] == 3.0).all() and (first[0][~on] == 3.0).all() and (first[1][~on] == 5.0).all()
    check(first[0][:, :nq * d].reshape(T, nq, d), first[1], b, c, q, d, dtype)


def _mixed(rng, ctxs, sizes, roots=1):
    return [(x, random_tree(rng, m, roots=min(roots, m))) for x, m in zip(ctxs, sizes)]


BORDERS = [0, 1, 2, 31, 33, 120, 123, 127, 128, 129, 200, 250, 256, 260, None, 5]
SIZES = [5, 1, 7, 1, 9, 8, 5, 1, 3, 128, 30, 6, 1, 12, 2, 33]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_one_token_over_a_short_cache(dtype, d):
    _run(1, dtype, 1, 1, d, 16, [(3, [-1])])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,head_major", [(16, False), (1, False), (24, True), (64, True), (100, False)])
def test_lengths_at_the_borders(dtype, d, page, head_major):
    _run(11, dtype, 4, 2, d, page, _mixed(np.random.default_rng(2), BORDERS, SIZES), head_major, tail=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,head_major", [(16, False), (1, False), (24, True), (100, False), (256, True)])
@pytest.mark.parametrize("nq,nkv", [(2, 2), (3, 1)])
def test_few_rows_at_the_borders(dtype, d, page, head_major, nq, nkv):
    """At most 16 rows per sequence on average (and some with more): the other kernel."""
    sizes = [2, 1, 3, 1, 4, 8, 5, 1, 3, 20, 1, 6, 1, 5, 2, 7]
    seqs = _mixed(np.random.default_rng(32), BORDERS, sizes, roots=2)
    assert sum(sizes) * nq // nkv <= 16 * len(sizes)
    _run(31, dtype, nq, nkv, d, page, seqs, head_major, tail=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [[(5000, 4)], [(9000, 3), (40, 7), (2100, 1)], [(20000, 1), (7, 1)]])
def test_few_rows_split_over_ctas(dtype, seqs):
    rng = np.random.default_rng(33)
    for d in (64, 128):
        _run(34, dtype, 4, 1, d, 64, [(x, random_tree(rng, m)) for x, m in seqs])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (3, 3), (7, 1), (16, 2), (17, 1), (40, 2), (71, 1)])
def test_group_sizes(dtype, nq, nkv):
    """Rows are tokens times heads of a group: blocks of rows end inside a token."""
    _run(12, dtype, nq, nkv, 128, 16, _mixed(np.random.default_rng(3), [70, 0, 300], [9, 40, 2]))
    _run(12, dtype, nq, nkv, 64, 16, _mixed(np.random.default_rng(3), [70, 0, 300], [1, 2, 1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256])
def test_rows_at_the_tiles_borders(dtype, m):
    rng = np.random.default_rng(m)
    _run(13, dtype, 2, 2, 64, 32, [(45, random_tree(rng, m)), (0, random_tree(rng, m, roots=3))])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [[(5000, 5)], [(9000, 70), (40, 3), (2100, 1)], [(700, 256)]])
def test_items_split_over_ctas(dtype, d, seqs):
    rng = np.random.default_rng(4)
    _run(14, dtype, 4, 1, d, 64, [(x, random_tree(rng, m)) for x, m in seqs])


def test_more_sequences_than_ctas():
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(0, 400, 300)]
    _run(15, "bf16", 4, 4, 64, 16, _mixed(rng, ctx, [int(m) for m in rng.integers(1, 9, 300)]), tail=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_items_of_one_unit_between_longer_ones(dtype, d):
    """Some sequences of a single unit, some of many, with one block of rows and with two halves:
    the streams that share the work go through items that one of them has no part in."""
    rng = np.random.default_rng(35)
    ctx = [int(x) for x in np.exp(rng.uniform(np.log(5), np.log(2500), 40))]
    _run(36, dtype, 8, 2, d, 16, _mixed(rng, ctx, [int(m) for m in rng.integers(1, 50, 40)]), tail=2)
    _run(37, dtype, 4, 2, d, 32, _mixed(rng, sorted(ctx), [20] * 40))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,head_major", [(8, False), (16, True), (24, False), (32, False), (64, True)])
def test_long_sequences_over_small_pages(d, page, head_major):
    """Batches that average more than 1000 tokens, short sequences and one with two halves of
    rows among them; groups of 2 and of 3 heads."""
    rng = np.random.default_rng(38)
    seqs = _mixed(rng, [2500, 1517, 30, None, 900, 4001, 1150], [12, 40, 70, 3, 100, 5, 1], roots=2)
    for nq, nkv in ((4, 2), (3, 1)):
        _run(39, "bf16", nq, nkv, d, page, seqs, head_major, tail=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chains_need_no_parents(dtype):
    _run(16, dtype, 4, 2, 128, 16, [(30, drafts.chain(256)), (None, drafts.chain(2)), (130, drafts.chain(1)),
                                    (0, drafts.chain(150))], parents=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores far apart: the reference moves, weights vanish."""
    rng = np.random.default_rng(6)
    _run(17, dtype, 4, 2, 128, 16, _mixed(rng, [900, 3, 140], [20, 9, 33]), scale=40.0)


def test_siblings_do_not_see_each_other():
    """Keys of tokens outside a row's path have no say, whatever they hold."""
    rng = np.random.default_rng(7)
    tree = [-1, 0, 0, 1, 1, 2, 2]
    for dtype in ("bf16", "f32"):
        b = Batch([(21, tree)])
        c = Cache(rng, b.lens, 8, 2, 64, dtype)
        q = dev(values(rng, (7, 2 * 64), dtype), dtype)
        plan = b.plan(2, 2, 64)
        outs = []
        for k, v in ((1.0, 1.0), (float("nan"), 7.0), (float("inf"), -2.0), (-3e38, 0.0)):
            for j in (2, 5, 6):          # not on the path of tokens 0, 1, 3, 4
                pg, i = c.table[0][(21 + j) // 8], (21 + j) % 8
                c.tk[pg, i] = k
                c.tv[pg, i] = v
            o = torch.zeros((7, 128), dtype=TORCH[dtype], device="cuda")
            lse = torch.zeros((7, 2), device="cuda")
            mgb.mgb_attention_tree(plan, c.desc, q, 128, o, 128, lse)
            outs.append((o[[0, 1, 3, 4]], lse[[0, 1, 3, 4]]))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        for o, lse in outs[1:]:
            assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def _bad(seqs, nq=2, nkv=1, d=64, dtype="bf16", page=8, spoil=None, tail=0, **kw):
    """o, lse, the batch and its cache after a call that reports an index."""
    rng = np.random.default_rng(8)
    b = Batch(seqs, tail)
    c = Cache(rng, b.lens, page, nkv, d, dtype)
    q = values(rng, (b.tokens, nq, d), dtype)
    if spoil:
        spoil(b, c)
        c.ttable.copy_(ints(c.table))
    o = torch.full((b.tokens, nq * d), 3.0, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((b.tokens, nq), 5.0, device="cuda")
    plan = b.plan(nq, nkv, d, **kw)
    mgb.mgb_attention_tree(plan, c.desc, dev(q.reshape(b.tokens, -1), dtype), nq * d, o, nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
    return host(o).reshape(b.tokens, nq, d), host(lse), b, c, q


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_tokens_of_a_bad_page_are_left_out(dtype, entry):
    def spoil(b, c):
        c.table[1][3] = entry
    o, lse, b, c, q = _bad([(20, [-1, 0]), (60, [-1, 0, 0, 1]), (3, [-1])], dtype=dtype, spoil=spoil)
    keep = [p for p in range(60) if p // 8 != 3]
    pool = lambda x: x[c.table[1][np.array(keep + [60, 61, 62, 63]) // 8], np.array(keep + [60, 61, 62, 63]) % 8]
    k, v = pool(c.k), pool(c.v)
    seen = np.concatenate([np.ones((4, len(keep)), dtype=bool), drafts.visible(b.trees[1])], axis=1)
    for h in range(2):
        sc = np.where(seen, q[2:6, h] @ k[:, 0].T / 8.0, -np.inf)
        p = np.exp(sc - sc.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        tol = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -16) * (p @ np.abs(v[:, 0]))
        assert (np.abs(o[2:6, h] - p @ v[:, 0]) <= tol).all()
    on = np.array([0, 1, 6])
    ref, ref_lse, a, m = drafts.tree_attention(q, c.k, c.v, np.where(c.table == entry, 0, c.table), b.cu, b.lens,
                                               b.trees)
    check_attention(o[on], lse[on], ref[on], ref_lse[on], a[on], m[on], np.full((3, 2), 64), 64, dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_of_long_sequences_are_left_out(d):
    gone = [0, 17, 99, 100, 140]

    def spoil(b, c):
        c.table[0][gone] = [-1, 10 ** 6, -1, -7, 2 ** 31 - 1]
    o, lse, b, c, q = _bad([(1200, drafts.chain(9)), (1100, drafts.chain(12))], d=d, page=8, spoil=spoil)
    n = 1209
    keep = np.array([p for p in range(n) if p // 8 not in gone])
    k, v = (x[c.table[0][keep // 8], keep % 8] for x in (c.k, c.v))
    seen = keep[None, :] <= np.arange(1200, n)[:, None]
    for h in range(2):
        sc = np.where(seen, q[:9, h] @ k[:, 0].T / np.sqrt(d), -np.inf)
        p = np.exp(sc - sc.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert (np.abs(o[:9, h] - p @ v[:, 0]) <= 2.0 ** -7 * (p @ np.abs(v[:, 0]))).all()
    on = np.arange(9, 21)
    table = np.where((c.table < 0) | (c.table >= len(c.k)), 0, c.table)
    ref, ref_lse, a, m = drafts.tree_attention(q, c.k, c.v, table, b.cu, b.lens, b.trees)
    check_attention(o[on], lse[on], ref[on], ref_lse[on], a[on], m[on], np.full((12, 2), 1112), d, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_a_token_left(dtype):
    def spoil(b, c):
        c.table[0][:] = -1
    o, lse, b, c, q = _bad([(20, [-1, 0, 0]), (9, [-1])], dtype=dtype, spoil=spoil)
    assert np.isnan(o[:3]).all() and np.isneginf(lse[:3]).all()
    assert np.isfinite(o[3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw,dead", [
    (dict(lens=[22, -5, 4]), [1]), (dict(lens=[22, 2, 4]), [1]), (dict(lens=[22, 2 ** 31 - 1, 4]), [1]),
    (dict(lens=[22, 10 ** 6, 4]), [1]),
    (dict(cu=[0, 2, 1, 6]), [1, 2]), (dict(cu=[0, 2, 99, 6]), [1, 2]), (dict(cu=[1, 2, 5, 6]), [0, 1, 2]),
    (dict(cu=[0, -4, 5, 6]), [0, 1, 2]), (dict(cu=[0, 2, 5, 2 ** 31 - 1]), [2]),
])
def test_bad_lengths_and_offsets_leave_their_rows(dtype, kw, dead):
    seqs = [(20, [-1, 0]), (60, [-1, 0, 0]), (3, [-1])]
    o, lse, b, c, q = _bad(seqs, dtype=dtype, **kw)
    rows = [range(b.cu[s], b.cu[s + 1]) for s in range(3)]
    for s in range(3):
        if s in dead:
            assert (o[list(rows[s])] == 3.0).all() and (lse[list(rows[s])] == 5.0).all()
        else:
            assert np.isfinite(o[list(rows[s])]).all() and (lse[list(rows[s])] != 5.0).all()


def test_too_many_drafted_tokens():
    o, lse, b, c, q = _bad([(20, [-1, 0]), (300, drafts.chain(257)), (3, [-1])])
    assert (o[2:259] == 3.0).all() and np.isfinite(o[[0, 1, 259]]).all() and (lse[[0, 1, 259]] != 5.0).all()


@pytest.mark.parametrize("bad", [-2, 3, 4, 10 ** 9, -2 ** 31])
def test_a_bad_parent_is_the_last_cached_token(bad):
    """Token 3's parent is not below it."""
    rng = np.random.default_rng(8)
    outs = []
    for tree in ([-1, 0, 1, bad, 3], [-1, 0, 1, -1, 3]):
        if tree[3] == -1:
            b = Batch([(20, tree)])
            c = Cache(np.random.default_rng(8), b.lens, 8, 1, 64, "bf16")
            q = values(np.random.default_rng(9), (5, 2, 64), "bf16")
            o = torch.zeros((5, 128), dtype=torch.bfloat16, device="cuda")
            mgb.mgb_attention_tree(b.plan(2, 1, 64), c.desc, dev(q.reshape(5, -1), "bf16"), 128, o, 128)
            assert mgb.mgb_device_status() == mgb.MGB_OK
        else:
            b = Batch([(20, tree)])
            c = Cache(np.random.default_rng(8), b.lens, 8, 1, 64, "bf16")
            q = values(np.random.default_rng(9), (5, 2, 64), "bf16")
            o = torch.zeros((5, 128), dtype=torch.bfloat16, device="cuda")
            mgb.mgb_attention_tree(b.plan(2, 1, 64), c.desc, dev(q.reshape(5, -1), "bf16"), 128, o, 128)
            assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
        outs.append(o)
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_replayed_with_other_trees_and_lengths(dtype):
    """Prepare and attention in one graph follow the offsets, lengths and parents."""
    rng = np.random.default_rng(10)
    nq, nkv, d, page, T, n = 4, 2, 64, 16, 40, 3
    c = Cache(rng, [700, 700, 700], page, nkv, d, dtype)
    q = values(rng, (T, nq, d), dtype)
    tq = dev(q.reshape(T, -1), dtype)
    cu, lens, parents = ints([0] * (n + 1)), ints([0] * n), ints([-1] * T)
    ws = torch.empty(mgb.mgb_attention_tree_ws_bytes(n, T, nq, nkv, d), dtype=torch.uint8, device="cuda")
    o = torch.zeros((T, nq * d), dtype=TORCH[dtype], device="cuda")

    def step():
        plan = mgb.mgb_attention_tree_prepare(n, T, nq, nkv, d, cu, lens, parents, ws)
        mgb.mgb_attention_tree(plan, c.desc, tq, nq * d, o, nq * d)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seqs in ([(600, 10), (3, 5), (None, 2)], [(1, 40), (None, 0), (20, 0)], [(30, 1), (650, 20), (200, 19)]):
        b = Batch([(x, random_tree(rng, m)) for x, m in seqs])
        b.tokens, b.parents = T, b.parents + [-1] * (T - len(b.parents))
        cu.copy_(ints(b.cu))
        lens.copy_(ints(b.lens))
        parents.copy_(ints(b.parents))
        o.fill_(3.0)
        graph.replay()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        got = host(o).reshape(T, nq, d)
        on = np.zeros(T, dtype=bool)
        on[:b.cu[-1]] = Batch(
            [(x, t) for (x, _), t in zip(seqs, b.trees)]).live()
        assert (got[~on] == 3.0).all()
        ref, _, a, m = drafts.tree_attention(q, c.k, c.v, c.table, b.cu, b.lens, b.trees)
        check_attention(got[on], None, ref[on], None, a[on], m[on], np.full((int(on.sum()), nq), 700), d, dtype)
