"""GPU parity of the cache's operators for drafted tokens: append by depth, accepted
paths moved to the front, pages copied."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import HALF_STEP, TORCH, Cache, dev, host, ints, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def same(a, b):
    return ((a == b) | (np.isnan(a) & np.isnan(b))).all()


def rounded(got, want, scale, dtype):
    """got is want rounded once; the rotation's three float32 steps are off by 2^-22 of the pair."""
    ok = np.isnan(want) & np.isnan(got)
    tol = HALF_STEP[dtype] * (np.abs(want) + 2.0 ** -22 * scale) + 2.0 ** -22 * scale
    return (ok | (np.abs(got - want) <= tol)).all()


def _append(seed, dtype, nq, nkv, d, page, seqs, rot, interleaved, head_major=False, tail=0, inplace=False,
            parents=True):
    rng = np.random.default_rng(seed)
    b = Batch(seqs, tail)
    T = b.tokens
    c = Cache(rng, b.lens, page, nkv, d, dtype, head_major)
    q, k, v = (values(rng, (T, h, d), dtype) for h in (nq, nkv, nkv))
    rope = rope_table(max(b.lens) + 1, rot) if rot else None
    w = (nq + 2 * nkv) * d
    qkv = dev(np.concatenate([x.reshape(T, -1) for x in (q, k, v)], axis=1), dtype)
    tk, tv = qkv[:, nq * d:], qkv[:, (nq + nkv) * d:]
    q_out = qkv if inplace else torch.full((T, nq * d), 3.0, dtype=TORCH[dtype], device="cuda")
    k_out = tk if inplace else torch.full((T, nkv * d), 3.0, dtype=TORCH[dtype], device="cuda")
    desc = mgb.kv_append_desc(T, b.n, nq, rot, interleaved, rope.shape[0] if rot else 0)
    plan = b.plan(nq, nkv, d, parents=parents)
    mgb.mgb_kv_append_tree(plan, desc, c.desc, rope, qkv, tk, tv, w, w, q_out, w if inplace else nq * d, k_out,
                           w if inplace else nkv * d)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    wq, wk, kp, vp = drafts.append_tree(q, k, v, b.cu, b.lens, b.trees, host(rope) if rot else None, interleaved,
                                        c.table, c.k, c.v)
    on = b.live()
    got_q = host(q_out)[:, :nq * d].reshape(T, nq, d)
    got_k = host(k_out)[:, :nkv * d].reshape(T, nkv, d)
    big = 8.0
    assert rounded(got_q[on], wq[on], big, dtype) and rounded(got_k[on], wk[on], big, dtype)
    off = ~on
    assert same(got_q[off], q[off] if inplace else np.full_like(q[off], 3.0))
    assert same(got_k[off], k[off] if inplace else np.full_like(k[off], 3.0))
    pools = [host(x) for x in (c.tk, c.tv)]
    assert rounded(pools[0], kp, big, dtype) and same(pools[1], vp)
    # what was cached before, and slots of no sequence, are as they were
    fresh = np.zeros(c.k.shape[:2], dtype=bool)
    for s, n in enumerate(b.lens):
        p = np.arange(n - len(b.trees[s]), n) if n else np.arange(0)
        fresh[c.table[s][p // page], p % page] = True
    assert same(pools[0][~fresh], c.k[~fresh]) and same(pools[1][~fresh], c.v[~fresh])


SEQS = [(20, 7), (0, 1), (None, 3), (127, 33), (3, 0), (300, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (32, False), (0, False)])
@pytest.mark.parametrize("page,head_major", [(16, False), (1, True), (100, False)])
def test_append_by_depth(dtype, rot, interleaved, page, head_major):
    rng = np.random.default_rng(20)
    seqs = [(x, random_tree(rng, m, roots=min(m, 2))) for x, m in SEQS]
    _append(21, dtype, 4, 2, 64, page, seqs, rot, interleaved, head_major, tail=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_in_place_and_many(dtype):
    rng = np.random.default_rng(22)
    _append(23, dtype, 6, 2, 128, 16, [(9, random_tree(rng, 6)), (40, random_tree(rng, 11))], 128, False, inplace=True)
    _append(24, dtype, 4, 1, 64, 32, [(int(x), drafts.chain(16)) for x in rng.integers(0, 200, 40)], 64, False,
            parents=False)


def test_append_reports_places_outside():
    b = Batch([(20, [-1, 0, 0]), (5, [-1])])
    for what in ("page", "rope", "cap"):
        c = Cache(np.random.default_rng(25), b.lens, 8, 1, 64, "bf16")
        rows = 21 if what == "rope" else 60           # token 0 has position 20, its children 21
        if what == "page":
            c.table[0][2] = 10 ** 6
            c.ttable.copy_(ints(c.table))
        if what == "cap":
            c.desc = mgb.kv_cache(c.tk, c.tv, c.ttable[:, :2])   # 16 slots
        before = host(c.tk)
        x = torch.ones((4, 192), dtype=torch.bfloat16, device="cuda")
        q = torch.full((4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        mgb.mgb_kv_append_tree(b.plan(1, 1, 64), mgb.kv_append_desc(4, 2, 1, 64, False, rows), c.desc,
                               rope_table(rows, 64), x, x[:, 64:], x[:, 128:], 192, 192, q, 64, None, 0)
        assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
        got, q = host(c.tk), host(q)
        dead = [0, 1, 2] if what != "rope" else [1, 2]
        assert (q[dead] == 3.0).all() and (q[3] != 3.0).all()
        changed = {(int(p), int(i)) for p, i, _, _ in np.argwhere(~((got == before) | (np.isnan(got) & np.isnan(before))))}
        own = {(int(c.table[1][0]), 5)} | ({(int(c.table[0][2]), 4)} if what == "rope" else set())
        assert changed <= own and changed


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,head_major,nkv,d", [(16, False, 2, 64), (1, True, 3, 128), (24, True, 1, 64),
                                                   (100, False, 17, 128)])
def test_accepted_paths_move_to_the_front(dtype, page, head_major, nkv, d):
    rng = np.random.default_rng(26)
    # token 1's path is one step behind itself: every slot read is written by the step after
    seqs = [(20, random_tree(rng, 40)), (0, [-1, -1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]), (None, [-1, 0]),
            (127, random_tree(rng, 256, branch=1)), (9, []), (130, drafts.chain(20)), (63, random_tree(rng, 9)),
            (5, [-1] * 8 + list(range(7, 250)))]
    b = Batch(seqs, tail=3)
    accepted = [39, 11, -1, 255, -1, 19, -1, 250]
    c = Cache(rng, b.lens, page, nkv, d, dtype, head_major)
    plan = b.plan(2 * nkv, nkv, d)
    new = torch.full((b.n,), -9, dtype=torch.int32, device="cuda")
    mgb.mgb_kv_accept(plan, c.desc, ints(accepted), new)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    (kp, vp), lens = drafts.accept((c.k, c.v), c.table, b.cu, b.lens, b.trees, accepted)
    assert new.tolist() == lens
    # behind the new length nothing is promised; the rest is exact
    for got, want, old in ((host(c.tk), kp, c.k), (host(c.tv), vp, c.v)):
        assert same(got, want)
    assert lens[1] == 11 and lens[7] == 5 + 244


def test_accept_reports_and_leaves():
    for what in ("leaf", "page", "cap"):
        b = Batch([(20, [-1, 0, 0, 2]), (5, [-1, 0, 0])])
        c = Cache(np.random.default_rng(27), b.lens, 8, 1, 64, "bf16")
        accepted = [4 if what == "leaf" else 3, 2]
        if what == "page":
            c.table[0][2] = -3
            c.ttable.copy_(ints(c.table))
        if what == "cap":
            c.desc = mgb.kv_cache(c.tk, c.tv, c.ttable[:, :2])
        before = host(c.tk)
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        mgb.mgb_kv_accept(b.plan(1, 1, 64), c.desc, ints(accepted), new)
        assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
        assert new.tolist() == [20 if what == "leaf" else 23, 7]
        got = host(c.tk)
        want = np.array(before)
        p = c.table[1][0]
        want[p, 6] = before[p, 7]
        assert same(got, want)


def test_accept_writes_the_lengths_it_was_prepared_from():
    b = Batch([(20, [-1, 0, 0, 2]), (None, [-1])])
    c = Cache(np.random.default_rng(28), b.lens, 8, 1, 64, "bf16")
    lens = ints(b.lens)
    ws = torch.empty(mgb.mgb_attention_tree_ws_bytes(2, 5, 1, 1, 64), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_tree_prepare(2, 5, 1, 1, 64, ints(b.cu), lens, ints(b.parents), ws)
    for _ in range(2):   # two layers' caches would each get a call: the same lengths
        mgb.mgb_kv_accept(plan, c.desc, ints([3, -1]), lens)
        assert lens.tolist() == [23, 0]
    assert mgb.mgb_device_status() == mgb.MGB_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,head_major,nkv,d", [(16, False, 2, 64), (1, True, 3, 24), (24, True, 1, 128),
                                                   (100, False, 5, 40), (256, True, 8, 128)])
def test_pages_are_copied(dtype, page, head_major, nkv, d):
    rng = np.random.default_rng(29)
    n_pages = 40
    c = Cache(rng, [n_pages * page - page], page, nkv, d, dtype, head_major, extra=1)
    order = rng.permutation(n_pages)
    src = list(order[:3]) + [order[0], order[0], order[4]]        # one page read three times
    dst = list(order[10:15]) + [order[4]]                         # the last one onto itself
    slots = [int(x) for x in rng.integers(0, page + 1, 5)] + [page]
    slots[1], slots[2] = page, 0
    mgb.mgb_kv_copy_pages(c.desc, ints(src), ints(dst), ints(slots))
    assert mgb.mgb_device_status() == mgb.MGB_OK
    for got, old in ((host(c.tk), c.k), (host(c.tv), c.v)):
        want = np.array(old)
        for a, b, n in zip(src, dst, slots):
            want[b, :n] = old[a, :n]
        assert same(got, want)
    mgb.mgb_kv_copy_pages(c.desc, ints(src[:1]), ints(order[20:21]))
    mgb.mgb_kv_copy_pages(c.desc, ints([]), ints([]))
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert same(host(c.tk)[order[20]], c.k[src[0]])


@pytest.mark.parametrize("src,dst,n", [(-1, 2, 3), (40, 2, 3), (1, -1, 3), (1, 2 ** 31 - 1, 3), (1, 2, 9), (1, 2, -1)])
def test_bad_copies_are_reported_and_skipped(src, dst, n):
    c = Cache(np.random.default_rng(30), [39 * 8], 8, 2, 64, "bf16", extra=1)
    mgb.mgb_kv_copy_pages(c.desc, ints([src, 5]), ints([dst, 6]), ints([n, 4]))
    assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
    want = np.array(c.k)
    want[6, :4] = c.k[5, :4]
    assert same(host(c.tk), want)


def test_copy_counts_must_agree():
    c = Cache(np.random.default_rng(31), [8], 8, 1, 64, "bf16")
    with pytest.raises(ValueError):
        mgb.mgb_kv_copy_pages(c.desc, ints([0, 1]), ints([1]))
    with pytest.raises(ValueError):
        mgb.mgb_kv_copy_pages(c.desc, ints([0]), ints([1]), ints([1, 1]))
