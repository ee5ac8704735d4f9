"""GPU tests of the operators for drafted tokens beside those in test_gpu_kv_tree.py and
test_gpu_tree_more.py: vectors next to each other, many sequences with a bad offset, the time
that many sequences take, accepts and page copies in a captured graph, a drafted chain against
single steps."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import Cache, host, ints
from tests.test_gpu_drafts_run import Net
from tests.util import TOL, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


@pytest.mark.parametrize("lens_first", [True, False])
def test_accepted_indices_and_new_lengths_next_to_each_other(lens_first):
    rng = np.random.default_rng(80)
    b = Batch([(20, random_tree(rng, 9)), (0, random_tree(rng, 4)), (None, [-1]), (300, random_tree(rng, 30))])
    accepted = [8, 2, -1, 29]
    c = Cache(rng, b.lens, 16, 2, 64, "bf16")
    both = ints([-9] * 10)
    new, old = (both[1:5], both[5:9]) if lens_first else (both[5:9], both[1:5])
    old.copy_(ints(accepted))
    mgb.mgb_kv_accept(b.plan(4, 2, 64), c.desc, old, new)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    (kp, vp), lens = drafts.accept((c.k, c.v), c.table, b.cu, b.lens, b.trees, accepted)
    assert new.tolist() == lens and old.tolist() == accepted and both[0] == both[9] == -9
    for got, want in ((host(c.tk), kp), (host(c.tv), vp)):
        assert ((got == want) | (np.isnan(got) & np.isnan(want))).all()


@pytest.mark.parametrize("n", [4096, 4097, 30000])
@pytest.mark.parametrize("where", [0, 1, 0.4, 1.0, None])
@pytest.mark.parametrize("empty", [True, False])
def test_many_sequences_with_a_bad_offset(n, where, empty):
    """Sequences of one row, or some without; from the first bad offset on they count as empty."""
    nq, d = 2, 64
    rng = np.random.default_rng(81)
    rows = (rng.random(n) < 0.6) if empty else np.ones(n, dtype=bool)
    cu = np.concatenate([[0], np.cumsum(rows)])
    T, last = int(cu[-1]), n
    if where is not None:
        # the offset behind sequence `last`: below the one before, or past the rows
        last = int(where * (n - 1)) if isinstance(where, float) else where
        cu[last + 1] = -1 if where == 1 else T + 1
        if where == 0.4:
            cu[last + 1:last + 900:7] = 2 ** 31 - 1    # and some more
    x = torch.randn((T, (nq + 2) * d), device="cuda").bfloat16()
    pool = torch.full((2, n, 1, 1, d), 7.0, device="cuda", dtype=torch.bfloat16)
    cache = mgb.kv_cache(pool[0], pool[1], torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1))
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    ws = torch.full((mgb.mgb_attention_tree_ws_bytes(n, T, nq, 1, d),), 0xC3, dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_tree_prepare(n, T, nq, 1, d, ints(cu), lens, ints([-1] * T), ws)
    bad = where is not None
    assert mgb.mgb_device_status() == (mgb.MGB_ERR_INDEX if bad else mgb.MGB_OK)
    w, o = x.shape[1], torch.full((T, nq * d), 3.0, device="cuda", dtype=torch.bfloat16)
    mgb.mgb_kv_append_tree(plan, mgb.kv_append_desc(T, n, nq, 0, False, 0), cache, None, x, x[:, nq * d:],
                           x[:, (nq + 1) * d:], w, w, None, 0, None, 0)
    mgb.mgb_attention_tree(plan, cache, x, w, o, nq * d)
    new = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    mgb.mgb_kv_accept(plan, cache, torch.full_like(lens, -1), new)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    seen = int(cu[last]) if bad else T          # rows in front of the bad offset
    v = x[:, (nq + 1) * d:]
    assert torch.equal(o[:seen], v[:seen].repeat(1, nq)) and bool((o[seen:] == 3.0).all())
    on = np.zeros(n, dtype=bool)
    on[:last] = rows[:last]
    on = torch.from_numpy(on).cuda()
    assert torch.equal(pool[1][on][:, 0, 0], v[:seen]) and bool((pool[:, ~on] == 7.0).all())
    assert torch.equal(new, torch.where(on, 0, 1).int())


def test_time_of_a_prepare_goes_with_the_sequences():
    """Not with their square: 70000 sequences against 17500 (4 times as many)."""
    times = []
    for n in (17500, 70000):
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        lens = torch.full((n,), 40, dtype=torch.int32, device="cuda")
        ws = torch.empty(mgb.mgb_attention_tree_ws_bytes(n, n, 2, 2, 64), dtype=torch.uint8, device="cuda")
        best = []
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(4):
                mgb.mgb_attention_tree_prepare(n, n, 2, 2, 64, cu, lens, None, ws)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        times.append(min(best))
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert times[1] < 8 * times[0], times


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accepts_and_copies_are_replayed_with_other_indices(dtype):
    """Prepare, accept and page copies in one graph, whose offsets, trees, leaves, pages and numbers
    of slots change between the replays; one replay's indices are bad."""
    rng = np.random.default_rng(82)
    n, T, page, nkv, d, copies = 4, 60, 16, 2, 64, 3
    c = Cache(rng, [page * 6] * n, page, nkv, d, dtype, extra=4)
    cu, lens, parents, accepted = (ints([0] * (n + 1)), ints([0] * n), ints([-1] * T), ints([-1] * n))
    new, src, dst, slots = ints([-9] * n), ints([0] * copies), ints([0] * copies), ints([0] * copies)
    ws = torch.empty(mgb.mgb_attention_tree_ws_bytes(n, T, 4, nkv, d), dtype=torch.uint8, device="cuda")

    def step():
        plan = mgb.mgb_attention_tree_prepare(n, T, 4, nkv, d, cu, lens, parents, ws)
        mgb.mgb_kv_accept(plan, c.desc, accepted, new)
        mgb.mgb_kv_copy_pages(c.desc, src, dst, slots)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()              # (nothing drafted, page 0 onto itself)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pools = [c.k, c.v]
    for replay in range(6):
        sizes = [int(m) for m in rng.integers(1, 15, n)]
        b = Batch([(None if m == 3 else int(rng.integers(0, 6 * page - m + 1)), random_tree(rng, m)) for m in sizes])
        leaf = [int(rng.integers(-1, m)) for m in sizes]
        order = rng.permutation(c.n_pages)
        a, z, k = order[:copies], order[copies:2 * copies], rng.integers(0, page + 1, copies)
        bad = replay == 3
        cu.copy_(ints(b.cu)), lens.copy_(ints(b.lens)), parents.copy_(ints(b.parents + [-1] * (T - b.tokens)))
        accepted.copy_(ints([leaf[0], leaf[1], leaf[2], 99 if bad else leaf[3]]))
        src.copy_(ints(a)), dst.copy_(ints([z[0], z[1], c.n_pages if bad else z[2]])), slots.copy_(ints(k))
        graph.replay()
        assert mgb.mgb_device_status() == (mgb.MGB_ERR_INDEX if bad else mgb.MGB_OK)
        if bad:
            leaf[3], k[2] = -1, 0
        pools, want = drafts.accept(pools, c.table, b.cu, b.lens, b.trees, leaf)
        for x in pools:
            for i, j, m in zip(a, z, k):
                x[j, :m] = x[i, :m]
        assert new.tolist() == want
        for got, x in ((host(c.tk), pools[0]), (host(c.tv), pools[1])):
            assert ((got == x) | (np.isnan(got) & np.isnan(x))).all()


@pytest.mark.parametrize("shape", [LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True),
                                   LayerShape(1, 1, 256, 8, 1, 128, 512, causal=True),
                                   LayerShape(1, 1, 128, 4, 2, 64, 256, dtype="f32", causal=True)])
@pytest.mark.parametrize("m", [1, 3, 17])
def test_a_drafted_chain_gives_what_single_steps_give(shape, m):
    """Two layers of each: a result is within 2 TOL of the float64 layers, so two are within 4 of each
    other; the caches, which a step more may have left at the same distance, too."""
    prompts, outs = [40, 1, 200], []
    for chain in (True, False):
        rng = np.random.default_rng(83)
        n = len(prompts)
        net = Net(shape, 64, False, n, 16)
        for layer in net.layers:
            layer.k_pool.zero_(), layer.v_pool.zero_()
        table, cu = ints(net.table), np.cumsum([0] + prompts)
        net.run(net.rows(rng, int(cu[-1])), ServingBatch(shape, table, ints(prompts), ints(cu), int(cu[-1])))
        x = net.rows(rng, n * m).reshape(n, m, -1)
        if chain:
            lens = ints([p + m for p in prompts])
            batch = ServingBatch(shape, table, lens, ints(np.arange(n + 1) * m), n * m, drafted=True)
            y = host(net.run(x.reshape(n * m, -1), batch)).reshape(n, m, -1)
            for layer in net.layers:
                layer.accept(batch, ints([m - 1] * n), lens)
            assert lens.tolist() == [p + m for p in prompts]
        else:
            y = np.stack([host(net.run(x[:, i].copy(), ServingBatch(shape, table, ints([p + i + 1 for p in prompts]))))
                          for i in range(m)], axis=1)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append((y, [host(t) for layer in net.layers for t in (layer.k_pool, layer.v_pool)]))
    tol = 4 * TOL[shape.dtype][0]
    for a, b in zip(outs[0][0].reshape(-1, shape.hidden), outs[1][0].reshape(-1, shape.hidden)):
        assert rel_l2(a, b) < tol
    for a, b in zip(outs[0][1], outs[1][1]):
        assert rel_l2(a, b) < tol
