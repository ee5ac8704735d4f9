"""The operators for drafted tokens where calls meet: offsets past 2^32 elements, rows far
apart, 70000 sequences, plans on two streams, one plan for several layers, shared pages,
calls without rows, NaN, infinities and scores of any size."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import TORCH, Cache, dev, ints, values

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _attend(plan, cache, q, o=None, lse=None):
    T, w = q.shape
    o = torch.full_like(q, 3.0) if o is None else o
    mgb.mgb_attention_tree(plan, cache, q, w, o, w, lse)
    return o


# query heads, KV heads, page, trees: the decode step's kernel; K and V by TMA; V by threads; row by row
FORMS = [(2, 2, 1040, [3, 2]), (16, 2, 1152, [9, 4]), (4, 2, 1040, [9, 14]), (4, 2, 1041, [9, 14])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_pages_past_two_to_the_32_elements(dtype, form):
    """Append, attention, accept and page copies: the bits of a small pool."""
    nq, nkv, page, sizes = FORMS[form]
    d, pages = 64, 6
    far = (1 << 30) + (1 << 20)      # elements between pages: the last two begin past 2^32
    if torch.cuda.mem_get_info()[0] < 7 * far * TORCH[dtype].itemsize:
        pytest.skip("not enough free memory")
    rng = np.random.default_rng(50)
    big = torch.empty(((pages - 1) * far + (1 << 20),), dtype=TORCH[dtype], device="cuda")
    view = lambda at: big[at:].as_strided((pages, page, nkv, d), (far, nkv * d, d, 1), big.storage_offset() + at)
    near = torch.zeros((2, pages, page, nkv, d), dtype=TORCH[dtype], device="cuda").normal_()
    pk, pv = view(0), view(1 << 19)
    pk.copy_(near[0])
    pv.copy_(near[1])
    ctx = [2 * page - 7, 1200 if form == 2 else 90]
    b = Batch([(c, random_tree(rng, m)) for c, m in zip(ctx, sizes)])
    table = ints([[4, 0, 3], [1, 2, -1]])
    qkv = dev(values(rng, (b.tokens, (nq + 2 * nkv) * d), dtype), dtype)
    w, rope = qkv.shape[1], rope_table(4096, d)
    accepted = ints([sizes[0] - 1, sizes[1] - 1])
    outs = []
    for k, v in ((pk, pv), (near[0], near[1])):
        cache = mgb.kv_cache(k, v, table)
        plan = b.plan(nq, nkv, d)
        q = torch.zeros((b.tokens, nq * d), dtype=qkv.dtype, device="cuda")
        mgb.mgb_kv_append_tree(plan, mgb.kv_append_desc(b.tokens, b.n, nq, d, False, 4096), cache, rope, qkv,
                               qkv[:, nq * d:], qkv[:, (nq + nkv) * d:], w, w, q, nq * d, None, 0)
        o = _attend(plan, cache, q)
        lens = ints([0, 0])
        mgb.mgb_kv_accept(plan, cache, accepted, lens)
        mgb.mgb_kv_copy_pages(cache, ints([4, 3]), ints([5, 2]), ints([page, 7]))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append((o, lens))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert bool(outs[0][0].isfinite().all()) and not bool((outs[0][0] == 3.0).all())
    assert torch.equal(pk, near[0]) and torch.equal(pv, near[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv", [(2, 2), (16, 2), (12, 2)])
def test_rows_far_apart(dtype, nq, nkv):
    """Rows of q and o 2^30 elements apart."""
    far, d = 1 << 30, 64
    rng = np.random.default_rng(51)
    b = Batch([(40, [-1, 0, 0, 1])])
    n = b.tokens
    if torch.cuda.mem_get_info()[0] < (n + 1) * far * TORCH[dtype].itemsize:
        pytest.skip("not enough free memory")
    c = Cache(rng, b.lens, 16, nkv, d, dtype)
    q = dev(values(rng, (n, nq * d), dtype), dtype)
    big = torch.empty(((n - 1) * far + 2 * nq * d,), dtype=TORCH[dtype], device="cuda")
    view = lambda at: big[at:].as_strided((n, nq * d), (far, 1), at)
    view(0).copy_(q)
    plan = b.plan(nq, nkv, d)
    o = _attend(plan, c.desc, q)
    mgb.mgb_attention_tree(plan, c.desc, view(0), far, view(nq * d), far)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert torch.equal(view(nq * d), o) and torch.equal(view(0), q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 32])
def test_more_sequences_than_a_grid_is_wide(dtype, nq):
    """70000 sequences of a drafted token or none, some of them padding: each sees itself."""
    n, d = 70000, 64
    gen = torch.Generator(device="cuda").manual_seed(7)
    ones = (torch.rand(n, generator=gen, device="cuda") < 0.7).to(torch.int32)
    cu = torch.cat([ints([0]), ones.cumsum(0).to(torch.int32)])
    T = int(cu[-1])
    lens = ones * (torch.rand(n, generator=gen, device="cuda") < 0.8).to(torch.int32)
    x = torch.randn((T, 2 * d), generator=gen, device="cuda").to(TORCH[dtype])
    pool = torch.zeros((2, n, 1, 1, d), device="cuda", dtype=TORCH[dtype])
    cache = mgb.kv_cache(pool[0], pool[1], torch.arange(n, dtype=torch.int32, device="cuda").flip(0).view(n, 1))
    ws = torch.empty(mgb.mgb_attention_tree_ws_bytes(n, T, nq, 1, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_tree_prepare(n, T, nq, 1, d, cu, lens, None, ws)
    mgb.mgb_kv_append_tree(plan, mgb.kv_append_desc(T, n, nq, 0, False, 0), cache, None, None, x, x[:, d:], 0, 2 * d,
                           None, 0, None, 0)
    live = (lens > 0)[ones.bool()]
    q = torch.randn((T, nq * d), generator=gen, device="cuda").to(TORCH[dtype])
    o = _attend(plan, cache, q)
    new = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    mgb.mgb_kv_accept(plan, cache, lens - 1, new)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    want = x[:, d:].repeat(1, nq)
    assert torch.equal(o[live], want[live]) and bool((o[~live] == 3.0).all())
    assert torch.equal(new, lens)
    kept = pool[1].flip(0)[lens > 0][:, 0, 0]
    assert torch.equal(kept, x[live][:, d:]) and not bool((pool.flip(1)[:, lens == 0] != 0).any())


def _job(seed, dtype, nq, nkv, d, page, seqs):
    rng = np.random.default_rng(seed)
    b = Batch([(c, random_tree(rng, m)) for c, m in seqs])
    c = Cache(rng, b.lens, page, nkv, d, dtype)
    return b.plan(nq, nkv, d), c, dev(values(rng, (b.tokens, nq * d), dtype), dtype)


def test_plans_on_streams_of_their_own():
    """Kernels of all forms at the same time, each with its own plan."""
    jobs = [_job(60, "bf16", 8, 2, 128, 16, [(3000, 9), (70, 30), (1500, 60)]),
            _job(61, "bf16", 4, 4, 64, 24, [(700, 3), (20, 1), (4000, 2)]),
            _job(62, "f32", 8, 2, 64, 16, [(600, 9), (33, 14)]),
            _job(63, "bf16", 4, 2, 64, 7, [(600, 19), (33, 34)])]
    alone = [_attend(p, c.desc, q) for p, c, q in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = [torch.zeros_like(q) for _, _, q in jobs]
        torch.cuda.synchronize()
        for _ in range(3):
            for st, (p, c, q), o in zip(streams, jobs, outs):
                with torch.cuda.stream(st):
                    _attend(p, c.desc, q, o)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert mgb.mgb_device_status() == mgb.MGB_OK


@pytest.mark.parametrize("d,sizes", [(128, (20, 33, 5)), (64, (2, 3, 4)), (64, (20, 33, 5)), (128, (1, 2, 1))])
def test_one_plan_for_layers_of_two_types_and_in_two_graphs(d, sizes):
    """Caches of both types under one plan, in two graphs that are replayed by turns; with twelve
    rows per sequence at head dim 64 the types go to different kernels."""
    rng = np.random.default_rng(64)
    nq, nkv = 8, 2
    b = Batch([(x, random_tree(rng, m)) for x, m in zip((2500, 17, 400), sizes)])
    plan = b.plan(nq, nkv, d)
    layers = []
    for dtype in ("bf16", "f32", "bf16"):
        c = Cache(rng, b.lens, 16, nkv, d, dtype)
        q = dev(values(rng, (b.tokens, nq * d), dtype), dtype)
        layers.append((c, q, _attend(plan, c.desc, q), torch.zeros_like(q)))
    torch.cuda.synchronize()
    graphs = []
    for first in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c, q, _, o in layers[first:]:
                _attend(plan, c.desc, q, o)
        graphs.append(g)
    for g in graphs * 3:
        for x in layers:
            x[3].zero_()
        g.replay()
        for c, q, want, o in layers[graphs.index(g):]:
            assert torch.equal(o, want)
    assert mgb.mgb_device_status() == mgb.MGB_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 7])
def test_sequences_that_share_pages(dtype, m):
    """A common prefix held once: the same bits as with a copy per sequence."""
    nq, nkv, d, page, n, common, own = 8, 2, 128, 16, 5, 40, 4
    rng = np.random.default_rng(65)
    b = Batch([(common * page + 3 + 7 * s, random_tree(rng, m)) for s in range(n)])
    prefix = torch.randn((2, common, page, nkv, d), device="cuda")
    tails = torch.randn((2, n * own, page, nkv, d), device="cuda")
    q = torch.randn((b.tokens, nq * d), device="cuda").to(TORCH[dtype])
    outs = []
    for shared in (True, False):
        copies = 1 if shared else n
        pool = torch.cat([prefix] * copies + [tails], dim=1).to(TORCH[dtype])
        at = np.array([[(0 if shared else s * common) + i for i in range(common)]
                       + [copies * common + s * own + i for i in range(own)] for s in range(n)])
        outs.append(_attend(b.plan(nq, nkv, d), mgb.kv_cache(pool[0], pool[1], ints(at)), q))
        assert mgb.mgb_device_status() == mgb.MGB_OK
    assert torch.equal(*outs) and bool((outs[0] != 3.0).any())


@pytest.mark.parametrize("n,tokens", [(0, 0), (0, 5), (3, 0), (3, 5)])
def test_nothing_to_do(n, tokens):
    """No sequences, no rows, or rows that no sequence owns: nothing is written."""
    nq, nkv, d = 4, 2, 64
    ws = torch.full((mgb.mgb_attention_tree_ws_bytes(n, tokens, nq, nkv, d) + 16,), 0xC3, dtype=torch.uint8,
                    device="cuda")
    lens = [7, 0, 9][:n]
    plan = mgb.mgb_attention_tree_prepare(n, tokens, nq, nkv, d, ints([0] * (n + 1)), ints(lens),
                                          ints([-9] * tokens), ws)
    pool = torch.full((2, 4, 16, nkv, d), 2.0, dtype=torch.bfloat16, device="cuda")
    cache = mgb.kv_cache(pool[0], pool[1], ints([[0, 1]] * max(n, 1)))
    x = torch.ones((max(tokens, 1), (nq + 2 * nkv) * d), dtype=torch.bfloat16, device="cuda")
    w, o = x.shape[1], torch.full((max(tokens, 1), nq * d), 3.0, dtype=torch.bfloat16, device="cuda")
    mgb.mgb_kv_append_tree(plan, mgb.kv_append_desc(tokens, n, nq, 0, False, 0), cache, None, x, x[:, nq * d:],
                           x[:, (nq + nkv) * d:], w, w, o, nq * d, None, 0)
    mgb.mgb_attention_tree(plan, cache, x, w, o, nq * d)
    new = torch.full((max(n, 1),), 9, dtype=torch.int32, device="cuda")
    mgb.mgb_kv_accept(plan, cache, ints([-1] * max(n, 1)), new)
    none = ints([0])[:0]
    mgb.mgb_kv_copy_pages(cache, none, none, none)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert bool((pool == 2.0).all()) and bool((o == 3.0).all())
    assert new.tolist() == (lens if n else [9])


def _rows(q, k, v, ctx, m, d, page=16, tree=None):
    """q [n, m, nq, d]; k, v [n, tokens, nkv, d], pages in order; ctx + m tokens each."""
    n, _, nq, _ = q.shape
    T, nkv = k.shape[1:3]
    pool = lambda x: x.reshape(n * T // page, page, nkv, d)
    cache = mgb.kv_cache(pool(k), pool(v), ints(np.arange(n * T // page).reshape(n, -1)))
    b = Batch([(ctx, drafts.chain(m) if tree is None else tree)] * n)
    lse = torch.full((n * m, nq), 3.0, device="cuda")
    o = _attend(b.plan(nq, nkv, d), cache, q.reshape(n * m, nq * d), lse=lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    return o.view(n, m, nq, d), lse.view(n, m, nq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx", [1, 40, 3000])
@pytest.mark.parametrize("m", [2, 9, 60])
def test_nan_and_infinity(dtype, d, ctx, m):
    """Per sequence one row's query is NaN, or all scores of a KV head -inf, or one score +inf or
    NaN, or only some -inf; the other heads and rows keep their bits."""
    rng = np.random.default_rng(66)
    n, nq, nkv, T = 5, 8, 2, 3200
    q, k, v = (dev(values(rng, s, dtype), dtype) for s in ((n, m, nq, d), (n, T, nkv, d), (n, T, nkv, d)))
    q[:, :, 4:, 0] = 0.0                       # heads 0 .. 3 read KV head 0, 4 .. 7 head 1
    want, wlse = _rows(q, k, v, ctx, m, d)
    q, k = q.clone(), k.clone()
    at = ctx // 2
    q[0, m // 2, 2, 5] = float("nan")
    q[1:, :, 0:4, 0] = 1.0
    k[1, :ctx + m, 0, 0] = -INF
    k[2, at, 0, 0] = INF
    k[3, at, 0, 0] = float("nan")
    k[4, at, 0, 0] = -INF
    o, lse = _rows(q, k, v, ctx, m, d)
    assert bool(o[0, m // 2, 2].isnan().all()) and bool(lse[0, m // 2, 2].isnan())
    assert bool(o[1, :, :4].isnan().all()) and bool((lse[1, :, :4] == -INF).all())
    assert bool(o[2, :, :4].isnan().all())                    # inf - inf
    assert bool(o[3, :, :4].isnan().all()) and bool(lse[3, :, :4].isnan().all())
    assert bool(o[4, :, :4].isfinite().all()) and bool(lse[4, :, :4].isfinite().all())
    same = torch.ones((n, m, nq), dtype=torch.bool, device="cuda")
    same[0, m // 2, 2] = False
    same[1:, :, :4] = False
    assert torch.equal(o[same], want[same]) and torch.equal(lse[same], wlse[same])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,nq", [(2, 2), (13, 2), (70, 4)])
@pytest.mark.parametrize("size", [2.0 ** 20, 1e9, 1e30, 2e37])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_equal_scores(dtype, d, m, nq, size, sign):
    """Scores that are all the same large number, up to near the type's lowest: every visible
    key has the same weight. (n additions in float32; in bf16 the weights' parts, 2^-16; the
    output's half step.)"""
    rng = np.random.default_rng(67)
    ctx, T = 300, 384
    q, k, v = (dev(values(rng, s, dtype), dtype) for s in ((1, m, nq, d), (1, T, 1, d), (1, T, 1, d)))
    q.zero_()
    q[..., 0] = float(d) ** 0.5
    k[..., 0] = sign * size
    tree = random_tree(rng, m)
    o, lse = _rows(q, k, v, ctx, m, d, tree=tree)
    score = float(q[0, 0, 0, 0].double() * k[0, 0, 0, 0].double()) / d ** 0.5
    half = torch.finfo(TORCH[dtype]).eps / 2
    for i in (0, 1, m // 2, m - 1):
        keys = list(range(ctx)) + [ctx + j for j in drafts.path(tree, i)]
        x = v[0, keys, 0].double()
        mean, mag = x.mean(0), x.abs().mean(0)
        e = (len(keys) + 4) * 2.0 ** -23 + (2.0 ** -16 if dtype == "bf16" else 0.0)
        for h in range(nq):
            err = (o[0, i, h].double() - mean).abs()
            assert bool((err <= mag * e * (1 + half) + half * mean.abs()).all())
            assert abs(float(lse[0, i, h]) - (score + np.log(len(keys)))) <= 2.0 ** -21 * abs(score)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,nq,page", [(2, 2, 16), (13, 2, 16), (13, 2, 5), (70, 4, 16)])
@pytest.mark.parametrize("ctx", [120, 2900])
def test_weights_are_held_in_two_parts(d, m, nq, page, ctx):
    """bf16: beside the output's half step the weights are off by 2^-16, not by 2^-8: values of
    one sign, whose errors do not cancel, all of which a single key offsets to about zero."""
    rng = np.random.default_rng(68)
    T = (ctx + m + page - 1) // page * page
    q, k, v = (values(rng, s, "bf16") for s in ((1, m, nq, d), (1, T, 1, d), (1, T, 1, d)))
    q, v = q / 8, np.abs(v)                     # (small scores, whose own error is small)
    v[0, 0] = 0.0
    sc = np.einsum("mhd,td->mht", q[0], k[0, :, 0]) / d ** 0.5
    seen = np.arange(T)[None, :] <= ctx + np.arange(m)[:, None]
    p = np.where(seen[:, None], np.exp(sc - np.where(seen[:, None], sc, -INF).max(-1, keepdims=True)), 0.0)
    p /= p.sum(-1, keepdims=True)
    # the first key's value takes what the others add up to in row 0, head 0, rounded
    rest = p[0, 0] @ v[0, :, 0]
    v[0, 0, 0] = torch.tensor(-rest / p[0, 0, 0]).bfloat16().double().numpy()
    ref, mag = p @ v[0, :, 0], p @ np.abs(v[0, :, 0])
    o, _ = _rows(*(dev(x, "bf16") for x in (q, k, v)), ctx, m, d, page)
    qk = np.einsum("mhd,td->mht", np.abs(q[0]), np.abs(k[0, :, 0])).max() / d ** 0.5
    score = d * 2.0 ** -23 * qk + 2.0 ** -22 * (1 + qk)
    e = 2 * score + 2.0 ** -21 + (ctx + m) * 2.0 ** -23 + 2.0 ** -16
    assert e < 2.0 ** -10
    tol = e * mag + 2.0 ** -8 * (np.abs(ref) + e * mag)
    assert (np.abs(o[0].double().cpu().numpy() - ref) <= tol).all()
