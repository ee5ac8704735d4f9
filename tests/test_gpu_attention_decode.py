"""GPU parity of mgb_attention_decode against the float64 oracle: lengths
around the unit and slice borders, empty sequences, page sizes and layouts,
group sizes, splits over many CTAs, poisoned unused slots, strides, repeats,
graph replay, device-side index errors."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import serving
from tests.serving_util import MGB, TORCH, Cache, check_attention, dev, host, ints, values
from tests.util import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _sums(q, c, lens):
    """sum p |v| [n, nq, d] and max_j sum |q k| / sqrt(d) [n, nq]."""
    n, nq, d = q.shape
    g = nq // c.k.shape[2]
    a, m = np.zeros((n, nq, d)), np.zeros((n, nq))
    for s in range(n):
        if lens[s] == 0:
            continue
        k, v = (serving.gather_cache(x, c.table[s], lens[s]) for x in (c.k, c.v))
        for h in range(nq):
            x = k[:, h // g] @ q[s, h] / np.sqrt(d)
            p = np.exp(x - x.max())
            a[s, h] = (p / p.sum()) @ np.abs(v[:, h // g])
            m[s, h] = (np.abs(k[:, h // g]) @ np.abs(q[s, h])).max() / np.sqrt(d)
    return a, m


def _plan(lens, nq, nkv, d, guard=None):
    n = mgb.mgb_attention_decode_ws_bytes(len(lens), nq, nkv, d)
    ws = guard.empty((n,), torch.uint8) if guard else torch.empty(n, dtype=torch.uint8, device="cuda")
    ws.fill_(0xC3)   # whatever was there before
    return mgb.mgb_attention_decode_prepare(len(lens), nq, nkv, d, ints(lens), ws), ws


def _run(seed, dtype, nq, nkv, d, page, lens, head_major=False, scale=1.0):
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, page, nkv, d, dtype, head_major)
    n = len(lens)
    q = values(rng, (n, nq, d), dtype, scale)
    wide = dev(np.concatenate([q.reshape(n, -1), values(rng, (n, 16), dtype)], axis=1), dtype)
    g = Guarded()
    o = g.empty((n, nq * d + 32), TORCH[dtype], 3.0)
    lse = g.empty((n, nq), torch.float32)
    plan, ws = _plan(lens, nq, nkv, d, g)
    first = None
    for _ in range(2):   # the second call finds the counters as the first left them
        mgb.mgb_attention_decode(plan, c.desc, wide, nq * d + 16, o, nq * d + 32, lse)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        now = host(o), host(lse)
        if first is not None:
            assert (now[0] == first[0]).all() and (now[1] == first[1]).all()
        first = now
    g.check()
    assert (first[0][:, nq * d:] == 3.0).all()
    got = first[0][:, :nq * d].reshape(n, nq, d)
    ref, ref_lse = serving.decode_attention(q, c.k, c.v, c.table, lens)
    a, m = _sums(q, c, lens)
    check_attention(got, first[1], ref, ref_lse, a, m, np.array(lens)[:, None] * np.ones(nq), d, dtype)
    for s, x in enumerate(lens):
        if x == 0:
            assert (got[s] == 0).all()


BORDERS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,head_major", [(16, False), (1, False), (24, True), (64, True), (100, False)])
def test_lengths_at_the_borders(dtype, d, page, head_major):
    _run(11, dtype, 4, 2, d, page, BORDERS, head_major)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (2, 1), (3, 3), (7, 1), (16, 2), (16, 1), (17, 1), (40, 2),
                                    (32, 1), (71, 1)])
def test_group_sizes(dtype, nq, nkv):
    """Up to 16 query heads share an item; larger groups take several, the last one smaller."""
    _run(12, dtype, nq, nkv, 128, 16, [70, 0, 300, 5])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("lens", [[1], [4000], [2500, 1, 0, 3300], [700] * 5])
def test_split_over_the_length(dtype, d, lens):
    """One KV head: a long sequence is split over many CTAs and joined."""
    _run(13, dtype, 8, 1, d, 32, lens)


def test_range_of_lengths_and_many_items():
    """More items than CTAs: ranges that begin and end inside items."""
    rng = np.random.default_rng(14)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(900), size=90))]
    _run(14, "bf16", 16, 8, 64, 16, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores of +-200: the running maximum moves often, most weights vanish."""
    _run(15, dtype, 8, 2, 128, 16, [500, 65, 1000], scale=20.0)


def test_more_sequences_than_the_scan_block():
    lens = [(i * 7) % 5 for i in range(1500)]
    _run(16, "bf16", 1, 1, 64, 4, lens)


def test_no_lse_no_sequences():
    rng = np.random.default_rng(1)
    c = Cache(rng, [9], 4, 1, 64, "bf16")
    q = dev(values(rng, (1, 64), "bf16"), "bf16")
    a, b = torch.empty_like(q), torch.empty_like(q)
    plan, ws = _plan([9], 1, 1, 64)
    mgb.mgb_attention_decode(plan, c.desc, q, 64, a, 64, torch.empty((1, 1), device="cuda"))
    mgb.mgb_attention_decode(plan, c.desc, q, 64, b, 64, None)
    assert torch.equal(a, b)
    plan, ws = _plan([], 1, 1, 64)
    mgb.mgb_attention_decode(plan, c.desc, q, 64, a.fill_(5), 64, None)
    assert mgb.mgb_device_status() == mgb.MGB_OK and (a == 5).all()


def test_layers_share_a_plan_and_streams_have_their_own():
    """One prepare serves several caches in turn; two plans run side by side
    on two streams."""
    rng = np.random.default_rng(2)
    lens, nq, nkv, d = [1300, 40, 2100], 4, 1, 128
    caches = [Cache(rng, lens, 16, nkv, d, "bf16") for _ in range(3)]
    q = values(rng, (3, nq, d), "bf16")
    tq = dev(q.reshape(3, -1), "bf16")
    outs = [torch.empty_like(tq) for _ in caches]
    plan, ws = _plan(lens, nq, nkv, d)
    for c, o in zip(caches, outs):
        mgb.mgb_attention_decode(plan, c.desc, tq, nq * d, o, nq * d)
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [_plan(lens, nq, nkv, d) for _ in streams]
    torch.cuda.synchronize()
    again = [[torch.empty_like(tq) for _ in caches] for _ in streams]
    for _ in range(5):
        for st, (p, _w), os in zip(streams, plans, again):
            for c, o in zip(caches, os):
                mgb.mgb_attention_decode(p, c.desc, tq, nq * d, o, nq * d, None, st)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    torch.cuda.synchronize()
    for i, c in enumerate(caches):
        ref, _ = serving.decode_attention(q, c.k, c.v, c.table, lens)
        a, m = _sums(q, c, lens)
        check_attention(host(outs[i]).reshape(3, nq, d), None, ref, None, a, m,
                        np.array(lens)[:, None] * np.ones(nq), d, "bf16")
        assert all(torch.equal(outs[i], os[i]) for os in again)


def test_captured_step_follows_the_lengths():
    rng = np.random.default_rng(3)
    most, nq, nkv, d = [700, 90, 1500], 8, 2, 64
    c = Cache(rng, most, 16, nkv, d, "bf16")
    q = values(rng, (3, nq, d), "bf16")
    tq, o = dev(q.reshape(3, -1), "bf16"), torch.zeros((3, nq * d), device="cuda", dtype=torch.bfloat16)
    lens = ints(most)
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(3, nq, nkv, d), dtype=torch.uint8, device="cuda")

    def step():
        plan = mgb.mgb_attention_decode_prepare(3, nq, nkv, d, lens, ws)
        mgb.mgb_attention_decode(plan, c.desc, tq, nq * d, o, nq * d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for now in ([700, 90, 1500], [1, 0, 1499], [64, 65, 66]):
        lens.copy_(ints(now))
        g.replay()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        ref, _ = serving.decode_attention(q, c.k, c.v, c.table, now)
        a, m = _sums(q, c, now)
        check_attention(host(o).reshape(3, nq, d), None, ref, None, a, m,
                        np.array(now)[:, None] * np.ones(nq), d, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["page_high", "page_low", "length", "negative"])
def test_bad_indices_are_reported(dtype, what):
    """A bad page or length of one sequence is an error; the others' results
    do not change."""
    rng = np.random.default_rng(4)
    lens, nq, nkv, d = [50, 40, 30], 2, 1, 64
    c = Cache(rng, lens, 16, nkv, d, dtype)
    q = dev(values(rng, (3, nq * d), dtype), dtype)
    good, bad = torch.empty_like(q), torch.empty_like(q)
    plan, ws = _plan(lens, nq, nkv, d)
    mgb.mgb_attention_decode(plan, c.desc, q, nq * d, good, nq * d)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    if what == "page_high":
        c.ttable[1, 2] = c.n_pages
    elif what == "page_low":
        c.ttable[1, 0] = -1
    else:
        lens = [50, 65 if what == "length" else -3, 30]
    plan, ws = _plan(lens, nq, nkv, d)
    mgb.mgb_attention_decode(plan, c.desc, q, nq * d, bad, nq * d)
    assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
    assert torch.equal(bad[0], good[0]) and torch.equal(bad[2], good[2])
    if what == "negative":
        assert (bad[1] == 0).all()
    assert mgb.mgb_device_status() == mgb.MGB_OK
