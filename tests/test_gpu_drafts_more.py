"""GPU tests of the operators for drafted tokens beside those in test_gpu_kv_tree.py and
test_gpu_tree_more.py: vectors next to each other, many sequences with a bad offset, the time
that many sequences take."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import drafts
from tests.drafts_util import Batch, random_tree
from tests.serving_util import Cache, host, ints

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
