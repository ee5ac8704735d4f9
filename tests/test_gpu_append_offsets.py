"""Row offsets of mgb_kv_append that are not what they must be: each is
reported, and a row is stored only where its own sequence's new rows go."""
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from tests.serving_util import ints

pytestmark = pytest.mark.gpu

PAGE, PAGES, D = 8, 4, 64


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _append(cu, lens, tokens, nq=2, whole=False, dtype=torch.bfloat16):
    """(status, rows of q_out written, {(sequence, position)} written): sequence s has pages
    PAGES s .. of its own."""
    n = len(lens)
    qkv = torch.randn((tokens, (nq + 2) * D), device="cuda").to(dtype)
    pool = torch.zeros((2, n * PAGES, PAGE, 1, D), device="cuda", dtype=dtype)
    table = ints([[s * PAGES + i for i in range(PAGES)] for s in range(n)])
    out = torch.zeros((tokens, nq * D), device="cuda", dtype=dtype)
    desc = mgb.kv_append_desc(tokens, n, nq, D, False, 64, **(dict(whole=True) if whole else {}))
    mgb.mgb_kv_append(desc, mgb.kv_cache(pool[0], pool[1], table), None if cu is None else ints(cu),
                      ints(lens), rope_table(64, D), qkv, qkv[:, nq * D:], qkv[:, (nq + 1) * D:],
                      (nq + 2) * D, (nq + 2) * D, out, nq * D, None, 0)
    status = mgb.mgb_device_status()
    rows = [t for t in range(tokens) if bool((out[t] != 0).any())]
    slots = (pool != 0).any(-1).all(0).view(n, PAGES * PAGE)
    assert bool((slots == (pool != 0).any(-1).any(0).view(n, -1)).all())
    return status, rows, {(s, p) for s in range(n) for p in range(PAGES * PAGE) if bool(slots[s, p])}


@pytest.mark.parametrize("cu,lens,tokens,rows,slots", [
    # rows before the first offset belong to no sequence
    ([2, 4], [10], 6, [2, 3], {(0, 8), (0, 9)}),
    # decreasing: no row may go behind its sequence's length
    ([0, 5, 3], [9, 9], 6, [0, 1, 2], {(0, 4), (0, 5), (0, 6)}),
    ([0, 3, 2], [3, 0], 4, [0, 1], {(0, 0), (0, 1)}),
    # outside [0, tokens]
    ([-1, 4], [6], 6, [], set()),
    ([0, 9], [9], 6, [], set()),
    ([0, 2, 8], [2, 0], 6, [0, 1], {(0, 0), (0, 1)}),          # .. the end of a padding sequence
    ([0, 2, 2 ** 31 - 1], [2, 5], 6, [0, 1], {(0, 0), (0, 1)}),
    ([-2 ** 31, 2, 4], [2, 4], 6, [2, 3], {(1, 2), (1, 3)}),
    # bad offsets of sequences that no row is looked up in
    ([0, 2, -7, 4], [2, 3, 4], 2, None, None),
])
@pytest.mark.parametrize("nq", [2, 70])
def test_bad_offsets(cu, lens, tokens, rows, slots, nq):
    for dtype in (torch.bfloat16, torch.float32):
        st, r, w = _append(cu, lens, tokens, nq, dtype=dtype)
        assert st == mgb.MGB_ERR_INDEX
        if rows is not None:
            assert r == rows and w == slots
        own = {(s, lens[s] - (cu[s + 1] - cu[s]) + i) for s in range(len(lens))
               for i in range(min(max(cu[s + 1] - cu[s], 0), 64))}
        assert w <= own                       # never over what a sequence had cached, nor behind its end
        assert mgb.mgb_device_status() == mgb.MGB_OK


def test_bad_offset_far_behind_the_rows():
    """Thousands of sequences, one bad offset, whichever block looks."""
    n = 3000
    good = [min(t, 40) for t in range(n + 1)]
    lens = [1] * 40 + [0] * (n - 40)
    assert _append(good, lens, 40)[0] == mgb.MGB_OK
    for at in (41, 1500, n):
        cu = list(good)
        cu[at] = 39
        assert _append(cu, lens, 40)[0] == mgb.MGB_ERR_INDEX


@pytest.mark.parametrize("cu,lens,tokens", [([0, 0, 0], [5, 0], 3), ([0, 3, 3, 6], [3, 0, 20], 9), ([0, 4], [0], 4)])
def test_good_offsets_are_not_reported(cu, lens, tokens):
    st, rows, slots = _append(cu, lens, tokens)
    assert st == mgb.MGB_OK
    want = {(s, lens[s] - (cu[s + 1] - cu[s]) + i) for s in range(len(lens)) if lens[s]
            for i in range(cu[s + 1] - cu[s])}
    assert slots == want and len(rows) == len(want)


@pytest.mark.parametrize("value", [150, -1, 10 ** 9, 701])
def test_bad_offset_in_a_large_step(value):
    """The form for many tokens: 350 sequences of two rows, one offset wrong."""
    cu = [2 * s for s in range(351)]
    cu[100] = value
    lens = [3] * 350
    st, rows, w = _append(cu, lens, 700)
    assert st == mgb.MGB_ERR_INDEX
    assert w <= {(s, 1 + i) for s in range(350) for i in range(2)}
    good = [s for s in range(350) if s not in (99, 100)]
    if value >= 0:
        # sequences on one side of the bad offset at least are served in full
        assert {(s, 1 + i) for s in good if s < 64 for i in range(2)} <= w


@pytest.mark.parametrize("cu,lens,tokens,bad", [
    ([0, 3, 6], [5, 3], 6, [0]),              # the first continues two cached tokens
    ([0, 3, 6], [3, 2], 6, [1]),              # more rows than tokens
    ([0, 3, 6, 8], [3, 0, 2], 9, []),         # a padding sequence, a row of none
    ([0, 1, 1, 2], [1, 7, 4], 2, [2]),        # no rows: nothing to attend, not looked at
    (None, [1, 2, 1], 3, [1]),
])
def test_whole_sequences(cu, lens, tokens, bad):
    st, rows, slots = _append(cu, lens, tokens, whole=True)
    assert st == (mgb.MGB_ERR_INDEX if bad else mgb.MGB_OK)
    at = cu or list(range(tokens + 1))
    good = [s for s in range(len(lens)) if s not in bad and lens[s] and at[s + 1] > at[s]]
    assert slots == {(s, p) for s in good for p in range(lens[s])}
    assert rows == [t for s in good for t in range(at[s], at[s + 1])]


def test_a_prompt_batch_over_cached_tokens_is_reported():
    """Packed attention sees the new rows alone: the runner's packed step of a sequence
    that already has tokens in the cache must not pass for a right one."""
    import numpy as np
    from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
    from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)
    pools = torch.zeros((2, 8, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    layer = ServingLayer(shape, layer_inputs(shape), pools[0], pools[1], rope_table(32, 64))
    table, cu = ints(np.arange(8).reshape(2, 4)), ints([0, 5, 9])
    x = torch.randn((9, 128), device="cuda").bfloat16()
    layer.step(x, ServingBatch(shape, table, ints([5, 4]), cu, 9))
    assert mgb.mgb_device_status() == mgb.MGB_OK
    before = pools.clone()
    layer.step(x, ServingBatch(shape, table, ints([5, 8]), cu, 9))
    assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
    assert torch.equal(pools, before)      # the first stored what it had, the second nothing
