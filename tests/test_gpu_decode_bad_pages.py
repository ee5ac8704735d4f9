"""mgb_attention_decode with bad pages and lengths: the result of every
sequence is defined. A token whose page is bad is left out; a sequence longer
than its row of the table counts as empty. Neither depends on what shared
memory held, and neither changes another sequence's bits."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import serving
from tests.serving_util import Cache, check_attention, dev, host, ints, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _decode(c, q, lens, nq, nkv, d):
    n = len(lens)
    ws = torch.full((mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d),), 0xC3, dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, ints(lens), ws)
    o, lse = torch.full_like(q, 3.0), torch.full((n, nq), 3.0, device="cuda")
    mgb.mgb_attention_decode(plan, c.desc, q, nq * d, o, nq * d, lse)
    return mgb.mgb_device_status(), o, lse


def _check(c, q, got, lse, s, keep, d, dtype):
    """Sequence s against the tokens `keep` alone."""
    qs = host(q)[s].reshape(-1, d)
    nq = qs.shape[0]
    k, v = (x[c.table[s][keep // c.k.shape[1]], keep % c.k.shape[1]] for x in (c.k, c.v))
    g = nq // k.shape[1]
    ref, a = np.zeros((nq, d)), np.zeros((nq, d))
    rl, m = np.zeros(nq), np.zeros(nq)
    for h in range(nq):
        x = k[:, h // g] @ qs[h] / np.sqrt(d)
        p = np.exp(x - x.max())
        rl[h] = x.max() + np.log(p.sum())
        p /= p.sum()
        ref[h], a[h] = p @ v[:, h // g], p @ np.abs(v[:, h // g])
        m[h] = (np.abs(k[:, h // g]) @ np.abs(qs[h])).max() / np.sqrt(d)
    check_attention(host(got)[s].reshape(nq, d), host(lse)[s], ref, rl, a, m, np.full(nq, len(keep)), d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("lens", [[50, 150, 300], [900, 4000, 30]])
def test_tokens_of_bad_pages_are_left_out(dtype, d, page, lens):
    """Every third page of sequence 1, single tokens up to whole stages."""
    rng = np.random.default_rng(31)
    nq, nkv = 8, 2
    c = Cache(rng, lens, page, nkv, d, dtype)
    q = dev(values(rng, (3, nq * d), dtype), dtype)
    st, good, glse = _decode(c, q, lens, nq, nkv, d)
    assert st == mgb.MGB_OK
    used = (lens[1] + page - 1) // page
    gone = list(range(1, used, 3))
    for i, at in enumerate(gone):
        c.ttable[1, at] = [c.n_pages, -1, 2 ** 31 - 1, -2 ** 31][i % 4]
    st, bad, blse = _decode(c, q, lens, nq, nkv, d)
    assert st == mgb.MGB_ERR_INDEX
    for s in (0, 2):
        assert torch.equal(bad[s], good[s]) and torch.equal(blse[s], glse[s])
    t = np.arange(lens[1])
    _check(c, q, bad, blse, 1, t[~np.isin(t // page, gone)], d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 700, 5000])
def test_a_sequence_of_bad_pages_only(dtype, n):
    """A softmax over no token: 0 / 0, log 0."""
    rng = np.random.default_rng(32)
    nq, nkv, d, lens = 4, 2, 128, [600, n, 65]
    c = Cache(rng, lens, 16, nkv, d, dtype)
    q = dev(values(rng, (3, nq * d), dtype), dtype)
    _, good, glse = _decode(c, q, lens, nq, nkv, d)
    c.ttable[1] = -1
    for _ in range(3):
        st, bad, blse = _decode(c, q, lens, nq, nkv, d)
        assert st == mgb.MGB_ERR_INDEX
        assert bool(bad[1].isnan().all()) and bool((blse[1] == float("-inf")).all())
        for s in (0, 2):
            assert torch.equal(bad[s], good[s]) and torch.equal(blse[s], glse[s])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("over", [65, 129, 400, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("where", [0, 1, 2])
def test_a_length_past_the_table_counts_as_empty(dtype, d, over, where):
    rng = np.random.default_rng(33)
    nq, nkv, lens = 4, 2, [64, 33, 50]
    c = Cache(rng, lens, 16, nkv, d, dtype)          # four entries per row: 64 tokens
    q = dev(values(rng, (3, nq * d), dtype), dtype)
    _, good, glse = _decode(c, q, lens, nq, nkv, d)
    wrong = list(lens)
    wrong[where] = over
    st, bad, blse = _decode(c, q, wrong, nq, nkv, d)
    assert st == mgb.MGB_ERR_INDEX
    assert bool((bad[where] == 0).all()) and bool((blse[where] == float("-inf")).all())
    for s in range(3):
        if s != where:
            assert torch.equal(bad[s], good[s]) and torch.equal(blse[s], glse[s])
    st, again, _ = _decode(c, q, lens, nq, nkv, d)
    assert st == mgb.MGB_OK and torch.equal(again, good)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_and_too_long_sequences_side_by_side(dtype):
    """Split items next to lengths past the table, with a plan used twice."""
    rng = np.random.default_rng(34)
    nq, nkv, d = 16, 2, 128
    lens = [3000, 0, 2900, 64, 1]
    c = Cache(rng, lens, 16, nkv, d, dtype)
    q = dev(values(rng, (5, nq * d), dtype), dtype)
    wrong = [3000, 9000, 2900, 3009, 1]               # 188 entries: 3008 tokens
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(5, nq, nkv, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(5, nq, nkv, d, ints(wrong), ws)
    runs = []
    for _ in range(3):
        o, lse = torch.full_like(q, 3.0), torch.full((5, nq), 3.0, device="cuda")
        mgb.mgb_attention_decode(plan, c.desc, q, nq * d, o, nq * d, lse)
        assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
        runs.append((o, lse))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
    o, lse = runs[0]
    assert bool((o[[1, 3]] == 0).all()) and bool((lse[[1, 3]] == float("-inf")).all())
    for s in (0, 2, 4):
        _check(c, q, o, lse, s, np.arange(lens[s]), d, dtype)
