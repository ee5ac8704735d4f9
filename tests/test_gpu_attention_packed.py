"""GPU parity of mgb_attention_packed_fwd against the float64 oracle: lengths
around the tile borders, empty sequences, rows of no sequence, group sizes,
strides, values of one sequence kept out of the others, the dense kernel on
equal lengths, long sequences, repeats, graph replay, bad row offsets."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import serving
from tests.serving_util import MGB, TORCH, check_attention, dev, host, ints, values
from tests.util import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _plan(cu, tokens, causal, guard=None):
    n = mgb.mgb_attention_packed_ws_bytes(len(cu) - 1, tokens)
    ws = guard.empty((n,), torch.uint8) if guard else torch.empty(n, dtype=torch.uint8, device="cuda")
    ws.fill_(0xC3)
    return mgb.mgb_attention_packed_prepare(len(cu) - 1, tokens, causal, ints(cu), ws)


def _sums(q, k, v, cu, causal):
    """sum p |v| [T, nq, d], max over visible keys of sum |q k| / sqrt(d) [T, nq], visible keys [T, nq]."""
    T, nq, d = q.shape
    g = nq // k.shape[1]
    a, m, n = np.zeros((T, nq, d)), np.zeros((T, nq)), np.ones((T, nq))
    for s, e in zip(cu[:-1], cu[1:]):
        L = e - s
        if L <= 0:
            continue
        seen = np.tril(np.ones((L, L), dtype=bool)) if causal else np.ones((L, L), dtype=bool)
        n[s:e] = seen.sum(1)[:, None]
        for h in range(nq):
            x = np.where(seen, q[s:e, h] @ k[s:e, h // g].T / np.sqrt(d), -np.inf)
            p = np.exp(x - x.max(1, keepdims=True))
            a[s:e, h] = p / p.sum(1, keepdims=True) @ np.abs(v[s:e, h // g])
            y = np.abs(q[s:e, h]) @ np.abs(k[s:e, h // g]).T / np.sqrt(d)
            m[s:e, h] = np.where(seen, y, 0).max(1)
    return a, m, n


def _run(seed, dtype, nq, nkv, d, causal, lens, tail=0, scale=1.0, poison=None, pad_cols=0):
    rng = np.random.default_rng(seed)
    cu = np.cumsum([0] + list(lens))
    T = int(cu[-1]) + tail
    x = values(rng, (T, nq + 2 * nkv, d), dtype)
    x[:, :nq] = values(rng, (T, nq, d), dtype, scale)
    given = x.copy()
    if tail:
        given[cu[-1]:] = np.nan
    if poison is not None:
        given[cu[poison]:cu[poison + 1]] = np.nan
    w = (nq + 2 * nkv) * d + pad_cols
    flat = np.full((T, w), np.nan)
    flat[:, :w - pad_cols] = given.reshape(T, -1)
    qkv = dev(flat, dtype)
    g = Guarded()
    o = g.empty((T, nq * d + pad_cols), TORCH[dtype], 3.0)
    lse = g.empty((nq, T), torch.float32, 3.0)
    plan = _plan(cu, T, causal, g)
    runs = []
    for _ in range(2):
        mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, MGB[dtype], qkv, qkv[:, nq * d:],
                                     qkv[:, (nq + nkv) * d:], w, w, o, nq * d + pad_cols, lse)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        runs.append((host(o), host(lse)))
    g.check()
    for a, b in zip(*runs):
        np.testing.assert_array_equal(a, b)
    got, glse = runs[0]
    assert (got[:, nq * d:] == 3.0).all()
    got = got[:, :nq * d].reshape(T, nq, d)
    live = np.zeros(T, dtype=bool)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        live[a:b] = s != poison
    behind = slice(cu[-1], None)
    assert (got[behind] == 3.0).all() and (glse[:, behind] == 3.0).all()
    q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
    ref, rlse = serving.packed_attention(q, k, v, cu, causal)
    a, m, n = _sums(q, k, v, cu, causal)
    check_attention(got[live], glse.T[live], ref[live], rlse.T[live], a[live], m[live], n[live], d, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[1, 0, 127, 128, 129, 2, 255, 256, 257, 0], [5000, 3, 700], [0, 0], [1]])
def test_work_lists(lens, causal):
    """The plan's lists hold every block of 256 (128) query rows once, longest first."""
    cu = [int(x) for x in np.cumsum([0] + lens)]
    T, n = cu[-1] + 5, len(lens)
    plan = _plan(cu, T, causal)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    ws = plan.tensors[0].cpu().numpy()
    up = lambda x: (x + 255) // 256 * 256
    counts = ws[:32].view(np.int32)[[0, 4]]
    at = 256 + up(8 * (n + 1))
    for R, count in zip((256, 128), counts):
        room = T // R + min(n, T)
        got = ws[at:at + 16 * room].view(np.int32).reshape(-1, 4)[:count]
        want = sorted((cu[s], lens[s], q0, 0) for s in range(n) for q0 in range(0, lens[s], R))
        assert sorted(map(tuple, got.tolist())) == want and count <= room
        cost = [(min(L, q0 + R) if causal else L) // 128 for _, L, q0, _ in got.tolist()]
        assert all(a >= b - 1 for a, b in zip(cost, cost[1:]))
        at += up(16 * room)


BORDERS = [1, 0, 127, 128, 129, 2, 255, 256, 257, 0, 63, 65, 385, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_at_the_borders(dtype, d, causal):
    _run(21, dtype, 4, 2, d, causal, BORDERS, tail=9)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (3, 3), (7, 1), (20, 4), (32, 8)])
def test_group_sizes(dtype, nq, nkv):
    _run(22, dtype, nq, nkv, 128, True, [70, 300, 5], pad_cols=24)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("poison", [0, 1, 2])
def test_sequences_do_not_touch_each_other(dtype, causal, poison):
    """One sequence's values are NaN, and so are the rows behind the last: the
    other sequences, which share tiles with them, come out right."""
    _run(23, dtype, 2, 1, 64, causal, [100, 90, 140], tail=30, poison=poison)
    _run(23, dtype, 2, 1, 128, causal, [100, 90, 140], tail=200, poison=poison)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(dtype):
    _run(24, dtype, 4, 2, 128, True, [300, 513], scale=20.0)


@pytest.mark.parametrize("dtype,lens", [("f32", [1]), ("bf16", [1]), ("f32", [1100, 3]), ("bf16", [2900, 3])])
def test_one_token_and_long(dtype, lens):
    _run(25, dtype, 2, 1, 64, True, lens)


def test_more_items_than_ctas():
    """Every CTA takes several items; more sequences than the scan's block."""
    rng = np.random.default_rng(26)
    _run(26, "bf16", 2, 2, 64, True, [int(x) for x in rng.integers(0, 5, size=1300)], tail=2)
    _run(27, "bf16", 16, 4, 64, True, [int(x) for x in rng.integers(0, 600, size=14)])


@pytest.mark.parametrize("causal", [True, False])
def test_equal_lengths_match_the_dense_kernel(causal):
    B, S, nq, nkv, d = 3, 384, 4, 2, 128
    qkv = torch.randn((B * S, (nq + 2 * nkv) * d), device="cuda").bfloat16()
    w = qkv.shape[1]
    a = (qkv, qkv[:, nq * d:], qkv[:, (nq + nkv) * d:], w, w)
    o1, o2 = (torch.empty((B * S, nq * d), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    l1 = torch.empty((B, nq, S), device="cuda")
    l2 = torch.empty((nq, B * S), device="cuda")
    mgb.mgb_attention_fwd(B, S, nq, nkv, d, causal, mgb.MGB_BF16, *a, o1, l1)
    mgb.mgb_attention_packed_fwd(_plan([0, S, 2 * S, 3 * S], B * S, causal), nq, nkv, d, mgb.MGB_BF16, *a,
                                 o2, nq * d, l2)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    # two roundings to bf16 of nearly the same value, and of nearly the same weights
    assert (o1.float() - o2.float()).norm() <= 2.0 ** -8 * o1.float().norm()
    assert (l1.transpose(0, 1).reshape(nq, -1) - l2).abs().max() <= 1e-5 * l1.abs().max()


def test_nothing_to_do():
    z = torch.zeros((0, 64), device="cuda", dtype=torch.bfloat16)
    for cu, T in (([0], 0), ([0, 0], 0)):
        mgb.mgb_attention_packed_fwd(_plan(cu, T, True), 1, 1, 64, mgb.MGB_BF16, z, z, z, 64, 64, z, 64)
    x = torch.full((5, 64), 2.0, device="cuda", dtype=torch.bfloat16)
    o = x.clone()
    mgb.mgb_attention_packed_fwd(_plan([0, 0, 0], 5, True), 1, 1, 64, mgb.MGB_BF16, x, x, x, 64, 64, o, 64)
    assert mgb.mgb_device_status() == mgb.MGB_OK and torch.equal(o, x)


def test_captured_batch_follows_the_offsets():
    rng = np.random.default_rng(28)
    T, nq, nkv, d = 700, 4, 2, 64
    x = values(rng, (T, nq + 2 * nkv, d), "bf16")
    qkv = dev(x.reshape(T, -1), "bf16")
    w = qkv.shape[1]
    cu = ints([0, 300, 600, 700])
    ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(3, T), dtype=torch.uint8, device="cuda")
    o = torch.zeros((T, nq * d), device="cuda", dtype=torch.bfloat16)

    def step():
        plan = mgb.mgb_attention_packed_prepare(3, T, True, cu, ws)
        mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, mgb.MGB_BF16, qkv, qkv[:, nq * d:],
                                     qkv[:, (nq + nkv) * d:], w, w, o, nq * d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for now in ([0, 300, 600, 700], [0, 1, 1, 690], [0, 128, 384, 500]):
        cu.copy_(ints(now))
        o.fill_(3.0)
        g.replay()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
        ref, _ = serving.packed_attention(q, k, v, now)
        a, m, n = _sums(q, k, v, now, True)
        got, end = host(o).reshape(T, nq, d), now[-1]
        check_attention(got[:end], None, ref[:end], None, a[:end], m[:end], n[:end], d, "bf16")
        assert (got[end:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 40, 30, 30], [0, 40, 101, 101], [-1, 40, 60, 60], [0, 40, -5, -5]])
def test_bad_offsets_are_reported(dtype, cu):
    """A sequence with bad offsets counts as empty; the good ones are served."""
    x = torch.randn((100, 3 * 64), device="cuda").to(TORCH[dtype])
    o, r = (torch.zeros((100, 64), device="cuda", dtype=TORCH[dtype]) for _ in range(2))
    call = lambda plan, out: mgb.mgb_attention_packed_fwd(plan, 1, 1, 64, MGB[dtype], x, x[:, 64:], x[:, 128:],
                                                          192, 192, out, 64)
    call(_plan(cu, 100, True), o)
    assert mgb.mgb_device_status() == mgb.MGB_ERR_INDEX
    if cu[0] == 0:  # the first sequence is a good one
        call(_plan([0, cu[1]], 100, True), r)
        assert torch.equal(o[:cu[1]], r[:cu[1]]) and bool((o[:cu[1]] != 0).any())
    assert mgb.mgb_device_status() == mgb.MGB_OK
