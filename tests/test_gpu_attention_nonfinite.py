"""NaN and infinity in what the serving attention kernels see: results follow
the definition, softmax over the visible keys, row by row; log-sum-exp too. What
is masked (tokens behind the length, later keys of a causal sequence) has no say."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from tests.serving_util import MGB, TORCH, dev, ints, values

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _decode(q, k, v, lens, d, page=16):
    """q [n, nq, d]; k, v [n, tokens, nkv, d], pages in order."""
    n, nq, _ = q.shape
    T, nkv = k.shape[1:3]
    pool = lambda x: x.reshape(n * T // page, page, nkv, d)
    cache = mgb.kv_cache(pool(k), pool(v), ints(np.arange(n * T // page).reshape(n, -1)))
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, ints(lens), ws)
    o, lse = torch.full_like(q, 3.0), torch.full((n, nq), 3.0, device="cuda")
    mgb.mgb_attention_decode(plan, cache, q, nq * d, o, nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    return o, lse


def _packed(x, cu, nq, nkv, d, dtype, causal):
    """x [T, nq + 2 nkv, d]."""
    T, w = x.shape[0], (nq + 2 * nkv) * d
    flat = x.reshape(T, w)
    ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(len(cu) - 1, T), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_packed_prepare(len(cu) - 1, T, causal, ints(cu), ws)
    o, lse = torch.full((T, nq, d), 3.0, dtype=x.dtype, device="cuda"), torch.full((nq, T), 3.0, device="cuda")
    mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, MGB[dtype], flat, flat[:, nq * d:], flat[:, (nq + nkv) * d:],
                                 w, w, o, nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [1, 40, 3000])
def test_decode(dtype, d, length):
    """Per sequence one head's query is NaN, or all its scores -inf, or one score
    +inf or NaN, or only some -inf; the other heads keep their bits."""
    rng = np.random.default_rng(41)
    n, nq, nkv, T = 5, 8, 2, 3008
    q, k, v = (dev(values(rng, s, dtype), dtype) for s in ((n, nq, d), (n, T, nkv, d), (n, T, nkv, d)))
    q[:, 4:, 0] = 0.0                       # heads 0 .. 3 read KV head 0, 4 .. 7 head 1
    lens = [length] * n
    want, wlse = _decode(q, k, v, lens, d)
    q, k = q.clone(), k.clone()
    at = length // 2
    q[0, 2, 5] = float("nan")
    q[1, 0:4, 0], k[1, :length, 0, 0] = 1.0, -INF          # all of KV head 0's scores
    q[2, 0:4, 0], k[2, at, 0, 0] = 1.0, INF
    q[3, 0:4, 0], k[3, at, 0, 0] = 1.0, float("nan")
    q[4, 0:4, 0], k[4, at, 0, 0] = 1.0, -INF               # one key less
    o, lse = _decode(q, k, v, lens, d)
    assert bool(o[0, 2].isnan().all()) and bool(lse[0, 2].isnan())
    assert bool(o[1, :4].isnan().all()) and bool((lse[1, :4] == -INF).all())
    assert bool(o[2, :4].isnan().all())                    # inf - inf
    assert bool(o[3, :4].isnan().all()) and bool(lse[3, :4].isnan().all())
    if length == 1:
        assert bool(o[4, :4].isnan().all()) and bool((lse[4, :4] == -INF).all())
    else:
        assert bool(o[4, :4].isfinite().all()) and bool(lse[4, :4].isfinite().all())
    others = [(0, h) for h in (0, 1, 3, 4, 5, 6, 7)] + [(s, h) for s in range(1, 5) for h in range(4, 8)]
    for s, h in others:
        assert torch.equal(o[s, h], want[s, h]) and torch.equal(lse[s, h], wlse[s, h])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_behind_the_length(dtype, d):
    """Slots behind the length hold NaN and infinity."""
    rng = np.random.default_rng(42)
    n, nq, nkv, T = 4, 4, 1, 2048
    q, k, v = (dev(values(rng, s, dtype), dtype) for s in ((n, nq, d), (n, T, nkv, d), (n, T, nkv, d)))
    lens = [0, 1, 77, 1999]
    want, wlse = _decode(q, k, v, lens, d)
    for s, m in enumerate(lens):
        k[s, m:], v[s, m:] = float("nan"), INF
    o, lse = _decode(q, k, v, lens, d)
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    assert bool(o.isfinite().all()) and bool(lse[1:].isfinite().all()) and bool((o[0] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("length", [1, 90, 300, 700])
def test_packed(dtype, d, causal, length):
    rng = np.random.default_rng(43)
    nq, nkv = 4, 2
    cu = [0, length, 2 * length, 2 * length + 50]
    T = cu[-1]
    x = dev(values(rng, (T, nq + 2 * nkv, d), dtype), dtype)
    x[:, 2:4, 0] = 0.0                                     # queries of KV head 1
    want, wlse = _packed(x, cu, nq, nkv, d, dtype, causal)
    x = x.clone()
    row = length // 2
    x[row, 0, 3] = float("nan")                            # one query of sequence 0
    x[length:2 * length, 0:2, 0] = 1.0                     # sequence 1, heads 0 and 1:
    x[length:2 * length, nq, 0] = -INF                     # .. every score -inf
    o, lse = _packed(x, cu, nq, nkv, d, dtype, causal)
    assert bool(o[row, 0].isnan().all()) and bool(lse[0, row].isnan())
    assert bool(o[length:2 * length, :2].isnan().all()) and bool((lse[:2, length:2 * length] == -INF).all())
    same = torch.ones((T, nq), dtype=torch.bool, device="cuda")
    same[row, 0] = False
    same[length:2 * length, :2] = False
    for a, b in ((o, want), (lse.T, wlse.T)):
        assert bool((a == b)[same].all())
