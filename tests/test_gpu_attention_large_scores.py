"""Large scores in the serving attention kernels, at both head dims and with
and without a mask: the running reference moves late and often, so the sums and
the outputs so far are rescaled in every part of a kernel's pipeline."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import serving
from tests.serving_util import MGB, Cache, check_attention, dev, host, ints, values
from tests.test_gpu_attention_decode import _sums as decode_sums
from tests.test_gpu_attention_packed import _plan, _sums

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _scale(kind, n):
    """The keys' scale along a sequence."""
    t = np.arange(n) / max(n - 1, 1)
    return {"flat": np.full(n, 20.0), "growing": 0.1 * 400.0 ** t, "steps": 2.0 ** (np.arange(n) // 128 % 9),
            "falling": 40.0 * 400.0 ** -t}[kind]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["flat", "growing", "steps", "falling"])
def test_packed(dtype, d, causal, kind):
    rng = np.random.default_rng(51)
    nq, nkv, lens = 2, 1, [513, 1100, 77]
    cu = np.cumsum([0] + lens)
    T = int(cu[-1])
    x = values(rng, (T, nq + 2 * nkv, d), "f32")
    for s, n in enumerate(lens):
        x[cu[s]:cu[s + 1], nq:nq + nkv] *= _scale(kind, n)[:, None, None]
    qkv = dev(x.reshape(T, -1), dtype)
    x = host(qkv).reshape(x.shape)
    w = qkv.shape[1]
    o, lse = torch.empty((T, nq * d), dtype=qkv.dtype, device="cuda"), torch.empty((nq, T), device="cuda")
    mgb.mgb_attention_packed_fwd(_plan(cu, T, causal), nq, nkv, d, MGB[dtype], qkv, qkv[:, nq * d:],
                                 qkv[:, (nq + nkv) * d:], w, w, o, nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
    ref, rlse = serving.packed_attention(q, k, v, cu, causal)
    a, m, n = _sums(q, k, v, cu, causal)
    check_attention(host(o).reshape(T, nq, d), host(lse).T, ref, rlse.T, a, m, n, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["flat", "growing", "steps", "falling"])
@pytest.mark.parametrize("nq,nkv", [(4, 2), (16, 1)])
def test_decode(dtype, d, kind, nq, nkv):
    rng = np.random.default_rng(52)
    lens = [500, 65, 1100, 4500]
    c = Cache(rng, lens, 16, nkv, d, dtype)
    for s, n in enumerate(lens):
        p = np.arange(n)
        c.k[c.table[s][p // 16], p % 16] *= _scale(kind, n)[:, None, None]
    c.tk.copy_(dev(c.k, dtype))
    c.k = host(c.tk)
    q = values(rng, (4, nq, d), dtype)
    tq = dev(q.reshape(4, -1), dtype)
    o, lse = torch.empty_like(tq), torch.empty((4, nq), device="cuda")
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(4, nq, nkv, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(4, nq, nkv, d, ints(lens), ws)
    mgb.mgb_attention_decode(plan, c.desc, tq, nq * d, o, nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    ref, rlse = serving.decode_attention(q, c.k, c.v, c.table, lens)
    a, m = decode_sums(q, c, lens)
    check_attention(host(o).reshape(4, nq, d), host(lse), ref, rlse, a, m, np.array(lens)[:, None] * np.ones(nq),
                    d, dtype)
