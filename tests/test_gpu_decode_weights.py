"""The softmax weights of mgb_attention_decode keep 16 bits beside their leading
one: in bf16 the result is off by its own rounding and little else."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from oracle import serving
from tests.serving_util import Cache, dev, host, ints, values
from tests.test_gpu_attention_decode import _sums

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv", [(4, 4), (8, 2), (16, 1), (32, 1)])
@pytest.mark.parametrize("lens", [[1, 2, 40, 300], [3000, 17, 900]])
def test_weights_in_two_parts(d, nq, nkv, lens):
    """With A = sum p |v|: a weight is off by 2^-16 relative (two bf16 parts, the second at
    most 2^-8 of the first and off by 2^-8 of itself) and by the score's error, as in
    serving_util; the output by half a step of its own."""
    rng = np.random.default_rng(61)
    n = len(lens)
    c = Cache(rng, lens, 16, nkv, d, "bf16")
    q = values(rng, (n, nq, d), "bf16")
    tq = dev(q.reshape(n, -1), "bf16")
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, ints(lens), ws)
    o = torch.empty_like(tq)
    mgb.mgb_attention_decode(plan, c.desc, tq, nq * d, o, nq * d)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    got = host(o).reshape(n, nq, d)
    ref, _ = serving.decode_attention(q, c.k, c.v, c.table, lens)
    a, qk = _sums(q, c, lens)
    score = d * 2.0 ** -23 * qk + 2.0 ** -22 * (1 + qk)
    e = (2 * score + 2.0 ** -21 + np.array(lens)[:, None] * 2.0 ** -23 + 2.0 ** -16)[..., None]
    tol = e * a + 2.0 ** -8 * (np.abs(ref) + e * a)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.abs(got - ref)[bad].max(), tol[bad].min())
