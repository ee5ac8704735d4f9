"""A sequence's rows of mgb_attention_packed_fwd depend on that sequence alone,
bit for bit: not on what lies in the other rows of the batch."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from tests.serving_util import MGB, TORCH, dev, ints, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _run(x, cu, nq, nkv, d, dtype, causal):
    T, w = x.shape
    ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(len(cu) - 1, T), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_packed_prepare(len(cu) - 1, T, causal, ints(cu), ws)
    o, lse = torch.zeros((T, nq * d), dtype=x.dtype, device="cuda"), torch.zeros((nq, T), device="cuda")
    mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, MGB[dtype], x, x[:, nq * d:], x[:, (nq + nkv) * d:], w, w, o,
                                 nq * d, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[17, 111], [100, 90, 140], [130, 1, 400], [300, 33, 257]])
def test_bits_do_not_depend_on_the_neighbours(dtype, d, causal, lens):
    nq, nkv, tail = 4, 2, 150
    gen = torch.Generator(device="cuda").manual_seed(5)
    cu = [int(c) for c in np.cumsum([0] + lens)]
    T = cu[-1] + tail
    x = (torch.randn((T, (nq + 2 * nkv) * d), generator=gen, device="cuda") * 1.5).to(TORCH[dtype])
    want = _run(x, cu, nq, nkv, d, dtype, causal)
    kinds = [lambda r: torch.zeros_like(r), lambda r: r * 64, lambda r: torch.full_like(r, float("nan")),
             lambda r: torch.full_like(r, float("inf")), lambda r: torch.full_like(r, -3e38)]
    for s in range(len(lens)):
        mine = slice(cu[s], cu[s + 1])
        for other in kinds:
            y = other(x)
            y[mine] = x[mine]
            o, lse = _run(y, cu, nq, nkv, d, dtype, causal)
            assert torch.equal(o[mine], want[0][mine]) and torch.equal(lse[:, mine], want[1][:, mine])
        # .. and alone
        alone = x[mine].contiguous()
        o, lse = _run(alone, [0, lens[s]], nq, nkv, d, dtype, causal)
        assert torch.equal(o, want[0][mine]) and torch.equal(lse, want[1][:, mine])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_packed_keys_that_are_masked(dtype, d, bad):
    """A later key's NaN or infinity does not reach the rows that do not see it,
    whether its tile is theirs or not."""
    rng = np.random.default_rng(44)
    nq, nkv, cu = 2, 1, [0, 420]
    x = dev(values(rng, (420, nq + 2 * nkv, d), dtype), dtype)
    want, wlse = _run(x.reshape(420, -1), cu, nq, nkv, d, dtype, True)
    for at in (1, 100, 129, 400):
        y = x.clone()
        y[at, nq] = bad
        o, lse = _run(y.reshape(420, -1), cu, nq, nkv, d, dtype, True)
        assert torch.equal(o[:at], want[:at]) and torch.equal(lse[:, :at], wlse[:, :at])
