"""Refusals of the serving runner and of outputs laid on their inputs (no GPU
needed: everything is turned down before any launch)."""
import ctypes

import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer
from tests.test_serving_host import P, _cache, lib  # noqa: F401 (fixture)

SHAPE = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)


def test_decode_output_on_its_queries(lib):  # noqa: F811
    plan = mgb.AttentionDecodePlan(n_seqs=3, n_q_heads=4, n_kv_heads=2, head_dim=64, ws=P, ws_bytes=1 << 30)
    call = lambda o: lib.mgb_attention_decode(ctypes.byref(plan), ctypes.byref(_cache()), P, 256, o, 256, None,
                                              None)
    assert call(P) == mgb.MGB_ERR_INVALID_ARG


@pytest.mark.parametrize("on", ["q", "k", "v"])
def test_packed_output_on_its_inputs(lib, on):  # noqa: F811
    plan = mgb.AttentionPackedPlan(n_seqs=3, tokens=50, causal=1, ws=P, ws_bytes=1 << 30)
    a = dict(q=2 * P, k=3 * P, v=4 * P)
    assert lib.mgb_attention_packed_fwd(ctypes.byref(plan), 4, 2, 64, mgb.MGB_BF16, a["q"], a["k"], a["v"], 512,
                                        512, a[on], 512, None, None) == mgb.MGB_ERR_INVALID_ARG


def _ints(*a):
    return torch.tensor(a, dtype=torch.int32)


@pytest.mark.parametrize("kw", [
    dict(lens=torch.tensor([1, 2])), dict(lens=_ints(1, 2, 3, 4)[::2]), dict(lens=_ints(1, 2).view(1, 2)),
    dict(table=torch.zeros((3, 4), dtype=torch.int32)), dict(table=_ints(1, 2)),
    dict(cu=torch.tensor([0, 1, 3]), tokens=3), dict(cu=_ints(0, 1), tokens=3), dict(cu=_ints(0, 1, 3)),
])
def test_batch_refuses(kw):
    a = dict(lens=_ints(1, 2), table=torch.zeros((2, 4), dtype=torch.int32), cu=None, tokens=None)
    a.update(kw)
    with pytest.raises(ValueError):
        ServingBatch(SHAPE, a["table"], a["lens"], a["cu"], a["tokens"])


def _pool(dtype=torch.bfloat16, nkv=2, d=64):
    return torch.zeros((4, 8, nkv, d), dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(k=_pool(torch.float32)), dict(k=_pool(nkv=4)), dict(k=_pool(d=128)),
    dict(rope=torch.zeros((9, 32, 2), dtype=torch.float64)), dict(rope=torch.zeros((9, 64))),
    dict(rope=torch.zeros((18, 32, 2))[::2]),
])
def test_layer_refuses(kw):
    a = dict(k=_pool(), rope=None)
    a.update(kw)
    with pytest.raises(ValueError):
        ServingLayer(SHAPE, layer_inputs(SHAPE), a["k"], torch.zeros_like(a["k"]), a["rope"])


@pytest.mark.parametrize("x", [
    torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((3, 64), dtype=torch.bfloat16),
    torch.zeros((3, 128)), torch.zeros((128, 3), dtype=torch.bfloat16).t(),
])
def test_step_refuses_rows_that_are_not_the_batchs(x):
    layer = ServingLayer(SHAPE, layer_inputs(SHAPE), _pool(), _pool())
    batch = ServingBatch.__new__(ServingBatch)
    batch.tokens, batch.cu_seqlens, batch.seq_lens = 3, None, _ints(1, 2, 3)
    batch.block_table = torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        layer.step(x, batch)
