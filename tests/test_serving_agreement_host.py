"""Serving calls whose parts do not belong together are turned down on the host
before any launch: a batch prepared for other heads or another mask than the
layer's, tensors on different devices (no GPU needed)."""
import dataclasses
import os

import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb, runner
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer

SHAPE = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)


@pytest.fixture
def recorded(monkeypatch):
    """The library's calls, recorded instead of made."""
    calls = []

    def fake(name):
        def f(*a, **k):
            calls.append(name)
            return object()
        return f
    for name in ("mgb_attention_decode_prepare", "mgb_attention_packed_prepare", "mgb_gemm_ex",
                 "mgb_layernorm_fwd", "mgb_kv_append", "mgb_attention_decode", "mgb_attention_packed_fwd"):
        monkeypatch.setattr(mgb, name, fake(name))
    monkeypatch.setattr(runner, "DEVICE", "cpu")
    monkeypatch.setattr(mgb, "mgb_attention_decode_ws_bytes", lambda *a: 256)
    monkeypatch.setattr(mgb, "mgb_attention_packed_ws_bytes", lambda *a: 256)
    return calls


def _ints(*a):
    return torch.tensor(a, dtype=torch.int32)


def _batch(shape, n, packed):
    table = torch.zeros((n, 4), dtype=torch.int32)
    lens = torch.ones(n, dtype=torch.int32)
    cu = torch.arange(n + 1, dtype=torch.int32) if packed else None
    return ServingBatch(shape, table, lens, cu, n if packed else None)


def _layer(shape=SHAPE):
    pool = torch.zeros((4, 8, shape.n_kv_heads, shape.head_dim), dtype=torch.bfloat16)
    return ServingLayer(shape, layer_inputs(shape), pool, torch.zeros_like(pool))


def _x(n):
    return torch.zeros((n, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("other", [dict(n_q_heads=8), dict(n_q_heads=2), dict(n_q_heads=4, n_kv_heads=4),
                                   dict(n_q_heads=8, n_kv_heads=4), dict(head_dim=128)])
@pytest.mark.parametrize("n", [1, 3])
def test_a_decode_batch_of_other_heads(recorded, other, n):
    """One sequence is the case that nothing else catches: its rows have no stride to check,
    and the plan's heads would be written over the end of the layer's one output row."""
    layer, batch = _layer(), _batch(dataclasses.replace(SHAPE, **other), n, False)
    del recorded[:]
    with pytest.raises(ValueError, match="heads"):
        layer.step(_x(n), batch)
    assert recorded == []


def test_a_packed_batch_of_another_mask(recorded):
    layer, batch = _layer(), _batch(dataclasses.replace(SHAPE, causal=False), 3, True)
    del recorded[:]
    with pytest.raises(ValueError, match="causal"):
        layer.step(_x(3), batch)
    assert recorded == []


@pytest.mark.parametrize("packed", [False, True])
def test_a_batch_serves_layers_that_differ_elsewhere(recorded, packed):
    """Width, activation and, packed, heads may differ from layer to layer."""
    for other in [dict(), dict(ffn=512, act="swiglu")] + ([dict(n_q_heads=8)] if packed else []):
        batch = _batch(dataclasses.replace(SHAPE, **other), 3, packed)
        del recorded[:]
        _layer().step(_x(3), batch)
        assert recorded[-1] in ("mgb_gemm_ex", "mgb_layernorm_fwd") and len(recorded) >= 7


META = torch.device("meta")   # a device that is not the others'


@pytest.mark.parametrize("which", range(3))
def test_cache_tensors_of_different_devices(which):
    pools = [torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16) for _ in range(2)]
    a = pools + [torch.zeros((3, 2), dtype=torch.int32)]
    a[which] = a[which].to(META)
    with pytest.raises(ValueError, match="device"):
        mgb.kv_cache(*a)


@pytest.mark.parametrize("which", ["table", "lens", "cu"])
def test_batch_tensors_of_different_devices(recorded, which):
    a = dict(table=torch.zeros((3, 4), dtype=torch.int32), lens=_ints(1, 1, 1), cu=_ints(0, 1, 2, 3))
    a[which] = a[which].to(META)
    with pytest.raises(ValueError, match="device"):
        ServingBatch(SHAPE, a["table"], a["lens"], a["cu"], 3)
    assert recorded == []


def test_layer_and_step_tensors_of_different_devices(recorded):
    pool = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16)
    for k, v, rope in [(pool, pool.to(META), None), (pool, pool, torch.zeros((9, 32, 2), device=META))]:
        with pytest.raises(ValueError, match="device"):
            ServingLayer(SHAPE, layer_inputs(SHAPE), k, v, rope)
    layer, batch = _layer(), _batch(SHAPE, 3, False)
    with pytest.raises(ValueError, match="device"):
        layer.step(_x(3).to(META), batch)
    batch.seq_lens = batch.seq_lens.to(META)
    with pytest.raises(ValueError, match="device"):
        layer.step(_x(3), batch)


@pytest.mark.parametrize("packed", [False, True])
def test_a_batch_on_the_host(recorded, monkeypatch, packed):
    monkeypatch.setattr(runner, "DEVICE", "cuda")
    with pytest.raises(ValueError, match="device"):
        _batch(SHAPE, 3, packed)
    assert recorded == []


def test_append_descriptor_of_whole_sequences():
    import ctypes
    from tests.test_serving_host import _cache, P
    if not os.path.exists(mgb.LIB_PATH):
        from megatron_transformer_layer_fwd_gb300 import build
        build.build()
    d = mgb.kv_append_desc(5, 3, 4, 64, False, 100)
    assert d.whole == 0 and mgb.kv_append_desc(5, 3, 4, 64, False, 100, whole=True).whole == 1
    for bad in (2, -1):
        d.whole = bad
        assert mgb.load().mgb_kv_append(ctypes.byref(d), ctypes.byref(_cache()), P, P, P, P, P, P, 256, 256, 2 * P,
                                        256, 2 * P, 128, None) == mgb.MGB_ERR_INVALID_ARG
