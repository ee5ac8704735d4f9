"""Layers and batches at the ends of their ranges through the serving runner:
no biases, no affine norms, one row, no rows, every sequence padding."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs, round_to_bf16
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer, rope_table, to_device, torch_dtype
from oracle import serving
from tests.serving_util import host, ints
from tests.util import TOL, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _layer(shape, n, rope=None):
    pools = torch.zeros((2, n * 4, 16, shape.n_kv_heads, shape.head_dim), dtype=torch_dtype(shape.dtype),
                        device="cuda")
    a = layer_inputs(shape, seed=1, random_affine=shape.ln_affine)
    table = ints(np.arange(n * 4).reshape(n, 4))
    return ServingLayer(shape, a, pools[0], pools[1], rope), a, table, pools


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(has_bias=False), dict(ln_affine=False), dict(has_bias=False, ln_affine=False),
                                dict(norm_pos="post", has_bias=False, act="swiglu"),
                                dict(causal=False)])
def test_a_prompt_and_a_step(dtype, kw):
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, dtype=dtype, **{"causal": True, **kw})
    rope = rope_table(64, 64)
    layer, a, table, _ = _layer(shape, 1, rope)
    rows = np.random.default_rng(3).standard_normal((20, 128))
    if dtype == "bf16":
        rows = round_to_bf16(rows)
    x = to_device(rows, torch_dtype(dtype))
    y = layer.step(x[:19], ServingBatch(shape, table, ints([19]), ints([0, 19]), 19))
    want = serving.layer_fwd(shape, a, rows[:19], host(rope))
    assert rel_l2(host(y), want) < TOL[dtype][0]
    if shape.causal:      # (without the mask a later row would change the earlier ones)
        z = layer.step(x[19:], ServingBatch(shape, table, ints([20])))
        want = serving.layer_fwd(shape, a, rows, host(rope))[19:]
        assert rel_l2(host(z), want) < TOL[dtype][0]
    assert mgb.mgb_device_status() == mgb.MGB_OK


def test_no_rows():
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)
    layer, _, table, pools = _layer(shape, 3)
    x = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    y = layer.step(x, ServingBatch(shape, table, ints([0, 0, 0]), ints([0, 0, 0, 0]), 0))
    assert y.shape == (0, 128)
    y = layer.step(x, ServingBatch(shape, table[:0], ints(np.zeros(0, dtype=np.int32))))
    assert y.shape == (0, 128) and y.dtype == torch.bfloat16
    assert mgb.mgb_device_status() == mgb.MGB_OK and not bool((pools != 0).any())


def test_padding_only():
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)
    layer, _, table, pools = _layer(shape, 3)
    x = torch.randn((3, 128), device="cuda").bfloat16()
    y = layer.step(x, ServingBatch(shape, table, ints([0, 0, 0])))
    assert bool(y.isfinite().all()) and not bool((pools != 0).any())
    assert mgb.mgb_device_status() == mgb.MGB_OK
