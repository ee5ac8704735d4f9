"""The serving runner on a stream that is not torch's current one: every fill
and every temporary of a step belongs to the step's stream, whatever other work
is under way on the current one."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer, rope_table
from tests.serving_util import ints

pytestmark = pytest.mark.gpu

SHAPE = LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True)
DELAY = 20_000_000  # cycles: 10 to 15 ms of a stream


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _setup(packed):
    n, page = 3, 16
    pools = torch.zeros((2, n * 4, page, 2, 64), dtype=torch.bfloat16, device="cuda")
    layer = ServingLayer(SHAPE, layer_inputs(SHAPE, seed=2, random_affine=True), pools[0], pools[1],
                         rope_table(64, 64))
    table = ints(np.arange(n * 4).reshape(n, 4))
    lens = [30, 1, 9] if packed else [1, 1, 1]
    cu = ints(np.cumsum([0] + lens)) if packed else None
    rows = sum(lens) + (5 if packed else 0)   # five rows of no sequence
    x = torch.randn((rows, 256), generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda").bfloat16()
    lens = ints(lens)
    return layer, pools, x, lambda **kw: ServingBatch(SHAPE, table, lens, cu, rows if packed else None, **kw)


def _poison(rows):
    """Fills what the allocator has free for the current stream with NaN (0xff): blocks
    of a step's sizes (rows of 256, 512 and 1024 numbers) and others."""
    sizes = [2 * rows * w for w in (256, 512, 1024)] * 12 + [1 << k for k in range(9, 20)] * 4
    junk = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for size in sizes]
    del junk


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("late", ["current", "step"])
def test_a_step_on_another_stream(packed, handle, late):
    """`late`: the stream that other work holds up. Behind the current one's, an
    output cleared there would be cleared too late; behind the step's, temporaries
    that went back to the current stream would be overwritten before they are read."""
    layer, pools, x, batch = _setup(packed)
    want = layer.step(x, batch())
    assert mgb.mgb_device_status() == mgb.MGB_OK
    want_pools = pools.clone()
    s = torch.cuda.Stream()
    for _ in range(3):
        pools.zero_()
        _poison(x.shape[0])
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.current_stream() if late == "current" else s):
            torch.cuda._sleep(DELAY)
        stream = s.cuda_stream if handle else s
        b = batch(stream=stream)
        got = layer.step(x, b, stream=stream)
        del b
        _poison(x.shape[0])
        s.synchronize()
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert torch.equal(got, want) and torch.equal(pools, want_pools)


def test_a_batch_prepared_on_one_stream_and_used_on_another():
    layer, pools, x, batch = _setup(False)
    want = layer.step(x, batch())
    a, s = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    b = batch(stream=a)
    s.wait_stream(a)
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    got = layer.step(x, b, stream=s)
    del b                       # its workspace must not be handed out while s still uses it
    with torch.cuda.stream(a):
        _poison(x.shape[0])
    torch.cuda.synchronize()
    assert mgb.mgb_device_status() == mgb.MGB_OK and torch.equal(got, want)


def test_a_step_captured_on_a_given_stream():
    layer, pools, x, batch = _setup(False)
    want = layer.step(x, batch())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer.step(x, batch(stream=s), stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = layer.step(x, batch(stream=s), stream=s)
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK and torch.equal(got, want)
