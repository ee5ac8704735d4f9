"""The serving operators together, as a program runs them: a batch of prompts
of different lengths through two layers into the paged caches, then steps of one
token per sequence with a sequence that ends on the way, every row against the
float64 layer on the whole sequence. Pages are handed out as lengths grow."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs, round_to_bf16
from megatron_transformer_layer_fwd_gb300.runner import (ServingBatch, ServingLayer, rope_table, to_device,
                                                         torch_dtype)
from oracle import serving
from tests.serving_util import host, ints
from tests.util import TOL, rel_l2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,rot,interleaved", [
    (LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True), 64, False),
    (LayerShape(1, 1, 256, 4, 1, 128, 512, norm_pos="post", causal=True), 32, True),
    (LayerShape(1, 1, 128, 4, 4, 64, 256, causal=True), 0, False),
    (LayerShape(1, 1, 128, 4, 2, 64, 256, dtype="f32", causal=True), 64, False),
])
def test_prompts_then_steps(mgb_lib, shape, rot, interleaved):
    rng = np.random.default_rng(6)
    layers, page, H = 2, 16, shape.hidden
    prompts, steps, ends = [5, 130, 33, 1], 4, {2: 2}   # sequence 2 ends before step 2
    n, most = len(prompts), max(prompts) + steps
    arrays = [layer_inputs(shape, seed=i, random_affine=True) for i in range(layers)]
    rope = rope_table(most, rot) if rot else None
    width = (most + page - 1) // page
    n_pages = n * width
    pools = lambda: torch.full((n_pages, page, shape.n_kv_heads, shape.head_dim), float("nan"),
                               dtype=torch_dtype(shape.dtype), device="cuda")
    net = [ServingLayer(shape, a, pools(), pools(), rope, interleaved) for a in arrays]
    free = list(rng.permutation(n_pages))
    table = np.full((n, width), -1)

    def grow(lens):
        for s, x in enumerate(lens):
            for i in range((x + page - 1) // page):
                if table[s, i] < 0:
                    table[s, i] = free.pop()
        return ints(table)

    rows = [rng.standard_normal((p + steps, H)) for p in prompts]
    if shape.dtype == "bf16":
        rows = [round_to_bf16(r) for r in rows]
    rope64 = host(rope) if rot else None
    want = []
    for r in rows:
        for a in arrays:
            r = serving.layer_fwd(shape, a, r, rope64, interleaved)
        want.append(r)

    def run(x, batch):
        y = to_device(x, torch_dtype(shape.dtype))
        for layer in net:
            y = layer.step(y, batch)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        return host(y)

    tol = layers * TOL[shape.dtype][0]
    cu, T = np.cumsum([0] + prompts), sum(prompts) + 3      # three rows of no sequence
    x = np.zeros((T, H))
    for s, p in enumerate(prompts):
        x[cu[s]:cu[s + 1]] = rows[s][:p]
    y = run(x, ServingBatch(shape, grow(prompts), ints(prompts), ints(cu), T))
    for s, p in enumerate(prompts):
        assert rel_l2(y[cu[s]:cu[s + 1]], want[s][:p]) < tol
    lens = list(prompts)
    for step in range(steps):
        lens = [0 if ends.get(s, steps) <= step else p + step + 1 for s, p in enumerate(prompts)]
        x = np.stack([rows[s][p + step] for s, p in enumerate(prompts)])
        y = run(x, ServingBatch(shape, grow(lens), ints(lens)))
        assert np.isfinite(y).all()
        for s, p in enumerate(prompts):
            if lens[s]:
                assert rel_l2(y[s], want[s][p + step]) < tol, (step, s)


def test_a_step_is_captured_once_and_replayed(mgb_lib):
    """The decode step with its prepare in one graph: replays follow the lengths
    and the rows on the device, bit for bit what eager steps give."""
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, act="swiglu", causal=True)
    arr = layer_inputs(shape, seed=3, random_affine=True)
    rope = rope_table(64, 64)
    n, page = 3, 8
    table = ints(np.arange(n * 8).reshape(n, 8))
    outs = []
    for captured in (False, True):
        pool = torch.zeros((2, n * 8, page, 2, 64), dtype=torch.bfloat16, device="cuda")
        layer = ServingLayer(shape, arr, pool[0], pool[1], rope)
        lens = ints([1, 1, 0])
        x = torch.zeros((n, 128), dtype=torch.bfloat16, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(4)
        step = lambda: layer.step(x, ServingBatch(shape, table, lens))
        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            pool.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = step()
        got = []
        for t in range(1, 50):
            x.copy_(torch.randn((n, 128), generator=gen, device="cuda"))
            lens.copy_(ints([t, max(t - 3, 0), 0 if t < 9 else t - 8]))
            if captured:
                graph.replay()
            else:
                y = step()
            got.append(y.clone())
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append(torch.stack(got))
    assert torch.equal(outs[0], outs[1]) and bool(torch.isfinite(outs[0].float()).all())
