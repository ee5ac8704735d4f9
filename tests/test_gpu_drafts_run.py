"""Drafted tokens as a program runs them: prompts into the caches of two layers, a step that
checks trees of guesses, one path of each kept, the next trees over what was kept, a sequence
that goes on in two ways, and plain steps behind; every row against the float64 layer on the
whole sequence that it stands for."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs, round_to_bf16
from megatron_transformer_layer_fwd_gb300.runner import (ServingBatch, ServingLayer, rope_table, to_device,
                                                         torch_dtype)
from oracle import drafts, serving
from tests.drafts_util import Batch, random_tree
from tests.serving_util import host, ints
from tests.util import TOL, rel_l2

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


class Net:
    """Two layers, their caches, and the float64 layers beside them."""

    def __init__(self, shape, rot, interleaved, n, width, page=16, extra=4):
        self.shape, self.page = shape, page
        arrays = [layer_inputs(shape, seed=i, random_affine=True) for i in range(2)]
        rope = rope_table(width * page, rot) if rot else None
        self.n_pages = n * width + extra
        pools = lambda: torch.full((self.n_pages, page, shape.n_kv_heads, shape.head_dim), float("nan"),
                                   dtype=torch_dtype(shape.dtype), device="cuda")
        self.layers = [ServingLayer(shape, a, pools(), pools(), rope, interleaved) for a in arrays]
        self.oracle = lambda r: [r := serving.layer_fwd(shape, a, r, host(rope) if rot else None, interleaved)
                                 for a in arrays][-1]
        order = np.random.default_rng(1).permutation(self.n_pages)
        self.table, self.spare = order[:n * width].reshape(n, width), list(order[n * width:])

    def rows(self, rng, n):
        x = rng.standard_normal((n, self.shape.hidden))
        return round_to_bf16(x) if self.shape.dtype == "bf16" else x

    def run(self, x, batch, stream=None):
        y = to_device(x, torch_dtype(self.shape.dtype))
        for layer in self.layers:
            y = layer.step(y, batch, stream)
        return y


@pytest.mark.parametrize("shape,rot,interleaved", [
    (LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True), 64, False),
    (LayerShape(1, 1, 256, 8, 1, 128, 512, norm_pos="post", causal=True), 32, True),
    (LayerShape(1, 1, 128, 4, 4, 64, 256, causal=True), 0, False),
    (LayerShape(1, 1, 128, 4, 2, 64, 256, dtype="f32", causal=True), 64, False),
])
@pytest.mark.parametrize("sizes", [[[3, 12, 1, 0], [7, 1, 5, 4]], [[30, 12, 40, 60], [64, 33, 5, 20]]])
def test_trees_are_checked_and_kept(shape, rot, interleaved, sizes):
    rng = np.random.default_rng(7)
    prompts = [5, 130, 33, 1]
    n = len(prompts)
    net = Net(shape, rot, interleaved, n, 20)
    table = ints(net.table)
    tol = 2 * TOL[shape.dtype][0]
    seqs = [net.rows(rng, p) for p in prompts]          # what each sequence's cache holds
    cu = np.cumsum([0] + prompts)
    lens = ints(prompts)
    net.run(np.concatenate(seqs), ServingBatch(shape, table, lens, ints(cu), int(cu[-1])))
    for step in range(2):
        b = Batch([(len(q), random_tree(rng, m, roots=min(m, 1 + step))) for q, m in zip(seqs, sizes[step])], tail=2)
        new = [net.rows(rng, m) for m in sizes[step]]
        lens.copy_(ints(b.lens))
        batch = ServingBatch(shape, table, lens, ints(b.cu), b.tokens, drafted=True, parents=ints(b.parents))
        y = host(net.run(np.concatenate(new + [net.rows(rng, 2)]), batch))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        accepted = []
        for s in range(n):
            for t in range(sizes[step][s]):
                keep = drafts.path(b.trees[s], t)
                if t % 4 == 0 or t + 1 == sizes[step][s]:     # (each costs a layer of the whole sequence)
                    want = net.oracle(np.concatenate([seqs[s], new[s][keep]]))[-1]
                    assert rel_l2(y[b.cu[s] + t], want) < tol, (step, s, t)
            leaf = int(rng.integers(-1, sizes[step][s])) if sizes[step][s] else -1
            accepted.append(leaf)
            seqs[s] = np.concatenate([seqs[s], new[s][drafts.path(b.trees[s], leaf)]])
        for layer in net.layers:   # the second call's plan still has the drafted lengths
            layer.accept(batch, ints(accepted), lens)
        assert lens.tolist() == [len(q) for q in seqs]
    # sequence 2 becomes a second way of sequence 1: full pages shared, the last one copied
    page = net.page
    full, part = divmod(len(seqs[1]), page)
    net.table[2, :full] = net.table[1, :full]
    net.table[2, full] = net.spare.pop()
    seqs[2] = seqs[1].copy()
    table = ints(net.table)
    for layer in net.layers:
        layer.copy_pages(ints([net.table[1, full]]), ints([net.table[2, full]]), ints([part]))
    for step in range(2):
        x = net.rows(rng, n)
        seqs = [np.concatenate([q, x[s:s + 1]]) for s, q in enumerate(seqs)]
        y = host(net.run(x, ServingBatch(shape, table, ints([len(q) for q in seqs]))))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        for s in range(n):
            assert rel_l2(y[s], net.oracle(seqs[s])[-1]) < tol, (step, s)


def test_a_prompt_in_pieces():
    """Chains over what is cached: the same rows as the prompt in one."""
    shape = LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True)
    rng = np.random.default_rng(8)
    net = Net(shape, 64, False, 2, 50)
    table, total = ints(net.table), [600, 333]
    x = [net.rows(rng, t) for t in total]
    got, at = [[], []], 0
    while any(at < t for t in total):
        take = [max(0, min(256, t - at)) for t in total]
        cu = np.cumsum([0] + take)
        lens = [min(at + 256, t) for t in total]
        rows = np.concatenate([v[at:at + m] for v, m in zip(x, take)])
        y = host(net.run(rows, ServingBatch(shape, table, ints(lens), ints(cu), int(cu[-1]), drafted=True)))
        for s in range(2):
            got[s].append(y[cu[s]:cu[s + 1]])
        at += 256
    assert mgb.mgb_device_status() == mgb.MGB_OK
    for s in range(2):
        assert rel_l2(np.concatenate(got[s]), net.oracle(x[s])) < 2 * TOL["bf16"][0]


def test_a_drafted_step_is_captured_and_replayed():
    """Prepare, step and accept in one graph: replays follow rows, trees, lengths and choices on
    the device, bit for bit what eager steps give; the lengths go on in place."""
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, act="swiglu", causal=True)
    n, T = 3, 24
    outs = []
    for captured in (False, True):
        rng = np.random.default_rng(9)
        net = Net(shape, 64, False, n, 20)
        for layer in net.layers:
            layer.k_pool.zero_(), layer.v_pool.zero_()
        table, lens, cu, parents, accepted = (ints(net.table), ints([0] * n), ints([0] * (n + 1)), ints([-1] * T),
                                              ints([-1] * n))
        full = ints([0] * n)     # the lengths with the drafted tokens
        x = torch.zeros((T, 128), dtype=torch.bfloat16, device="cuda")

        def step():
            full.copy_(lens + (cu[1:] - cu[:-1]))
            batch = ServingBatch(shape, table, full, cu, T, drafted=True, parents=parents)
            y = x
            for layer in net.layers:
                y = layer.step(y, batch)
            for layer in net.layers:
                layer.accept(batch, accepted, lens)
            return y
        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            for layer in net.layers:
                layer.k_pool.zero_(), layer.v_pool.zero_()
            lens.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = step()
        got = []
        for _ in range(12):
            m = [int(k) for k in rng.integers(1, 9, n)]
            trees = [random_tree(rng, k) for k in m]
            cu.copy_(ints(np.cumsum([0] + m)))
            parents.copy_(ints(sum(trees, []) + [-1] * (T - sum(m))))
            accepted.copy_(ints([int(rng.integers(0, k)) for k in m]))
            x.copy_(torch.from_numpy(rng.standard_normal((T, 128))))
            if captured:
                graph.replay()
            else:
                y = step()
            got.append((y[:sum(m)].clone(), lens.clone()))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append(got)
    for (a, la), (b, lb) in zip(*outs):
        assert torch.equal(a, b) and torch.equal(la, lb) and bool(torch.isfinite(a.float()).all())
    assert outs[0][-1][1].max() > 20


def test_on_a_stream_of_its_own():
    """A step, its accept and a page copy on a stream that is not the current one."""
    shape = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)
    outs = []
    for own in (False, True):
        rng = np.random.default_rng(10)
        net = Net(shape, 64, False, 1, 6)
        b = Batch([(0, random_tree(rng, 9))])
        s = torch.cuda.Stream() if own else None
        x = net.rows(rng, 9)
        args = [ints(v) for v in (net.table, b.lens, b.cu, b.parents, [8], [0])]
        torch.cuda.synchronize()
        batch = ServingBatch(shape, args[0], args[1], args[2], 9, stream=s, drafted=True, parents=args[3])
        y = to_device(x, torch.bfloat16)
        torch.cuda.synchronize()
        for layer in net.layers:
            y = layer.step(y, batch, s)
            layer.accept(batch, args[4], args[5], s)
            layer.copy_pages(args[0][0, :1].clone() if s is None else args[0][0, :1], ints([int(net.spare[0])]), None, s)
        if own:
            s.synchronize()
        assert mgb.mgb_device_status(s) == mgb.MGB_OK
        outs.append((y.clone(), args[5].tolist(),
                     [torch.equal(la.k_pool[net.spare[0]].nan_to_num(), la.k_pool[net.table[0, 0]].nan_to_num())
                      for la in net.layers]))
    assert torch.equal(outs[0][0], outs[1][0]) and outs[0][1] == outs[1][1] and all(outs[1][2]) and all(outs[0][2])
