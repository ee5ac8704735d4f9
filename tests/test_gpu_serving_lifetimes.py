"""Index tensors that a program drops as soon as a call has returned: what is still to run on
another stream, or in a captured graph that is replayed later, reads them all the same."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer, rope_table
from tests.drafts_util import random_tree
from tests.serving_util import ints

pytestmark = pytest.mark.gpu

SHAPE = LayerShape(1, 1, 256, 4, 2, 64, 512, act="swiglu", causal=True)
DELAY = 20_000_000  # cycles: 10 to 15 ms of a stream
NEW = [5, 1, 9]     # rows per sequence, where there are several


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


class Case:
    """A layer and, made anew for every call, the index tensors of a step."""

    def __init__(self, kind):
        self.kind, page, n = kind, 16, 3
        self.pools = torch.zeros((2, n * 4, page, 2, 64), dtype=torch.bfloat16, device="cuda")
        self.layer = ServingLayer(SHAPE, layer_inputs(SHAPE, seed=2, random_affine=True), self.pools[0],
                                  self.pools[1], rope_table(64, 64))
        self.rows = n if kind == "decode" else sum(NEW)
        g = torch.Generator(device="cuda").manual_seed(3)
        self.x = torch.randn((self.rows, 256), generator=g, device="cuda").bfloat16()
        self.cached = torch.randn(self.pools.shape, generator=g, device="cuda").bfloat16()
        rng = np.random.default_rng(4)
        self.trees = [random_tree(rng, m) for m in NEW]

    def index(self):
        """Arguments of ServingBatch behind the shape."""
        table = ints(np.arange(12).reshape(3, 4))
        if self.kind == "decode":
            return dict(block_table=table, seq_lens=ints([31, 2, 10]))
        cu = ints(np.cumsum([0] + NEW))
        a = dict(block_table=table, seq_lens=ints(NEW), cu_seqlens=cu, tokens=self.rows)
        if self.kind != "packed":
            a.update(seq_lens=ints([30 + NEW[0], NEW[1], 20 + NEW[2]]), drafted=True)
        if self.kind == "drafted":
            a["parents"] = ints(sum(self.trees, []))
        return a

    def reset(self):
        self.pools.copy_(self.cached)

    def want(self):
        self.reset()
        y = self.layer.step(self.x, ServingBatch(SHAPE, **self.index()))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        return y, self.pools.clone()


def _poison():
    """Fills what the allocator has free for the current stream with -1: the smallest blocks, as
    index tensors take, and larger ones."""
    junk = [torch.full((size // 4,), -1, dtype=torch.int32, device="cuda")
            for size in [512] * 400 + [1 << k for k in range(10, 20)] * 4]
    del junk


def _busy(s):
    """Holds up stream s behind what the current stream has done so far."""
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)


KINDS = ["decode", "packed", "drafted", "chains"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("handle", [False, True])
def test_a_batch_made_on_a_busy_stream_from_temporaries(kind, handle):
    c = Case(kind)
    want, pools = c.want()
    s = torch.cuda.Stream()
    for _ in range(3):
        c.reset()
        torch.cuda.synchronize()
        keep, dropped = c.index(), c.index()   # the first stay for the step below
        _busy(s)
        b = ServingBatch(SHAPE, **dropped, stream=s.cuda_stream if handle else s)
        b.block_table, b.seq_lens, b.cu_seqlens = keep["block_table"], keep["seq_lens"], keep.get("cu_seqlens")
        b.parents = None
        del dropped
        _poison()
        got = c.layer.step(c.x, b, stream=s)
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert torch.equal(got, want) and torch.equal(c.pools, pools)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("handle", [False, True])
def test_a_step_on_a_busy_stream_and_nothing_kept(kind, handle):
    c = Case(kind)
    want, pools = c.want()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    for _ in range(3):
        c.reset()
        torch.cuda.synchronize()
        dropped = c.index()
        x = c.x.clone()
        _busy(s)
        b = ServingBatch(SHAPE, **dropped, stream=stream)
        got = c.layer.step(x, b, stream=stream)
        del dropped, b, x
        _poison()
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert torch.equal(got, want) and torch.equal(c.pools, pools)


@pytest.mark.parametrize("kind", KINDS)
def test_a_batch_of_one_stream_in_a_step_of_the_current_one(kind):
    """The workspace goes back to the stream that it was made on, where other work takes it."""
    c = Case(kind)
    want, pools = c.want()
    a, index = torch.cuda.Stream(), c.index()
    for _ in range(3):
        c.reset()
        torch.cuda.synchronize()
        b = ServingBatch(SHAPE, **index, stream=a)
        torch.cuda.current_stream().wait_stream(a)
        torch.cuda._sleep(DELAY)
        got = c.layer.step(c.x, b)
        size = b.ws.numel()
        del b
        with torch.cuda.stream(a):
            junk = [torch.full((size,), 0xC3, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        del junk
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert torch.equal(got, want) and torch.equal(c.pools, pools)


@pytest.mark.parametrize("handle", [False, True])
def test_an_accept_and_copies_on_a_busy_stream_and_nothing_kept(handle):
    """The paths of the last tokens, then page 0 to page 3 and half of page 4 to page 7."""
    c = Case("drafted")
    c.want()
    after, new, outs = c.pools.clone(), torch.zeros(3, dtype=torch.int32, device="cuda"), []
    last = [m - 1 for m in NEW]
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    for own in (False, True, True):
        c.pools.copy_(after)
        new.zero_()
        torch.cuda.synchronize()
        b = ServingBatch(SHAPE, **c.index())
        a = [ints(last), ints([0, 4]), ints([3, 7]), ints([16, 8])]
        if own:
            _busy(s)
        c.layer.accept(b, a[0], new, stream if own else None)
        del b
        c.layer.copy_pages(*a[1:], stream if own else None)
        del a
        if own:
            _poison()
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append((c.pools.clone(), new.tolist()))
    assert all(torch.equal(p, outs[0][0]) and n == outs[0][1] for p, n in outs[1:])
    assert outs[0][1][0] > 30 and not torch.equal(outs[0][0], after)


def test_a_captured_batch_is_all_that_a_replay_needs():
    c = Case("drafted")
    want, pools = c.want()
    index = c.index()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.layer.step(c.x, ServingBatch(SHAPE, **index))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        batch = ServingBatch(SHAPE, **index)
        got = c.layer.step(c.x, batch)
    del index
    for _ in range(2):
        _poison()
        c.reset()
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert torch.equal(got, want) and torch.equal(c.pools, pools)
    del batch
