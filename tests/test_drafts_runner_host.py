"""Refusals of the runner for drafted tokens (no GPU needed: before any launch)."""
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb, runner
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer

SHAPE = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)


def ints(*a):
    return torch.tensor(a, dtype=torch.int32)


TABLE = torch.zeros((2, 4), dtype=torch.int32)


@pytest.mark.parametrize("kw", [
    dict(cu_seqlens=None, tokens=None), dict(parents=ints(-1, -1)), dict(parents=torch.tensor([-1, -1, 0])),
    dict(parents=ints(-1, 0, 1, 2, 3, 4)[::2]), dict(drafted=False, parents=ints(-1, -1, 0)), dict(tokens=None),
])
def test_batch_refuses(kw):
    a = dict(cu_seqlens=ints(0, 1, 3), tokens=3, drafted=True, parents=ints(-1, -1, 0))
    a.update(kw)
    with pytest.raises(ValueError):
        ServingBatch(SHAPE, TABLE, ints(5, 6), **a)


def test_batch_refuses_parents_elsewhere(monkeypatch):
    monkeypatch.setattr(runner, "DEVICE", "cpu")
    with pytest.raises(ValueError, match="one GPU device"):
        ServingBatch(SHAPE, TABLE, ints(5, 6), ints(0, 1, 3), 3, drafted=True,
                     parents=torch.empty(3, dtype=torch.int32, device="meta"))


class FakeBatch:
    def __init__(self, **kw):
        self.drafted, self.heads, self.seq_lens = True, (4, 2, 64), ints(5, 6)
        self.block_table, self.ws, self.plan, self.cu_seqlens, self.tokens = TABLE, None, None, ints(0, 1, 3), 3
        self.causal = True
        self.__dict__.update(kw)


def _layer():
    pool = torch.zeros((8, 16, 2, 64), dtype=torch.bfloat16)
    return ServingLayer(SHAPE, layer_inputs(SHAPE, seed=1), pool, pool.clone())


@pytest.mark.parametrize("kw", [dict(drafted=False), dict(heads=(8, 2, 64))])
def test_accept_refuses_batches(kw):
    with pytest.raises(ValueError):
        _layer().accept(FakeBatch(**kw), ints(0, 0))


@pytest.mark.parametrize("a", [
    (ints(0, 0, 0),), (torch.tensor([0, 0]),), (ints(0, 0, 0, 0)[::2],), (ints(0, 0), ints(0)),
    (torch.empty(2, dtype=torch.int32, device="meta"),), (ints(0, 0), torch.empty(2, dtype=torch.int32, device="meta")),
])
def test_accept_refuses_vectors(a):
    with pytest.raises(ValueError):
        _layer().accept(FakeBatch(), *a)


def test_step_refuses_other_heads():
    with pytest.raises(ValueError, match="other heads"):
        _layer().step(torch.zeros((3, 128), dtype=torch.bfloat16), FakeBatch(heads=(2, 2, 64)))


@pytest.mark.parametrize("a", [
    (ints(0, 1), ints(2)), (torch.tensor([0]), ints(1)), (ints(0), torch.tensor([1])), (ints(0), ints(1), ints(1, 2)),
    (ints(0, 1, 2, 3)[::2], ints(1, 2)), (ints(0).view(1, 1), ints(1).view(1, 1)),
    (ints(0), torch.empty(1, dtype=torch.int32, device="meta")),
])
def test_copies_refuse_vectors(a, monkeypatch):
    monkeypatch.setattr(runner, "DEVICE", "cpu")
    with pytest.raises(ValueError):
        _layer().copy_pages(*a)


def test_copies_refuse_host_pools():
    with pytest.raises(ValueError, match="GPU"):
        _layer().copy_pages(ints(0), ints(1))


def test_page_copies_of_different_numbers():
    with pytest.raises(ValueError):
        mgb.mgb_kv_copy_pages(None, ints(0, 1), ints(1))
