"""Which tensors a batch and a layer keep, and which they say are in use on a stream that is
not the current one (no GPU needed: the library's calls and torch's streams are stood in for)."""
import contextlib

import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb, runner
from megatron_transformer_layer_fwd_gb300.inputs import LayerShape, layer_inputs
from megatron_transformer_layer_fwd_gb300.runner import ServingBatch, ServingLayer

SHAPE = LayerShape(1, 1, 128, 4, 2, 64, 256, causal=True)
OTHER = object()     # a stream


@pytest.fixture
def used(monkeypatch):
    """The tensors that were recorded as used on OTHER, by address."""
    seen = set()

    def record(t, stream):
        assert stream is OTHER
        seen.add(t.data_ptr())
    for name in ("mgb_attention_decode_prepare", "mgb_attention_packed_prepare", "mgb_attention_tree_prepare",
                 "mgb_gemm_ex", "mgb_layernorm_fwd", "mgb_kv_append", "mgb_kv_append_tree", "mgb_attention_decode",
                 "mgb_attention_packed_fwd", "mgb_attention_tree", "mgb_kv_accept", "mgb_kv_copy_pages"):
        monkeypatch.setattr(mgb, name, lambda *a, **k: object())
    for name in ("decode", "packed", "tree"):
        monkeypatch.setattr(mgb, f"mgb_attention_{name}_ws_bytes", lambda *a: 256)
    monkeypatch.setattr(runner, "DEVICE", "cpu")
    monkeypatch.setattr(runner, "_on", lambda stream, device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: OTHER)
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    return seen


def _ints(*a):
    return torch.tensor(a, dtype=torch.int32)


def _batch(kind, stream=None):
    """A batch of two sequences and the tensors that its plan is made from."""
    lens, cu, parents = _ints(5, 6), _ints(0, 2, 3), _ints(-1, 0, -1)
    table = torch.zeros((2, 4), dtype=torch.int32)
    kw = {"decode": {}, "packed": dict(cu_seqlens=cu, tokens=3),
          "drafted": dict(cu_seqlens=cu, tokens=3, drafted=True, parents=parents),
          "chains": dict(cu_seqlens=cu, tokens=3, drafted=True)}[kind]
    made_from = [lens] + ([] if kind == "decode" else [cu]) + ([parents] if kind == "drafted" else [])
    return ServingBatch(SHAPE, table, lens, stream=stream, **kw), made_from


KINDS = ["decode", "packed", "drafted", "chains"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_plan_made_on_a_given_stream_holds_what_it_is_made_from(used, kind):
    _, made_from = _batch(kind, OTHER)
    assert {t.data_ptr() for t in made_from} <= used


@pytest.mark.parametrize("kind", KINDS)
def test_a_batch_keeps_what_a_replayed_prepare_reads(used, kind):
    b, made_from = _batch(kind)
    held = [b.seq_lens, b.cu_seqlens, b.parents]
    assert all(any(t is h for h in held) for t in made_from)


def _layer():
    pool = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16)
    return ServingLayer(SHAPE, layer_inputs(SHAPE), pool, torch.zeros_like(pool))


@pytest.mark.parametrize("kind", KINDS)
def test_a_step_on_a_given_stream_holds_the_batch(used, kind):
    b, made_from = _batch(kind)
    x = torch.zeros((b.tokens, 128), dtype=torch.bfloat16)
    _layer().step(x, b, stream=OTHER)
    read = [x, b.ws, b.block_table] + ([b.seq_lens, b.cu_seqlens] if kind == "packed" else [b.seq_lens])
    assert {t.data_ptr() for t in read} <= used


@pytest.mark.parametrize("kind", ["drafted", "chains"])
def test_an_accept_on_a_given_stream_holds_the_batch(used, kind):
    b, _ = _batch(kind)
    accepted, new_lens = _ints(0, -1), _ints(0, 0)
    _layer().accept(b, accepted, new_lens, stream=OTHER)
    assert {t.data_ptr() for t in (accepted, new_lens, b.ws, b.block_table)} <= used


def test_page_copies_on_a_given_stream_hold_their_lists(used):
    lists = _ints(0, 1), _ints(2, 3), _ints(8, 4)
    _layer().copy_pages(*lists, stream=OTHER)
    assert {t.data_ptr() for t in lists} <= used


@pytest.mark.parametrize("kind", KINDS)
def test_a_workspace_of_another_stream_is_held_by_a_step_on_the_current_one(used, kind):
    b, _ = _batch(kind, OTHER)
    used.clear()
    layer = _layer()
    layer.step(torch.zeros((b.tokens, 128), dtype=torch.bfloat16), b)
    assert used == {b.ws.data_ptr()}
    if kind in ("drafted", "chains"):
        used.clear()
        layer.accept(b, _ints(0, -1))
        assert used == {b.ws.data_ptr()}


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_is_recorded_on_one_stream(used, kind):
    b, _ = _batch(kind)
    _layer().step(torch.zeros((b.tokens, 128), dtype=torch.bfloat16), b)
    assert not used
