"""Rows whose offsets pass 2^31 elements: the last rows of long packed
activations, and rows far apart, give the bits of the same rows in small tensors."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from tests.serving_util import MGB, TORCH, ints

pytestmark = pytest.mark.gpu

NQ, NKV, D = 4, 2, 128
W = (NQ + 2 * NKV) * D
ROWS = (1 << 31) // W + 70001          # of W numbers: past 2^31 elements


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _room(numbers, dtype):
    if torch.cuda.mem_get_info()[0] < 3 * numbers * TORCH[dtype].itemsize:
        pytest.skip("not enough free memory")


def _attend(x, cu, dtype):
    T = x.shape[0]
    ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(len(cu) - 1, T), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_packed_prepare(len(cu) - 1, T, True, ints(cu), ws)
    o = torch.zeros((T, NQ * D), dtype=x.dtype, device="cuda")
    lse = torch.zeros((NQ, T), device="cuda")
    mgb.mgb_attention_packed_fwd(plan, NQ, NKV, D, MGB[dtype], x, x[:, NQ * D:], x[:, (NQ + NKV) * D:], W, W, o,
                                 NQ * D, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_rows_past_two_to_the_31(dtype):
    _room(ROWS * W, dtype)
    near = torch.randn((300, W), device="cuda").to(TORCH[dtype])
    x = torch.zeros((ROWS, W), dtype=TORCH[dtype], device="cuda")
    x[-301:-1] = near
    want, wlse = _attend(near, [0, 170, 300], dtype)
    o, lse = _attend(x, [ROWS - 301, ROWS - 131, ROWS - 1], dtype)
    assert torch.equal(o[-301:-1], want) and torch.equal(lse[:, -301:-1], wlse)
    assert not bool((o[:-301] != 0).any()) and not bool((o[-1] != 0).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_appended_rows_past_two_to_the_31(dtype):
    """The rows before the last sequence are a padding sequence's."""
    _room(ROWS * W, dtype)
    near = torch.randn((50, W), device="cuda").to(TORCH[dtype])
    x = torch.zeros((ROWS, W), dtype=TORCH[dtype], device="cuda")
    x[-51:-1] = near
    rope, table = rope_table(64, D), ints([[0, 1, 2, 3], [4, 5, 6, 7]])
    outs = []
    for y, cu in ((near, [0, 0, 50]), (x, [0, ROWS - 51, ROWS - 1])):
        pool = torch.zeros((2, 8, 16, NKV, D), dtype=TORCH[dtype], device="cuda")
        T = y.shape[0]
        mgb.mgb_kv_append(mgb.kv_append_desc(T, 2, NQ, D, True, 64), mgb.kv_cache(pool[0], pool[1], table), ints(cu),
                          ints([0, 60]), rope, y, y[:, NQ * D:], y[:, (NQ + NKV) * D:], W, W, y, W, y[:, NQ * D:], W)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append(pool)
    assert torch.equal(*outs) and bool((outs[0] != 0).any())
    assert torch.equal(x[-51:-1], near) and not bool((x[:-51] != 0).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_rows_far_apart(dtype):
    """Query and output rows 2^30 elements apart, four sequences: past 2^31."""
    far, n = 1 << 30, 4
    _room(n * far, dtype)
    pool = torch.randn((2, 16, 16, NKV, D), device="cuda").to(TORCH[dtype])
    cache = mgb.kv_cache(pool[0], pool[1], ints(np.arange(16).reshape(4, 4)))
    lens = ints([64, 1, 0, 37])
    q = torch.randn((n, NQ * D), device="cuda").to(TORCH[dtype])
    big = torch.empty(((n - 1) * far + 2 * NQ * D,), dtype=TORCH[dtype], device="cuda")
    view = lambda at: big[at:].as_strided((n, NQ * D), (far, 1), at)
    view(0).copy_(q)
    view(NQ * D).fill_(3.0)
    outs = []
    for a, o, ld in ((q, torch.zeros_like(q), NQ * D), (view(0), view(NQ * D), far)):
        ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, NQ, NKV, D), dtype=torch.uint8, device="cuda")
        plan = mgb.mgb_attention_decode_prepare(n, NQ, NKV, D, lens, ws)
        mgb.mgb_attention_decode(plan, cache, a, ld, o, ld)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append(o.clone())
    assert torch.equal(*outs) and torch.equal(view(0), q)


def test_more_sequences_than_a_grid_is_wide():
    """70000 sequences of a token or none, each form."""
    n = 70000
    gen = torch.Generator(device="cuda").manual_seed(7)
    ones = (torch.rand(n, generator=gen, device="cuda") < 0.7).to(torch.int32)
    cu = torch.cat([ints([0]), ones.cumsum(0).to(torch.int32)])
    T = int(cu[-1])
    x = torch.randn((T, 3 * 64), generator=gen, device="cuda").bfloat16()
    o = torch.zeros((T, 64), device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(mgb.mgb_attention_packed_ws_bytes(n, T), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_packed_prepare(n, T, True, cu, ws)
    mgb.mgb_attention_packed_fwd(plan, 1, 1, 64, mgb.MGB_BF16, x, x[:, 64:], x[:, 128:], 192, 192, o, 64)
    assert torch.equal(o, x[:, 128:])               # one key each
    pool = torch.zeros((2, n, 1, 1, 64), device="cuda", dtype=torch.bfloat16)
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).view(n, 1)
    cache = mgb.kv_cache(pool[0], pool[1], table)
    mgb.mgb_kv_append(mgb.kv_append_desc(T, n, 1, 0, False, 0), cache, cu, ones, None, None, x[:, 64:], x[:, 128:], 192,
                      192, None, 0, None, 0)
    alive = ones.bool()
    assert torch.equal(pool[1].flip(0)[alive][:, 0, 0], x[:, 128:]) and not bool((pool.flip(1)[:, ~alive] != 0).any())
    q = torch.randn((n, 64), generator=gen, device="cuda").bfloat16()
    od = torch.full_like(q, 3.0)
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, 1, 1, 64), dtype=torch.uint8, device="cuda")
    mgb.mgb_attention_decode(mgb.mgb_attention_decode_prepare(n, 1, 1, 64, ones, ws), cache, q, 64, od, 64)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert torch.equal(od[alive], x[:, 128:]) and not bool((od[~alive] != 0).any())
