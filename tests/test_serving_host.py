"""Refusals of the serving entry points, before any launch (no GPU needed):
every bad size, stride, alignment, dtype and missing pointer is turned down
with the documented status."""
import ctypes
import os

import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb

P = 4096  # a non-NULL, aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mgb.LIB_PATH):
        from megatron_transformer_layer_fwd_gb300 import build
        build.build()
    return mgb.load()


def _cache(**kw):
    a = dict(k=P, v=P, block_table=P, stride_page=16 * 2 * 64, stride_token=2 * 64, stride_head=64,
             ld_table=8, n_pages=100, page_size=16, max_pages=8, n_kv_heads=2, head_dim=64,
             dtype=mgb.MGB_BF16)
    a.update(kw)
    return mgb.KVCache(**a)


BAD_CACHE = [
    (dict(dtype=2), mgb.MGB_ERR_INVALID_ARG), (dict(n_pages=0), mgb.MGB_ERR_INVALID_ARG),
    (dict(page_size=0), mgb.MGB_ERR_INVALID_ARG), (dict(max_pages=0), mgb.MGB_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), mgb.MGB_ERR_INVALID_ARG), (dict(k=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(v=None), mgb.MGB_ERR_INVALID_ARG), (dict(block_table=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_table=7), mgb.MGB_ERR_INVALID_ARG), (dict(stride_token=56), mgb.MGB_ERR_INVALID_ARG),
    (dict(stride_head=56), mgb.MGB_ERR_INVALID_ARG), (dict(stride_page=-8), mgb.MGB_ERR_INVALID_ARG),
    (dict(stride_page=8), mgb.MGB_ERR_INVALID_ARG),
    (dict(k=P + 8), mgb.MGB_ERR_MISALIGNED), (dict(v=P + 2), mgb.MGB_ERR_MISALIGNED),
    (dict(stride_token=132), mgb.MGB_ERR_MISALIGNED), (dict(stride_page=2052), mgb.MGB_ERR_MISALIGNED),
    (dict(block_table=P + 1), mgb.MGB_ERR_MISALIGNED),
]


def _append(lib, cache=None, desc=None, **kw):
    a = dict(cu=P, lens=P, rope=P, q=P, k=P, v=P, ld_q=256, ld_kv=256, q_out=2 * P, ld_qo=256,
             k_out=2 * P, ld_ko=128)
    a.update(kw)
    d = dict(tokens=5, n_seqs=3, n_q_heads=4, rot_dim=64, interleaved=0, rope_len=100)
    d.update(desc or {})
    return lib.mgb_kv_append(ctypes.byref(mgb.KVAppendDesc(**d)), ctypes.byref(cache or _cache()),
                             a["cu"], a["lens"], a["rope"], a["q"], a["k"], a["v"], a["ld_q"], a["ld_kv"],
                             a["q_out"], a["ld_qo"], a["k_out"], a["ld_ko"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_append_rejects_bad_caches(lib, kw, status):
    assert _append(lib, _cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(desc=dict(tokens=-1)), mgb.MGB_ERR_INVALID_ARG),
    (dict(desc=dict(n_seqs=-1)), mgb.MGB_ERR_INVALID_ARG),
    (dict(desc=dict(rot_dim=-16)), mgb.MGB_ERR_INVALID_ARG),
    (dict(desc=dict(rot_dim=24)), mgb.MGB_ERR_UNSUPPORTED),
    (dict(desc=dict(rot_dim=80)), mgb.MGB_ERR_INVALID_ARG),          # more than head_dim
    (dict(desc=dict(interleaved=2)), mgb.MGB_ERR_INVALID_ARG),
    (dict(desc=dict(rope_len=0)), mgb.MGB_ERR_INVALID_ARG),
    (dict(desc=dict(n_q_heads=0)), mgb.MGB_ERR_INVALID_ARG),
    (dict(rope=None), mgb.MGB_ERR_INVALID_ARG), (dict(rope=P + 4), mgb.MGB_ERR_MISALIGNED),
    (dict(cu=None), mgb.MGB_ERR_INVALID_ARG),                         # tokens != n_seqs
    (dict(lens=None), mgb.MGB_ERR_INVALID_ARG), (dict(q=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(k=None), mgb.MGB_ERR_INVALID_ARG), (dict(v=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_q=248), mgb.MGB_ERR_INVALID_ARG), (dict(ld_kv=120), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_qo=248), mgb.MGB_ERR_INVALID_ARG), (dict(ld_ko=120), mgb.MGB_ERR_INVALID_ARG),
    (dict(q_out=P, ld_qo=264), mgb.MGB_ERR_INVALID_ARG),              # in place, other stride
    (dict(k_out=P, ld_ko=128), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_q=260), mgb.MGB_ERR_MISALIGNED), (dict(q=P + 8), mgb.MGB_ERR_MISALIGNED),
    (dict(k_out=P + 4), mgb.MGB_ERR_MISALIGNED), (dict(cu=P + 2), mgb.MGB_ERR_MISALIGNED),
    (dict(lens=P + 1), mgb.MGB_ERR_MISALIGNED),
])
def test_append_rejects_bad_arguments(lib, kw, status):
    assert _append(lib, **kw) == status


def test_append_head_dims(lib):
    assert _append(lib, _cache(head_dim=264, stride_head=264, stride_token=528, stride_page=16 * 528),
                   ld_q=4096, ld_qo=4096, ld_kv=4096, ld_ko=4096) == mgb.MGB_ERR_UNSUPPORTED
    assert _append(lib, _cache(head_dim=24), ld_q=4096) == mgb.MGB_ERR_UNSUPPORTED   # bf16: 16s
    # float32 in steps of 8: past every check but the device's
    ok = _append(lib, _cache(head_dim=24, dtype=mgb.MGB_F32), desc=dict(rot_dim=8))
    assert ok in (mgb.MGB_ERR_ARCH, mgb.MGB_ERR_CUDA) or torch.cuda.is_available()


def _ws(lib, n=3, nq=4, nkv=2, d=64):
    return lib.mgb_attention_decode_ws_bytes(n, nq, nkv, d)


@pytest.mark.parametrize("a", [(-1, 4, 2, 64), (3, 0, 2, 64), (3, 4, 0, 64), (3, 4, 3, 64), (3, 4, 2, 96)])
def test_decode_workspace_of_bad_shapes_is_zero(lib, a):
    assert lib.mgb_attention_decode_ws_bytes(*a) == 0


@pytest.mark.parametrize("a,status", [
    ((-1, 4, 2, 64, P, P), mgb.MGB_ERR_INVALID_ARG), ((3, 4, 3, 64, P, P), mgb.MGB_ERR_INVALID_ARG),
    ((3, 4, 2, 80, P, P), mgb.MGB_ERR_UNSUPPORTED), ((3, 4, 2, 64, None, P), mgb.MGB_ERR_INVALID_ARG),
    ((3, 4, 2, 64, P, None), mgb.MGB_ERR_INVALID_ARG), ((3, 4, 2, 64, P, P + 8), mgb.MGB_ERR_MISALIGNED),
    ((3, 4, 2, 64, P + 2, P), mgb.MGB_ERR_MISALIGNED),
])
def test_decode_prepare_rejects(lib, a, status):
    plan = mgb.AttentionDecodePlan()
    n, nq, nkv, d, lens, ws = a
    assert lib.mgb_attention_decode_prepare(n, nq, nkv, d, lens, ws, 1 << 30, ctypes.byref(plan),
                                            None) == status
    if status != mgb.MGB_ERR_UNSUPPORTED:
        assert plan.ws is None


def test_decode_prepare_small_workspace_and_no_plan(lib):
    plan = mgb.AttentionDecodePlan()
    assert lib.mgb_attention_decode_prepare(3, 4, 2, 64, P, P, _ws(lib) - 1, ctypes.byref(plan),
                                            None) == mgb.MGB_ERR_WORKSPACE_TOO_SMALL
    assert lib.mgb_attention_decode_prepare(3, 4, 2, 64, P, P, 1 << 30, None, None) == mgb.MGB_ERR_INVALID_ARG


def _decode(lib, cache=None, plan=None, **kw):
    p = dict(n_seqs=3, n_q_heads=4, n_kv_heads=2, head_dim=64, ws=P, ws_bytes=1 << 30)
    p.update(plan or {})
    a = dict(q=P, ld_q=256, o=P, ld_o=256, lse=P)
    a.update(kw)
    return lib.mgb_attention_decode(ctypes.byref(mgb.AttentionDecodePlan(**p)),
                                    ctypes.byref(cache or _cache()), a["q"], a["ld_q"], a["o"], a["ld_o"],
                                    a["lse"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_decode_rejects_bad_caches(lib, kw, status):
    assert _decode(lib, _cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(plan=dict(ws=None)), mgb.MGB_ERR_INVALID_ARG),
    (dict(plan=dict(ws_bytes=1000)), mgb.MGB_ERR_WORKSPACE_TOO_SMALL),
    (dict(plan=dict(ws=P + 8)), mgb.MGB_ERR_MISALIGNED),
    (dict(plan=dict(n_kv_heads=4)), mgb.MGB_ERR_INVALID_ARG),        # not the cache's
    (dict(plan=dict(head_dim=128)), mgb.MGB_ERR_INVALID_ARG),
    (dict(plan=dict(n_seqs=-1)), mgb.MGB_ERR_INVALID_ARG),
    (dict(q=None), mgb.MGB_ERR_INVALID_ARG), (dict(o=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_q=248), mgb.MGB_ERR_INVALID_ARG), (dict(ld_o=0), mgb.MGB_ERR_INVALID_ARG),
    (dict(q=P + 8), mgb.MGB_ERR_MISALIGNED), (dict(o=P + 4), mgb.MGB_ERR_MISALIGNED),
    (dict(ld_o=260), mgb.MGB_ERR_MISALIGNED), (dict(lse=P + 2), mgb.MGB_ERR_MISALIGNED),
])
def test_decode_rejects_bad_arguments(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_packed_workspace(lib):
    assert lib.mgb_attention_packed_ws_bytes(-1, 5) == 0 and lib.mgb_attention_packed_ws_bytes(2, -1) == 0
    # an entry per 128 (256) rows and sequence, bounded by the rows
    assert lib.mgb_attention_packed_ws_bytes(1 << 20, 10) < 20 << 20
    assert lib.mgb_attention_packed_ws_bytes(8, 1 << 20) >= 16 * ((1 << 13) + (1 << 12))


@pytest.mark.parametrize("a,status", [
    ((-1, 9, 1, P, P), mgb.MGB_ERR_INVALID_ARG), ((2, -9, 1, P, P), mgb.MGB_ERR_INVALID_ARG),
    ((2, 9, 2, P, P), mgb.MGB_ERR_INVALID_ARG), ((2, 9, 1, None, P), mgb.MGB_ERR_INVALID_ARG),
    ((2, 9, 1, P, None), mgb.MGB_ERR_INVALID_ARG), ((2, 9, 1, P + 2, P), mgb.MGB_ERR_MISALIGNED),
    ((2, 9, 1, P, P + 4), mgb.MGB_ERR_MISALIGNED),
])
def test_packed_prepare_rejects(lib, a, status):
    plan = mgb.AttentionPackedPlan()
    n, tokens, causal, cu, ws = a
    assert lib.mgb_attention_packed_prepare(n, tokens, causal, cu, ws, 1 << 30, ctypes.byref(plan),
                                            None) == status
    assert plan.ws is None


def test_packed_prepare_small_workspace_and_no_plan(lib):
    plan = mgb.AttentionPackedPlan()
    size = lib.mgb_attention_packed_ws_bytes(2, 900)
    assert lib.mgb_attention_packed_prepare(2, 900, 1, P, P, size - 1, ctypes.byref(plan),
                                            None) == mgb.MGB_ERR_WORKSPACE_TOO_SMALL
    assert lib.mgb_attention_packed_prepare(2, 9, 1, P, P, 1 << 30, None, None) == mgb.MGB_ERR_INVALID_ARG


def _packed(lib, plan=None, nq=4, nkv=2, d=64, dtype=mgb.MGB_BF16, **kw):
    p = dict(n_seqs=3, tokens=50, causal=1, ws=P, ws_bytes=1 << 30)
    p.update(plan or {})
    a = dict(q=P, k=P, v=P, ld_q=512, ld_kv=512, o=2 * P, ld_o=256, lse=P)
    a.update(kw)
    return lib.mgb_attention_packed_fwd(ctypes.byref(mgb.AttentionPackedPlan(**p)), nq, nkv, d, dtype,
                                        a["q"], a["k"], a["v"], a["ld_q"], a["ld_kv"], a["o"], a["ld_o"],
                                        a["lse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(plan=dict(ws=None)), mgb.MGB_ERR_INVALID_ARG), (dict(plan=dict(tokens=-1)), mgb.MGB_ERR_INVALID_ARG),
    (dict(plan=dict(causal=3)), mgb.MGB_ERR_INVALID_ARG),
    (dict(plan=dict(ws_bytes=100)), mgb.MGB_ERR_WORKSPACE_TOO_SMALL),
    (dict(plan=dict(ws=P + 8)), mgb.MGB_ERR_MISALIGNED),
    (dict(nq=0), mgb.MGB_ERR_INVALID_ARG), (dict(nkv=3), mgb.MGB_ERR_INVALID_ARG),
    (dict(nkv=0), mgb.MGB_ERR_INVALID_ARG), (dict(dtype=2), mgb.MGB_ERR_INVALID_ARG),
    (dict(d=96), mgb.MGB_ERR_UNSUPPORTED), (dict(d=32, dtype=mgb.MGB_F32), mgb.MGB_ERR_UNSUPPORTED),
    (dict(plan=dict(tokens=1 << 30), nq=1 << 20, nkv=1, ld_q=1 << 27, ld_o=1 << 27), mgb.MGB_ERR_UNSUPPORTED),
    (dict(ld_q=248), mgb.MGB_ERR_INVALID_ARG), (dict(ld_kv=120), mgb.MGB_ERR_INVALID_ARG),
    (dict(ld_o=248), mgb.MGB_ERR_INVALID_ARG), (dict(q=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(k=None), mgb.MGB_ERR_INVALID_ARG), (dict(v=None), mgb.MGB_ERR_INVALID_ARG),
    (dict(o=None), mgb.MGB_ERR_INVALID_ARG), (dict(ld_q=516), mgb.MGB_ERR_MISALIGNED),
    (dict(ld_kv=516), mgb.MGB_ERR_MISALIGNED), (dict(ld_o=260), mgb.MGB_ERR_MISALIGNED),
    (dict(v=P + 8), mgb.MGB_ERR_MISALIGNED), (dict(lse=P + 2), mgb.MGB_ERR_MISALIGNED),
])
def test_packed_rejects_bad_arguments(lib, kw, status):
    assert _packed(lib, **kw) == status


def test_fault_injection_and_status_text(lib, monkeypatch):
    assert mgb.status_string(mgb.MGB_ERR_INDEX) not in ("", "unknown status")
    monkeypatch.setenv("MGB_FAULT", "validate")
    assert _append(lib) == mgb.MGB_ERR_INVALID_ARG
    assert _decode(lib) == mgb.MGB_ERR_INVALID_ARG
    assert _packed(lib) == mgb.MGB_ERR_INVALID_ARG


def test_kv_cache_helper_checks_its_tensors():
    k, v = torch.zeros((2, 5, 4, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((3, 2), dtype=torch.int32)
    c = mgb.kv_cache(k, v, t)
    assert (c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.max_pages, c.dtype) == (5, 4, 2, 64, 2, 1)
    assert (c.stride_page, c.stride_token, c.stride_head, c.ld_table) == (512, 128, 64, 2)
    h = mgb.kv_cache(*(x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v)), t)
    assert (h.stride_page, h.stride_token, h.stride_head) == (512, 64, 256)
    for bad in [(k, v[:4], t), (k[0], v[0], t), (k, v.float(), t), (k, v, t.long()), (k, v, t[0]),
                (k.half(), v.half(), t), (k, v.transpose(1, 2).contiguous().transpose(1, 2), t),
                (k, v, t.t()), (k.transpose(2, 3), v.transpose(2, 3), t)]:
        with pytest.raises(ValueError):
            mgb.kv_cache(*bad)
