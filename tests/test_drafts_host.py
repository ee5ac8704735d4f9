"""Refusals of the entry points for drafted tokens, before any launch (no GPU needed)."""
import ctypes
import os

import pytest

from megatron_transformer_layer_fwd_gb300 import mgb
from tests.test_serving_host import BAD_CACHE, P, _cache

INV, UNS, MIS, SMALL = (mgb.MGB_ERR_INVALID_ARG, mgb.MGB_ERR_UNSUPPORTED, mgb.MGB_ERR_MISALIGNED,
                        mgb.MGB_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mgb.LIB_PATH):
        from megatron_transformer_layer_fwd_gb300 import build
        build.build()
    return mgb.load()


def _plan(lib, **kw):
    a = dict(n_seqs=3, tokens=5, n_q_heads=4, n_kv_heads=2, head_dim=64, ws=P)
    a.update(kw)
    size = a.pop("ws_bytes", None)
    if size is None:
        size = lib.mgb_attention_tree_ws_bytes(a["n_seqs"], a["tokens"], a["n_q_heads"], a["n_kv_heads"],
                                               a["head_dim"])
    return mgb.AttentionTreePlan(ws_bytes=size, **a)


BAD_PLAN = [(dict(n_seqs=-1), INV), (dict(tokens=-1), INV), (dict(n_q_heads=3), INV), (dict(n_q_heads=0), INV),
            (dict(n_kv_heads=0), INV), (dict(ws=None), INV), (dict(ws=P + 8), MIS), (dict(head_dim=96), UNS),
            (dict(ws_bytes=1000), SMALL)]


@pytest.mark.parametrize("a", [(-1, 5, 4, 2, 64), (3, -1, 4, 2, 64), (3, 5, 0, 2, 64), (3, 5, 4, 0, 64),
                               (3, 5, 4, 3, 64), (3, 5, 4, 2, 80)])
def test_workspace_of_bad_shapes_is_zero(lib, a):
    assert lib.mgb_attention_tree_ws_bytes(*a) == 0


def test_limit_is_the_headers(lib):
    text = open(mgb.HEADER).read()
    assert f"#define MGB_TREE_MAX_TOKENS {mgb.TREE_MAX_TOKENS}\n" in text


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INV), (dict(tokens=-1), INV), (dict(nq=3), INV), (dict(d=80), UNS), (dict(cu=None), INV),
    (dict(lens=None), INV), (dict(ws=None), INV), (dict(ws=P + 8), MIS), (dict(cu=P + 2), MIS),
    (dict(lens=P + 1), MIS), (dict(parents=P + 3), MIS), (dict(size=100), SMALL), (dict(plan=None), INV),
])
def test_prepare_rejects(lib, kw, status):
    a = dict(n=3, tokens=5, nq=4, nkv=2, d=64, cu=P, lens=P, parents=P, ws=P,
             size=lib.mgb_attention_tree_ws_bytes(3, 5, 4, 2, 64), plan=ctypes.byref(mgb.AttentionTreePlan()))
    a.update(kw)
    assert lib.mgb_attention_tree_prepare(a["n"], a["tokens"], a["nq"], a["nkv"], a["d"], a["cu"], a["lens"],
                                          a["parents"], a["ws"], a["size"], a["plan"], None) == status


def _tree(lib, plan=None, cache=None, **kw):
    a = dict(q=P, ld_q=256, o=2 * P, ld_o=256, lse=P)
    a.update(kw)
    return lib.mgb_attention_tree(ctypes.byref(plan or _plan(lib)), ctypes.byref(cache or _cache()), a["q"],
                                  a["ld_q"], a["o"], a["ld_o"], a["lse"], None)


def _append(lib, plan=None, cache=None, desc=None, **kw):
    a = dict(rope=P, q=P, k=P, v=P, ld_q=256, ld_kv=256, q_out=2 * P, ld_qo=256, k_out=2 * P, ld_ko=128)
    a.update(kw)
    d = dict(tokens=5, n_seqs=3, n_q_heads=4, rot_dim=64, interleaved=0, rope_len=100)
    d.update(desc or {})
    return lib.mgb_kv_append_tree(ctypes.byref(plan or _plan(lib)), ctypes.byref(mgb.KVAppendDesc(**d)),
                                  ctypes.byref(cache or _cache()), a["rope"], a["q"], a["k"], a["v"], a["ld_q"],
                                  a["ld_kv"], a["q_out"], a["ld_qo"], a["k_out"], a["ld_ko"], None)


def _accept(lib, plan=None, cache=None, accepted=P, new_lens=2 * P):
    return lib.mgb_kv_accept(ctypes.byref(plan or _plan(lib)), ctypes.byref(cache or _cache()), accepted, new_lens,
                             None)


@pytest.mark.parametrize("call", [_tree, _append, _accept])
@pytest.mark.parametrize("kw,status", BAD_PLAN)
def test_bad_plans(lib, call, kw, status):
    assert call(lib, plan=_plan(lib, **kw)) == status


@pytest.mark.parametrize("call", [_tree, _append, _accept])
@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(n_kv_heads=1), INV), (dict(head_dim=128, stride_head=128, stride_token=256, stride_page=4096), INV)])
def test_bad_caches(lib, call, kw, status):
    assert call(lib, cache=_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(o=None), INV), (dict(o=P), INV), (dict(ld_q=248), INV), (dict(ld_o=248), INV),
    (dict(ld_q=260), MIS), (dict(ld_o=260), MIS), (dict(q=P + 8), MIS), (dict(o=P + 8), MIS), (dict(lse=P + 2), MIS),
])
def test_attention_rejects(lib, kw, status):
    assert _tree(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(desc=dict(tokens=6)), INV), (dict(desc=dict(n_seqs=2)), INV), (dict(desc=dict(n_q_heads=2)), INV),
    (dict(desc=dict(whole=1)), INV), (dict(desc=dict(rot_dim=24)), UNS), (dict(desc=dict(rope_len=0)), INV),
    (dict(rope=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(ld_q=248), INV),
    (dict(ld_kv=120), INV), (dict(q_out=P, ld_qo=264), INV), (dict(k=P + 8), MIS), (dict(ld_ko=132), MIS),
])
def test_append_rejects(lib, kw, status):
    assert _append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(accepted=None), INV), (dict(accepted=P + 2), MIS), (dict(new_lens=P + 1), MIS), (dict(new_lens=P), INV),
])
def test_accept_rejects(lib, kw, status):
    assert _accept(lib, **kw) == status


def _copy(lib, cache=None, n=2, src=P, dst=P, slots=P):
    return lib.mgb_kv_copy_pages(ctypes.byref(cache or _cache()), n, src, dst, slots, None)


@pytest.mark.parametrize("kw,status", [x for x in BAD_CACHE if not {"block_table", "ld_table"} & set(x[0])] + [
    (dict(block_table=P + 1), MIS), (dict(head_dim=60), UNS)])
def test_copy_bad_caches(lib, kw, status):
    assert _copy(lib, cache=_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INV), (dict(src=None), INV), (dict(dst=None), INV), (dict(src=P + 1), MIS), (dict(dst=P + 2), MIS),
    (dict(slots=P + 3), MIS),
])
def test_copy_rejects(lib, kw, status):
    assert _copy(lib, **kw) == status


def test_no_plan(lib):
    c, d = ctypes.byref(_cache()), ctypes.byref(mgb.KVAppendDesc(tokens=5, n_seqs=3, n_q_heads=4))
    assert lib.mgb_attention_tree(None, c, P, 256, 2 * P, 256, None, None) == INV
    assert lib.mgb_kv_accept(None, c, P, None, None) == INV
    assert lib.mgb_kv_append_tree(None, d, c, P, P, P, P, 256, 256, None, 0, None, 0, None) == INV
