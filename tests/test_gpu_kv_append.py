"""GPU parity of mgb_kv_append against the float64 oracle: dtypes, rotation
forms, page sizes and layouts, ragged and empty sequences, padding, in-place
outputs, untouched slots and rows, device-side index errors, graph replay."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from oracle import serving
from tests.serving_util import HALF_STEP, Cache, dev, host, ints, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built(mgb_lib):
    return mgb_lib


def _check_rotated(got, x, rows, rot, interleaved, dtype):
    """a c - b s in float32 with one fused multiply-add: the product b s and the
    sum are rounded to half a float32 step each, the result once to dtype."""
    ref = serving.rope_rotate(x, rows, interleaved) if rot else x
    step = np.abs(x).max(axis=-1, keepdims=True) * 2.0 ** -24 * (4 if rot else 0)
    tol = step + (HALF_STEP[dtype] if rot else 0.0) * (np.abs(ref) + step)
    if rot and rot < x.shape[-1]:
        tol[..., rot:] = 0.0
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


def _run(seed, dtype, nq, nkv, d, rot, interleaved, page, new, ctx, head_major=False, tail=0,
         in_place=False, want_q=True, want_k=True, cu_null=False):
    rng = np.random.default_rng(seed)
    lens = [0 if c < 0 else n + c for n, c in zip(new, ctx)]
    cu = np.cumsum([0] + list(new))
    T = int(cu[-1]) + tail
    w = (nq + 2 * nkv) * d
    x = values(rng, (T, nq + 2 * nkv, d), dtype)
    c = Cache(rng, lens, page, nkv, d, dtype, head_major)
    before = [t.clone() for t in (c.tk, c.tv)]
    rope_len = max([1] + lens)
    rope = rope_table(rope_len, rot) if rot else None
    qkv = dev(x.reshape(T, w), dtype)
    q, k, v = qkv, qkv[:, nq * d:], qkv[:, (nq + nkv) * d:]
    if in_place:
        q_out, ldq, k_out, ldk = q, w, k, w
        old_q, old_k = x[:, :nq].copy(), x[:, nq:nq + nkv].copy()
    else:
        q_out = torch.full((T, nq * d + 16), 7.0, dtype=qkv.dtype, device="cuda")
        k_out = torch.full((T, nkv * d), 7.0, dtype=qkv.dtype, device="cuda")
        ldq, ldk = nq * d + 16, nkv * d
        old_q, old_k = np.full((T, nq, d), 7.0), np.full((T, nkv, d), 7.0)
    desc = mgb.kv_append_desc(T, len(new), nq, rot, interleaved, rope_len if rot else 0)
    mgb.mgb_kv_append(desc, c.desc, None if cu_null else ints(cu), ints(lens), rope,
                      q if want_q else None, k, v, w, w, q_out if want_q else None, ldq,
                      k_out if want_k else None, ldk)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    gq = host(q_out)[:, :nq * d].reshape(T, nq, d)
    gk = host(k_out)[:, :nkv * d].reshape(T, nkv, d)
    if not in_place:
        assert (host(q_out)[:, nq * d:] == 7.0).all()
    rows64 = host(rope) if rot else None
    expect_slots = np.zeros(c.k.shape[:2], dtype=bool)
    pk, pv = host(c.tk), host(c.tv)
    for t, (s, p) in enumerate(serving.append_positions(cu, lens, T)):
        if s < 0 or not want_q:
            assert (gq[t] == old_q[t]).all()
        if s < 0 or not want_k:
            assert (gk[t] == old_k[t]).all()
        if s < 0:
            continue
        row = rows64[p:p + 1] if rot else None
        if want_q:
            _check_rotated(gq[t:t + 1], x[t:t + 1, :nq], row, rot, interleaved, dtype)
        slot = c.table[s][p // page], p % page
        expect_slots[slot] = True
        if want_k:
            assert (gk[t] == pk[slot]).all()
        _check_rotated(pk[slot][None], x[t:t + 1, nq:nq + nkv], row, rot, interleaved, dtype)
        assert (pv[slot] == x[t, nq + nkv:]).all()
    for pool, b in ((c.tk, before[0]), (c.tv, before[1])):
        same = (pool.contiguous().view(torch.uint8) == b.contiguous().view(torch.uint8))
        same = same.view(*c.k.shape[:2], -1).all(-1).cpu().numpy()
        assert same[~expect_slots].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (64, 16), (128, 96), (256, 32), (32, 0)])
def test_rotation_forms(dtype, interleaved, d, rot):
    _run(1, dtype, 4, 2, d, rot, interleaved, 16, [5, 3], [0, 30])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,head_major", [(1, False), (16, True), (24, False), (64, True), (7, True)])
def test_pages_and_layouts(dtype, page, head_major):
    _run(2, dtype, 3, 3, 64, 64, False, page, [1, 0, 40, 7, 1], [63, 5, 23, -1, 0], head_major, tail=3)


@pytest.mark.parametrize("nq,nkv", [(1, 1), (32, 8), (71, 1), (5, 5), (64, 16)])
def test_head_counts(nq, nkv):
    """From fewer units than a warp to more than a block's threads."""
    _run(3, "bf16", nq, nkv, 128, 128, False, 16, [3, 9], [100, 2], tail=1)
    _run(3, "f32", nq, nkv, 64, 32, True, 16, [3, 9], [100, 2])


@pytest.mark.parametrize("n", [1, 2, 33, 40, 1100])
def test_one_token_per_sequence(n):
    rng = np.random.default_rng(n)
    ctx = [int(rng.integers(0, 300)) if rng.random() < 0.9 else -1 for _ in range(n)]
    _run(4, "bf16", 4, 1, 64, 64, False, 32, [1] * n, ctx, cu_null=True)


def test_many_sequences_search():
    """More sequences than one round of the 32-way search covers, many of them empty."""
    rng = np.random.default_rng(8)
    new = [int(x) for x in rng.integers(0, 4, size=1500)]
    _run(5, "bf16", 2, 1, 32, 32, False, 8, new, [int(x) for x in rng.integers(0, 9, size=1500)], tail=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_optional_outputs(dtype):
    _run(6, dtype, 4, 2, 128, 128, False, 16, [17, 4], [9, 0], in_place=True, tail=2)
    _run(6, dtype, 4, 2, 128, 64, True, 16, [17, 4], [9, 0], in_place=True)
    _run(6, dtype, 4, 2, 128, 128, False, 16, [17, 4], [9, 0], want_q=False)
    _run(6, dtype, 4, 2, 128, 128, False, 16, [17, 4], [9, 0], want_k=False)


def _simple(lens, new, table=None, rope_len=64, page=8, pages=4, max_pages=2):
    T = sum(new)
    qkv = torch.randn((T, 4 * 64), device="cuda").bfloat16()
    pool = torch.zeros((2, pages, page, 1, 64), device="cuda", dtype=torch.bfloat16)
    table = ints(table if table is not None else [[i % pages] * max_pages for i in range(len(lens))])
    out = torch.zeros((T, 128), device="cuda", dtype=torch.bfloat16)
    mgb.mgb_kv_append(mgb.kv_append_desc(T, len(lens), 2, 64, False, rope_len),
                      mgb.kv_cache(pool[0], pool[1], table), ints(np.cumsum([0] + new)), ints(lens),
                      rope_table(rope_len, 64), qkv, qkv[:, 128:], qkv[:, 192:], 256, 256, out, 128, None, 0)
    return mgb.mgb_device_status(), out, pool


@pytest.mark.parametrize("lens,bad,kw", [
    ([2, -1], [2, 3], {}), ([2, 1], [2], {}),               # position below 0 (-1, then 0)
    ([2, 17], [3], {}),                                     # past the table (15, then 16)
    ([2, 9], [3], dict(rope_len=8)),                        # past the rotary table (7, then 8)
    ([2, 3], [2, 3], dict(table=[[0, 0], [4, 0]])), ([2, 3], [2, 3], dict(table=[[0, 0], [-1, 0]])),
])
def test_bad_indices_are_reported_and_skipped(lens, bad, kw):
    """Rows of the second sequence are out of range: an error, no store for
    them, and the other rows served as usual."""
    st, out, pool = _simple(lens, [2, 2], **kw)
    assert st == mgb.MGB_ERR_INDEX
    assert [t for t in range(4) if not bool((out[t] != 0).any())] == bad
    assert int((pool[0] != 0).any(-1).sum()) == 4 - len(bad)
    assert mgb.mgb_device_status() == mgb.MGB_OK            # read and cleared


def test_no_tokens():
    st, out, pool = _simple([3, 4], [0, 0])
    assert st == mgb.MGB_OK and (pool == 0).all()


def test_captured_step_follows_the_lengths():
    """A captured append replays with new lengths and new values."""
    n, d, page = 3, 64, 4
    qkv = torch.randn((n, 3 * d), device="cuda").bfloat16()
    pool = torch.zeros((2, 9, page, 1, d), device="cuda", dtype=torch.bfloat16)
    cache = mgb.kv_cache(pool[0], pool[1], ints(np.arange(9).reshape(3, 3)))
    lens = ints([1, 1, 1])
    desc = mgb.kv_append_desc(n, n, 1, 0, False, 0)
    call = lambda: mgb.mgb_kv_append(desc, cache, None, lens, None, None, qkv[:, d:], qkv[:, 2 * d:],
                                     3 * d, 3 * d, None, 0, None, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for step in range(1, 12):
        qkv.normal_()
        lens.fill_(step)
        g.replay()
        flat = pool.view(2, 3, 3 * page, d)
        assert torch.equal(flat[0][:, step - 1], qkv[:, d:2 * d])
        assert torch.equal(flat[1][:, step - 1], qkv[:, 2 * d:])
    assert mgb.mgb_device_status() == mgb.MGB_OK
