"""Serving calls that the per-operator suites do not make: outputs that are only
16-byte aligned, separate q, k, v tensors, pages past 2^32 elements, pages two
sequences share, offsets that overlap, one packed plan on two streams, and a
captured fork and join of the three operators."""
import numpy as np
import pytest
import torch

from megatron_transformer_layer_fwd_gb300 import mgb
from megatron_transformer_layer_fwd_gb300.runner import rope_table
from oracle import serving
from tests.serving_util import MGB, TORCH, check_attention, dev, host, ints, values
from tests.test_gpu_attention_packed import _plan, _sums

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_packed_separate_tensors_and_16_byte_outputs(dtype, d, shift):
    """o begins `shift` 16-byte vectors behind a 32-byte boundary, and every row of a
    stride that is an odd number of vectors changes sides."""
    rng = np.random.default_rng(shift)
    nq, nkv, lens = 6, 2, [200, 0, 57, 300]
    cu, T, vn = np.cumsum([0] + lens), sum(lens), 16 // TORCH[dtype].itemsize
    q, k, v = (values(rng, (T, h, d), dtype) for h in (nq, nkv, nkv))
    ld_q, ld_kv, ld_o = nq * d + vn, nkv * d + 3 * vn, nq * d + vn * (1 if shift else 2)

    def rows(x, ld):
        t = torch.full((T, ld), float("nan"), dtype=TORCH[dtype], device="cuda")
        t[:, :x.shape[1] * d] = dev(x.reshape(T, -1), dtype)
        return t
    out = torch.full((T * ld_o + shift * vn,), 3.0, dtype=TORCH[dtype], device="cuda")
    o = out[shift * vn:].view(T, ld_o)
    lse = torch.empty((nq, T), device="cuda")
    mgb.mgb_attention_packed_fwd(_plan(cu, T, True), nq, nkv, d, MGB[dtype], rows(q, ld_q), rows(k, ld_kv),
                                 rows(v, ld_kv), ld_q, ld_kv, o, ld_o, lse)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    ref, rlse = serving.packed_attention(q, k, v, cu, True)
    a, m, n = _sums(q, k, v, cu, True)
    got = host(o)
    assert (got[:, nq * d:] == 3.0).all() and (host(out[:shift * vn]) == 3.0).all()
    check_attention(got[:, :nq * d].reshape(T, nq, d), host(lse).T, ref, rlse.T, a, m, n, d, dtype)


@pytest.mark.parametrize("cu,good", [
    ([0, 60, 0, 60, 100], [0, 60, 60, 60, 100]),                  # the third shares the first's rows
    ([0, 60, 50, 70, 100], [0, 60, 60, 70, 100]),                 # .. and part of them: only 70 .. 100 stays
    ([0, 100] * 1100, [0] + [100] * 2199),                        # past the scan's block
    ([0] * 1024 + [40, 30, 100, 20, 90], [0] * 1024 + [40] * 5),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_that_overlap(dtype, cu, good):
    """Sequences that begin before the end of an earlier one are empty and reported."""
    x = torch.randn((100, 3 * 64), device="cuda").to(TORCH[dtype])
    outs = []
    for c, status in ((cu, mgb.MGB_ERR_INDEX), (good, mgb.MGB_OK)):
        o = torch.zeros((100, 64), device="cuda", dtype=TORCH[dtype])
        mgb.mgb_attention_packed_fwd(_plan(c, 100, True), 1, 1, 64, MGB[dtype], x, x[:, 64:], x[:, 128:], 192,
                                     192, o, 64)
        assert mgb.mgb_device_status() == status
        outs.append(o)
    if cu[2] == 50:
        outs[1][60:70] = 0
    assert torch.equal(outs[0], outs[1]) and bool((outs[0][:40] != 0).any())


def _serve(cache, n, nq, nkv, d, lens, qkv, rope):
    """One appended token per sequence, then attention; the queries and the output."""
    w = (nq + 2 * nkv) * d
    q, o = (torch.zeros((n, nq * d), dtype=qkv.dtype, device="cuda") for _ in range(2))
    mgb.mgb_kv_append(mgb.kv_append_desc(n, n, nq, d, False, rope.shape[0]), cache, None, lens, rope, qkv,
                      qkv[:, nq * d:], qkv[:, (nq + nkv) * d:], w, w, q, nq * d, None, 0)
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d), dtype=torch.uint8, device="cuda")
    plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, lens, ws)
    mgb.mgb_attention_decode(plan, cache, q, nq * d, o, nq * d)
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_past_two_to_the_32_elements(dtype):
    nq, nkv, d, page, pages = 4, 2, 64, 16, 5
    far = (1 << 30) + (1 << 20)      # elements between pages: the last begins past 2^32
    es = TORCH[dtype].itemsize
    if torch.cuda.mem_get_info()[0] < 5 * far * es:
        pytest.skip("not enough free memory")
    big = torch.empty(((pages - 1) * far + (1 << 20),), dtype=TORCH[dtype], device="cuda")
    view = lambda at: big[at:].as_strided((pages, page, nkv, d), (far, nkv * d, d, 1), big.storage_offset() + at)
    near = torch.zeros((2, pages, page, nkv, d), dtype=TORCH[dtype], device="cuda")
    near.normal_()
    pk, pv = view(0), view(1 << 19)
    pk.copy_(near[0])
    pv.copy_(near[1])
    table, lens = ints([[4, 0, 3, -1], [1, -1, -1, -1], [2, 4, -1, -1]]), ints([37, 9, 16])
    table[2, 0] = 2
    qkv = torch.randn((3, (nq + 2 * nkv) * d), device="cuda").to(TORCH[dtype])
    rope = rope_table(64, d)
    a = _serve(mgb.kv_cache(pk, pv, table), 3, nq, nkv, d, lens, qkv, rope)
    b = _serve(mgb.kv_cache(near[0], near[1], table), 3, nq, nkv, d, lens, qkv, rope)
    assert mgb.mgb_device_status() == mgb.MGB_OK
    assert torch.equal(a, b) and bool((a != 0).any())
    assert torch.equal(pk, near[0]) and torch.equal(pv, near[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_share_pages(dtype):
    """A common prefix held once: the same bits as with a copy per sequence."""
    nq, nkv, d, page, n, common = 8, 2, 128, 16, 5, 40
    lens = ints([common * page + 3 + 7 * s for s in range(n)])
    own = 3
    prefix = torch.randn((2, common, page, nkv, d), device="cuda")
    tails = torch.randn((2, n * own, page, nkv, d), device="cuda")
    q = torch.randn((n, nq * d), device="cuda").to(TORCH[dtype])
    outs = []
    for shared in (True, False):
        copies = 1 if shared else n
        pool = torch.cat([prefix] * copies + [tails], dim=1).to(TORCH[dtype])
        at = np.array([[(0 if shared else s * common) + i for i in range(common)]
                       + [copies * common + s * own + i for i in range(own)] for s in range(n)])
        cache = mgb.kv_cache(pool[0], pool[1], ints(at))
        ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d), dtype=torch.uint8, device="cuda")
        plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, lens, ws)
        o = torch.zeros_like(q)
        mgb.mgb_attention_decode(plan, cache, q, nq * d, o, nq * d)
        assert mgb.mgb_device_status() == mgb.MGB_OK
        outs.append(o)
    assert torch.equal(*outs) and bool((outs[0] != 0).any())


def test_one_packed_plan_on_two_streams():
    """Layers of different heads and types read one plan at the same time."""
    lens = [700, 3, 0, 1200, 64]
    cu, T = np.cumsum([0] + lens), sum(lens)
    plan = _plan(cu, T, True)
    torch.cuda.synchronize()
    kinds = [("bf16", 16, 4, 128), ("bf16", 8, 8, 64), ("f32", 4, 1, 64)]
    jobs = []
    for dtype, nq, nkv, d in kinds:
        w = (nq + 2 * nkv) * d
        x = torch.randn((T, w), device="cuda").to(TORCH[dtype])
        jobs.append((dtype, nq, nkv, d, w, x))

    def run(job, o):
        dtype, nq, nkv, d, w, x = job
        mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, MGB[dtype], x, x[:, nq * d:], x[:, (nq + nkv) * d:], w, w,
                                     o, nq * d)
    make = lambda: [torch.zeros((T, j[1] * j[3]), dtype=TORCH[j[0]], device="cuda") for j in jobs]
    alone = make()
    for j, o in zip(jobs, alone):
        run(j, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = make()
        torch.cuda.synchronize()
        for _ in range(3):
            for st, j, o in zip(streams, jobs, outs):
                with torch.cuda.stream(st):
                    run(j, o)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert mgb.mgb_device_status() == mgb.MGB_OK


def test_captured_fork_and_join():
    """Two layers' appends on a forked stream, their attentions joined behind it,
    prompts beside it: replays give the bits of eager calls in one stream."""
    nq, nkv, d, page, n, T = 4, 2, 64, 8, 3, 200
    w = (nq + 2 * nkv) * d
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)
    table, lens, rope = ints(np.arange(n * 8).reshape(n, 8)), ints([5, 60, 1]), rope_table(64, d)
    cu = ints([0, 90, 150])
    pools, qkv, prompt = new(2, 2, n * 8, page, nkv, d), new(2, n, w), new(T, w)
    start = pools.clone()
    q, o = torch.zeros((2, n, nq * d), dtype=torch.bfloat16, device="cuda"), new(2, n, nq * d)
    op = torch.zeros((T, nq * d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mgb.mgb_attention_decode_ws_bytes(n, nq, nkv, d), dtype=torch.uint8, device="cuda")
    wp = torch.empty(mgb.mgb_attention_packed_ws_bytes(2, T), dtype=torch.uint8, device="cuda")
    desc = mgb.kv_append_desc(n, n, nq, d, False, 64)
    caches = [mgb.kv_cache(pools[i, 0], pools[i, 1], table) for i in range(2)]

    def append(i):
        mgb.mgb_kv_append(desc, caches[i], None, lens, rope, qkv[i], qkv[i][:, nq * d:],
                          qkv[i][:, (nq + nkv) * d:], w, w, q[i], nq * d, None, 0)

    def step(fork):
        main = torch.cuda.current_stream()
        side = torch.cuda.Stream() if fork else main
        side.wait_stream(main)
        with torch.cuda.stream(side):
            append(0)
            append(1)
        plan = mgb.mgb_attention_decode_prepare(n, nq, nkv, d, lens, ws)
        packed = mgb.mgb_attention_packed_prepare(2, T, True, cu, wp)
        mgb.mgb_attention_packed_fwd(packed, nq, nkv, d, mgb.MGB_BF16, prompt, prompt[:, nq * d:],
                                     prompt[:, (nq + nkv) * d:], w, w, op, nq * d)
        main.wait_stream(side)
        for i in range(2):
            mgb.mgb_attention_decode(plan, caches[i], q[i], nq * d, o[i], nq * d)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(False)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(True)
    for now in ([5, 60, 1], [0, 64, 33], [2, 2, 2]):
        got = []
        for replay in (False, True):
            lens.copy_(ints(now))
            pools.copy_(start)
            o.fill_(0)
            op.fill_(0)
            if replay:
                graph.replay()
            else:
                step(False)
            got.append((o.clone(), op.clone(), pools.clone()))
        assert mgb.mgb_device_status() == mgb.MGB_OK
        assert all(torch.equal(a, b) for a, b in zip(*got)) and bool((got[0][0] != 0).any())
