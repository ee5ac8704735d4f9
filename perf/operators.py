"""The serving operators and the sizes they are measured at.

Three operators that a program which runs a trained layer calls one after the
other: `append` (a step's keys and values into a paged cache, queries and keys
rotated by their positions on the way), `packed` (attention over a batch of
prompts of different lengths laid one behind the other) and `decode` (attention
of one new token per sequence over the paged cache).

A case names an operator and its sizes. Sequence lengths are drawn from the
case itself (log-uniform between its bounds), values from the seed. With
`own` false `run` computes the operators in elementary float32 torch
operations; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    gqa = dict(nq=32, nkv=8, d=128, dtype="bf16")   # the grouped-head layer of the benchmark
    mha = dict(nq=16, nkv=16, d=128, dtype="bf16")  # the causal layer with as many key heads
    return [
        # a prompt batch enters the cache: 8192 tokens of a few sequences
        dict(name="append_prompts", op="append", **gqa, seqs=5, new_lo=600, new_hi=3000, ctx_lo=0,
             ctx_hi=0, page=64, head_major=False, rot=128, interleaved=False, pad=0, tail=7),
        # one user, one token: nothing but latency
        dict(name="append_one_token", op="append", **gqa, seqs=1, new_lo=1, new_hi=1, ctx_lo=4321,
             ctx_hi=4321, page=16, head_major=False, rot=128, interleaved=False, pad=0, tail=0),
        # a decode step of a padded batch, float32, a quarter of each head rotated in pairs
        dict(name="append_step_f32_partial", op="append", nq=16, nkv=4, d=64, dtype="f32", seqs=96,
             new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=60000, page=32, head_major=True, rot=16,
             interleaved=True, pad=5, tail=0),
        # two long documents, as many tokens as the benchmark's layer step
        dict(name="packed_long", op="packed", **gqa, seqs=2, len_lo=4000, len_hi=4200, causal=True,
             tail=0, lse=True, plan="kept"),
        # a batch of chat prompts, most of them short; the plan is made in the pass
        dict(name="packed_ragged", op="packed", **mha, seqs=48, len_lo=9, len_hi=1500, causal=True,
             tail=21, lse=False, plan="made"),
        # one short prompt: latency
        dict(name="packed_one_short", op="packed", nq=16, nkv=16, d=64, dtype="bf16", seqs=1,
             len_lo=37, len_hi=37, causal=True, tail=0, lse=False, plan="kept"),
        # encoder-style batch without the causal mask, float32 and small heads
        dict(name="packed_f32_full", op="packed", nq=8, nkv=2, d=64, dtype="f32", seqs=6, len_lo=100,
             len_hi=900, causal=False, tail=3, lse=True, plan="kept"),
        # one user with a short history; the plan is made in the pass
        dict(name="decode_one_short", op="decode", **gqa, seqs=1, len_lo=77, len_hi=77, page=16,
             head_major=False, pad=0, lse=False, plan="made"),
        # one user with a very long document
        dict(name="decode_one_long", op="decode", **gqa, seqs=1, len_lo=131001, len_hi=131001,
             page=64, head_major=False, pad=0, lse=False, plan="kept"),
        # a serving batch of mixed histories
        dict(name="decode_ragged", op="decode", **gqa, seqs=64, len_lo=33, len_hi=16000, page=16,
             head_major=False, pad=3, lse=True, plan="kept"),
        # many short histories, every query head with its own key head
        dict(name="decode_many_mha", op="decode", nq=16, nkv=16, d=64, dtype="bf16", seqs=200,
             len_lo=20, len_hi=1200, page=24, head_major=True, pad=0, lse=False, plan="made"),
        # float32 cache
        dict(name="decode_f32", op="decode", nq=16, nkv=4, d=128, dtype="f32", seqs=12, len_lo=5,
             len_hi=5000, page=32, head_major=False, pad=1, lse=True, plan="kept"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "packed", "decode"])
    nkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if nkv * group > 64:
        group = 64 // nkv
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = dict(op=op, nq=nkv * group, nkv=nkv, d=rng.choice([64, 128]), dtype=dtype)
    if op == "packed":
        budget = 8192 if dtype == "bf16" else 1024   # tokens
        seqs = _log_int(rng, 1, 100)
        hi = max(1, min(4200 if dtype == "bf16" else 900, budget // seqs))
        lo = _log_int(rng, 1, hi)
        if c["nq"] * hi > 32 * 4200:
            hi = max(lo, 32 * 4200 // c["nq"])
        c.update(seqs=seqs, len_lo=lo, len_hi=hi, causal=rng.random() < 0.75,
                 tail=rng.choice([0, 0, 1, 13]), lse=rng.random() < 0.5,
                 plan=rng.choice(["kept", "made"]))
        return c
    c.update(page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128, 256]), head_major=rng.random() < 0.5,
             pad=rng.choice([0, 0, 1, 4]))
    if op == "append":
        seqs = _log_int(rng, 1, 200)
        hi = _log_int(rng, 1, max(1, 6000 // seqs))
        ctx = _log_int(rng, 1, max(2, 60000 // max(1, seqs // 4)))
        rot = rng.choice([0, 16, 32, 64, c["d"]])
        c.update(seqs=seqs, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=0 if ctx < 4 else ctx // 4,
                 ctx_hi=ctx, rot=rot, interleaved=rng.random() < 0.4, tail=rng.choice([0, 0, 5]))
        if c["new_hi"] > 1:
            c["pad"] = 0
        return c
    seqs = _log_int(rng, 1, 220)
    per_token = nkv * c["d"] * (2 if dtype == "bf16" else 4)      # half a cached token's bytes
    room = int(130000 * 8 * 128 * 2 / per_token / seqs)           # as many bytes as the largest case
    hi = _log_int(rng, 1, max(1, min(room, 131000)))
    c.update(seqs=seqs, len_lo=_log_int(rng, 1, hi), len_hi=hi, lse=rng.random() < 0.5,
             plan=rng.choice(["kept", "made"]))
    return c


def _spread(n, lo, hi, salt):
    """n lengths between lo and hi (log-uniform), the same for every seed."""
    rng = random.Random(1000003 * n + 101 * lo + hi + 7919 * salt)
    return [int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(n)]


def _new_and_ctx(c):
    """append: (new tokens, tokens cached before) per sequence, padding last."""
    pad = c["pad"]
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"], 1) + [1] * pad
    ctx = _spread(c["seqs"], c["ctx_lo"], c["ctx_hi"], 2) + [-1] * pad
    return new, ctx


def _lens(c):
    return _spread(c["seqs"], c["len_lo"], c["len_hi"], 3) + [0] * c.get("pad", 0)


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _pages(gen, c, counts, margin=3):
    """A shuffled block table with pages for counts[s] tokens, and the pool size."""
    need = [(n + c["page"] - 1) // c["page"] for n in counts]
    n_pages = sum(need) + margin
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(need))
    table = torch.zeros((len(counts), width), dtype=torch.int32, device="cuda")
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    return table, n_pages


def _pool(c, n_pages, dtype, fill):
    """[n_pages, page, nkv, d] view of a pool stored token-major or head-major."""
    if c["head_major"]:
        return fill((n_pages, c["nkv"], c["page"], c["d"]), dtype).transpose(1, 2)
    return fill((n_pages, c["page"], c["nkv"], c["d"]), dtype)


def _rope_rows(positions, rot, base=10000.0):
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    p = torch.arange(positions, device="cuda", dtype=torch.float64)
    a = p[:, None] * torch.exp(j * (-2.0 * math.log(base) / rot))[None, :]
    return torch.stack((torch.cos(a), torch.sin(a)), dim=-1).to(torch.float32).contiguous()


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1 + 7 * seed)
    dt = _DTYPES[c["dtype"]]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    s = {"case": c}
    if c["op"] == "append":
        new, ctx = _new_and_ctx(c)
        total = sum(new) + c["tail"]
        lens = [a + b for a, b in zip(new, ctx)]
        s["tokens"] = total
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32,
                               device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["table"], n_pages = _pages(gen, c, lens)
        s["qkv"] = _randn(gen, (total, (nq + 2 * nkv) * d), dt)
        fill = lambda shape, t: _randn(gen, shape, t)
        s["k_pool"], s["v_pool"] = (_pool(c, n_pages, dt, fill) for _ in range(2))
        s["rope_len"] = max(1, max(lens))
        s["rope"] = _rope_rows(s["rope_len"], c["rot"]) if c["rot"] else None
        s["q_out"] = torch.zeros((total, nq * d), dtype=dt, device="cuda")
        s["k_out"] = torch.zeros((total, nkv * d), dtype=dt, device="cuda")
        return s
    lens = _lens(c)
    if c["op"] == "packed":
        total = sum(lens) + c["tail"]
        s["tokens"] = total
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                               device="cuda")
        s["qkv"] = _randn(gen, (total, (nq + 2 * nkv) * d), dt)
        s["o"] = torch.zeros((total, nq * d), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((nq, total), dtype=torch.float32, device="cuda") if c["lse"] else None
        return s
    n = len(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"], n_pages = _pages(gen, c, lens)
    fill = lambda shape, t: _randn(gen, shape, t)
    s["k_pool"], s["v_pool"] = (_pool(c, n_pages, dt, fill) for _ in range(2))
    s["q"] = _randn(gen, (n, (nq + 2 * nkv) * d), dt, 1.5)  # the query columns of a fused projection
    s["o"] = torch.zeros((n, nq * d), dtype=dt, device="cuda")
    s["lse"] = torch.zeros((n, nq), dtype=torch.float32, device="cuda") if c["lse"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    # the lengths are the program's own: it laid the batch out
    s["host_lens"] = _new_and_ctx(c) if c["op"] == "append" else _lens(c)
    if own:
        from megatron_transformer_layer_fwd_gb300 import mgb
        if c["op"] != "packed":
            s["cache"] = mgb.kv_cache(s["k_pool"], s["v_pool"], s["table"])
        if c["op"] == "append":
            s["desc"] = mgb.kv_append_desc(s["tokens"], s["lens"].numel(), c["nq"], c["rot"],
                                           c["interleaved"], s["rope_len"] if c["rot"] else 0)
        elif c["op"] == "packed":
            s["ws"] = torch.empty(mgb.mgb_attention_packed_ws_bytes(len(_lens(c)), s["tokens"]),
                                  dtype=torch.uint8, device="cuda")
            s["plan"] = _packed_plan(s)
        else:
            s["ws"] = torch.empty(
                mgb.mgb_attention_decode_ws_bytes(s["lens"].numel(), c["nq"], c["nkv"], c["d"]),
                dtype=torch.uint8, device="cuda")
            s["plan"] = _decode_plan(s)
    return s


# ------------------------------------------------------------------ the library's calls
def _packed_plan(s):
    from megatron_transformer_layer_fwd_gb300 import mgb
    c = s["case"]
    return mgb.mgb_attention_packed_prepare(s["cu"].numel() - 1, s["tokens"], c["causal"], s["cu"], s["ws"])


def _decode_plan(s):
    from megatron_transformer_layer_fwd_gb300 import mgb
    c = s["case"]
    return mgb.mgb_attention_decode_prepare(s["lens"].numel(), c["nq"], c["nkv"], c["d"], s["lens"], s["ws"])


def _run_own(s):
    from megatron_transformer_layer_fwd_gb300 import mgb
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    w = (nq + 2 * nkv) * d
    if c["op"] == "append":
        qkv = s["qkv"]
        mgb.mgb_kv_append(s["desc"], s["cache"], s["cu"], s["lens"], s["rope"], qkv, qkv[:, nq * d:],
                          qkv[:, (nq + nkv) * d:], w, w, s["q_out"], nq * d, s["k_out"], nkv * d)
        return s["q_out"], s["k_out"], s["k_pool"], s["v_pool"]
    if c["op"] == "packed":
        plan = _packed_plan(s) if c["plan"] == "made" else s["plan"]
        qkv = s["qkv"]
        dt = mgb.MGB_BF16 if c["dtype"] == "bf16" else mgb.MGB_F32
        mgb.mgb_attention_packed_fwd(plan, nq, nkv, d, dt, qkv, qkv[:, nq * d:],
                                     qkv[:, (nq + nkv) * d:], w, w, s["o"], nq * d, s["lse"])
    else:
        plan = _decode_plan(s) if c["plan"] == "made" else s["plan"]
        mgb.mgb_attention_decode(plan, s["cache"], s["q"], w, s["o"], nq * d, s["lse"])
    return (s["o"], s["lse"]) if c["lse"] else (s["o"],)


# ------------------------------------------------------------------ plain forms
def _rotate_plain(x, rows, c):
    """x [T, heads, d] float32, rows [T, rot/2, 2]."""
    rot = c["rot"]
    if rot == 0:
        return x
    cs, sn = rows[:, None, :, 0], rows[:, None, :, 1]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cs - b * sn, a * sn + b * cs), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * cs - b * sn, a * sn + b * cs), dim=-1)
    return torch.cat((r, x[..., rot:]), dim=-1)


def _append_plain(s):
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    T, cu, lens = s["tokens"], s["cu"].long(), s["lens"].long()
    t = torch.arange(T, device="cuda")
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    inside = seq < lens.numel()
    seq = seq.clamp(max=lens.numel() - 1)
    pos = lens[seq] - (cu[seq + 1] - cu[seq]) + t - cu[seq]
    ok = (inside & (pos >= 0))
    t, seq, pos = t[ok], seq[ok], pos[ok]
    x = s["qkv"][t].float().view(-1, nq + 2 * nkv, d)
    rows = s["rope"][pos] if c["rot"] else None
    q = _rotate_plain(x[:, :nq], rows, c)
    k = _rotate_plain(x[:, nq:nq + nkv], rows, c)
    dt = s["qkv"].dtype
    s["q_out"][t] = q.reshape(-1, nq * d).to(dt)
    s["k_out"][t] = k.reshape(-1, nkv * d).to(dt)
    page = s["table"].long()[seq, pos // c["page"]]
    s["k_pool"][page, pos % c["page"]] = k.to(dt)
    s["v_pool"][page, pos % c["page"]] = x[:, nq + nkv:].to(dt)
    return s["q_out"], s["k_out"], s["k_pool"], s["v_pool"]


def _softmax_plain(q, k, v, group, causal):
    """q [L, nq, d], k and v [N, nkv, d], float32 -> o [L, nq, d], lse [nq, L]."""
    L, nq, d = q.shape
    nkv = k.shape[1]
    qh = q.permute(1, 0, 2).reshape(nkv, group * L, d)
    sc = torch.matmul(qh, k.permute(1, 2, 0)) * (1.0 / math.sqrt(d))
    sc = sc.view(nkv, group, L, -1)
    if causal:
        i = torch.arange(L, device=q.device)
        sc = sc.masked_fill(i[None, :] > i[:, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul((e / z).view(nkv, group * L, -1), v.permute(1, 0, 2))
    lse = (m + torch.log(z)).view(nq, L)
    return o.view(nq, L, d).permute(1, 0, 2), lse


def _packed_plain(s):
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    at = 0
    for n in s["host_lens"]:
        if n:
            x = s["qkv"][at:at + n].float().view(n, nq + 2 * nkv, d)
            o, lse = _softmax_plain(x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:], nq // nkv, c["causal"])
            s["o"][at:at + n] = o.reshape(n, nq * d).to(s["o"].dtype)
            if s["lse"] is not None:
                s["lse"][:, at:at + n] = lse
        at += n
    return (s["o"], s["lse"]) if c["lse"] else (s["o"],)


def _decode_plain(s):
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            s["o"][b] = 0
            if s["lse"] is not None:
                s["lse"][b] = float("-inf")
            continue
        pages = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
        k = s["k_pool"][pages].reshape(-1, nkv, d)[:n].float()
        v = s["v_pool"][pages].reshape(-1, nkv, d)[:n].float()
        q = s["q"][b:b + 1, :nq * d].float().view(1, nq, d)
        o, lse = _softmax_plain(q, k, v, nq // nkv, False)
        s["o"][b] = o.reshape(-1).to(s["o"].dtype)
        if s["lse"] is not None:
            s["lse"][b] = lse[:, 0]
    return (s["o"], s["lse"]) if c["lse"] else (s["o"],)


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append_plain, "packed": _packed_plain, "decode": _decode_plain}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        new, ctx = _new_and_ctx(c)
        live = sum(n for n, x in zip(new, ctx) if x >= 0)
        rows = live * (2 * nq + 5 * nkv) * d * es       # q, k, v in; q', k', cache k' and v out
        ids = 4 * (2 * len(new) + 1) + 4 * live
        return {"bytes": rows + ids + 4 * c["rot"] * live, "flops": 3 * live * (nq + nkv) * c["rot"]}
    lens = _lens(c)
    if c["op"] == "packed":
        pairs = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens)
        by = sum(lens) * (2 * nq + 2 * nkv) * d * es + (4 * nq * sum(lens) if c["lse"] else 0)
        return {"bytes": by, "flops": 4 * d * nq * pairs}
    n = sum(lens)
    by = 2 * n * nkv * d * es + len(lens) * (2 * nq * d * es + (4 * nq if c["lse"] else 0))
    return {"bytes": by + 4 * (n // c["page"] + 2 * len(lens)), "flops": 4 * d * nq * n}


# ------------------------------------------------------------------ 64-bit results
def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e11:
        return None
    s = _inputs(c, seed)
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    g = nq // nkv
    if c["op"] == "append":
        q_out, k_out = s["q_out"].double(), s["k_out"].double()
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        x = s["qkv"].double()
        new, ctx = _new_and_ctx(c)
        rot, at = c["rot"], 0
        for b, (n, start) in enumerate(zip(new, ctx)):
            if start >= 0:
                y = x[at:at + n].reshape(n, nq + 2 * nkv, d).clone()
                if rot:
                    th = s["rope"][start:start + n].double()
                    z = torch.complex(th[..., 0], th[..., 1])[:, None]
                    h = y[:, :nq + nkv, :rot]
                    h = h.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
                        h.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                    w = torch.view_as_real(torch.view_as_complex(h.contiguous()) * z)
                    y[:, :nq + nkv, :rot] = (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)
                q_out[at:at + n] = y[:, :nq].flatten(1)
                k_out[at:at + n] = y[:, nq:nq + nkv].flatten(1)
                p = torch.arange(start, start + n, device="cuda")
                rowp = s["table"][b].long()[p // c["page"]]
                kp[rowp, p % c["page"]] = y[:, nq:nq + nkv]
                vp[rowp, p % c["page"]] = y[:, nq + nkv:]
            at += n
        return q_out, k_out, kp, vp
    o = s["o"].double()
    lse = s["lse"].double() if c["lse"] else None
    at = 0
    for b, n in enumerate(_lens(c)):
        if c["op"] == "decode":
            if n == 0:
                if lse is not None:
                    lse[b] = float("-inf")
                continue
            p = torch.arange(n, device="cuda")
            where = s["table"][b].long()[p // c["page"]]
            k, v = (s[t][where, p % c["page"]].double() for t in ("k_pool", "v_pool"))
            q = s["q"][b:b + 1, :nq * d].double().reshape(1, nq, d)
        else:
            y = s["qkv"][at:at + n].double().reshape(n, nq + 2 * nkv, d)
            q, k, v = y[:, :nq], y[:, nq:nq + nkv], y[:, nq + nkv:]
        for h in range(nq):
            a = (q[:, h] @ k[:, h // g].T) / math.sqrt(d)
            if c["op"] == "packed" and c["causal"]:
                a = a + torch.triu(torch.full_like(a, float("-inf")), 1)
            z = torch.logsumexp(a, dim=1)
            r = torch.exp(a - z[:, None]) @ v[:, h // g]
            if c["op"] == "decode":
                o[b, h * d:(h + 1) * d] = r[0]
                if lse is not None:
                    lse[b, h] = z[0]
            else:
                o[at:at + n, h * d:(h + 1) * d] = r
                if lse is not None:
                    lse[h, at:at + n] = z
        at += n
    return (o, lse) if c["lse"] else (o,)
