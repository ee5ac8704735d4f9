"""Operators for several new tokens per sequence over a paged cache, and the
sizes they are measured at.

A program that drafts tokens and checks them in one step calls them one after
the other: `append` (the drafted tokens' keys and values enter the cache, rotated
by their depth in the tree), `tree` (attention of every drafted token over the
cached tokens, its ancestors and itself), `accept` (the accepted path of each
tree moves to the front of its slots) and, where a sequence goes on in more than
one way, `copy` (slots of pages to other pages).

A case names an operator and its sizes. Lengths and trees are drawn from the
case itself, values from the seed. With `own` false `run` computes the operators
in elementary float32 torch operations; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    gqa = dict(nq=32, nkv=8, d=128, dtype="bf16")   # the grouped-head layer of the benchmark
    mha = dict(nq=16, nkv=16, d=64, dtype="bf16")   # as many key heads, small ones
    return [
        # one user, a short history, a chain of five guesses; the plan is made in the pass
        dict(name="tree_one_chain", op="tree", **gqa, seqs=1, ctx_lo=77, ctx_hi=77, new_lo=5, new_hi=5,
             branch=0, page=16, head_major=False, pad=0, tail=0, lse=False, plan="made"),
        # one user with a very long document and a wide tree
        dict(name="tree_one_long", op="tree", **gqa, seqs=1, ctx_lo=130940, ctx_hi=130940, new_lo=61,
             new_hi=61, branch=3, page=64, head_major=False, pad=0, tail=0, lse=False, plan="kept"),
        # a serving batch of mixed histories, small trees of different sizes
        dict(name="tree_ragged", op="tree", **gqa, seqs=32, ctx_lo=33, ctx_hi=16000, new_lo=2, new_hi=24,
             branch=2, page=16, head_major=False, pad=3, tail=5, lse=True, plan="kept"),
        # many short histories, every query head with its own key head; the plan is made in the pass
        dict(name="tree_many_mha", op="tree", **mha, seqs=96, ctx_lo=20, ctx_hi=1200, new_lo=1, new_hi=8,
             branch=2, page=24, head_major=True, pad=0, tail=0, lse=False, plan="made"),
        # two prompts continue over what is cached of them, a piece of 256 tokens each
        dict(name="tree_prompt_pieces", op="tree", **gqa, seqs=2, ctx_lo=7000, ctx_hi=9000, new_lo=256,
             new_hi=256, branch=0, page=32, head_major=False, pad=0, tail=0, lse=True, plan="kept"),
        # float32 cache
        dict(name="tree_f32", op="tree", nq=16, nkv=4, d=128, dtype="f32", seqs=8, ctx_lo=5, ctx_hi=3000,
             new_lo=3, new_hi=20, branch=2, page=32, head_major=False, pad=1, tail=0, lse=True, plan="kept"),
        # the drafted tokens of a serving batch enter the cache
        dict(name="append_trees", op="append", **gqa, seqs=64, ctx_lo=33, ctx_hi=16000, new_lo=4, new_hi=61,
             branch=3, page=16, head_major=False, pad=0, tail=3, rot=128, interleaved=False),
        # one user, float32, a quarter of each head rotated in pairs: latency
        dict(name="append_one_f32", op="append", nq=16, nkv=4, d=64, dtype="f32", seqs=1, ctx_lo=4321,
             ctx_hi=4321, new_lo=7, new_hi=7, branch=2, page=32, head_major=True, pad=0, tail=0, rot=16,
             interleaved=True),
        # a path is accepted in each tree of a serving batch
        dict(name="accept_batch", op="accept", **gqa, seqs=200, ctx_lo=33, ctx_hi=4000, new_lo=8, new_hi=61,
             branch=2, page=16, head_major=False, pad=5, tail=0),
        # one user: latency
        dict(name="accept_one", op="accept", **gqa, seqs=1, ctx_lo=4321, ctx_hi=4321, new_lo=25, new_hi=25,
             branch=2, page=64, head_major=False, pad=0, tail=0),
        # one sequence goes on in four ways: its last page, half filled
        dict(name="copy_fork", op="copy", **gqa, copies=3, page=64, head_major=False, full=False),
        # long sequences move to other pages
        dict(name="copy_many", op="copy", **gqa, copies=1000, page=64, head_major=False, full=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "append", "accept", "copy"])
    nkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if nkv * group > 64:
        group = 64 // nkv
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    c = dict(op=op, nq=nkv * group, nkv=nkv, d=rng.choice([64, 128]), dtype=dtype,
             page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 128, 256]), head_major=rng.random() < 0.5)
    per_token = nkv * c["d"] * (2 if dtype == "bf16" else 4)      # half a cached token's bytes
    if op == "copy":
        room = int(1000 * 64 * 8 * 128 * 2 / per_token / c["page"])
        c.update(copies=_log_int(rng, 1, min(3000, room)), full=rng.random() < 0.5)
        return c
    seqs = _log_int(rng, 1, 200)
    new_hi = _log_int(rng, 1, min(256, max(1, 4000 // seqs)))
    room = int(130000 * 8 * 128 * 2 / per_token / seqs)           # as many bytes as the largest case
    ctx_hi = _log_int(rng, 1, max(1, min(room, 130900)))
    if op == "tree":                                              # .. and as many operations
        rate = 61 * 130000 * 32 * 128 if dtype == "bf16" else 8 * 10 * 1500 * 16 * 128 * 8
        while seqs * new_hi * (ctx_hi + new_hi) * c["nq"] * c["d"] > rate:
            if ctx_hi >= new_hi:
                ctx_hi = max(1, ctx_hi // 2)
            else:
                new_hi //= 2
    c.update(seqs=seqs, ctx_lo=_log_int(rng, 1, ctx_hi), ctx_hi=ctx_hi, new_lo=rng.randint(1, new_hi),
             new_hi=new_hi, branch=rng.choice([0, 1, 2, 3, 4]), pad=rng.choice([0, 0, 1, 4]),
             tail=rng.choice([0, 0, 1, 13]))
    if op == "tree":
        c.update(lse=rng.random() < 0.5, plan=rng.choice(["kept", "made"]))
    if op == "append":
        c.update(rot=rng.choice([0, 16, 32, 64, c["d"]]), interleaved=rng.random() < 0.4)
    return c


def _spread(n, lo, hi, salt):
    """n lengths between lo and hi (log-uniform), the same for every seed."""
    rng = random.Random(1000003 * n + 101 * lo + hi + 7919 * salt)
    return [int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1 for _ in range(n)]


def _batch(c):
    """Per sequence: drafted tokens, tokens cached before (-1: padding), and the
    parent of each drafted token in its sequence (-1: the last cached token)."""
    new = _spread(c["seqs"], c["new_lo"], c["new_hi"], 1) + [1] * c["pad"]
    ctx = _spread(c["seqs"], c["ctx_lo"], c["ctx_hi"], 2) + [-1] * c["pad"]
    rng = random.Random(31 * c["seqs"] + c["new_hi"])
    trees = []
    for n in new:
        if c["branch"] == 0:
            trees.append([i - 1 for i in range(n)])
        else:  # level by level, about `branch` children each
            trees.append([-1 if i == 0 else max(0, (i - 1) // c["branch"] - rng.randint(0, 1))
                          for i in range(n)])
    return new, ctx, trees


def _path(tree, i):
    out = []
    while i >= 0:
        out.append(i)
        i = tree[i]
    return out[::-1]


def _accepted(c):
    """The last token of the accepted path per sequence (-1: none), such that
    accepting it again changes nothing: every token of the path stays, or comes
    from behind the path. Where there is such a path of some tokens, not the first alone."""
    new, ctx, trees = _batch(c)
    rng = random.Random(17 * c["seqs"] + c["new_hi"])
    out = []
    for x, tree in zip(ctx, trees):
        pick = -1
        if x >= 0 and rng.random() < 0.9:
            for i in rng.sample(range(len(tree)), len(tree)):
                p = _path(tree, i)
                if all(a == k or a >= len(p) for k, a in enumerate(p)):
                    pick = i
                    if len(p) > 2 and p[-1] >= len(p):
                        break
        out.append(pick)
    return out


# ------------------------------------------------------------------ inputs
def _randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


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


def _pool(gen, c, n_pages):
    """[n_pages, page, nkv, d] view of a pool stored token-major or head-major."""
    dt = _DTYPES[c["dtype"]]
    if c["head_major"]:
        return _randn(gen, (n_pages, c["nkv"], c["page"], c["d"]), dt).transpose(1, 2)
    return _randn(gen, (n_pages, c["page"], c["nkv"], c["d"]), dt)


def _rope_rows(positions, rot, base=10000.0):
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    p = torch.arange(positions, device="cuda", dtype=torch.float64)
    a = p[:, None] * torch.exp(j * (-2.0 * math.log(base) / rot))[None, :]
    return torch.stack((torch.cos(a), torch.sin(a)), dim=-1).to(torch.float32).contiguous()


def _slots(c):
    """copy: slots per page."""
    if c["full"]:
        return [c["page"]] * c["copies"]
    rng = random.Random(c["copies"])
    return [rng.randint(min(c["page"], (c["page"] + 1) // 2), c["page"]) for _ in range(c["copies"])]


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1 + 7 * seed)
    dt = _DTYPES[c["dtype"]]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    s = {"case": c}
    if c["op"] == "copy":
        n_pages = 2 * c["copies"] + 5
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        # a fork's copies are of one page, moved pages are each their own
        s["src"] = order[:c["copies"]].contiguous() if c["full"] else order[:1].repeat(c["copies"])
        s["dst"] = order[c["copies"]:2 * c["copies"]].contiguous()
        s["slots"] = _ints(_slots(c))
        s["table"] = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        s["k_pool"], s["v_pool"] = (_pool(gen, c, n_pages) for _ in range(2))
        return s
    new, ctx, trees = _batch(c)
    lens = [n + x if x >= 0 else 0 for n, x in zip(new, ctx)]
    total = sum(new) + c["tail"]
    s["tokens"] = total
    s["cu"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    s["lens"] = _ints(lens)
    s["parents"] = _ints([p for t in trees for p in t] + [-1] * c["tail"]) if c["branch"] else None
    s["table"], n_pages = _pages(gen, c, lens)
    s["k_pool"], s["v_pool"] = (_pool(gen, c, n_pages) for _ in range(2))
    if c["op"] == "accept":
        s["leaf"] = _ints(_accepted(c))
        s["new_lens"] = torch.zeros(len(new), dtype=torch.int32, device="cuda")
        return s
    s["qkv"] = _randn(gen, (total, (nq + 2 * nkv) * d), dt, 1.5 if c["op"] == "tree" else 1.0)
    if c["op"] == "append":
        s["rope_len"] = max(1, max(lens))
        s["rope"] = _rope_rows(s["rope_len"], c["rot"]) if c["rot"] else None
        s["q_out"] = torch.zeros((total, nq * d), dtype=dt, device="cuda")
        s["k_out"] = torch.zeros((total, nkv * d), dtype=dt, device="cuda")
    else:
        s["o"] = torch.zeros((total, nq * d), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((total, nq), dtype=torch.float32, device="cuda") if c["lse"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    if c["op"] != "copy":
        # lengths and trees are the program's own: it laid the batch out
        s["host"] = _batch(c)
        if c["op"] == "accept":
            s["host_leaf"] = _accepted(c)
    if own:
        from megatron_transformer_layer_fwd_gb300 import mgb
        s["cache"] = mgb.kv_cache(s["k_pool"], s["v_pool"], s["table"])
        if c["op"] != "copy":
            s["ws"] = torch.empty(mgb.mgb_attention_tree_ws_bytes(
                s["lens"].numel(), s["tokens"], c["nq"], c["nkv"], c["d"]), dtype=torch.uint8, device="cuda")
            s["plan"] = _plan(s)
        if c["op"] == "append":
            s["desc"] = mgb.kv_append_desc(s["tokens"], s["lens"].numel(), c["nq"], c["rot"],
                                           c["interleaved"], s["rope_len"] if c["rot"] else 0)
    return s


# ------------------------------------------------------------------ the library's calls
def _plan(s):
    from megatron_transformer_layer_fwd_gb300 import mgb
    c = s["case"]
    return mgb.mgb_attention_tree_prepare(s["lens"].numel(), s["tokens"], c["nq"], c["nkv"], c["d"], s["cu"],
                                          s["lens"], s["parents"], s["ws"])


def _run_own(s):
    from megatron_transformer_layer_fwd_gb300 import mgb
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    w = (nq + 2 * nkv) * d
    if c["op"] == "tree":
        plan = _plan(s) if c["plan"] == "made" else s["plan"]
        mgb.mgb_attention_tree(plan, s["cache"], s["qkv"], w, s["o"], nq * d, s["lse"])
        return (s["o"], s["lse"]) if c["lse"] else (s["o"],)
    if c["op"] == "append":
        qkv = s["qkv"]
        mgb.mgb_kv_append_tree(s["plan"], s["desc"], s["cache"], s["rope"], qkv, qkv[:, nq * d:],
                               qkv[:, (nq + nkv) * d:], w, w, s["q_out"], nq * d, s["k_out"], nkv * d)
        return s["q_out"], s["k_out"], s["k_pool"], s["v_pool"]
    if c["op"] == "accept":
        mgb.mgb_kv_accept(s["plan"], s["cache"], s["leaf"], s["new_lens"])
        return s["new_lens"], s["k_pool"], s["v_pool"]
    mgb.mgb_kv_copy_pages(s["cache"], s["src"], s["dst"], s["slots"])
    return s["k_pool"], s["v_pool"]


# ------------------------------------------------------------------ plain forms
def _visible(parents, n, steps):
    """[n, n] whether token i of a tree descends from token j or is it, from its
    parents (None: a chain); no path is longer than `steps`."""
    i = torch.arange(n, device="cuda")
    if parents is None:
        return i[None, :] <= i[:, None]
    seen = i[None, :] == i[:, None]
    at = parents.long()
    for _ in range(steps):
        seen = seen | (at[:, None] == i[None, :])
        at = torch.where(at >= 0, parents.long()[at.clamp(min=0)], at)
    return seen


def _steps(c, tree):
    return 0 if c["branch"] == 0 else max(len(_path(tree, i)) for i in range(len(tree)))


def _tree_plain(s):
    c = s["case"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    g = nq // nkv
    at = 0
    for b, (n, x, tree) in enumerate(zip(*s["host"])):
        if x >= 0:
            seen = _visible(s["parents"][at:at + n] if c["branch"] else None, n, _steps(c, tree))
            pages = s["table"][b, :(x + n + c["page"] - 1) // c["page"]].long()
            k = s["k_pool"][pages].reshape(-1, nkv, d)[:x + n].float()
            v = s["v_pool"][pages].reshape(-1, nkv, d)[:x + n].float()
            q = s["qkv"][at:at + n, :nq * d].float().view(n, nq, d)
            # row n i + t: head i of the group, token t
            qh = q.permute(1, 0, 2).reshape(nkv, g * n, d)
            sc = torch.matmul(qh, k.permute(1, 2, 0)) * (1.0 / math.sqrt(d))
            hide = torch.cat((torch.zeros((n, x), dtype=torch.bool, device="cuda"), ~seen), dim=1)
            sc = sc.view(nkv, g, n, x + n).masked_fill(hide, float("-inf"))
            m = sc.amax(-1, keepdim=True)
            e = torch.exp(sc - m)
            z = e.sum(-1, keepdim=True)
            o = torch.matmul((e / z).view(nkv, g * n, -1), v.permute(1, 0, 2))
            s["o"][at:at + n] = o.view(nq, n, d).permute(1, 0, 2).reshape(n, nq * d).to(s["o"].dtype)
            if s["lse"] is not None:
                s["lse"][at:at + n] = (m + torch.log(z)).view(nq, n).T
        at += n
    return (s["o"], s["lse"]) if c["lse"] else (s["o"],)


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
    first, ctx = cu[seq], lens[seq] - (cu[seq + 1] - cu[seq])
    depth = t - first
    if c["branch"]:
        depth = torch.zeros_like(t)
        at = torch.where(s["parents"] >= 0, s["parents"].long() + first, -1)
        for _ in range(max(_steps(c, tree) for tree in s["host"][2])):
            depth += at >= 0
            up = s["parents"].long()[at.clamp(min=0)]
            at = torch.where((at >= 0) & (up >= 0), up + first, -1)
    ok = inside & (ctx >= 0)
    t, seq, slot, pos = t[ok], seq[ok], (ctx + t - first)[ok], (ctx + depth)[ok]
    x = s["qkv"][t].float().view(-1, nq + 2 * nkv, d)
    rows = s["rope"][pos] if c["rot"] else None
    q = _rotate_plain(x[:, :nq], rows, c)
    k = _rotate_plain(x[:, nq:nq + nkv], rows, c)
    dt = s["qkv"].dtype
    s["q_out"][t] = q.reshape(-1, nq * d).to(dt)
    s["k_out"][t] = k.reshape(-1, nkv * d).to(dt)
    page = s["table"].long()[seq, slot // c["page"]]
    s["k_pool"][page, slot % c["page"]] = k.to(dt)
    s["v_pool"][page, slot % c["page"]] = x[:, nq + nkv:].to(dt)
    return s["q_out"], s["k_out"], s["k_pool"], s["v_pool"]


def _accept_plain(s):
    c = s["case"]
    at = 0
    for b, (n, x, tree) in enumerate(zip(*s["host"])):
        leaf = s["host_leaf"][b]
        length = x
        if x >= 0 and leaf >= 0:
            seen = _visible(s["parents"][at:at + n] if c["branch"] else None, n, _steps(c, tree))
            path = torch.nonzero(seen[leaf]).flatten()
            length = x + path.numel()
            src, dst = x + path, torch.arange(x, length, device="cuda")
            row = s["table"][b].long()
            for pool in (s["k_pool"], s["v_pool"]):
                moved = pool[row[src // c["page"]], src % c["page"]]
                pool[row[dst // c["page"]], dst % c["page"]] = moved
        s["new_lens"][b] = max(0, length)
        at += n
    return s["new_lens"], s["k_pool"], s["v_pool"]


def _copy_plain(s):
    c = s["case"]
    i = torch.arange(c["page"], device="cuda")
    take = i[None, :] < s["slots"][:, None]
    src = s["src"].long()[:, None].expand_as(take)[take]
    dst = s["dst"].long()[:, None].expand_as(take)[take]
    slot = i[None, :].expand_as(take)[take]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[dst, slot] = pool[src, slot]
    return s["k_pool"], s["v_pool"]


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree_plain, "append": _append_plain, "accept": _accept_plain, "copy": _copy_plain}[
        state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "copy":
        return {"bytes": sum(_slots(c)) * 4 * nkv * d * es + 12 * c["copies"], "flops": 0}
    new, ctx, trees = _batch(c)
    ids = 4 * (2 * len(new) + 1) + (4 * sum(new) if c["branch"] else 0)
    if c["op"] == "accept":
        by = ids + 8 * len(new)
        for leaf, x, tree in zip(_accepted(c), ctx, trees):
            if x >= 0 and leaf >= 0:
                by += sum(a != k for k, a in enumerate(_path(tree, leaf))) * (4 * nkv * d * es + 8)
        return {"bytes": by, "flops": 0}
    if c["op"] == "append":
        live = sum(n for n, x in zip(new, ctx) if x >= 0)
        rows = live * (2 * nq + 5 * nkv) * d * es       # q, k, v in; q', k', cache k' and v out
        return {"bytes": rows + ids + 4 * live + 4 * c["rot"] * live, "flops": 3 * live * (nq + nkv) * c["rot"]}
    by, pairs = ids, 0
    for n, x, tree in zip(new, ctx, trees):
        if x >= 0:
            by += 2 * (x + n) * nkv * d * es + n * (2 * nq * d * es + (4 * nq if c["lse"] else 0))
            by += 4 * ((x + n) // c["page"] + 1)
            deep = []
            for i in range(n):
                deep.append(1 + (deep[tree[i]] if tree[i] >= 0 else 0))
            pairs += n * x + sum(deep)
    return {"bytes": by, "flops": 4 * d * nq * pairs}


# ------------------------------------------------------------------ 64-bit results
def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e11:
        return None
    s = _inputs(c, seed)
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    if c["op"] == "copy":
        for n, src, dst in zip(_slots(c), s["src"].tolist(), s["dst"].tolist()):
            kp[dst, :n] = s["k_pool"][src, :n].double()
            vp[dst, :n] = s["v_pool"][src, :n].double()
        return kp, vp
    new, ctx, trees = _batch(c)
    where = lambda b, p: (s["table"][b].long()[p // page], p % page)
    if c["op"] == "accept":
        lens = []
        for b, (x, tree, leaf) in enumerate(zip(ctx, trees, _accepted(c))):
            path = _path(tree, leaf) if x >= 0 else []
            for k, a in enumerate(path):
                (sp, si), (dp, di) = where(b, x + a), where(b, x + k)
                kp[dp, di] = s["k_pool"][sp, si].double()
                vp[dp, di] = s["v_pool"][sp, si].double()
            lens.append(max(0, x) + len(path))
        return _ints(lens), kp, vp
    at = 0
    if c["op"] == "append":
        q_out, k_out = s["q_out"].double(), s["k_out"].double()
        rot = c["rot"]
        for b, (n, x, tree) in enumerate(zip(new, ctx, trees)):
            if x >= 0:
                y = s["qkv"][at:at + n].double().reshape(n, nq + 2 * nkv, d).clone()
                if rot:
                    pos = torch.tensor([x + len(_path(tree, i)) - 1 for i in range(n)], device="cuda")
                    th = s["rope"][pos].double()
                    z = torch.complex(th[..., 0], th[..., 1])[:, None]
                    h = y[:, :nq + nkv, :rot]
                    h = h.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
                        h.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
                    w = torch.view_as_real(torch.view_as_complex(h.contiguous()) * z)
                    y[:, :nq + nkv, :rot] = (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)
                q_out[at:at + n] = y[:, :nq].flatten(1)
                k_out[at:at + n] = y[:, nq:nq + nkv].flatten(1)
                pg, i = where(b, torch.arange(x, x + n, device="cuda"))
                kp[pg, i] = y[:, nq:nq + nkv]
                vp[pg, i] = y[:, nq + nkv:]
            at += n
        return q_out, k_out, kp, vp
    o = s["o"].double()
    lse = s["lse"].double() if c["lse"] else None
    for b, (n, x, tree) in enumerate(zip(new, ctx, trees)):
        if x >= 0:
            pg, i = where(b, torch.arange(x + n, device="cuda"))
            k, v = kp[pg, i], vp[pg, i]
            off = torch.full((n, x + n), float("-inf"), dtype=torch.float64)
            off[:, :x] = 0
            for t in range(n):
                off[t, [x + a for a in _path(tree, t)]] = 0
            off = off.cuda()
            for h in range(nq):
                q = s["qkv"][at:at + n, h * d:(h + 1) * d].double()
                a = (q @ k[:, h // (nq // nkv)].T) / math.sqrt(d) + off
                z = torch.logsumexp(a, dim=1)
                o[at:at + n, h * d:(h + 1) * d] = torch.exp(a - z[:, None]) @ v[:, h // (nq // nkv)]
                if lse is not None:
                    lse[at:at + n, h] = z
        at += n
    return (o, lse) if c["lse"] else (o,)
