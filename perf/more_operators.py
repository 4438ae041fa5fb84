"""Drafted trees over the paged cache, and tokens under several adapters, as
measured workloads.

A server that drafts a tree of continuations per request and has the model
verify all of it in one step runs, beside what a plain step runs: the trees'
positions and ancestor masks (``tables``), attention in which a drafted token
sees the cache and its own ancestors (``attend``), and afterwards the walk
along the tokens that the model itself chose, with the pages past them given
back and the accepted tokens' keys and values moved to their places
(``verify``). Tokens under several adapters each, with a router's weights, are
sorted by adapter on the GPU, their rows copied out, and the adapters' results
brought back and added up (``route``), with the gradients of both
(``route_grad``). ``run`` computes each in plain torch operations, or, with
``own`` set, through the library.

Layouts: K and V caches [pages, kv_heads, page, head_dim] (a leading dimension
for the layers); block_table [requests, max_blocks]; a tree's parents are
indices into its request's new tokens; bit m of a token's mask words is its
request's new token m.
"""
import math
import random

import numpy as np
import torch

own = False

# Head layouts of this repository's layer workloads: the 7B layer is 4096
# wide with k/v as wide as q (32 heads of 128), the 70B slice is 8192 wide
# with k/v of 1024 (64 heads of 128 on 8).
HEADS_7B = {"heads": 32, "kv_heads": 32, "head_dim": 128}
HEADS_70B = {"heads": 64, "kv_heads": 8, "head_dim": 128}
VOCABULARY = 32000


def _tables(name, batch, lo, hi, ctx_lo, ctx_hi, lengths):
    """batch trees of lo..hi tokens behind ctx_lo..ctx_hi cached ones."""
    return {"name": name, "op": "tables", "batch": batch, "lo": lo, "hi": hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "lengths": lengths}


def _attend(name, layout, dtype, page, batch, lo, hi, ctx_lo, ctx_hi, lengths, window=0, sinks=0):
    return {"name": name, "op": "attend", **layout, "dtype": dtype, "page": page, "batch": batch, "lo": lo, "hi": hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lengths": lengths, "window": window, "sinks": sinks}


def _verify(name, layout, dtype, page, batch, lo, hi, ctx_lo, ctx_hi, layers, lengths):
    return {"name": name, "op": "verify", "kv_heads": layout["kv_heads"], "head_dim": layout["head_dim"], "dtype": dtype,
            "page": page, "batch": batch, "lo": lo, "hi": hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "layers": layers,
            "lengths": lengths}


def _route(name, op, tokens, choices, adapters, width, dtype, absent, base=False):
    """tokens rows of `width` with `choices` of `adapters` adapters each, a share `absent` of the choices being none;
    base: the results are added to the layer's own output."""
    return {"name": name, "op": op, "tokens": tokens, "choices": choices, "adapters": adapters, "width": width,
            "dtype": dtype, "absent": absent, "base": base}


def listed():
    return [
        # A verification step of the 64-request batch, trees of some 64 tokens.
        _tables("tables_64", 64, 26, 64, 128, 1024, 1),
        # Many requests with trees of all sizes, single tokens among them.
        _tables("tables_mixed", 512, 1, 256, 0, 4096, 2),
        # Trees over ragged contexts, 7B layer: every query head has its own keys.
        _attend("tree_7b", HEADS_7B, "bf16", 16, 64, 17, 64, 0, 2047, 3),
        # The largest: 128 requests of the 70B slice, trees of 64 tokens.
        _attend("tree_70b", HEADS_70B, "bf16", 64, 128, 64, 64, 127, 4095, 4),
        # One request with a long context: few rows, the work lies along the cache.
        _attend("tree_one", HEADS_70B, "bf16", 16, 1, 25, 25, 31000, 31000, 5),
        # Binary32, odd sizes, heads of 64 in groups of 5, a window and a few first tokens.
        _attend("tree_f32_window", {"heads": 10, "kv_heads": 2, "head_dim": 64}, "f32", 16, 3, 1, 13, 0, 700, 6,
                window=256, sinks=4),
        # The end of the 64-request step: tokens accepted, pages back, one layer's keys and values moved.
        _verify("verify_7b", HEADS_7B, "bf16", 16, 64, 26, 64, 0, 200, 1, 7),
        # 256 requests with trees of all sizes, eight layers of the 70B slice's cache at once.
        _verify("verify_70b", HEADS_70B, "bf16", 64, 256, 1, 128, 0, 200, 8, 8),
        # A decode step: 64 tokens, two of 64 adapters each.
        _route("route_decode", "route", 64, 2, 64, 4096, "bf16", 0.1),
        # A prefill batch of 8 prompts, four of a 2000-slot pool's adapters each, added to the layer's output.
        _route("route_prefill", "route", 4583, 4, 2000, 8192, "bf16", 0.05, base=True),
        # The router's training step over 7B-wide rows.
        _route("grad_7b", "route_grad", 4583, 2, 64, 4096, "bf16", 0.05),
        # Binary32, odd sizes.
        _route("grad_f32_odd", "route_grad", 517, 3, 7, 1000, "f32", 0.2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    lengths = rng.randrange(1 << 20)
    op = rng.choice(["tables", "attend", "attend", "attend", "verify", "route", "route", "route_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    head_dim = rng.choice([64, 80, 96, 128, 128, 128])
    kv_heads, group = rng.choice([(32, 1), (8, 8), (8, 4), (4, 5), (1, 8), (2, 7)])
    layout = {"heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim}
    hi = _log_int(rng, 1, 256)
    lo = rng.choice([1, max(1, hi // 2), hi])
    if op == "tables":
        c = _tables("", _log_int(rng, 1, 512), lo, hi, 0, _log_int(rng, 64, 4096), lengths)
    elif op == "verify":
        batch = _log_int(rng, 1, 256)
        c = _verify("", layout, dtype, page, batch, lo, min(hi, 128), 0, _log_int(rng, 8, 256),
                    rng.choice([1, 2, 8]) if batch <= 64 and kv_heads < 32 else 1, lengths)
        c["lo"] = min(c["lo"], c["hi"])
    elif op == "attend":
        batch = _log_int(rng, 1, 128)
        ctx_hi = _log_int(rng, 16, 32768 if batch <= 2 else 4096)
        window, sinks = (rng.choice([256, 300, 1024, 2000]), rng.choice([0, 1, 4, 30])) if rng.random() < 0.3 else (0, 0)
        c = _attend("", layout, dtype, page, batch, lo, hi, rng.choice([0, ctx_hi // 2]), ctx_hi, lengths, window, sinks)
        most = next(x for x in listed() if x["name"] == "tree_70b")

        def cost(x):  # of the padded plain form; binary32 products are ten times as dear
            return (x["batch"] * x["hi"] * (x["ctx_hi"] + x["hi"]) * x["heads"] * x["head_dim"]
                    * (8 if x["dtype"] == "f32" else 1))
        while cost(c) > cost(most) and c["batch"] > 1:
            c["batch"] = (c["batch"] + 1) // 2
        while cost(c) > cost(most):
            c["ctx_hi"], c["ctx_lo"] = c["ctx_hi"] // 2, c["ctx_lo"] // 2
    else:
        tokens, choices = _log_int(rng, 1, 8192), rng.choice([1, 2, 3, 4, 6, 8])
        adapters = max(choices, _log_int(rng, 1, 2000))
        width = 8 * _log_int(rng, 8, 1024)
        size = 2 if dtype == "bf16" else 4
        most = 4583 * 4 * 8192 * 2 if op == "route" else 4583 * 2 * 4096 * 2
        c = _route("", op, max(1, min(tokens, most // (choices * width * size))), choices, adapters, width, dtype,
                   rng.choice([0.0, 0.05, 0.3]), op == "route" and rng.random() < 0.5)
    del c["name"]
    return c


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tree(n, rng):
    """Parents of a tree of n tokens, level after level: the first is the root, and a level's tokens hang on the level
    before in order."""
    parent = np.full(n, -1, np.int32)
    level = max(1, round((n - 1) / rng.integers(3, 9)))
    before, at, width = 0, 1, 1
    while at < n:
        take = min(level, n - at)
        parent[at:at + take] = before + np.sort(rng.integers(0, width, take))
        before, at, width = at, at + take, take
    return parent


def _shape(case):
    """(trees, cached lengths) of the batch: the same for every seed."""
    r = np.random.default_rng(case["lengths"])
    new = r.integers(case["lo"], case["hi"] + 1, case["batch"])
    ctx = r.integers(case["ctx_lo"], case["ctx_hi"] + 1, case["batch"])
    return [_tree(int(n), r) for n in new], [int(c) for c in ctx]


def _depths(parent):
    depth = np.zeros(len(parent), np.int64)
    for i in range(1, len(parent)):
        depth[i] = depth[parent[i]] + 1 if parent[i] >= 0 else 0
    return depth


def _int32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _pages(lengths, page):
    return [-(-n // page) for n in lengths]


def _random_blocks(counts, rng, extra_pages=0):
    """A block table whose rows hold `counts` pages each, drawn from a shuffled
    pool; entries past a row's count are -1. Returns (table, left-over pages)."""
    total = sum(counts) + extra_pages
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(counts), max(1, max(counts))), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:]


def _starts(trees):
    return np.concatenate([[0], np.cumsum([len(p) for p in trees])])


def _words(case):
    return -(-case["hi"] // 32)


def _prepare_tables(case, seed):
    rng = np.random.default_rng(seed)
    trees, ctx = _shape(case)
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, len(ctx))
    parent = np.concatenate(trees)
    return {"parent": _int32(parent), "q_start": _int32(_starts(trees)), "kv_len": _int32([c + len(p) for c, p in zip(ctx, trees)]),
            "position": _int32(np.zeros(len(parent))), "mask": _int32(np.zeros((len(parent), _words(case))))}


def _ancestors(trees, words):
    """Mask words [T, words] on the host."""
    out = np.zeros((sum(map(len, trees)), words), np.uint32)
    at = 0
    for parent in trees:
        for i, p in enumerate(parent):
            if p >= 0:
                out[at + i] = out[at + p]
            out[at + i, i // 32] |= np.uint32(1 << (i % 32))
        at += len(parent)
    return out.view(np.int32)


def _prepare_attend(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, page = DTYPES[case["dtype"]], case["page"]
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    trees, ctx = _shape(case)
    kv = [len(p) + c for p, c in zip(trees, ctx)]
    table, _ = _random_blocks(_pages(kv, page), rng)
    num_pages, n = sum(_pages(kv, page)), sum(map(len, trees))
    fused = torch.randn(n, (hq + 2 * hk) * d, generator=gen, device="cuda").to(dtype)
    K = torch.randn(num_pages, hk, page, d, generator=gen, device="cuda", dtype=dtype)
    V = torch.randn(num_pages, hk, page, d, generator=gen, device="cuda", dtype=dtype)
    return {"q": fused[:, :hq * d].view(n, hq, d), "K": K, "V": V, "block_table": torch.from_numpy(table).cuda(),
            "q_start": _int32(_starts(trees)), "kv_len": _int32(kv), "max_q_len": max(map(len, trees)),
            "mask": torch.from_numpy(_ancestors(trees, _words(case))).cuda(), "scale": d ** -0.5,
            "window": case["window"], "sinks": case["sinks"],
            "out": torch.empty(n, hq, d, dtype=dtype, device="cuda"),
            "lse": torch.empty(n, hq, dtype=torch.float32, device="cuda")}


def _accepted_path(parent, rng):
    """The tokens from the root to a random one, cut so that none is moved to the place of another accepted one: a
    second pass over the same state then moves the same rows again."""
    path, i = [], int(rng.integers(0, len(parent)))
    while i >= 0:
        path.append(i)
        i = int(parent[i])
    path = path[::-1]
    while any(p != d and p < len(path) for d, p in enumerate(path)):
        path.pop()
    return path


def _prepare_verify(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, page = DTYPES[case["dtype"]], case["page"]
    trees, ctx = _shape(case)
    start = _starts(trees)
    refused = case["lengths"] % len(trees) if len(trees) > 8 else -1  # a request that the pool had no pages for
    kv = [c + (len(p) if b != refused else 0) for b, (p, c) in enumerate(zip(trees, ctx))]
    token = rng.integers(0, VOCABULARY, int(start[-1])).astype(np.int32)
    target = rng.integers(VOCABULARY, 2 * VOCABULARY, int(start[-1])).astype(np.int32)  # not drafted, but:
    free = 17 + case["lengths"] % 200
    table, left = _random_blocks(_pages(kv, page), rng, free + 8)  # 8 that requests outside this step hold
    num_pages = sum(_pages(kv, page)) + free + 8
    slot = np.full(int(start[-1]), -1, np.int32)
    for b, parent in enumerate(trees):
        path = _accepted_path(parent, rng)
        for i, j in zip(path, path[1:]):
            target[start[b] + i] = token[start[b] + j]
        if b != refused:
            at = ctx[b] + np.arange(len(parent))
            slot[start[b]:start[b + 1]] = table[b, at // page] * page + at % page
    head = int(rng.integers(0, num_pages))
    ring = np.full(num_pages, -1, np.int32)
    ring[(head + np.arange(free)) % num_pages] = left[:free]
    K, V = (torch.randn(case["layers"], num_pages, case["kv_heads"], page, case["head_dim"], generator=gen, device="cuda",
                        dtype=dtype) for _ in range(2))
    T, B = int(start[-1]), len(trees)
    return {"parent": _int32(np.concatenate(trees)), "token": _int32(token), "target": _int32(target), "slot": _int32(slot),
            "q_start": _int32(start), "kv_len": _int32(kv), "page": page, "block_table": torch.from_numpy(table).cuda(),
            "free_pages": torch.from_numpy(ring).cuda(), "pool_in": _int32([head, free, 0, T]),
            "pool_out": _int32([0] * 4), "path": _int32(np.zeros(T)), "accepted": _int32(np.zeros(B)),
            "next_token": _int32(np.zeros(B)), "kept_len": _int32(np.zeros(B)), "K": K, "V": V}


def _choices(case, rng):
    """Distinct adapters per token, some far more popular than others; absent ones are -1."""
    T, k, P = case["tokens"], case["choices"], case["adapters"]
    score = np.log(np.arange(1, P + 1) ** -0.8)[rng.permutation(P)] + rng.gumbel(size=(T, P))
    ids = np.argpartition(-score, k - 1, axis=1)[:, :k].astype(np.int32) if k < P else np.tile(np.arange(P, dtype=np.int32), (T, 1))
    ids = rng.permuted(ids, axis=1)
    ids[rng.random((T, k)) < case["absent"]] = -1
    return ids


def _prepare_route(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, T, k, P, d = DTYPES[case["dtype"]], case["tokens"], case["choices"], case["adapters"], case["width"]

    def rows(n):
        return torch.randn(n, d, generator=gen, device="cuda").to(dtype)

    choice = _choices(case, rng)
    weight = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), 1)
    if case["op"] == "route":
        S = min(P, T * k)
        return {"choice": torch.from_numpy(choice).cuda(), "adapters": P, "X": rows(T), "Ys": rows(T * k), "weight": weight,
                "base": rows(T) if case["base"] else None, "seg_start": _int32(np.zeros(S + 1)), "seg_adapter": _int32(np.zeros(S)),
                "order": _int32(np.zeros(T * k)), "place": _int32(np.zeros((T, k))), "Xs": rows(T * k), "Y": rows(T)}
    order = np.argsort(np.where(choice.reshape(-1) < 0, P, choice.reshape(-1)), kind="stable")
    place = np.empty(T * k, np.int32)
    place[order] = np.arange(T * k)
    place[choice.reshape(-1) < 0] = -1
    return {"place": _int32(place.reshape(T, k)), "weight": weight, "Ys": rows(T * k), "dY": rows(T), "dXs": rows(T * k),
            "dYs": rows(T * k), "dweight": torch.empty(T, k, device="cuda"), "dX": rows(T)}


def prepare(case, seed):
    make = {"tables": _prepare_tables, "attend": _prepare_attend, "verify": _prepare_verify, "route": _prepare_route,
            "route_grad": _prepare_route}[case["op"]]
    return {"op": case["op"], **make(case, seed)}


def _plain_tables(s):
    parent, start = s["parent"].long(), s["q_start"].long()
    T, words = s["mask"].shape
    row = torch.arange(T, device=parent.device)
    of = torch.searchsorted(start, row, right=True) - 1
    at = row - start[of]
    seen = torch.zeros(T, words * 32, dtype=torch.bool, device=parent.device)
    up = torch.where((parent >= 0) & (parent < at), parent, -1)  # this token's ancestor, one level further each time
    depth = torch.full_like(row, -1)
    now = at
    for _ in range(words * 32):
        live = now >= 0
        if not bool(live.any()):
            break
        seen.scatter_(1, now.clamp(min=0)[:, None], seen.gather(1, now.clamp(min=0)[:, None]) | live[:, None])
        depth += live
        now = torch.where(live, up[start[of] + now.clamp(min=0)], -1)
    bit = torch.arange(32, device=parent.device)
    word = (seen.view(T, words, 32).long() << bit).sum(-1)
    s["mask"].copy_(torch.where(word >= 1 << 31, word - (1 << 32), word))
    s["position"].copy_(s["kv_len"].long()[of] - (start[1:] - start[:-1])[of] + depth)
    return {"position": s["position"], "mask": s["mask"]}


def _plain_attend(s):
    q, K, V, table = s["q"], s["K"], s["V"], s["block_table"]
    batch, page, hk, d = table.shape[0], K.shape[2], K.shape[1], K.shape[3]
    hq, nq, nk = q.shape[1], s["max_q_len"], table.shape[1] * K.shape[2]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    row = torch.arange(nq, device=q.device)
    token = (start[:-1, None] + row).clamp(max=q.shape[0] - 1)
    group = hq // hk
    # queries [batch, hk, group * nq, d], keys and values [batch, hk, nk, d], padded to the longest
    qs = q[token].float().view(batch, nq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, group * nq, d)
    blocks = table.long().clamp(min=0)
    key = torch.arange(nk, device=q.device)
    ks = K[blocks].float().permute(0, 2, 4, 1, 3).reshape(batch, hk, d, nk).contiguous()
    score = torch.matmul(qs, ks).mul_(s["scale"]).view(batch, hk, group, nq, nk)
    del ks
    bits = ((s["mask"][token].long()[..., None] >> torch.arange(32, device=q.device)) & 1).bool().flatten(2)
    cached = (kv - n)[:, None, None]
    drafted = key - cached  # of the request's new tokens, where not negative
    seen = drafted < 0
    if s["window"] > 0:
        pos = (kv - n)[:, None] + bits.sum(-1) - 1
        seen = seen & ((key > pos[..., None] - s["window"]) | (key < s["sinks"]))
    inside = (drafted >= 0) & (drafted < n[:, None, None])
    at = drafted.clamp(0, bits.shape[-1] - 1).expand(batch, nq, nk)
    seen = seen | (inside & bits.gather(2, at))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(top.clamp(min=-3e38)).exp_()
    total = score.sum(-1, keepdim=True)
    vs = V[blocks].float().permute(0, 2, 1, 3, 4).reshape(batch, hk, nk, d)
    vs.mul_((key < kv[:, None])[:, None, :, None])
    out = torch.matmul(score.view(batch, hk, group * nq, nk), vs).view(batch, hk, group, nq, d)
    out = out / total.clamp(min=1e-38)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    real = torch.nonzero((row < n[:, None]).view(-1)).view(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch * nq, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(batch * nq, hq)
    s["out"].copy_(out[real])
    s["lse"].copy_(lse[real])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_verify(s):
    parent, token, target, slot = s["parent"].long(), s["token"], s["target"], s["slot"].long()
    start, kv, page, ring = s["q_start"].long(), s["kv_len"].long(), s["page"], s["free_pages"]
    T, B, pages = parent.numel(), kv.numel(), ring.numel()
    n = start[1:] - start[:-1]
    row = torch.arange(T, device=parent.device)
    of = torch.searchsorted(start, row, right=True) - 1
    live = (n > 0) & (slot[start[:-1].clamp(max=T - 1)] >= 0)
    served = live.clone()  # the others have no slots: nothing of them is accepted
    cur = torch.zeros_like(kv)
    path = torch.full_like(row, -1)
    accepted, last = torch.zeros_like(kv), torch.full_like(kv, -1)
    for depth in range(int(n.max())):
        if not bool(live.any()):
            break
        path = torch.where((row - start[of] == depth) & live[of], cur[of], path)
        accepted += live
        chosen = target[(start[:-1] + cur).clamp(max=T - 1)]
        last = torch.where(live, chosen.long(), last)
        child = live[of] & (parent == cur[of]) & (token == chosen[of]) & (row - start[of] > parent)
        nxt = torch.full_like(kv, T).scatter_reduce(0, of, torch.where(child, row - start[of], T), "amin")
        live = live & (nxt < T)
        cur = torch.where(live, nxt, cur)
    kept = torch.where(served, kv - n + accepted, kv)
    back = (kv + page - 1) // page - (kept + page - 1) // page
    upto = back.cumsum(0)
    first, width = (kept + page - 1) // page, s["block_table"].shape[1]
    column = torch.arange(width, device=parent.device)
    mine = (column >= first[:, None]) & (column < (first + back)[:, None])
    rank = (upto - back)[:, None] + column - first[:, None]
    head, count = s["pool_in"][0].long(), s["pool_in"][1].long()
    wide = torch.cat([ring, ring[:1]])
    wide.scatter_(0, torch.where(mine, (head + count + rank) % pages, pages).view(-1), s["block_table"].view(-1))
    ring.copy_(wide[:pages])
    s["pool_out"].copy_(torch.stack([head, count + back.sum(), s["pool_in"][2].long(), s["pool_in"][3].long()]))
    for name, x in (("path", path), ("accepted", accepted), ("next_token", last), ("kept_len", kept)):
        s[name].copy_(x)
    moved = torch.nonzero((path >= 0) & (path != row - start[of])).view(-1)
    src, dst = slot[start[of[moved]] + path[moved]], slot[moved]
    for c in (s["K"], s["V"]):
        c[:, dst // page, :, dst % page] = c[:, src // page, :, src % page]
    return {k: s[k] for k in ("path", "accepted", "next_token", "kept_len", "pool_out", "free_pages", "K", "V")}


def _weighted(rows, place, weight, base):
    total = torch.zeros(place.shape[0], rows.shape[1], device=rows.device) if base is None else base.float()
    for j in range(place.shape[1]):
        at = place[:, j].long()
        x = rows[at.clamp(min=0)].float()
        x = x if weight is None else x * weight[:, j, None]
        total = total + torch.where(at[:, None] >= 0, x, 0.0)
    return total


def _plain_route(s):
    choice, P = s["choice"], s["adapters"]
    T, k = choice.shape
    flat = choice.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < P), flat, P)
    order = torch.argsort(flat, stable=True)
    valid = (flat < P).sum()
    where = torch.arange(T * k, device=flat.device)
    place = torch.empty_like(flat)
    place[order] = where
    s["place"].copy_(torch.where(flat < P, place, -1).view(T, k))
    s["order"].copy_(torch.where(where < valid, order, -1))
    ends = (flat[None, :] < torch.arange(1, P + 1, device=flat.device)[:, None]).sum(1) if P * T * k < 1 << 24 else \
        torch.searchsorted(flat[order].contiguous(), torch.arange(1, P + 1, device=flat.device))
    size = torch.diff(ends, prepend=ends.new_zeros(1))
    used = torch.cumsum(size > 0, 0)
    S = s["seg_adapter"].numel()
    to = torch.where(size > 0, used - 1, S)
    start = torch.full((S + 2,), 0, dtype=torch.long, device=flat.device)
    start[:] = valid
    start.scatter_(0, torch.where(size > 0, used - 1, S + 1), ends - size)
    adapter = torch.zeros(S + 1, dtype=torch.long, device=flat.device)
    adapter.scatter_(0, to, torch.arange(P, device=flat.device))
    start[S] = valid
    s["seg_start"].copy_(start[:S + 1])
    s["seg_adapter"].copy_(adapter[:S])
    at = s["order"].long()
    s["Xs"].copy_(torch.where(at[:, None] >= 0, s["X"][at.clamp(min=0) // k], s["Xs"]))
    s["Y"].copy_(_weighted(s["Ys"], s["place"], s["weight"], s["base"]))
    return {k: s[k] for k in ("seg_start", "seg_adapter", "order", "place", "Xs", "Y")}


def _plain_route_grad(s):
    place, weight, dY = s["place"], s["weight"], s["dY"].float()
    for j in range(place.shape[1]):
        at = place[:, j].long()
        has = at >= 0
        dots = (dY * s["Ys"][at.clamp(min=0)].float()).sum(1)
        s["dweight"][:, j] = torch.where(has, dots, 0.0)
        t = torch.nonzero(has).view(-1)
        s["dYs"][at[t]] = (dY[t] * weight[t, j, None]).to(s["dYs"].dtype)
    s["dX"].copy_(_weighted(s["dXs"], place, None, None))
    return {k: s[k] for k in ("dYs", "dweight", "dX")}


def run(s):
    if not own:
        return {"tables": _plain_tables, "attend": _plain_attend, "verify": _plain_verify, "route": _plain_route,
                "route_grad": _plain_route_grad}[s["op"]](s)
    import segmented_gather_gemm_sgmv_amd as sg
    if s["op"] == "tables":
        sg.sgmv_tree_tables(s["parent"], s["q_start"], s["kv_len"], s["position"], s["mask"])
        return {"position": s["position"], "mask": s["mask"]}
    if s["op"] == "attend":
        sg.sgmv_tree_attention(s["out"], s["q"], s["K"], s["V"], s["block_table"], s["q_start"], s["kv_len"], s["mask"],
                               s["scale"], s["max_q_len"], window=s["window"], sinks=s["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "verify":
        sg.sgmv_tree_accept(s["parent"], s["token"], s["target"], s["slot"], s["q_start"], s["kv_len"], s["page"],
                            s["block_table"], s["free_pages"], s["pool_in"], s["pool_out"], s["path"], s["accepted"],
                            s["next_token"], s["kept_len"])
        sg.sgmv_kv_commit(s["K"], s["V"], s["slot"], s["q_start"], s["path"])
        return {k: s[k] for k in ("path", "accepted", "next_token", "kept_len", "pool_out", "free_pages", "K", "V")}
    if s["op"] == "route":
        sg.sgmv_sort_tokens(s["choice"], s["adapters"], s["seg_start"], s["seg_adapter"], s["order"], s["place"])
        sg.sgmv_spread_rows(s["Xs"], s["X"], s["place"])
        sg.sgmv_combine_rows(s["Y"], s["Ys"], s["place"], s["weight"], base=s["base"])
        return {k: s[k] for k in ("seg_start", "seg_adapter", "order", "place", "Xs", "Y")}
    sg.sgmv_combine_rows_grad(s["dYs"], s["dweight"], s["dY"], s["Ys"], s["place"], s["weight"])
    sg.sgmv_combine_rows(s["dX"], s["dXs"], s["place"])
    return {k: s[k] for k in ("dYs", "dweight", "dX")}


def work(case):
    if case["op"] in ("route", "route_grad"):
        T, k, d, size = case["tokens"], case["choices"], case["width"], 2 if case["dtype"] == "bf16" else 4
        N = int(round(T * k * (1 - case["absent"])))
        if case["op"] == "route":
            rows = T + N + N + T + (T if case["base"] else 0)
            return {"bytes": size * d * rows + 4 * (4 * T * k + 2 * min(case["adapters"], T * k)), "flops": 2 * N * d}
        return {"bytes": size * d * (T + 2 * N + N + T) + 4 * 3 * T * k, "flops": 4 * N * d}
    trees, ctx = _shape(case)
    T, B = sum(map(len, trees)), len(trees)
    if case["op"] == "tables":
        return {"bytes": 4 * (T * (2 + _words(case)) + 2 * B + 1), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "verify":
        # the accepted tokens are the tree's depth at most: half of that moves
        moved = sum(int(_depths(p).max()) for p in trees) // 2
        return {"bytes": 4 * (5 * T + 7 * B) + 4 * moved * case["layers"] * case["kv_heads"] * case["head_dim"] * size,
                "flops": 0}
    hq, hk, d, window = case["heads"], case["kv_heads"], case["head_dim"], case["window"]
    keys = pairs = 0
    for parent, c in zip(trees, ctx):
        depth = _depths(parent)
        first = np.maximum(c + depth - window + 1, 0) if window else np.zeros(len(parent), np.int64)
        first = np.minimum(first, c)
        sunk = np.minimum(first, case["sinks"])
        keys += c - int(first.min()) + int(sunk.min()) + len(parent)
        pairs += int((c - first + sunk + depth + 1).sum())
    tables = 4 * (2 * B + 1 + keys // case["page"] + T * _words(case))
    return {"bytes": 2 * size * hk * d * keys + T * hq * (2 * size * d + 4) + tables, "flops": 4 * hq * d * pairs}


def _exact_attend(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    trees, ctx = _shape(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (parent, c) in enumerate(zip(trees, ctx)):
        n = len(parent)
        pages = s["block_table"][b, :_pages([n + c], case["page"])[0]].long()
        k, v = (x[pages].double().transpose(0, 1).reshape(hk, -1, d)[:, :n + c] for x in (s["K"], s["V"]))
        hidden = np.zeros((n, n + c), bool)
        hidden[:, c:] = True
        depth = _depths(parent)
        for i in range(n):
            if case["window"]:
                hidden[i, case["sinks"]:max(0, c + depth[i] - case["window"] + 1)] = True
            j = i
            while j >= 0:
                hidden[i, c + j] = False
                j = parent[j]
        hidden = torch.from_numpy(hidden).cuda()
        step = max(1, (1 << 27) // max(1, n * (n + c)))  # heads at a time
        for h in range(0, hq, step):
            heads = torch.arange(h, min(hq, h + step), device="cuda")
            kk, vv = k[heads // (hq // hk)], v[heads // (hq // hk)]
            score = s["q"][at:at + n, heads].double().transpose(0, 1).contiguous() @ kk.transpose(1, 2).contiguous()
            score = (score * d ** -0.5).masked_fill(hidden, -math.inf)
            lse[at:at + n, heads] = torch.logsumexp(score, -1).T
            out[at:at + n, heads] = (torch.softmax(score, -1) @ vv.contiguous()).transpose(0, 1)
        at += n
    return {"out": out, "lse": lse}


def _exact_verify(case, seed):
    """The cache's rows after the moves; the whole numbers have no other value than the plain form's."""
    s = prepare(case, seed)
    K, V = s["K"].clone(), s["V"].clone()
    parent, token, target, slot, start = (s[k].tolist() for k in ("parent", "token", "target", "slot", "q_start"))
    page = case["page"]
    src, dst = [], []
    for q0, q1 in zip(start, start[1:]):
        if slot[q0] < 0:
            continue
        cur, depth = 0, 0
        while cur is not None:
            if cur != depth:
                src.append(slot[q0 + cur])
                dst.append(slot[q0 + depth])
            cur = next((j for j in range(cur + 1, q1 - q0) if parent[q0 + j] == cur and token[q0 + j] == target[q0 + cur]), None)
            depth += 1
    for x, old in ((K, s["K"]), (V, s["V"])):
        for i, j in zip(src, dst):
            x[:, j // page, :, j % page] = old[:, i // page, :, i % page]
    return {"path": None, "accepted": None, "next_token": None, "kept_len": None, "pool_out": None, "free_pages": None,
            "K": K.double(), "V": V.double()}


def _exact_route(case, seed):
    s = prepare(case, seed)
    T, k = case["tokens"], case["choices"]
    if case["op"] == "route":
        choice = s["choice"].cpu().numpy().reshape(-1)
        order = [i for _, i in sorted((c, i) for i, c in enumerate(choice) if c >= 0)]
        place = np.full(T * k, -1)
        place[order] = np.arange(len(order))
        Xs = s["Xs"].double()
        Xs[:len(order)] = s["X"].double()[torch.tensor(order, device="cuda") // k]
        place = torch.from_numpy(place.reshape(T, k)).cuda()
        zero = torch.zeros(1, case["width"], dtype=torch.float64, device="cuda")
        Y = torch.zeros(T, case["width"], dtype=torch.float64, device="cuda") if s["base"] is None else s["base"].double()
        rows = torch.cat([s["Ys"].double(), zero])  # an absent choice's index, -1, is the row of zeros
        for j in range(k):
            Y += s["weight"][:, j, None].double() * rows[place[:, j]]
        return {"seg_start": None, "seg_adapter": None, "order": None, "place": None, "Xs": Xs, "Y": Y}
    place = s["place"].long()
    dYs, dweight = s["dYs"].double(), torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dX = torch.zeros(T, case["width"], dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(place[:, j] >= 0).view(-1)
        at = place[t, j]
        dYs[at] = s["weight"][t, j, None].double() * s["dY"][t].double()
        dweight[t, j] = (s["dY"][t].double() * s["Ys"][at].double()).sum(1)
        dX[t] += s["dXs"][at].double()
    return {"dYs": dYs, "dweight": dweight, "dX": dX}


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    return {"attend": _exact_attend, "verify": _exact_verify}.get(case["op"], _exact_route)(case, seed)
