"""The paged key/value-cache operators as measured workloads.

A multi-LoRA server runs, between the q/k/v projections and the o projection
of a layer (the projections whose adapters SGMV applies), four things: it
gives the step's tokens their cache slots, it rotates q and k and writes k
and v to the cache, and the step's queries attend to the cache, over all of
it or over a window with a few first tokens. ``run`` computes each of them
in plain torch operations, or, with ``own`` set, through the library.

Layouts: K and V caches [pages, kv_heads, page, head_dim]; block_table
[requests, max_blocks]; q, k, v rows are slices of one fused projection
output, so their row stride is that of the fused row.
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


def _tables(name, batch, new_lo, new_hi, ctx_lo, ctx_hi, page, ended, free_share, lengths):
    return {"name": name, "op": "tables", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "page": page, "ended": ended, "free_share": free_share, "lengths": lengths}


def _append(name, tokens, layout, dtype, page, rot_dim, interleaved, base, scaling, max_position):
    return {"name": name, "op": "append", "tokens": tokens, **layout, "dtype": dtype, "page": page,
            "rot_dim": rot_dim, "interleaved": interleaved, "base": base, "scaling": scaling,
            "max_position": max_position}


def _attend(name, layout, dtype, page, batch, new_lo, new_hi, ctx_lo, ctx_hi, lengths, singles=0, window=0, sinks=0):
    """batch requests with new_lo..new_hi new tokens each behind ctx_lo..ctx_hi
    cached ones; the first `singles` of them add one token only."""
    return {"name": name, "op": "attend", **layout, "dtype": dtype, "page": page, "batch": batch, "new_lo": new_lo,
            "new_hi": new_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "lengths": lengths, "singles": singles,
            "window": window, "sinks": sinks}


def listed():
    return [
        # A decode step of the 64-request batch: one token each, a few need a new page.
        _tables("tables_decode", 64, 1, 1, 128, 1024, 16, 0.0, 1.0, 1),
        # A busy scheduler's step: 512 requests, prompt chunks and single tokens mixed, ended requests
        # giving their pages back, and a pool too small for the last ones.
        _tables("tables_mixed", 512, 1, 256, 0, 4096, 16, 0.1, 0.9, 2),
        # The decode step's rotation and cache write, 7B layer.
        _append("append_decode_7b", 64, HEADS_7B, "bf16", 16, 128, False, 10000.0, 1.0, 4096),
        # A prefill batch of 8 prompts of some 570 tokens, 70B layer, positions scaled for a long context.
        _append("append_prefill_70b", 4583, HEADS_70B, "bf16", 64, 128, False, 500000.0, 8.0, 131072),
        # Decode, one query head per cached head, ragged contexts, 7B layer.
        _attend("decode_7b", HEADS_7B, "bf16", 16, 64, 1, 1, 0, 2047, 3),
        # The largest decode: 512 requests of the 70B slice.
        _attend("decode_70b", HEADS_70B, "bf16", 64, 512, 1, 1, 127, 4095, 4),
        # One request with a long context: few rows, the work lies along the cache.
        _attend("decode_long", HEADS_70B, "bf16", 16, 1, 1, 1, 131000, 131000, 5),
        # Prefill: 8 prompts' chunks of 128..1024 tokens (the prefill workload), part of each cached before.
        _attend("chunk_70b", HEADS_70B, "bf16", 64, 8, 128, 1024, 0, 4096, 6),
        # A step that mixes 48 decodes with 4 prompt chunks, 7B layer.
        _attend("mixed_7b", HEADS_7B, "bf16", 16, 52, 100, 512, 1, 1500, 7, singles=48),
        # Binary32, odd sizes, heads of 64 in groups of 5, a few tokens per request.
        _attend("chunk_f32_small", {"heads": 10, "kv_heads": 2, "head_dim": 64}, "f32", 16, 3, 1, 7, 0, 200, 8),
        # Window and sinks: decode far into the context, and a long prompt's chunks.
        _attend("window_decode_7b", HEADS_7B, "bf16", 16, 64, 1, 1, 2000, 8191, 9, window=1024, sinks=4),
        _attend("window_chunk_70b", HEADS_70B, "bf16", 64, 2, 2048, 2048, 2048, 6144, 10, window=1024, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    lengths = rng.randrange(1 << 20)
    op = rng.choice(["tables", "append", "attend", "attend", "window"])
    if op == "tables":
        batch = _log_int(rng, 1, 512)
        c = _tables("", batch, 1, _log_int(rng, 1, 256), 0, _log_int(rng, 64, 4096), page, rng.choice([0.0, 0.1, 0.3]),
                    rng.choice([1.0, 1.0, 0.8]), lengths)
    elif op == "append":
        head_dim = rng.choice([64, 80, 96, 128, 128])
        kv_heads, group = rng.choice([(32, 1), (8, 8), (8, 4), (4, 5), (1, 8), (2, 7)])
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 32])
        c = _append("", _log_int(rng, 1, 4608), {"heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim},
                    rng.choice(["bf16", "bf16", "f32"]), page, rot, rng.random() < 0.5, rng.choice([10000.0, 500000.0]),
                    rng.choice([1.0, 4.0, 8.0]), rng.choice([4096, 8192, 131072]))
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        head_dim = rng.choice([64, 80, 128, 128, 128])
        kv_heads, group = rng.choice([(32, 1), (8, 8), (8, 4), (4, 5), (1, 8), (2, 7)])
        layout = {"heads": kv_heads * group, "kv_heads": kv_heads, "head_dim": head_dim}
        window, sinks = (rng.choice([100, 256, 1024, 2000]), rng.choice([0, 1, 4, 30])) if op == "window" else (0, 0)
        if rng.random() < 0.5:  # decode
            batch = _log_int(rng, 1, 256)
            c = _attend("", layout, dtype, page, batch, 1, rng.choice([1, 1, 4]), 0, _log_int(rng, 64, 8192 if batch < 32 else 2048),
                        lengths, window=window, sinks=sinks)
        else:  # chunks, some with decodes beside them
            batch = rng.randint(1, 6)
            singles = rng.choice([0, 0, rng.randint(1, 20)])
            c = _attend("", layout, dtype, page, batch + singles, 1, _log_int(rng, 8, 1024 if dtype == "bf16" else 256),
                        0, _log_int(rng, 64, 4096), lengths, singles=singles, window=window, sinks=sinks)
    del c["name"]
    return c


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(case):
    """(new, ctx) per request: the batch's shape, the same for every seed."""
    r = random.Random(case["lengths"])
    new, ctx = [], []
    for b in range(case["batch"]):
        single = b < case.get("singles", 0) or (case["op"] == "tables" and r.random() < 0.5)
        new.append(1 if single else r.randint(case["new_lo"], case["new_hi"]))
        ctx.append(r.randint(case["ctx_lo"], case["ctx_hi"]))
        if case["op"] == "tables" and r.random() < case["ended"]:
            new[-1] = -1
    return new, ctx


def _pages(lengths, page):
    return [-(-n // page) for n in lengths]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


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


def _prepare_tables(case, seed):
    rng = np.random.default_rng(seed)
    new, ctx = _lengths(case)
    page = case["page"]
    have = _pages(ctx, page)
    want = _pages([c + max(n, 0) for c, n in zip(ctx, new)], page)
    need = sum(w - h for w, h, n in zip(want, have, new) if n >= 0)
    free = int(need * case["free_share"]) + (1 if case["free_share"] >= 1 else 0)
    others = 64  # pages of the pool that requests outside this step hold
    table, left = _random_blocks(have, rng, free + others)
    wide = np.full((len(new), max(1, max(want))), -1, np.int32)
    wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
    num_pages = sum(have) + free + others
    head = int(rng.integers(0, num_pages))  # the free pages sit in a ring, starting anywhere
    ring = np.full(num_pages, -1, np.int32)
    ring[(head + np.arange(free)) % num_pages] = left[:free]
    tokens = sum(max(n, 0) for n in new)
    return {"page": page, "seq_len": _int32(ctx), "new_len": _int32(new), "block_table": torch.from_numpy(wide).cuda(),
            "free_pages": torch.from_numpy(ring).cuda(), "pool_in": _int32([head, free, 0, 0]),
            "pool_out": _int32([0, 0, 0, 0]), "q_start": _int32([0] * (len(new) + 1)), "kv_len": _int32([0] * len(new)),
            "position": _int32([0] * tokens), "slot": _int32([0] * tokens)}


def _angles(case):
    """Rotation angles [max_position, rot_dim / 2] in 64 bits."""
    half = case["rot_dim"] // 2
    freq = case["base"] ** (-torch.arange(half, dtype=torch.float64, device="cuda") * 2 / case["rot_dim"])
    return torch.arange(case["max_position"], dtype=torch.float64, device="cuda")[:, None] / case["scaling"] * freq


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, n, page = DTYPES[case["dtype"]], case["tokens"], case["page"]
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    num_pages = -(-n // page) + 8
    fused = torch.randn(n, (hq + 2 * hk) * d, generator=gen, device="cuda").to(dtype)
    cache = torch.randn(2, num_pages, hk, page, d, generator=gen, device="cuda").to(dtype)
    slots = (rng.permutation(num_pages)[:, None] * page + np.arange(page)).reshape(-1)[:n].astype(np.int32)
    if n > 8:
        slots[rng.integers(0, n)] = -1  # a token without a slot: rotated, not written
    start = rng.integers(0, max(1, case["max_position"] - n))
    position = ((start + np.arange(n)) % case["max_position"]).astype(np.int32)
    angle = _angles(case)
    table = torch.stack([angle.cos(), angle.sin()], -1).to(torch.float32).contiguous()
    q, k, v = fused.split([hq * d, hk * d, hk * d], dim=1)
    return {"q": q.view(n, hq, d), "k": k.view(n, hk, d), "v": v.view(n, hk, d), "K": cache[0], "V": cache[1],
            "position": torch.from_numpy(position).cuda(), "slot": torch.from_numpy(slots).cuda(), "table": table,
            "interleaved": case["interleaved"], "q_out": torch.empty(n, hq, d, dtype=dtype, device="cuda")}


def _prepare_attend(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, page = DTYPES[case["dtype"]], case["page"]
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    new, ctx = _lengths(case)
    kv = [n + c for n, c in zip(new, ctx)]
    table, _ = _random_blocks(_pages(kv, page), rng)
    num_pages, n = sum(_pages(kv, page)), sum(new)
    fused = torch.randn(n, (hq + 2 * hk) * d, generator=gen, device="cuda").to(dtype)
    K = torch.randn(num_pages, hk, page, d, generator=gen, device="cuda", dtype=dtype)
    V = torch.randn(num_pages, hk, page, d, generator=gen, device="cuda", dtype=dtype)
    return {"q": fused[:, :hq * d].view(n, hq, d), "K": K, "V": V, "block_table": torch.from_numpy(table).cuda(),
            "q_start": _int32([0] + list(np.cumsum(new))), "kv_len": _int32(kv), "max_q_len": max(new),
            "scale": d ** -0.5, "window": case["window"], "sinks": case["sinks"],
            "out": torch.empty(n, hq, d, dtype=dtype, device="cuda"),
            "lse": torch.empty(n, hq, dtype=torch.float32, device="cuda")}


def prepare(case, seed):
    make = {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend}[case["op"]]
    return {"op": case["op"], **make(case, seed)}


def _plain_tables(s):
    page, table, ring = s["page"], s["block_table"], s["free_pages"]
    rows, width, pages, n = table.shape[0], table.shape[1], ring.numel(), s["slot"].numel()
    seq, ended = s["seq_len"].long().clamp(min=0), s["new_len"] < 0
    new = s["new_len"].long().clamp(min=0)
    head, count = s["pool_in"][0].long(), s["pool_in"][1].long()
    have = ((seq + page - 1) // page).clamp(max=width)
    want = (seq + new + page - 1) // page
    need = torch.where(ended | (want > width), 0, want - have)
    upto = need.cumsum(0)
    granted = ~ended & (want <= width) & ((need == 0) | (upto <= count))
    taken = torch.where(granted & (need > 0), upto, 0).amax()
    column = torch.arange(width, device=table.device)
    back = column[None, :] < torch.where(ended, have, 0)[:, None]  # the ended requests' pages, in order
    rank = back.view(-1).long().cumsum(0).view(rows, width) - 1
    wide = torch.cat([ring, ring[:1]])
    wide.scatter_(0, torch.where(back, (head + count + rank) % pages, pages).view(-1), table.view(-1))
    nth = column[None, :] - have[:, None]
    fresh = granted[:, None] & (nth >= 0) & (nth < need[:, None])
    page_of = ring[((head + (upto - need)[:, None] + nth) % pages)]
    table.copy_(torch.where(fresh, page_of, table))
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    token = torch.arange(n, device=table.device)
    of = torch.searchsorted(start, token, right=True) - 1
    inside, of = of < rows, of.clamp(max=rows - 1)
    pos = seq[of] + token - start[of]
    cell = table[of, (pos // page).clamp(max=width - 1)].long()
    s["slot"].copy_(torch.where(inside & granted[of], cell * page + pos % page, -1))
    s["position"].copy_(torch.where(inside, pos, -1))
    s["q_start"].copy_(start)
    s["kv_len"].copy_(torch.where(ended, 0, torch.where(granted, seq + new, seq)))
    ring.copy_(wide[:pages])
    refused = (~ended & ~granted).sum()
    s["pool_out"].copy_(torch.stack([(head + taken) % pages, count - taken + back.sum(), refused, start[-1]]))
    return {k: s[k] for k in ("block_table", "free_pages", "pool_out", "q_start", "kv_len", "position", "slot")}


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_append(s):
    turn = s["table"][s["position"].long()]
    cos, sin = turn[:, None, :, 0], turn[:, None, :, 1]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, s["interleaved"]))
    k = _rotated(s["k"], cos, sin, s["interleaved"]).to(s["K"].dtype)
    page = s["K"].shape[2]
    slot = s["slot"].long()
    has = torch.nonzero(slot >= 0).view(-1)  # a token without a slot writes nothing
    cell, at = slot[has] // page, slot[has] % page
    s["K"][cell, :, at] = k[has]
    s["V"][cell, :, at] = s["v"][has]
    return {"q_out": s["q_out"], "K": s["K"], "V": s["V"]}


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
    pos = (kv - n)[:, None] + row
    seen = key <= pos[..., None]
    if s["window"] > 0:
        seen &= (key > pos[..., None] - s["window"]) | (key < s["sinks"])
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


def run(s):
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    import segmented_gather_gemm_sgmv_amd as sg
    if s["op"] == "tables":
        sg.sgmv_kv_tables(s["seq_len"], s["new_len"], s["block_table"], s["page"], s["free_pages"], s["pool_in"],
                          s["pool_out"], s["q_start"], s["kv_len"], s["position"], s["slot"])
        return {k: s[k] for k in ("block_table", "free_pages", "pool_out", "q_start", "kv_len", "position", "slot")}
    if s["op"] == "append":
        sg.sgmv_rope_append(s["q_out"], s["q"], s["k"], s["v"], s["K"], s["V"], s["position"], s["slot"], s["table"],
                            s["interleaved"])
        return {"q_out": s["q_out"], "K": s["K"], "V": s["V"]}
    sg.sgmv_paged_attention(s["out"], s["q"], s["K"], s["V"], s["block_table"], s["q_start"], s["kv_len"], s["scale"],
                            s["max_q_len"], window=s["window"], sinks=s["sinks"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _keys_seen(new, ctx, window, sinks):
    """(keys read at all, query-key pairs) of one request."""
    pos = np.arange(ctx, ctx + new, dtype=np.int64)
    if not window:
        return ctx + new, int((pos + 1).sum())
    first = np.maximum(pos - window + 1, 0)
    pairs = pos + 1 - first + np.minimum(first, sinks)
    return int(ctx + new - first[0] + min(first[0], sinks)), int(pairs.sum())


def work(case):
    if case["op"] == "tables":
        new, ctx = _lengths(case)
        page, tokens = case["page"], sum(max(n, 0) for n in new)
        fresh = sum(w - h for w, h, n in zip(_pages([c + max(n, 0) for c, n in zip(ctx, new)], page), _pages(ctx, page), new) if n >= 0)
        back = sum(h for h, n in zip(_pages(ctx, page), new) if n < 0)
        return {"bytes": 4 * (4 * len(new) + 2 * tokens + 2 * fresh + 2 * back + 8), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        n = case["tokens"]
        return {"bytes": n * (2 * size * d * (hq + 2 * hk) + 4 * case["rot_dim"] + 8),
                "flops": 3 * n * case["rot_dim"] * (hq + hk)}
    new, ctx = _lengths(case)
    seen = [_keys_seen(n, c, case["window"], case["sinks"]) for n, c in zip(new, ctx)]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    tables = 4 * (2 * len(new) + 1 + sum(_pages([k for k, _ in seen], case["page"])))
    return {"bytes": 2 * size * hk * d * keys + sum(new) * hq * (2 * size * d + 4) + tables, "flops": 4 * hq * d * pairs}


def _exact_append(case, seed):
    s = prepare(case, seed)
    rot, half = case["rot_dim"], case["rot_dim"] // 2
    angle = _angles(case)[s["position"].long()][:, None, :]
    first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)

    def turn(x):
        x = x.double()
        y = x.clone()
        y[..., first] = x[..., first] * angle.cos() - x[..., second] * angle.sin()
        y[..., second] = x[..., first] * angle.sin() + x[..., second] * angle.cos()
        return y

    K, V = s["K"].double(), s["V"].double()
    has = s["slot"] >= 0
    at = s["slot"][has].long()
    K[at // case["page"], :, at % case["page"]] = turn(s["k"])[has]
    V[at // case["page"], :, at % case["page"]] = s["v"][has].double()
    return {"q_out": turn(s["q"]), "K": K, "V": V}


def _exact_attend(case, seed):
    s = prepare(case, seed)
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    new, ctx = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pages = s["block_table"][b, :_pages([n + c], case["page"])[0]].long()
        k, v = (x[pages].double().transpose(0, 1).reshape(hk, -1, d)[:, :n + c] for x in (s["K"], s["V"]))
        p = torch.arange(c, c + n, device="cuda")[:, None]
        j = torch.arange(n + c, device="cuda")[None, :]
        hidden = j > p
        if case["window"]:
            hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
        step = max(1, (1 << 27) // max(1, n * (n + c)))  # heads at a time
        for h in range(0, hq, step):
            heads = torch.arange(h, min(hq, h + step), device="cuda")
            kk, vv = k[heads // (hq // hk)], v[heads // (hq // hk)]
            score = s["q"][at:at + n, heads].double().transpose(0, 1).contiguous() @ kk.transpose(1, 2).contiguous()
            score = (score * case["head_dim"] ** -0.5).masked_fill(hidden, -math.inf)
            lse[at:at + n, heads] = torch.logsumexp(score, -1).T
            out[at:at + n, heads] = (torch.softmax(score, -1) @ vv.contiguous()).transpose(0, 1)
        at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    return _exact_append(case, seed) if case["op"] == "append" else _exact_attend(case, seed)
