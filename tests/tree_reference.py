"""Plain 64-bit implementations of the drafted-tree operators, and the error
bounds that the GPU tests hold the kernels to. No code is shared with the
library."""
from __future__ import annotations

import numpy as np

from .kv_reference import U16, U32


def random_tree(rng, n, branch=3):
    """Parents of a random tree: token 0 is the root, others hang on any earlier one (near ones more often)."""
    return np.array([-1] + [int(rng.integers(max(0, (i - 1) // branch - 2), i)) for i in range(1, n)], np.int32)[:n]


def tables(parents, kv_len, T, words):
    """parents: a list of arrays, one per request. Returns (position [T], mask [T, words] uint32)."""
    position, mask = np.full(T, -1, np.int64), np.zeros((T, words), np.uint32)
    at = 0
    for parent, kv in zip(parents, kv_len):
        n = len(parent)
        for i in range(min(n, 32 * words)):
            j, depth = i, -1
            while True:
                mask[at + i, j // 32] |= np.uint32(1 << (j % 32))
                depth += 1
                p = int(parent[j])
                if not 0 <= p < j:
                    break
                j = p
            position[at + i] = kv - n + depth
        at += n
    return position, mask


def bits_of(mask, n):
    """mask [words] -> the first n bits."""
    return ((mask[:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)[:n].astype(bool)


def seen_keys(mask, c, n, window, sinks):
    """Keys (indices in the request) that a token with this mask sees."""
    drafted = bits_of(mask, n)
    p = c - 1 + int(drafted.sum())
    cached = [j for j in range(c) if window == 0 or j > p - window or j < sinks]
    return np.array(cached + [c + m for m in np.flatnonzero(drafted)], np.int64)


def attend(q, K, V, block_table, q_start, kv_len, mask, scale, window=0, sinks=0, bf16=False):
    """q [T, hq, d], K, V [pages, hk, page, d], all float64. Returns out, lse,
    and bounds on their errors (derived as those of the causal call)."""
    T, hq, d = q.shape
    hk, page = K.shape[1], K.shape[2]
    group = hq // hk
    out, lse = np.zeros_like(q), np.full((T, hq), -np.inf)
    tol_out, tol_lse = np.zeros_like(q), np.zeros((T, hq))
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        for i in range(n):
            row = q_start[b] + i
            seen = seen_keys(mask[row], kv - n, n, window, sinks)
            if not len(seen):
                continue
            k, v = K[block_table[b, seen // page], :, seen % page], V[block_table[b, seen // page], :, seen % page]
            for h in range(hq):
                kh, vh = k[:, h // group], v[:, h // group]
                s = kh @ q[row, h] * scale
                top = s.max()
                w = np.exp(s - top)
                out[row, h] = w @ vh / w.sum()
                lse[row, h] = top + np.log(w.sum())
                # Scores: d products summed in fp32, times scale and log2 e; the exponent's own rounding; the
                # exponential to 2 ulp; sums over the keys; bf16 weights hold 16 significant bits.
                ds = ((d + 2) * (np.abs(kh) @ np.abs(q[row, h])).max() * scale + 4 * np.abs(s).max()) * U32
                dw = 2 * ds + (len(seen) + 16) * U32 + (2.0 ** -16 if bf16 else 0)
                mass = w @ np.abs(vh) / w.sum()
                tol_out[row, h] = dw * mass * 1.01 + (U16 if bf16 else U32) * np.abs(out[row, h]) * 1.01
                tol_lse[row, h] = ds + (len(seen) + 16) * U32 + 4 * U32 * abs(lse[row, h])
    return out, lse, tol_out, tol_lse


def accept(parents, token, target, slot, q_start, kv_len, page, block_table, ring, pool, T):
    """One step, request by request. Returns a dict of arrays."""
    path, accepted, nxt, kept, back = np.full(T, -1, np.int64), [], [], [], []
    for b, parent in enumerate(parents):
        n, q0, kv = len(parent), int(q_start[b]), int(kv_len[b])
        if n == 0 or slot[q0] < 0:
            accepted.append(0)
            nxt.append(-1)
            kept.append(kv)
            continue
        walk = [0]
        while True:
            i = walk[-1]
            child = [j for j in range(i + 1, min(n, 1024)) if parent[j] == i and token[q0 + j] == target[q0 + i]]
            if not child:
                break
            walk.append(child[0])
        path[q0:q0 + len(walk)] = walk
        accepted.append(len(walk))
        nxt.append(int(target[q0 + walk[-1]]))
        kept.append(kv - n + len(walk))
        back += list(block_table[b, -(-kept[-1] // page):-(-kv // page)])
    ring = np.array(ring).copy()
    for i, p in enumerate(back):
        ring[(int(pool[0]) + int(pool[1]) + i) % len(ring)] = p
    return {"path": path, "accepted": np.array(accepted, np.int64), "next_token": np.array(nxt, np.int64),
            "kept_len": np.array(kept, np.int64), "free_pages": ring,
            "pool_out": np.array([pool[0], pool[1] + len(back), pool[2], pool[3]])}
