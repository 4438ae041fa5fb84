"""Plain 64-bit implementations of the paged-cache operators, and the error
bounds that the GPU tests hold the kernels to. No code is shared with the
library."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # unit roundoff of binary32
U16 = 2.0 ** -8    # unit roundoff of bfloat16


def tables(seq_len, new_len, block_table, page, ring, pool, T):
    """One step, request by request, on plain lists. Returns a dict of arrays."""
    seq_len, new_len = list(map(int, seq_len)), list(map(int, new_len))
    table, ring = np.array(block_table, np.int32), np.array(ring, np.int32)
    P, width = len(ring), table.shape[1]
    head, count = int(pool[0]), int(pool[1])
    before = table.copy()
    q_start, kv, refused, position, slot = [0], [], 0, [], []
    taken, stuck, returned = 0, False, []
    for b, (L, n) in enumerate(zip(seq_len, new_len)):
        have = -(-L // page)
        if n < 0:
            returned += list(before[b, :have])
            kv.append(0)
            q_start.append(q_start[-1])
            continue
        want = -(-(L + n) // page)
        ok = want <= width
        if ok and want > have:
            if stuck or taken + want - have > count:
                ok, stuck = False, True
            else:
                for i in range(have, want):
                    table[b, i] = ring[(head + taken) % P]
                    taken += 1
        refused += not ok
        kv.append(L + n if ok else L)
        q_start.append(q_start[-1] + n)
        for p in range(L, L + n):
            position.append(p)
            slot.append(int(table[b, p // page]) * page + p % page if ok else -1)
    out_ring = ring.copy()
    for i, p in enumerate(returned):
        out_ring[(head + count + i) % P] = p
    pad = T - len(position)
    return {"block_table": table, "free_pages": out_ring,
            "pool_out": np.array([(head + taken) % P, count - taken + len(returned), refused, q_start[-1]], np.int32),
            "q_start": np.array(q_start, np.int32), "kv_len": np.array(kv, np.int32),
            "position": np.array(position + [-1] * pad, np.int32)[:T],
            "slot": np.array(slot + [-1] * pad, np.int32)[:T]}


def rope_angles(max_position, rot_dim, base):
    i = np.arange(rot_dim // 2)
    return np.arange(max_position)[:, None] * float(base) ** (-2.0 * i / rot_dim)


def rotate(x, angle, interleaved):
    """x [T, heads, D] float64, angle [T, rot/2]. Returns (rotated, |a| + |b| of
    each element's pair, 0 past the rotated part)."""
    half = angle.shape[1]
    y, size = x.copy(), np.zeros_like(x)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(angle[:, i])[:, None], np.sin(angle[:, i])[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def rope_bound(y, size, bf16):
    """Two fp32 products and a sum of table values rounded once (4 roundings of
    at most |a| + |b|), then one rounding to the storage type."""
    return (U16 if bf16 else U32) * np.abs(y) * 1.01 + 4 * U32 * size


def attend(q, K, V, block_table, q_start, kv_len, scale, window=0, sinks=0, bf16=False):
    """q [T, hq, d], K, V [pages, hk, page, d], all float64. Returns out, lse,
    and bounds on their errors."""
    T, hq, d = q.shape
    hk, page = K.shape[1], K.shape[2]
    out, lse = np.zeros_like(q), np.full((T, hq), -np.inf)
    tol_out, tol_lse = np.zeros_like(q), np.zeros((T, hq))
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        for i in range(n):
            p = kv - n + i
            seen = [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]
            if not seen:
                continue
            seen = np.array(seen)
            cells = (block_table[b, seen // page], slice(None), seen % page)
            k, v = K[cells[0], :, cells[2]], V[cells[0], :, cells[2]]
            for h in range(hq):
                row = q_start[b] + i
                kh, vh = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
                s = kh @ q[row, h] * scale
                top = s.max()
                w = np.exp(s - top)
                out[row, h] = w @ vh / w.sum()
                lse[row, h] = top + np.log(w.sum())
                # Scores: d products summed in fp32, times scale and log2 e; the exponent's own
                # rounding; the exponential to 2 ulp; sums over the keys.
                ds = ((d + 2) * (np.abs(kh) @ np.abs(q[row, h])).max() * scale + 4 * np.abs(s).max()) * U32
                dw = 2 * ds + (len(seen) + 16) * U32
                mass = w @ np.abs(vh) / w.sum()
                tol_out[row, h] = (dw + (U16 if bf16 else 0)) * mass * 1.01 + (U16 if bf16 else U32) * np.abs(out[row, h]) * 1.01
                tol_lse[row, h] = ds + (len(seen) + 16) * U32 + 4 * U32 * abs(lse[row, h])
    return out, lse, tol_out, tol_lse
