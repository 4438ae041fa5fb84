"""The paged-cache operators on the GPU against plain 64-bit implementations
(tests/kv_reference.py), to error bounds derived there."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import kv_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, what=""):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    same = got == want  # infinities too
    err = np.where(same, 0.0, np.abs(np.where(same, 0, got) - np.where(same, 0, want)))
    worst = np.max(err - tol, initial=-1.0)
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


# -- block tables and slots ----------------------------------------------------
def tables_case(rng, B, page, max_new, max_ctx, ended, free_share=1.0, slack=0, T_extra=0):
    seq = rng.integers(0, max_ctx + 1, B)
    new = rng.integers(0, max_new + 1, B)
    new[rng.random(B) < ended] = -1
    have = -(-seq // page)
    want = -(-(seq + np.maximum(new, 0)) // page)
    need = int(np.where(new >= 0, want - have, 0).sum())
    free = int(need * free_share) + slack
    P = int(have.sum()) + free + 3
    order = rng.permutation(P).astype(np.int32)
    table = np.full((B, max(1, int(want.max(initial=1)))), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    head = int(rng.integers(0, P))
    ring = np.full(P, -1, np.int32)
    ring[(head + np.arange(free)) % P] = order[at:at + free]
    return seq, new, table, ring, [head, free, 0, 0], int(np.maximum(new, 0).sum()) + T_extra


def run_tables(dev, seq, new, table, page, ring, pool, T, stream=None):
    B = len(seq)
    t = dict(seq_len=ints(seq, dev), new_len=ints(new, dev), block_table=ints(table, dev), free_pages=ints(ring, dev),
             pool_in=ints(pool, dev), pool_out=ints([7] * 4, dev), q_start=ints([7] * (B + 1), dev),
             kv_len=ints([7] * B, dev), position=ints([7] * T, dev), slot=ints([7] * T, dev))
    sg.sgmv_kv_tables(t["seq_len"], t["new_len"], t["block_table"], page, t["free_pages"], t["pool_in"], t["pool_out"],
                      t["q_start"], t["kv_len"], t["position"], t["slot"])
    torch.cuda.synchronize()
    return t


@pytest.mark.parametrize("B,page,max_new,max_ctx,ended,free_share,slack,T_extra", [
    (1, 16, 0, 40, 0.0, 1.0, 0, 0),        # nothing to add
    (1, 16, 33, 0, 0.0, 1.0, 0, 5),        # a first prompt, and tokens past the last
    (64, 16, 1, 100, 0.0, 1.0, 4, 0),      # decode
    (65, 32, 1, 300, 0.2, 1.0, 0, 0),      # some ended
    (257, 16, 90, 200, 0.3, 1.0, 9, 3),    # mixed, over one scan block
    (300, 64, 70, 500, 0.1, 0.6, 0, 0),    # a pool that runs out
    (40, 16, 200, 50, 0.0, 0.0, 0, 0),     # no free page at all
    (2500, 16, 5, 60, 0.1, 0.95, 0, 0),    # many requests
    (8192, 16, 2, 20, 0.05, 1.0, 0, 0),    # as many as a call takes
])
def test_tables(dev, B, page, max_new, max_ctx, ended, free_share, slack, T_extra):
    rng = np.random.default_rng(B * 1000 + page)
    seq, new, table, ring, pool, T = tables_case(rng, B, page, max_new, max_ctx, ended, free_share, slack, T_extra)
    want = ref.tables(seq, new, table, page, ring, pool, T)
    got = run_tables(dev, seq, new, table, page, ring, pool, T)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k


def test_tables_narrow_row_and_no_requests(dev):
    """A request too long for its row is refused and takes no page from the
    others; a step without requests still writes its outputs."""
    table = np.array([[5, -1], [6, 7], [8, -1]], np.int32)
    ring = np.arange(10, dtype=np.int32)
    args = ([10, 20, 16], [10, 30, 1], table, 16, ring, [9, 4, 0, 0], 41)
    got, want = run_tables(dev, *args), ref.tables(*args)
    for k, v in want.items():
        assert np.array_equal(got[k].cpu().numpy(), v), k
    assert want["pool_out"].tolist() == [1, 2, 1, 41]
    got = run_tables(dev, [], [], np.zeros((0, 2), np.int32), 16, ring, [3, 2, 0, 0], 4)
    assert got["pool_out"].tolist() == [3, 2, 0, 0] and got["q_start"].tolist() == [0]
    assert got["slot"].tolist() == [-1] * 4 and got["position"].tolist() == [-1] * 4


def test_tables_steps_follow_one_another(dev):
    """Twenty steps with the pool and the lengths carried on the device: at
    every step each page is free or in one row, once."""
    rng = np.random.default_rng(3)
    B, page, P, width = 9, 16, 60, 8
    lens, pool = [ints([0] * B, dev), ints([0] * B, dev)], [ints([0, P, 0, 0], dev), ints([0] * 4, dev)]
    table, ring = ints(np.full((B, width), -1), dev), ints(rng.permutation(P), dev)
    host_table, host_ring = table.cpu().numpy(), ring.cpu().numpy()
    for step in range(20):
        a, z = step % 2, 1 - step % 2
        new = rng.integers(0, 40, B)
        new[rng.random(B) < 0.25] = -1
        T = int(np.maximum(new, 0).sum())
        want = ref.tables(lens[a].tolist(), new, host_table, page, host_ring, pool[a].tolist(), T)
        pos, slot, q_start = ints([0] * T, dev), ints([0] * T, dev), ints([0] * (B + 1), dev)
        sg.sgmv_kv_tables(lens[a], ints(new, dev), table, page, ring, pool[a], pool[z], q_start, lens[z], pos, slot)
        got = dict(block_table=table, free_pages=ring, pool_out=pool[z], q_start=q_start, kv_len=lens[z], position=pos,
                   slot=slot)
        for k, v in want.items():
            assert np.array_equal(got[k].cpu().numpy(), v), (step, k)
        host_table, host_ring = want["block_table"], want["free_pages"]
        head, count = want["pool_out"][:2]
        held = [p for b in range(B) for p in host_table[b, :-(-int(want["kv_len"][b]) // page)]]
        free = [host_ring[(head + i) % P] for i in range(count)]
        assert sorted(held + free) == list(range(P)), step


# -- rotary positions and the write to the cache ---------------------------------
@pytest.mark.parametrize("kind,kw", [(sg.SGMV_ROPE_PLAIN, {}), (sg.SGMV_ROPE_LINEAR, dict(factor=8.0)),
                                     (sg.SGMV_ROPE_BY_PARTS, dict(factor=16.0, original_max=4096))])
def test_rope_table(dev, kind, kw):
    rot, base, n = 64, 10000.0, 5000
    got = f64(sg.sgmv_rope_table(n, rot, base, kind, device=dev, **kw))
    i = np.arange(rot // 2)
    f, size = base ** (-2.0 * i / rot), 1.0
    if kind == sg.SGMV_ROPE_LINEAR:
        f = f / kw["factor"]
    if kind == sg.SGMV_ROPE_BY_PARTS:
        turns = kw["original_max"] * f / (2 * np.pi)      # turns of each pair over the original length
        low = np.floor(np.interp(-np.log(32.0), -np.log(turns), i))
        high = np.ceil(np.interp(-np.log(1.0), -np.log(turns), i))
        w = 1 - np.clip((i - low) / (high - low), 0, 1)
        assert w[0] == 1 and w[-1] == 0 and ((w > 0) & (w < 1)).any()
        f, size = f * w + f / kw["factor"] * (1 - w), 0.1 * np.log(kw["factor"]) + 1
    angle = np.arange(n)[:, None] * f
    # one rounding to fp32, and 2^-52 of the angle and of its frequency's power (a few ulp)
    tol = U = ref.U32 * size * 1.01 + 16 * 2.0 ** -52 * (1 + angle) * size
    assert (np.abs(got[..., 0] - np.cos(angle) * size) <= tol).all()
    assert (np.abs(got[..., 1] - np.sin(angle) * size) <= U).all()


def rope_case(rng, dev, T, hq, hk, D, dtype, page, pages, max_position, fused=True, pad=0):
    width = (hq + 2 * hk) * D + pad
    x = torch.tensor(rng.standard_normal((T, width)), dtype=F32).to(dtype).to(dev)
    q, k, v = x[:, :hq * D].view(T, hq, D), x[:, hq * D:(hq + hk) * D].view(T, hk, D), x[:, (hq + hk) * D:(hq + 2 * hk) * D].view(T, hk, D)
    K, V = (torch.tensor(rng.standard_normal((pages, hk, page, D)), dtype=F32).to(dtype).to(dev) for _ in range(2))
    slot = rng.permutation(pages * page)[:T].astype(np.int32)
    position = rng.integers(0, max_position, T).astype(np.int32)
    return q, k, v, K, V, position, slot


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,hq,hk,D,rot,page", [(1, 8, 1, 128, 128, 16), (7, 32, 32, 128, 128, 16), (65, 5, 5, 80, 32, 32),
                                                (33, 14, 2, 64, 64, 64), (3, 1, 1, 16, 16, 16), (130, 6, 3, 72, 48, 128),
                                                (20, 4, 2, 96, 0, 16), (9, 71, 1, 64, 16, 256),
                                                # rotated parts of every run length
                                                (11, 4, 2, 80, 40, 16), (8, 3, 1, 64, 36, 32), (8, 2, 2, 40, 2, 16),
                                                (7, 5, 5, 128, 126, 16), (10, 6, 2, 24, 24, 16)])
def test_rope_append(dev, dtype, interleaved, T, hq, hk, D, rot, page):
    rng = np.random.default_rng(T * 7 + D)
    n = 999
    q, k, v, K, V, position, slot = rope_case(rng, dev, T, hq, hk, D, dtype, page, T // page + 3, n, pad=8)
    if T > 6:
        slot[2], slot[4] = -1, K.shape[0] * page     # no slot; one outside the cache
        position[3], position[5] = -1, n             # left out
    table = sg.sgmv_rope_table(n, rot, 10000.0, device=dev) if rot else None
    q_out = torch.full((T, hq * D + 16), 7.0, dtype=dtype, device=dev)[:, 8:8 + hq * D].view(T, hq, D)
    K0, V0 = f64(K), f64(V)
    sg.sgmv_rope_append(q_out, q, k, v, K, V, ints(position, dev), ints(slot, dev), table, interleaved)
    torch.cuda.synchronize()
    used = (position >= 0) & ((position < n) | (rot == 0))  # without a table every position >= 0 is taken
    angle = ref.rope_angles(n, rot, 10000.0)[np.clip(position, 0, n - 1)] if rot else np.zeros((T, 0))
    bf16 = dtype is BF16
    yq, sq = ref.rotate(f64(q), angle, interleaved)
    yk, sk = ref.rotate(f64(k), angle, interleaved)
    want_q = np.where(used[:, None, None], yq, 7.0)
    within(q_out, want_q, np.where(used[:, None, None], ref.rope_bound(yq, sq, bf16), 0), "q")
    tol_K = np.zeros_like(K0)
    for t in range(T):
        if used[t] and 0 <= slot[t] < K.shape[0] * page:
            K0[slot[t] // page, :, slot[t] % page] = yk[t]
            tol_K[slot[t] // page, :, slot[t] % page] = ref.rope_bound(yk, sk, bf16)[t]
            V0[slot[t] // page, :, slot[t] % page] = f64(v)[t]
    within(K, K0, tol_K, "K")
    assert np.array_equal(f64(V), V0)


def test_rope_in_place_and_parts(dev):
    """q_out may be q; q alone; k and v alone: each equals the whole call."""
    rng = np.random.default_rng(5)
    q, k, v, K, V, position, slot = rope_case(rng, dev, 50, 8, 2, 64, BF16, 16, 6, 100)
    pos, sl, table = ints(position, dev), ints(slot, dev), sg.sgmv_rope_table(100, 64, device=dev)
    whole, K1, V1 = torch.empty(50, 8, 64, dtype=BF16, device=dev), K.clone(), V.clone()
    sg.sgmv_rope_append(whole, q, k, v, K1, V1, pos, sl, table)
    alone = torch.empty_like(whole)
    sg.sgmv_rope_append(alone, q, None, None, None, None, pos, None, table)
    K2, V2 = K.clone(), V.clone()
    sg.sgmv_rope_append(None, None, k, v, K2, V2, pos, sl, table)
    sg.sgmv_rope_append(q, q, k, v, K, V, pos, sl, table)
    torch.cuda.synchronize()
    assert torch.equal(alone, whole) and torch.equal(q.contiguous(), whole)
    assert torch.equal(K1, K2) and torch.equal(V1, V2) and torch.equal(K1, K) and torch.equal(V1, V)


# -- attention -------------------------------------------------------------------
def paged(rng, dev, new, ctx, hq, hk, D, dtype, page, extra_width=2, garbage=float("nan"), std=1.0):
    """A paged batch. Cells and pages that no token has hold `garbage`, and
    table entries past a request's pages are out of range."""
    B = len(new)
    kv = [n + c for n, c in zip(new, ctx)]
    count = [-(-n // page) for n in kv]
    pages = sum(count) + 2
    order = rng.permutation(pages)
    table = np.full((B, max(1, max(count, default=1)) + extra_width), 1 << 30, np.int32)
    K = np.full((pages, hk, page, D), garbage)
    V = np.full((pages, hk, page, D), garbage)
    at = 0
    for b in range(B):
        table[b, :count[b]] = order[at:at + count[b]]
        at += count[b]
        for j in range(kv[b]):
            K[table[b, j // page], :, j % page] = rng.standard_normal((hk, D)) * std
            V[table[b, j // page], :, j % page] = rng.standard_normal((hk, D)) * std
    T = sum(new)
    row = torch.tensor(rng.standard_normal((T, hq * D + 24)) * std, dtype=F32).to(dtype).to(dev)
    q = row[:, 8:8 + hq * D].view(T, hq, D)
    K, V = (torch.tensor(x, dtype=F32).to(dtype).to(dev) for x in (K, V))
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return q, K, V, table, q_start, np.array(kv, np.int32)


def attend(dev, q, K, V, table, q_start, kv, window=0, sinks=0, scale=None, max_q_len=None, want_lse=True):
    T, hq, D = q.shape
    out = torch.full((T, hq * D + 8), 7.0, dtype=q.dtype, device=dev)[:, :hq * D].view(T, hq, D)
    lse = torch.full((T, hq), 7.0, dtype=F32, device=dev) if want_lse else None
    n = int(np.diff(q_start).max(initial=0)) if max_q_len is None else max_q_len
    sg.sgmv_paged_attention(out, q, K, V, ints(table, dev), ints(q_start, dev), ints(kv, dev),
                            D ** -0.5 if scale is None else scale, n, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    ws = sg.attention_workspace(dev, D, q.dtype)
    assert int(ws[:4096].sum()) == 0   # the counters are zero again
    return out, lse


def check_attention(dev, rng, new, ctx, hq, hk, D, dtype, page, window=0, sinks=0, std=1.0):
    q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, hq, hk, D, dtype, page, std=std)
    out, lse = attend(dev, q, K, V, table, q_start, kv, window, sinks)
    o, l, to, tl = ref.attend(f64(q), f64(K), f64(V), table, q_start, kv, D ** -0.5, window, sinks, dtype is BF16)
    within(out, o, to, "out")
    within(lse, l, tl, "lse")


SHAPES = [  # new, ctx, hq, hk, D, page
    ([1], [0], 1, 1, 128, 16),                       # one token, one key
    ([1, 1, 1], [15, 16, 17], 4, 4, 64, 16),         # ends around a page's end
    ([1] * 5, [0, 31, 32, 63, 500], 8, 1, 128, 16),  # a group of 8, ends around a tile's
    ([1, 2, 3], [700, 3, 0], 14, 2, 80, 32),         # a group of 7, a head of 80
    ([4, 1], [250, 100], 8, 2, 64, 64),              # several tokens per request
    ([17, 1, 40], [0, 90, 5], 6, 3, 128, 16),        # chunks
    ([130], [70], 2, 1, 64, 16),                     # a chunk over row tiles
    ([33, 5], [127, 300], 16, 2, 128, 128),          # 264 packed rows
    ([3, 1], [40, 9], 10, 2, 8, 16),                 # the narrowest head
    ([1, 3], [40, 1200], 48, 1, 96, 256),            # a group of 48
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(dev, dtype, case):
    check_attention(dev, np.random.default_rng(case), *SHAPES[case][:5], dtype, SHAPES[case][5])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (33, 4), (100, 40), (64, 1), (5000, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_attention_window(dev, dtype, window, sinks):
    rng = np.random.default_rng(window % 1000 + sinks % 7)
    check_attention(dev, rng, [1, 1, 37, 1, 2], [400, 30, 150, 0, 65], 8, 2, 64, dtype, 16, window, sinks)
    check_attention(dev, rng, [70, 1], [300, 257], 4, 4, 128, dtype, 32, window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("std", [0.05, 6.0])
def test_attention_flat_and_peaked(dev, dtype, std):
    """Nearly equal weights, and scores in the hundreds, where the running
    reference point moves often."""
    rng = np.random.default_rng(11)
    check_attention(dev, rng, [1, 20], [600, 200], 8, 2, 64, dtype, 16, std=std)


def uniform(dev, new, ctx, hq, hk, D, dtype, page, window=0, sinks=0, seed=0, device_table=None):
    """q = 0: every visible key weighs exactly 1, so lse is log(count) and out
    is an integer sum over the count. One key too many or too few shows."""
    rng = np.random.default_rng(seed)
    B, kv = len(new), np.array([n + c for n, c in zip(new, ctx)], np.int32)
    count = -(-kv // page)
    order = rng.permutation(int(count.sum()) + 1)
    table = np.full((B, int(count.max())), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :count[b]] = order[at:at + count[b]]
        at += count[b]
    gen = torch.Generator(dev).manual_seed(seed)
    shape = (len(order), hk, page, D)
    K = torch.randn(shape, generator=gen, device=dev).to(dtype)
    V = torch.randint(-2, 3, shape, generator=gen, device=dev).to(dtype)
    q = torch.zeros(sum(new), hq, D, dtype=dtype, device=dev)
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out, lse = attend(dev, q, K, V, table, q_start, kv, window, sinks)
    for b in range(B):
        cells = torch.tensor(table[b, :count[b]], device=dev).long()
        v = V[cells].double().transpose(0, 1).reshape(hk, -1, D)[:, :kv[b]]
        upto = torch.cat([v.new_zeros(hk, 1, D), v.cumsum(1)], 1)
        p = torch.arange(ctx[b], ctx[b] + new[b], device=dev)
        lo = (p - window + 1).clamp(min=0) if window else torch.zeros_like(p)
        first = lo.clamp(max=sinks)
        total = upto[:, p + 1] - upto[:, lo] + upto[:, first]
        number = (p + 1 - lo + first).double()
        want = (total / number[:, None]).transpose(0, 1).repeat_interleave(hq // hk, 1)
        got = out[q_start[b]:q_start[b + 1]].double()
        u = ref.U16 if dtype is BF16 else 2 * ref.U32  # one rounding (of a quotient by a reciprocal in fp32)
        assert ((got - want).abs() <= 1.01 * u * want.abs() + 3 * ref.U32 * want.abs()).all(), b
        got = lse[q_start[b]:q_start[b + 1]].double()
        assert ((got - number.log()[:, None]).abs() <= 4 * ref.U32 * (1 + number.log()[:, None])).all(), b


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 4), (257, 70)])
def test_every_key_once(dev, dtype, window, sinks):
    uniform(dev, [1] * 30, list(range(0, 6000, 200)), 8, 2, 128, dtype, 16, window, sinks, 1)          # ragged decode
    uniform(dev, [1], [40000], 16, 2, 64, dtype, 32, window, sinks, 2)                                  # split many ways
    uniform(dev, [300, 1, 511, 64], [0, 2000, 1900, 4000], 4, 2, 128, dtype, 64, window, sinks, 3)      # chunks beside decode
    uniform(dev, [1500], [300], 8, 1, 64, dtype, 16, window, sinks, 4)                                  # one long chunk
    uniform(dev, [1] * 600, [b % 97 for b in range(600)], 5, 1, 64, dtype, 16, window, sinks, 5)        # many requests
    uniform(dev, [2, 5, 1] * 100, [b * 13 % 500 for b in range(300)], 12, 4, 72, dtype, 16, window, sinks, 6)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_rows_that_see_nothing(dev, dtype):
    """No cached token, fewer cached than new, and rows of no request."""
    rng = np.random.default_rng(2)
    q, K, V, table, _, _ = paged(rng, dev, [5, 6, 3, 4], [10, 10, 0, 3], 4, 2, 64, dtype, 16)
    q_start, kv = np.array([0, 5, 11, 14, 14], np.int32), np.array([0, 4, 3, 9], np.int32)
    out, lse = attend(dev, q, K, V, table, q_start, kv)
    o, l, to, tl = ref.attend(f64(q)[:14], f64(K), f64(V), table, q_start, kv, 64 ** -0.5, bf16=dtype is BF16)
    within(out[:14], o, to)
    within(lse[:14], l, tl)
    assert np.isinf(l[:7]).all() and (f64(out[:7]) == 0).all()
    assert (out[14:] == 7).all() and (lse[14:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_infinite_and_nan_inputs_stay_in_their_rows(dev, dtype):
    """A NaN query spoils its own row only; NaN and infinite keys and values
    before the window, which no row of the request sees, spoil nothing."""
    rng = np.random.default_rng(4)
    q, K, V, table, q_start, kv = paged(rng, dev, [1, 1, 20], [300, 300, 200], 4, 2, 64, dtype, 16)
    out, lse = attend(dev, q, K, V, table, q_start, kv, 50, 3)
    K2, V2 = K.clone(), V.clone()
    for b in range(3):
        first = kv[b] - (q_start[b + 1] - q_start[b]) - 50 + 1
        for j in range(3, first):
            K2[table[b, j // 16], :, j % 16] = float("nan") if j % 2 else float("inf")
            V2[table[b, j // 16], :, j % 16] = float("nan") if j % 3 else float("-inf")
    out2, lse2 = attend(dev, q, K2, V2, table, q_start, kv, 50, 3)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    q3 = q.clone()
    q3[7, 2] = float("nan")
    out3, lse3 = attend(dev, q3, K, V, table, q_start, kv, 50, 3)
    assert out3[7, 2].isnan().all() and lse3[7, 2].isnan()
    keep = torch.ones(22, 4, dtype=torch.bool, device=dev)
    keep[7, 2] = False
    assert torch.equal(out3[keep], out[keep]) and torch.equal(lse3[keep], lse[keep])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,hq,hk,D,window,sinks", [
    ([7, 1], [90, 40], 4, 2, 64, 0, 0),        # streamed in both types
    ([15, 2], [100, 30], 2, 1, 128, 20, 3),
    ([40, 1], [70, 90], 6, 2, 80, 0, 0),       # several row tiles, a narrower head
    ([150, 33], [20, 300], 8, 2, 128, 64, 5),
    ([200], [100], 1, 1, 64, 33, 70),
    ([1, 1], [400, 31], 8, 1, 128, 0, 0),      # single tokens: a value's infinity stays one
])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dev, dtype, new, ctx, hq, hk, D, window, sinks):
    """Causal masks and windows hide a key from some rows of a request and not
    from others; a NaN or an infinity in one column of its value belongs to the
    others' same column alone."""
    rng = np.random.default_rng(sum(new) + D)
    q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, hq, hk, D, dtype, 16)
    clean, odd = f64(V), V.clone()
    want = np.zeros(q.shape)   # what each element gets from values that are not finite
    for b in range(len(new)):
        p = np.arange(ctx[b], kv[b])
        keys = {int(kv[b]) - 1, int(kv[b]) - 2, ctx[b], ctx[b] + new[b] // 2, max(ctx[b] - 7, 0), 1}
        for n, j in enumerate(sorted(keys)):
            x = [float("nan"), float("inf"), float("-inf")][n % 3]
            head, cols = n % hk, [(11 * n) % D, D - 1 - n]
            seen = (j <= p) & ((j > p - window) | (j < sinks) | (window == 0))
            for c in cols:
                odd[table[b, j // 16], head, j % 16, c] = x
                clean[table[b, j // 16], head, j % 16, c] = 0.0
                for h in range(head * (hq // hk), (head + 1) * (hq // hk)):
                    want[q_start[b]:q_start[b + 1], h, c] += np.where(seen, x, 0.0)
    out, lse = attend(dev, q, K, odd, table, q_start, kv, window, sinks)
    o, l, to, tl = ref.attend(f64(q), f64(K), clean, table, q_start, kv, D ** -0.5, window, sinks, dtype is BF16)
    spoilt, got = ~np.isfinite(want), f64(out)
    assert spoilt.any() and not spoilt.all()
    assert np.array_equal(got[spoilt], want[spoilt], equal_nan=True)
    got[spoilt] = o[spoilt]
    within(torch.tensor(got), o, to, "out")
    within(lse, l, tl, "lse")


def test_same_bits_twice_without_lse_and_on_another_stream(dev):
    rng = np.random.default_rng(6)
    for new, ctx in (([1] * 3, [5000, 900, 40]), ([100, 1], [3000, 2500])):
        q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, 8, 2, 64, BF16, 16)
        a, la = attend(dev, q, K, V, table, q_start, kv)
        b, _ = attend(dev, q, K, V, table, q_start, kv, want_lse=False)
        assert torch.equal(a, b)
        s = torch.cuda.Stream(dev)
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            c, lc = attend(dev, q, K, V, table, q_start, kv)
        assert torch.equal(a, c) and torch.equal(la, lc)


def test_max_q_len_cuts_the_rows(dev):
    rng = np.random.default_rng(8)
    q, K, V, table, q_start, kv = paged(rng, dev, [9, 2], [100, 40], 4, 1, 64, BF16, 16)
    cut, lse = attend(dev, q, K, V, table, q_start, kv, max_q_len=4)
    done = [0, 1, 2, 3, 9, 10]
    o, l, to, tl = ref.attend(f64(q), f64(K), f64(V), table, q_start, kv, 64 ** -0.5, bf16=True)
    within(cut[done], o[done], to[done])
    within(lse[done], l[done], tl[done])
    assert (cut[4:9] == 7).all() and (lse[4:9] == 7).all()


def test_bad_metadata_touches_nothing_else(dev):
    """Offsets that decrease, lengths past the table, page ids out of range:
    results are unspecified, but the call ends, its counters are zero again,
    and the next call is right."""
    rng = np.random.default_rng(9)
    q, K, V, table, q_start, kv = paged(rng, dev, [3, 1, 8], [400, 2000, 64], 8, 2, 64, BF16, 16, garbage=0.0)
    for bad_start, bad_kv, bad_table in (([9, 3, -5, 40], kv, table), (q_start, [1 << 30, -7, 2 ** 31 - 1], table),
                                         (q_start, kv, np.full_like(table, -9)), ([0, 12, 0, 12], kv, table)):
        attend(dev, q, K, V, bad_table, np.array(bad_start, np.int32), np.array(bad_kv), max_q_len=8)
    out, lse = attend(dev, q, K, V, table, q_start, kv)
    o, l, to, tl = ref.attend(f64(q), f64(K), f64(V), table, q_start, kv, 64 ** -0.5, bf16=True)
    within(out, o, to)
    within(lse, l, tl)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_cache_past_32_bits(dev, dtype):
    """Cells whose byte offset passes 2^32 in both caches are written by
    sgmv_rope_append and read by attention."""
    hk, page, D = 8, 64, 128
    pages = (5 << 30) // (hk * page * D * (2 if dtype is BF16 else 4))
    K = torch.zeros(pages, hk, page, D, dtype=dtype, device=dev)
    V = torch.zeros_like(K)
    rng = np.random.default_rng(10)
    new, ctx = [90, 1], [0, 200]
    table = np.array([[pages - 1, pages - 3, -1, -1], [pages - 2, 0, pages - 5, pages - 4]], np.int32)
    total = 90 + 201
    k, v = (torch.tensor(rng.standard_normal((total, hk, D)), dtype=F32).to(dtype).to(dev) for _ in range(2))
    at = [(0, j) for j in range(90)] + [(1, j) for j in range(201)]
    slot = np.array([table[b, j // page] * page + j % page for b, j in at], np.int32)
    sg.sgmv_rope_append(None, None, k, v, K, V, ints([j for _, j in at], dev), ints(slot, dev), None)
    for i in (0, 89, 90, 290):
        assert torch.equal(K[slot[i] // page, :, slot[i] % page], k[i])
        assert torch.equal(V[slot[i] // page, :, slot[i] % page], v[i])
    q = torch.tensor(rng.standard_normal((91, 16, D)), dtype=F32).to(dtype).to(dev)
    q_start, kv = np.array([0, 90, 91], np.int32), np.array([90, 201], np.int32)
    out, lse = attend(dev, q, K, V, table, q_start, kv)
    use = sorted({int(p) for row in table for p in row if p >= 0})
    small = np.array([[use.index(p) if p >= 0 else 0 for p in row] for row in table])
    o, l, to, tl = ref.attend(f64(q), f64(K[use]), f64(V[use]), small, q_start, kv, D ** -0.5, bf16=dtype is BF16)
    within(out, o, to)
    within(lse, l, tl)


def test_graph_of_a_step(dev):
    """A step's write and attention captured in a graph and replayed, with
    eager work between, gives the eager result every time."""
    rng = np.random.default_rng(12)
    q, K, V, table, q_start, kv = paged(rng, dev, [1] * 6, [700, 20, 1500, 33, 4000, 0], 8, 2, 128, BF16, 16, garbage=0.0)
    T = 6
    k, v = (torch.tensor(rng.standard_normal((T, 2, 128)), dtype=F32).to(BF16).to(dev) for _ in range(2))
    slot = ints([table[b, (kv[b] - 1) // 16] * 16 + (kv[b] - 1) % 16 for b in range(T)], dev)
    pos, tab = ints(kv - 1, dev), sg.sgmv_rope_table(5000, 128, device=dev)
    args = (ints(table, dev), ints(q_start, dev), ints(kv, dev))
    qr, out = torch.empty(T, 8, 128, dtype=BF16, device=dev), torch.empty(T, 8, 128, dtype=BF16, device=dev)

    def step():
        sg.sgmv_rope_append(qr, q, k, v, K, V, pos, slot, tab)
        sg.sgmv_paged_attention(out, qr, K, V, *args, 128 ** -0.5, 1)

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        out.zero_()
        K[slot.long() // 16, :, slot.long() % 16] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert float(out.float().sum()) == float(want.float().sum())


# -- the operators together ---------------------------------------------------------
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_serving_layer_against_dense(dev, dtype, window):
    """examples/lora_attention_layer.py: prompts, single tokens, ended requests
    and new ones in their place, with adapters, against a dense recomputation.

    fp32: every stage's sums of up to 256 terms are off by at most 256 2^-24 of
    their terms' sizes, and some eight such stages follow one another. bf16:
    eight roundings of 2^-8 on the way (projections, deltas, rotation, weights,
    output), those before the softmax acting through scores of order one."""
    import importlib.util
    from pathlib import Path
    spec = importlib.util.spec_from_file_location(
        "lora_attention_layer", Path(__file__).resolve().parents[1] / "examples" / "lora_attention_layer.py")
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(256, 8, 2, 64, 16, 4, 6, 64, 16, 256, dtype, dev, window, 3)
    worst, seconds = example.serve(layer, 256, 6, 14, 60)
    assert len(seconds) == 14
    assert worst <= (2.0 ** -4 if dtype is BF16 else 8 * 256 * 2.0 ** -24), worst


def test_slots_are_kept_for_another_stream(dev):
    """A step of another size replaces position and slot; a stream that still
    reads the old ones keeps their memory."""
    cache = sg.PagedKVCache(8, 16, 1, 64, 2, 4, dtype=F32, device=dev)
    x = torch.ones(5, 1, 64, device=dev)
    cache.step(ints([3, 2], dev), 5)
    old = {cache.position.data_ptr(), cache.slot.data_ptr()}
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)   # tens of milliseconds
        cache.append(torch.empty_like(x), x, x, x, None)
    cache.step(ints([1, 1], dev), 2)
    assert not old & {cache.position.data_ptr(), cache.slot.data_ptr()}
    torch.cuda.synchronize()
    assert float(cache.K.sum()) == 5 * 64 and float(cache.V.sum()) == 5 * 64


def test_binding_refusals(dev):
    """What the Python calls refuse before the library is reached."""
    q = torch.zeros(3, 4, 64, dtype=BF16, device=dev)
    K = torch.zeros(5, 2, 16, 64, dtype=BF16, device=dev)
    table, starts, lens = ints(np.zeros((2, 3)), dev), ints([0, 1, 3], dev), ints([1, 2], dev)

    def attend(out=q, q=q, K=K, V=K, table=table, starts=starts, lens=lens, lse=None, ws=None, n=2, scale=0.1):
        return sg.sgmv_paged_attention(out, q, K, V, table, starts, lens, scale, n, lse=lse, workspace_buf=ws)

    attend(out=torch.empty_like(q))
    bad = [dict(out=q[:2]), dict(out=q.float()), dict(K=K.float()), dict(V=K[:4]), dict(K=K[..., :32], V=K[..., :32]),
           dict(table=table[:1]), dict(table=table.long()), dict(starts=starts[:2]), dict(lens=lens.float()),
           dict(lse=torch.zeros(3, 4, dtype=BF16, device=dev)), dict(lse=torch.zeros(4, 3, device=dev)),
           dict(q=q.transpose(0, 1)), dict(q=q.cpu()), dict(q=q.half(), out=q.half(), K=K.half(), V=K.half()), dict(q=None)]
    for b in bad:
        with pytest.raises((ValueError, TypeError, AttributeError)):
            attend(**b)
    for b in (dict(scale=0.0), dict(scale=float("nan")), dict(n=-1), dict(ws=torch.zeros(256, dtype=torch.uint8, device=dev))):
        with pytest.raises(sg.SGMVError):
            attend(**b)

    pos, tab = ints([0, 1, 2], dev), torch.zeros(9, 32, 2, device=dev)

    def rope(q_out=q, q=q, k=K[:3, :, 0], v=K[:3, :, 0], K=K, V=K, pos=pos, slot=pos, tab=tab):
        sg.sgmv_rope_append(q_out, q, k.contiguous() if k is not None else None, v, K, V, pos, slot, tab)

    kv = torch.zeros(3, 2, 64, dtype=BF16, device=dev)
    for b in [dict(q_out=None), dict(k=kv, v=kv[:2]), dict(k=kv, v=kv.float()), dict(k=kv, v=kv, slot=None),
              dict(k=kv, v=kv, slot=pos[:2]), dict(k=kv, v=kv, pos=pos[:2]), dict(k=kv, v=kv, tab=tab[..., :1]),
              dict(k=kv, v=kv, tab=tab.double()), dict(q=None, q_out=None, k=None), dict(k=kv[:, :1], v=kv[:, :1])]:
        with pytest.raises((ValueError, TypeError)):
            rope(**b)

    seq = ints([3, 4], dev)
    with pytest.raises(ValueError):
        sg.sgmv_kv_tables(seq, ints([1], dev), table, 16, pos, ints([0] * 4, dev), ints([0] * 4, dev), starts, lens, pos, pos)
    with pytest.raises(ValueError):
        sg.sgmv_kv_tables(seq, seq, table, 16, pos, ints([0] * 3, dev), ints([0] * 4, dev), starts, lens, pos, pos)
    with pytest.raises(sg.SGMVError):
        sg.sgmv_kv_tables(seq, seq, table, 17, pos, ints([0] * 4, dev), ints([0] * 4, dev), starts, lens, pos, pos)
