"""The drafted-tree operators on the GPU against plain 64-bit implementations
(tests/tree_reference.py), to error bounds derived there."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import tree_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def words_tensor(mask, dev):
    return torch.from_numpy(mask.view(np.int32)).to(dev)


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, tol, what=""):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    same = (got == want) | np.isnan(want)  # infinities too
    err = np.where(same, 0.0, np.abs(np.where(same, 0, got) - np.where(same, 0, want)))
    worst = np.max(err - np.where(same, np.inf, tol), initial=-1.0)
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


def starts(parents):
    return np.concatenate([[0], np.cumsum([len(p) for p in parents])]).astype(np.int64)


# -- positions and masks -------------------------------------------------------------
def run_tables(dev, parents, kv, T, words, flat=None):
    flat = np.concatenate(list(parents) + [np.full(T - starts(parents)[-1], 5)]) if flat is None else flat
    position, mask = ints([77] * T, dev), torch.full((T, words), 77, dtype=torch.int32, device=dev)
    sg.sgmv_tree_tables(ints(flat, dev), ints(starts(parents), dev), ints(kv, dev), position, mask)
    want_position, want_mask = ref.tables(parents, kv, T, words)
    assert np.array_equal(position.cpu().numpy(), want_position)
    assert np.array_equal(mask.cpu().numpy().view(np.uint32), want_mask)


@pytest.mark.parametrize("sizes,words,tail", [
    ([1], 1, 0), ([0], 1, 3), ([0, 1, 0, 2], 1, 0), ([32, 33, 31], 2, 5), ([64] * 70, 2, 0), ([255, 256, 257, 1], 9, 1),
    ([1024, 3], 32, 0), ([40, 7, 70], 1, 0), ([1, 1, 1], 4, 0)])
def test_tree_tables(dev, sizes, words, tail):
    rng = np.random.default_rng(sum(sizes) + words)
    parents = [ref.random_tree(rng, n) for n in sizes]
    run_tables(dev, parents, [n + int(rng.integers(0, 5000)) for n in sizes], sum(sizes) + tail, words)


def test_tree_tables_chain_and_odd_parents(dev):
    chain = np.arange(-1, 1023)
    star = np.array([-1] + [0] * 99)
    odd = np.array([0, 1, 0, 7, 3, -9, 2 ** 31 - 1, -2 ** 31, 6, 5])  # own index, later ones and any value: roots
    run_tables(dev, [chain, star, odd], [1024, 4000, 10], 1134, 32)
    run_tables(dev, [odd], [3], 12, 1)  # longer than its cache: positions may be negative, nothing is touched elsewhere


def test_tree_tables_bad_starts(dev):
    """Offsets that decrease or leave the step's rows: nothing outside the outputs is touched."""
    T = 50
    buf = torch.full((3, T), 7, dtype=torch.int32, device=dev)
    sg.sgmv_tree_tables(ints(np.zeros(T), dev), ints([-5, 2 ** 30, 3, 10 ** 6], dev), ints([9, 9, 9], dev), buf[1], buf[1:2].new_zeros(T, 2))
    assert bool((buf[0] == 7).all()) and bool((buf[2] == 7).all())


# -- attention -------------------------------------------------------------------------
def make(dev, rng, sizes, ctx, hq, hk, d, dtype, page, words=None, masks="tree", poison=True, fused=True):
    """A step's operands on the device and as float64, with poison in every cell that no token of a request holds."""
    B, T = len(sizes), sum(sizes)
    kv = [c + n for c, n in zip(ctx, sizes)]
    counts = [-(-x // page) for x in kv]
    pages = sum(counts) + 2
    order = rng.permutation(pages)
    table = np.full((B, max(1, max(counts)) + 1), -7, np.int64)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    gen = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    K, V = (torch.randn(pages, hk, page, d, generator=gen).to(dtype) for _ in range(2))
    if poison:
        held = np.zeros((pages, page), bool)
        for b in range(B):
            j = np.arange(kv[b])
            held[table[b, j // page], j % page] = True
        free = torch.from_numpy(~held)[:, None, :, None].expand_as(K)
        K = torch.where(free, torch.tensor(float("nan"), dtype=dtype), K)
        V = torch.where(free, torch.tensor(float("inf"), dtype=dtype), V)
    rows = torch.randn(T, (hq + 2 * hk) * d if fused else hq * d, generator=gen).to(dtype)
    words = words or max(1, -(-max(sizes + [1]) // 32))
    parents = [ref.random_tree(rng, n) for n in sizes]
    if masks == "tree":
        mask = ref.tables(parents, kv, T, words)[1]
    else:  # any bits, some rows with none
        mask = rng.integers(0, 1 << 32, (T, words), dtype=np.uint64).astype(np.uint32)
        mask[rng.random(T) < 0.3] = 0
    x = dict(q=rows.to(dev)[:, :hq * d].view(T, hq, d), K=K.to(dev), V=V.to(dev), block_table=ints(table, dev),
             q_start=ints(starts(parents), dev), kv_len=ints(kv, dev), mask=words_tensor(mask, dev))
    h = dict(q=f64(rows)[:, :hq * d].reshape(T, hq, d), K=f64(K), V=f64(V), block_table=table, q_start=starts(parents),
             kv_len=kv, mask=mask)
    return x, h


def attend(x, scale, max_q, window=0, sinks=0, **kw):
    out = torch.full_like(x["q"], 99.0, memory_format=torch.contiguous_format)
    lse = torch.full(x["q"].shape[:2], 99.0, device=out.device)
    sg.sgmv_tree_attention(out, x["q"], x["K"], x["V"], x["block_table"], x["q_start"], x["kv_len"], x["mask"], scale, max_q,
                           window=window, sinks=sinks, lse=lse, **kw)
    return out, lse


def check(dev, rng, sizes, ctx, hq, hk, d, dtype, page, window=0, sinks=0, max_q=None, **kw):
    x, h = make(dev, rng, sizes, ctx, hq, hk, d, dtype, page, **kw)
    scale = d ** -0.5
    out, lse = attend(x, scale, max_q or max(sizes), window, sinks)
    want_out, want_lse, tol_out, tol_lse = ref.attend(**h, scale=scale, window=window, sinks=sinks, bf16=dtype == BF16)
    within(out, want_out, tol_out, "out")
    within(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,ctx,hq,hk,d,page", [
    ([1], [0], 4, 4, 64, 16),                              # one token, nothing cached
    ([5], [0], 8, 2, 128, 16),                             # a tree with nothing before it
    ([13, 1, 0, 9], [70, 200, 10, 0], 10, 2, 64, 16),      # streamed; a request without tokens
    ([33, 40], [127, 300], 4, 4, 128, 16),                 # more rows than are streamed, two words
    ([64, 64], [64, 31], 8, 1, 128, 64),                   # 512 rows a request
    ([65, 3, 100], [500, 700, 1], 6, 2, 80, 32),           # tiles and streams in one launch
    ([17], [1000], 7, 1, 96, 128),
    ([200], [90], 4, 2, 72, 256),
    ([31, 2], [33, 250], 3, 3, 8, 16)])
def test_tree_attention(dev, dtype, sizes, ctx, hq, hk, d, page):
    check(dev, np.random.default_rng(sum(sizes) + d), sizes, ctx, hq, hk, d, dtype, page)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,most,ctx,hq,hk,d", [
    (64, 6, 150, 4, 1, 64),       # as many requests as a wave has lanes; up to 24 rows, streamed in bf16
    (65, 9, 90, 2, 2, 64),        # two per lane
    (70, 20, 60, 16, 16, 8),      # more groups than the GPU runs at once, few rows each
    (600, 3, 40, 2, 1, 64),       # more than eight per lane
    (130, 40, 300, 4, 2, 128)])
def test_many_requests(dev, dtype, B, most, ctx, hq, hk, d):
    """Items found among many requests, the longest first; every tenth request without tokens, some without a cache."""
    rng = np.random.default_rng(B)
    sizes = [int(n) if b % 10 else 0 for b, n in enumerate(rng.integers(1, most + 1, B))]
    check(dev, rng, sizes, [int(c) if b % 7 else 0 for b, c in enumerate(rng.integers(0, ctx + 1, B))], hq, hk, d, dtype, 16)


@pytest.mark.parametrize("sizes,ctx", [([6, 3], [3000, 700]), ([30, 2, 9], [2500, 1, 4000])])
def test_splits_beside_whole_groups(dev, sizes, ctx):
    check(dev, np.random.default_rng(sum(ctx)), sizes, ctx, 4, 1, 64, BF16, 16)
    check(dev, np.random.default_rng(sum(ctx)), sizes, ctx, 4, 1, 64, F32, 16)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,ctx,group", [([20, 7], [40, 0], 2), ([60, 90], [0, 100], 1), ([33], [31], 4)])
def test_any_mask(dev, dtype, sizes, ctx, group):
    """Bits of tokens behind the row's own and of tokens that there are not, and rows without any."""
    check(dev, np.random.default_rng(group), sizes, ctx, 2 * group, 2, 64, dtype, 16, masks="any")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,ctx,window,sinks", [
    ([20, 7], [300, 5], 64, 0), ([20, 13], [300, 700], 20, 3), ([70, 90], [400, 40], 100, 1), ([64], [64], 64, 100),
    ([5, 6, 7], [1000, 31, 32], 33, 30), ([40], [500], 10 ** 9, 4)])
def test_tree_window(dev, dtype, sizes, ctx, window, sinks):
    rng = np.random.default_rng(window % 1000 + sinks)
    check(dev, rng, sizes, ctx, 4, 2, 64, dtype, 16, window, sinks)
    check(dev, rng, sizes, ctx, 4, 2, 64, dtype, 32, window, sinks, masks="any")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 40])
def test_long_context_is_split(dev, dtype, n):
    check(dev, np.random.default_rng(n), [n], [9000], 2, 1, 128, dtype, 64)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,ctx", [(9, 50), (70, 50), (9, 9000), (70, 9000)], ids=["9", "70", "9split", "70split"])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(dev, dtype, n, ctx):
    """NaN and infinities in drafted tokens' keys and values, and in a cached value: a row is what the formula says, and
    a row that does not see them is bitwise what it is without them."""
    rng = np.random.default_rng(n)
    x, h = make(dev, rng, [n], [ctx], 4, 2, 64, dtype, 16)
    clean, clean_lse = attend(x, 0.125, n)
    cell = lambda m: (int(h["block_table"][0, (ctx + m) // 16]), (ctx + m) % 16)  # noqa: E731
    hit = [2, n - 1]
    for m, (k, v) in zip(hit, [(None, float("inf")), (float("nan"), 3.0)]):
        p, o = cell(m)
        if k is not None:
            x["K"][p, :, o] = k
        x["V"][p, :, o] = v
    out, lse = attend(x, 0.125, n)
    sees = np.stack([ref.bits_of(h["mask"][i], n) for i in range(n)])
    for i in range(n):
        if not sees[i, hit[0]] and not sees[i, hit[1]]:
            assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i]), i
        elif sees[i, hit[1]]:
            assert bool(out[i].isnan().all()) and bool(lse[i].isnan().all()), i
        else:
            assert bool((out[i] == float("inf")).all()) and torch.equal(lse[i], clean_lse[i]), i


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,ctx", [(9, 300), (70, 300), (9, 9000), (70, 9000)])
def test_cached_values_that_are_not_finite(dev, dtype, n, ctx):
    """A cached infinity that every row sees, in a part of its own where the keys are split, and one that a window hides
    from every row: the first is every row's result in its column, the second nobody's."""
    rng = np.random.default_rng(ctx + n)
    x, h = make(dev, rng, [n], [ctx], 4, 2, 64, dtype, 16)
    cell = lambda j: (int(h["block_table"][0, j // 16]), j % 16)  # noqa: E731
    for window in (0, 200):
        clean, clean_lse = attend(x, 0.125, n, window)
        V = x["V"].clone()
        p, o = cell(ctx - 30)
        V[p, 0, o, 5], V[p, 1, o, 60] = float("-inf"), float("nan")
        hidden = cell(40)
        if window:
            V[hidden[0], :, hidden[1]] = float("nan")
        out, lse = attend(dict(x, V=V), 0.125, n, window)
        assert torch.equal(lse, clean_lse)
        assert bool((out[:, :2, 5] == float("-inf")).all()) and bool(out[:, 2:, 60].isnan().all())
        out[:, :2, 5], out[:, 2:, 60] = clean[:, :2, 5], clean[:, 2:, 60]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_rows_of_no_request_are_left_and_refused_ones_stay_inside(dev, dtype):
    rng = np.random.default_rng(3)
    x, h = make(dev, rng, [40, 6], [30, 20], 4, 2, 64, dtype, 16)
    T = 60
    q = torch.randn(T, 4, 64, device=dev).to(dtype)
    q[:46] = x["q"]
    mask = torch.zeros(T, 2, dtype=torch.int32, device=dev)
    mask[:46] = x["mask"]
    x["q"], x["mask"] = q, mask
    out, lse = attend(x, 0.125, 40)
    assert bool((out[46:] == 99).all()) and bool((lse[46:] == 99).all())
    x["kv_len"] = ints([30, 3], dev)  # the first one's step was refused; the second's cache is shorter than its tokens
    again, _ = attend(x, 0.125, 40)
    assert bool((again[46:] == 99).all())
    x["block_table"].fill_(2 ** 30)  # pages that are not there
    x["q_start"] = ints([5, -3, 2 ** 30], dev)
    attend(x, 0.125, 40)


def test_a_causal_mask_is_the_causal_call(dev):
    """To the bounds of both, a chain of tokens is a chunk."""
    rng = np.random.default_rng(8)
    x, h = make(dev, rng, [70, 20], [200, 300], 8, 2, 128, BF16, 16)
    h["mask"] = ref.tables([np.arange(-1, 69), np.arange(-1, 19)], h["kv_len"], 90, 3)[1]
    x["mask"] = words_tensor(h["mask"], dev)
    out, lse = attend(x, 0.09, 70)
    plain, plain_lse = torch.empty_like(out), torch.empty_like(lse)
    sg.sgmv_paged_attention(plain, x["q"], x["K"], x["V"], x["block_table"], x["q_start"], x["kv_len"], 0.09, 70, lse=plain_lse)
    want, want_lse, tol, tol_lse = ref.attend(**h, scale=0.09, bf16=True)
    within(out, want, tol)
    within(out, f64(plain), 2 * tol)
    within(lse, f64(plain_lse), 2 * tol_lse)


def test_repeated_calls_give_the_same_bits(dev):
    rng = np.random.default_rng(9)
    for sizes, ctx in (([3], [20000]), ([64, 9], [9000, 100])):
        x, _ = make(dev, rng, sizes, ctx, 8, 1, 128, BF16, 64)
        first = attend(x, 0.1, max(sizes))
        for _ in range(5):
            again = attend(x, 0.1, max(sizes))
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("n", [6, 40])
def test_a_cache_past_32_bits(dev, n):
    """Pages whose offsets pass 2^31 elements and 2^32 bytes: attention (streamed and tiled), and the accepted rows' moves."""
    pages, hk, page, d = 20000, 8, 128, 128          # 5.2 GB of K and of V
    if torch.cuda.mem_get_info(dev)[0] < 24 << 30:
        pytest.skip("needs 24 GB of GPU memory")
    rng = np.random.default_rng(n)
    small, h = make(dev, rng, [n], [300], hk, hk, d, BF16, page)
    used = h["block_table"][0, :-(-(300 + n) // page)]
    K, V = (torch.empty(pages, hk, page, d, dtype=BF16, device=dev) for _ in range(2))
    where = pages - 1 - np.arange(len(used)) * 7
    for i, p in enumerate(used):
        K[where[i]], V[where[i]] = small["K"][p], small["V"][p]
    table = np.full((1, 5), -1)
    table[0, :len(used)] = where
    x = dict(small, K=K, V=V, block_table=ints(table, dev))
    got, want = attend(x, 0.1, n), attend(small, 0.1, n)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    slot = where[(300 + np.arange(n)) // page].astype(np.int64) * page + (300 + np.arange(n)) % page
    before = K[slot[3] // page, :, slot[3] % page].clone()
    path = np.full(n, -1)
    path[:2] = [0, 3]
    sg.sgmv_kv_commit(K, V, ints(slot, dev), ints([0, n], dev), ints(path, dev))
    assert torch.equal(K[slot[1] // page, :, slot[1] % page], before)


# -- acceptance ------------------------------------------------------------------------
def accept_case(rng, sizes, ctx, page, agree, vocabulary=50, refused=(), free=7):
    parents = [ref.random_tree(rng, n) for n in sizes]
    T, q_start = sum(sizes), starts(parents)
    kv = [c + (0 if b in refused else n) for b, (n, c) in enumerate(zip(sizes, ctx))]
    counts = [-(-x // page) for x in kv]
    P = sum(counts) + free + 3
    order = rng.permutation(P)
    table = np.full((len(sizes), max([1] + counts)), -1, np.int64)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    head = int(rng.integers(0, P))
    ring = np.full(P, -1, np.int64)
    ring[(head + np.arange(free)) % P] = order[at:at + free]
    token = rng.integers(0, vocabulary, T)
    target = rng.integers(0, vocabulary, T)
    slot = np.full(T, -1, np.int64)
    for b, parent in enumerate(parents):
        q0 = q_start[b]
        for i in range(len(parent)):
            child = [j for j in range(i + 1, len(parent)) if parent[j] == i]
            if child and rng.random() < agree:
                target[q0 + i] = token[q0 + rng.choice(child)]
            if b not in refused:
                j = ctx[b] + i
                slot[q0 + i] = table[b, j // page] * page + j % page
    return dict(parents=parents, token=token, target=target, slot=slot, q_start=q_start, kv_len=kv, page=page,
                block_table=table, ring=ring, pool=[head, free, len(refused), T], T=T)


def run_accept(dev, c, tail=0):
    B, T = len(c["parents"]), c["T"] + tail
    pad = lambda v, x: np.concatenate([v, np.full(tail, x)])  # noqa: E731
    parent = np.concatenate([np.zeros(0, np.int64), *c["parents"]])
    t = dict(path=ints([7] * T, dev), accepted=ints([7] * B, dev), next_token=ints([7] * B, dev), kept_len=ints([7] * B, dev),
             free_pages=ints(c["ring"], dev), pool_out=ints([7] * 4, dev))
    table = ints(c["block_table"], dev).view(B, -1)
    sg.sgmv_tree_accept(ints(pad(parent, 0), dev), ints(pad(c["token"], 1), dev), ints(pad(c["target"], 1), dev),
                        ints(pad(c["slot"], 3), dev), ints(c["q_start"], dev), ints(c["kv_len"], dev), c["page"], table,
                        t["free_pages"], ints(c["pool"], dev), t["pool_out"], t["path"], t["accepted"], t["next_token"], t["kept_len"])
    want = ref.accept(**dict(c, T=T))
    for k, v in want.items():
        assert np.array_equal(t[k].cpu().numpy(), v), k
    assert torch.equal(table, ints(c["block_table"], dev).view(B, -1))
    return want


@pytest.mark.parametrize("B,lo,hi,page,agree,refused", [
    (1, 1, 1, 16, 1.0, ()), (1, 64, 64, 16, 1.0, ()), (3, 0, 5, 16, 0.5, (1,)), (65, 1, 70, 16, 0.8, (0, 64)),
    (300, 1, 30, 32, 0.9, (7, 8, 9)), (7, 200, 400, 16, 1.0, ()), (5, 0, 0, 64, 0.0, ())])
def test_tree_accept(dev, B, lo, hi, page, agree, refused):
    rng = np.random.default_rng(B + hi)
    sizes = [int(n) for n in rng.integers(lo, hi + 1, B)]
    run_accept(dev, accept_case(rng, sizes, [int(x) for x in rng.integers(0, 90, B)], page, agree, refused=refused),
               tail=B % 4)


@pytest.mark.parametrize("sizes,tail", [
    ([64] * 64, 0), ([64] * 64, 1), ([64] * 63 + [0], 64), ([1] * 64, 3), ([1] * 65, 0), ([0] * 31 + [4096], 0), ([17] * 16 + [0] * 3, 2)],
    ids=["4096", "4097", "tail", "64of1", "65of1", "one", "odd"])
def test_accept_of_full_and_empty_workgroups(dev, sizes, tail):
    rng = np.random.default_rng(len(sizes) + tail)
    refused = (2, 5) if len(sizes) > 16 else ()
    run_accept(dev, accept_case(rng, sizes, [int(x) for x in rng.integers(0, 90, len(sizes))], 16, 0.9, refused=refused), tail=tail)


def test_accept_of_large_steps(dev):
    """Chains longer than what is looked at, and many requests' pages that wrap round the ring's end."""
    rng = np.random.default_rng(3)
    c = accept_case(rng, [1030, 3100], [5, 0], 16, 0.0)
    c["parents"] = [np.arange(-1, 1029), np.arange(-1, 3099)]
    c["token"], c["target"] = np.arange(4130), np.arange(1, 4131)
    assert run_accept(dev, c)["accepted"].tolist() == [1024, 1024]
    c = accept_case(rng, [90] * 70, [int(x) for x in rng.integers(0, 50, 70)], 16, 1.0, vocabulary=2, free=0)
    c["pool"][0] = len(c["ring"]) - 2
    run_accept(dev, c)


def test_accept_of_large_steps_with_bad_device_values(dev):
    rng = np.random.default_rng(5)
    c = accept_case(rng, [2100, 2100], [10, 20], 16, 0.7)
    T, big = 4200, 2 ** 30
    guard = torch.full((9, T), 7, dtype=torch.int32, device=dev)
    for parent, q_start, kv, pool in (
            (rng.integers(-big, big, T), [0, 2100, T], [big, -big], [-5, big, 0, 0]),
            (np.arange(T), [-9, big, 3], [0, 5], [big, -1, 0, 0])):
        ring = torch.full((3, len(c["ring"])), 7, dtype=torch.int32, device=dev)
        sg.sgmv_tree_accept(ints(parent, dev), ints(c["token"], dev), ints(c["token"], dev), ints(c["slot"], dev), ints(q_start, dev),
                            ints(kv, dev), 16, ints(c["block_table"], dev), ring[1], ints(pool, dev), guard[1, :4], guard[3],
                            guard[5, :2], guard[5, 2:4], guard[5, 4:6])
        assert bool((ring[[0, 2]] == 7).all())
        assert bool((guard[[0, 2, 4, 6, 7, 8]] == 7).all()) and bool((guard[5, 6:] == 7).all()) and bool((guard[1, 4:] == 7).all())


def test_accept_ties_chain_and_ring(dev):
    rng = np.random.default_rng(2)
    c = accept_case(rng, [90, 8], [10, 0], 16, 1.0, vocabulary=2)      # many children hold the same token: the first
    run_accept(dev, c)
    c = accept_case(rng, [1030], [5], 16, 0.0)                          # a chain, longer than what is looked at
    c["parents"] = [np.arange(-1, 1029)]
    c["token"], c["target"] = np.arange(1030), np.arange(1, 1031)
    assert run_accept(dev, c)["accepted"][0] == 1024
    c = accept_case(rng, [100, 100, 100], [3, 4, 5], 16, 0.0, free=0)   # the pages returned wrap round the ring's end
    c["pool"][0] = len(c["ring"]) - 2
    run_accept(dev, c)
    empty = dict(parents=[], token=np.zeros(0), target=np.zeros(0), slot=np.zeros(0), q_start=np.zeros(1), kv_len=[], page=16,
                 block_table=np.zeros((0, 3)), ring=np.arange(4), pool=[1, 2, 0, 0], T=0)
    t = dict(free_pages=ints(empty["ring"], dev), pool_out=ints([7] * 4, dev))
    none = ints([], dev)
    sg.sgmv_tree_accept(none, none, none, none, ints([0], dev), none, 16, none.view(0, 0), t["free_pages"], ints([1, 2, 0, 0], dev),
                        t["pool_out"], none, none, none, none)
    assert t["pool_out"].tolist() == [1, 2, 0, 0]


def test_accept_with_bad_device_values(dev):
    """Any parents, lengths and pool: nothing outside the outputs is touched (guarded buffers), and the call ends."""
    rng = np.random.default_rng(4)
    c = accept_case(rng, [40, 40], [10, 20], 16, 0.7)
    T, big = 80, 2 ** 30
    guard = torch.full((9, T), 7, dtype=torch.int32, device=dev)
    for parent, q_start, kv, pool in (
            (rng.integers(-big, big, T), [0, 40, 80], [big, -big], [-5, big, 0, 0]),
            (np.arange(T), [-9, big, 3], [0, 5], [big, -1, 0, 0]),
            (np.zeros(T), [0, 80, 80], [3, 2 ** 31 - 1], [0, len(c["ring"]), 0, 0])):
        ring = torch.full((3, len(c["ring"])), 7, dtype=torch.int32, device=dev)
        sg.sgmv_tree_accept(ints(parent, dev), ints(c["token"], dev), ints(c["token"], dev), ints(c["slot"], dev), ints(q_start, dev),
                            ints(kv, dev), 16, ints(c["block_table"], dev), ring[1], ints(pool, dev), guard[1, :4], guard[3],
                            guard[5, :2], guard[5, 2:4], guard[5, 4:6])
        assert bool((ring[[0, 2]] == 7).all())
        assert bool((guard[[0, 2, 4, 6, 7, 8]] == 7).all()) and bool((guard[5, 6:] == 7).all()) and bool((guard[1, 4:] == 7).all())


# -- commit ------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layers,hk,d,page,B", [(0, 2, 128, 16, 3), (1, 3, 8, 16, 5), (4, 8, 64, 32, 70), (2, 32, 128, 16, 9), (3, 5, 80, 64, 2)])
def test_kv_commit(dev, dtype, layers, hk, d, page, B):
    """layers 0: one layer's cache, without the dimension."""
    rng = np.random.default_rng(B + d)
    sizes = [int(n) for n in rng.integers(0, 150, B)]
    T, cells = sum(sizes), (sum(sizes) // page + 3) * page
    slot = rng.permutation(cells)[:T]
    slot[rng.random(T) < 0.03] = -1
    slot[rng.random(T) < 0.03] = cells + 5
    path = np.full(T, -1, np.int64)
    q_start = np.concatenate([[0], np.cumsum(sizes)])
    shape = (cells // page, hk, page, d)
    K, V = (torch.randn(*((layers,) if layers else ()), *shape, device=dev).to(dtype) for _ in range(2))
    want = [f64(K).reshape(-1, *shape), f64(V).reshape(-1, *shape)]
    for b, n in enumerate(sizes):
        take = np.sort(rng.permutation(n)[:rng.integers(0, n + 1)]) if b % 3 else np.arange(rng.integers(0, n + 1))
        path[q_start[b]:q_start[b] + len(take)] = take
        for x in want:
            old = x.copy()
            for i, m in enumerate(take):
                src, dst = slot[q_start[b] + m], slot[q_start[b] + i]
                if 0 <= src < cells and 0 <= dst < cells:
                    x[:, dst // page, :, dst % page] = old[:, src // page, :, src % page]
    sg.sgmv_kv_commit(K, V, ints(slot, dev), ints(q_start, dev), ints(path, dev))
    assert np.array_equal(f64(K).reshape(want[0].shape), want[0]) and np.array_equal(f64(V).reshape(want[1].shape), want[1])


def test_commit_with_bad_device_values(dev):
    buf = torch.full((4, 6, 2, 16, 8), 7.0, device=dev)
    rng = np.random.default_rng(1)
    for path, q_start in ((rng.integers(-2 ** 30, 2 ** 30, 50), [0, 30, 50]), (np.arange(50)[::-1].copy(), [0, 50, 50]),
                          (np.full(50, 49), [-7, 2 ** 30, 3])):
        sg.sgmv_kv_commit(buf[1], buf[2], ints(rng.integers(-2 ** 31, 2 ** 31, 50), dev), ints(q_start, dev), ints(path, dev))
        sg.sgmv_kv_commit(buf[1], buf[2], ints(rng.integers(0, 96, 50), dev), ints(q_start, dev), ints(path, dev))
    assert bool((buf == 7).all())


# -- refusals ------------------------------------------------------------------------------
def test_refusals(dev):
    x, _ = make(dev, np.random.default_rng(0), [5], [20], 4, 2, 64, BF16, 16)
    with pytest.raises(sg.SGMVError):
        attend(x, 0.1, 33)                       # a word holds 32 tokens
    with pytest.raises(sg.SGMVError):
        attend(x, 0.1, 5, window=4)
    for bad in (x["mask"][:4], x["mask"].long(), x["mask"][0], x["mask"].cpu()):
        with pytest.raises(ValueError):
            attend(dict(x, mask=bad), 0.1, 5)
    with pytest.raises((ValueError, TypeError)):
        sg.sgmv_kv_commit(x["K"], x["V"].float(), x["q_start"], x["q_start"], x["q_start"])
    with pytest.raises(ValueError):
        sg.sgmv_kv_commit(x["K"].transpose(0, 1), x["V"].transpose(0, 1), x["q_start"], x["q_start"], x["q_start"])
    with pytest.raises(ValueError):
        sg.sgmv_tree_tables(x["q_start"], x["q_start"], x["kv_len"], x["kv_len"], x["mask"])
