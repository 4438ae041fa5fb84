"""Several adapters per token on the GPU: the sort, rows out and back, and their
gradients against plain 64-bit implementations; and a mixture of adapters with
the SGMV calls between them."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from .kv_reference import U16, U32

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


def sort_reference(choice, P, S):
    flat = choice.reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < P), flat, P)
    order = np.argsort(flat, kind="stable")
    N = int((flat < P).sum())
    place = np.empty(len(flat), np.int64)
    place[order] = np.arange(len(flat))
    place[flat == P] = -1
    order[N:] = -1
    used, first = np.unique(flat[flat < P], return_counts=True)
    start, adapter = np.full(S + 1, N), np.zeros(S, np.int64)
    start[:len(used)] = np.concatenate([[0], np.cumsum(first)])[:-1] if len(used) else []
    adapter[:len(used)] = used
    return start, adapter, order, place.reshape(choice.shape)


def run_sort(dev, choice, P, spare=0, **kw):
    T, k = choice.shape
    S = min(P, T * k) + spare
    out = [torch.full(n, 77, dtype=torch.int32, device=dev) for n in ((S + 1,), (S,), (T * k,), (T, k))]
    sg.sgmv_sort_tokens(torch.from_numpy(choice.astype(np.int32)).to(dev), P, *out, **kw)
    return out, sort_reference(choice, P, S)


@pytest.mark.parametrize("T,k,P,absent", [
    (0, 1, 4, 0.0), (1, 1, 1, 0.0), (1, 1, 1, 1.0), (7, 3, 0, 0.0), (63, 1, 5, 0.1), (64, 1, 64, 0.0), (65, 1, 2000, 0.0),
    (64, 2, 64, 0.1), (500, 8, 256, 0.05), (512, 8, 257, 0.0), (513, 8, 3, 0.3), (4097, 1, 1, 0.0), (4583, 4, 2000, 0.05),
    (4583, 8, 1025, 0.0), (66000, 2, 4096, 0.0), (300, 64, 1024, 0.5), (70001, 3, 64, 0.01)])
def test_sort(dev, T, k, P, absent):
    rng = np.random.default_rng(T + k + P)
    choice = rng.integers(0, max(P, 1), (T, k))
    choice[rng.random((T, k)) < 0.3] = P // 2          # one that most take
    choice[rng.random((T, k)) < absent] = -1
    choice[rng.random((T, k)) < absent / 3] = P        # one past the pool's end
    for spare in (0, 3):
        got, want = run_sort(dev, choice, P, spare)
        for g, w, name in zip(got, want, ("seg_start", "seg_adapter", "order", "place")):
            assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("T,k,P", [(1 << 23, 2, 4096), ((1 << 24) - 5, 1, 130)])
def test_sort_of_the_most_choices(dev, T, k, P):
    choice = np.random.default_rng(P).integers(-1, P, (T, k), dtype=np.int32)
    got, want = run_sort(dev, choice, P)
    for g, w, name in zip(got, want, ("seg_start", "seg_adapter", "order", "place")):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("T", [50, 5000])
def test_sort_of_one_choice_is_the_host_grouping(dev, T):
    """With one adapter per token: what sgmv_build_segments gives, and the gathered calls take order as rows."""
    rng = np.random.default_rng(T)
    choice = rng.integers(0, 40, (T, 1))
    (start, adapter, order, _), _ = run_sort(dev, choice, 40)
    perm, seg_start, seg_adapter = sg.sgmv_build_segments(choice.reshape(-1))
    n = len(seg_adapter)
    assert np.array_equal(order.cpu().numpy(), perm)
    assert np.array_equal(start.cpu().numpy()[:n + 1], seg_start) and np.array_equal(adapter.cpu().numpy()[:n], seg_adapter)
    A, B = (torch.randn(40, 16, 64, device=dev).bfloat16() for _ in range(2))
    X, Y = (torch.randn(T, 64, device=dev).bfloat16() for _ in range(2))
    A_ptrs, B_ptrs = sg.sgmv_pool_pointers(A), sg.sgmv_pool_pointers(B)
    by_host = sg.sgmv_fused_gather(Y.clone(), X, ints(perm, dev), A_ptrs, B_ptrs, ints(seg_start, dev), ints(seg_adapter, dev), 16, 32.0)
    by_device = sg.sgmv_fused_gather(Y.clone(), X, order, A_ptrs, B_ptrs, start, adapter, 16, 32.0)
    assert torch.equal(by_host, by_device)


def test_tokens_without_an_adapter_are_left_by_the_gathered_call(dev):
    """Some tokens have no adapter: order, with its -1 past the last row, is still what the gathered calls take."""
    rng = np.random.default_rng(12)
    T, P = 400, 6
    choice = rng.integers(-1, P, (T, 1))
    (start, adapter, order, _), _ = run_sort(dev, choice, P)
    A, B = (torch.randn(P, 16, 64, device=dev).bfloat16() for _ in range(2))
    X, Y = (torch.randn(T, 64, device=dev).bfloat16() for _ in range(2))
    got = sg.sgmv_fused_gather(Y.clone(), X, order, sg.sgmv_pool_pointers(A), sg.sgmv_pool_pointers(B), start, adapter, 16, 16.0)
    k = torch.from_numpy(np.maximum(choice[:, 0], 0)).to(dev)
    v = (X.double()[:, None] * A.double()[k]).sum(-1)
    want = Y.double() + torch.where(torch.from_numpy(choice >= 0).to(dev), (v[..., None] * B.double()[k]).sum(1), 0.0)
    assert torch.equal(got[choice[:, 0] < 0], Y[choice[:, 0] < 0])
    # fp32 sums of the width and the rank, V in 16 bits (2^-16 of the terms), one rounding
    tol = U16 * want.abs() * 1.01 + 2.0 ** -15 * (v.abs()[..., None] * B.double()[k].abs()).sum(1)
    assert bool(((got.double() - want).abs() <= tol).all())


def test_one_adapter_twice(dev):
    """Both of a token's choices may be one adapter: two rows, and both weights."""
    choice = np.array([[3, 3], [1, 3], [3, 1]])
    (start, adapter, order, place), want = run_sort(dev, choice, 5)
    assert np.array_equal(order.cpu().numpy(), want[2]) and adapter.tolist()[:2] == [1, 3] and start.tolist()[:3] == [0, 2, 6]
    X = torch.randn(3, 16, device=dev)
    Xs = sg.sgmv_spread_rows(torch.zeros(6, 16, device=dev), X, place)
    weight = torch.tensor([[1.0, 2.0], [0.5, 0.25], [4.0, 8.0]], device=dev)
    Y = sg.sgmv_combine_rows(torch.empty_like(X), Xs, place, weight)
    assert torch.allclose(Y, X * weight.sum(1, keepdim=True), rtol=4 * U32, atol=0)


def test_sort_takes_any_values(dev):
    rng = np.random.default_rng(0)
    choice = rng.integers(-2 ** 31, 2 ** 31, (3000, 2))
    choice[::7] = rng.integers(0, 9, choice[::7].shape)
    got, want = run_sort(dev, choice, 9)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))


def test_sort_with_a_workspace_of_the_callers(dev):
    rng = np.random.default_rng(1)
    choice = rng.integers(0, 100, (20000, 2))
    need = sg.lib.sgmv_sort_tokens_workspace_bytes(20000, 2, 100)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev)
    got, want = run_sort(dev, choice, 100, workspace_buf=ws)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want)) and bool((ws[need:] == 255).all())
    with pytest.raises(sg.SGMVError):
        run_sort(dev, choice, 100, workspace_buf=ws[:need - 16])


# -- rows --------------------------------------------------------------------------------
def case(dev, rng, T, k, d, dtype, spare=5, wide=0):
    """Places of T tokens' choices in rows of a random order, some absent, some outside; rows wider than d by `wide`."""
    rows = T * k + spare
    place = rng.permutation(rows)[:T * k].reshape(T, k)
    place[rng.random((T, k)) < 0.2] = -1
    odd = rng.random((T, k)) < 0.05
    place[odd] = rng.choice([rows, rows + 7, -2 ** 31, 2 ** 31 - 1], odd.sum())
    gen = torch.Generator().manual_seed(int(rng.integers(1 << 30)))

    def tensor(n):
        return torch.randn(n, d + wide, generator=gen).to(dtype).to(dev)[:, :d]
    weight = torch.randn(T, k, generator=gen).to(dev)
    return place, (place >= 0) & (place < rows), rows, tensor, weight


SHAPES = [(1, 1, 8), (3, 2, 24), (64, 2, 4096), (70, 3, 520), (33, 5, 512), (129, 8, 64), (20, 64, 136), (5, 4, 8192), (300, 1, 1000)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("wide", [0, 16])
def test_spread(dev, dtype, T, k, d, wide):
    place, has, rows, tensor, _ = case(dev, np.random.default_rng(T + d), T, k, d, dtype, wide=wide)
    X, Xs = tensor(T), tensor(rows)
    want = f64(Xs)
    t, j = np.nonzero(has)
    want[place[t, j]] = f64(X)[t]
    sg.sgmv_spread_rows(Xs, X, ints(place, dev))
    assert np.array_equal(f64(Xs), want)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("weighted,base", [(True, None), (False, None), (True, "other"), (True, "self")])
def test_combine(dev, dtype, T, k, d, weighted, base):
    place, has, rows, tensor, weight = case(dev, np.random.default_rng(T + d + 1), T, k, d, dtype, wide=8 if base == "other" else 0)
    Ys, Y = tensor(rows), tensor(T)
    other = tensor(T) if base == "other" else Y if base == "self" else None
    w = f64(weight) if weighted else np.ones((T, k))
    want = np.zeros((T, d)) if other is None else f64(other)
    size = np.abs(want)
    for j in range(k):
        y = np.where(has[:, j, None], f64(Ys)[np.where(has[:, j], place[:, j], 0)], 0.0)
        want, size = want + w[:, j, None] * y, size + np.abs(w[:, j, None] * y)
    sg.sgmv_combine_rows(Y, Ys, ints(place, dev), weight if weighted else None, base=other)
    # k products and sums in fp32, then one rounding
    tol = (U16 if dtype == BF16 else U32) * np.abs(want) * 1.01 + 2 * (k + 1) * U32 * size
    assert np.all(np.abs(f64(Y) - want) <= tol)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,d", SHAPES)
@pytest.mark.parametrize("weighted,which", [(True, "both"), (False, "both"), (True, "rows"), (True, "weights")])
def test_combine_grad(dev, dtype, T, k, d, weighted, which):
    place, has, rows, tensor, weight = case(dev, np.random.default_rng(T + d + 2), T, k, d, dtype, wide=8 if k == 2 else 0)
    Ys, dY, dYs = tensor(rows), tensor(T), tensor(rows)
    want = f64(dYs)
    w = f64(weight) if weighted else np.ones((T, k))
    t, j = np.nonzero(has)
    want[place[t, j]] = w[t, j, None] * f64(dY)[t]
    dots, size = np.zeros((T, k)), np.zeros((T, k))
    dots[t, j] = (f64(dY)[t] * f64(Ys)[place[t, j]]).sum(1)
    size[t, j] = np.abs(f64(dY)[t] * f64(Ys)[place[t, j]]).sum(1)
    dweight = torch.full((T, k), 99.0, device=dev)
    both = which == "both"
    sg.sgmv_combine_rows_grad(dYs if both or which == "rows" else None, dweight if both or which == "weights" else None, dY,
                              Ys if which != "rows" else None, ints(place, dev), weight if weighted else None)
    if which != "weights":  # one product, rounded to fp32 and to the type
        assert np.all(np.abs(f64(dYs) - want) <= ((U16 if dtype == BF16 else 0) + U32) * np.abs(want) * 1.01)
    if which != "rows":     # a sum of d products, in any order
        assert np.all(np.abs(f64(dweight) - dots) <= (d + 2) * U32 * size)


def test_gradients_are_those_of_differences(dev):
    """combine is linear in the rows and in the weights: differences along a direction are exact but for rounding."""
    rng = np.random.default_rng(5)
    place, has, rows, tensor, weight = case(dev, rng, 40, 3, 64, F32)
    Ys, G, step, wstep = tensor(rows), tensor(40), tensor(rows), torch.randn(40, 3, device=dev)
    p = ints(place, dev)

    def value(y, w):
        return float((sg.sgmv_combine_rows(torch.empty_like(G), y, p, w).double() * G.double()).sum())

    dYs, dweight = torch.zeros_like(Ys), torch.zeros_like(weight)
    sg.sgmv_combine_rows_grad(dYs, dweight, G, Ys, p, weight)
    for got, diff in ((float((dYs.double() * step.double()).sum()), value(Ys + step, weight) - value(Ys, weight)),
                      (float((dweight.double() * wstep.double()).sum()), value(Ys, weight + wstep) - value(Ys, weight))):
        # every value is a sum of some 40 * 64 * 3 terms of size ~ 1, each off by a few 2^-24
        assert abs(got - diff) < 40 * 64 * 3 * 16 * U32
    X, dXs = tensor(40), tensor(rows)
    Xs = sg.sgmv_spread_rows(torch.zeros_like(dXs), X, p)
    dX = sg.sgmv_combine_rows(torch.empty_like(X), dXs, p)
    assert abs(float((Xs.double() * dXs.double()).sum()) - float((X.double() * dX.double()).sum())) < 40 * 64 * 3 * 16 * U32


def test_rows_that_are_not_finite(dev):
    """An absent choice's weight, and rows that no choice has, change nothing; a weight of 0 over an infinity is NaN."""
    Ys = torch.randn(6, 64, device=dev)
    Ys[4], Ys[5] = float("nan"), float("inf")
    place = ints([[0, -1], [1, 5], [2, 5]], dev)
    weight = torch.tensor([[1.0, float("nan")], [1.0, 0.0], [1.0, 1.0]], device=dev)
    Y = sg.sgmv_combine_rows(torch.empty(3, 64, device=dev), Ys, place, weight)
    assert torch.equal(Y[0], Ys[0]) and bool(Y[1].isnan().all()) and bool((Y[2] == float("inf")).all())
    dYs, dweight = torch.full_like(Ys, 9.0), torch.empty(3, 2, device=dev)
    sg.sgmv_combine_rows_grad(dYs, dweight, torch.ones(3, 64, device=dev), Ys, place, weight)
    assert float(dweight[0, 1]) == 0 and bool((dYs[3:5] == 9).all()) and float(dweight[2, 1]) == float("inf")


def test_offsets_past_32_bits(dev):
    """Rows whose offsets pass 2^31 bytes and 2^31 elements, by their stride."""
    free = torch.cuda.mem_get_info(dev)[0]
    if free < 12 << 30:
        pytest.skip("needs 12 GB of GPU memory")
    stride = (1 << 30) + 64
    big = torch.zeros(2 * stride + stride // 8, dtype=BF16, device=dev)
    Xs = big.as_strided((3, 64), (stride, 1))
    X = torch.randn(3, 64, device=dev).bfloat16()
    place = ints([[2], [0], [1]], dev)
    sg.sgmv_spread_rows(Xs, X, place)
    assert torch.equal(Xs[place.view(-1).long()], X)
    assert torch.equal(sg.sgmv_combine_rows(torch.empty_like(X), Xs, place), X)
    assert torch.equal(sg.sgmv_combine_rows(Xs, X, place, base=Xs)[0], (X[2].float() + X[1].float()).bfloat16())


def test_refusals(dev):
    place, _, rows, tensor, weight = case(dev, np.random.default_rng(6), 4, 2, 64, F32)
    X, Xs, p = tensor(4), tensor(rows), ints(place, dev)
    for bad in (lambda: sg.sgmv_spread_rows(Xs.bfloat16(), X, p), lambda: sg.sgmv_spread_rows(Xs, X.half(), p),
                lambda: sg.sgmv_spread_rows(Xs[:, :56], X, p), lambda: sg.sgmv_spread_rows(Xs, X[:3], p),
                lambda: sg.sgmv_spread_rows(Xs, X, p.long()), lambda: sg.sgmv_spread_rows(Xs, X, p.t()),
                lambda: sg.sgmv_combine_rows(X, Xs, p, weight.double()), lambda: sg.sgmv_combine_rows(X, Xs, p, weight[:, :1]),
                lambda: sg.sgmv_combine_rows(X, Xs, p, weight, base=X.bfloat16()),
                lambda: sg.sgmv_combine_rows(X, Xs.t().contiguous().t(), p), lambda: sg.sgmv_combine_rows(X, Xs, p.cpu()),
                lambda: sg.sgmv_combine_rows_grad(None, None, X, Xs, p), lambda: sg.sgmv_combine_rows_grad(Xs, weight, X, None, p),
                lambda: sg.sgmv_combine_rows_grad(Xs, weight, X, Xs[1:], p), lambda: sg.sgmv_sort_tokens(p[0], 4, p, p, p, p)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(sg.SGMVError):
        sg.sgmv_spread_rows(Xs[:, :60], X[:, :60], p)
    with pytest.raises(sg.SGMVError):  # rows that start 4 bytes past a multiple of 16
        sg.sgmv_spread_rows(Xs[:, 1:57], X[:, :56], p)
    with pytest.raises(sg.SGMVError):
        run_sort(dev, np.zeros((4, 2)), 4097)


# -- a mixture of adapters -----------------------------------------------------------------
@pytest.mark.parametrize("dtype,T,d_in,d_out", [(F32, 37, 64, 128), (BF16, 300, 256, 192)])
def test_mixture_of_adapters_and_its_gradients(dev, dtype, T, d_in, d_out):
    """Y = base + sum_j w_j (alpha / r) X A_k B_k over two adapters per token, and the gradients of X and of the weights
    through frozen adapters, against the same in 64 bits."""
    P, k, r, alpha = 9, 2, 16, 24.0
    rng = np.random.default_rng(T)
    gen = torch.Generator(dev).manual_seed(T)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    A, B = normal(P, r, d_in, std=d_in ** -0.5), normal(P, r, d_out, std=r ** -0.5)
    A_ptrs, B_ptrs = sg.sgmv_pool_pointers(A), sg.sgmv_pool_pointers(B)
    X, base, dY = normal(T, d_in), normal(T, d_out), normal(T, d_out)
    choice = np.stack([rng.permutation(P)[:k] for _ in range(T)])
    choice[rng.random((T, k)) < 0.2] = -1
    weight = torch.softmax(torch.randn(T, k, generator=gen, device=dev), 1)
    (start, adapter, order, place), _ = run_sort(dev, choice, P)
    Xs = sg.sgmv_spread_rows(torch.zeros(T * k, d_in, dtype=dtype, device=dev), X, place)
    Ys = sg.sgmv_fused(torch.zeros(T * k, d_out, dtype=dtype, device=dev), Xs, A_ptrs, B_ptrs, start, adapter, r, alpha)
    Y = sg.sgmv_combine_rows(base.clone(), Ys, place, weight, base=base)
    dYs, dweight = torch.zeros_like(Ys), torch.empty_like(weight)
    sg.sgmv_combine_rows_grad(dYs, dweight, dY, Ys, place, weight)
    dXs = sg.sgmv_fused(torch.zeros_like(Xs), dYs, B_ptrs, A_ptrs, start, adapter, r, alpha)
    dX = sg.sgmv_combine_rows(torch.empty_like(X), dXs, place)

    X64, w64 = X.double().requires_grad_(), weight.double().requires_grad_()
    want = base.double()
    for j in range(k):
        at = torch.from_numpy(np.maximum(choice[:, j], 0)).to(dev)
        on = torch.from_numpy(choice[:, j] >= 0).to(dev)
        v = (X64[:, None] * A.double()[at]).sum(-1)
        delta = alpha / r * (v[..., None] * B.double()[at]).sum(1)
        want = want + torch.where(on, w64[:, j], 0.0)[:, None] * delta
    (want * dY.double()).sum().backward()
    # Stored once per step in the type (Xs is exact; Ys or dYs, dXs, the sum), sums of the rank and the width in fp32:
    # four roundings and a part of them, of the results' norms, which the mixture's terms pass by less than 2.
    unit = U16 if dtype == BF16 else U32
    for got, ref in ((Y, want.detach()), (dX, X64.grad), (dweight, w64.grad)):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err < (8 if dtype == BF16 else 64) * unit, err
