"""Row calls that move more than 256 MiB, whose results are written as streams,
and calls just below that: against 64 bits, and against the same rows taken in
smaller calls, bit for bit. The last-level cache holds 256 MiB. And as many
tokens as one launch has workgroups for."""
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from .kv_reference import U16, U32

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LIMIT = 256 << 20


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def tokens_of(rows_each, d, dtype, above):
    """Tokens of a call that moves rows_each rows for each: the most that do not pass the limit, or one more."""
    size = rows_each * d * (2 if dtype == BF16 else 4)
    T = LIMIT // size
    assert T * size <= LIMIT < (T + 1) * size
    return T + above


def case(dev, T, k, d, dtype):
    """Places of T tokens' choices in rows of a random order, a fifth of them absent, some outside; values in each type."""
    gen = torch.Generator(dev).manual_seed(T + d)
    rows = T * k + 3
    place = torch.randperm(rows, generator=gen, device=dev)[:T * k].view(T, k).int()
    draw = torch.rand(T, k, generator=gen, device=dev)
    place = torch.where(draw < 0.2, -1, torch.where(draw < 0.22, rows + 5, place)).int().contiguous()

    def tensor(n):
        return torch.randn(n, d, generator=gen, device=dev).to(dtype)
    return place, (place >= 0) & (place < rows), rows, tensor, torch.randn(T, k, generator=gen, device=dev)


def parts(T):
    """Runs of tokens small enough for a call of each to be below the limit, in any case below."""
    step = T // 3 + 1
    return [slice(i, min(i + step, T)) for i in range(0, T, step)]


ABOVE = pytest.mark.parametrize("above", [0, 1], ids=["below", "above"])
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@TYPES
@ABOVE
@pytest.mark.parametrize("k,d", [(2, 8192), (5, 1000)])
def test_spread(dev, dtype, above, k, d):
    T = tokens_of(k + 1, d, dtype, above)
    place, has, rows, tensor, _ = case(dev, T, k, d, dtype)
    X, Xs = tensor(T), tensor(rows)
    small, want = Xs.clone(), Xs.clone()
    for j in range(k):
        want[place[has[:, j], j].long()] = X[has[:, j]]
    sg.sgmv_spread_rows(Xs, X, place)
    for p in parts(T):
        sg.sgmv_spread_rows(small, X[p], place[p])
    assert torch.equal(Xs, want) and torch.equal(small, want)


@TYPES
@ABOVE
@pytest.mark.parametrize("k,d,weighted,base", [(2, 8192, True, True), (5, 1000, False, False)])
def test_combine(dev, dtype, above, k, d, weighted, base):
    T = tokens_of(k + (2 if base else 1), d, dtype, above)
    place, has, rows, tensor, weight = case(dev, T, k, d, dtype)
    Ys, under = tensor(rows), tensor(T) if base else None
    w = weight if weighted else None
    Y = sg.sgmv_combine_rows(tensor(T), Ys, place, w, base=under)
    small = torch.empty_like(Y)
    for p in parts(T):
        sg.sgmv_combine_rows(small[p], Ys, place[p], None if w is None else w[p], base=None if under is None else under[p])
    assert torch.equal(Y, small)
    for p in parts(T):
        want = under[p].double() if base else torch.zeros(Y[p].shape, dtype=torch.float64, device=dev)
        size = want.abs()
        for j in range(k):
            y = torch.where(has[p, j, None], Ys[torch.where(has[p, j], place[p, j], 0).long()].double(), 0.0)
            y = y * w[p, j, None].double() if weighted else y
            want, size = want + y, size + y.abs()
        # k products and sums in fp32, then one rounding
        tol = (U16 if dtype == BF16 else U32) * want.abs() * 1.01 + 2 * (k + 1) * U32 * size
        assert bool(((Y[p].double() - want).abs() <= tol).all())


@TYPES
@ABOVE
@pytest.mark.parametrize("k,d,which", [(2, 8192, "both"), (5, 1000, "both"), (2, 8192, "rows"), (2, 8192, "weights")])
def test_combine_grad(dev, dtype, above, k, d, which):
    T = tokens_of(k * (2 if which == "both" else 1) + 1, d, dtype, above)
    place, has, rows, tensor, weight = case(dev, T, k, d, dtype)
    Ys, dY, dYs = tensor(rows), tensor(T), tensor(rows)
    left, small, dweight = dYs.clone(), dYs.clone(), torch.full((T, k), 99.0, device=dev)
    small_weight = torch.full_like(dweight, 77.0)

    def call(dYs, dweight, p):
        sg.sgmv_combine_rows_grad(None if which == "weights" else dYs, None if which == "rows" else dweight[p], dY[p],
                                  None if which == "rows" else Ys, place[p], weight[p])

    call(dYs, dweight, slice(0, T))
    for p in parts(T):
        call(small, small_weight, p)
    assert torch.equal(dYs, small)
    if which != "rows":
        assert torch.equal(dweight, small_weight)
    taken = torch.zeros(rows, dtype=torch.bool, device=dev)
    for j in range(k):
        taken[place[has[:, j], j].long()] = True
    assert torch.equal(dYs[~taken], left[~taken]), "rows that no choice has"
    for p in parts(T):
        g = dY[p].double()
        for j in range(k):
            on = has[p, j]
            at = torch.where(on, place[p, j], 0).long()
            if which != "weights":  # one product, rounded to fp32 and to the type
                want = weight[p, j, None].double() * g
                tol = ((U16 if dtype == BF16 else 0) + U32) * want.abs() * 1.01
                assert bool(((dYs[at].double() - want).abs() <= tol)[on].all())
            if which != "rows":  # a sum of d products, in any order
                terms = torch.where(on[:, None], g * Ys[at].double(), 0.0)
                assert bool(((dweight[p, j].double() - terms.sum(1)).abs() <= (d + 2) * U32 * terms.abs().sum(1)).all())


def test_the_most_tokens(dev):
    """The gradient takes a workgroup per token, of which one launch has fewer than 2^24."""
    T, d = (1 << 24) - 1, 8
    gen = torch.Generator(dev).manual_seed(2)
    place = torch.randperm(T, generator=gen, device=dev).int().view(T, 1)
    dY, Ys = (torch.randn(T, d, generator=gen, device=dev) for _ in range(2))
    weight = torch.randn(T, 1, generator=gen, device=dev)
    dYs, dweight = torch.zeros_like(Ys), torch.zeros_like(weight)
    sg.sgmv_combine_rows_grad(dYs, dweight, dY, Ys, place, weight)
    at = place[:, 0].long()
    assert torch.equal(dYs[at], weight * dY)
    terms = dY.double() * Ys[at].double()
    assert bool(((dweight[:, 0].double() - terms.sum(1)).abs() <= (d + 2) * U32 * terms.abs().sum(1)).all())
    with pytest.raises(sg.SGMVError):
        sg.sgmv_combine_rows_grad(None, torch.zeros(T + 1, 1, device=dev), torch.zeros(T + 1, d, device=dev), Ys,
                                  torch.zeros(T + 1, 1, dtype=torch.int32, device=dev))


def test_the_most_segments(dev):
    """2^31 - 1 segments, all but three of them empty."""
    S = 2 ** 31 - 1
    if torch.cuda.mem_get_info(dev)[0] < 24 << 30:
        pytest.skip("needs 24 GB of GPU memory")
    choice = torch.tensor([[3], [1], [3], [-1], [0]], dtype=torch.int32, device=dev)
    start, adapter = (torch.full((n,), 77, dtype=torch.int32, device=dev) for n in (S + 1, S))
    order, place = torch.empty(5, dtype=torch.int32, device=dev), torch.empty_like(choice)
    sg.sgmv_sort_tokens(choice, 4, start, adapter, order, place)
    assert order.tolist() == [4, 1, 0, 2, -1] and place.view(-1).tolist() == [2, 1, 3, -1, 0]
    assert start[:3].tolist() == [0, 1, 2] and adapter[:3].tolist() == [0, 1, 3]
    step = 1 << 28
    assert all(bool((start[max(i, 3):i + step] == 4).all()) for i in range(0, S + 1, step))
    assert all(bool((adapter[max(i, 3):i + step] == 0).all()) for i in range(0, S, step))
