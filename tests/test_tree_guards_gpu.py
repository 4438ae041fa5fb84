"""What drafted trees' calls leave alone, whatever their tables hold: caches in
which every element is its own value between guards, and outputs between
guards."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import commit_reference as ref
from .test_tree_gpu import make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


# -- commit ------------------------------------------------------------------------------
class OnDevice:
    """The buffer of `caches` on the GPU, and its K and V as the call takes them."""

    def __init__(self, caches, dtype, dev):
        self.raw = torch.from_numpy(caches.buf.copy()).to(dev)
        slabs = self.raw.view(dtype).view(4, *caches.shape)
        self.K, self.V = (slabs[i] if caches.layers > 1 else slabs[i, 0] for i in (1, 2))

    def now(self):
        return self.raw.cpu().numpy()


KINDS = [(BF16, 16), (F32, 32)]


@pytest.mark.parametrize("dtype,bits", KINDS, ids=["bf16", "f32"])
@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("sizes", [[40, 0, 50], [120], [1, 2, 3, 64, 30]])
def test_commit_with_slots_outside_the_cache(dev, dtype, bits, layers, sizes):
    """Rows whose slots are a little before or behind the cache are left out, and all others go where they should."""
    c = ref.Caches(layers, 8, 2, 16, 8, bits)
    for seed in range(3):
        slot, q_start, path = ref.rising_case(np.random.default_rng(seed), c, sizes)
        x = OnDevice(c, dtype, dev)
        sg.sgmv_kv_commit(x.K, x.V, ints(slot, dev), ints(q_start, dev), ints(path, dev))
        assert np.array_equal(x.now(), ref.commit(c, slot, q_start, path))


@pytest.mark.parametrize("dtype,bits", KINDS, ids=["bf16", "f32"])
@pytest.mark.parametrize("layers", [1, 3])
def test_commit_with_any_device_values(dev, dtype, bits, layers):
    """Paths that fall or leave the request, slots that tokens share or that are any number, starts that decrease: rows
    move within their cache, layer and head, if at all, and nothing outside is touched."""
    c = ref.Caches(layers, 6, 2, 16, 8, bits)
    rng = np.random.default_rng(1)
    for path, q_start in ((rng.integers(-2 ** 30, 2 ** 30, 50), [0, 30, 50]), (np.arange(50)[::-1].copy(), [0, 50, 50]),
                          (np.full(50, 49), [-7, 2 ** 30, 3]), (rng.integers(0, 50, 50), [0, 25, 50])):
        for slot in (rng.integers(-2 ** 31, 2 ** 31, 50), rng.integers(0, 96, 50), rng.integers(-96, 192, 50)):
            x = OnDevice(c, dtype, dev)
            sg.sgmv_kv_commit(x.K, x.V, ints(slot, dev), ints(q_start, dev), ints(path, dev))
            after = x.now()
            assert c.guards_are_left(after) and c.every_piece_is_one_of_its_head(after)


# -- attention ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes,ctx,hq,hk,d", [
    ([9, 6], [30, 20], 4, 4, 64),        # streamed
    ([40, 6], [30, 20], 4, 2, 64),       # tiles, halves of them
    ([60, 20], [300, 20], 8, 2, 72),     # whole tiles, a narrower head
    ([40, 3], [9000, 700], 2, 1, 128)],  # splits, and their sum
    ids=["streamed", "halves", "tiles", "splits"])
def test_attention_with_any_device_values_stays_inside(dev, dtype, sizes, ctx, hq, hk, d):
    """Pages that are not there, starts that decrease or leave the rows, lengths of any size: outputs lie between guards
    that keep their bits, and the operands keep theirs."""
    x, _ = make(dev, np.random.default_rng(7), sizes, ctx, hq, hk, d, dtype, 16)
    T, most = sum(sizes), max(sizes)
    out = torch.full((3, T, hq, d), 99.0, dtype=dtype, device=dev)
    lse = torch.full((3, T, hq), 99.0, device=dev)
    kept = {n: v.clone() for n, v in x.items()}

    def bits(t):
        return t.contiguous().view(torch.uint8)

    for table, q_start, kv_len in ((2 ** 30, [0, sizes[0], T], None), (-1, [0, sizes[0], T], None),
                                   (None, [5, -3, 2 ** 30], None), (None, [0, 2 ** 31 - 1, 3], None),
                                   (None, [-2 ** 31, T, -1], None), (None, [0, sizes[0], T], [2 ** 31 - 1, -2 ** 31]),
                                   (2 ** 31 - 1, [2, 2 ** 30, T], [2 ** 31 - 1, 2 ** 30])):
        y = dict(x, q_start=ints(q_start, dev))
        y["block_table"] = x["block_table"] if table is None else torch.full_like(x["block_table"], table)
        y["kv_len"] = x["kv_len"] if kv_len is None else ints(kv_len, dev)
        for window, sinks in ((0, 0), (most + 10, 3)):
            sg.sgmv_tree_attention(out[1], y["q"], y["K"], y["V"], y["block_table"], y["q_start"], y["kv_len"], y["mask"], 0.125,
                                   most, window=window, sinks=sinks, lse=lse[1])
            assert bool((out[[0, 2]] == 99).all()) and bool((lse[[0, 2]] == 99).all()), (table, q_start, kv_len, window)
    assert all(torch.equal(bits(x[n]), bits(kept[n])) for n in x)
