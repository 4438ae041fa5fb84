"""How exactly the attention kernels hold a row's weights, and that a row's bits
are its own: against tests/kv_reference.py, on inputs made so that an error of
the weights is not hidden by the result's own rounding."""
import numpy as np
import pytest
import torch

from . import kv_reference as ref
from .test_kv_gpu import BF16, F32, attend, dev, f64, ints, paged, within  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu

# new, ctx, hq, hk, D: streamed requests, tiled ones, both in a launch, one request alone, split groups
LAYOUTS = [
    ([1, 1], [500, 700], 8, 1, 128),
    ([3, 4], [500, 720], 8, 2, 64),
    ([40, 150], [600, 500], 8, 2, 128),
    ([1, 40, 2], [700, 480, 600], 16, 2, 64),
    ([100], [500], 4, 4, 80),
    ([60, 33], [500, 640], 6, 3, 32),
    ([9], [2000], 32, 2, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,hq,hk,D", LAYOUTS)
def test_weights_hold_16_bits(dev, dtype, new, ctx, hq, hk, D):  # noqa: F811
    """Of 16 neighbouring keys one has the score 0 and the value 1, the others
    the score -t and the value -1. 15 exp(-t) is 1.037, so the result nearly
    cancels and its own rounding is small; and exp(-t) lies near the middle of
    two bf16 values (off by 0.79 * 2^-8), the same way at every key, so weights
    of 8 bits would shift the result by 1.6e-3."""
    t = 2.671875                       # exact in bf16, as are q and k below
    assert abs(float(torch.tensor(np.exp(-t)).bfloat16()) / np.exp(-t) - 1) > 0.75 * 2.0 ** -8
    rng = np.random.default_rng(0)
    q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, hq, hk, D, dtype, 16)
    cell = torch.arange(16, device=dev) % 16 == 0
    K.zero_()
    V.fill_(-1)
    V[:, :, cell] = 1
    K[:, :, ~cell, 0] = -t
    q.zero_()
    q[:, :, 0] = 8
    out, _ = attend(dev, q, K, V, table, q_start, kv, scale=0.125)
    bf16 = dtype is BF16
    o, _, tol, _ = ref.attend(f64(q), f64(K), f64(V), table, q_start, kv, 0.125, bf16=bf16)
    assert np.abs(o).max() < 0.05      # rounded to within 2e-4
    if bf16:                           # the reference's bound grants every weight 2^-8; here 2^-16 (sum w |V| / sum w is 1)
        tol = tol - 1.01 * (ref.U16 - 2.0 ** -16)
    assert tol.max() < 4e-4
    within(out, o, tol, "out")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,hq,hk,D", [([15], [420], 4, 2, 64), ([8, 7], [500, 410], 12, 3, 128),  # streamed in both types
                                             ([60], [400], 4, 2, 64), ([150, 70], [330, 700], 8, 4, 128)])
def test_a_row_is_its_own(dev, dtype, new, ctx, hq, hk, D):  # noqa: F811
    """The last token's key, whatever it holds, leaves the bits of the tokens
    before it as they are. Scores grow along the context (by less than the
    slack within which a reference point may stay), so rows that followed
    another row's change of reference point would be rounded differently."""
    rng = np.random.default_rng(D + len(new))
    q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, hq, hk, D, dtype, 16)
    last = [(table[b, (kv[b] - 1) // 16], (kv[b] - 1) % 16) for b in range(len(new))]
    for b in range(len(new)):
        for j in range(kv[b]):
            K[table[b, j // 16], :, j % 16] *= 0.3 + j / kv[b]
    before = np.concatenate([np.arange(q_start[b], q_start[b + 1] - 1) for b in range(len(new))])
    out, lse = attend(dev, q, K, V, table, q_start, kv)
    for factor in (60.0, -60.0, 1e4):
        K2 = K.clone()
        for page, at in last:
            K2[page, :, at] *= factor
        out2, lse2 = attend(dev, q, K2, V, table, q_start, kv)
        assert not torch.equal(lse, lse2)
        assert torch.equal(lse[before], lse2[before]), factor
        assert torch.equal(out[before], out2[before]), factor
