"""Attention at every head width that has a kernel of its own or is padded to
one, and the state that calls leave behind: against tests/kv_reference.py."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import kv_reference as ref
from .test_kv_gpu import BF16, F32, check_attention, dev, f64, ints, uniform, within  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def counters_are_zero(dev):  # noqa: F811
    """All counters of every workspace, the streamed items' of a mixed launch among them."""
    yield
    torch.cuda.synchronize()
    for key, ws in sg._attention_workspaces.items():
        assert int(ws[:sg.SGMV_ATTENTION_COUNTER_BYTES].count_nonzero()) == 0, key


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 56, 64, 72, 88, 96, 104, 112, 120, 128])
def test_head_widths(dev, dtype, D):  # noqa: F811
    rng = np.random.default_rng(D)
    check_attention(dev, rng, [1, 3], [200, 77], 8, 2, D, dtype, 16)             # streamed in both types
    check_attention(dev, rng, [45, 2, 70], [60, 300, 0], 6, 2, D, dtype, 32)     # tiles in bf16, and a short request beside them
    check_attention(dev, rng, [90], [130], 4, 1, D, dtype, 16, window=50, sinks=3)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [24, 56, 88, 120])
def test_head_widths_split_over_long_contexts(dev, dtype, D):  # noqa: F811
    uniform(dev, [1, 1], [9000, 30], 8, 2, D, dtype, 16, 0, 0, 1)
    uniform(dev, [60, 1, 2], [5000, 7000, 400], 4, 2, D, dtype, 64, 0, 0, 2)     # tile items and streamed items, both split
    uniform(dev, [80, 1], [4000, 6000], 4, 1, D, dtype, 32, 3000, 70, 3)


def test_a_refused_request_changes_nothing_of_the_others(dev):  # noqa: F811
    """A pool too small for the second request: its slots are -1, its length
    stays, the others are served; offered again when pages are back, it is
    right."""
    rng = np.random.default_rng(7)
    cache = sg.PagedKVCache(6, 16, 2, 64, 3, 8, dtype=F32, device=dev)
    held = [[], [], []]

    def step(new):
        T = sum(max(n, 0) for n in new)
        q, k, v = (torch.tensor(rng.standard_normal((T, h, 64)), dtype=F32, device=dev) for h in (4, 2, 2))
        cache.step(ints(new, dev), T)
        cache.append(q, q, k, v, None)
        out = cache.attend(torch.empty_like(q), q, 0.125, max(new))
        slot, kv, start = cache.slot.tolist(), cache.kv_len.tolist(), cache.q_start.tolist()
        for b, n in enumerate(new):
            rows = slice(start[b], start[b + 1])
            if n < 0:
                held[b] = []
            elif n > 0 and min(slot[rows]) >= 0:
                held[b].append((k[rows], v[rows]))
                K, V = (f64(torch.cat([x[i] for x in held[b]]))[None].transpose(0, 2, 1, 3) for i in (0, 1))
                o, _, tol, _ = ref.attend(f64(q[rows]), K, V, np.zeros((1, 1), int), [0, n], [kv[b]], 0.125)
                within(out[rows], o, tol, (new, b))
            elif n > 0:
                assert set(slot[rows]) == {-1}
                assert kv[b] == sum(len(x[0]) for x in held[b])
        return [slot[start[b]] for b in range(3) if new[b] > 0], int(cache.pool[2])

    assert step([40, 17, 0])[1] == 0                      # 3 + 2 of 6 pages
    slots, refused = step([1, 40, 2])                     # the second needs 2 more pages, the third one
    assert slots[0] >= 0 and slots[1:] == [-1, -1] and refused == 2
    assert step([-1, 1, 0])[1] == 0                       # the first ends, the second goes on in its page
    assert step([0, 40, 2])[1] == 0                       # served from the pages that came back
    assert step([3, 1, 1])[1] == 0
