"""What the paged-cache calls do with memory, streams, devices, threads and
arguments, apart from their results."""
import threading
import time

import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from .test_kv_gpu import dev  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_rope_table_is_allocated_on_its_stream(dev, raw):  # noqa: F811
    """Memory freed on the current stream, whose work there may still be
    pending, is not what another stream writes the table to."""
    side = torch.cuda.Stream(dev)
    want = sg.sgmv_rope_table(30011, 128, device=dev)
    ahead = [torch.empty_like(want) for _ in range(3)]
    freed = {x.data_ptr() for x in ahead}
    del ahead
    table = sg.sgmv_rope_table(30011, 128, device=dev, stream=side.cuda_stream if raw else side)
    assert table.data_ptr() not in freed
    torch.cuda.synchronize()
    assert torch.equal(table, want)
    again = torch.empty_like(want)   # those blocks are the current stream's still
    assert again.data_ptr() in freed


def test_a_flag_without_a_truth_value_is_refused(dev):  # noqa: F811
    """The error is the value's own, and nothing is launched."""
    q = torch.ones(3, 2, 64, device=dev)
    out, pos = torch.zeros_like(q), torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(RuntimeError, match="ambiguous"):
        sg.sgmv_rope_append(out, q, None, None, None, None, pos, None, None, torch.zeros(2))
    torch.cuda.synchronize()
    assert float(out.sum()) == 0
    sg.sgmv_rope_append(out, q, None, None, None, None, pos, None, None, torch.ones(1))
    assert torch.equal(out, q)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_a_cache_on_a_device_that_is_not_the_current_one(dev):  # noqa: F811
    """Calls are made on their operands' device, and those of two devices are
    refused (two ranks of one process, or a second model's cache)."""
    here, there = [], []
    for device, results in ((dev, here), (torch.device("cuda", 1), there)):
        gen = torch.Generator("cpu").manual_seed(1)
        cache = sg.PagedKVCache(64, 16, 2, 64, 2, 16, device=device)
        table = sg.sgmv_rope_table(256, 64, device=device)
        for new in ([40, 200], [1, 1]):
            q, k, v = (torch.randn(sum(new), h, 64, generator=gen).bfloat16().to(device) for h in (8, 2, 2))
            cache.step(torch.tensor(new, dtype=torch.int32, device=device), sum(new))
            cache.append(q, q, k, v, table)
            results.append(cache.attend(torch.empty_like(q), q, 0.125, max(new)).cpu())
            assert torch.cuda.current_device() == 0
    for a, b in zip(here, there):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="device"):
        cache.step(torch.tensor([1, 1], dtype=torch.int32, device=dev), 2)
    with pytest.raises(ValueError, match="device"):
        cache.attend(torch.empty_like(q), q.to(dev), 0.125, 1)


def test_other_threads_run_while_a_launch_waits(dev):  # noqa: F811
    """A launch waits while the GPU's queue is full (here: behind half a second
    of other work). Python's other threads go on meanwhile."""
    q, pos = torch.zeros(1, 1, 64, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    sg.sgmv_rope_append(q, q, None, None, None, None, pos, None, None)
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        torch.cuda._sleep(1_200_000_000)
        longest = 0.0
        for _ in range(25000):
            began = time.perf_counter()
            sg.sgmv_rope_append(q, q, None, None, None, None, pos, None, None)
            longest = max(longest, time.perf_counter() - began)
        torch.cuda.synchronize()
    finally:
        stop.set()
        thread.join()
    print(f"longest call {longest * 1e3:.0f} ms, longest gap {gaps[0] * 1e3:.0f} ms")
    assert gaps[0] < max(0.05, longest / 3), (gaps[0], longest)
