"""The paged-cache calls captured into graphs: what a graph holds is its own, in
whatever order and beside whatever it is replayed."""
import gc
import weakref

import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from .test_kv_gpu import BF16, F32, dev, ints, paged  # noqa: F401 (dev: the fixture)

pytestmark = pytest.mark.gpu


def capture(graph, stream=None):
    """torch.cuda.graph, with nothing left whose collection could end a graph while another is captured."""
    gc.collect()
    return torch.cuda.graph(graph, stream=stream)


def attention_case(dev, dtype, seed, new, ctx, hq=8, hk=2, D=56):  # noqa: F811
    rng = np.random.default_rng(seed)
    q, K, V, table, q_start, kv = paged(rng, dev, new, ctx, hq, hk, D, dtype, 16, garbage=0.0)
    out = torch.empty(q.shape, dtype=dtype, device=dev)
    args = (q, K, V, ints(table, dev), ints(q_start, dev), ints(kv, dev), D ** -0.5, max(new))
    return out, args


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_graphs_without_warm_up_replayed_in_any_order(dev, dtype):  # noqa: F811
    """Two graphs captured on one stream that has seen no call before; the
    second is replayed first, eager calls on that stream come between, and at
    the end both are replayed side by side."""
    stream = torch.cuda.Stream(dev)
    cases = [attention_case(dev, dtype, 1, [1, 1, 1], [5000, 2200, 40]), attention_case(dev, dtype, 2, [40, 1], [2600, 3000])]
    known = set(sg._attention_workspaces)
    graphs = []
    for out, args in cases:
        graph = torch.cuda.CUDAGraph()
        with capture(graph, stream):
            sg.sgmv_paged_attention(out, *args)
        graphs.append(graph)
    assert set(sg._attention_workspaces) == known, "a workspace that belongs to a graph is kept for other calls"
    wants = [sg.sgmv_paged_attention(torch.empty_like(out), *args) for out, args in cases]
    assert all(bool(w.isfinite().all()) and float(w.abs().max()) > 0 for w in wants)

    def check(i):
        torch.cuda.synchronize()
        assert torch.equal(cases[i][0], wants[i]), i
        cases[i][0].zero_()

    for i in (1, 0, 1, 1, 0):
        graphs[i].replay()
        check(i)
        with torch.cuda.stream(stream):
            out, args = cases[1 - i]
            sg.sgmv_paged_attention(out, *args)
        check(1 - i)
    side = [torch.cuda.Stream(dev), torch.cuda.Stream(dev)]
    for _ in range(10):
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        check(0)
        check(1)


def test_no_workspace_is_made_for_other_calls_during_a_capture(dev):  # noqa: F811
    stream, x = torch.cuda.Stream(dev), torch.zeros(8, device=dev)
    before = sg.attention_workspace(dev, 24, F32, stream)
    graph = torch.cuda.CUDAGraph()
    with capture(graph, stream):
        x.add_(1)
        with pytest.raises(RuntimeError, match="captured"):
            sg.attention_workspace(dev, 48, F32)
        with pytest.raises(RuntimeError, match="captured"):
            sg.attention_workspace(dev, 48, F32, stream)
        assert sg.attention_workspace(dev, 24, F32) is before
    graph.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 8


def test_captured_call_with_a_workspace_of_the_callers(dev):  # noqa: F811
    out, args = attention_case(dev, BF16, 3, [1, 1], [4000, 90])
    want = sg.sgmv_paged_attention(torch.empty_like(out), *args)
    ws = torch.zeros_like(sg.attention_workspace(dev, 56, BF16))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with capture(graph):
        sg.sgmv_paged_attention(out, *args, workspace_buf=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert int(ws[:sg.SGMV_ATTENTION_COUNTER_BYTES].sum()) == 0 and int(ws.count_nonzero()) > 0


class Layer:
    """One cache and what a step of it reads and writes, at fixed places per number of tokens."""

    def __init__(self, dev):  # noqa: F811
        self.dev, self.B = dev, 3
        self.cache = sg.PagedKVCache(64, 16, 2, 64, self.B, 16, dtype=F32, device=dev)
        self.table = sg.sgmv_rope_table(256, 64, device=dev)
        self.io = {}

    def buffers(self, T):
        if T not in self.io:
            self.io[T] = [torch.zeros(T, h, 64, device=self.dev) for h in (8, 2, 2, 8, 8)]
        return self.io[T]

    def fill(self, T, seed):
        gen = torch.Generator(self.dev).manual_seed(seed)
        for x in self.buffers(T)[:3]:
            x.copy_(torch.randn(x.shape, generator=gen, device=self.dev))

    def step(self, new, T, most):
        q, k, v, turned, out = self.buffers(T)
        self.cache.step(new, T)
        self.cache.append(turned, q, k, v, self.table)
        self.cache.attend(out, turned, 0.125, most)


@pytest.mark.parametrize("warm", [True, False], ids=["warm", "cold"])
def test_captured_steps_between_steps_of_other_sizes(dev, warm):  # noqa: F811
    """Two decode steps in a graph, replayed between eager steps of another
    number of tokens and of the same, against a second cache that takes every
    step eagerly. What the allocator gave out in the meantime is not written."""
    stream = torch.cuda.Stream(dev)
    graphed, eager = Layer(dev), Layer(dev)
    one, chunk = ints([1, 1, 1], dev), ints([9, 0, 4], dev)
    seed = [0]

    def same(T):
        assert torch.equal(graphed.cache.kv_len, eager.cache.kv_len) and torch.equal(graphed.cache.pool, eager.cache.pool)
        assert torch.equal(graphed.cache.block_table, eager.cache.block_table)
        assert torch.equal(graphed.cache.K, eager.cache.K) and torch.equal(graphed.cache.V, eager.cache.V)
        assert torch.equal(graphed.buffers(T)[4], eager.buffers(T)[4])

    def both(T, f):
        seed[0] += 1
        for layer in (graphed, eager):
            layer.fill(T, seed[0])
            f(layer)
        torch.cuda.synchronize()
        same(T)

    both(58, lambda x: x.step(ints([30, 11, 17], dev), 58, 30))
    both(13, lambda x: x.step(chunk, 13, 9))
    if warm:
        stream.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(stream):
            both(3, lambda x: x.step(one, 3, 1))
            both(3, lambda x: x.step(one, 3, 1))
    else:
        graphed.buffers(3)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with capture(graph, stream):
        for _ in range(2):
            graphed.step(one, 3, 1)
    slots = [weakref.ref(graphed.cache.position), weakref.ref(graphed.cache.slot)]
    both(13, lambda x: x.step(chunk, 13, 9))
    both(13, lambda x: x.step(chunk, 13, 9))
    assert all(s() is not None for s in slots), "the graph's position and slot are no longer the cache's"
    others = [torch.full((3,), 77, dtype=torch.int32, device=dev) for _ in range(2000)]

    def two(layer):
        if layer is graphed:
            graph.replay()
        else:
            for _ in range(2):
                layer.step(one, 3, 1)

    for _ in range(3):
        both(3, two)
        both(13, lambda x: x.step(chunk, 13, 9))
        both(13, lambda x: x.step(chunk, 13, 9))
        both(3, lambda x: x.step(one, 3, 1))   # where the graph's slots are
        assert graphed.cache.slot is slots[1]()
        both(3, lambda x: x.step(one, 3, 1))
    assert bool((torch.stack(others) == 77).all())
    assert int(eager.cache.pool[2]) == 0


def test_captured_layer_calls_read_the_next_steps_slots(dev):  # noqa: F811
    """Only the layer's calls are captured: every eager step of that many
    tokens, whatever came between, gives its slots to the graph."""
    graphed, eager = Layer(dev), Layer(dev)
    for x in (graphed, eager):
        x.fill(4, 1)
        x.step(ints([2, 2, 0], dev), 4, 2)
    graph = torch.cuda.CUDAGraph()
    q, k, v, turned, _ = graphed.buffers(4)
    torch.cuda.synchronize()
    with capture(graph):
        graphed.cache.append(turned, q, k, v, graphed.table)
    held = weakref.ref(graphed.cache.slot)
    for x in (graphed, eager):
        x.fill(1, 2)
        x.step(ints([0, 0, 1], dev), 1, 1)
    assert held() is not None
    for x in (graphed, eager):
        x.fill(4, 3)
    graphed.cache.step(ints([1, 1, 2], dev), 4)
    assert graphed.cache.slot is held()
    graph.replay()
    eager.step(ints([1, 1, 2], dev), 4, 2)
    torch.cuda.synchronize()
    assert torch.equal(graphed.cache.K, eager.cache.K) and torch.equal(graphed.cache.V, eager.cache.V)
    assert torch.equal(turned, eager.buffers(4)[3])
