"""The paged-cache calls captured into graphs: what a graph holds is its own, in
whatever order and beside whatever it is replayed."""
import gc

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
