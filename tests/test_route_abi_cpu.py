"""Refusals of the entry points for several adapters per token, on the CPU:
every call below ends in its argument checks (or is a no-op) before anything is
enqueued."""
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

P = [0x100000 * (i + 1) for i in range(16)]   # fake addresses, never dereferenced
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE = -1, -2, -4, -5, -6


def sort(**kw):
    a = dict(choice=P[0], T=40, k=3, adapters=64, start=P[1], adapter=P[2], S=64, order=P[3], place=P[4], ws=None, ws_bytes=0)
    a.update(kw)
    return sg.lib.sgmv_sort_tokens(*a.values(), None)


def test_sort_refusals():
    for k in ("choice", "start", "adapter", "order", "place"):
        assert sort(**{k: None}) == NULL, k
    for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(T=1 << 24, k=2), dict(adapters=-1), dict(adapters=4097), dict(S=63),
                dict(S=-1), dict(T=20, k=2, S=39)):
        assert sort(**bad) == SHAPE, bad
    need = sg.lib.sgmv_sort_tokens_workspace_bytes(20000, 3, 64)
    assert need > 0
    big = dict(T=20000, ws_bytes=need)
    for bad in (dict(big), dict(big, ws=P[5] + 4), dict(big, ws=P[5], ws_bytes=need - 1)):
        assert sort(**bad) == WORKSPACE, bad


def test_sort_workspace_bytes():
    f = sg.lib.sgmv_sort_tokens_workspace_bytes
    assert f(-1, 1, 4) == 0 and f(4, 0, 4) == 0 and f(4, 65, 4) == 0 and f(4, 1, 4097) == 0 and f(1 << 24, 2, 4) == 0
    assert f(64, 2, 2000) == 0 and f(0, 1, 4) == 0


def spread(**kw):
    a = dict(Xs=P[0], ss=64, rows=90, X=P[1], xs=64, place=P[2], T=40, k=3, d=64, dt=1)
    a.update(kw)
    return sg.lib.sgmv_spread_rows(*a.values(), None)


def combine(**kw):
    a = dict(Y=P[0], ys=64, base=P[1], bs=64, Ys=P[2], ss=64, rows=90, place=P[3], weight=P[4], T=40, k=3, d=64, dt=1)
    a.update(kw)
    return sg.lib.sgmv_combine_rows(*a.values(), None)


def grad(**kw):
    a = dict(dYs=P[0], ds=64, dw=P[1], dY=P[2], ys=64, Ys=P[3], ss=64, rows=90, place=P[4], weight=P[5], T=40, k=3, d=64, dt=1)
    a.update(kw)
    return sg.lib.sgmv_combine_rows_grad(*a.values(), None)


@pytest.mark.parametrize("call,needed,strides", [
    (spread, ("Xs", "X", "place"), ("ss", "xs")),
    (combine, ("Y", "Ys", "place"), ("ys", "bs", "ss")),
    (grad, ("dY", "Ys", "place"), ("ds", "ys", "ss")),
])
def test_rows_refusals(call, needed, strides):
    for k in needed:
        assert call(**{k: None}) == NULL, k
    for bad in [dict(T=-1), dict(rows=-1), dict(k=0), dict(k=65), dict(d=0), dict(d=12), dict(d=-8), dict(T=1 << 24)]:
        assert call(**bad) == SHAPE, bad
    for s in strides:
        assert call(**{s: 56}) == SHAPE and call(**{s: -64}) == SHAPE and call(**{s: 1 << 40}) == SHAPE, s
        assert call(**{s: 68}) == ALIGN and call(dt=0, **{s: 66}) == ALIGN, s
    for k in needed:
        if k != "place":
            assert call(**{k: P[7] + 8}) == ALIGN, k
    assert call(dt=2) == DTYPE
    assert call(T=0, place=None) == 0
    assert call(T=1 << 21, k=8, d=1 << 15, **{s: 1 << 15 for s in strides}) == SHAPE  # more workgroups than a launch holds


def test_rows_left_out():
    assert grad(dYs=None, dw=None) == NULL
    assert combine(base=P[1] + 8) == ALIGN
    assert spread(rows=0, Xs=None) == 0


@pytest.mark.parametrize("call", [
    lambda x, i: sg.sgmv_sort_tokens(i, 4, i[0], i[0], i[0], i),
    lambda x, i: sg.sgmv_spread_rows(x, x, i),
    lambda x, i: sg.sgmv_combine_rows(x, x, i),
    lambda x, i: sg.sgmv_combine_rows_grad(x, x, x, x, i),
])
def test_binding_refuses_host_tensors(call):
    with pytest.raises((ValueError, TypeError)):
        call(torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32))
