"""Refusals of the drafted-tree entry points, on the CPU: every call below ends
in its argument checks (or is a no-op) before anything is enqueued."""
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

P = [0x100000 * (i + 1) for i in range(24)]   # fake addresses, never dereferenced
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE = -1, -2, -4, -5, -6


def tables(**kw):
    a = dict(parent=P[0], q_start=P[1], kv_len=P[2], B=4, position=P[3], mask=P[4], words=2, T=50)
    a.update(kw)
    return sg.lib.sgmv_tree_tables(*a.values(), None)


def test_tables_refusals():
    for k in ("parent", "q_start", "kv_len", "position", "mask"):
        assert tables(**{k: None}) == NULL, k
    for bad in (dict(B=-1), dict(B=8193), dict(T=-1), dict(T=(1 << 24) + 1), dict(words=0), dict(words=33), dict(words=-1)):
        assert tables(**bad) == SHAPE, bad
    assert tables(T=0, parent=None, position=None, mask=None) == 0


def attention(**kw):
    a = dict(out=P[0], os=1024, lse=None, q=P[1], qs=1024, hq=8, K=P[2], V=P[3], pages=10, hk=2, page=16, D=128,
             table=P[4], width=8, q_start=P[5], kv_len=P[6], mask=P[8], words=2, B=4, T=90, max_q=64, scale=0.1, window=0,
             sinks=0, dt=1, ws=P[7], ws_bytes=1 << 30)
    a.update(kw)
    return sg.lib.sgmv_tree_attention(*a.values(), None)


def test_attention_refusals():
    for k in ("out", "q", "K", "V", "table", "q_start", "kv_len", "mask"):
        assert attention(**{k: None}) == NULL, k
    for bad in (dict(words=0), dict(words=33), dict(words=-1), dict(words=1), dict(max_q=65), dict(window=63), dict(window=1),
                dict(hq=7), dict(hk=0), dict(D=12), dict(D=136), dict(page=20), dict(pages=0), dict(width=-1),
                dict(width=(1 << 26) + 1), dict(B=-1), dict(B=8193), dict(T=-1), dict(max_q=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(qs=1016), dict(os=8)):
        assert attention(**bad) == SHAPE, bad
    for bad in (dict(q=P[1] + 8), dict(out=P[0] + 8), dict(K=P[2] + 8), dict(V=P[3] + 2), dict(qs=1028), dict(os=1026)):
        assert attention(**bad) == ALIGN, bad
    assert attention(dt=2) == DTYPE
    need = sg.lib.sgmv_paged_attention_workspace_bytes(128, 1)
    for bad in (dict(ws=None), dict(ws=P[7] + 16), dict(ws_bytes=need - 1)):
        assert attention(**bad) == WORKSPACE, bad
    for none in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert attention(**none, q=None, out=None, mask=None, ws=None) == 0, none


def accept(**kw):
    a = dict(parent=P[0], token=P[1], target=P[2], slot=P[3], q_start=P[4], kv_len=P[5], B=4, page=16, table=P[6], width=8,
             free=P[7], pages=10, pool_in=P[8], pool_out=P[9], path=P[10], accepted=P[11], next=P[12], kept=P[13], T=50)
    a.update(kw)
    return sg.lib.sgmv_tree_accept(*a.values(), None)


def test_accept_refusals():
    for k in ("parent", "token", "target", "slot", "q_start", "kv_len", "table", "free", "pool_in", "pool_out", "path",
              "accepted", "next", "kept"):
        assert accept(**{k: None}) == NULL, k
    for bad in (dict(B=-1), dict(B=8193), dict(T=-1), dict(T=(1 << 24) + 1), dict(page=24), dict(page=8), dict(pages=0),
                dict(pages=1 << 28), dict(width=-1), dict(width=1 << 28), dict(B=4096, width=1 << 20)):
        assert accept(**bad) == SHAPE, bad


def commit(**kw):
    a = dict(K=P[0], V=P[1], layers=3, stride=10 * 2 * 16 * 128, pages=10, hk=2, page=16, D=128, slot=P[2], q_start=P[3],
             path=P[4], B=4, T=50, dt=1)
    a.update(kw)
    return sg.lib.sgmv_kv_commit(*a.values(), None)


def test_commit_refusals():
    for k in ("K", "V", "slot", "q_start", "path"):
        assert commit(**{k: None}) == NULL, k
    for bad in (dict(layers=-1), dict(stride=10 * 2 * 16 * 128 - 8), dict(stride=0), dict(stride=1 << 40), dict(pages=0),
                dict(hk=0), dict(hk=65537), dict(page=12), dict(D=0), dict(D=136), dict(D=20), dict(B=-1), dict(B=8193),
                dict(T=-1), dict(T=(1 << 24) + 1), dict(layers=1 << 20, hk=1, pages=1, D=128, stride=16 * 128)):
        assert commit(**bad) == SHAPE, bad
    for bad in (dict(K=P[0] + 8), dict(V=P[1] + 2), dict(stride=10 * 2 * 16 * 128 + 4)):
        assert commit(**bad) == ALIGN, bad
    assert commit(dt=2) == DTYPE
    for none in (dict(layers=0), dict(B=0), dict(T=0)):
        assert commit(**none, slot=None, path=None) == 0, none


@pytest.mark.parametrize("call", [
    lambda x, i: sg.sgmv_tree_tables(i, i, i, i, i[None]),
    lambda x, i: sg.sgmv_tree_attention(x, x, x[None], x[None], i[None], i, i, i[None], 1.0, 1),
    lambda x, i: sg.sgmv_tree_accept(i, i, i, i, i, i, 16, i[None], i, i, i, i, i, i, i),
    lambda x, i: sg.sgmv_kv_commit(x[None], x[None], i, i, i),
])
def test_binding_refuses_host_tensors(call):
    with pytest.raises((ValueError, TypeError)):
        call(torch.zeros(2, 2, 16), torch.zeros(2, dtype=torch.int32))
