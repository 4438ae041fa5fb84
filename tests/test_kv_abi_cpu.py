"""Refusals of the paged-cache entry points, on the CPU: every call below ends
in its argument checks (or is a no-op) before anything is enqueued."""
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

P = [0x100000 * (i + 1) for i in range(16)]   # fake addresses, never dereferenced
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE = -1, -2, -4, -5, -6


def tables(**kw):
    a = dict(seq=P[0], new=P[1], B=4, table=P[2], width=8, page=16, free=P[3], pages=10, pool_in=P[4], pool_out=P[5],
             q_start=P[6], kv_len=P[7], position=P[8], slot=P[9], T=7)
    a.update(kw)
    return sg.lib.sgmv_kv_tables(*a.values(), None)


def test_tables_refusals():
    for k in ("seq", "new", "table", "free", "pool_in", "pool_out", "q_start", "kv_len", "position", "slot"):
        assert tables(**{k: None}) == NULL, k
    for bad in (dict(B=-1), dict(B=8193), dict(width=-1), dict(T=-1), dict(page=0), dict(page=15), dict(page=24),
                dict(page=8), dict(page=512), dict(pages=0), dict(pages=-1), dict(pages=1 << 28), dict(B=4096, T=1 << 20),
                dict(B=4096, width=1 << 20), dict(width=1 << 28)):
        assert tables(**bad) == SHAPE, bad


def rope(**kw):
    a = dict(q_out=P[0], qos=1024, q=P[1], qs=1024, hq=8, k=P[2], ks=256, v=P[3], vs=256, K=P[4], V=P[5], pages=10, hk=2,
             page=16, D=128, position=P[6], slot=P[7], T=3, table=P[8], max_position=100, rot=128, inter=0, dt=1)
    a.update(kw)
    return sg.lib.sgmv_rope_append(*a.values(), None)


def test_rope_refusals():
    for k in ("q_out", "q", "k", "v", "K", "V", "position", "slot", "table"):
        assert rope(**{k: None}) == NULL, k
    for bad in (dict(T=-1), dict(hq=-1), dict(hk=-1), dict(D=0), dict(D=12), dict(D=136), dict(rot=-16), dict(rot=144),
                dict(rot=7), dict(rot=41), dict(page=17), dict(pages=0), dict(qs=1016), dict(qos=0), dict(ks=255),
                dict(vs=128), dict(max_position=-1), dict(T=(1 << 24) + 1), dict(hq=70000, qs=1 << 24, qos=1 << 24)):
        assert rope(**bad) == SHAPE, bad
    for bad in (dict(q=P[1] + 8), dict(q_out=P[0] + 2), dict(k=P[2] + 4), dict(v=P[3] + 8), dict(K=P[4] + 8),
                dict(V=P[5] + 8), dict(table=P[8] + 4), dict(qs=1028), dict(ks=257)):
        assert rope(**bad) == ALIGN, bad
    assert rope(dt=2) == DTYPE
    assert rope(T=0, q=None, k=None) == 0
    assert rope(hq=0, hk=0, q=None, k=None, position=None) == 0


def rope_table(**kw):
    a = dict(table=P[0], n=100, rot=64, base=10000.0, kind=0, factor=1.0, fast=32.0, slow=1.0, orig=0)
    a.update(kw)
    return sg.lib.sgmv_rope_table(*a.values(), None)


def test_rope_table_refusals():
    parts = dict(kind=2, factor=4.0, orig=4096)
    for bad in (dict(n=-1), dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                dict(kind=3), dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=1, factor=float("nan")),
                dict(parts, orig=0), dict(parts, factor=0.5), dict(parts, slow=0.0), dict(parts, fast=1.0)):
        assert rope_table(**bad) == SHAPE, bad
    assert rope_table(table=None) == NULL and rope_table(table=P[0] + 8) == ALIGN
    assert rope_table(n=0, table=None) == 0


def attention(**kw):
    a = dict(out=P[0], os=1024, lse=None, q=P[1], qs=1024, hq=8, K=P[2], V=P[3], pages=10, hk=2, page=16, D=128,
             table=P[4], width=8, q_start=P[5], kv_len=P[6], B=4, T=9, max_q=3, scale=0.1, window=0, sinks=0, dt=1,
             ws=P[7], ws_bytes=1 << 30)
    a.update(kw)
    return sg.lib.sgmv_paged_attention(*a.values(), None)


def test_attention_refusals():
    for k in ("out", "q", "K", "V", "table", "q_start", "kv_len"):
        assert attention(**{k: None}) == NULL, k
    for bad in (dict(hq=7), dict(hq=0), dict(hk=0), dict(hk=-2), dict(D=0), dict(D=12), dict(D=136), dict(page=20),
                dict(pages=0), dict(pages=1 << 28), dict(width=-1), dict(width=1 << 28), dict(B=-1), dict(B=8193),
                dict(T=-1), dict(T=(1 << 24) + 1, hq=2, hk=1), dict(T=1 << 24, hq=256, qs=1 << 20), dict(max_q=-1), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(qs=1016),
                dict(os=8)):
        assert attention(**bad) == SHAPE, bad
    for bad in (dict(q=P[1] + 8), dict(out=P[0] + 8), dict(K=P[2] + 8), dict(V=P[3] + 2), dict(qs=1028), dict(os=1026)):
        assert attention(**bad) == ALIGN, bad
    assert attention(dt=2) == DTYPE and attention(dt=-1) == DTYPE
    need = sg.lib.sgmv_paged_attention_workspace_bytes(128, 1)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=P[7] + 16), dict(ws_bytes=need - 1)):
        assert attention(**bad) == WORKSPACE, bad
    for none in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert attention(**none, q=None, out=None, ws=None) == 0, none


def test_attention_positions_stay_in_31_bits():
    """The end of the key tile past the last position has to be an int too."""
    assert attention(width=(1 << 26) + 1) == SHAPE
    assert attention(width=1 << 26, T=0) == 0


def test_attention_workspace_bytes():
    f = sg.lib.sgmv_paged_attention_workspace_bytes
    assert f(12, 1) == 0 and f(136, 1) == 0 and f(0, 1) == 0 and f(64, 2) == 0
    assert 0 < f(64, 1) <= f(128, 1) and f(80, 0) == f(128, 0)


@pytest.mark.parametrize("call", [
    lambda x: sg.sgmv_paged_attention(x, x, x[None], x[None], x[0], x, x, 1.0, 1),
    lambda x: sg.sgmv_rope_append(x, x, x, x, x[None], x[None], x[0, 0], x[0, 0], None),
    lambda x: sg.sgmv_kv_tables(x, x, x[0], 16, x, x, x, x, x, x, x),
])
def test_binding_refuses_host_tensors(call):
    with pytest.raises((ValueError, TypeError)):
        call(torch.zeros(2, 2, 16, dtype=torch.float32))
