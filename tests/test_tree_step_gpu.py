"""Whole steps that verify drafted trees, as a server runs them: PagedKVCache with
draft, attend, accept and commit against a dense recomputation of the accepted
sequences; captured and replayed, on side streams, beside other calls."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import tree_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


class Model:
    """q, k and v of a token are rows of random tables, by its id and its position's rotation: what it attends to is then
    known from the accepted tokens alone."""

    def __init__(self, dev, vocabulary, hq, hk, d, layers, dtype=torch.float32):
        gen = torch.Generator(dev).manual_seed(1)
        self.q = torch.randn(layers, vocabulary, hq, d, generator=gen, device=dev).to(dtype)
        self.k, self.v = (torch.randn(layers, vocabulary, hk, d, generator=gen, device=dev).to(dtype) for _ in range(2))
        self.table = sg.sgmv_rope_table(512, d, device=dev)
        self.d, self.group, self.layers = d, hq // hk, layers

    def turned(self, x, position):
        angle = self.table.double()[position]
        cos, sin = angle[..., 0][:, None], angle[..., 1][:, None]
        a, b = x.double()[..., :self.d // 2], x.double()[..., self.d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def dense(self, layer, tokens, last):
        """Attention of the last `last` of a sequence's tokens, in 64 bits."""
        t = torch.as_tensor(tokens, device=self.q.device)
        position = torch.arange(len(tokens), device=t.device)
        k = self.turned(self.k[layer, t], position).repeat_interleave(self.group, 1).transpose(0, 1)
        v = self.v[layer, t].double().repeat_interleave(self.group, 1).transpose(0, 1)
        q = self.turned(self.q[layer, t], position).transpose(0, 1)[:, -last:]
        score = q @ k.transpose(1, 2).contiguous() * self.d ** -0.5
        hidden = position[None, :] > position[-last:, None]
        return (torch.softmax(score.masked_fill(hidden, -torch.inf), -1) @ v.contiguous()).transpose(0, 1)


def close(got, want):
    assert float((got.double() - want).abs().max()) < 2e-5  # binary32, a few hundred keys, values of size 1


def test_drafted_steps_are_plain_decoding(dev):
    """Prompts, then steps of random trees whose accepted tokens grow the sequences; single tokens and ended requests in
    between. Every accepted token's attention is that of its sequence, and no page is lost."""
    rng = np.random.default_rng(0)
    requests, vocabulary, layers, pages = 5, 40, 2, 120
    model = Model(dev, vocabulary, 4, 2, 64, layers)
    cache = sg.PagedKVCache(pages, 16, 2, 64, requests, 30, layers, dtype=torch.float32, device=dev)
    seq = [[] for _ in range(requests)]

    def run(new_tokens, parents=None, ended=()):
        new = [-1 if b in ended else len(t) for b, t in enumerate(new_tokens)]
        T = sum(len(t) for t in new_tokens)
        flat = np.concatenate([np.asarray(t, np.int64) for t in new_tokens])
        cache.step(ints(new, dev), T)
        words = -(-max(new) // 32)
        mask = torch.empty(T, words, dtype=torch.int32, device=dev) if parents is not None else None
        if parents is not None:
            cache.draft(ints(np.concatenate(parents), dev), mask)
        ids = torch.as_tensor(flat, device=dev)
        outs = []
        for layer in range(layers):
            q = model.q[layer, ids].clone()
            cache.append(q, q, model.k[layer, ids], model.v[layer, ids], model.table, layer=layer)
            outs.append(cache.attend(torch.empty_like(q), q, model.d ** -0.5, max(new), layer=layer, mask=mask))
        return flat, outs

    for step in range(12):
        ended = [b for b in range(requests) if seq[b] and step > 2 and rng.random() < 0.1]
        for b in ended:
            seq[b] = []
        fresh = {b: rng.integers(0, vocabulary, rng.integers(1, 50)).tolist() for b in range(requests)
                 if not seq[b] and b not in ended}
        if fresh or step % 4 == 3:  # a plain step: prompts, single tokens beside them
            tokens = [fresh.get(b, [] if b in ended else [int(rng.integers(0, vocabulary))]) for b in range(requests)]
            _, outs = run(tokens, ended=ended)
            at = 0
            for b, t in enumerate(tokens):
                seq[b] = seq[b] + t
                for layer in range(layers):
                    if t:
                        close(outs[layer][at:at + len(t)], model.dense(layer, seq[b], len(t)))
                at += len(t)
            continue
        parents = [np.zeros(0, np.int32) if b in ended else ref.random_tree(rng, int(rng.integers(1, 60))) for b in range(requests)]
        tokens = [rng.integers(0, vocabulary, len(p)).tolist() for p in parents]
        flat, outs = run(tokens, parents, ended)
        target = rng.integers(0, vocabulary, len(flat))
        start = np.concatenate([[0], np.cumsum([len(p) for p in parents])])
        for b, p in enumerate(parents):  # the model agrees with a drafted child more often than chance
            for i in range(len(p)):
                child = np.flatnonzero(p == i)
                if len(child) and rng.random() < 0.8:
                    target[start[b] + i] = flat[start[b] + rng.choice(child)]
        path, accepted, nxt = ints([7] * len(flat), dev), ints([7] * requests, dev), ints([7] * requests, dev)
        cache.accept(ints(np.concatenate(parents), dev), ints(flat, dev), ints(target, dev), path, accepted, nxt)
        cache.commit(path)
        walks, counts = path.cpu().numpy(), accepted.cpu().numpy()
        for b, p in enumerate(parents):
            walk = walks[start[b]:start[b] + counts[b]]
            assert len(p) == 0 or (counts[b] >= 1 and walk[0] == 0)
            seq[b] = seq[b] + [int(flat[start[b] + i]) for i in walk]
            for layer in range(layers):
                if len(walk):
                    close(outs[layer][start[b] + torch.as_tensor(walk, device=dev).long()], model.dense(layer, seq[b], len(walk)))
            if len(walk):
                assert int(nxt[b]) == target[start[b] + walk[-1]]
        lengths = cache.kv_len.cpu().numpy()
        assert [int(x) for x in lengths] == [len(s) for s in seq]
        assert int(cache.pool[1]) == pages - sum(-(-len(s) // 16) for s in seq), "pages lost or doubled"
        held = [int(p) for b in range(requests) for p in cache.block_table[b, :-(-len(seq[b]) // 16)].cpu()]
        free = [int(cache.free_pages[(int(cache.pool[0]) + i) % pages]) for i in range(int(cache.pool[1]))]
        assert sorted(held + free) == list(range(pages))


def drafted_step(dev, B=3, n=20, layers=2):
    """A cache with prompts, and a function that runs one drafted step on it from static inputs."""
    rng = np.random.default_rng(4)
    model = Model(dev, 50, 4, 2, 64, layers)
    cache = sg.PagedKVCache(60, 16, 2, 64, B, 20, layers, dtype=torch.float32, device=dev)
    prompt = torch.as_tensor(rng.integers(0, 50, B * 30), device=dev)
    cache.step(ints([30] * B, dev), B * 30)
    for layer in range(layers):
        q = model.q[layer, prompt].clone()
        cache.append(q, q, model.k[layer, prompt], model.v[layer, prompt], model.table, layer=layer)
    T = B * n
    x = dict(new=ints([n] * B, dev), parent=ints(np.concatenate([ref.random_tree(rng, n) for _ in range(B)]), dev),
             token=ints(rng.integers(0, 3, T), dev), target=ints(rng.integers(0, 3, T), dev),
             mask=torch.zeros(T, 1, dtype=torch.int32, device=dev), path=ints([0] * T, dev), accepted=ints([0] * B, dev),
             next=ints([0] * B, dev), out=[torch.zeros(T, 4, 64, device=dev) for _ in range(layers)])

    def step():
        cache.step(x["new"], T)
        cache.draft(x["parent"], x["mask"])
        ids = x["token"].long()
        for layer in range(layers):
            q = model.q[layer].index_select(0, ids)
            cache.append(q, q, model.k[layer].index_select(0, ids), model.v[layer].index_select(0, ids), model.table, layer=layer)
            cache.attend(x["out"][layer], q, 0.125, n, layer=layer, mask=x["mask"])
        cache.accept(x["parent"], x["token"], x["target"], x["path"], x["accepted"], x["next"])
        cache.commit(x["path"])

    def state():
        return [t.clone() for t in (cache.K, cache.V, cache.kv_len, cache.pool, cache.free_pages, cache.block_table, x["mask"],
                                    x["path"], x["accepted"], x["next"], *x["out"])]

    def restore(saved):
        for t, s in zip((cache.K, cache.V, cache.kv_len, cache.pool, cache.free_pages, cache.block_table), saved):
            t.copy_(s)
    return step, state, restore, x


def test_a_captured_step_replays(dev):
    """One drafted step is an even number of changes: it is captured by itself, and replayed between eager work, every
    replay from other tokens."""
    step, state, restore, x = drafted_step(dev)
    before = state()
    step()  # eager, so that what the library keeps is there
    torch.cuda.synchronize()
    restore(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(4):
        rng = np.random.default_rng(replay)
        x["token"].copy_(ints(rng.integers(0, 3, x["token"].numel()), dev))
        x["target"].copy_(ints(rng.integers(0, 3, x["token"].numel()), dev))
        restore(before)
        step()
        want = state()
        restore(before)
        graph.replay()
        torch.cuda.synchronize()
        for i, (g, w) in enumerate(zip(state(), want)):
            assert torch.equal(g, w), (replay, i)


def test_two_attention_graphs_replay_beside_each_other(dev):
    """Captured tree attention over a context that is split: graphs have workspaces of their own."""
    from .test_tree_gpu import attend, make
    x, _ = make(dev, np.random.default_rng(5), [20], [9000], 4, 1, 64, torch.bfloat16, 64)
    y, _ = make(dev, np.random.default_rng(6), [20], [7000], 4, 1, 64, torch.bfloat16, 64)
    want = [attend(z, 0.125, 20)[0].clone() for z in (x, y)]
    graphs, outs = [], []
    for z in (x, y):
        out = torch.empty_like(want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sg.sgmv_tree_attention(out, z["q"], z["K"], z["V"], z["block_table"], z["q_start"], z["kv_len"], z["mask"], 0.125, 20)
        graphs.append(g)
        outs.append(out)
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
        eager = attend(x, 0.125, 20)[0]
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])


def test_routing_is_captured(dev):
    rng = np.random.default_rng(7)
    T, k, P, d = 6000, 2, 300, 64
    choice, weight = ints(rng.integers(-1, P, (T, k)), dev), torch.rand(T, k, device=dev)
    X = torch.randn(T, d, device=dev)
    S = P
    t = dict(start=ints([0] * (S + 1), dev), adapter=ints([0] * S, dev), order=ints([0] * T * k, dev), place=ints(np.zeros((T, k)), dev),
             Xs=torch.zeros(T * k, d, device=dev), Y=torch.zeros(T, d, device=dev), dYs=torch.zeros(T * k, d, device=dev),
             dw=torch.zeros(T, k, device=dev))

    def run():
        sg.sgmv_sort_tokens(choice, P, t["start"], t["adapter"], t["order"], t["place"])
        sg.sgmv_spread_rows(t["Xs"], X, t["place"])
        sg.sgmv_combine_rows(t["Y"], t["Xs"], t["place"], weight)
        sg.sgmv_combine_rows_grad(t["dYs"], t["dw"], X, t["Xs"], t["place"], weight)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for replay in range(4):
        choice.copy_(ints(rng.integers(-1, P, (T, k)), dev))
        for v in t.values():
            v.zero_()
        run()
        want = {n: v.clone() for n, v in t.items()}
        for v in t.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t[n], want[n]) for n in t), replay


def test_on_a_stream_of_the_callers(dev):
    """stream=: the calls run behind what that stream holds, and the workspace of the sort belongs to it."""
    rng = np.random.default_rng(8)
    side = torch.cuda.Stream()
    T, P = 30000, 50
    choice_host = rng.integers(0, P, (T, 1))
    choice = torch.full((T, 1), -1, dtype=torch.int32, device=dev)
    out = [ints(np.zeros(n), dev) for n in ((P + 1,), (P,), (T,), (T, 1))]
    parent, kv = ints(np.arange(-1, 63), dev), ints([64], dev)
    position, mask = ints([0] * 64, dev), torch.zeros(64, 2, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        choice.copy_(torch.from_numpy(choice_host.astype(np.int32)).pin_memory(), non_blocking=True)
    sg.sgmv_sort_tokens(choice, P, *out, stream=side)
    sg.sgmv_tree_tables(parent, ints([0, 64], dev), kv, position, mask, stream=side.cuda_stream)
    side.synchronize()
    assert np.array_equal(out[2].cpu().numpy(), np.argsort(choice_host.reshape(-1), kind="stable"))
    assert position.tolist() == list(range(64))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_on_a_device_that_is_not_current():
    other = torch.device("cuda", 1)
    test_drafted_steps_are_plain_decoding(other)


def test_operands_of_two_devices_are_refused(dev):
    x = torch.zeros(4, 64, device=dev)
    with pytest.raises((ValueError, TypeError)):
        sg.sgmv_spread_rows(x, x, torch.zeros(4, 1, dtype=torch.int32))
