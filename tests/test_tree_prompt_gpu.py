"""A prompt chunk, single tokens and a tree in one drafted step: the chunk is a
chain whose targets are its own next tokens, and is kept whole."""
import numpy as np
import pytest
import torch

import segmented_gather_gemm_sgmv_amd as sg

from . import tree_reference as ref
from .test_tree_step_gpu import Model, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


@pytest.mark.parametrize("prompt", [2, 50, 200])
def test_a_prompt_beside_trees_is_kept_whole(dev, prompt):
    rng = np.random.default_rng(prompt)
    layers, vocabulary, pages = 2, 30, 60
    model = Model(dev, vocabulary, 4, 2, 64, layers)
    cache = sg.PagedKVCache(pages, 16, 2, 64, 4, 20, layers, dtype=torch.float32, device=dev)
    seq = [[] for _ in range(4)]

    def run(tokens, parents=None):
        T, most = sum(map(len, tokens)), max(map(len, tokens))
        cache.step(ints([len(t) for t in tokens], dev), T)
        mask = None
        if parents is not None:
            mask = torch.empty(T, -(-most // 32), dtype=torch.int32, device=dev)
            cache.draft(ints(np.concatenate(parents), dev), mask)
        ids = torch.as_tensor(np.concatenate(tokens), device=dev).long()
        outs = []
        for layer in range(layers):
            q = model.q[layer, ids].clone()
            cache.append(q, q, model.k[layer, ids], model.v[layer, ids], model.table, layer=layer)
            outs.append(cache.attend(torch.empty_like(q), q, 0.125, most, layer=layer, mask=mask))
        return outs

    # Request 0 is half way through its prompt, 1 and 2 decode, 3 is new: its whole prompt is in the drafted step.
    before = [rng.integers(0, vocabulary, n) for n in (33, 20, 5, 0)]
    run(before)
    parents = [np.arange(-1, prompt - 1), ref.random_tree(rng, 25), np.array([-1]), np.arange(-1, 39)]
    tokens = [rng.integers(0, vocabulary, len(p)) for p in parents]
    own = [rng.integers(0, vocabulary, len(p)) for p in parents]  # what the model says
    target = [np.concatenate([t[1:], o[-1:]]) if b in (0, 3) else o for b, (t, o) in enumerate(zip(tokens, own))]
    outs = run(tokens, parents)
    T = sum(map(len, tokens))
    path, accepted, nxt = ints([7] * T, dev), ints([7] * 4, dev), ints([7] * 4, dev)
    cache.accept(ints(np.concatenate(parents), dev), ints(np.concatenate(tokens), dev), ints(np.concatenate(target), dev), path,
                 accepted, nxt)
    cache.commit(path)
    walk, count = path.cpu().numpy(), accepted.tolist()
    assert count[0] == prompt and count[2] == 1 and count[3] == 40 and count[1] >= 1
    start = np.concatenate([[0], np.cumsum([len(t) for t in tokens])])
    for b in range(4):
        kept = walk[start[b]:start[b] + count[b]]
        seq[b] = [*before[b], *tokens[b][kept]]
        for layer in range(layers):
            close(outs[layer][start[b] + torch.as_tensor(kept, device=dev).long()], model.dense(layer, seq[b], count[b]))
        assert int(nxt[b]) == target[b][kept[-1]]
    assert cache.kv_len.tolist() == [len(s) for s in seq]
    assert int(cache.pool[1]) == pages - sum(-(-len(s) // 16) for s in seq)
    # and a plain step behind it
    outs = run([np.array([int(x)]) for x in nxt])
    for b in range(4):
        for layer in range(layers):
            close(outs[layer][b:b + 1], model.dense(layer, [*seq[b], int(nxt[b])], 1))
