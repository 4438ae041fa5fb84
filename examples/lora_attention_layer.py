"""The attention half of a decoder layer served to requests with adapters of
their own: a few prompts, then single tokens, requests that end and others
that take their place.

    python examples/lora_attention_layer.py            # 7B-wide layer, bf16
    python examples/lora_attention_layer.py --small    # a narrow one in fp32

Per step: q/k/v projections (torch matmul) with every request's LoRA deltas in
one launch (sgmv_fused_layer, the batch left in token order), slots for the
step's tokens (PagedKVCache.step), rotation and cache write, attention over
the cache, o projection with its deltas (sgmv_fused_gather). At the end every
token's output is compared with a dense recomputation in 64 bits.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_gemm_sgmv_amd as sg  # noqa: E402


class Layer:
    """Random weights and adapters of one layer, and its cache."""

    def __init__(self, hidden, heads, kv_heads, head_dim, rank, adapters, requests, pages, page_size, max_len, dtype,
                 device, window, sinks, seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=gen, device=device) * std).to(dtype)

        self.heads, self.kv_heads, self.head_dim, self.rank, self.alpha = heads, kv_heads, head_dim, rank, 2.0 * rank
        self.dtype, self.device, self.window, self.sinks, self.base = dtype, device, window, sinks, 10000.0
        self.widths = {"q": heads * head_dim, "k": kv_heads * head_dim, "v": kv_heads * head_dim}
        self.W = {n: normal(hidden, w, std=hidden ** -0.5) for n, w in self.widths.items()}
        self.W["o"] = normal(heads * head_dim, hidden, std=(heads * head_dim) ** -0.5)
        self.A = {n: normal(adapters, rank, w.shape[0], std=w.shape[0] ** -0.5) for n, w in self.W.items()}
        self.B = {n: normal(adapters, rank, w.shape[1], std=0.3 * rank ** -0.5) for n, w in self.W.items()}
        self.A_ptrs = {n: sg.sgmv_pool_pointers(a) for n, a in self.A.items()}
        self.B_ptrs = {n: sg.sgmv_pool_pointers(b) for n, b in self.B.items()}
        self.table = sg.sgmv_rope_table(max_len, head_dim, self.base, device=device)
        self.cache = sg.PagedKVCache(pages, page_size, kv_heads, head_dim, requests, -(-max_len // page_size),
                                     dtype=dtype, device=device)

    def step(self, x, token_adapter, new_len):
        """x [T, hidden]: the step's tokens, request after request."""
        T, D = x.shape[0], self.head_dim
        perm, seg_start, seg_adapter = sg.sgmv_build_segments(token_adapter)
        rows, seg_start, seg_adapter, lens = (torch.from_numpy(np.asarray(a, np.int32)).to(self.device)
                                              for a in (perm, seg_start, seg_adapter, new_len))
        y = {n: x @ self.W[n] for n in "qkv"}
        sg.sgmv_fused_layer([(y[n], x, self.A_ptrs[n], self.B_ptrs[n]) for n in "qkv"], seg_start, seg_adapter,
                            self.rank, self.alpha, rows=rows)
        q, k, v = (y[n].view(T, -1, D) for n in "qkv")
        self.cache.step(lens, T)
        self.cache.append(q, q, k, v, self.table)
        out = torch.empty_like(q)
        self.cache.attend(out, q, D ** -0.5, int(max(new_len)), self.window, self.sinks)
        out = out.view(T, -1)
        z = out @ self.W["o"]
        sg.sgmv_fused_gather(z, out, rows, self.A_ptrs["o"], self.B_ptrs["o"], seg_start, seg_adapter, self.rank,
                             self.alpha)
        return z

    def dense(self, x, adapter):
        """One request's whole sequence in 64 bits."""
        x = x.double()
        n, D = x.shape[0], self.head_dim

        def project(name, t):
            delta = t @ self.A[name][adapter].double().T @ self.B[name][adapter].double()
            return t @ self.W[name].double() + self.alpha / self.rank * delta

        q, k, v = (project(name, x).view(n, -1, D).transpose(0, 1) for name in "qkv")
        pos = torch.arange(n, device=x.device)
        angle = pos[:, None].double() * self.base ** (-torch.arange(D // 2, device=x.device).double() * 2 / D)
        cos, sin = angle.cos(), angle.sin()

        def turn(t):
            a, b = t[..., :D // 2], t[..., D // 2:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

        group = self.heads // self.kv_heads
        k, v = turn(k).repeat_interleave(group, 0), v.repeat_interleave(group, 0)
        score = turn(q) @ k.transpose(1, 2).contiguous() * D ** -0.5
        hidden = pos[None, :] > pos[:, None]
        if self.window:
            hidden |= (pos[None, :] <= pos[:, None] - self.window) & (pos[None, :] >= self.sinks)
        weight = torch.softmax(score.masked_fill(hidden, -torch.inf), -1)
        return project("o", (weight @ v.contiguous()).transpose(0, 1).reshape(n, -1))


def serve(layer: Layer, hidden: int, requests: int, steps: int, prompt: int, seed: int = 1):
    """Random traffic; returns the worst relative error (2-norm) of a request's
    outputs against the dense recomputation, and the seconds per step."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(layer.device).manual_seed(seed)
    live, done = {}, []
    seconds = []
    for step in range(steps):
        new = np.zeros(requests, np.int64)
        for b in range(requests):
            if b in live and step > 1 and rng.random() < 0.15:
                done.append(live.pop(b))
                new[b] = -1                       # ended: its pages go back
            elif b in live:
                new[b] = 1
            elif rng.random() < 0.7:
                new[b] = rng.integers(1, prompt + 1)
                live[b] = {"adapter": int(rng.integers(0, layer.A["q"].shape[0])), "x": [], "z": []}
        counts = np.maximum(new, 0)
        x = torch.randn(int(counts.sum()), hidden, generator=gen, device=layer.device).to(layer.dtype)
        adapter = np.concatenate([np.full(counts[b], live[b]["adapter"]) for b in range(requests) if counts[b]]
                                 or [np.zeros(0)]).astype(np.int32)
        if not len(adapter):
            continue
        torch.cuda.synchronize()
        began = time.perf_counter()
        z = layer.step(x, adapter, new)
        torch.cuda.synchronize()
        seconds.append(time.perf_counter() - began)
        assert int(layer.cache.pool[2]) == 0, "the pool is too small for this traffic"
        at = 0
        for b in range(requests):
            if counts[b]:
                live[b]["x"].append(x[at:at + counts[b]])
                live[b]["z"].append(z[at:at + counts[b]])
                at += counts[b]
    worst = 0.0
    for r in done + list(live.values()):
        want, got = layer.dense(torch.cat(r["x"]), r["adapter"]), torch.cat(r["z"]).double()
        worst = max(worst, float((got - want).norm() / want.norm()))
    return worst, seconds


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--small", action="store_true")
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=4)
    a = ap.parse_args()
    hidden, heads, kv_heads, dim = (256, 8, 2, 64) if a.small else (4096, 32, 32, 128)
    dtype = torch.float32 if a.small else torch.bfloat16
    layer = Layer(hidden, heads, kv_heads, dim, 16, 8, 16, 1024, 16, 2048, dtype, torch.device("cuda", 0), a.window, a.sinks)
    worst, seconds = serve(layer, hidden, 16, a.steps, 300)
    print(f"{len(seconds)} steps, median {np.median(seconds) * 1e6:.0f} us; worst relative error {worst:.2e}")


if __name__ == "__main__":
    main()
