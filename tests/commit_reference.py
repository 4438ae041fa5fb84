"""A host model of sgmv_kv_commit on raw memory, and the checks that its GPU
tests make on what a call leaves behind. K and V lie in one buffer between two
guards, every element its own bit pattern, so that a row that went elsewhere,
into the other cache or out of both shows. No code is shared with the library."""
from __future__ import annotations

import numpy as np

GUARD = -1


class Caches:
    """Slabs [guard, K, V, guard] of one buffer, as integers of an element's size: K's and V's elements are 0, 1, 2, ...
    through both."""

    def __init__(self, layers, pages, heads, page, d, bits):
        self.shape = (layers, pages, heads, page, d)
        self.layers, self.pages, self.heads, self.page, self.d, self.bits = layers, pages, heads, page, d, bits
        self.size = int(np.prod(self.shape))
        assert 2 * self.size < 1 << (bits - 1)
        self.piece = 128 // bits  # elements that move together
        self.buf = np.full(4 * self.size, GUARD, np.int32 if bits == 32 else np.int16)
        self.buf[self.size:3 * self.size] = np.arange(2 * self.size)

    def guards_are_left(self, after):
        return bool((after[:self.size] == GUARD).all() and (after[3 * self.size:] == GUARD).all())

    def every_piece_is_one_of_its_head(self, after):
        """Each 16 bytes of a cache are 16 bytes that some row of the same cache, layer and head held there."""
        got = after[self.size:3 * self.size].astype(np.int64)
        whole = got.reshape(-1, self.piece)
        together = (whole == whole[:, :1] + np.arange(self.piece)).all() and (whole[:, 0] % self.piece == 0).all()
        inside = (got >= 0).all() and (got < 2 * self.size).all()
        home = np.stack(np.unravel_index(np.arange(2 * self.size), (2, *self.shape)))
        come = np.stack(np.unravel_index(np.clip(got, 0, 2 * self.size - 1), (2, *self.shape)))
        same = all((home[i] == come[i]).all() for i in (0, 1, 3, 5))  # cache, layer, head, column
        return bool(together and inside and same)


def commit(caches, slot, q_start, path, checked=True):
    """The buffer after the call, for slots that no two tokens share and paths that rise. Without `checked` a destination
    outside the cache is written all the same, wherever in the buffer it lies."""
    c, cells, T = caches, caches.pages * caches.page, len(slot)
    old, new = c.buf, c.buf.copy()
    for lo, hi in zip(q_start, q_start[1:]):
        lo = min(max(int(lo), 0), T)
        hi = min(max(int(hi), lo), T)
        for i in range(hi - lo):
            src = int(path[lo + i])
            if not i < src < hi - lo:
                continue
            a, b = int(slot[lo + src]), int(slot[lo + i])
            if not 0 <= a < cells or (checked and not 0 <= b < cells):
                continue
            for cache in (0, 1):
                for layer in range(c.layers):
                    for head in range(c.heads):
                        def at(s):
                            row = ((layer * c.pages + s // c.page) * c.heads + head) * c.page + s % c.page
                            return (1 + cache) * c.size + row * c.d
                        if 0 <= at(b) <= len(new) - c.d:
                            new[at(b):at(b) + c.d] = old[at(a):at(a) + c.d]
    return new


def rising_case(rng, caches, sizes):
    """Slots of which some lie just outside the cache, none of them twice, and rising paths."""
    cells, T = caches.pages * caches.page, sum(sizes)
    inside = rng.permutation(cells)
    outside = np.concatenate([-1 - np.arange(cells // 2), cells + np.arange(cells // 2)])
    slot = inside[:T].copy()
    bad = rng.random(T) < 0.3
    slot[bad] = rng.permutation(outside)[:bad.sum()]
    path, q_start = np.full(T, -1), np.concatenate([[0], np.cumsum(sizes)])
    for lo, n in zip(q_start, sizes):
        take = np.sort(rng.permutation(n)[:(n + 1) // 2])
        path[lo:lo + len(take)] = take
    return slot, q_start, path
