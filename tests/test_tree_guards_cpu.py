"""The checks of tests/commit_reference.py see what they are there for: a host
model that lacks a bounds check, or puts a row into the wrong head or cache,
fails them."""
import numpy as np
import pytest

from . import commit_reference as ref


def caches(layers=1, bits=32):
    return ref.Caches(layers, 8, 2, 16, 8, bits)


@pytest.mark.parametrize("layers,bits", [(1, 32), (2, 32), (1, 16), (2, 16)])
@pytest.mark.parametrize("seed", range(3))
def test_a_write_outside_the_caches_is_seen(layers, bits, seed):
    c = caches(layers, bits)
    slot, q_start, path = ref.rising_case(np.random.default_rng(seed), c, [40, 0, 50])
    right, wrong = ref.commit(c, slot, q_start, path), ref.commit(c, slot, q_start, path, checked=False)
    assert not np.array_equal(right, c.buf), "rows move"
    assert c.guards_are_left(right) and c.every_piece_is_one_of_its_head(right)
    assert not np.array_equal(wrong, right)
    assert not (c.guards_are_left(wrong) and c.every_piece_is_one_of_its_head(wrong))


def test_wrong_places_inside_are_seen():
    c = caches()
    body = slice(c.size, 3 * c.size)
    for other in (c.size, 16 * 8, 4):  # V's row in K's place, the next head's row, the row's next piece
        wrong = c.buf.copy()
        wrong[c.size:c.size + 4] = c.buf[c.size + other:c.size + other + 4]
        assert not c.every_piece_is_one_of_its_head(wrong), other
    wrong = c.buf.copy()
    wrong[c.size] = c.buf[c.size + 8]  # half of a piece
    assert not c.every_piece_is_one_of_its_head(wrong)
    moved = c.buf.copy()
    moved[c.size:c.size + 8] = c.buf[c.size + 8:c.size + 16]  # the head's next row
    assert c.every_piece_is_one_of_its_head(moved) and c.every_piece_is_one_of_its_head(c.buf)
    assert not np.array_equal(moved[body], c.buf[body])
