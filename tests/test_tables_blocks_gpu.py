"""Block tables: entries outside the pool in the rows of requests that end.  They are
flagged, do not go onto the stack and so come back to no other request."""

import numpy as np
import pytest

from _serving import plain_tables
from test_tables_gpu import make, run

pytestmark = pytest.mark.gpu

BLOCK = 128


def _check(num_blocks, cached, new, table, free, count, max_tokens):
    """The plain rules with each ended request's row reduced to the blocks in it."""
    got, flags = run(num_blocks, cached, new, table, free, count, max_tokens)
    c, t, any_bad = [int(x) for x in cached], np.array(table), False
    for s, n in enumerate(new):
        if n == -1 and c[s] >= 0:
            row = [int(b) for b in t[s, :-(-c[s] // BLOCK)]]
            good = [b for b in row if 0 <= b < num_blocks]
            if len(good) < len(row):
                any_bad = True
                t[s, :len(good)], c[s] = good, BLOCK * len(good)
    want, bad = plain_tables(num_blocks, c, [int(x) for x in new], t, np.array(free), count, max_tokens)
    for s, n in enumerate(new):
        if n == -1:
            want["table"][s] = table[s]  # the rows of ended requests stay as they are
    for k, v in want.items():
        assert np.array_equal(got[k], np.atleast_1d(v)), (k, np.argwhere(got[k] != np.atleast_1d(v))[:5])
    assert (flags != 0) == (bad or any_bad)
    if any_bad:
        assert flags & 1
    return got


def test_one_bad_entry():
    # three returned entries of which the middle one is no block; two free blocks, four wanted
    for bad in (-1, 8, 2 ** 31 - 1, -2 ** 31):
        got = _check(8, [300, 5, 0], [-1, 260, 200], np.array([[4, bad, 6, -1], [7, -1, -1, -1], [-1, -1, -1, -1]]),
                     np.array([0, 1, -6, -6, -6, -6]), 2, 460)
        assert got["table"][1].tolist() == [7, 6, 4, -1] and got["table"][2].tolist() == [1, 0, -1, -1]
        assert got["free_count"][0] == 0


def test_only_bad_entries():
    _check(8, [300, 5], [-1, 0], np.array([[-1, 9, -7], [7, -1, -1]]), np.array([0, 1, -6, -6]), 2, 3)
    _check(8, [300, 128], [-1, -1], np.array([[-1, 9, -7], [7, -1, -1]]), np.array([0, 1, -6, -6]), 2, 0)


@pytest.mark.parametrize("S,share", [(3, 0.5), (40, 0.02), (40, 0.3), (700, 0.01), (3000, 0.5)])
@pytest.mark.parametrize("max_cached", [900, 9000])
def test_random_bad_entries(S, share, max_cached):
    rng = np.random.default_rng(S)
    pool, cached, new, table, free, count, tokens = make(S, 200, max_cached if S < 1000 else 900, seed=S + 1, ends=0.4, spare=5 * S)
    table = table.copy()
    for s in np.flatnonzero(new == -1):
        n = -(-cached[s] // BLOCK)
        hit = rng.random(n) < share
        table[s, :n][hit] = rng.choice([-1, pool, pool + 7, -2 ** 31], n)[hit]
    _check(pool, cached, new, table, free, count, tokens)


def test_bad_entries_and_a_stack_without_room():
    # room for three of the returned blocks: those in front
    _check(9, [600, 300], [-1, -1], np.array([[4, -1, 5, 6, 7], [8, 9, 3, -1, -1]]), np.array([0, 1, -6, -6, -6]), 2, 2)
    _check(9, [600], [-1], np.array([[4, 5, 6, 7, -1]]), np.array([0, 1, -6, -6, -6]), 2, 2)


def test_a_bad_entry_does_not_come_around():
    # taken off the stack once (flagged, -1 in the row); when its request ends it is gone
    table, free = np.full((2, 4), -1), np.array([3, 77, 2, -6])
    got, flags = run(8, [0, 0], [200, 0], table, free, 3, 200)
    assert flags == 1 and got["table"][0].tolist() == [2, -1, -1, -1] and int(got["free_count"][0]) == 1
    got = _check(8, [200, 0], [-1, 200], got["table"], got["free"], 1, 200)
    assert got["table"][1].tolist() == [2, 3, -1, -1] and int(got["free_count"][0]) == 0
