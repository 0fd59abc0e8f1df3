"""Block tables at the ends of their ranges: token counts whose sums pass 2^31."""

import numpy as np
import pytest
import torch

from test_tables_gpu import run

pytestmark = pytest.mark.gpu

MOST = 1 << 30  # where the sums saturate


def _blocks(t):
    return -(-t // 128)


def _check(cached, new, max_nb, pool, max_tokens):
    """Every request's documented outcome; tables start empty but for the blocks that cached tokens have."""
    S = len(cached)
    table = torch.full((S, max_nb), -5, dtype=torch.int32)
    at = 0
    for s in range(S):
        n = _blocks(cached[s])
        table[s, :n] = torch.arange(at, at + n)
        at += n
    free = np.arange(at, pool)
    got, flags = run(pool, cached, new, table, free, len(free), max_tokens)
    slots, pos, lens, offs = [], np.zeros(max_tokens, np.int64), [], []
    stack, tokens, wanted, refused = list(free), 0, 0, False
    rows = {}
    for s in range(S):
        offs.append(min(tokens, MOST))
        for i in range(min(new[s], max(0, max_tokens - tokens))):
            pos[tokens + i] = cached[s] + i
        tokens, wanted = tokens + new[s], wanted + _blocks(cached[s] + new[s]) - _blocks(cached[s])
        ok = tokens <= max_tokens and wanted <= len(free)
        lens.append(cached[s] + (new[s] if ok else 0))
        refused |= not ok and new[s] > 0
        if ok and new[s]:
            row = list(table[s, :_blocks(cached[s])].tolist())
            row += [stack.pop() for _ in range(_blocks(cached[s] + new[s]) - _blocks(cached[s]))]
            rows[s] = row
            slots += [row[p // 128] * 128 + p % 128 for p in range(cached[s], cached[s] + new[s])]
    offs.append(min(tokens, MOST))
    assert (flags != 0) == refused
    assert np.array_equal(got["seq_lens"], lens) and np.array_equal(got["offsets"], offs)
    assert np.array_equal(got["slots"], slots + [-1] * (max_tokens - len(slots)))
    assert np.array_equal(got["positions"], pos)
    assert int(got["free_count"][0]) == len(stack) and np.array_equal(got["free"][:len(stack)], stack)
    for s, row in rows.items():
        table[s, :len(row)] = torch.tensor(row)
    assert np.array_equal(got["table"], table.numpy())


@pytest.mark.parametrize("giants", [1, 2, 3, 5])
def test_sums_of_requests_as_long_as_a_table(giants):
    # each is 2^30 tokens: two of them pass 2^31
    _check([100, 0, 7] + [0] * giants + [5, 9], [30, 200, 0] + [MOST] * giants + [3, 0], 1 << 23, 40, 300)


@pytest.mark.parametrize("S", [40, 512, 3000, 8192])
def test_sums_over_lanes_warps_and_threads(S):
    # from 2^20 tokens each: two halves of a scan saturate wherever the halves meet
    each = 1 << 20 if S > 2048 else 1 << 24
    cached, new = [0] * S, [each] * S
    new[0], new[1], new[2], cached[2], new[S // 2], new[-1] = 50, 0, 129, 100, 0, 1
    _check(cached, new, each // 128, 30, 400)


def test_sums_that_end_at_the_limit():
    _check([0, 0, 0], [10, MOST - 10, 1], 1 << 23, 20, 64)
    _check([0, 0], [MOST - 1, 1], 1 << 23, 20, 64)
