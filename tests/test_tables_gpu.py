"""Block tables from request lengths (msa_build_tables) against the documented
rules applied one request after the other: growth, ends, waiting requests, a
stack that runs out, token places that run out, malformed requests and blocks."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _serving import plain_tables

pytestmark = pytest.mark.gpu


def run(num_blocks, cached, new, table, free, count, max_tokens, stream=None):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    S = len(cached)
    t, f = dev(table), dev(free)
    out = {k: torch.full((n,), -77, dtype=torch.int32, device="cuda")
           for k, n in (("seq_lens", S), ("offsets", S + 1), ("slots", max_tokens), ("positions", max_tokens), ("free_count", 1))}
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_build_tables(num_blocks, dev(cached), dev(new), t, f, dev([count]), out["seq_lens"], out["offsets"], out["slots"],
                         out["positions"], out["free_count"], ws, stream)
    st, flags = msa.msa_read_device_status(ws)
    got = {k: v.cpu().numpy() for k, v in out.items()}
    got.update(table=t.cpu().numpy(), free=f.cpu().numpy())
    return got, flags


def make(S, max_new, max_cached, seed, ends=0.2, waits=0.2, spare=10):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, max_cached + 1, S)
    new = rng.integers(1, max_new + 1, S)
    new[rng.random(S) < waits] = 0
    new[rng.random(S) < ends] = -1
    max_nb = int((cached + np.maximum(new, 0)).max()) // 128 + 2
    had = -(-cached // 128)
    pool = int(had.sum() + (-(-(cached + np.maximum(new, 0)) // 128) - had).sum()) + spare
    perm = rng.permutation(pool)
    table = np.full((S, max_nb), -5)
    at = 0
    for s in range(S):
        table[s, :had[s]] = perm[at:at + had[s]]
        at += had[s]
    free = np.full(pool, -6)
    free[:pool - at] = perm[at:]
    return pool, cached, new, table, free, pool - at, int(np.maximum(new, 0).sum()) + 3


def check(args, fault=None):
    got, flags = run(*args)
    want, bad = plain_tables(*[np.asarray(a).tolist() if i in (1, 2) else a for i, a in enumerate(args)])
    for k, v in want.items():
        assert np.array_equal(got[k], np.atleast_1d(v)), (k, np.argwhere(got[k] != np.atleast_1d(v))[:5])
    assert (flags != 0) == bad
    if fault is not None:
        assert bad == fault
    return got


@pytest.mark.parametrize("S,max_new,max_cached", [(1, 1, 0), (1, 1, 128), (1, 129, 127), (7, 1, 1000), (32, 8, 5000), (250, 700, 3000),
                                                  (1000, 3, 300), (8192, 2, 200), (3, 40000, 10)])
def test_random_steps(S, max_new, max_cached):
    check(make(S, max_new, max_cached, seed=S + max_new), fault=False)


def test_nothing_to_do():
    check((4, [0, 130], [0, 0], np.array([[-1, -1], [2, 3]]), np.array([0, 1]), 2, 5), fault=False)
    check((4, [0, 130], [-1, -1], np.array([[-1, -1], [2, 3]]), np.array([0, 1, 9, 9]), 2, 0), fault=False)


def test_returned_blocks_are_taken_in_the_same_call():
    # two free blocks, three returned, four wanted: all three returned ones and one free one
    args = (8, [300, 5, 0], [-1, 260, 200], np.array([[4, 5, 6, -1], [7, -1, -1, -1], [-1, -1, -1, -1]]),
            np.array([0, 1, -6, -6, -6, -6]), 2, 460)
    got = check(args, fault=False)
    assert got["table"][1].tolist() == [7, 6, 5, -1] and got["table"][2].tolist() == [4, 1, -1, -1]
    assert got["free_count"][0] == 1


def test_the_stack_runs_out():
    pool, cached, new, table, free, count, tokens = make(40, 500, 800, seed=3, ends=0.1)
    got = check((pool, cached, new, table, free, min(count, 20), tokens), fault=True)
    assert got["free_count"][0] >= 0


def test_token_places_run_out():
    pool, cached, new, table, free, count, tokens = make(40, 500, 800, seed=4, ends=0.1)
    check((pool, cached, new, table, free, count, tokens // 2), fault=True)


def test_malformed_requests_count_as_empty():
    pool, cached, new, table, free, count, tokens = make(20, 50, 500, seed=5, ends=0.0)
    cached, new = cached.copy(), new.copy()
    cached[3], new[7], new[11] = -1, -2, table.shape[1] * 128 + 1
    new[12], cached[13] = 2 ** 31 - 1, 2 ** 31 - 1
    check((pool, cached, new, table, free, count, tokens), fault=True)


def test_blocks_outside_the_pool():
    pool, cached, new, table, free, count, tokens = make(12, 300, 500, seed=6, ends=0.0, waits=0.0)
    table, free = table.copy(), free.copy()
    s = int(np.argmax(cached % 128 != 0))
    table[s, cached[s] // 128] = pool       # the block its next token falls into
    free[count - 2] = -3
    check((pool, cached, new, table, free, count, tokens), fault=True)


def test_a_stack_without_room_for_what_comes_back():
    check((8, [300, 5], [-1, 0], np.array([[4, 5, 6], [7, -1, -1]]), np.array([0, 1, -6]), 2, 2), fault=True)


def test_replayed_steps_carry_their_state_in_device_memory():
    # five decode steps as replays of one graph: lengths and stack size copied back on the device
    S, steps = 5, 200
    pool, cached, _, table, free, count, _ = make(S, 1, 200, seed=7, ends=0.0, waits=0.0, spare=20)
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    table = np.concatenate([table, np.full((S, 3), -5)], 1)
    c, n, t, f, k = dev(cached), dev(np.ones(S)), dev(table), dev(free), dev([count])
    lens, offs, slots, pos, k2 = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (S, S + 1, S, S, 1))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def step():
        msa.msa_build_tables(pool, c, n, t, f, k, lens, offs, slots, pos, k2, ws)
        c.copy_(lens)
        k.copy_(k2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    assert msa.msa_read_device_status(ws)[1] == 0
    ref = (table, free, count)
    cur = list(cached)
    for _ in range(steps):
        want, bad = plain_tables(pool, [int(x) for x in cur], [1] * S, ref[0], ref[1], ref[2], S)
        assert not bad
        ref, cur = (want["table"], want["free"], want["free_count"]), want["seq_lens"]
    assert np.array_equal(t.cpu().numpy(), ref[0]) and int(k[0]) == ref[2]
    assert np.array_equal(c.cpu().numpy(), cur) and np.array_equal(slots.cpu().numpy(), want["slots"])
