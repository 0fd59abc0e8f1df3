"""Insert into caches with one scale for each block and head, bit for bit against the documented
operations taken one by one, and the read of tokens back out of caches of every format."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _blocks import BLOCK, DIM, KINDS, code_values, empty_cache, plain_insert, same_bits, spans, status_words, to_host

pytestmark = pytest.mark.gpu


def _rows(T, H, seed, spread=0.4, extra=0):
    """k and v as slices of one projection's rows (their strides are the projection's)."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, 2 * H + extra, DIM), generator=gen) * torch.exp(spread * torch.randn((T, 2 * H + extra, 1), generator=gen))
    x = x.bfloat16().cuda()
    return x[:, extra:extra + H], x[:, extra + H:]


def _insert(cache, first, end, offsets, table, k, v, want=0):
    """Run the insert and hold it against plain_insert, the whole pool bit for bit."""
    ref = to_host(cache)
    plain_insert(cache.kv_dtype, ref, first, end, offsets, np.asarray(table), k.float().cpu().numpy(), v.float().cpu().numpy(),
                 cache.num_blocks)
    ws = status_words()
    msa.msa_block_insert(cache, spans(first, end, offsets, table), k, v, ws)
    assert msa.msa_read_device_status(ws)[1] == want
    got = to_host(cache)
    for name, x in ref.items():
        assert same_bits(got[name], x), (name, np.argwhere(got[name] != x)[:4])
    return got


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("first,n", [(0, 1), (0, 128), (0, 129), (5, 1), (127, 1), (127, 2), (128, 1), (100, 300), (1, 127), (255, 700)])
def test_one_span(kv, first, n):
    H = 2
    cache = empty_cache(kv, 10, H, seed=n)
    table = np.random.default_rng(n).permutation(10)[None, :9]
    cache.k_scale.copy_(torch.rand(10, H).cuda() * 0.02 + 0.005)  # blocks that go on: some grow, some do not
    cache.v_scale.copy_(torch.rand(10, H).cuda() * 0.02 + 0.005)
    k, v = _rows(n, H, seed=first + n, extra=3)
    _insert(cache, [first], [first + n], [0], table, k, v)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("H", [1, 3, 8])
def test_many_spans(kv, H):
    # more than one chunk of 256 sequences; waiting, ended and refused requests among them; rows between the spans
    rng = np.random.default_rng(H)
    S, pool = 600, 1500
    first = rng.integers(0, 200, S)
    n = rng.integers(0, 4, S) * rng.integers(0, 40, S)
    end = np.where(rng.random(S) < 0.1, 0, first + n)
    blocks = [-(-max(a, b) // BLOCK) for a, b in zip(first, end)]
    table = np.full((S, 4), -99)
    order, at = rng.permutation(pool), 0
    for s in range(S):
        table[s, :blocks[s]] = order[at:at + blocks[s]]
        at += blocks[s]
    offsets, T = [], 0
    for s in range(S):
        T += int(rng.integers(0, 3))
        offsets.append(T)
        T += max(0, int(end[s] - first[s]))
    cache = empty_cache(kv, pool, H, seed=H)
    k, v = _rows(T + 5, H, seed=1)
    _insert(cache, first, end, offsets, table, k, v)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("S,most", [(31, 1), (257, 3), (5000, 2), (40, 9)])
def test_a_steps_few_tokens(kv, S, most):
    # 1 to `most` tokens a request, and one request that brings many more; more sequences than CTAs x 256
    rng = np.random.default_rng(S)
    H = 1 if S > 1000 else 4
    first = rng.integers(0, 250, S)
    n = rng.integers(0, most + 1, S)
    n[S // 2] = min(300, 4 * S) if most < 9 else 300
    end = first + n
    pool = 6 * S
    table = rng.permutation(pool).reshape(S, 6)
    offsets = np.cumsum(n) - n
    cache = empty_cache(kv, pool, H, seed=S)
    cache.k_scale.copy_(torch.rand(pool, H).cuda() * 0.03 + 0.005)
    k, v = _rows(int(n.sum()), H, seed=S, spread=0.8)
    _insert(cache, first, end, offsets, table, k, v)


@pytest.mark.parametrize("kv", KINDS)
def test_special_values_one_token_at_a_time(kv):
    # infinities, NaN, zeros, the smallest and the largest numbers in single tokens that go on in blocks, some of which grow
    H, S = 1, 12
    cache = empty_cache(kv, S, H, seed=30)
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.tensor([1e-38, 1e-3, 1.0, 1e30] * 3).view(S, 1).cuda())
    k, v = (t.clone() for t in _rows(S, H, seed=31))
    for i, x in enumerate((0.0, -0.0, 1e-40, 3e38, float("inf"), float("-inf"), float("nan"), 1e-30, 1e20, -3.3e38, 1.0, 2.0 ** -126)):
        k[i, 0, 3 * i] = x
        v[i] = x
    first = np.arange(S) * 10 + 1
    _insert(cache, first, first + 1, np.arange(S), np.arange(S)[:, None], k, v)
    _insert(cache, np.zeros(S), np.ones(S), np.arange(S), np.arange(S)[:, None], k, v)  # and in blocks that begin


@pytest.mark.parametrize("kv", KINDS)
def test_special_values(kv):
    # rows of zeros, of the smallest numbers, near the largest, with infinities and NaN, and blocks without a finite element
    H, T = 2, 8 * BLOCK
    k, v = _rows(T, H, seed=2)
    k, v = k.clone(), v.clone()
    k[:BLOCK] = 0
    k[1, 0, 0], k[2, 0, 1] = -0.0, 1e-40
    k[BLOCK:2 * BLOCK] *= 2.0 ** -126
    k[2 * BLOCK:3 * BLOCK] *= 2.0 ** 120
    k[3 * BLOCK + 5, 0, 7], k[3 * BLOCK + 6, 0, 8] = float("inf"), float("-inf")
    k[3 * BLOCK + 7, 1, 9] = float("nan")
    k[4 * BLOCK:5 * BLOCK] = float("nan")
    k[5 * BLOCK:6 * BLOCK, 0], k[5 * BLOCK:6 * BLOCK, 1] = float("inf"), float("-inf")
    k[6 * BLOCK:7 * BLOCK] *= 1e-38
    k[6 * BLOCK + 3, 0, 0], k[6 * BLOCK + 9, 0, 3] = float("inf"), 3.0e38
    v[:, 0, 0] = 3.3e38
    cache = empty_cache(kv, 9, H, seed=3)
    got = _insert(cache, [0], [T], [0], np.arange(8)[None], k, v)
    assert np.isfinite(got["k_scale"][:8]).all() and (got["k_scale"][:8] >= 2.0 ** -126).all()
    if kv == "fp8_block":
        assert got["k"][0, 0, 1, 0] == 0x80 and (got["k"][4] & 0x7F == 0x7F).all()  # the sign of a zero, and NaN


@pytest.mark.parametrize("kv", KINDS)
def test_old_scales_of_any_bits(kv):
    # a span goes on in blocks whose scale is zero, negative, subnormal, infinite, NaN or the largest number
    olds = [0.0, -1.0, 1e-40, float("inf"), float("nan"), 3.4e38, 2.0 ** -126, 2.0 ** -149, 2.0 ** -20, 1.0]
    S, H = len(olds), 1
    cache = empty_cache(kv, S, H, seed=4)
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.tensor(olds).view(S, 1).cuda())
    first = np.arange(S) * 12 + 1
    k, v = _rows(S, H, seed=5)
    _insert(cache, first, first + 1, np.arange(S), np.arange(S)[:, None], k, (v.float() * 1e30).bfloat16())


@pytest.mark.parametrize("kv", KINDS)
def test_a_block_that_grows_token_by_token(kv):
    # 128 tokens one after the other, larger and larger: the codes of what was inserted first are off by less than a
    # step of the final scale (INT8: 1/2 + 1/4 + ...), E4M3 by its own half step and what its subnormals lose
    H = 2
    cache = empty_cache(kv, 3, H, seed=6)
    gen = torch.Generator().manual_seed(7)
    x = (torch.randn((BLOCK, 2 * H, DIM), generator=gen) * torch.exp2(torch.arange(BLOCK) / 16.0).view(-1, 1, 1)).bfloat16().cuda()
    for t in range(BLOCK):
        got = _insert(cache, [t], [t + 1], [0], [[1]], x[t:t + 1, :H], x[t:t + 1, H:])
    want = x.float().cpu().numpy().astype(np.float64)
    for h in range(H):
        for name, w in (("k", want[:, h]), ("v", want[:, H + h])):
            s = float(got[name + "_scale"][1, h])
            err = np.abs(code_values(kv, got[name][1, h]) * s - w)
            step = s if kv == "int8_block" else 2.0 ** -4 * np.abs(w) * 1.01 + 2.0 ** -9 * s
            assert (err <= step).all()
            assert s <= 2.01 * np.abs(w).max() / (127 if kv == "int8_block" else 448)


@pytest.mark.parametrize("kv", KINDS)
def test_in_one_go_or_in_pieces_the_scale_is_near(kv):
    # a prompt in one call has amax / Q exactly; in pieces at most twice that
    H, T = 4, 300
    k, v = _rows(T, H, seed=8)
    one, many = empty_cache(kv, 4, H), empty_cache(kv, 4, H)
    a = _insert(one, [0], [T], [0], [[2, 0, 1]], k, v)
    t = 0
    for n in (1, 40, 87, 1, 2, 120, 49):
        b = _insert(many, [t], [t + n], [0], [[2, 0, 1]], k[t:t + n], v[t:t + n])
        t += n
    assert t == T
    ratio = b["k_scale"][[2, 0, 1]] / a["k_scale"][[2, 0, 1]]
    assert (ratio >= 1 - 2.0 ** -23).all() and (ratio < 2.0 + 2.0 ** -22).all()


@pytest.mark.parametrize("kv", KINDS)
def test_faults_are_flagged_and_skipped(kv):
    H = 2
    cache = empty_cache(kv, 12, H, seed=9)
    table = np.arange(12).reshape(6, 2)
    first, end = [-1, 10, 0, 250, 5, 3], [3, 20, 9, 257, 9, 140]
    offsets = [0, 40, 64, 0, -1, 0]
    table[5, 0] = 12
    k, v = _rows(140, H, seed=10)
    # only sequences 1 and 2 and the second block of 5 are sound
    _insert(cache, first, end, offsets, table, k, v, want=1 | 2 | 16)
    cache = empty_cache(kv, 12, H, seed=9)
    table[5, 0], first[5], end[5] = -1, 0, 5
    _insert(cache, first[5:], end[5:], [0], table[5:], k, v, want=1)
    _insert(cache, [0], [141], [0], [[1, 2]], k, v, want=16)  # one row too few
    _insert(cache, [2 ** 31 - 2], [2 ** 31 - 1], [0], [[1, 2]], k, v, want=2)
    _insert(cache, [-2 ** 31], [2 ** 31 - 1], [0], [[1, 2]], k, v, want=2)
    _insert(cache, [0], [3], [2 ** 31 - 1], [[1, 2]], k, v, want=16)


@pytest.mark.parametrize("kv", KINDS)
def test_insert_past_32_bits(kv):
    H, pool = 8, 41000  # 5.4 GB for K and for V
    t = {n: torch.zeros((pool, H, BLOCK, DIM), dtype=torch.int8 if kv == "int8_block" else torch.uint8, device="cuda") for n in "kv"}
    sc = {n + "_scale": torch.ones((pool, H), device="cuda") for n in "kv"}
    cache = msa.PagedCache(kv_dtype=kv, index_dtype="bf16", num_blocks=pool, num_kv_heads=H, idx=None, **t, **sc)
    k, v = _rows(200, H, seed=11)
    last = np.array([[pool - 1, pool - 2]])
    ws = status_words()
    sp = spans([0], [200], [0], last)
    msa.msa_block_insert(cache, sp, k, v, ws)
    ref = {n: np.zeros((2, H, BLOCK, DIM), np.int8 if kv == "int8_block" else np.uint8) for n in "kv"}
    ref.update({n + "_scale": np.ones((2, H), np.float32) for n in "kv"})
    plain_insert(kv, ref, [0], [200], [0], np.array([[1, 0]]), k.float().cpu().numpy(), v.float().cpu().numpy(), 2)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert same_bits(getattr(cache, n)[-2:].cpu().numpy(), ref[n])
    ko, vo = torch.zeros((2, 200, H, DIM), dtype=torch.bfloat16, device="cuda")
    msa.msa_cache_read(cache, sp, ko, vo, ws)
    assert msa.msa_read_device_status(ws)[1] == 0
    x = np.concatenate([code_values(kv, ref["k"][1]), code_values(kv, ref["k"][0])], 1)[:, :200].astype(np.float32)
    s = np.repeat(ref["k_scale"][[1, 0]], BLOCK, 0)[:200].T[..., None]
    assert torch.equal(ko.cpu(), torch.from_numpy((x * s).transpose(1, 0, 2)).bfloat16())


# ---------------------------------------------------------------- read

def _any_cache(kv, pool, H, seed):
    """Codes of all bits; scales of sound sizes."""
    gen = torch.Generator().manual_seed(seed)
    t, kw = {}, {}
    for name in ("k", "v"):
        width = {"bf16": 256, "nvfp4": 64}.get(kv, 128)
        raw = torch.randint(0, 256, (pool, H, BLOCK, width), generator=gen, dtype=torch.uint8)
        t[name] = (raw.view(torch.bfloat16) if kv == "bf16" else raw.view(torch.int8) if kv == "int8_block" else raw).cuda()
        if kv in ("fp8", *KINDS):
            shape = (pool, H, BLOCK) if kv == "fp8" else (pool, H)
            t[name + "_scale"] = torch.exp(3 * torch.randn(shape, generator=gen)).cuda()
        if kv == "nvfp4":
            t[name + "_sf"] = torch.randint(0, 127, (pool, H, BLOCK, 8), generator=gen, dtype=torch.uint8).cuda()
            kw[name + "_global"] = 0.0123 if name == "k" else 0.5
    return msa.PagedCache(kv_dtype=kv, index_dtype="bf16", num_blocks=pool, num_kv_heads=H, idx=None, **t, **kw)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4", *KINDS])
@pytest.mark.parametrize("mode", ["exact", "e4m3"])
@pytest.mark.parametrize("H", [1, 2, 5])
def test_read_is_the_dequantized_value(kv, mode, H):
    if mode == "e4m3" and kv != "nvfp4":
        mode = "exact"
    pool = 40
    cache = _any_cache(kv, pool, H, seed=H)
    cache.nvfp4_mode = mode
    rng = np.random.default_rng(H)
    first = np.array([0, 5, 127, 128, 300, 7, 0, 50])
    end = np.array([1, 5, 129, 400, 20, 320, 128, 51])
    table = np.stack([rng.permutation(pool)[:4] for _ in first])  # blocks may be shared
    offsets = np.array([3, 4, 4, 10, 0, 290, 610, 740])
    T = 745
    # what the library says of each block, in fp32
    every = torch.arange(pool, dtype=torch.int32, device="cuda")
    val = {}
    for which, name in ((0, "k"), (1, "v")):
        val[name] = torch.empty((pool, H, BLOCK, DIM), device="cuda")
        msa.msa_dequant_debug(cache, which, every, val[name])
        if kv in KINDS:  # and what the formats are
            want = code_values(kv, getattr(cache, name).cpu().numpy()).astype(np.float32) * getattr(cache, name + "_scale").cpu().numpy()[..., None, None]
            assert np.array_equal(val[name].cpu().numpy(), want, equal_nan=True)
    wide = torch.full((T, 2 * H + 1, DIM), 9.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = wide[:, :H], wide[:, H + 1:]
    ws = status_words()
    sp = spans(first, end, offsets, table)
    msa.msa_cache_read(cache, sp, ko, vo, ws)
    assert msa.msa_read_device_status(ws)[1] == 0
    want = torch.full_like(wide, 9.0)
    for s in range(len(first)):
        for p in range(first[s], end[s]):
            row = offsets[s] + p - first[s]
            want[row, :H] = val["k"][table[s, p // BLOCK], :, p % BLOCK].bfloat16()
            want[row, H + 1:] = val["v"][table[s, p // BLOCK], :, p % BLOCK].bfloat16()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(wide.float()), nan)
    bits = lambda x: x.masked_fill(nan, 0).view(torch.int16)  # noqa: E731
    assert torch.equal(bits(wide), bits(want))
    if kv == "bf16":  # every bit, those of a NaN too
        raw = cache.k.view(torch.int16)
        assert torch.equal(wide[10, :H].view(torch.int16), raw[table[3, 1], :, 0])
    only = torch.full((T, H, DIM), 9.0, dtype=torch.bfloat16, device="cuda")
    msa.msa_cache_read(cache, sp, None, only, ws)
    assert torch.equal(only.view(torch.int16), wide[:, H + 1:].contiguous().view(torch.int16))
    only.fill_(9.0)
    msa.msa_cache_read(cache, sp, only, None, ws)
    assert torch.equal(only.view(torch.int16), wide[:, :H].contiguous().view(torch.int16))


def test_read_faults():
    cache = _any_cache("int8_block", 6, 2, seed=1)
    out = torch.full((2, 100, 2, DIM), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = status_words()
    for first, end, off, table, want in ((0, 10, 91, [[0, 1]], 16), (-1, 10, 0, [[0, 1]], 2), (0, 257, 0, [[0, 1]], 2), (0, 10, 0, [[6, 1]], 1),
                                         (0, 10, 0, [[-1, 1]], 1), (0, 10, -1, [[0, 1]], 16)):
        msa.msa_cache_read(cache, spans([first], [end], [off], table), out[0], out[1], ws)
        assert msa.msa_read_device_status(ws)[1] == want
        assert (out == 9).all()
    msa.msa_cache_read(cache, spans([0], [0], [0], [[0, 1]]), out[0], out[1], ws)
    msa.msa_cache_read(cache, spans([0], [0], [0], [[0, 1]]), out[0][:0], out[1][:0], ws)
    assert msa.msa_read_device_status(ws)[1] == 0 and (out == 9).all()


@pytest.mark.parametrize("kv", KINDS)
def test_captured_insert_and_read(kv):
    # one graph that inserts a step's tokens and reads the prefix back, replayed as the lengths go on, on another stream
    H, S = 2, 3
    cache = empty_cache(kv, 12, H, seed=12)
    ref = to_host(cache)
    table = np.arange(12).reshape(S, 4)[:, ::-1].copy()
    lens = np.array([0, 126, 255])
    sp = spans(lens, lens, [0, 2, 4], table)  # no tokens yet
    pre = spans(np.zeros(S), np.zeros(S), [0, 400, 800], table)
    k, v = (t.clone() for t in _rows(2 * S, H, seed=13))
    ko, vo = torch.zeros((2, 1200, H, DIM), dtype=torch.bfloat16, device="cuda")
    ws = status_words()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        msa.msa_block_insert(cache, sp, k, v, ws)
        msa.msa_cache_read(cache, pre, ko, vo, ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            msa.msa_block_insert(cache, sp, k, v, ws)
            msa.msa_cache_read(cache, pre, ko, vo, ws)
    torch.cuda.synchronize()
    # what the blocks held before belongs to no one: a known state
    for name in ("k", "v"):
        getattr(cache, name + "_scale").fill_(0.01)
        ref[name + "_scale"][:] = 0.01
    for step in range(4):
        a, b = _rows(2 * S, H, seed=20 + step)
        k.copy_(a)
        v.copy_(b)
        sp.first.copy_(torch.from_numpy(lens).int())
        sp.end.copy_(torch.from_numpy(lens + 2).int())
        pre.end.copy_(torch.from_numpy(lens + 2).int())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        plain_insert(kv, ref, lens, lens + 2, [0, 2, 4], table, a.float().cpu().numpy(), b.float().cpu().numpy(), 12)
        got = to_host(cache)
        for name, x in ref.items():
            assert same_bits(got[name], x), (step, name)
        for s in range(S):
            n = lens[s] + 2
            blocks = table[s, :-(-n // BLOCK)]
            x = np.concatenate([code_values(kv, ref["v"][p]).astype(np.float32) * ref["v_scale"][p][:, None, None] for p in blocks], 1)[:, :n]
            want = torch.from_numpy(x.transpose(1, 0, 2).copy()).bfloat16()
            assert torch.equal(torch.nan_to_num(vo[400 * s:400 * s + n].cpu().float()), torch.nan_to_num(want.float()))
        lens = lens + 2
    assert msa.msa_read_device_status(ws)[1] == 0


@pytest.mark.parametrize("kv", KINDS)
def test_from_one_format_to_another(kv):
    # rows read out of an FP8 cache with token scales and inserted into one with block scales
    H, T = 2, 300
    src, dst = _any_cache("fp8", 4, H, seed=14), empty_cache(kv, 5, H, seed=15)
    src.k.masked_fill_(src.k & 0x7F == 0x7F, 0)
    src.v.masked_fill_(src.v & 0x7F == 0x7F, 0)
    ko, vo = torch.zeros((2, T, H, DIM), dtype=torch.bfloat16, device="cuda")
    ws = status_words()
    msa.msa_cache_read(src, spans([0], [T], [0], [[3, 0, 2]]), ko, vo, ws)
    got = _insert(dst, [0], [T], [0], [[4, 1, 2]], ko, vo)
    x = ko.float().cpu().numpy().astype(np.float64)
    for b, p in enumerate((4, 1, 2)):
        rows = x[b * BLOCK:(b + 1) * BLOCK].transpose(1, 0, 2)
        s = got["k_scale"][p].astype(np.float64)[:, None, None]
        err = np.abs(code_values(kv, got["k"][p])[:, :rows.shape[1]] * s - rows)
        assert (err <= (s / 2 if kv == "int8_block" else 2.0 ** -4 * np.abs(rows) + 2.0 ** -10 * s) * (1 + 1e-6)).all()
