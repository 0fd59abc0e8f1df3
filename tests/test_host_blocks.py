"""Caches with one scale for each block and head, without a GPU: what the entry points refuse before any
launch, and the documented insert's own bounds."""

import ctypes

import numpy as np
import pytest
import torch

from _blocks import BLOCK, DIM, KINDS, TOP, code_values, growth, plain_insert
from test_host_serving import _Elsewhere, _refused, lib, on_device_0  # noqa: F401  (fixtures)
from test_host_types import _passes

ref = ctypes.byref
bf, i32, u8, i8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.int8, torch.float32


# places far from one another: the cache holds 100 blocks of 4 heads (6,553,600 bytes of codes, 1,600 of scales)
K, V, KS, VS, ROWS_K, ROWS_V, WS = (i << 28 for i in range(1, 8))
SPANS = tuple(i << 20 for i in range(1, 5))


def _structs(kv=8, **over):
    import block_sparse_attention_03_gb300 as msa
    c = msa.MsaCacheT(kv, 1, 100, 128, 4, 128, 128, K, V, None, None, KS, VS, 80, None, 96, 0, 0, 0)
    b = msa.MsaBatchT(2, 1, 50, 16, 32)
    f = msa.MsaConfigT(16, 0, 0, 128 ** -0.5, 128 ** -0.5, 0)
    sp = msa.MsaSpansT(2, 50, *SPANS)
    for k, v in over.items():
        obj, field = k.split("__")
        setattr({"c": c, "b": b, "f": f, "s": sp}[obj], field, v)
    return c, b, f, sp


@pytest.mark.parametrize("name", ["msa_block_insert", "msa_cache_read"])
@pytest.mark.parametrize("kv", [8, 9])
def test_span_refusals(lib, name, kv):  # noqa: F811
    import block_sparse_attention_03_gb300 as msa
    read = name == "msa_cache_read"

    def call(tokens=4, k=(ROWS_K, 4096), v=(ROWS_V, 4096), ws=WS, size=256, cache=True, spans=True, **over):
        c, _, _, sp = _structs(kv, **over)
        rows = [None if x is None else ref(msa.MsaRowsT(*x)) for x in (k, v)]
        return getattr(lib, name)(ref(c) if cache else None, ref(sp) if spans else None, tokens, *rows, ctypes.c_void_p(ws), size, None)

    assert call(tokens=0) == 0 and call(tokens=0, k=None, v=None) == 0
    assert call(cache=False) == 1 and call(spans=False) == 1 and call(tokens=-1) == 1 and call(ws=None) == 1 and call(ws=WS + 2) == 1
    assert call(size=255) == 3
    for bad in (dict(c__k=None), dict(c__v=17), dict(c__k_scale=None), dict(c__v_scale=20), dict(s__num_seqs=0),
                dict(s__max_blocks_per_seq=0), dict(s__first=None), dict(s__end=None), dict(s__token_offsets=None),
                dict(s__block_table=None), dict(s__first=18), dict(s__end=33), dict(s__token_offsets=50), dict(s__block_table=67)):
        assert call(**bad) == 1, bad
    assert call(tokens=(1 << 27) + 1) == 2 and call(s__max_blocks_per_seq=(1 << 23) + 1) == 2 and call(c__num_kv_heads=9) == 2 and call(c__head_dim=64) == 2
    for bad in ((None, 4096), (24, 4096), (ROWS_K, 4100), (ROWS_K, -8)):
        assert call(k=bad, v=bad) == 1 and call(k=bad) == 1 and call(v=(bad[0] and bad[0] + ROWS_V - ROWS_K, bad[1])) == 1, bad
    for unknown in (3, 7, 10):
        assert call(c__kv_dtype=unknown) == 2
    if read:  # one of the two is enough; the rows of two tokens may not lie on top of each other
        assert call(k=None, v=None) == 0 and call(k=(ROWS_K, 504)) == 1 and call(v=(ROWS_V, 0)) == 1
    else:
        assert call(k=None) == 1 and call(v=None) == 1
        for other in (0, 1):  # the formats that msa_cache_insert writes
            assert call(c__kv_dtype=other, c__k_sf=16, c__v_sf=16) == 2


ROW = 4 * 128  # elements of a token's heads


@pytest.mark.parametrize("kv", [8, 9])
def test_what_a_span_call_writes_overlaps_nothing(lib, kv):  # noqa: F811
    import block_sparse_attention_03_gb300 as msa

    def call(name, k, v, tokens=5, stride=(4096, 4096), **over):
        c, _, _, sp = _structs(kv, **over)
        rows = [None if x is None else ref(msa.MsaRowsT(x, n)) for x, n in zip((k, v), stride)]
        return getattr(lib, name)(ref(c), ref(sp), tokens, *rows, ctypes.c_void_p(over.get("ws", WS)), 256, None)

    codes, scales, rows = 100 * 4 * 128 * 128, 1600, (4 * 4096 + ROW) * 2
    for name in ("msa_block_insert", "msa_cache_read"):
        for start, size in ((K, codes), (V, codes), (KS, scales), (VS, scales)):
            for at in (start, start + size - 16, start - rows + 16):  # inside, the last bytes, the first
                assert call(name, at, ROWS_V) == 1 and call(name, ROWS_K, at) == 1
    for name, start, size in (("c__k", K, codes), ("c__v", V, codes), ("c__k_scale", KS, scales), ("c__v_scale", VS, scales)):
        for other in ("s__first", "s__end", "s__token_offsets", "s__block_table"):
            assert call("msa_block_insert", ROWS_K, ROWS_V, **{other: start + size - 4}) == 1, (name, other)
        for other in {"c__k", "c__v", "c__k_scale", "c__v_scale"} - {name}:
            assert call("msa_block_insert", ROWS_K, ROWS_V, **{other: start + size - 16}) == 1, (name, other)
    for other in ("s__first", "s__end", "s__token_offsets", "s__block_table"):
        assert call("msa_cache_read", ROWS_K, ROWS_V, **{other: ROWS_K + rows - 4}) == 1
        assert call("msa_cache_read", ROWS_K, ROWS_V, **{other: ROWS_V}) == 1
    # K and V of the same rows: side by side or one behind the other, never on top of each other
    read = lambda d, **a: call("msa_cache_read", ROWS_K, ROWS_K + 2 * d, **a)  # noqa: E731
    for d in (0, 8, ROW - 8, 4096 - ROW + 8, 4096, 4 * 4096 - ROW + 8, 4 * 4096 + ROW - 8, -8, 8 - ROW, -4096, 8 - 4096 - ROW, -4 * 4096):
        assert read(d) == 1, d
    assert read(ROW, stride=(4096, 8192)) == 1 and read(0, tokens=1) == 1 and read(ROW - 8, tokens=1) == 1


def test_what_the_other_calls_refuse_of_a_cache_with_block_scales(lib):  # noqa: F811
    import block_sparse_attention_03_gb300 as msa
    ws = ctypes.c_void_p(4096)
    q = msa.MsaQueryT(16, 0, 1.0)
    rope, row = msa.msa_rope_init(128, 1e4), msa.MsaRowsT(16, 4096)
    for kv in (8, 9):
        c, b, f, _ = _structs(kv)
        # the index keys alone: K and V are written by msa_block_insert
        assert lib.msa_cache_insert(ref(c), 0, 16, None, None, 16, ws, 256, None) == 0
        for k, v in ((16, 16), (16, None), (None, 16)):
            assert lib.msa_cache_insert(ref(c), 4, 16, k, v, 16, ws, 256, None) == 2
        assert lib.msa_rope_insert(ref(c), ref(rope), 0, 16, 16, 16, ref(row), ref(q), None, None, None, None, None, None, ws, 256, None) == 0
        for k, v in ((ref(row), ref(row)), (ref(row), None), (None, ref(row))):
            assert lib.msa_rope_insert(ref(c), ref(rope), 4, 16, 16, 16, ref(row), ref(q), None, None, k, v, None, None, ws, 256, None) == 2
        # an index cache has no such format
        c2, _, _, _ = _structs(kv, c__index_dtype=kv)
        assert lib.msa_indexer_score(ref(c2), ref(b), ref(f), ref(q), 16, ws, 1 << 20, None) == 2
        assert lib.msa_cache_insert(ref(c2), 4, 16, None, None, 16, ws, 256, None) == 2

        def dense(hq=16, out=16, ws=ws, size=1 << 30, **over):
            c, b, f, _ = _structs(kv, **over)
            return lib.msa_dense_attend(ref(c), ref(b), ref(f), ref(q), hq, out, None, ws, size, None)

        need = lib.msa_dense_workspace_size(ref(c), ref(b), 16)
        assert need > 256 and dense(size=need - 1) == 3
        assert dense(c__k_scale=None) == 1 and dense(c__v_scale=4) == 1 and dense(hq=4 * 65) == 2 and dense(b__q_per_seq=9) == 2

        def sparse(hq=16, out=16, ws=ws, size=1 << 30, lists=16, lse=None, **over):
            c, b, f, _ = _structs(kv, **over)
            return lib.msa_sparse_attend(ref(c), ref(b), ref(f), ref(q), hq, lists, out, lse, ws, size, None)

        need = lib.msa_workspace_size(ref(c), ref(b), ref(f), 16)
        assert need > 256 and sparse(size=need - 1) == 3
        assert sparse(hq=4 * 65) == 2 and sparse(hq=15) == 1 and sparse(lists=None) == 1 and sparse(out=24) == 1
        assert sparse(lists=18) == 1 and sparse(lse=66) == 1 and sparse(ws=ctypes.c_void_p(4104)) == 1
        assert sparse(b__seq_lens=17) == 1 and sparse(b__block_table=18) == 1 and sparse(f__topk=5) == 2
        # the attend's part does not grow with the batch: the pooled scores alone do
        c3, b3, f3, _ = _structs(kv, b__num_seqs=4)
        assert lib.msa_workspace_size(ref(c3), ref(b3), ref(f3), 16) - need <= 2 * 4 * 50 * 4 + 256


def z(*s, dt=bf, at=0):
    return _Elsewhere(torch.zeros(s, dtype=dt), at)


def cut(*s, dt=i32):
    return _Elsewhere(torch.zeros((*s, 2), dtype=dt)[..., 0])


def _cache(msa, kv="int8_block", **over):
    t = dict(k=z(2, 2, 128, 128, dt=i8), v=z(2, 2, 128, 128, dt=u8), k_scale=z(2, 2, dt=f32), v_scale=z(2, 2, dt=f32))
    if kv == "fp8_block":
        t["k"] = z(2, 2, 128, 128, dt=torch.float8_e4m3fn)
    return msa.PagedCache(kv, "bf16", 2, 2, idx=None, **{**t, **over})


@pytest.mark.parametrize("kv", [8, 9])
def test_places_of_a_sequences_lists_are_counted_in_32_bits(lib, kv):  # noqa: F811
    for tokens, topk, ok in ((1 << 25, 32, False), (1 << 25, 16, True), (1 << 24, 32, True), (1 << 26, 16, False)):
        c, b, f, _ = _structs(kv, b__num_seqs=1, b__q_per_seq=tokens, b__max_blocks_per_seq=1 << 19, f__topk=topk)
        assert (lib.msa_workspace_size(ref(c), ref(b), ref(f), 16) > 0) == ok, (tokens, topk)




@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("name", ["msa_block_insert", "msa_cache_read"])
def test_python_refuses_what_the_kernels_would_misread(on_device_0, kv, name):  # noqa: F811
    msa = on_device_0

    def call(first, end, offsets, table, k, v, ws, **over):
        getattr(msa, name)(_cache(msa, kv, **over), msa.Spans(first, end, offsets, table), k, v, ws, stream=0)

    good = dict(first=z(3, dt=i32), end=z(3, dt=i32), offsets=z(4, dt=i32), table=z(3, 5, dt=i32), k=z(7, 2, 128), v=z(7, 2, 128),
                ws=z(256, dt=u8))
    bad = [("offsets", z(2, dt=i32)), ("table", z(2, 5, dt=i32)), ("table", z(15, dt=i32)), ("table", cut(3, 5)), ("ws", z(256, dt=u8, at=1)),
           ("k", z(6, 2, 128)), ("k", z(7, 1, 128)), ("v", z(7, 2, 64)), ("v", z(7, 2, 128, dt=torch.float16)),
           ("k", z(7, 2, 128, at=-1)), ("v", cut(7, 2, 128, dt=bf)), ("v", _Elsewhere(torch.zeros(7, 128, 2, dtype=bf).transpose(1, 2)))]
    for n in ("first", "end", "offsets"):
        bad += [(n, z(3, dt=torch.int64)), (n, z(3, dt=i32, at=1)), (n, cut(3))]
    bad += [("first", z(2, dt=i32)), ("end", z(4, dt=i32))]
    bad += [("k_scale", z(2, 1, dt=f32)), ("v_scale", z(2, 2, dt=bf)), ("k_scale", cut(2, 2, dt=f32)), ("v_scale", z(2, 2, dt=f32, at=1)),
            ("k", None) if name == "msa_block_insert" else ("k", z(7, 2, 127)),
            ("v", None) if name == "msa_block_insert" else ("v", z(7, 2, 127))]
    caches = [b for b in bad if b[0].endswith("_scale")]
    _refused(msa, call, good, [b for b in bad if b not in caches])
    for field, t in caches:
        with pytest.raises(msa.MsaError):
            call(**good, **{field: t})
    wide = torch.zeros(7, 5, 128, dtype=bf)
    _passes(call, **{**good, "k": _Elsewhere(wide[:, :2]), "v": _Elsewhere(wide[:, 3:])})


@pytest.mark.parametrize("kv", KINDS)
def test_python_looks_at_the_cache_in_every_attend(on_device_0, kv):  # noqa: F811
    msa = on_device_0
    batch, cfg, q = msa.Batch(z(3, dt=i32), z(3, 5, dt=i32)), msa.Config(), msa.Query(z(3, 4, 128))

    def dense(cache):
        msa.msa_dense_attend(cache, batch, cfg, q, 4, z(3, 4, 128), None, z(4096, dt=u8), stream=0)

    def sparse(cache):
        msa.msa_sparse_attend(cache, batch, cfg, q, 4, z(3, 2, 16, dt=i32), z(3, 4, 128), None, z(4096, dt=u8), stream=0)

    def decode(cache):
        msa.msa_decode(cache, batch, cfg, msa.Query(z(3, 2, 128)), q, 4, z(3, 2, 16, dt=i32), z(3, 4, 128), None, z(4096, dt=u8), stream=0)

    def noalloc(cache):
        msa.msa_decode_noalloc(cache, batch, cfg, msa.Query(z(3, 2, 128)), q, 4, z(3, 2, 16, dt=i32), z(3, 4, 128), None, stream=0)

    for call in (dense, sparse, decode, noalloc):
        _passes(call, cache=_cache(msa, kv))
        for over in (dict(k_scale=z(2, 1, dt=f32)), dict(v=z(1, 2, 128, 128, dt=u8)), dict(k=z(2, 2, 128, 128)),
                     dict(v_scale=z(2, 2, dt=f32, at=1))):
            with pytest.raises(msa.MsaError):
                call(cache=_cache(msa, kv, **over))


@pytest.mark.parametrize("kv", KINDS)
def test_python_refuses_what_the_sparse_attend_would_misread(on_device_0, kv):  # noqa: F811
    msa = on_device_0
    cache = _cache(msa, kv)

    def call(lens, table, q, lists, out, lse, ws, kind="bf16"):
        msa.msa_sparse_attend(cache, msa.Batch(lens, table, 2), msa.Config(topk=8), msa.Query(q, kind), 4, lists, out, lse, ws, stream=0)

    good = dict(lens=z(3, dt=i32), table=z(3, 5, dt=i32), q=z(6, 4, 128), lists=z(6, 2, 8, dt=i32), out=z(6, 4, 128), lse=z(6, 4, dt=f32),
                ws=z(4096, dt=u8))
    _refused(msa, call, good, [("lens", z(3, dt=torch.int64)), ("lens", cut(3)), ("table", z(2, 5, dt=i32)), ("table", z(15, dt=i32)),
                               ("table", cut(3, 5)), ("q", z(3, 4, 128)), ("q", z(6, 4, 128, dt=u8)), ("q", z(6, 4, 128, at=1)),
                               ("lists", z(6, 2, 16, dt=i32)), ("lists", z(6, 2, 8, dt=torch.int64)), ("lists", cut(6, 2, 8)),
                               ("lists", z(6, 2, 8, dt=i32, at=-1)), ("out", z(6, 4, 128, dt=f32)), ("out", cut(6, 4, 128, dt=bf)),
                               ("lse", z(3, 4, dt=f32)), ("lse", z(6, 4)), ("ws", z(4096, dt=u8, at=1)), ("kind", "fp8")])
    _passes(call, **{**good, "lse": None})


def test_growth_is_the_least_power_of_two():
    rng = np.random.default_rng(1)
    for a, b in np.float32(np.exp(rng.uniform(-80, 80, (500, 2)))):
        n = growth(a, b)
        assert np.ldexp(np.float64(a), n) >= b and (n == 0 or np.ldexp(np.float64(a), n - 1) < b)
    assert growth(np.float32(1), np.float32(1)) == 0 and growth(np.float32(1), np.nextafter(np.float32(1), np.float32(2))) == 1


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("pieces", [[300], [1] * 140, [1, 127, 1, 128, 40], [100, 200]])
def test_the_documented_insert_keeps_every_element(kv, pieces):
    # whatever the pieces: INT8 within a step of the present scale, E4M3 within its half step and a step of its subnormals
    rng = np.random.default_rng(len(pieces))
    T, H = sum(pieces), 2
    x = torch.from_numpy(rng.standard_normal((2, T, H, DIM)) * np.exp(rng.standard_normal((2, T, H, 1)))).bfloat16().float().numpy()
    cache = {n: np.full((4, H, BLOCK, DIM), 77, np.int8 if kv == "int8_block" else np.uint8) for n in "kv"}
    cache.update({n + "_scale": np.full((4, H), np.nan, np.float32) for n in "kv"})
    t = 0
    for n in pieces:
        plain_insert(kv, cache, [t], [t + n], [0], np.array([[2, 0, 3]]), x[0, t:t + n], x[1, t:t + n], 4)
        t += n
    for i, name in enumerate("kv"):
        for p in range(T):
            phys = (2, 0, 3)[p // BLOCK]
            s = cache[name + "_scale"][phys].astype(np.float64)[:, None]
            got = code_values(kv, cache[name][phys, :, p % BLOCK]) * s
            want = x[i, p].astype(np.float64)
            bound = s if kv == "int8_block" else 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -9 * s
            assert (np.abs(got - want) <= bound).all(), (name, p)
        assert (cache[name][1] == 77).all() and np.isnan(cache[name + "_scale"][1]).all()
        for blk in range(-(-T // BLOCK)):
            amax = np.abs(x[i, blk * BLOCK:(blk + 1) * BLOCK]).max((0, 2)).astype(np.float64) / float(TOP[kv])
            ratio = cache[name + "_scale"][(2, 0, 3)[blk]] / amax
            assert (ratio >= 1 - 2.0 ** -23).all() and (ratio <= 2 * (1 + 2.0 ** -22)).all()
