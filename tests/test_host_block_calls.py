"""What the binding looks at in every call over caches with block scales, beside test_host_blocks.py (no GPU is touched)."""

import dataclasses
from types import SimpleNamespace

import pytest
import torch

from test_host_blocks import KINDS, _cache, f32, i32, u8, z
from test_host_serving import on_device_0  # noqa: F401  (a fixture)
from test_host_types import _passes, _tensors


@pytest.mark.parametrize("kv", KINDS)
def test_the_sparse_attend_does_not_go_without_lists(on_device_0, kv):  # noqa: F811
    msa = on_device_0

    def call(lists):
        msa.msa_sparse_attend(_cache(msa, kv), msa.Batch(z(3, dt=i32), z(3, 5, dt=i32), 2), msa.Config(topk=8),
                              msa.Query(z(6, 4, 128)), 4, lists, z(6, 4, 128), z(6, 4, dt=f32), z(4096, dt=u8), stream=0)

    with pytest.raises(msa.MsaError) as e:
        call(None)
    assert e.value.status == 1 and "msa_sparse_attend" in str(e.value)
    _passes(call, lists=z(6, 2, 8, dt=i32))


def _calls(msa, cache):
    """Each call over the holders of a batch, a query or spans: the holder's tensors by name, and the call."""
    batch, query = msa.Batch(z(3, dt=i32), z(3, 5, dt=i32), 2), msa.Query(z(6, 4, 128))
    spans = msa.Spans(z(3, dt=i32), z(3, dt=i32), z(4, dt=i32), z(3, 5, dt=i32))
    attends = {"seq_lens": batch.seq_lens, "block_table": batch.block_table, "data": query.data}
    pieces = {n: getattr(spans, n) for n in ("first", "end", "token_offsets", "block_table")}
    ws = z(4096, dt=u8)
    yield attends, lambda: msa.msa_dense_attend(cache, batch, msa.Config(), query, 4, z(6, 4, 128), None, ws, stream=0)
    if cache.kv_dtype != "bf16":
        yield attends, lambda: msa.msa_sparse_attend(cache, batch, msa.Config(topk=8), query, 4, z(6, 2, 8, dt=i32), z(6, 4, 128), None,
                                                     ws, stream=0)
        yield pieces, lambda: msa.msa_block_insert(cache, spans, z(7, 2, 128), z(7, 2, 128), ws, stream=0)
    yield pieces, lambda: msa.msa_cache_read(cache, spans, z(7, 2, 128), None, ws, stream=0)


def _plain_cache(msa, kv):
    return _cache(msa, kv) if kv != "bf16" else msa.PagedCache(kv, "bf16", 2, 2, z(2, 2, 128, 128), z(2, 2, 128, 128), None)


@pytest.mark.parametrize("kv", [*KINDS, "bf16"])
def test_types_and_devices_are_looked_at_in_every_call(on_device_0, kv):  # noqa: F811
    # t.data = other gives a tensor another type, or another device, under the same holder
    msa = on_device_0
    for tensors, call in _calls(msa, _plain_cache(msa, kv)):
        for name, t in tensors.items():
            _passes(call)
            was = t._t
            t._t.data = torch.zeros(t.shape, dtype=torch.float16 if name == "data" else torch.int64)
            with pytest.raises(msa.MsaError):
                call()
            t._t = was.new_zeros(was.shape, dtype=torch.bfloat16 if name == "data" else i32)
            _passes(call)
            t._at = 1
            with pytest.raises(msa.MsaError):
                call()
            t._at = -1
            with pytest.raises(msa.MsaError):
                call()
            t._at = 0
        _passes(call)


def _cache_calls(msa, kv):
    """Each call that looks at the cache's K and V, as a function of the cache."""
    batch, cfg, q = msa.Batch(z(3, dt=i32), z(3, 5, dt=i32)), msa.Config(), msa.Query(z(3, 4, 128))
    lists, out, ws, rope = z(3, 2, 16, dt=i32), z(3, 4, 128), z(4096, dt=u8), msa.MsaRopeT()
    rope.axes = 1
    spans = msa.Spans(z(3, dt=i32), z(3, dt=i32), z(4, dt=i32), z(3, 5, dt=i32))
    rows = z(3, 2, 128)
    yield lambda c: msa.msa_dense_attend(c, batch, cfg, q, 4, out, None, ws, stream=0)
    yield lambda c: msa.msa_cache_read(c, spans, rows, None, ws, stream=0)
    blk = kv in KINDS
    kv_rows = None if blk else rows
    yield lambda c: msa.msa_rope_insert(c, rope, z(3, dt=i32), z(3, dt=i32), z(3, 4, 128), msa.Query(z(3, 4, 128)), None, None, kv_rows,
                                        kv_rows, None, None, ws, stream=0)
    if blk:
        yield lambda c: msa.msa_block_insert(c, spans, rows, rows, ws, stream=0)
        yield lambda c: msa.msa_sparse_attend(c, batch, cfg, q, 4, lists, out, None, ws, stream=0)
        yield lambda c: msa.msa_decode(c, batch, cfg, msa.Query(rows), q, 4, lists, out, None, ws, stream=0)
        yield lambda c: msa.msa_decode_noalloc(c, batch, cfg, msa.Query(rows), q, 4, lists, out, None, stream=0)


def _taken(msa, kv):
    """A cache whose tensors may change in place."""
    if kv in KINDS:
        return _cache(msa, kv), ("k", "v", "k_scale", "v_scale")
    t = _tensors(kv, "bf16")
    return msa.PagedCache(kv, "bf16", 2, 2, **t, k_global=1.0, v_global=1.0), [n for n in t if n != "idx"]


@pytest.mark.parametrize("kv", [*KINDS, "bf16", "fp8", "nvfp4"])
def test_the_caches_tensors_are_looked_at_in_every_call(on_device_0, kv):  # noqa: F811
    msa = on_device_0
    for i in range(len(list(_cache_calls(msa, kv)))):
        cache, names = _taken(msa, kv)
        call = list(_cache_calls(msa, kv))[i]
        for name in names:
            t = getattr(cache, name)
            real, shape = t._t, t.shape
            address = real.data_ptr()
            _passes(call, c=cache)
            t._t.resize_(1, *shape[1:])  # at the same address
            assert real.data_ptr() == address
            with pytest.raises(msa.MsaError):
                call(cache)
            t._t.resize_(shape)
            _passes(call, c=cache)
            t._t.as_strided_(shape, [0] * len(shape))
            assert real.data_ptr() == address
            with pytest.raises(msa.MsaError):
                call(cache)
            t._t = real.new_zeros(shape)
            _passes(call, c=cache)  # at another address
            t._t.data = torch.zeros(shape, dtype=torch.float64)
            with pytest.raises(msa.MsaError):
                call(cache)
            t._t = real.new_zeros(shape)
            t._at = 1
            with pytest.raises(msa.MsaError):
                call(cache)
            t._at = 0
            _passes(call, c=cache)


@pytest.mark.parametrize("at", [-1, 1])
@pytest.mark.parametrize("kv", KINDS)
def test_a_cache_that_is_not_on_the_current_device(on_device_0, kv, at):  # noqa: F811
    msa = on_device_0
    for call in _cache_calls(msa, kv):
        cache = _cache(msa, kv)
        _passes(call, c=cache)
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(cache, name)._at = at
        with pytest.raises(msa.MsaError):
            call(cache)


def test_holders_of_a_callers_own(on_device_0):  # noqa: F811
    # anything with the fields will do, changed in place or not
    msa = on_device_0
    cfg = SimpleNamespace(**{f.name: f.default for f in dataclasses.fields(msa.Config)})
    batch, q = SimpleNamespace(seq_lens=z(3, dt=i32), block_table=z(3, 5, dt=i32), q_per_seq=1), SimpleNamespace(data=z(3, 4, 128), dtype="bf16", scale=1.0)

    def call(kv="bf16"):
        msa.msa_dense_attend(_plain_cache(msa, kv), batch, cfg, q, 4, z(3, 4, 128), None, z(4096, dt=u8), stream=0)

    for kv in (*KINDS, "bf16"):
        _passes(call, kv=kv)
    batch.seq_lens = z(2, dt=i32)
    with pytest.raises(msa.MsaError):
        call()
    spans = SimpleNamespace(first=z(3, dt=i32), end=z(3, dt=i32), token_offsets=z(4, dt=i32), block_table=z(3, 5, dt=i32))
    _passes(lambda: msa.msa_cache_read(_cache(msa), spans, z(7, 2, 128), None, z(256, dt=u8), stream=0))


def test_settings_follow_their_fields():
    import block_sparse_attention_03_gb300 as msa
    cfg = msa.Config()
    own = SimpleNamespace(**{f.name: f.default for f in dataclasses.fields(msa.Config)})
    seen = set()

    def same():  # (behind the struct: padding up to the next one's place)
        want = bytes(cfg.struct())
        assert msa._config_bytes(cfg) == msa._config_bytes(own) == want.ljust(len(msa._config_bytes(own)), b"\0")

    for name, value in (("topk", 8), ("init_blocks", 1), ("local_blocks", 2), ("index_scale", 0.5), ("sm_scale", 0.25),
                        ("score_type", "other"), ("prefill_select", "indexer")):
        same()
        seen.add(msa._config_bytes(cfg))
        setattr(cfg, name, value)
        setattr(own, name, value)
    same()
    assert len(seen) == 7
