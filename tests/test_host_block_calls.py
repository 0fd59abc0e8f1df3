"""What the binding looks at in every call over caches with block scales, beside test_host_blocks.py (no GPU is touched)."""

import pytest
import torch

from test_host_blocks import KINDS, _cache, f32, i32, u8, z
from test_host_serving import on_device_0  # noqa: F401  (a fixture)
from test_host_types import _passes


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
