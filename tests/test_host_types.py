"""Types, sizes and devices that the Python binding of the serving calls refuses before
the library is reached (no GPU is touched)."""

import pytest
import torch

from test_host_serving import _Elsewhere, _refused, on_device_0  # noqa: F401  (a fixture)

bf, i32, u8, f32, e4m3 = torch.bfloat16, torch.int32, torch.uint8, torch.float32, torch.float8_e4m3fn


def z(*s, dt=bf, at=0):
    return _Elsewhere(torch.zeros(s, dtype=dt), at)


def _passes(call, **good):
    with pytest.raises(AssertionError):  # the fixture's library: the call was not refused
        call(**good)


def test_query_and_lse_types(on_device_0):  # noqa: F811
    msa = on_device_0
    cache = msa.PagedCache("bf16", "bf16", 2, 2, z(2, 2, 128, 128), z(2, 2, 128, 128), None)
    ws = z(4096, dt=u8)

    def dense(kind, data, lse):
        msa.msa_dense_attend(cache, msa.Batch(z(3, dt=i32), z(3, 5, dt=i32), 2), msa.Config(), msa.Query(data, kind), 4, z(6, 4, 128),
                             lse, ws, stream=0)

    good = dict(kind="bf16", data=z(6, 4, 128), lse=z(6, 4, dt=f32))
    _refused(msa, dense, good, [("data", z(6, 4, 128, dt=torch.float16)), ("data", z(6, 4, 128, dt=torch.int16)),
                                ("data", z(6, 4, 128, dt=u8)), ("kind", "fp8"), ("kind", "nvfp4"), ("lse", z(6, 4, dt=i32))])
    codes = dict(good, kind="fp8", data=z(6, 4, 128, dt=u8))
    _refused(msa, dense, codes, [("data", z(6, 4, 128, dt=torch.float8_e5m2)), ("data", z(6, 4, 128, dt=torch.bool)), ("kind", "bf16")])
    _passes(dense, **dict(codes, data=z(6, 4, 128, dt=e4m3)))
    _passes(dense, **dict(good, lse=None))


def test_rotary_insert_query_types(on_device_0):  # noqa: F811
    msa = on_device_0
    cache = msa.PagedCache("bf16", "bf16", 2, 2, z(2, 2, 128, 128), z(2, 2, 128, 128), None)
    rope = msa.MsaRopeT()
    rope.axes = 1

    def insert(kind, qo, ikind, iqo):
        msa.msa_rope_insert(cache, rope, z(3, dt=i32), z(3, dt=i32), z(3, 4, 128), msa.Query(qo, kind), z(3, 2, 128),
                            msa.Query(iqo, ikind), z(3, 2, 128), z(3, 2, 128), None, None, z(4096, dt=u8), stream=0)

    good = dict(kind="bf16", qo=z(3, 4, 128), ikind="fp8", iqo=z(3, 2, 128, dt=u8))
    _refused(msa, insert, good, [("qo", z(3, 4, 128, dt=torch.float16)), ("iqo", z(3, 2, 128, dt=torch.float8_e5m2)),
                                 ("ikind", "bf16"), ("kind", "fp8")])
    _passes(insert, **dict(good, iqo=z(3, 2, 128, dt=e4m3)))


FORMATS = {"bf16": {"": (bf, 128)}, "fp8": {"": (u8, 128), "_scale": (f32, 1)}, "nvfp4": {"": (u8, 64), "_sf": (u8, 8)}}
WRONG = {bf: torch.float16, u8: torch.float8_e5m2, f32: i32}


def _tensors(kv, idx, blocks=2, heads=2):
    got = {}
    for name, kind, h in (("k", kv, (heads,)), ("v", kv, (heads,)), ("idx", idx, ())):
        for part, (dt, width) in FORMATS[kind].items():
            got[name + part] = z(*((blocks, *h, 128) + (() if width == 1 else (width,))), dt=dt)
    return got


def _calls(msa, kv, idx):
    ws = z(4096, dt=u8)
    rope = msa.MsaRopeT()
    rope.axes = 1
    glob = dict(k_global=1.0, v_global=1.0, idx_global=1.0)

    def dense(**t):
        cache = t.pop("cache", None) or msa.PagedCache(kv, idx, 2, 2, **t, **glob)
        msa.msa_dense_attend(cache, msa.Batch(z(3, dt=i32), z(3, 5, dt=i32), 2), msa.Config(), msa.Query(z(6, 4, 128)), 4,
                             z(6, 4, 128), None, ws, stream=0)

    def insert(index=True, **t):
        cache = t.pop("cache", None) or msa.PagedCache(kv, idx, 2, 2, **t, **glob)
        msa.msa_rope_insert(cache, rope, z(3, dt=i32), z(3, dt=i32), z(3, 4, 128), msa.Query(z(3, 4, 128)), None, None, z(3, 2, 128),
                            z(3, 2, 128), z(3, 128) if index else None, None, ws, stream=0)

    return dense, insert


@pytest.mark.parametrize("kv,idx", [("bf16", "fp8"), ("fp8", "nvfp4"), ("nvfp4", "bf16")])
def test_every_tensor_of_the_cache(on_device_0, kv, idx):  # noqa: F811
    msa = on_device_0
    dense, insert = _calls(msa, kv, idx)
    good = _tensors(kv, idx)
    for name, t in good.items():
        shape, dt = t.shape, t.dtype
        bad = [z(*shape, dt=WRONG[dt]), z(*shape, dt=dt, at=1), z(*shape, dt=dt, at=-1), z(1, *shape[1:], dt=dt),
               _Elsewhere(torch.zeros((*shape, 2), dtype=dt)[..., 0])]
        if name.startswith("idx"):
            for x in bad:
                with pytest.raises(msa.MsaError):
                    insert(**{**good, name: x})
                _passes(dense, **{**good, name: x})  # not read
                _passes(insert, **{**good, name: x}, index=False)
        else:
            _refused(msa, dense, good, [(name, x) for x in bad])
            _refused(msa, insert, good, [(name, x) for x in bad])
    _passes(dense, **_tensors(kv, idx, blocks=3))  # more blocks than the pool uses


def test_the_check_follows_the_fields(on_device_0):  # noqa: F811
    msa = on_device_0
    dense, insert = _calls(msa, "fp8", "fp8")
    good = _tensors("fp8", "fp8")
    cache = msa.PagedCache("fp8", "fp8", 2, 2, **good)
    for call in (dense, insert, dense, insert):
        _passes(call, cache=cache)
    cache.v_scale = z(2, 2, 128, dt=f32, at=1)
    for call in (dense, insert):
        with pytest.raises(msa.MsaError):
            call(cache=cache)
    cache.v_scale = good["v_scale"]
    _passes(dense, cache=cache)
    cache.idx_scale = z(2, 128, dt=i32)
    _passes(dense, cache=cache)
    with pytest.raises(msa.MsaError):
        insert(cache=cache)
    cache.idx_scale = good["idx_scale"]
    _passes(insert, cache=cache)
    cache.num_blocks = 3
    with pytest.raises(msa.MsaError):
        dense(cache=cache)
