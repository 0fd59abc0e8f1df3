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
