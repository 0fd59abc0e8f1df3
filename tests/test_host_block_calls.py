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
