"""What the rotary insert stores for rows that it does not turn is, byte for byte,
what msa_cache_insert stores, which divides: infinities, NaN, elements and
per-tensor scales of every size."""

import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from test_rope_gpu import _cache

pytestmark = pytest.mark.gpu


def _same_bytes(kv, k, v, ik, g=2.0 ** -8, kinds=("v",)):
    """Both inserts of k, v, index k (positions 0); the kinds named have to agree."""
    T, H = v.shape[0], v.shape[1]
    pool = -(-T // 128)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    a, ab = _cache(kv, kv, pool, H, g)
    b, bb = _cache(kv, kv, pool, H, g)
    msa.msa_cache_insert(a, slots, k, v, ik, ws)
    out = msa.Query(torch.empty_like(k))
    msa.msa_rope_insert(b, msa.msa_rope_init(16, 1e4), torch.zeros(T, dtype=torch.int32, device="cuda"), slots, k, out, None, None, k,
                        v, ik, None, ws)
    assert msa.msa_read_device_status(ws)[1] == 0
    for name in ab:
        if name.split("_")[0] in kinds:
            x, y = ab[name].view(torch.uint8), bb[name].view(torch.uint8)
            assert torch.equal(x, y), (name, (x != y).nonzero()[:4].tolist(), int((x != y).sum()))


def _rows(T, H, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, 128), generator=gen) * torch.exp(spread * torch.randn((T, H, 128), generator=gen))
    return (x * torch.exp(spread * torch.randn((T, H, 1), generator=gen))).bfloat16().cuda(), gen


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_elements_that_are_not_finite(kv):
    x, gen = _rows(256, 2, 40)
    at = torch.rand((256, 2, 128), generator=gen).cuda()
    x[at < 0.01] = float("inf")
    x[at > 0.99] = float("-inf")
    x[(at > 0.5) & (at < 0.503)] = float("nan")
    x[7] = float("nan")
    x[8] = float("-inf")
    k, ik = _rows(256, 2, 41)[0], _rows(256, 1, 42)[0].squeeze(1)
    _same_bytes(kv, k, x, ik)


def test_bf16_copies_the_bits():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(256, 2, 128).cuda()
    _same_bytes("bf16", _rows(256, 2, 52)[0], x, _rows(256, 1, 53)[0].squeeze(1))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_zeros_of_either_sign(kv):
    x, gen = _rows(256, 2, 49)
    at = torch.rand((256, 2, 128), generator=gen).cuda()
    x[at < 0.1] = 0.0
    x[at > 0.9] = -0.0
    x[5] = -0.0
    _same_bytes(kv, _rows(256, 2, 50)[0], x, _rows(256, 1, 51)[0].squeeze(1))


@pytest.mark.parametrize("g", [2.0 ** -8, 0.1234, 1e-10, 1e-25, 3e-30, 1e30])
def test_nvfp4_with_elements_far_beyond_the_scale(g):
    # quotients that pass fp32's range on either side, infinities among ordinary elements
    x, gen = _rows(256, 2, 43, spread=20.0)
    x[torch.rand((256, 2, 128), generator=gen).cuda() < 0.002] = float("-inf")
    x[9] = -3.0e38
    _same_bytes("nvfp4", _rows(256, 2, 44)[0], x, _rows(256, 1, 45)[0].squeeze(1), g)


@pytest.mark.parametrize("kv,g", [("fp8", 1.0), ("nvfp4", 2.0 ** -8), ("nvfp4", 0.0371)])
@pytest.mark.parametrize("spread", [0.0, 1.0, 6.0])
def test_quotients_are_those_of_a_division(kv, g, spread):
    # 16,384 tokens of 4 heads: 8.4 million quotients, of every mantissa and of sizes far apart
    x, _ = _rows(16384, 4, 46, spread)
    _same_bytes(kv, _rows(16384, 4, 47)[0], x, _rows(16384, 1, 48)[0].squeeze(1), g)
