"""Forms of the serving calls that the other tests leave out: NVFP4 products rounded
to E4M3 at every column count, the rotary insert with one of the two index tensors and
with the most heads, dense attends on several streams at once."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _serving import HALF, bind_dense, check_dense, dense_outputs, paged_case, plain_dense, plain_rope, run_dense
from test_rope_gpu import _cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qd", ["bf16", "fp8"])
@pytest.mark.parametrize("Q,r", [(1, 1), (1, 8), (4, 4), (3, 7), (8, 4), (5, 8), (8, 8), (6, 11)])
def test_rounded_products_at_every_column_count(qd, Q, r):
    c = paged_case([300, 0, Q, 131, 1], "nvfp4", qd, Q=Q, Hq=2 * r, H=2, seed=60 + Q)
    c["nv_mode"] = "e4m3"
    check_dense(c, *run_dense(c), plain_dense(c))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("T,Hq,H,index_q,index_k", [(3, 1024, 8, True, True), (5, 1024, 1, False, True), (70, 6, 3, True, False),
                                                    (40, 5, 5, False, True), (1, 1, 1, False, False)])
def test_one_of_the_index_tensors(kv, T, Hq, H, index_q, index_k):
    gen = torch.Generator().manual_seed(T + Hq)
    q, k, v, iq = (torch.randn((T, h, 128), generator=gen).bfloat16().cuda() for h in (Hq, H, H, H))
    ik = torch.randn((T, 128), generator=gen).bfloat16().cuda()
    cache, bufs = _cache(kv, kv, 1, H)
    pos = torch.randint(0, 5000, (2, T), generator=gen).int()
    out, iq_out = msa.Query(torch.zeros_like(q)), msa.Query(torch.zeros_like(iq)) if index_q else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_rope_insert(cache, msa.msa_rope_init(96, 1e4, [20, 28]), pos.cuda(), torch.arange(T, dtype=torch.int32).cuda(), q, out,
                        iq if index_q else None, iq_out, k, v, ik if index_k else None, None, ws)
    assert msa.msa_read_device_status(ws)[1] == 0

    def near(got, x):
        # angles to 2^-23 of half a turn, sine and cosine to two steps, two products and a sum: 6e-7 of the pair's length
        ref = plain_rope(x.float().cpu().numpy(), pos.numpy(), 96, 1e4, [20, 28], "halves")
        size = np.sqrt((ref ** 2).sum(-1, keepdims=True))
        assert (np.abs(got.float().cpu().numpy() - ref) <= HALF["bf16"] * np.abs(ref) + 1.3e-6 * size).all()

    near(out.data, q)
    if index_q:
        near(iq_out.data, iq)
    if kv == "bf16":
        near(bufs["k"][0, :, :T].transpose(0, 1), k)
        assert torch.equal(bufs["v"][0, :, :T].transpose(0, 1), v)
        if index_k:
            near(bufs["idx"][0, :T].unsqueeze(1), ik.unsqueeze(1))
    written = (bufs["idx"].view(torch.uint8)[0] != 0).any(-1)
    assert written[:T].all() if index_k else not written.any()
    assert not written[T:].any()


def test_several_streams_at_once():
    cases = [paged_case([3000, 500, 0, 1], kv, Q=2, Hq=8, H=2, seed=70 + i) for i, kv in enumerate(("fp8", "nvfp4", "bf16"))]
    calls = []
    for c in cases:
        cache, batch, q = bind_dense(c)
        ws = torch.empty(msa.msa_dense_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda")
        msa.msa_workspace_init(ws)
        calls.append((cache, batch, q, *dense_outputs(c), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for cache, batch, q, out, lse, ws, stream in calls:
            msa.msa_dense_attend(cache, batch, msa.default_config(), q, 8, out, lse, ws, stream)
    torch.cuda.synchronize()
    for c, (_, _, _, out, lse, ws, _) in zip(cases, calls):
        assert msa.msa_read_device_status(ws)[1] == 0
        check_dense(c, out, lse, plain_dense(c))
