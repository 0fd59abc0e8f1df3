"""Sparse attend over FP8 caches: blocks whose V scales are tiny behind ordinary
ones, against the dense attend over the same blocks (with as many blocks selected
as there are, both attend to the whole sequence)."""

import pytest
import torch

import block_sparse_attention_03_gb300 as msa
import msa_synth as ms

from _helpers import bind, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [1.2e-38, 1e-36, 3e-39])
@pytest.mark.parametrize("blocks", [(9,), (3, 5, 12)])
@pytest.mark.parametrize("q_per_seq", [1, 2])
def test_tiny_scales_behind_ordinary_ones(value, blocks, q_per_seq):
    # enough sequences that one split holds all of a sequence's blocks; V of one sign, so that sums grow
    S, T = 120, 2000
    w = ms.make_workload("fp8_decode", seq_lens=(T,) * S, q_per_seq=q_per_seq, seed=21)
    case = ms.make_case(w, device="cuda")
    cache, batch, iq, q = bind(case)
    cache.v.view(torch.uint8).bitwise_and_(0x7F)
    for b in blocks:
        phys = batch.block_table[:, b].long()
        cache.v_scale[phys] = value
    cfg = msa.default_config()
    rows = S * q_per_seq
    ws = workspace(cache, batch, cfg, w.num_q_heads)
    topk = torch.empty((rows, w.num_kv_heads, 16), dtype=torch.int32, device="cuda")
    out = torch.empty((rows, w.num_q_heads, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((rows, w.num_q_heads), dtype=torch.float32, device="cuda")
    msa.msa_decode(cache, batch, cfg, iq, q, w.num_q_heads, topk, out, lse, ws)
    assert msa.msa_read_device_status(ws)[1] == 0 and (topk >= 0).all()
    dws = torch.empty(msa.msa_dense_workspace_size(cache, batch, w.num_q_heads), dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(dws)
    dout, dlse = torch.empty_like(out), torch.empty_like(lse)
    msa.msa_dense_attend(cache, batch, cfg, q, w.num_q_heads, dout, dlse, dws)
    assert msa.msa_read_device_status(dws)[1] == 0
    assert torch.isfinite(out.float()).all() and (dlse - lse).abs().max() < 1e-4
    # each side rounds once to bf16; the sparse path's weights are two e4m3 terms (2^-8)
    a, b = out.float(), dout.float()
    assert ((a - b).abs() <= 2 * 2.0 ** -8 * b.abs() + 2.0 ** -8 * b.abs().amax()).all()
