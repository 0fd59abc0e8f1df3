"""The serving operators as a model runs them, step after step over one cache:
block tables from the requests' lengths, rotary insert of the step's tokens,
dense attend (and the sparse path) over what was inserted, against a 64-bit
model of each request that keeps plain lists of rows."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa
from oracle import msa_oracle as O

from _serving import HALF, plain_rope
from test_rope_gpu import _cache

pytestmark = pytest.mark.gpu

THETA = 1.0e4


def _dequant_all(kv, bufs, name, g):
    raw = bufs[name].cpu()
    raw = raw.view(torch.int16).numpy().view(np.uint16) if kv == "bf16" else raw.numpy()
    return O._dequant(kv, raw, bufs[name + "_scale"].cpu().numpy() if kv == "fp8" else None,
                      bufs[name + "_sf"].cpu().numpy() if kv == "nvfp4" else None, g).astype(np.float64)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_prompts_then_decode_then_an_end(kv):
    gen = torch.Generator().manual_seed(1)
    S, Hq, H, pool, max_nb, g = 4, 8, 2, 24, 8, 2.0 ** -8
    cache, bufs = _cache(kv, kv, pool, H, g)
    rope = msa.msa_rope_init(64, THETA)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cached, table, free, count = i32(S), i32(S, max_nb), torch.arange(pool, dtype=torch.int32, device="cuda"), i32(1)
    count.fill_(pool)
    seq_lens, offs, count2 = i32(S), i32(S + 1), i32(1)
    batch = msa.Batch(seq_lens, table, 1)
    ws = torch.empty(max(msa.msa_dense_workspace_size(cache, batch, Hq),
                         msa.msa_workspace_size(cache, batch, msa.default_config(32), Hq)), dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    keys = [[] for _ in range(S)]  # K as the rotation gives it, before the cache's rounding
    lens = [0] * S
    # prompts of 300, 1, 129 and 0 tokens; then decode steps; then request 0 ends and request 3 begins in its blocks
    plan = [[300, 1, 129, 0]] + [[1, 1, 1, 0]] * 3 + [[-1, 1, 1, 700]] + [[0, 1, 1, 1]] * 2
    for new in plan:
        T = sum(max(0, n) for n in new)
        total = Hq + 3 * H + 1
        qkv = torch.randn((T, total, 128), generator=gen).bfloat16().cuda()
        q, k, v, iq, ik = qkv.split([Hq, H, H, H, 1], dim=1)
        slots, pos = i32(T + 2), i32(T + 2)
        msa.msa_build_tables(pool, cached, torch.tensor(new, dtype=torch.int32, device="cuda"), table, free, count, seq_lens, offs,
                             slots, pos, count2, ws)
        q_out = msa.Query(torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device="cuda"))
        iq_out = msa.Query(torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda"))
        msa.msa_rope_insert(cache, rope, pos[:T], slots[:T], q, q_out, iq, iq_out, k, v, ik.squeeze(1), None, ws)
        # the last token of every request attends to its whole sequence
        offs_h = offs.cpu().tolist()
        last = [max(0, offs_h[s + 1] - 1) if new[s] > 0 else 0 for s in range(S)]
        qd = msa.Query(q_out.data[last].contiguous())
        iqd = msa.Query(iq_out.data[last].contiguous())
        out = torch.full((S, Hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((S, Hq), dtype=torch.float32, device="cuda")
        msa.msa_dense_attend(cache, batch, msa.default_config(), qd, Hq, out, lse, ws)
        assert msa.msa_read_device_status(ws)[1] == 0
        cached.copy_(seq_lens)
        count.copy_(count2)
        # ---- the 64-bit model
        kh = k.float().cpu().numpy()
        for s, n in enumerate(new):
            if n < 0:
                lens[s], keys[s] = 0, []
            if n > 0:
                p = np.arange(lens[s], lens[s] + n)
                rot = plain_rope(kh[offs_h[s]:offs_h[s] + n], [p], 64, THETA, [32], "halves")
                keys[s].append(rot)
                lens[s] += n
        assert seq_lens.cpu().tolist() == lens
        tb, Kd, Vd = table.cpu().numpy(), _dequant_all(kv, bufs, "k", g), _dequant_all(kv, bufs, "v", g)
        qh = qd.data.float().cpu().numpy().astype(np.float64)
        held = set()
        for s in range(S):
            T_s = lens[s]
            blocks = tb[s, :-(-T_s // 128)].tolist()
            assert not held & set(blocks) and len(set(blocks)) == len(blocks)  # no block belongs to two requests
            held |= set(blocks)
            if T_s == 0:
                assert (out[s] == 0).all() and torch.isneginf(lse[s]).all()
                continue
            K = np.concatenate([Kd[b] for b in blocks], 1)[:, :T_s]
            V = np.concatenate([Vd[b] for b in blocks], 1)[:, :T_s]
            want = np.concatenate(keys[s]).transpose(1, 0, 2)
            # the cache holds the rotated keys to its format: bf16 half a step, e4m3 with the row's scale, e2m1 with its group's
            size = np.abs(want).max(-1, keepdims=True)
            step = {"bf16": HALF["bf16"] * np.abs(want), "fp8": HALF["fp8"] * np.abs(want) + 2.0 ** -10 * size / 448,
                    "nvfp4": size / 6 * (1 + 2.0 ** -4) + 2.0 ** -4 * np.abs(want)}[kv]
            assert (np.abs(K - want) <= step + 1e-5 * size).all(), (s, T_s)
            if new[s] <= 0:
                continue
            for h in range(Hq):
                x = K[h // (Hq // H)] @ qh[s, h] * 128 ** -0.5
                p = np.exp(x - x.max())
                ref = p @ V[h // (Hq // H)] / p.sum()
                mass = p @ np.abs(V[h // (Hq // H)]) / p.sum()
                err = np.abs(out[s, h].float().cpu().numpy() - ref)
                assert (err <= HALF["bf16"] * np.abs(ref) + 2.0 ** -9 * mass).all(), (s, h)
                assert abs(float(lse[s, h]) - (x.max() + np.log(p.sum()))) < 1e-3
        # the sparse path over the same cache selects every block here (at most 8 of 32)
        live = [s for s in range(S) if lens[s] > 0 and new[s] > 0]
        sb = msa.Batch(seq_lens[live].contiguous(), table[live].contiguous(), 1)
        topk = torch.zeros((len(live), H, 32), dtype=torch.int32, device="cuda")
        sout = torch.zeros((len(live), Hq, 128), dtype=torch.bfloat16, device="cuda")
        msa.msa_decode(cache, sb, msa.default_config(32), msa.Query(iqd.data[live].contiguous()), msa.Query(qd.data[live].contiguous()), Hq,
                       topk, sout, None, ws)
        assert msa.msa_read_device_status(ws)[1] == 0
        a, b = sout.float(), out[live].float()
        assert ((a - b).abs() <= 2.0 ** -6 * (b.abs() + b.abs().amax(-1, keepdim=True))).all()
