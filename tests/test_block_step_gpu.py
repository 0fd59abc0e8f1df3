"""Caches with one scale for each block and head as a model runs them, step after step: block tables
from the requests' lengths, rotary positions of queries, keys and index keys, the block insert, the dense and
the sparse attend over what was inserted, and the read of a prefix, against a 64-bit model of each request."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _blocks import BLOCK, DIM, KINDS, code_values, empty_cache, workspace
from _serving import HALF, plain_rope

pytestmark = pytest.mark.gpu

THETA = 1.0e4


@pytest.mark.parametrize("kv,index", [("int8_block", "fp8"), ("fp8_block", "bf16")])
def test_prompts_then_decode_then_an_end(kv, index):
    gen = torch.Generator().manual_seed(1)
    S, Hq, H, pool, max_nb = 5, 8, 2, 24, 8
    cache = empty_cache(kv, pool, H, seed=2, index=index)  # whatever the memory held
    cache.idx = torch.zeros((pool, BLOCK, DIM), dtype=torch.bfloat16 if index == "bf16" else torch.uint8, device="cuda")
    if index == "fp8":
        cache.idx_scale = torch.zeros((pool, BLOCK), dtype=torch.float32, device="cuda")
    rope = msa.msa_rope_init(64, THETA)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cached, table, free, count = i32(S), i32(S, max_nb), torch.arange(pool, dtype=torch.int32, device="cuda"), i32(1)
    count.fill_(pool)
    seq_lens, offs, count2 = i32(S), i32(S + 1), i32(1)
    batch = msa.Batch(seq_lens, table, 1)
    spans = msa.Spans(cached, seq_lens, offs, table)  # beside the tables: the step's new tokens
    prefix = msa.Spans(i32(S), seq_lens, i32(S), table)
    cfg = msa.default_config(32)
    ws = workspace(max(msa.msa_dense_workspace_size(cache, batch, Hq), msa.msa_workspace_size(cache, batch, cfg, Hq)))
    keys, vals, lens = [[] for _ in range(S)], [[] for _ in range(S)], [0] * S
    # prompts, decode steps, an end whose blocks another request takes, a long one, and one (the last) that is refused: 7 of its 8
    # blocks are there
    plan = [([300, 1, 129, 0, 0], 0)] + [([1, 1, 1, 0, 0], 0)] * 3 + [([-1, 1, 1, 700, 0], 0)] + [([0, 1, 1, 1, 0], 0)] * 2 + \
        [([1000, 1, 1, 1, 0], 0), ([1, 1, 1, 1, 1000], 16)]
    for step, (new, fault) in enumerate(plan):
        T = sum(max(0, n) for n in new)
        qkv = torch.randn((T, Hq + 3 * H + 1, DIM), generator=gen)
        qkv = (qkv * torch.exp(0.5 * torch.randn((T, Hq + 3 * H + 1, 1), generator=gen)) * 1.3 ** step).bfloat16().cuda()
        q, k, v, iq, ik = qkv.split([Hq, H, H, H, 1], dim=1)
        slots, pos = i32(T), i32(T)
        msa.msa_build_tables(pool, cached, torch.tensor(new, dtype=torch.int32, device="cuda"), table, free, count, seq_lens, offs,
                             slots, pos, count2, ws)
        bf = lambda h: torch.zeros((T, h, DIM), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        q_out, iq_out, k_out = msa.Query(bf(Hq)), msa.Query(bf(H)), msa.Query(bf(H))
        msa.msa_rope_insert(cache, rope, pos, slots, q, q_out, iq, iq_out, None, None, ik.squeeze(1), None, ws)
        msa.msa_rope_insert(cache, rope, pos, slots, k, k_out, None, None, None, None, None, None, ws)
        msa.msa_block_insert(cache, spans, k_out.data, v, ws)
        offs_h = offs.cpu().tolist()
        last = [max(0, offs_h[s + 1] - 1) if new[s] > 0 else 0 for s in range(S)]
        qd, iqd = msa.Query(q_out.data[last].contiguous()), msa.Query(iq_out.data[last].contiguous())
        out = torch.full((S, Hq, DIM), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((S, Hq), dtype=torch.float32, device="cuda")
        msa.msa_dense_attend(cache, batch, msa.default_config(), qd, Hq, out, lse, ws)
        assert msa.msa_read_device_status(ws)[1] == fault
        # ---- the 64-bit model
        kh, vh = k.float().cpu().numpy(), v.float().cpu().numpy()
        for s, n in enumerate(new):
            if n < 0:
                lens[s], keys[s], vals[s] = 0, [], []
            if n > 0 and not (fault and s == S - 1):
                p = np.arange(lens[s], lens[s] + n)
                rows = slice(offs_h[s], offs_h[s] + n)
                keys[s].append(plain_rope(kh[rows], [p], 64, THETA, [32], "halves"))
                vals[s].append(vh[rows])
                lens[s] += n
        assert seq_lens.cpu().tolist() == lens
        # what the cache holds: the rotated keys, rounded to bf16 and then to the block's format
        tb = table.cpu().numpy()
        scales = {n: getattr(cache, n + "_scale").double().cpu().numpy() for n in "kv"}
        held = {n: code_values(kv, getattr(cache, n).cpu().numpy()) * scales[n][..., None, None] for n in "kv"}
        prefix.token_offsets.copy_(torch.tensor(np.cumsum([0] + lens[:-1]), dtype=torch.int32))
        total = sum(lens)
        back = torch.full((2, total + 1, H, DIM), 9.0, dtype=torch.bfloat16, device="cuda")
        msa.msa_cache_read(cache, prefix, back[0], back[1], ws)
        assert msa.msa_read_device_status(ws)[1] == 0 and (back[:, total] == 9).all()
        qh = qd.data.float().cpu().numpy().astype(np.float64)
        at = 0
        for s in range(S):
            T_s = lens[s]
            blocks = tb[s, :-(-T_s // BLOCK)]
            if T_s == 0:
                assert (out[s] == 0).all() and torch.isneginf(lse[s]).all()
                continue
            got = {}
            for name, rows in (("k", keys[s]), ("v", vals[s])):
                got[name] = np.concatenate([held[name][b] for b in blocks], 1)[:, :T_s]
                want = np.concatenate(rows).transpose(1, 0, 2)
                sc = np.repeat(scales[name][blocks].T, BLOCK, 1)[:, :T_s, None]
                step_size = sc if kv == "int8_block" else HALF["fp8"] * np.abs(want) * 1.01 + 2.0 ** -9 * sc
                assert (np.abs(got[name] - want) <= step_size + (2.0 ** -7 * np.abs(want) + 1e-5 if name == "k" else 0)).all(), (name, s)
                rows_back = back["kv".index(name), at:at + T_s].float().cpu().numpy().transpose(1, 0, 2)
                assert (np.abs(rows_back - got[name]) <= HALF["bf16"] * np.abs(got[name])).all()
            at += T_s
            if new[s] <= 0 or (fault and s == S - 1):
                continue
            for h in range(Hq):
                K, V = got["k"][h // (Hq // H)], got["v"][h // (Hq // H)]
                x = K @ qh[s, h] * DIM ** -0.5
                p = np.exp(x - x.max())
                ref, mass = p @ V / p.sum(), p @ np.abs(V) / p.sum()
                # weights far below the largest: one times its block's V scale is held as f16, 4 over the largest such
                # product, so below f16's normal numbers (2^-14) it is off by up to half of 2^-24: over 4, 2^-27 of that
                # largest product for each key, times the key's code
                vs = np.repeat(scales["v"][blocks][:, h // (Hq // H)], BLOCK)[:T_s]
                low = 2.0 ** -27 * (p * vs).max() * np.abs(V / vs[:, None]).sum(0) / p.sum()
                err = np.abs(out[s, h].float().cpu().numpy() - ref)
                assert (err <= HALF["bf16"] * np.abs(ref) + 2.0 ** -9 * mass + low).all(), (s, h)
                assert abs(float(lse[s, h]) - (x.max() + np.log(p.sum()))) < 1e-3
        # the sparse path over the same cache selects every block here (at most 8 of 32)
        live = [s for s in range(S) if lens[s] > 0 and new[s] > 0 and not (fault and s == S - 1)]
        sb = msa.Batch(seq_lens[live].contiguous(), table[live].contiguous(), 1)
        topk = torch.zeros((len(live), H, 32), dtype=torch.int32, device="cuda")
        sout = torch.zeros((len(live), Hq, DIM), dtype=torch.bfloat16, device="cuda")
        slse = torch.zeros((len(live), Hq), dtype=torch.float32, device="cuda")
        msa.msa_decode(cache, sb, cfg, msa.Query(iqd.data[live].contiguous()), msa.Query(qd.data[live].contiguous()), Hq,
                       topk, sout, slse, ws)
        assert msa.msa_read_device_status(ws)[1] == 0
        a, b = sout.float(), out[live].float()
        assert ((a - b).abs() <= 2.0 ** -7 * (b.abs() + b.abs().amax(-1, keepdim=True))).all()
        assert (slse - lse[live]).abs().max() < 1e-4
        cached.copy_(seq_lens)
        count.copy_(count2)


@pytest.mark.parametrize("kv", KINDS)
def test_rotary_insert_and_cache_insert_of_the_rest(kv):
    # queries and index keys come out as over any other cache, and K and V of the block cache stay as they are
    gen = torch.Generator().manual_seed(3)
    T, Hq, H, pool = 70, 4, 2, 3
    qkv = torch.randn((T, Hq + H + 2 * H + 1, DIM), generator=gen).bfloat16().cuda()
    q, iq, k, v, ik = qkv.split([Hq, H, H, H, 1], dim=1)
    ik = ik.squeeze(1)
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(pool * BLOCK, generator=gen)[:T].to(torch.int32).cuda()
    slots[5] = -1
    rope, norm = msa.msa_rope_init(128, THETA), msa.QkNorm(*(torch.randn(DIM, generator=gen).bfloat16().cuda() for _ in range(4)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    got = []
    for which in (kv, "fp8"):
        if which == "fp8":
            cache = msa.PagedCache("fp8", "fp8", pool, H, z(pool, H, BLOCK, DIM), z(pool, H, BLOCK, DIM), z(pool, BLOCK, DIM),
                                   k_scale=z(pool, H, BLOCK, dt=torch.float32), v_scale=z(pool, H, BLOCK, dt=torch.float32))
        else:
            cache = empty_cache(kv, pool, H, seed=4, index="fp8")
            cache.idx = z(pool, BLOCK, DIM)
        cache.idx_scale = z(pool, BLOCK, dt=torch.float32)
        before = [cache.k.clone(), cache.v.clone(), cache.k_scale.clone(), cache.v_scale.clone()]
        qo, iqo = z(T, Hq, DIM, dt=torch.bfloat16), z(T, H, DIM, dt=torch.uint8)
        kk, vv = (k, v) if which == "fp8" else (None, None)
        msa.msa_rope_insert(cache, rope, pos, slots, q, msa.Query(qo), iq, msa.Query(iqo, "fp8", 0.05), kk, vv, ik, norm, ws)
        idx = (cache.idx.clone(), cache.idx_scale.clone())
        cache.idx.zero_()
        msa.msa_cache_insert(cache, slots, kk if kk is None else kk.contiguous(), vv if vv is None else vv.contiguous(), ik.contiguous(), ws)
        got.append((qo, iqo, *idx, cache.idx, cache.idx_scale))
        assert msa.msa_read_device_status(ws)[1] == 0
        if which != "fp8":
            for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    with pytest.raises(msa.MsaError):
        msa.msa_rope_insert(cache if cache.kv_dtype == kv else empty_cache(kv, pool, H), rope, pos, slots, q, msa.Query(qo), None, None, k, v,
                            None, norm, ws)
