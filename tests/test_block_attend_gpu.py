"""Dense and sparse attend over caches with one scale for each block and head, against a plain
64-bit attention: head layouts and column counts, lengths of zero and one, causal rows, garbage in
every row that no query may see, scales far apart, lists with holes, faults."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _blocks import BLOCK, KINDS, attend_case, bind, check_attend, outputs, plain_attend, run_attend, select, workspace

pytestmark = pytest.mark.gpu

FORMATS = [(kv, qd) for kv in KINDS for qd in ("bf16", "fp8")]


def _gpu(lists):
    return torch.from_numpy(lists).cuda()


@pytest.mark.parametrize("kv,qd", FORMATS)
@pytest.mark.parametrize("length", [1, 15, 33, 127, 128, 129, 700])
def test_one_sequence(kv, qd, length):
    c = attend_case(kv, [length], qd, seed=length)
    check_attend(*run_attend(c), plain_attend(c))
    lists = select(c, 4, seed=length)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))


@pytest.mark.parametrize("kv,qd", FORMATS)
@pytest.mark.parametrize("Q,r,H", [(1, 1, 3), (7, 1, 1), (3, 4, 2), (8, 3, 1), (2, 16, 2), (8, 5, 1), (8, 8, 1), (6, 11, 1), (8, 16, 1)])
def test_columns(kv, qd, Q, r, H):
    c = attend_case(kv, [300, 0, Q, 131, max(1, Q - 1)], qd, Q=Q, Hq=r * H, H=H, seed=10 * Q + r)
    check_attend(*run_attend(c), plain_attend(c))


@pytest.mark.parametrize("kv,qd", FORMATS)
@pytest.mark.parametrize("Q,r,H,K", [(1, 1, 1, 8), (3, 4, 8, 16), (1, 12, 2, 32), (2, 17, 1, 4), (9, 24, 1, 8), (1, 33, 1, 16),
                                     (1, 64, 2, 4)])
def test_sparse_columns(kv, qd, Q, r, H, K):
    c = attend_case(kv, [2000, Q, 131, 900], qd, Q=Q, Hq=r * H, H=H, seed=10 * Q + r)
    lists = select(c, K, seed=r)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("Q,K,r,H", [(1, 16, 4, 2), (1, 32, 1, 8), (3, 32, 2, 2), (8, 8, 5, 1), (2, 4, 33, 1)])
@pytest.mark.parametrize("lens", ["short", "one long", "long and short"])
def test_lists_longer_than_the_sequences(kv, Q, K, r, H, lens):
    # more than 32 sequences, most with fewer blocks than a list has places; the entries in any order, padding among them
    gen = np.random.default_rng(K + Q)
    n = 37
    got = gen.integers(Q, 700, n)
    if lens == "one long":
        got[n // 2] = 128 * K + 700
    elif lens == "long and short":
        got[::2] = 128 * K + gen.integers(0, 900, len(got[::2]))
    got[:3] = Q, 128, 129
    c = attend_case(kv, [0] + [int(t) for t in got] + [0], Q=Q, Hq=r * H, H=H, seed=K)
    mine = gen.permuted(select(c, K, seed=Q), axis=-1)
    out, lse = run_attend(c, _gpu(mine), want=2)  # (the empty sequences)
    check_attend(out, lse, plain_attend(c, mine))


@pytest.mark.parametrize("kv", KINDS)
def test_many_ragged_sequences(kv):
    rng = np.random.default_rng(5)
    c = attend_case(kv, [int(x) for x in rng.integers(0, 900, 90)], Hq=4, H=2, seed=6)
    check_attend(*run_attend(c), plain_attend(c))
    c = attend_case(kv, [int(x) for x in rng.integers(1, 2000, 70)], Hq=8, H=2, seed=7)
    lists = select(c, 8, seed=1)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))


@pytest.mark.parametrize("kv,qd,Q,r", [("int8_block", "bf16", 1, 4), ("fp8_block", "fp8", 8, 4), ("int8_block", "fp8", 4, 16)])
def test_long_sequence_is_joined(kv, qd, Q, r):
    c = attend_case(kv, [20011, 37], qd, Q=Q, Hq=r, H=1, seed=8)
    check_attend(*run_attend(c), plain_attend(c))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("Q,r,H", [(1, 4, 2), (2, 6, 1), (6, 4, 1), (8, 4, 1), (3, 16, 1), (8, 8, 1)])
def test_as_many_segments_as_teams(kv, Q, r, H):
    rng = np.random.default_rng(100 * Q + r)
    lens = [int(x) for x in rng.choice([0, 1, 2, 63, 64, 65, 128, 129, 200, 257], 320 // H)] + [4003]
    rng.shuffle(lens)
    c = attend_case(kv, lens, Q=Q, Hq=r * H, H=H, seed=Q + r)
    check_attend(*run_attend(c), plain_attend(c))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("long,short", [(30000, 90), (60000, 100), (9000, 200)])
def test_a_long_sequence_among_many_short_ones(kv, long, short):
    # more segments than a quarter of the runs, and some that cross more than 32 of them, first, last and in between
    for at in (0, short // 2, short):
        lens = [100] * short
        lens.insert(at, long)
        c = attend_case(kv, lens, Hq=4, H=1, seed=at)
        out, lse = run_attend(c)
        ref = plain_attend({**c, "lens": [t if t == long or i < 3 else 0 for i, t in enumerate(lens)]})
        rows = [i for i, t in enumerate(lens) if t == long or i < 3]
        check_attend(out, lse, ref, rows=rows)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("r", [4, 16])
@pytest.mark.parametrize("qsize,scale_spread", [(6.0, 2.0), (1.0, 8.0), (0.01, 12.0)])
def test_large_logits_and_scales_far_apart(kv, r, qsize, scale_spread):
    c = attend_case(kv, [5000, 129], Q=2, Hq=r, H=1, seed=9, spread=1.0, qsize=qsize)
    rng = np.random.default_rng(3)  # V's scales alone, so that the logits stay those of the case
    new = c["rows_v_scale"] * torch.from_numpy(np.exp(scale_spread * rng.standard_normal(c["rows_v_scale"].shape))).float()
    c["rows_v_scale"] = new
    c["v_scale"][c["place"].cuda()] = new.cuda()
    check_attend(*run_attend(c), plain_attend(c))
    lists = select(c, 16, seed=4)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("first", [1e30, 1e-34])
def test_v_scales_from_one_end_of_fp32_to_the_other(kv, first):
    # the blocks in order: a huge one, then tiny ones (and the other way round)
    c = attend_case(kv, [128 * 9 + 5], Hq=4, H=1, seed=10)
    n = len(c["place"])
    scale = torch.tensor([[first if b < 3 else 1e-34 if first > 1 else 1e30] for b in range(n)])
    index = {int(p): i for i, p in enumerate(c["place"])}
    for b in range(n):
        c["rows_v_scale"][index[int(c["table"][0, b])]] = scale[b]
    c["v_scale"][c["place"].cuda()] = c["rows_v_scale"].cuda()
    check_attend(*run_attend(c), plain_attend(c))


@pytest.mark.parametrize("kv", KINDS)
def test_scales_that_are_not_finite_reach_only_who_sees_them(kv):
    # five new tokens, the last two in a block of their own whose scales are NaN and infinite
    Q, T = 5, 258
    c = attend_case(kv, [T], Q=Q, Hq=4, H=1, seed=11)
    clean = plain_attend(c)
    blk = int(c["table"][0, 2])
    c["k_scale"][blk, 0], c["v_scale"][blk, 0] = float("nan"), float("inf")
    out, lse = run_attend(c)
    check_attend(out, lse, clean, rows=slice(0, 3))
    assert torch.isnan(out[3:].float()).any(-1).all() and torch.isnan(lse[3:]).all()
    lists = select(c, 4)
    out, lse = run_attend(c, _gpu(lists))
    check_attend(out, lse, clean, rows=slice(0, 3))
    assert torch.isnan(lse[3:]).all()


def test_a_later_tokens_nan_codes_reach_no_earlier_row():
    Q, T = 5, 260
    for r in (1, 4, 8):
        c = attend_case("fp8_block", [T], Q=Q, Hq=r, H=1, seed=12)
        clean = plain_attend(c)
        for t in (T - 2, T - 1):
            c["k"][int(c["table"][0, t // BLOCK]), 0, t % BLOCK] = 0x7F
            c["v"][int(c["table"][0, t // BLOCK]), 0, t % BLOCK] = 0xFF
        out, lse = run_attend(c)
        check_attend(out, lse, clean, rows=slice(0, 3))
        assert torch.isnan(out[3:].float()).any(-1).all()


@pytest.mark.parametrize("kv", KINDS)
def test_a_query_that_is_not_finite_gives_nan(kv):
    c = attend_case(kv, [200, 200, 0], Hq=4, H=2, seed=13)
    clean = plain_attend(c)
    c["q"][0, 1, 5], c["q"][1, 2, 7], c["q"][2, 0, 0] = float("inf"), float("nan"), float("nan")
    out, lse = run_attend(c)
    assert torch.isnan(out[0, 1].float()).all() and torch.isnan(out[1, 2].float()).all() and torch.isnan(lse[0, 1])
    out[0, 1], out[1, 2] = torch.tensor(clean[0][0, 1]).cuda().bfloat16(), torch.tensor(clean[0][1, 2]).cuda().bfloat16()
    lse[0, 1], lse[1, 2] = float(clean[1][0, 1]), float(clean[1][1, 2])
    check_attend(out, lse, clean)  # the sequence without keys among them


@pytest.mark.parametrize("kv", KINDS)
def test_all_codes_zero(kv):
    c = attend_case(kv, [300], Hq=4, H=2, seed=14)
    for name in ("k", "v"):
        c["rows_" + name].zero_()
        c["rows_" + name + "_scale"].fill_(2.0 ** -126)
        c[name].zero_()
        c[name + "_scale"].fill_(2.0 ** -126)
    check_attend(*run_attend(c), plain_attend(c))


@pytest.mark.parametrize("kv", KINDS)
def test_faults_in_lengths_and_tables(kv):
    c = attend_case(kv, [300, 400, 500, 600], Hq=4, H=2, seed=15)
    clean = plain_attend(c)
    c["lens"][0], c["lens"][2] = -3, c["table"].shape[1] * BLOCK + 1
    good = int(c["table"][3, 1])
    c["table"][3, 1] = c["pool"]
    out, lse = run_attend(c, want=3)  # bad block, bad length
    for row in (0, 2):
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()
    check_attend(out, lse, clean, rows=slice(1, 2))
    assert torch.isfinite(lse[3]).all()
    # the sparse attend: the same, and entries that count for nothing
    lists = np.full((4, 2, 8), -1, np.int32)
    lists[1, 0, :3] = [3, 0, 2]        # any order
    lists[1, 1, 5] = 1                 # behind holes
    lists[3, 0, :8] = [0, 0, 1, 5, 4, 2, 2, -7]  # repeated, outside the pool, not there yet
    out, lse = run_attend(c, _gpu(lists), want=1 | 2 | 4)
    c["lens"][0], c["lens"][2], c["table"][3, 1] = 300, 500, good
    lists[3, 0] = [0, 4, 2, -1, -1, -1, -1, -1]
    ref = plain_attend(c, lists)
    check_attend(out, lse, ref, rows=[1, 3])
    assert torch.isneginf(lse[3, 2:]).all() and (out[3, 2:] == 0).all()  # an empty list
    for row in (0, 2):
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()


@pytest.mark.parametrize("kv", KINDS)
def test_offsets_past_32_bits(kv):
    # 5.4 GB for K and for V, the sequences in the last blocks
    c = attend_case(kv, [1000, 77], Hq=8, H=8, seed=16, pool=41000, last=True)
    check_attend(*run_attend(c), plain_attend(c))
    lists = select(c, 4, seed=2)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))


@pytest.mark.parametrize("kv", KINDS)
def test_captured_calls_on_another_stream_and_a_shared_workspace(kv):
    # a dense and a sparse call in one graph and one workspace, replayed with other lengths and rows in the same memory
    a = attend_case(kv, [3000, 200], Hq=8, H=2, seed=17)
    b = attend_case(kv, [700, 1], Hq=8, H=2, seed=18, pool=a["pool"])
    cache, batch, q = bind(a)
    cfg = msa.default_config(8)
    ws = workspace(max(msa.msa_dense_workspace_size(cache, batch, 8), msa.msa_workspace_size(cache, batch, cfg, 8)))
    (out, lse), (sout, slse) = outputs(a), outputs(a)
    lists = _gpu(select(a, 8, seed=3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def calls():
        msa.msa_dense_attend(cache, batch, cfg, q, 8, out, lse, ws)
        msa.msa_sparse_attend(cache, batch, cfg, q, 8, lists, sout, slse, ws)

    with torch.cuda.stream(side):
        calls()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    for seed, c in enumerate((a, b, a)):
        mine = select(c, 8, seed=seed)
        for name in ("k", "v", "k_scale", "v_scale"):
            a[name][c["place"].cuda()] = c["rows_" + name].cuda()
        batch.seq_lens.copy_(torch.tensor(c["lens"], dtype=torch.int32))
        batch.block_table.fill_(-9)
        batch.block_table[:, :c["table"].shape[1]].copy_(c["table"])
        lists.copy_(_gpu(mine))
        saved = a["q"].clone()
        a["q"].copy_(c["q"])
        for t in (out, lse, sout, slse):
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws)[1] == 0
        check_attend(out, lse, plain_attend(c))
        check_attend(sout, slse, plain_attend(c, mine))
        first = out.clone(), sout.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first[0], out) and torch.equal(first[1], sout)  # equal calls give equal bits
        a["q"].copy_(saved)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("Q,index", [(1, "bf16"), (3, "fp8"), (1, "nvfp4"), (16, "fp8"), (12, "bf16")])
def test_the_whole_path(kv, Q, index):
    # index scores, top-k and attend in one call, the attend against the selection that it wrote; without a workspace too
    import msa_synth as ms
    c = attend_case(kv, [2500, 131, 1000], Q=Q, Hq=8, H=2, seed=19)
    cache, batch, q = bind(c)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((c["pool"], BLOCK, 128), generator=gen)
    cache.index_dtype = index
    if index == "bf16":
        cache.idx = x.bfloat16().cuda()
    elif index == "fp8":
        codes, scale = ms.quantize_fp8_rows(x)
        cache.idx, cache.idx_scale = codes.cuda(), scale.cuda()
    else:
        codes, sf, g = ms.quantize_nvfp4(x)
        cache.idx, cache.idx_sf, cache.idx_global = codes.cuda(), sf.cuda(), g
    iq = msa.Query(torch.randn((3 * Q, 2, 128), generator=gen).bfloat16().cuda())
    cfg = msa.default_config(4)
    ws = workspace(msa.msa_workspace_size(cache, batch, cfg, 8))
    topk = torch.full((3 * Q, 2, 4), -5, dtype=torch.int32, device="cuda")
    out, lse = outputs(c)
    msa.msa_decode(cache, batch, cfg, iq, q, 8, topk, out, lse, ws)
    assert msa.msa_read_device_status(ws)[1] == 0
    lists = topk.cpu().numpy()
    pos = np.array([t - Q + i for t in c["lens"] for i in range(Q)])
    assert (lists.max(-1) == (pos // BLOCK)[:, None]).all()  # the newest block is always there
    check_attend(out, lse, plain_attend(c, lists))
    # the selection is that of the stages called by themselves
    pooled = torch.empty((3 * Q, 2, batch.block_table.shape[1]), device="cuda")
    alone = torch.empty_like(topk)
    msa.msa_indexer_score(cache, batch, cfg, iq, pooled, ws)
    msa.msa_topk_blocks(batch, cfg, 2, pooled, alone, None, ws)
    assert torch.equal(alone, topk)
    (out2, lse2), topk2 = outputs(c), torch.empty_like(topk)
    status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    msa.msa_decode_noalloc(cache, batch, cfg, iq, q, 8, topk2, out2, lse2, status)
    assert status.cpu().tolist()[0] == 0
    assert torch.equal(topk2, topk) and torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("kv", KINDS)
def test_tables_so_wide_that_a_batch_takes_several_launches(kv):
    # units of a launch are counted in 32 bits, by the width of the table: 31 sequences of 64 segments and 2^20 blocks
    wide, most, Q, r, H = 1 << 20, 31, 8, 64, 8
    lens = [int(t) for t in np.random.default_rng(5).integers(Q, 300, 40)]
    lens[3] = lens[35] = 0
    c = attend_case(kv, lens, Q=Q, Hq=r * H, H=H, seed=23)
    cache, batch, q = bind(c)
    cfg = msa.default_config(16)
    table = torch.full((len(lens), wide), -(1 << 30), dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"].cuda()

    def call(a, b, table):
        part = msa.Batch(batch.seq_lens[a:b], table[a:b].contiguous(), Q)
        out = torch.full(((b - a) * Q, r * H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(((b - a) * Q, r * H), 7.0, device="cuda")
        ws = workspace(msa.msa_dense_workspace_size(cache, part, r * H))
        msa.msa_dense_attend(cache, part, cfg, msa.Query(q.data[a * Q:b * Q]), r * H, out, lse, ws)
        assert msa.msa_read_device_status(ws)[1] == 0
        return out, lse

    out, lse = call(0, len(lens), table)
    for a, b in ((0, most), (most, len(lens))):
        want, want_lse = call(a, b, c["table"].cuda())  # (the same segments, so the same runs)
        assert torch.equal(out[a * Q:b * Q], want) and torch.equal(lse[a * Q:b * Q], want_lse)
    assert (out[3 * Q:4 * Q] == 0).all() and torch.isfinite(lse[:3 * Q]).all()


@pytest.mark.parametrize("kv", KINDS)
def test_queries_near_the_largest_bf16(kv):
    c = attend_case(kv, [300, 131], Q=2, Hq=8, H=2, seed=29)
    c["q"] = (c["q"].float().clamp(-3, 3) * 1.1e38).bfloat16()
    assert c["q"].abs().max() > 3e38 and torch.isfinite(c["q"]).all()
    for name in ("k_scale", "rows_k_scale"):
        c[name] = c[name] * 2e-36
    check_attend(*run_attend(c), plain_attend(c))
    lists = select(c, 4, seed=3)
    check_attend(*run_attend(c, _gpu(lists)), plain_attend(c, lists))
