"""Dense attend (msa_dense_attend) against a plain 64-bit attention over the
dequantized cache: every format, head layout and column count, lengths of zero
and one, blocks that end inside a tile, causal rows, NaN and infinity in every
row that no query may see, faults in the lengths and tables."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa

from _serving import DIM, bind_dense, check_dense, dense_outputs, paged_case, plain_dense, run_dense

pytestmark = pytest.mark.gpu

FORMATS = [("bf16", "bf16"), ("bf16", "fp8"), ("fp8", "bf16"), ("fp8", "fp8"), ("nvfp4", "bf16"), ("nvfp4", "fp8")]


@pytest.mark.parametrize("kv,qd", FORMATS)
@pytest.mark.parametrize("length", [1, 15, 16, 63, 64, 65, 127, 128, 129, 700])
def test_one_sequence(kv, qd, length):
    c = paged_case([length], kv, qd, seed=length)
    check_dense(c, *run_dense(c), plain_dense(c))


# query columns: 1 and 7 (one half-filled tile), 12 (one tile), 24 and 32 (two), 40 and 64
# (four), 66 and 128 (several groups of columns)
@pytest.mark.parametrize("kv,qd", FORMATS)
@pytest.mark.parametrize("Q,r,H", [(1, 1, 3), (7, 1, 1), (3, 4, 2), (8, 3, 1), (2, 16, 2), (8, 5, 1), (8, 8, 1), (6, 11, 1), (8, 16, 1)])
def test_columns(kv, qd, Q, r, H):
    c = paged_case([300, 0, Q, 131, max(1, Q - 1)], kv, qd, Q=Q, Hq=r * H, H=H, seed=10 * Q + r)
    check_dense(c, *run_dense(c), plain_dense(c))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_many_ragged_sequences(kv):
    # more segments than CTAs, and segments that cross the runs' borders
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 900, 90)]
    c = paged_case(lens, kv, Hq=4, H=2, seed=6)
    check_dense(c, *run_dense(c), plain_dense(c))


@pytest.mark.parametrize("kv,qd,Q,r", [("bf16", "bf16", 1, 4), ("fp8", "bf16", 1, 4), ("fp8", "fp8", 8, 4), ("nvfp4", "fp8", 8, 4),
                                       ("fp8", "bf16", 1, 16), ("nvfp4", "bf16", 4, 16)])
def test_long_sequence_is_joined(kv, qd, Q, r):
    c = paged_case([20011, 37], kv, qd, Q=Q, Hq=r, H=1, seed=8)
    check_dense(c, *run_dense(c), plain_dense(c))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("Q,r,H", [(1, 4, 2), (2, 6, 1), (6, 4, 1), (8, 4, 1), (3, 16, 1), (8, 8, 1)])
def test_as_many_segments_as_teams(kv, Q, r, H):
    # 1 to 64 columns; about as many short sequences as there are teams, so that runs begin and end
    # inside, before and behind the places that stand for segment ends, beside one that spans many runs
    rng = np.random.default_rng(100 * Q + r)
    lens = [int(x) for x in rng.choice([0, 1, 2, 63, 64, 65, 128, 129, 200, 257], 320 // H)] + [4003]
    rng.shuffle(lens)
    c = paged_case(lens, kv, Q=Q, Hq=r * H, H=H, seed=Q + r)
    check_dense(c, *run_dense(c), plain_dense(c))


def test_large_logits_and_uneven_scales():
    # a few keys take nearly all of the weight, and V's scales span 2^20
    c = paged_case([5000, 129], "fp8", Hq=4, H=2, seed=9, spread=2.5, qsize=6.0)
    check_dense(c, *run_dense(c), plain_dense(c))


def test_nvfp4_product_rounded_to_e4m3():
    c = paged_case([900, 300], "nvfp4", Q=2, Hq=8, H=2, seed=10)
    c["nv_mode"] = "e4m3"
    check_dense(c, *run_dense(c), plain_dense(c))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("r", [1, 4, 8])
def test_a_later_tokens_nan_reaches_no_earlier_row(kv, r):
    # the last two of five new tokens hold NaN and infinity in K and V: rows 0 to 2 must not see it
    Q, T = 5, 260
    c = paged_case([T], kv, Q=Q, Hq=r, H=1, seed=11)
    clean = plain_dense(c)
    for t in (T - 2, T - 1):
        blk, off = int(c["table"][0, t // 128]), t % 128
        if kv == "bf16":
            c["k"][blk, 0, off] = float("nan")
            c["v"][blk, 0, off, ::2] = float("inf")
            c["v"][blk, 0, off, 1::2] = float("nan")
        elif kv == "fp8":
            c["v"][blk, 0, off] = 0x7F
            c["k_scale"][blk, 0, off] = float("nan")
            c["v_scale"][blk, 0, off] = float("inf")
        else:
            c["k_sf"][blk, 0, off] = 0x7F
            c["v_sf"][blk, 0, off] = 0x7F
    out, lse = run_dense(c)
    check_dense(c, out, lse, clean, rows=slice(0, 3))
    assert torch.isnan(out[3:].float()).any(-1).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_a_query_that_is_not_finite_gives_nan(kv):
    c = paged_case([200, 200], kv, Hq=4, H=2, seed=12)
    clean = plain_dense(c)
    c["q"][0, 1, 5] = float("inf")
    c["q"][1, 2, 7] = float("nan")
    out, lse = run_dense(c)
    bad = torch.zeros((2, 4), dtype=torch.bool)
    bad[0, 1] = bad[1, 2] = True
    assert torch.isnan(out.float().cpu()).all(-1).eq(bad).all() and torch.isnan(lse.cpu()).eq(bad).all()
    fill = torch.tensor(clean[0][bad.numpy()]).float().cuda()
    out[bad.cuda()] = fill.bfloat16()
    lse[bad.cuda()] = torch.tensor(clean[1][bad.numpy()]).float().cuda()
    check_dense(c, out, lse, clean)


def test_faults_in_lengths_and_tables():
    c = paged_case([300, 400, 500, 600], "fp8", Hq=4, H=2, seed=13)
    clean = plain_dense(c)
    lens = list(c["lens"])
    c["lens"][0], c["lens"][2] = -3, c["table"].shape[1] * 128 + 1
    c["table"][3, 1] = c["pool"]
    out, lse = run_dense(c, want=3)  # bad block, bad length
    for row in (0, 2):
        assert (out[row] == 0).all() and torch.isneginf(lse[row]).all()
    check_dense(c, out, lse, clean, rows=slice(1, 2))
    c["lens"] = lens
    c["table"][3, 1] = c["table"][3, 0]  # a block of the pool again for the plain form, which leaves it out
    check_dense(c, out, lse, plain_dense(c, skip_blocks=(1,)), rows=slice(3, 4))


def test_offsets_past_32_bits():
    # a pool of 5.4 GB for K and for V, the sequences in its last blocks
    c = paged_case([1000, 77], "fp8", Hq=8, H=8, seed=14, pool=41000)
    c["perm"], old = torch.arange(41000 - len(c["perm"]), 41000), c["perm"]
    for key in ("k", "v", "k_scale", "v_scale"):
        c[key][c["perm"].cuda()] = c["rows_" + key].cuda()
    where = {int(p): i for i, p in enumerate(old)}
    for s in range(2):
        for b in range(c["table"].shape[1]):
            if int(c["table"][s, b]) >= 0:
                c["table"][s, b] = int(c["perm"][where[int(c["table"][s, b])]])
    check_dense(c, *run_dense(c), plain_dense(c))


def test_equal_calls_give_equal_bits_and_workspaces_are_shared():
    import msa_synth as ms
    from _helpers import bind
    c = paged_case([7000, 3000, 1], "fp8", Hq=8, H=2, seed=15)
    cache, batch, q = bind_dense(c)
    w = ms.make_workload("fp8_decode", seq_lens=(3000, 1700), seed=7)
    case = ms.make_case(w, device="cuda")
    scache, sbatch, siq, sq = bind(case)
    cfg = msa.default_config()
    n = max(msa.msa_dense_workspace_size(cache, batch, 8), msa.msa_workspace_size(scache, sbatch, cfg, 16))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    first = run_dense(c)
    ref = plain_dense(c)
    topk = torch.empty((2, 4, 16), dtype=torch.int32, device="cuda")
    sout = torch.empty((2, 16, 128), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):  # the sparse path's leftovers in the workspace change nothing
        msa.msa_decode(scache, sbatch, cfg, siq, sq, 16, topk, sout, None, ws)
        again = run_dense(c, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    check_dense(c, *first, ref)


def test_captured_calls_on_another_stream():
    # two calls in one graph, replayed with other lengths, queries and cache rows in the same memory
    c = paged_case([900, 200], "fp8", Hq=4, H=2, seed=16)
    d = paged_case([700, 0], "fp8", Hq=4, H=2, seed=17, pool=c["pool"])
    cache, batch, q = bind_dense(c)
    ws = torch.empty(msa.msa_dense_workspace_size(cache, batch, 4), dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    out, lse = dense_outputs(c)
    out2, _ = dense_outputs(c)
    cfg = msa.default_config()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        msa.msa_dense_attend(cache, batch, cfg, q, 4, out, lse, ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            msa.msa_dense_attend(cache, batch, cfg, q, 4, out, lse, ws)
            msa.msa_dense_attend(cache, batch, cfg, q, 4, out2, None, ws)
    torch.cuda.synchronize()
    for x in (c, d, c):
        for key in ("k", "v", "k_scale", "v_scale"):
            c[key][x["perm"].cuda()] = x["rows_" + key].cuda()
        batch.seq_lens.copy_(torch.tensor(x["lens"], dtype=torch.int32))
        batch.block_table.fill_(-9)
        batch.block_table[:, :x["table"].shape[1]].copy_(x["table"][:, :batch.block_table.shape[1]])
        saved = c["q"].clone()
        c["q"].copy_(x["q"])
        out.fill_(3)
        out2.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert msa.msa_read_device_status(ws)[1] == 0
        check_dense(x, out, lse, plain_dense(x))
        assert torch.equal(out, out2)
        c["q"].copy_(saved)


def test_two_graphs_share_a_workspace():
    # of different column counts, so that they lay it out differently, replayed in turn
    a, b = paged_case([5000, 77], "fp8", Hq=4, H=2, seed=21), paged_case([900, 3000, 0], "nvfp4", Q=8, Hq=8, H=2, seed=22)
    cfg, calls = msa.default_config(), []
    for c in (a, b):
        cache, batch, q = bind_dense(c)
        calls.append((c, cache, batch, q, c["Hq"], *dense_outputs(c)))
    ws = torch.full((max(msa.msa_dense_workspace_size(x[1], x[2], x[4]) for x in calls),), 0x5a, dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    graphs = []
    for c, cache, batch, q, hq, out, lse in calls:
        msa.msa_dense_attend(cache, batch, cfg, q, hq, out, lse, ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            msa.msa_dense_attend(cache, batch, cfg, q, hq, out, lse, ws)
    refs = [plain_dense(c) for c, *_ in calls]
    for n in (0, 1, 1, 0, 1):
        calls[n][5].fill_(3)
        calls[n][6].fill_(3)
        graphs[n].replay()
        torch.cuda.synchronize()
        check_dense(calls[n][0], calls[n][5], calls[n][6], refs[n])
    assert msa.msa_read_device_status(ws)[1] == 0


def test_equals_the_sparse_attend_that_selects_every_block():
    # with topk at least the number of blocks the sparse path attends to the whole sequence
    import msa_synth as ms
    from _helpers import bind, workspace
    w = ms.make_workload("fp8_decode", seq_lens=(2000, 1100), seed=18)
    case = ms.make_case(w, device="cuda")
    cache, batch, iq, q = bind(case)
    cfg = msa.default_config()
    ws = workspace(cache, batch, cfg, 16)
    topk = torch.empty((2, 4, 16), dtype=torch.int32, device="cuda")
    out = torch.empty((2, 16, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 16), dtype=torch.float32, device="cuda")
    msa.msa_decode(cache, batch, cfg, iq, q, 16, topk, out, lse, ws)
    dws = torch.empty(msa.msa_dense_workspace_size(cache, batch, 16), dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(dws)
    dout, dlse = torch.empty_like(out), torch.empty_like(lse)
    msa.msa_dense_attend(cache, batch, cfg, q, 16, dout, dlse, dws)
    assert msa.msa_read_device_status(dws)[1] == 0
    assert (dlse - lse).abs().max() < 1e-4
    # each side rounds once to bf16; the sparse path's weights are two e4m3 terms (2^-8)
    a, b = out.float(), dout.float()
    assert ((a - b).abs() <= 2 * 2.0 ** -8 * b.abs() + 2.0 ** -8 * b.abs().amax()).all()
