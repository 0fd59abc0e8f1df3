"""Dense attend over FP8 caches whose V scales are far apart: scales near fp32's
smallest, large scales in rows that a query may not see, and large scales of keys
that weigh next to nothing.  Against the plain 64-bit attention."""

import numpy as np
import pytest
import torch

from oracle import msa_oracle as O

from _serving import DIM, check_dense, paged_case, plain_dense, run_dense

pytestmark = pytest.mark.gpu


def _codes(c, s, h, upto):
    index = {int(p): i for i, p in enumerate(c["perm"])}
    rows = [c["rows_v"][index[int(c["table"][s, b])], h].numpy() for b in range(-(-upto // 128))]
    with np.errstate(invalid="ignore"):
        return np.abs(O.e4m3_value(np.concatenate(rows)[:upto]).astype(np.float64))


def _scales(c, s, h, upto):
    index = {int(p): i for i, p in enumerate(c["perm"])}
    got = [c["rows_v_scale"][index[int(c["table"][s, b])], h].numpy() for b in range(-(-upto // 128))]
    return np.concatenate(got)[:upto].astype(np.float64)


def _reference(c):
    """plain_dense with the bound of weights below f16's normal range as the products give it: a
    column keeps p x vscale times 4 over the largest of them that it has met, so one below f16's
    normal numbers is off by half of 2^-24, 2^-27 of the largest (earlier steps' share decays with the
    largest itself; the sum of the weights is 1 or more): 2^-27 max(p vscale) sum |code| over the sum."""
    ref = plain_dense(c)
    q = c["q"].cpu()
    q = q.view(torch.int16).numpy().view(np.uint16) if c["qd"] == "bf16" else q.numpy()
    q = O.query_values(q, c["qd"], c["q_scale"]).astype(np.float64)
    index = {int(p): i for i, p in enumerate(c["perm"])}
    low, Q, r = ref[5] * 0, c["Q"], c["Hq"] // c["H"]
    for s, T in enumerate(c["lens"]):
        for h in range(c["H"] if T > 0 else 0):
            at = [index[int(c["table"][s, b])] for b in range(-(-T // 128))]
            with np.errstate(invalid="ignore"):
                k = np.concatenate([O.e4m3_value(c["rows_k"][i, h].numpy()).astype(np.float64) *
                                    c["rows_k_scale"][i, h].numpy().astype(np.float64)[:, None] for i in at])[:T]
            codes, vs = _codes(c, s, h, T), _scales(c, s, h, T)
            for i in range(Q):
                see = np.arange(T) <= T - Q + i
                for hh in range(h * r, (h + 1) * r):
                    x = k[see] @ q[s * Q + i, hh] * DIM ** -0.5
                    p = np.exp(x - x.max()) if see.any() else x
                    if see.any():
                        low[s * Q + i, hh] = 2.0 ** -27 * (p * vs[see]).max() * codes[see].sum(0) / p.sum()
    return ref[:5] + (low,)


def _set_scales(c, s, tokens, factor=None, value=None, codes=None):
    """V scales (and codes) of tokens of sequence s, in the cache and in the plain form's rows."""
    index = {int(p): i for i, p in enumerate(c["perm"])}
    for t in tokens:
        blk, off = int(c["table"][s, t // 128]), t % 128
        i = index[blk]
        new = c["rows_v_scale"][i, :, off] * factor if value is None else torch.full_like(c["rows_v_scale"][i, :, off], value)
        c["rows_v_scale"][i, :, off] = new
        c["v_scale"][blk, :, off] = new.cuda()
        if codes is not None:
            c["rows_v"][i, :, off] = codes
            c["v"][blk, :, off] = codes


@pytest.mark.parametrize("qd,Q,r", [("bf16", 1, 4), ("fp8", 2, 6), ("bf16", 4, 6), ("bf16", 8, 4), ("fp8", 8, 8)])
@pytest.mark.parametrize("runs", [1, 3, 9])
@pytest.mark.parametrize("codes", [None, 0])
def test_tiny_scales_behind_ordinary_ones(qd, Q, r, runs, codes):
    # V of one sign, so that the sums grow, then whole runs of 32 keys with scales of 1e-38 (the smallest
    # normal number is a usual floor for the scale of a row of zeros), with ordinary codes and with zeros
    T = 4096
    c = paged_case([T, 33 + Q], "fp8", qd, Q=Q, Hq=2 * r, H=2, seed=31)
    c["rows_v"] &= 0x7F
    c["v"] &= 0x7F
    for n in range(runs):
        at = 1024 + (512 if runs < 9 else 96) * n
        _set_scales(c, 0, range(at, at + 32 + 32 * (n % 3)), value=1e-38 if n % 2 == 0 else 3e-39, codes=codes)
    _set_scales(c, 1, range(32, 33), value=1e-38, codes=codes)
    check_dense(c, *run_dense(c), _reference(c))


@pytest.mark.parametrize("value", [1e-38, 3e-35])
@pytest.mark.parametrize("r", [1, 10])
def test_tiny_scales_in_long_segments(value, r):
    # enough sequences that each warp has added up many steps before the tiny scales come
    c = paged_case([2500] * 24, "fp8", "bf16", Q=1, Hq=8 * r, H=8, seed=37)
    c["rows_v"] &= 0x7F
    c["v"] &= 0x7F
    for s in range(24):
        for at in (1184, 1500, 2464):
            _set_scales(c, s, range(at, at + 64 if at < 2464 else 2500), value=value)
    check_dense(c, *run_dense(c), _reference(c))


@pytest.mark.parametrize("qd", ["bf16", "fp8"])
@pytest.mark.parametrize("r", [1, 4, 8])
@pytest.mark.parametrize("T", [20, 260])
@pytest.mark.parametrize("up", [20, 30, 60])
def test_a_later_tokens_large_scale_reaches_no_earlier_row(qd, r, T, up):
    Q = 5
    c = paged_case([T], "fp8", qd, Q=Q, Hq=r, H=1, seed=32)
    clean = _reference(c)
    _set_scales(c, 0, (T - 2, T - 1), factor=2.0 ** up)
    out, lse = run_dense(c)
    check_dense(c, out, lse, clean, rows=slice(0, 3))
    check_dense(c, out, lse, _reference(c), rows=slice(3, 5))


@pytest.mark.parametrize("up", [24, 60, 110])
@pytest.mark.parametrize("r,T", [(4, 30), (4, 700), (16, 700)])
def test_a_large_scale_that_weighs_next_to_nothing(up, r, T):
    # one key whose logits are far below the others': its weight times its scale is below theirs
    c = paged_case([T], "fp8", "bf16", Q=1, Hq=r, H=1, seed=33, spread=0.1)
    c["q"].copy_(c["q"].abs())
    t = T // 2
    blk, off = int(c["table"][0, t // 128]), t % 128
    i = {int(p): i for i, p in enumerate(c["perm"])}[blk]
    c["rows_k"][i, 0, off] = 0xFE  # -448
    c["k"][blk, 0, off] = 0xFE
    new = (up + 20) * np.log(2) * DIM ** 0.5 / (448 * c["q"].float().sum(-1).min().item())
    c["rows_k_scale"][i, 0, off] = new
    c["k_scale"][blk, 0, off] = new
    _set_scales(c, 0, (t,), factor=2.0 ** up)
    check_dense(c, *run_dense(c), _reference(c))


def test_scales_of_every_size():
    # scales from 2^-100 to 2^100 in no order: some row's largest product is anywhere in the sequence
    c = paged_case([1500, 129, 31], "fp8", "bf16", Q=2, Hq=8, H=2, seed=34)
    gen = torch.Generator().manual_seed(35)
    c["rows_v_scale"] *= torch.exp2(200 * torch.rand(c["rows_v_scale"].shape, generator=gen) - 100)
    c["v_scale"][c["perm"][:c["rows_v_scale"].shape[0]].cuda()] = c["rows_v_scale"].cuda()
    check_dense(c, *run_dense(c), _reference(c))


@pytest.mark.parametrize("value", [2.0 ** -120, 7.0e35, 3.0e38])
def test_a_cache_of_very_small_or_very_large_values(value):
    # 7e35 x 448 is close to bf16's largest number: sums of weighted rows stay below fp32's only with codes of 1
    c = paged_case([300, 17], "fp8", "fp8", Q=1, Hq=4, H=2, seed=36)
    code = None if value < 1 else 0x38 if value < 1e38 else 0x01  # 1 and 2^-9
    for s, T in enumerate(c["lens"]):
        _set_scales(c, s, range(T), value=value, codes=code)
    check_dense(c, *run_dense(c), _reference(c))
