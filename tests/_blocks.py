"""Caches with one scale for each block and head: builders of their inputs and plain
implementations of what writes and reads them.

plain_insert takes the documented operations one by one (an fp32 division, exponents and
mantissas compared, roundings to nearest even), so its codes and scales are compared for
equality; plain_attend is in 64 bits."""

from __future__ import annotations

import numpy as np
import torch

import block_sparse_attention_03_gb300 as msa
from oracle import msa_oracle as O

BLOCK, DIM = 128, 128
KINDS = ("int8_block", "fp8_block")
TOP = {"int8_block": np.float32(127), "fp8_block": np.float32(448)}
LEAST = np.float32(2.0 ** -126)
HALF_BF16 = 2.0 ** -8


def code_values(kv, codes):
    """fp64 values of codes (int8, or uint8 E4M3)."""
    if kv == "int8_block":
        return codes.view(np.int8).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return O.e4m3_value(codes.view(np.uint8)).astype(np.float64)


def codes_of(kv, x):
    """fp32 values as codes: nearest even, saturating, NaN as 0 (INT8) or NaN (E4M3)."""
    x = np.asarray(x, np.float32)
    if kv == "int8_block":
        with np.errstate(invalid="ignore"):
            return np.where(np.isnan(x), 0, np.clip(np.rint(x), -127, 127)).astype(np.int8)
    codes = torch.from_numpy(np.clip(x, np.float32(-448), np.float32(448))).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.where(np.isnan(x), np.uint8(0x7F), codes)


def growth(a, b):
    """The least k >= 0 with a 2^k >= b, of positive normal fp32 numbers."""
    (ma, ea), (mb, eb) = np.frexp(np.float32(a)), np.frexp(np.float32(b))
    return max(0, int(eb) - int(ea) + int(mb > ma))


def plain_insert(kv, cache, first, end, offsets, table, k, v, num_blocks):
    """Into cache {"k", "k_scale", "v", "v_scale"} (numpy, changed in place); k, v fp32 [T][H][128] of bf16 values."""
    T = len(k)
    for s in range(len(first)):
        a, b = int(first[s]), int(end[s])
        if b <= a or a < 0 or b > table.shape[1] * BLOCK or offsets[s] < 0 or offsets[s] + b - a > T:
            continue
        for blk in range(a // BLOCK, (b - 1) // BLOCK + 1):
            phys = int(table[s, blk])
            if not 0 <= phys < num_blocks:
                continue
            p0, p1 = max(a, blk * BLOCK), min(b, (blk + 1) * BLOCK)
            had = max(0, a - blk * BLOCK)
            for name, rows in (("k", k), ("v", v)):
                x = rows[offsets[s] + p0 - a:offsets[s] + p1 - a]
                for h in range(x.shape[1]):
                    y = x[:, h].astype(np.float32)
                    fine = np.abs(y[np.isfinite(y)])
                    amax = fine.max() if fine.size else np.float32(0)
                    need = max(np.float32(amax / TOP[kv]), LEAST)
                    data = cache[name][phys, h]
                    scale = need
                    if had:
                        old = cache[name + "_scale"][phys, h]
                        scale = old if np.isfinite(old) and old >= LEAST else LEAST
                        n = growth(scale, need)
                        if n:
                            scale = np.float32(np.ldexp(scale, n))
                            small = np.float32(np.ldexp(np.float32(1), -min(n, 126)))
                            data[:had] = codes_of(kv, code_values(kv, data[:had]).astype(np.float32) * small)
                    cache[name + "_scale"][phys, h] = scale
                    with np.errstate(invalid="ignore", over="ignore"):
                        data[p0 % BLOCK:p0 % BLOCK + p1 - p0] = codes_of(kv, y / scale)


def to_host(cache):
    return {n: getattr(cache, n).cpu().numpy().copy() for n in ("k", "v", "k_scale", "v_scale")}


def same_bits(a, b):
    return np.array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


def empty_cache(kv, pool, H, seed=0, index="bf16"):
    """A cache of which nothing is known: random codes, scales of any bits."""
    gen = torch.Generator().manual_seed(seed)
    t = {}
    for name in ("k", "v"):
        codes = torch.randint(0, 256, (pool, H, BLOCK, DIM), generator=gen, dtype=torch.uint8)
        t[name] = (codes.view(torch.int8) if kv == "int8_block" else codes).cuda()
        t[name + "_scale"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (pool, H), generator=gen).to(torch.int32).view(torch.float32).cuda()
    return msa.PagedCache(kv_dtype=kv, index_dtype=index, num_blocks=pool, num_kv_heads=H, idx=None, **t)


def status_words():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def spans(first, end, offsets, table):
    i = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).contiguous().cuda()  # noqa: E731
    return msa.Spans(i(first), i(end), i(offsets), i(table))


# ---------------------------------------------------------------- attends

def attend_case(kv, lens, qd="bf16", Q=1, Hq=4, H=2, seed=0, spread=0.5, scale_spread=0.0, qsize=1.0, pool=None, last=False):
    """Sequences of the given lengths in a cache with block scales.  Rows that no sequence holds are NaN
    (E4M3) or -128 (INT8), scales of blocks that none holds NaN, unused table entries far outside the pool.
    last: the sequences in the pool's last blocks."""
    gen = torch.Generator().manual_seed(seed)
    nbs = [-(-t // BLOCK) if t > 0 else 0 for t in lens]
    used = sum(nbs)
    pool = used + 2 if pool is None else pool
    max_nb = max(1, max(nbs)) + 1
    place = torch.randperm(used + 2 if not last else used, generator=gen)[:used] + (pool - used if last else 0)
    table = torch.full((len(lens), max_nb), -(1 << 30), dtype=torch.int32)
    holds = torch.zeros((used, BLOCK), dtype=torch.bool)
    at = 0
    for s, nb in enumerate(nbs):
        for b in range(nb):
            table[s, b] = int(place[at])
            holds[at, :min(BLOCK, lens[s] - b * BLOCK)] = True
            at += 1
    c = dict(kv=kv, qd=qd, Q=Q, Hq=Hq, H=H, lens=list(lens), table=table, pool=pool, place=place)
    dt = torch.int8 if kv == "int8_block" else torch.uint8
    hole = -128 if kv == "int8_block" else 0x7F
    for name in ("k", "v"):
        x = torch.randn((used, H, BLOCK, DIM), generator=gen) * torch.exp(spread * torch.randn((used, H, BLOCK, 1), generator=gen))
        x = x * holds[:, None, :, None]
        scale = (x.abs().amax((-1, -2)) / float(TOP[kv])).clamp(min=1e-30)
        rows = torch.from_numpy(codes_of(kv, (x / scale[..., None, None]).numpy()).copy())
        rows[~holds[:, None, :, None].expand_as(rows)] = hole
        scale = scale * torch.exp(scale_spread * torch.randn((used, H), generator=gen))
        full = torch.full((pool, H, BLOCK, DIM), hole, dtype=dt, device="cuda")
        fs = torch.full((pool, H), float("nan"), device="cuda")
        full[place.cuda()], fs[place.cuda()] = rows.cuda(), scale.cuda()
        c[name], c[name + "_scale"], c["rows_" + name], c["rows_" + name + "_scale"] = full, fs, rows, scale
    q = torch.randn((len(lens) * Q, Hq, DIM), generator=gen) * qsize
    if qd == "fp8":
        c["q_scale"] = 2.0 ** -6
        c["q"] = torch.from_numpy(codes_of("fp8_block", (q / c["q_scale"]).numpy()).copy()).cuda()
    else:
        c["q_scale"], c["q"] = 1.0, q.to(torch.bfloat16).cuda()
    return c


def bind(c):
    cache = msa.PagedCache(kv_dtype=c["kv"], index_dtype="bf16", num_blocks=c["pool"], num_kv_heads=c["H"], k=c["k"], v=c["v"],
                           idx=c.get("idx"), k_scale=c["k_scale"], v_scale=c["v_scale"])
    batch = msa.Batch(torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), c["table"].cuda(), c["Q"])
    return cache, batch, msa.Query(c["q"], c["qd"], c["q_scale"])


def outputs(c):
    rows = len(c["lens"]) * c["Q"]
    return (torch.full((rows, c["Hq"], DIM), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, c["Hq"]), 7.0, dtype=torch.float32, device="cuda"))


def workspace(n):
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    return ws


def run_attend(c, topk=None, want=0, ws=None, stream=None):
    """The dense attend, or the sparse one over the lists topk (int32 [rows][H][K] on the GPU)."""
    cache, batch, q = bind(c)
    cfg = msa.default_config(16 if topk is None else topk.shape[-1])
    if ws is None:
        ws = workspace(msa.msa_dense_workspace_size(cache, batch, c["Hq"]) if topk is None
                       else msa.msa_workspace_size(cache, batch, cfg, c["Hq"]))
    out, lse = outputs(c)
    if topk is None:
        msa.msa_dense_attend(cache, batch, cfg, q, c["Hq"], out, lse, ws, stream)
    else:
        msa.msa_sparse_attend(cache, batch, cfg, q, c["Hq"], topk, out, lse, ws, stream)
    st, flags = msa.msa_read_device_status(ws)
    assert flags == want, (st, flags)
    return out, lse


def _host(c, name, s, h, blocks):
    """(codes as fp64 [n][128], scale of each) of the given logical blocks of sequence s."""
    index = {int(p): i for i, p in enumerate(c["place"])}
    at = [index[int(c["table"][s, b])] for b in blocks]
    codes = code_values(c["kv"], np.concatenate([c["rows_" + name][i, h].numpy() for i in at]))
    return codes, np.repeat(np.array([c["rows_" + name + "_scale"][i, h].numpy() for i in at], np.float64), BLOCK)


def plain_attend(c, topk=None):
    """(out, lse, |v| average, logit error, keys seen, bound of small weights) of every row, in 64 bits; topk
    (numpy): the lists, entries that do not count taken out.

    A logit: 128 products summed in fp32 (at most 136 roundings of sums below sum |q k|); a bf16 query is f16
    after a power of two, exact to 2^-38 of the row's largest element; the scaled logit takes four roundings.
    A weight times its block's V scale is held as f16, 4 over the largest such product of the column so far:
    below f16's normal numbers it is off by half of 2^-24, 2^-27 of the largest."""
    q = c["q"].cpu()
    q = q.view(torch.int16).numpy().view(np.uint16) if c["qd"] == "bf16" else q.numpy()
    q = O.query_values(q, c["qd"], c["q_scale"]).astype(np.float64)
    Q, Hq, H = c["Q"], c["Hq"], c["H"]
    R, r = len(c["lens"]) * Q, Hq // H
    out, size, low = np.zeros((R, Hq, DIM)), np.zeros((R, Hq, DIM)), np.zeros((R, Hq, DIM))
    lse, ex, n = np.full((R, Hq), -np.inf), np.zeros((R, Hq)), np.zeros((R, Hq))
    for s, T in enumerate(c["lens"]):
        for h in range(H):
            for i in range(Q):
                row, pos = s * Q + i, T - Q + i
                if pos < 0:
                    continue
                blocks = list(range(pos // BLOCK + 1)) if topk is None else [b for b in topk[row, h] if b >= 0]
                if not blocks:
                    continue
                t = (np.array(blocks)[:, None] * BLOCK + np.arange(BLOCK)).reshape(-1)
                see = t <= pos
                (kc, ks), (vc, vs) = _host(c, "k", s, h, blocks), _host(c, "v", s, h, blocks)
                K, V = (kc * ks[:, None])[see], (vc * vs[:, None])[see]
                for hh in range(h * r, (h + 1) * r):
                    qv = q[row, hh]
                    x = K @ qv * DIM ** -0.5
                    mass = np.abs(K) @ np.abs(qv) * DIM ** -0.5
                    split = 2.0 ** -38 * np.abs(qv).max() * np.abs(K).sum(1) * DIM ** -0.5
                    ex[row, hh] = (mass * 136 * 2.0 ** -24 + split + np.abs(x) * 4 * 2.0 ** -23).max()
                    m = x.max()
                    p = np.exp(x - m)
                    lse[row, hh] = m + np.log(p.sum())
                    out[row, hh] = p @ V / p.sum()
                    size[row, hh] = p @ np.abs(V) / p.sum()
                    n[row, hh] = see.sum()
                    low[row, hh] = 2.0 ** -27 * (p * vs[see]).max() * np.abs(vc[see]).sum(0) / p.sum()
    return out, lse, size, ex, n, low


def check_attend(out, lse, ref, rows=None):
    """Half a step of bf16; before it every weight is off by the logit's error twice (itself and the sum's), ex2's
    2^-22 and the factors' roundings, its own rounding to f16 (2^-11), and the sums over n keys in fp32 by at most
    n / 8 roundings of a lane's run of them; and the bound of small weights."""
    rows = slice(None) if rows is None else rows
    got, gl = out.float().cpu().numpy().astype(np.float64)[rows], lse.cpu().numpy().astype(np.float64)[rows]
    o, l, size, ex, n, low = [x[rows] for x in ref]
    sums = (n / 8 + 64) * 2.0 ** -24
    weight = 2.0 ** -11 + 2 * ex + 2.0 ** -21 + 2 * sums
    tol = HALF_BF16 * np.abs(o) + (1 + HALF_BF16) * (size * weight[..., None] + low) + 1e-37
    assert np.isfinite(got).all()
    err = np.abs(got - o)
    assert (err <= tol).all(), (np.argwhere(err > tol)[:4], (err / tol).max())
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    ltol = ex + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, l)) + 2.0 ** -22
    lerr = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, l))
    assert (lerr <= ltol).all(), (lerr / ltol).max()


def select(c, K, seed=0, own=True):
    """Lists of K blocks that each (token, group) sees, its own among them, ascending, padded with -1."""
    rng = np.random.default_rng(seed)
    R, H = len(c["lens"]) * c["Q"], c["H"]
    got = np.full((R, H, K), -1, np.int32)
    for row in range(R):
        pos = c["lens"][row // c["Q"]] - c["Q"] + row % c["Q"]
        if pos < 0:
            continue
        last = pos // BLOCK
        for h in range(H):
            n = min(K, last + 1)
            pick = rng.choice(last + 1, n, replace=False)
            if own and last not in pick:
                pick[0] = last
            got[row, h, :n] = np.sort(pick)
    return got
