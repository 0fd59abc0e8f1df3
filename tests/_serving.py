"""Plain 64-bit implementations of the serving operators around the path
(dense attend, rotary insert, block tables) and builders of their inputs."""

from __future__ import annotations

import numpy as np
import torch

import block_sparse_attention_03_gb300 as msa
import msa_synth as ms
from oracle import msa_oracle as O

BLOCK, DIM = 128, 128
HALF = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4}  # half a step, relative


def _bits(x: torch.Tensor) -> torch.Tensor:
    return x.to(torch.bfloat16)


def paged_case(lens, kv="bf16", qd="bf16", Q=1, Hq=4, H=2, seed=0, spare=2, pool=None, spread=0.5, qsize=1.0):
    """A paged K / V cache holding sequences of the given lengths, on the GPU.  Rows that no
    sequence holds are NaN (codes, scales or elements); unused table entries are far outside the pool."""
    gen = torch.Generator().manual_seed(seed)
    nbs = [-(-t // BLOCK) if t > 0 else 0 for t in lens]
    used = sum(nbs)
    pool = used + spare if pool is None else pool
    max_nb = max(1, max(nbs)) + 1
    perm = torch.randperm(pool, generator=gen)[pool - used:] if pool > 10 * used else torch.randperm(pool, generator=gen)[:used]
    table = torch.full((len(lens), max_nb), -(1 << 30), dtype=torch.int32)
    holds = torch.zeros((used, BLOCK), dtype=torch.bool)
    at = 0
    for s, nb in enumerate(nbs):
        for b in range(nb):
            table[s, b] = int(perm[at])
            holds[at, :min(BLOCK, lens[s] - b * BLOCK)] = True
            at += 1
    case = dict(kv=kv, qd=qd, Q=Q, Hq=Hq, H=H, lens=list(lens), table=table, pool=pool, perm=perm, nv_mode="exact")
    for name in ("k", "v"):
        x = torch.randn((used, H, BLOCK, DIM), generator=gen)
        x = x * torch.exp(spread * torch.randn((used, H, BLOCK, 1), generator=gen))
        dead = ~holds[:, None, :, None].expand(used, H, BLOCK, DIM)
        full = {}
        if kv == "bf16":
            rows = _bits(x)
            rows[dead] = float("nan") if name == "k" else float("inf")
            full[name] = (rows, float("nan"))
        elif kv == "fp8":
            codes, scale = ms.quantize_fp8_rows(x)
            codes[dead] = 0x7F
            scale[dead[..., 0]] = float("nan")
            full[name], full[name + "_scale"] = (codes, 0x7F), (scale, float("nan"))
        else:
            codes, sf, g = ms.quantize_nvfp4(x)
            sf[dead[..., 0]] = 0x7F
            full[name], full[name + "_sf"] = (codes, 0x77), (sf, 0x7F)
            case[name + "_global"] = g
        for key, (rows, fill) in full.items():
            buf = torch.full((pool,) + tuple(rows.shape[1:]), fill, dtype=rows.dtype, device="cuda")
            buf[perm.cuda()] = rows.cuda()
            case[key] = buf
            case["rows_" + key] = rows  # by position in `perm`
    q = torch.randn((len(lens) * Q, Hq, DIM), generator=gen) * qsize
    if qd == "fp8":
        codes, scale = ms.quantize_fp8_tensor(q)
        case["q"], case["q_scale"] = codes.cuda(), scale
    else:
        case["q"], case["q_scale"] = _bits(q).cuda(), 1.0
    return case


def bind_dense(c):
    cache = msa.PagedCache(kv_dtype=c["kv"], index_dtype=c["kv"], num_blocks=c["pool"], num_kv_heads=c["H"], k=c["k"], v=c["v"],
                           idx=None, k_sf=c.get("k_sf"), v_sf=c.get("v_sf"), k_scale=c.get("k_scale"), v_scale=c.get("v_scale"),
                           k_global=c.get("k_global", 0.0), v_global=c.get("v_global", 0.0), nvfp4_mode=c["nv_mode"])
    batch = msa.Batch(torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), c["table"].cuda(), c["Q"])
    return cache, batch, msa.Query(c["q"], c["qd"], c["q_scale"])


def dense_outputs(c):
    rows = len(c["lens"]) * c["Q"]
    return (torch.full((rows, c["Hq"], DIM), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, c["Hq"]), 7.0, dtype=torch.float32, device="cuda"))


def run_dense(c, want=0, ws=None, stream=None):
    cache, batch, q = bind_dense(c)
    if ws is None:
        ws = torch.full((msa.msa_dense_workspace_size(cache, batch, c["Hq"]),), 0xFF, dtype=torch.uint8, device="cuda")
        msa.msa_workspace_init(ws)
    out, lse = dense_outputs(c)
    msa.msa_dense_attend(cache, batch, msa.default_config(), q, c["Hq"], out, lse, ws, stream)
    st, flags = msa.msa_read_device_status(ws)
    assert flags == want, (st, flags)
    return out, lse


def _host_rows(c, name, s, h, upto):
    """fp64 rows of K or V of the first `upto` tokens of sequence s."""
    index = {int(p): i for i, p in enumerate(c["perm"])}
    got = []
    for b in range(-(-upto // BLOCK)):
        i = index[int(c["table"][s, b])]
        raw = c["rows_" + name][i, h]
        raw = raw.view(torch.int16).numpy().view(np.uint16) if c["kv"] == "bf16" else raw.numpy()
        scale = c["rows_" + name + "_scale"][i, h].numpy() if c["kv"] == "fp8" else None
        sf = c["rows_" + name + "_sf"][i, h].numpy() if c["kv"] == "nvfp4" else None
        with np.errstate(invalid="ignore"):
            got.append(O._dequant(c["kv"], raw, scale, sf, c.get(name + "_global"), c["nv_mode"]).astype(np.float64))
    return np.concatenate(got)[:upto] if got else np.zeros((0, DIM))


def _scales(c, name, s, h, upto):
    """fp32 scales of the first `upto` tokens of sequence s (FP8)."""
    index = {int(p): i for i, p in enumerate(c["perm"])}
    got = [c["rows_" + name + "_scale"][index[int(c["table"][s, b])], h].numpy() for b in range(-(-upto // BLOCK))]
    return np.concatenate(got)[:upto].astype(np.float64)


def plain_dense(c, skip_blocks=()):
    """(out, lse, |v| average, logit error bound, keys, bound for weights below f16's normal range) of
    every row, in 64 bits.

    The error bound of a logit: q.k is summed in fp32 (128 products in tensor-core
    order: at most 136 roundings of partial sums below sum |q k|), a bf16 query
    meeting e4m3 keys is held in f16 after a scale that brings its row's largest
    element to 2^13 or more (exact above 2^-14, off by 2^-25 at most below: 2^-38 of the largest), and
    the scaled logit takes three more roundings in the log2 domain."""
    q = c["q"].cpu()
    q = q.view(torch.int16).numpy().view(np.uint16) if c["qd"] == "bf16" else q.numpy()
    q = O.query_values(q, c["qd"], c["q_scale"]).astype(np.float64)
    Q, Hq, H = c["Q"], c["Hq"], c["H"]
    R, r = len(c["lens"]) * Q, Hq // H
    out, lse = np.zeros((R, Hq, DIM)), np.full((R, Hq), -np.inf)
    size, ex, n, low = np.zeros((R, Hq, DIM)), np.zeros((R, Hq)), np.zeros((R, Hq)), np.zeros((R, Hq, DIM))
    scale = DIM ** -0.5
    for s, T in enumerate(c["lens"]):
        if T <= 0:
            continue
        for h in range(H):
            K, V = _host_rows(c, "k", s, h, T), _host_rows(c, "v", s, h, T)
            A = np.abs(V)
            if c["kv"] == "fp8":
                vs = _scales(c, "v", s, h, T)
                A = A * (vs.max() / vs * 2.0 ** 8)[:, None]
            for i in range(Q):
                see = np.arange(T) <= T - Q + i
                for b in skip_blocks:
                    see[b * BLOCK:(b + 1) * BLOCK] = False
                if not see.any():
                    continue
                for hh in range(h * r, (h + 1) * r):
                    row, x = s * Q + i, None
                    qv = q[row, hh]
                    x = K[see] @ qv * scale
                    mass = np.abs(K[see]) @ np.abs(qv) * scale
                    split = 2.0 ** -38 * np.abs(qv).max() * np.abs(K[see]).sum(1) * scale if c["kv"] == "fp8" and c["qd"] == "bf16" else 0.0
                    ex[row, hh] = (mass * 136 * 2.0 ** -24 + split + np.abs(x) * 3 * 2.0 ** -23).max()
                    m = x.max()
                    p = np.exp(x - m)
                    lse[row, hh] = m + np.log(p.sum())
                    out[row, hh] = p @ V[see] / p.sum()
                    size[row, hh] = p @ np.abs(V[see]) / p.sum()
                    n[row, hh] = see.sum()
                    low[row, hh] = 0 if c["kv"] == "bf16" else 2.0 ** -32 * A[see].sum(0)
    return out, lse, size, ex, n, low


def check_dense(c, out, lse, ref, rows=None):
    """Against plain_dense.  out: half a step of bf16; before it every weight is off by the logit's
    error twice (itself and the sum's), ex2's 2^-22 and its own rounding (2^-11 as f16, 2^-16 as two bf16
    terms), and the sums over n keys in fp32 by at most n / 8 roundings of a lane's run of them.
    As f16 a weight is kept as 2^7 w where the row's reference has w = 1 (its sum is 1 or more), so
    below 2^-14 it is off by half of 2^-24: 2^-32 |v| a key.  FP8 keeps 2^7 w times the key's scale over
    one that is at most 2^8 the largest: that much more, over the key's own scale."""
    o, l, size, ex, n, low = ref
    rows = slice(None) if rows is None else rows
    got, gl = out.float().cpu().numpy().astype(np.float64)[rows], lse.cpu().numpy().astype(np.float64)[rows]
    o, l, size, ex, n, low = o[rows], l[rows], size[rows], ex[rows], n[rows], low[rows]
    sums = (n / 8 + 64) * 2.0 ** -24
    weight = (2.0 ** -16 if c["kv"] == "bf16" else 2.0 ** -11) + 2 * ex + 2.0 ** -21 + 2 * sums
    tol = HALF["bf16"] * np.abs(o) + (1 + HALF["bf16"]) * size * weight[..., None] + (1 + HALF["bf16"]) * low + 1e-37
    assert np.isfinite(got).all()
    err = np.abs(got - o)
    assert (err <= tol).all(), (np.argwhere(err > tol)[:4], (err / tol).max())
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    ltol = ex + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, l)) + 2.0 ** -22
    lerr = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, l))
    assert (lerr <= ltol).all(), (lerr / ltol).max()


# ---------------------------------------------------------------- rotary insert

def plain_rope(x, positions, rotary, theta, sections, layout, w=None, eps=1e-6, offset=0.0):
    """x [T][heads][128] in 64 bits, normed (w given) and turned."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + np.asarray(w, np.float64))
    if positions is None:
        return x
    y = x.copy()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(rotary // 2):
        ang = np.asarray(positions[axis[i]], np.float64) * theta ** (-2.0 * i / rotary)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        u, v = (2 * i, 2 * i + 1) if layout == "adjacent" else (i, i + rotary // 2)
        y[..., u] = x[..., u] * c - x[..., v] * s
        y[..., v] = x[..., u] * s + x[..., v] * c
    return y


# ---------------------------------------------------------------- block tables

def plain_tables(num_blocks, cached, new, table, free, count, max_tokens):
    """The documented rules, one request after the other; returns the outputs and whether anything was refused."""
    S, max_nb = table.shape
    table, free = table.copy(), free.copy()
    cap = len(free)
    stack = list(free[:count])
    fault = False
    good = [c >= 0 and n >= -1 and c + max(n, 0) <= max_nb * BLOCK for c, n in zip(cached, new)]
    for s in range(S):
        if good[s] and new[s] == -1:
            stack += list(table[s, :-(-cached[s] // BLOCK)])
    fault |= len(stack) > cap or not all(good)
    stack = stack[:cap]
    total = len(stack)
    slots, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int64)
    lens, offsets = np.zeros(S, np.int64), np.zeros(S + 1, np.int64)
    wanted = tokens = taken = 0
    for s in range(S):
        add = max(new[s], 0) if good[s] else 0
        need = -(-(cached[s] + add) // BLOCK) - -(-cached[s] // BLOCK) if good[s] and add else 0
        offsets[s] = tokens
        lens[s] = cached[s] if good[s] and new[s] >= 0 else 0
        wanted, tokens = wanted + need, tokens + add
        ok = wanted <= total and tokens <= max_tokens
        for i in range(add):
            if offsets[s] + i < max_tokens:
                pos[offsets[s] + i] = cached[s] + i
        if not ok:
            fault |= add > 0
            continue
        lens[s] += add
        had = -(-cached[s] // BLOCK) if good[s] else 0
        for b in range(need):
            blk = stack[total - 1 - taken]
            taken += 1
            inside = 0 <= blk < num_blocks
            fault |= not inside
            table[s, had + b] = blk if inside else -1
        for i in range(add):
            p = cached[s] + i
            blk = table[s, p // BLOCK]
            if 0 <= blk < num_blocks:
                slots[offsets[s] + i] = blk * BLOCK + p % BLOCK
            else:
                fault = True
    offsets[S] = tokens
    left = total - taken
    free[:left] = stack[:left]
    return dict(table=table, free=free, seq_lens=lens, offsets=offsets, slots=slots, positions=pos, free_count=left), fault
