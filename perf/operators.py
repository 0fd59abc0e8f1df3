"""The serving operators around the sparse path, as they are measured: block
tables from request lengths, rotary positions with the cache insert, and the
dense attend over the paged cache.

Where ``own`` is false, ``run`` computes an operator in elementary torch
operations in 32 bits (angles in 64); where it is true it makes the library's calls."""

import math

import torch

own = False

BLOCK = 128
DIM = 128
THETA = 5.0e6
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one request of 4K tokens: the latency of a single decode step
        _attend("attend one bf16", "bf16", "bf16", 1, 4096, 4096),
        # a decode batch, contexts of 16K to 32K
        _attend("attend batch fp8", "fp8", "bf16", 32, 16384, 32768),
        # speculative verify: 8 new tokens on 128K
        _attend("attend verify nvfp4", "nvfp4", "fp8", 8, 131072, 131072, q_tokens=8),
        # four requests of 512K: the cache is far larger than any on-chip memory
        _attend("attend long fp8", "fp8", "bf16", 4, 524288, 524288),
        # short, ragged requests with padding rows, 16 heads a group, 3 new tokens
        _attend("attend ragged bf16", "bf16", "bf16", 61, 1, 9001, q_tokens=3, heads=32, kv_heads=2, empty=3),
        # a decode step's 32 tokens: latency
        _rope("rope step fp8", "fp8", 32, axes=1),
        # a prompt chunk of 8,192 tokens
        _rope("rope prompt fp8", "fp8", 8192, axes=1),
        # images: three axes, a partial rotation, e4m3 queries out
        _rope("rope images nvfp4", "nvfp4", 24571, axes=3, rotary=64, q_fp8=True),
        # an odd count with padding tokens, adjacent pairs, no norm
        _rope("rope odd bf16", "bf16", 1001, axes=3, norm=False, adjacent=True, padding=13),
        # a decode step of 32 requests, one token each
        _tables("tables step", 32, 1, 1, 30000, 0),
        # 253 prompts of ragged lengths while every seventh request ends
        _tables("tables prompts", 253, 1, 600, 3000, 7),
    ]


def _attend(name, kv, qd, seqs, lo, hi, q_tokens=1, heads=16, kv_heads=4, empty=0):
    return {"name": name, "op": "attend", "kv": kv, "qd": qd, "seqs": seqs, "lo": lo, "hi": hi, "q_tokens": q_tokens,
            "heads": heads, "kv_heads": kv_heads, "empty": empty}


def _rope(name, kv, tokens, axes=1, rotary=128, q_fp8=False, norm=True, adjacent=False, padding=0, heads=16, kv_heads=4):
    return {"name": name, "op": "rope", "kv": kv, "tokens": tokens, "axes": axes, "rotary": rotary, "q_fp8": q_fp8,
            "norm": norm, "adjacent": adjacent, "padding": padding, "heads": heads, "kv_heads": kv_heads}


def _tables(name, seqs, lo, hi, cached, ends):
    return {"name": name, "op": "tables", "seqs": seqs, "lo": lo, "hi": hi, "cached": cached, "ends": ends}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "rope", "tables"))
    if op == "attend":
        kv = rng.choice(("bf16", "fp8", "nvfp4"))
        kv_heads = rng.choice((1, 2, 4, 8))
        seqs = _log(rng, 1, 96)
        hi = _log(rng, 1, min(262144, 1500000 // (seqs * kv_heads)))
        lo = rng.randint(1, hi)
        c = _attend("", kv, "bf16" if kv == "bf16" else rng.choice(("bf16", "fp8")), seqs, lo, hi,
                    q_tokens=rng.choice((1, 1, 1, 2, 4, 5, 8)), heads=kv_heads * rng.choice((1, 2, 3, 4, 6, 8, 16)),
                    kv_heads=kv_heads, empty=rng.choice((0, 0, 1)) if seqs > 1 else 0)
    elif op == "rope":
        axes = rng.choice((1, 2, 3))
        c = _rope("", rng.choice(("bf16", "fp8", "nvfp4")), _log(rng, 1, 20000), axes=axes, rotary=rng.choice((32, 64, 96, 128)),
                  q_fp8=rng.random() < 0.3, norm=rng.random() < 0.7, adjacent=rng.random() < 0.3, padding=0,
                  kv_heads=rng.choice((1, 2, 4, 8)))
        c["heads"] = c["kv_heads"] * rng.choice((1, 2, 4, 5))
        c["padding"] = rng.randint(0, c["tokens"] // 4)
    else:
        seqs = _log(rng, 1, 500)
        hi = _log(rng, 1, 60000 // seqs)
        c = _tables("", seqs, rng.randint(0, hi), hi, _log(rng, 100, 30000), rng.choice((0, 0, 3, 11)))
    del c["name"]
    return c


# ------------------------------------------------------------------ what a case holds

def _lens(c):
    """The sequence lengths of an attend case: spread evenly over lo .. hi, the first `empty` of them 0."""
    n, span = c["seqs"], c["hi"] - c["lo"]
    lens = [c["lo"] + int(span * ((i * 0.6180339887498949) % 1.0) + 0.5) for i in range(n)]
    lens[-1] = c["hi"]
    return [0] * min(c["empty"], n - 1) + lens[min(c["empty"], n - 1):]


def _row_bytes(kv):
    return {"bf16": 256, "fp8": 132, "nvfp4": 72}[kv]


def work(c):
    if c["op"] == "attend":
        lens = _lens(c)
        rows = c["seqs"] * c["q_tokens"] * c["heads"]
        q = DIM if c["qd"] == "fp8" else 2 * DIM
        keys = sum(max(0, t - c["q_tokens"] + i + 1) for t in lens for i in range(c["q_tokens"]))
        return {"bytes": sum(lens) * c["kv_heads"] * 2 * _row_bytes(c["kv"]) + rows * (q + 2 * DIM + 4)
                + 4 * sum(-(-t // BLOCK) for t in lens), "flops": 4 * DIM * c["heads"] * keys}
    if c["op"] == "rope":
        h, g, live = c["heads"], c["kv_heads"], c["tokens"] - c["padding"]
        rows = h + 3 * g + 1  # q, k, v, index q, index k
        out = (h + g) * (DIM if c["q_fp8"] else 2 * DIM)
        rotated = h + 2 * g + 1
        return {"bytes": c["tokens"] * (rows * 2 * DIM + out + 4 * c["axes"] + 4) + live * (2 * g + 1) * _row_bytes(c["kv"]),
                "flops": c["tokens"] * rotated * (3 * c["rotary"] + (4 * DIM if c["norm"] else 0))}
    cached, new = _requests(c)
    tokens = sum(max(0, n) for n in new)
    return {"bytes": 8 * c["seqs"] + 4 * c["seqs"] + 8 * tokens + 4 * c["seqs"]
            + 8 * sum(_blocks(a + n) - _blocks(a) for a, n in zip(cached, new) if n > 0)
            + 8 * sum(_blocks(a) for a, n in zip(cached, new) if n < 0), "flops": 0}


def _blocks(t):
    return -(-t // BLOCK)


def _requests(c):
    """Tokens cached and tokens new of each request; -1 new: the request has ended and gives its blocks back."""
    cached, new = [], []
    for i in range(c["seqs"]):
        a, b = (i * 0.6180339887498949) % 1.0, (i * 0.7548776662466927 + 0.3) % 1.0
        cached.append(int(a * c["cached"]))
        new.append(c["lo"] + int((c["hi"] - c["lo"]) * b + 0.5))
        if c["ends"] and i % c["ends"] == c["ends"] - 1:
            new[-1] = -1
    return cached, new


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _fp8_rows(x):
    amax = x.abs().amax(dim=-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale.squeeze(-1).contiguous()


def _e2m1_codes(v):
    """The nearest e2m1 code, ties to the even one, +0 for what rounds to zero."""
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75).to(torch.uint8) + (m > 1.25).to(torch.uint8) + (m >= 1.75).to(torch.uint8)
            + (m > 2.5).to(torch.uint8) + (m >= 3.5).to(torch.uint8) + (m > 5.0).to(torch.uint8))
    return code | (((v < 0) & (code > 0)).to(torch.uint8) << 3)


def _nvfp4_rows(x, g):
    """Packed codes, e4m3 scale codes of 16 elements each, for the per-tensor scale g (an fp32 value)."""
    y = x.unflatten(-1, (-1, 16))
    sf = (y.abs().amax(dim=-1) / torch.tensor(6.0 * g, dtype=torch.float32, device=x.device)).clamp(0, 448.0).to(torch.float8_e4m3fn)
    den = (sf.float() * torch.tensor(g, dtype=torch.float32, device=x.device)).unsqueeze(-1)
    codes = _e2m1_codes(torch.where(den > 0, y / den, torch.zeros_like(y))).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sf.view(torch.uint8)


def _e2m1_pairs():
    """For each byte of two e2m1 codes the two values they stand for, in a type of 8 bits that holds them all."""
    e = torch.tensor(E2M1, dtype=torch.float32, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8).to(torch.int32)
    return (e.unsqueeze(0) | (e.unsqueeze(1) << 8)).flatten().to(torch.int16)


def prepare(case, seed):
    return {"attend": _prepare_attend, "rope": _prepare_rope, "tables": _prepare_tables}[case["op"]](case, seed)


def run(st):
    return {"attend": _run_attend, "rope": _run_rope, "tables": _run_tables}[st["op"]](st)


def exact(case, seed):
    """In 64 bits, from the definitions."""
    return {"attend": _exact_attend, "rope": _exact_rope, "tables": _exact_tables}[case["op"]](case, seed)


# ------------------------------------------------------------------ the dense attend

def _prepare_attend(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lens(c)
    nbs = torch.tensor([_blocks(t) for t in lens], device="cuda")
    max_nb, pool = int(max(1, max(_blocks(t) for t in lens))), sum(_blocks(t) for t in lens) + 3
    order = torch.randperm(pool, generator=gen, device="cuda")
    b = torch.arange(max_nb, device="cuda")
    at = (torch.cumsum(nbs, 0) - nbs).unsqueeze(1) + b
    held = b < nbs.unsqueeze(1)
    table = torch.where(held, order[at.clamp(max=pool - 1)], torch.full_like(at, -1)).to(torch.int32)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st = {"op": "attend", "kv": c["kv"], "qd": c["qd"], "q_tokens": c["q_tokens"], "heads": c["heads"],
          "kv_heads": c["kv_heads"], "pool": pool, "table": table, "seq_lens": seq_lens}
    # which rows of the pool hold a token: the others are whatever the memory held, NaN among it
    used = torch.zeros((pool, BLOCK), dtype=torch.bool, device="cuda")
    t = b.unsqueeze(1) * BLOCK + torch.arange(BLOCK, device="cuda")
    live = t.unsqueeze(0) < seq_lens.view(-1, 1, 1)
    used[table.clamp(min=0).long()[held]] = live[held]
    for name, spread in (("k", 0.25), ("v", 0.5)):
        x = _randn(gen, pool, c["kv_heads"], BLOCK, DIM)
        x *= torch.exp(spread * _randn(gen, pool, c["kv_heads"], BLOCK, 1))  # rows are of different sizes
        if c["kv"] == "bf16":
            st[name] = x.to(torch.bfloat16).masked_fill_(~used.view(pool, 1, BLOCK, 1), float("nan"))
        elif c["kv"] == "fp8":
            st[name], s = _fp8_rows(x)
            st[name + "_scale"] = s.masked_fill_(~used.unsqueeze(1), float("nan"))
        else:
            st[name + "_global"] = float(torch.tensor(2.0 ** -8 if name == "k" else 2.0 ** -7))
            st[name], sf = _nvfp4_rows(x, st[name + "_global"])
            st[name + "_sf"] = sf.masked_fill_(~used.view(pool, 1, BLOCK, 1), 0x7F)
        del x
    q = _randn(gen, c["seqs"] * c["q_tokens"], c["heads"], DIM)
    if c["qd"] == "fp8":
        st["q_scale"] = 2.0 ** -6
        st["q"] = (q / st["q_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        st["q_scale"], st["q"] = 1.0, q.to(torch.bfloat16)
    if own:
        import block_sparse_attention_03_gb300 as msa
        st["cache"] = msa.PagedCache(kv_dtype=c["kv"], index_dtype=c["kv"], num_blocks=pool, num_kv_heads=c["kv_heads"],
                                     k=st["k"], v=st["v"], idx=None, k_sf=st.get("k_sf"), v_sf=st.get("v_sf"),
                                     k_scale=st.get("k_scale"), v_scale=st.get("v_scale"),
                                     k_global=st.get("k_global", 0.0), v_global=st.get("v_global", 0.0))
        st["batch"] = msa.Batch(seq_lens, table, c["q_tokens"])
        st["cfg"] = msa.default_config()
        st["query"] = msa.Query(st["q"], c["qd"], st["q_scale"])
        st["out"] = torch.empty((c["seqs"] * c["q_tokens"], c["heads"], DIM), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((c["seqs"] * c["q_tokens"], c["heads"]), dtype=torch.float32, device="cuda")
        st["ws"] = torch.empty(msa.msa_dense_workspace_size(st["cache"], st["batch"], c["heads"]), dtype=torch.uint8, device="cuda")
        msa.msa_workspace_init(st["ws"])
    return st


def _values(st, name, table):
    """K or V of the blocks of `table`, in 32 bits: [S][H][tokens][128]."""
    x = st[name][table]
    if st["kv"] == "bf16":
        x = x.float()
    elif st["kv"] == "fp8":
        x = x.view(torch.float8_e4m3fn).float() * st[name + "_scale"][table].unsqueeze(-1)
    else:
        lut = torch.tensor(E2M1, dtype=torch.float32, device="cuda")
        x = torch.stack((lut[(x & 15).int()], lut[(x >> 4).int()]), dim=-1).flatten(-2)
        sf = st[name + "_sf"][table].view(torch.float8_e4m3fn).float()
        x = (x.unflatten(-1, (8, 16)) * sf.unsqueeze(-1)).flatten(-2) * st[name + "_global"]
    return x.transpose(1, 2).flatten(2, 3)


def _run_attend(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_dense_attend(st["cache"], st["batch"], st["cfg"], st["query"], st["heads"], st["out"], st["lse"], st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    lens, table, n, H = st["seq_lens"], st["table"], st["q_tokens"], st["kv_heads"]
    S, r = lens.shape[0], st["heads"] // H
    table = table.clamp(min=0).long()
    q = st["q"].view(torch.float8_e4m3fn).float() * st["q_scale"] if st["qd"] == "fp8" else st["q"].float()
    q = q.view(S, n, H, r, DIM).permute(0, 2, 1, 3, 4).reshape(S, H, n * r, DIM)
    t = torch.arange(table.shape[1] * BLOCK, device="cuda")
    last = lens.view(S, 1) - n + torch.arange(n, device="cuda")  # the last key that each new token sees
    sees = (t <= last.unsqueeze(-1)).view(S, 1, n, 1, -1)
    x = torch.matmul(q, _values(st, "k", table).transpose(-1, -2)) * (DIM ** -0.5)
    x = torch.where(sees, x.view(S, H, n, r, -1), torch.full((), -math.inf, device="cuda"))
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    total = p.sum(dim=-1, keepdim=True)
    v = torch.where((t < lens.view(S, 1)).view(S, 1, -1, 1), _values(st, "v", table), torch.zeros((), device="cuda"))
    o = torch.matmul(p.view(S, H, n * r, -1), v).view(S, H, n, r, DIM)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(S * n, st["heads"], DIM).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(S * n, st["heads"])}


def _code_values(exp_bits, man_bits, bias):
    """Values of the sign / exponent / mantissa codes of a small float format, in 64 bits."""
    got = []
    for code in range(1 << (1 + exp_bits + man_bits)):
        m, e = code & ((1 << man_bits) - 1), (code >> man_bits) & ((1 << exp_bits) - 1)
        v = math.ldexp(m, 1 - bias - man_bits) if e == 0 else math.ldexp((1 << man_bits) + m, e - bias - man_bits)
        got.append(-v if code >> (exp_bits + man_bits) else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _rows64(st, name, phys, h):
    raw = st[name][phys, h]
    if st["kv"] == "bf16":
        return raw.double().reshape(-1, DIM)
    if st["kv"] == "fp8":
        return (_code_values(4, 3, 7)[raw.int()] * st[name + "_scale"][phys, h].double().unsqueeze(-1)).reshape(-1, DIM)
    e2m1 = _code_values(2, 1, 1)
    both = torch.stack((e2m1[(raw & 15).int()], e2m1[(raw >> 4).int()]), -1).reshape(-1, 8, 16)
    sf = _code_values(4, 3, 7)[st[name + "_sf"][phys, h].int()].reshape(-1, 8, 1)
    return (both * sf * float(st[name + "_global"])).reshape(-1, DIM)


def _exact_attend(c, seed):
    st = _prepare_attend(c, seed)
    n, H, r = c["q_tokens"], c["kv_heads"], c["heads"] // c["kv_heads"]
    q = _code_values(4, 3, 7)[st["q"].int()] * st["q_scale"] if c["qd"] == "fp8" else st["q"].double()
    out = torch.zeros((c["seqs"] * n, c["heads"], DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"] * n, c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for s, T in enumerate(_lens(c)):
        if T == 0:
            continue
        phys = st["table"][s, :_blocks(T)].long()
        for h in range(H):
            keys, vals = (_rows64(st, name, phys, h)[:T] for name in ("k", "v"))
            for i in range(n):
                see = T - n + i + 1
                if see < 1:
                    continue
                x = keys[:see] @ q[s * n + i, h * r:(h + 1) * r].T / math.sqrt(DIM)
                z = torch.logsumexp(x, dim=0)
                lse[s * n + i, h * r:(h + 1) * r] = z
                out[s * n + i, h * r:(h + 1) * r] = torch.exp(x - z).T @ vals[:see]
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ rotary positions and the insert

def _sections(c):
    """How many frequency pairs each axis takes: the first a little more than the others, as for time, height, width."""
    pairs = c["rotary"] // 2
    rest = pairs // (c["axes"] + 1) if c["axes"] > 1 else 0
    return [pairs - rest * (c["axes"] - 1)] + [rest] * (c["axes"] - 1)


def _prepare_rope(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, Hq, H = c["tokens"], c["heads"], c["kv_heads"]
    live = T - c["padding"]
    pool = _blocks(T) + 1
    # the projection's output: one row a token with q, k, v, index q, index k side by side
    qkv = _randn(gen, T, Hq + 3 * H + 1, DIM)
    qkv = (qkv * torch.exp(0.5 * _randn(gen, T, Hq + 3 * H + 1, 1))).to(torch.bfloat16)
    q, k, v, iq, ik = qkv.split([Hq, H, H, H, 1], dim=1)
    base = torch.randint(0, 200000, (1,), generator=gen, device="cuda")
    t = torch.arange(T, device="cuda")
    # axis 0 counts on; the others run over the rows and columns of images 48 wide
    axes = [base + t, base + (t // 48) % 48, base + t % 48][:c["axes"]]
    # consecutive tokens sit in consecutive rows of a block, the blocks anywhere in the pool
    place = torch.randperm(pool, generator=gen, device="cuda")
    slots = place[t // BLOCK] * BLOCK + t % BLOCK
    slots = torch.where(t < live, slots, torch.full_like(slots, -1))
    st = {"op": "rope", "kv": c["kv"], "q_fp8": c["q_fp8"], "rotary": c["rotary"], "adjacent": c["adjacent"], "padding": c["padding"],
          "tokens": T, "heads": Hq, "kv_heads": H, "q": q, "k": k, "v": v, "index_q": iq, "index_k": ik.squeeze(1), "pool": pool,
          "sections": _sections(c), "positions": torch.stack(axes).to(torch.int32).contiguous(), "slots": slots.to(torch.int32),
          "q_scale": 2.0 ** -6}
    pair_axis = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
    st["pair_axis"] = torch.tensor(pair_axis, device="cuda")
    st["freq"] = THETA ** (-2.0 * torch.arange(c["rotary"] // 2, dtype=torch.float64, device="cuda") / c["rotary"])
    names = ("q", "k", "index_q", "index_k")
    st["norm"] = {n: (0.1 * _randn(gen, DIM)).to(torch.bfloat16) for n in names} if c["norm"] else None
    zeros = lambda *shape, dtype=torch.uint8: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    st["bufs"] = {}
    for name, h in (("k", (H,)), ("v", (H,)), ("idx", ())):
        if c["kv"] == "bf16":
            st["bufs"][name] = zeros(pool, *h, BLOCK, DIM, dtype=torch.bfloat16)
        elif c["kv"] == "fp8":
            st["bufs"][name] = zeros(pool, *h, BLOCK, DIM)
            st["bufs"][name + "_scale"] = zeros(pool, *h, BLOCK, dtype=torch.float32)
        else:
            st["bufs"][name] = zeros(pool, *h, BLOCK, DIM // 2)
            st["bufs"][name + "_sf"] = zeros(pool, *h, BLOCK, DIM // 16)
            st[name + "_global"] = 2.0 ** -8
    if c["kv"] == "nvfp4":
        st["pair"] = _e2m1_pairs()
    if own:
        import block_sparse_attention_03_gb300 as msa
        b = st["bufs"]
        st["cache"] = msa.PagedCache(kv_dtype=c["kv"], index_dtype=c["kv"], num_blocks=pool, num_kv_heads=H, k=b["k"], v=b["v"],
                                     idx=b["idx"], k_sf=b.get("k_sf"), v_sf=b.get("v_sf"), idx_sf=b.get("idx_sf"),
                                     k_scale=b.get("k_scale"), v_scale=b.get("v_scale"), idx_scale=b.get("idx_scale"),
                                     k_global=st.get("k_global", 0.0), v_global=st.get("v_global", 0.0),
                                     idx_global=st.get("idx_global", 0.0))
        st["rope"] = msa.msa_rope_init(c["rotary"], THETA, st["sections"], "adjacent" if c["adjacent"] else "halves")
        st["weights"] = msa.QkNorm(eps=EPS, offset=1.0, **st["norm"]) if c["norm"] else None
        q_dtype = torch.uint8 if c["q_fp8"] else torch.bfloat16
        kind = "fp8" if c["q_fp8"] else "bf16"
        st["q_out"] = msa.Query(torch.empty((T, Hq, DIM), dtype=q_dtype, device="cuda"), kind, st["q_scale"])
        st["index_q_out"] = msa.Query(torch.empty((T, H, DIM), dtype=q_dtype, device="cuda"), kind, st["q_scale"])
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return st


def _seen(st, q, iq):
    """The rotated queries and the caches, codes as the values that they stand for."""
    e4m3 = lambda x: x.view(torch.float8_e4m3fn)  # noqa: E731
    got = {"q": e4m3(q) if st["q_fp8"] else q, "index_q": e4m3(iq) if st["q_fp8"] else iq}
    for name, x in st["bufs"].items():
        if x.dtype != torch.uint8:
            got[name] = x
        elif st["kv"] == "nvfp4" and not name.endswith("_sf"):
            got[name] = e4m3(st["pair"][x.int()].view(torch.uint8))
        else:
            got[name] = e4m3(x)
    return got


def _turned(st, x, name, c, s):
    x = x.float()
    if st["norm"] is not None:
        w = st["norm"][name].float() + 1.0
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w
    r, p = st["rotary"], st["rotary"] // 2
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if st["adjacent"] else (x[..., :p], x[..., p:r])
    a, b = a * c - b * s, a * s + b * c
    both = torch.stack((a, b), dim=-1).flatten(-2) if st["adjacent"] else torch.cat((a, b), dim=-1)
    return torch.cat((both, x[..., r:]), dim=-1)


def _put(st, name, x, blk, off):
    """Rows x, of shape [T][H][128] or [T][128], into the cache at (block, offset)."""
    at = (blk, slice(None), off) if x.dim() == 3 else (blk, off)
    b = st["bufs"]
    if st["kv"] == "bf16":
        b[name][at] = x.to(torch.bfloat16)
    elif st["kv"] == "fp8":
        b[name][at], b[name + "_scale"][at] = _fp8_rows(x)
    else:
        b[name][at], b[name + "_sf"][at] = _nvfp4_rows(x, st[name + "_global"])


def _run_rope(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_rope_insert(st["cache"], st["rope"], st["positions"], st["slots"], st["q"], st["q_out"], st["index_q"],
                            st["index_q_out"], st["k"], st["v"], st["index_k"], st["weights"], st["ws"])
        return _seen(st, st["q_out"].data, st["index_q_out"].data)
    angle = st["positions"][st["pair_axis"]].T.double() * st["freq"]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    ch, sh = c.unsqueeze(1), s.unsqueeze(1)
    q, iq = _turned(st, st["q"], "q", ch, sh), _turned(st, st["index_q"], "index_q", ch, sh)
    k, ik, v = _turned(st, st["k"], "k", ch, sh), _turned(st, st["index_k"], "index_k", c, s), st["v"].float()
    if st["q_fp8"]:
        q, iq = ((x / st["q_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn) for x in (q, iq))
    else:
        q, iq = q.to(torch.bfloat16), iq.to(torch.bfloat16)
    slots = st["slots"].long()
    if st["padding"]:
        keep = slots >= 0
        slots, k, v, ik = slots[keep], k[keep], v[keep], ik[keep]
    blk, off = slots // BLOCK, slots % BLOCK
    _put(st, "k", k, blk, off)
    _put(st, "v", v, blk, off)
    _put(st, "idx", ik, blk, off)
    return _seen(st, q, iq)


def _exact_rope(c, seed):
    st = _prepare_rope(c, seed)
    T, p, r = c["tokens"], c["rotary"] // 2, c["rotary"]
    axis = [a for a, n in enumerate(_sections(c)) for _ in range(n)]
    turned = {}
    for name in ("q", "index_q", "k", "index_k", "v"):
        x = st[name].double()
        x = x.clone() if x.dim() == 3 else x.unsqueeze(1).clone()
        if name != "v":
            if c["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DIM + EPS) * (1 + st["norm"][name].double())
            y = x.clone()
            for i in range(p):
                angle = st["positions"][axis[i]].double() * (THETA ** (-2.0 * i / r))
                cos, sin = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
                u, w = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + p)
                y[..., u] = x[..., u] * cos - x[..., w] * sin
                y[..., w] = x[..., u] * sin + x[..., w] * cos
            x = y
        turned[name] = x
    scale = st["q_scale"] if c["q_fp8"] else 1.0
    got = {"q": turned["q"] / scale, "index_q": turned["index_q"] / scale}
    live = T - c["padding"]
    where = st["slots"][:live].long()
    for name, src in (("k", "k"), ("v", "v"), ("idx", "index_k")):
        x = turned[src][:live]
        buf = st["bufs"][name]
        rows = lambda width: torch.zeros((st["pool"], x.shape[1], BLOCK, width), dtype=torch.float64, device="cuda")  # noqa: E731
        fit = lambda full, width: full.reshape(tuple(buf.shape[:-1]) + (width,))  # noqa: E731
        full = rows(DIM)
        if c["kv"] == "fp8":
            amax = x.abs().amax(-1, keepdim=True)
            scales = rows(1)
            sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
            scales[where // BLOCK, :, where % BLOCK] = sc
            got[name + "_scale"] = fit(scales, 1).squeeze(-1)
            x = x / sc
        elif c["kv"] == "nvfp4":
            g = st[name + "_global"]
            sf = (x.reshape(live, -1, 8, 16).abs().amax(-1) / (6 * g)).clamp(max=448)
            scales = rows(8)
            scales[where // BLOCK, :, where % BLOCK] = sf
            got[name + "_sf"] = fit(scales, 8)
            got[name] = None  # a 4-bit code is a choice of one of eight sizes: its scale above is what is computed
            continue
        full[where // BLOCK, :, where % BLOCK] = x
        got[name] = fit(full, DIM)
    return got


# ------------------------------------------------------------------ block tables from request lengths

def _prepare_tables(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cached, new = _requests(c)
    S, tokens = c["seqs"], sum(max(0, n) for n in new)
    most = max(_blocks(a + max(0, n)) for a, n in zip(cached, new)) + 2
    held, wants = sum(_blocks(a) for a in cached), sum(_blocks(a + max(0, n)) for a, n in zip(cached, new))
    pool = max(held, wants) + 50
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    nbs = torch.tensor([_blocks(a) for a in cached], device="cuda")
    b = torch.arange(most, device="cuda")
    at = (torch.cumsum(nbs, 0) - nbs).unsqueeze(1) + b
    table = torch.where(b < nbs.unsqueeze(1), order[at.clamp(max=pool - 1)], torch.full_like(order[:1], -1))
    free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")  # a stack: the last of them is taken first
    free[:pool - held] = order[held:]
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    st = {"op": "tables", "pool": pool, "cached": ints(*cached), "new": ints(*new), "table": table.contiguous(), "free": free,
          "free_count": ints(pool - held), "max_tokens": tokens + 5 if tokens > 8 * S else max(S, tokens)}
    if own:
        st["out"] = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (S, S + 1, st["max_tokens"], st["max_tokens"], 1)]
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return st


def _run_tables(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        lens, offsets, slots, positions, count = st["out"]
        msa.msa_build_tables(st["pool"], st["cached"], st["new"], st["table"], st["free"], st["free_count"], lens, offsets, slots,
                             positions, count, st["ws"])
        return {"table": st["table"], "free": st["free"], "seq_lens": lens, "offsets": offsets, "slots": slots,
                "positions": positions, "free_count": count}
    cached, new, table, free = st["cached"].long(), st["new"].long(), st["table"], st["free"]
    S, most, cap = cached.shape[0], table.shape[1], free.shape[0]
    ends = new < 0
    add = new.clamp(min=0)
    had = (cached + BLOCK - 1) // BLOCK
    wants = torch.where(ends, torch.zeros_like(had), (cached + add + BLOCK - 1) // BLOCK - had)
    back = torch.where(ends, had, torch.zeros_like(had))
    upto, tok = torch.cumsum(wants, 0), torch.cumsum(add, 0)
    back_to = torch.cumsum(back, 0)
    count = st["free_count"].long()
    # the blocks given back, in the order of the requests, go on top of the stack
    i = torch.arange(cap, device="cuda")
    r = i - count
    owner = torch.searchsorted(back_to, r.clamp(min=0), right=True).clamp(max=S - 1)
    given = table[owner, (r - (back_to - back)[owner]).clamp(0, most - 1)]
    total = count + back_to[-1]
    stack = torch.where((r >= 0) & (i < total), given, free)
    # new blocks are taken from the top, request after request
    b = torch.arange(most, device="cuda").unsqueeze(0)
    nth = (upto - wants).unsqueeze(1) + b - had.unsqueeze(1)
    is_new = (b >= had.unsqueeze(1)) & (b < (had + wants).unsqueeze(1))
    table = torch.where(is_new, stack[(total - 1 - nth).clamp(0, cap - 1)], table)
    left = total - upto[-1]
    free = torch.where(i < left, stack, free)
    t = torch.arange(st["max_tokens"], device="cuda")
    s = torch.searchsorted(tok, t, right=True).clamp(max=S - 1)
    pos = cached[s] + t - (tok - add)[s]
    real = t < tok[-1]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slots = table[s, pos // BLOCK].long() * BLOCK + pos % BLOCK
    slots = torch.where(real, slots, torch.full_like(slots, -1))
    lens = torch.where(ends, torch.zeros_like(cached), cached + add)
    offsets = torch.cat((torch.zeros_like(tok[:1]), tok))
    return {"table": table, "free": free, "seq_lens": lens.int(), "offsets": offsets.int(), "slots": slots.int(),
            "positions": pos.int(), "free_count": left.int()}


def _exact_tables(c, seed):
    st = _prepare_tables(c, seed)
    cached, new = st["cached"].tolist(), st["new"].tolist()
    table, array = st["table"].tolist(), st["free"].tolist()
    stack = array[:int(st["free_count"])]
    for s, n in enumerate(new):
        if n < 0:
            stack += table[s][:_blocks(cached[s])]
    total = len(stack)
    slots, positions, offsets, lens = [], [], [0], []
    for s, n in enumerate(new):
        for b in range(_blocks(cached[s]), _blocks(cached[s] + max(0, n))):
            table[s][b] = stack.pop()
        for p in range(cached[s], cached[s] + max(0, n)):
            slots.append(table[s][p // BLOCK] * BLOCK + p % BLOCK)
            positions.append(p)
        offsets.append(len(slots))
        lens.append(cached[s] + n if n >= 0 else 0)
    array[:len(stack)] = stack
    pad = st["max_tokens"] - len(slots)
    ints = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    assert total - len(stack) == sum(_blocks(a + n) - _blocks(a) for a, n in zip(cached, new) if n > 0)
    return {"table": ints(table), "free": ints(array), "seq_lens": ints(lens), "offsets": ints(offsets),
            "slots": ints(slots + [-1] * pad), "positions": ints(positions + [0] * pad), "free_count": ints([len(stack)])}
