"""A cache in 8 bits with one scale for each block of 128 tokens and head, as it is measured:
writing new tokens into it, reading tokens back, and the dense and the sparse attend over it.

Where ``own`` is false, ``run`` computes an operator in elementary torch operations in
32 bits; where it is true it makes the library's calls."""

import math

import torch

own = False

BLOCK = 128
DIM = 128
LEAST = 2.0 ** -126  # the smallest scale
TOP = {"int8_block": 127.0, "fp8_block": 448.0}  # the largest code
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # a decode step: one new token for each of 32 requests somewhere in their blocks; latency
        _insert("insert step int8", "int8_block", 32, 1, 1, 30000),
        # a prompt chunk of 8,192 tokens that goes on in a block already begun
        _insert("insert prompt fp8", "fp8_block", 1, 8192, 8192, 57301),
        # 253 requests with 0 to 200 new tokens, every seventh of them ended, 8 heads
        _insert("insert ragged int8", "int8_block", 253, 0, 200, 4000, ends=7, kv_heads=8),
        # a shared prefix of 4K tokens for the layers that read rows
        _read("read one int8", "int8_block", 1, 4096, 4096, 0),
        # eight prefixes of 16K to 32K
        _read("read batch fp8", "fp8_block", 8, 16384, 32768, 0),
        # the ends of 61 ragged requests out of the older format with scales of 16 elements
        _read("read ragged nvfp4", "nvfp4", 61, 1, 900, 9001, kv_heads=2),
        # one request of 4K tokens: the latency of a single decode step
        _attend("attend one int8", "int8_block", "bf16", 1, 4096, 4096),
        # a decode batch, contexts of 16K to 32K
        _attend("attend batch fp8", "fp8_block", "bf16", 32, 16384, 32768),
        # speculative verify: 8 new tokens on 128K
        _attend("attend verify int8", "int8_block", "fp8", 8, 131072, 131072, q_tokens=8),
        # four requests of 512K: the cache is far larger than any on-chip memory
        _attend("attend long int8", "int8_block", "bf16", 4, 524288, 524288),
        # the sparse layers of the same decode batch, 16 blocks each
        _sparse("sparse batch int8", "int8_block", "bf16", 32, 16384, 32768),
        # and of the verify: every new token has blocks of its own
        _sparse("sparse verify fp8", "fp8_block", "fp8", 8, 131072, 131072, q_tokens=8),
    ]


def _insert(name, kv, seqs, lo, hi, cached, ends=0, kv_heads=4):
    return {"name": name, "op": "insert", "kv": kv, "seqs": seqs, "lo": lo, "hi": hi, "cached": cached, "ends": ends,
            "kv_heads": kv_heads}


def _read(name, kv, seqs, lo, hi, skip, kv_heads=4):
    return {"name": name, "op": "read", "kv": kv, "seqs": seqs, "lo": lo, "hi": hi, "cached": skip, "ends": 0, "kv_heads": kv_heads}


def _attend(name, kv, qd, seqs, lo, hi, q_tokens=1, heads=16, kv_heads=4, empty=0):
    return {"name": name, "op": "attend", "kv": kv, "qd": qd, "seqs": seqs, "lo": lo, "hi": hi, "q_tokens": q_tokens,
            "heads": heads, "kv_heads": kv_heads, "empty": empty}


def _sparse(name, kv, qd, seqs, lo, hi, q_tokens=1, heads=16, kv_heads=4, topk=16):
    return {"name": name, "op": "sparse", "kv": kv, "qd": qd, "seqs": seqs, "lo": lo, "hi": hi, "q_tokens": q_tokens,
            "heads": heads, "kv_heads": kv_heads, "topk": topk, "empty": 0}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("insert", "read", "attend", "sparse"))
    kv, kv_heads = rng.choice(("int8_block", "fp8_block")), rng.choice((1, 2, 4, 8))
    if op == "insert":
        seqs = _log(rng, 1, 300)
        hi = _log(rng, 1, 30000 // seqs)
        c = _insert("", kv, seqs, rng.randint(0, hi), hi, _log(rng, 1, 30000), ends=rng.choice((0, 0, 3, 11)), kv_heads=kv_heads)
    elif op == "read":
        kv = rng.choice((kv, kv, "bf16", "fp8", "nvfp4"))
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 1, 100000 // seqs)
        c = _read("", kv, seqs, rng.randint(0, hi), hi, _log(rng, 1, 5000), kv_heads=kv_heads)
    elif op == "attend":
        seqs = _log(rng, 1, 96)
        hi = _log(rng, 1, min(262144, 1500000 // (seqs * kv_heads)))
        c = _attend("", kv, rng.choice(("bf16", "fp8")), seqs, rng.randint(1, hi), hi, q_tokens=rng.choice((1, 1, 1, 2, 4, 5, 8)),
                    heads=kv_heads * rng.choice((1, 2, 3, 4, 6, 8, 16)), kv_heads=kv_heads,
                    empty=rng.choice((0, 0, 1)) if seqs > 1 else 0)
    else:
        q_tokens, topk = rng.choice((1, 1, 2, 4, 8)), rng.choice((4, 8, 16, 32))
        seqs = _log(rng, 1, 64 // q_tokens)
        hi = _log(rng, 130, min(100000, 1500000 // (seqs * kv_heads)))
        c = _sparse("", kv, rng.choice(("bf16", "fp8")), seqs, rng.randint(130, hi), hi, q_tokens=q_tokens,
                    heads=kv_heads * rng.choice((1, 2, 3, 4, 8, 16)), kv_heads=kv_heads, topk=topk)
    del c["name"]
    return c


# ------------------------------------------------------------------ what a case holds

def _blocks(t):
    return -(-t // BLOCK)


def _lens(c):
    """The sequence lengths of an attend case: spread evenly over lo .. hi, the first `empty` of them 0."""
    n, span = c["seqs"], c["hi"] - c["lo"]
    lens = [c["lo"] + int(span * ((i * 0.6180339887498949) % 1.0) + 0.5) for i in range(n)]
    lens[-1] = c["hi"]
    return [0] * min(c["empty"], n - 1) + lens[min(c["empty"], n - 1):]


def _spans(c):
    """First position and the one behind the last of each request's tokens in an insert or read case
    (behind the first: none; a request that has ended gives 0)."""
    first, end = [], []
    for i in range(c["seqs"]):
        a, b = (i * 0.6180339887498949 + 0.999) % 1.0, (i * 0.7548776662466927) % 1.0 if i else 1.0
        first.append(int(a * c["cached"]))
        end.append(first[-1] + c["lo"] + int((c["hi"] - c["lo"]) * b + 0.5))
        if c["ends"] and i % c["ends"] == c["ends"] - 1:
            end[-1] = 0
    return first, end


def _row_bytes(kv):
    return {"bf16": 256, "fp8": 132, "nvfp4": 72}.get(kv, 128)


def work(c):
    h = c["kv_heads"]
    if c["op"] in ("insert", "read"):
        first, end = _spans(c)
        live = [(a, b) for a, b in zip(first, end) if b > a]
        tokens, blocks = sum(b - a for a, b in live), sum(_blocks(b) - a // BLOCK for a, b in live)
        scales = 8 * h * blocks if c["kv"] in TOP else 0
        if c["op"] == "insert":
            scales += 8 * h * sum(a % BLOCK > 0 for a, _ in live)
        return {"bytes": tokens * 2 * h * (256 + _row_bytes(c["kv"])) + scales + 12 * c["seqs"] + 4 * blocks,
                "flops": tokens * 4 * h * DIM if c["op"] == "insert" else tokens * 2 * h * DIM}
    lens, n, q = _lens(c), c["q_tokens"], DIM if c["qd"] == "fp8" else 2 * DIM
    rows = c["seqs"] * n * c["heads"]
    side = rows * (q + 2 * DIM + 4)
    if c["op"] == "attend":
        keys = sum(max(0, t - n + i + 1) for t in lens for i in range(n))
        held = sum(lens)
        return {"bytes": h * (held * 2 * _row_bytes(c["kv"]) + 8 * sum(_blocks(t) for t in lens)) + side
                + 4 * sum(_blocks(t) for t in lens), "flops": 4 * DIM * c["heads"] * keys}
    blocks, picks = 0.0, 0
    for t in lens:  # blocks that any of the request's tokens selects, on average: its own, and the others by chance
        nb = _blocks(t)
        k = min(c["topk"], nb)
        blocks += 1 + (nb - 1) * (1 - (1 - (k - 1) / max(1, nb - 1)) ** n)
        picks += n * k
    return {"bytes": h * blocks * (2 * BLOCK * DIM + 8) + side + 4 * c["seqs"] * n * h * c["topk"],
            "flops": 4 * DIM * c["heads"] * picks * BLOCK}


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _e2m1_codes(v):
    """The nearest e2m1 code, ties to the even one, +0 for what rounds to zero."""
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75).to(torch.uint8) + (m > 1.25).to(torch.uint8) + (m >= 1.75).to(torch.uint8)
            + (m > 2.5).to(torch.uint8) + (m >= 3.5).to(torch.uint8) + (m > 5.0).to(torch.uint8))
    return code | (((v < 0) & (code > 0)).to(torch.uint8) << 3)


def _pool(gen, c, lens):
    """A pool of blocks in any order, a table of those that sequences of these lengths hold, and which rows hold a token."""
    nbs = torch.tensor([_blocks(t) for t in lens], device="cuda")
    max_nb, pool = max(1, max(_blocks(t) for t in lens)), sum(_blocks(t) for t in lens) + 3
    order = torch.randperm(pool, generator=gen, device="cuda")
    b = torch.arange(max_nb, device="cuda")
    at = (torch.cumsum(nbs, 0) - nbs).unsqueeze(1) + b
    held = b < nbs.unsqueeze(1)
    table = torch.where(held, order[at.clamp(max=pool - 1)], torch.full_like(at, -1)).to(torch.int32)
    used = torch.zeros((pool, BLOCK), dtype=torch.bool, device="cuda")
    t = b.unsqueeze(1) * BLOCK + torch.arange(BLOCK, device="cuda")
    live = t.unsqueeze(0) < torch.tensor(lens, device="cuda").view(-1, 1, 1)
    used[table.clamp(min=0).long()[held]] = live[held]
    return pool, table, used


def _fill(gen, c, pool, used, st):
    """K and V of the pool, rows of different sizes; rows without a token hold what the memory held, NaN among it."""
    kv, H = c["kv"], c["kv_heads"]
    hole = ~used.view(pool, 1, BLOCK, 1)
    for name, spread in (("k", 0.25), ("v", 0.5)):
        x = _randn(gen, pool, H, BLOCK, DIM)
        x *= torch.exp(spread * _randn(gen, pool, H, BLOCK, 1))
        if kv == "bf16":
            st[name] = x.to(torch.bfloat16).masked_fill_(hole, float("nan"))
        elif kv == "fp8":
            s = x.abs().amax(-1, keepdim=True) / 448.0
            st[name] = _e4m3(x / s)
            st[name + "_scale"] = s.squeeze(-1).masked_fill(~used.unsqueeze(1), float("nan")).contiguous()
        elif kv == "nvfp4":
            g = 2.0 ** -8 if name == "k" else 2.0 ** -7
            sf = (x.unflatten(-1, (8, 16)).abs().amax(-1) / (6.0 * g)).clamp(0, 448.0).to(torch.float8_e4m3fn)
            codes = _e2m1_codes((x.unflatten(-1, (8, 16)) / (sf.float() * g).clamp(min=1e-30).unsqueeze(-1)).flatten(-2))
            st[name], st[name + "_global"] = codes[..., 0::2] | (codes[..., 1::2] << 4), g
            st[name + "_sf"] = sf.view(torch.uint8).masked_fill(hole, 0x7F)
        else:
            x.masked_fill_(hole, 0.0)
            s = (x.abs().amax((-2, -1)) / TOP[kv]).clamp(min=LEAST)
            x /= s.view(pool, H, 1, 1)
            st[name] = x.round_().to(torch.int8).masked_fill_(hole, -127) if kv == "int8_block" else _e4m3(x).masked_fill_(hole, 0x7F)
            st[name + "_scale"] = s.masked_fill(~used.any(1).unsqueeze(1), float("nan"))
        del x


def _cache(st, c, pool):
    import block_sparse_attention_03_gb300 as msa
    return msa.PagedCache(kv_dtype=c["kv"], index_dtype="bf16", num_blocks=pool, num_kv_heads=c["kv_heads"], k=st["k"], v=st["v"],
                          idx=None, k_sf=st.get("k_sf"), v_sf=st.get("v_sf"), k_scale=st.get("k_scale"), v_scale=st.get("v_scale"),
                          k_global=st.get("k_global", 0.0), v_global=st.get("v_global", 0.0))


def _workspace(n):
    import block_sparse_attention_03_gb300 as msa
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    msa.msa_workspace_init(ws)
    return ws


def prepare(case, seed):
    return {"insert": _prepare_insert, "read": _prepare_read, "attend": _prepare_attend, "sparse": _prepare_attend}[case["op"]](case, seed)


def run(st):
    return {"insert": _run_insert, "read": _run_read, "attend": _run_attend, "sparse": _run_sparse}[st["op"]](st)


def exact(case, seed):
    """In 64 bits, from the definitions."""
    return {"insert": _exact_insert, "read": _exact_read, "attend": _exact_attend, "sparse": _exact_sparse}[case["op"]](case, seed)


# ------------------------------------------------------------------ spans of tokens: insert and read

def _prepare_span(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    first, end = _spans(c)
    lens = [max(a, b) for a, b in zip(first, end)]
    counts = [max(0, b - a) for a, b in zip(first, end)]
    pool, table, used = _pool(gen, c, lens)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets = [sum(counts[:i]) for i in range(len(counts) + 1)]
    st = {"op": c["op"], "kv": c["kv"], "kv_heads": c["kv_heads"], "table": table, "first": ints(first), "end": ints(end),
          "offsets": ints(offsets), "tokens": offsets[-1], "runs": sum(_blocks(b) - a // BLOCK for a, b in zip(first, end) if b > a)}
    return gen, st, pool, used, first


def _own_span(st, c, pool):
    import block_sparse_attention_03_gb300 as msa
    st["cache"] = _cache(st, c, pool)
    st["spans"] = msa.Spans(st["first"], st["end"], st["offsets"], st["table"])
    st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


def _prepare_insert(c, seed):
    gen, st, pool, used, first = _prepare_span(c, seed)
    H = c["kv_heads"]
    was = torch.zeros_like(used)  # the rows that hold a token before the call
    t = torch.arange(st["table"].shape[1] * BLOCK, device="cuda").view(1, -1, BLOCK)
    held = st["table"] >= 0
    was[st["table"].clamp(min=0).long()[held]] = (t < torch.tensor(first, device="cuda").view(-1, 1, 1))[held]
    _fill(gen, c, pool, was, st)
    for name in ("k", "v"):  # what a block held so far is now larger, now smaller than what comes
        st[name + "_scale"] *= torch.exp(0.3 * _randn(gen, pool, H) - 0.2)
    # the projection's output: one row a token with k and v heads side by side
    x = _randn(gen, max(1, st["tokens"]), 2 * H, DIM)
    x = (x * torch.exp(0.4 * _randn(gen, max(1, st["tokens"]), 2 * H, 1))).to(torch.bfloat16)[:st["tokens"]]
    st["k_new"], st["v_new"] = x.split([H, H], dim=1)
    st["top"] = torch.full((1,), TOP[c["kv"]], device="cuda")
    if own:
        _own_span(st, c, pool)
    return st


def _codes(st, x):
    return torch.round(x).clamp(-127, 127).to(torch.int8) if st["kv"] == "int8_block" else _e4m3(x)


def _seen(st):
    """The cache, E4M3 codes as the values that they stand for."""
    e4m3 = st["kv"] == "fp8_block"
    got = {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    got.update((n, st[n].view(torch.float8_e4m3fn) if e4m3 else st[n]) for n in ("k", "v"))
    return got


def _tokens(st):
    """For each row of the span's tokens: its block in the pool, its row there, its place among the blocks touched, and how
    many tokens its block held before."""
    offsets, n = st["offsets"].long(), st["tokens"]
    row = torch.arange(n, device="cuda")
    s = torch.searchsorted(offsets, row, right=True) - 1
    pos = st["first"].long()[s] + row - offsets[s]
    blk = pos // BLOCK
    phys = st["table"][s, blk].long()
    new = (pos % BLOCK == 0) | (row == offsets[s])
    return phys, pos % BLOCK, torch.cumsum(new, 0) - 1, (st["first"].long()[s] - blk * BLOCK).clamp(min=0)


def _run_insert(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_block_insert(st["cache"], st["spans"], st["k_new"], st["v_new"], st["ws"])
        return _seen(st)
    if st["tokens"] == 0:
        return _seen(st)
    phys, off, run_of, live = _tokens(st)
    n, H = st["runs"], st["kv_heads"]
    at = torch.zeros(n, dtype=torch.long, device="cuda").scatter_(0, run_of, phys)
    had = torch.zeros(n, dtype=torch.long, device="cuda").scatter_(0, run_of, live)
    for name in ("k", "v"):
        x, data, scale = st[name + "_new"].float(), st[name], st[name + "_scale"]
        amax = torch.zeros((n, H), device="cuda").index_reduce_(0, run_of, x.abs().amax(-1), "amax")
        need = (amax / st["top"]).clamp(min=LEAST)
        old = scale[at]
        m0, e0 = torch.frexp(old)
        m1, e1 = torch.frexp(need)
        k = (e1 - e0 + (m1 > m0)).clamp(min=0)  # the least with old x 2^k >= need
        k = torch.where((had > 0).unsqueeze(1), k, torch.zeros_like(k))
        pow2 = lambda e: ((e + 127) << 23).to(torch.int32).view(torch.float32)  # noqa: E731
        s = torch.where((had > 0).unsqueeze(1), old * pow2(k), need)
        held = data[at]
        was = held.float() if st["kv"] == "int8_block" else held.view(torch.float8_e4m3fn).float()
        moved = _codes(st, was * pow2(-k.clamp(max=126)).view(n, H, 1, 1))
        keep = (torch.arange(BLOCK, device="cuda") >= had.unsqueeze(1)).view(n, 1, BLOCK, 1) | (k == 0).view(n, H, 1, 1)
        data[at] = torch.where(keep, held, moved)
        scale[at] = s
        data[phys, :, off] = _codes(st, x / s[run_of].unsqueeze(-1))
    return _seen(st)


def _exact_insert(c, seed):
    st = _prepare_insert(c, seed)
    first, end = _spans(c)
    offsets, table = st["offsets"].tolist(), st["table"].tolist()
    small = c["kv"] == "fp8_block"
    got = {}
    for name in ("k", "v"):
        new, scale = st[name + "_new"].double(), st[name + "_scale"].double()
        # the codes of INT8 are choices among whole numbers: the scales are what is computed
        full = _code_values(4, 3, 7)[st[name].int()] if small else None
        for s, (a, b) in enumerate(zip(first, end)):
            for blk in range(a // BLOCK, _blocks(b) if b > a else 0):
                p0, p1, at = max(a, blk * BLOCK), min(b, (blk + 1) * BLOCK), table[s][blk]
                x = new[offsets[s] + p0 - a:offsets[s] + p1 - a]
                need = (x.abs().amax((0, 2)) / TOP[c["kv"]]).clamp(min=LEAST)
                had = max(0, a - blk * BLOCK)
                grow = torch.ones_like(need)
                if had:
                    grow = 2.0 ** torch.ceil(torch.log2(need / scale[at])).clamp(min=0)
                    need = scale[at] * grow
                scale[at] = need
                if small:
                    full[at, :, :had] /= grow.view(-1, 1, 1)
                    full[at, :, p0 - blk * BLOCK:p1 - blk * BLOCK] = (x / need.view(1, -1, 1)).transpose(0, 1)
        got[name], got[name + "_scale"] = full, scale
    return got


def _prepare_read(c, seed):
    gen, st, pool, used, _ = _prepare_span(c, seed)
    _fill(gen, c, pool, used, st)
    if own:
        _own_span(st, c, pool)
        st["out"] = [torch.empty((st["tokens"], c["kv_heads"], DIM), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    return st


def _values(st, name, at, row=None):
    """K or V in 32 bits: of the blocks `at` [..][H][128][128], or of their rows `row` [..][H][128]."""
    of = lambda x: x[at] if row is None else x[at, :, row]  # noqa: E731
    x = of(st[name])
    if st["kv"] == "bf16":
        return x.float()
    if st["kv"] == "fp8":
        return x.view(torch.float8_e4m3fn).float() * of(st[name + "_scale"]).unsqueeze(-1)
    if st["kv"] == "nvfp4":
        lut = torch.tensor(E2M1, dtype=torch.float32, device="cuda")
        x = torch.stack((lut[(x & 15).int()], lut[(x >> 4).int()]), dim=-1).flatten(-2)
        sf = of(st[name + "_sf"]).view(torch.float8_e4m3fn).float()
        return (x.unflatten(-1, (8, 16)) * sf.unsqueeze(-1)).flatten(-2) * st[name + "_global"]
    scale = st[name + "_scale"][at].unsqueeze(-1)
    return (x.float() if st["kv"] == "int8_block" else x.view(torch.float8_e4m3fn).float()) * (scale.unsqueeze(-1) if row is None else scale)


def _run_read(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_cache_read(st["cache"], st["spans"], st["out"][0], st["out"][1], st["ws"])
        return {"k": st["out"][0], "v": st["out"][1]}
    phys, off, _, _ = _tokens(st)
    return {"k": _values(st, "k", phys, off).to(torch.bfloat16), "v": _values(st, "v", phys, off).to(torch.bfloat16)}


def _exact_read(c, seed):
    st = _prepare_read(c, seed)
    first, end = _spans(c)
    table, offsets = st["table"].tolist(), st["offsets"].tolist()
    got = {name: torch.zeros((st["tokens"], c["kv_heads"], DIM), dtype=torch.float64, device="cuda") for name in ("k", "v")}
    for s, (a, b) in enumerate(zip(first, end)):
        for blk in range(a // BLOCK, _blocks(b) if b > a else 0):
            p0, p1 = max(a, blk * BLOCK), min(b, (blk + 1) * BLOCK)
            to = offsets[s] - a
            for name in ("k", "v"):
                for h in range(c["kv_heads"]):
                    rows = _rows64(st, name, table[s][blk], h)
                    got[name][to + p0:to + p1, h] = rows[p0 - blk * BLOCK:p1 - blk * BLOCK]
    return got


# ------------------------------------------------------------------ the attends

def _prepare_attend(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens, n = _lens(c), c["q_tokens"]
    pool, table, used = _pool(gen, c, lens)
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st = {"op": c["op"], "kv": c["kv"], "qd": c["qd"], "q_tokens": n, "heads": c["heads"], "kv_heads": c["kv_heads"],
          "table": table, "seq_lens": seq_lens}
    _fill(gen, c, pool, used, st)
    rows = c["seqs"] * n
    q = _randn(gen, rows, c["heads"], DIM)
    if c["qd"] == "fp8":
        st["q_scale"] = 2.0 ** -6
        st["q"] = _e4m3(q / st["q_scale"])
    else:
        st["q_scale"], st["q"] = 1.0, q.to(torch.bfloat16)
    if c["op"] == "sparse":
        # a selection: each token's own block and others that it sees, ascending, -1 where there are no more
        last = (seq_lens.long().view(-1, 1) - n + torch.arange(n, device="cuda")).view(rows, 1, 1) // BLOCK
        b = torch.arange(max(table.shape[1], c["topk"]), device="cuda")
        score = torch.rand((rows, c["kv_heads"], b.shape[0]), generator=gen, device="cuda")
        score = torch.where(b < last, score, torch.where(b == last, torch.full_like(score, 2.0), torch.full_like(score, -1.0)))
        best, idx = score.topk(c["topk"], dim=-1)
        idx = torch.where(best >= 0, idx, torch.full_like(idx, 1 << 30)).sort(dim=-1).values
        st["topk"] = torch.where(idx < (1 << 30), idx, torch.full_like(idx, -1)).to(torch.int32).contiguous()
    if own:
        import block_sparse_attention_03_gb300 as msa
        st["cache"] = _cache(st, c, pool)
        st["batch"] = msa.Batch(seq_lens, table, n)
        st["cfg"] = msa.default_config(c.get("topk", 16))
        st["query"] = msa.Query(st["q"], c["qd"], st["q_scale"])
        st["out"] = torch.empty((rows, c["heads"], DIM), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty((rows, c["heads"]), dtype=torch.float32, device="cuda")
        st["ws"] = _workspace(msa.msa_workspace_size(st["cache"], st["batch"], st["cfg"], c["heads"]) if c["op"] == "sparse"
                              else msa.msa_dense_workspace_size(st["cache"], st["batch"], c["heads"]))
    return st


def _softmax(x, sees):
    """Weights, their sums and the largest logits over the last axis of x, where `sees`."""
    x = torch.where(sees, x, torch.full((), -math.inf, device="cuda"))
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    return p, p.sum(dim=-1, keepdim=True), m


def _queries(st):
    return st["q"].view(torch.float8_e4m3fn).float() * st["q_scale"] if st["qd"] == "fp8" else st["q"].float()


def _run_attend(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_dense_attend(st["cache"], st["batch"], st["cfg"], st["query"], st["heads"], st["out"], st["lse"], st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    lens, n, H = st["seq_lens"], st["q_tokens"], st["kv_heads"]
    S, r = lens.shape[0], st["heads"] // H
    table = st["table"].clamp(min=0).long()
    q = _queries(st).view(S, n, H, r, DIM).permute(0, 2, 1, 3, 4).reshape(S, H, n * r, DIM)
    t = torch.arange(table.shape[1] * BLOCK, device="cuda")
    last = lens.view(S, 1) - n + torch.arange(n, device="cuda")  # the last key that each new token sees
    sees = (t <= last.unsqueeze(-1)).view(S, 1, n, 1, -1)
    x = torch.matmul(q, _values(st, "k", table).transpose(1, 2).flatten(2, 3).transpose(-1, -2)) * (DIM ** -0.5)
    p, total, m = _softmax(x.view(S, H, n, r, -1), sees)
    del x
    v = _values(st, "v", table).transpose(1, 2).flatten(2, 3)
    v = torch.where((t < lens.view(S, 1)).view(S, 1, -1, 1), v, torch.zeros((), device="cuda"))
    o = torch.matmul(p.view(S, H, n * r, -1), v).view(S, H, n, r, DIM)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(S * n, st["heads"], DIM).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(S * n, st["heads"])}


def _run_sparse(st):
    if own:
        import block_sparse_attention_03_gb300 as msa
        msa.msa_sparse_attend(st["cache"], st["batch"], st["cfg"], st["query"], st["heads"], st["topk"], st["out"], st["lse"], st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    lens, n, H, idx = st["seq_lens"], st["q_tokens"], st["kv_heads"], st["topk"].long()
    S, r = lens.shape[0], st["heads"] // H
    rows, K = S * n, idx.shape[-1]
    row = torch.arange(rows, device="cuda")
    last = (lens.view(S, 1) - n + torch.arange(n, device="cuda")).view(rows, 1, 1, 1)
    key = idx.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device="cuda")
    sees = ((idx >= 0).unsqueeze(-1) & (key <= last)).view(rows, H, 1, K * BLOCK)
    at = st["table"][(row // n).view(rows, 1, 1), idx.clamp(min=0)].clamp(min=0).long()
    head = torch.arange(H, device="cuda").view(1, H, 1)

    def picked(name):  # [rows][H][K x 128][128]
        x = st[name][at, head]
        x = x.float() if st["kv"] == "int8_block" else x.view(torch.float8_e4m3fn).float()
        return (x * st[name + "_scale"][at, head].view(rows, H, K, 1, 1)).flatten(2, 3)

    q = _queries(st).view(rows, H, r, DIM)
    p, total, m = _softmax(torch.matmul(q, picked("k").transpose(-1, -2)) * (DIM ** -0.5), sees)
    v = torch.where(sees.transpose(-1, -2), picked("v"), torch.zeros((), device="cuda"))
    o = torch.matmul(p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"out": o.reshape(rows, st["heads"], DIM).to(torch.bfloat16), "lse": (m + torch.log(total)).reshape(rows, st["heads"])}


def _code_values(exp_bits, man_bits, bias):
    """Values of the sign / exponent / mantissa codes of a small float format, in 64 bits."""
    got = []
    for code in range(1 << (1 + exp_bits + man_bits)):
        m, e = code & ((1 << man_bits) - 1), (code >> man_bits) & ((1 << exp_bits) - 1)
        v = math.ldexp(m, 1 - bias - man_bits) if e == 0 else math.ldexp((1 << man_bits) + m, e - bias - man_bits)
        if exp_bits == 4 and code & 0x7F == 0x7F:
            v = math.nan
        got.append(-v if code >> (exp_bits + man_bits) else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _rows64(st, name, phys, h):
    """Rows of a block, or of several one after another, of one head."""
    raw = st[name][phys, h]
    if st["kv"] == "bf16":
        return raw.double().reshape(-1, DIM)
    if st["kv"] == "nvfp4":
        e2m1 = _code_values(2, 1, 1)
        both = torch.stack((e2m1[(raw & 15).int()], e2m1[(raw >> 4).int()]), -1).reshape(-1, 8, 16)
        sf = _code_values(4, 3, 7)[st[name + "_sf"][phys, h].int()].reshape(-1, 8, 1)
        return (both * sf * float(st[name + "_global"])).reshape(-1, DIM)
    x = raw.double() if st["kv"] == "int8_block" else _code_values(4, 3, 7)[raw.int()]
    scale = st[name + "_scale"][phys, h].double()
    return (x * (scale.unsqueeze(-1) if st["kv"] == "fp8" else scale.view(-1, 1, 1))).reshape(-1, DIM)


def _attended(keys, vals, q):
    x = keys @ q.T / math.sqrt(DIM)
    z = torch.logsumexp(x, dim=0)
    return torch.exp(x - z).T @ vals, z


def _exact_outputs(c, st):
    q = _code_values(4, 3, 7)[st["q"].int()] * st["q_scale"] if c["qd"] == "fp8" else st["q"].double()
    rows = c["seqs"] * c["q_tokens"]
    return (q, torch.zeros((rows, c["heads"], DIM), dtype=torch.float64, device="cuda"),
            torch.full((rows, c["heads"]), -math.inf, dtype=torch.float64, device="cuda"))


def _exact_attend(c, seed):
    st = _prepare_attend(c, seed)
    n, H, r = c["q_tokens"], c["kv_heads"], c["heads"] // c["kv_heads"]
    q, out, lse = _exact_outputs(c, st)
    for s, T in enumerate(_lens(c)):
        phys = st["table"][s, :_blocks(T)].long()
        for h in range(H if T else 0):
            keys, vals = (_rows64(st, name, phys, h)[:T] for name in ("k", "v"))
            for i in range(n):
                see, at = T - n + i + 1, (s * n + i, slice(h * r, (h + 1) * r))
                if see >= 1:
                    out[at], lse[at] = _attended(keys[:see], vals[:see], q[at])
    return {"out": out, "lse": lse}


def _exact_sparse(c, seed):
    st = _prepare_attend(c, seed)
    n, H, r = c["q_tokens"], c["kv_heads"], c["heads"] // c["kv_heads"]
    q, out, lse = _exact_outputs(c, st)
    picks, table = st["topk"].tolist(), st["table"].tolist()
    for s, T in enumerate(_lens(c)):
        for i in range(n):
            see = T - n + i + 1
            for h in range(H):
                mine = [b for b in picks[s * n + i][h] if b >= 0]  # ascending: the last may hold keys that are not seen
                phys = torch.tensor([table[s][b] for b in mine], device="cuda")
                upto = (len(mine) - 1) * BLOCK + see - mine[-1] * BLOCK
                keys, vals = (_rows64(st, name, phys, h)[:upto] for name in ("k", "v"))
                at = (s * n + i, slice(h * r, (h + 1) * r))
                out[at], lse[at] = _attended(keys, vals, q[at])
    return {"out": out, "lse": lse}
