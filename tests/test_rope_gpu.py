"""Rotary insert (msa_rope_insert) against a plain 64-bit norm and rotation and
the formats' rounding rules: layouts, partial rotations, several axes, far and
negative positions, strided inputs, padding and faulty slots, odd head counts."""

import numpy as np
import pytest
import torch

import block_sparse_attention_03_gb300 as msa
from oracle import msa_oracle as O

from _serving import HALF, plain_rope

pytestmark = pytest.mark.gpu

THETA = 5.0e6


def _cache(kv, idx, pool, H, g=2.0 ** -8):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    bufs, kw = {}, {}
    for name, dt, heads in (("k", kv, (H,)), ("v", kv, (H,)), ("idx", idx, ())):
        if dt == "bf16":
            bufs[name] = z(pool, *heads, 128, 128, dt=torch.bfloat16)
        elif dt == "fp8":
            bufs[name], bufs[name + "_scale"] = z(pool, *heads, 128, 128), z(pool, *heads, 128, dt=torch.float32)
        else:
            bufs[name], bufs[name + "_sf"] = z(pool, *heads, 128, 64), z(pool, *heads, 128, 8)
            kw[name + "_global"] = g
    cache = msa.PagedCache(kv_dtype=kv, index_dtype=idx, num_blocks=pool, num_kv_heads=H, **bufs, **kw)
    return cache, bufs


def _check_query(got, fp8, scale, ref, slack):
    if fp8:
        v = O.e4m3_value(got.cpu().numpy()) * scale
        ref_c = np.clip(ref, -448 * scale, 448 * scale)
        tol = HALF["fp8"] * np.abs(ref_c) + 2.0 ** -10 * scale + 2 * slack
        assert (np.abs(v - ref_c) <= tol).all()
    else:
        v = got.float().cpu().numpy()
        assert (np.abs(v - ref) <= HALF["bf16"] * np.abs(ref) + 2 * slack).all()


def _check_rows(bufs, name, dt, slots, ref, slack, g=2.0 ** -8):
    """ref [T][heads][128]; slack: bound of the fp32 error of each element before the format's rounding."""
    live = [t for t, s in enumerate(slots) if 0 <= s < bufs[name].shape[0] * 128]
    blk, off = np.array([slots[t] // 128 for t in live], int), np.array([slots[t] % 128 for t in live], int)
    ref, slack = ref[live], slack[live]

    def rows(key):
        x = bufs[key].float().cpu().numpy() if bufs[key].dtype != torch.uint8 else bufs[key].cpu().numpy()
        return x[blk, :, off] if name != "idx" else x[blk, off][:, None]

    x = rows(name)
    if dt == "bf16":
        assert (np.abs(x - ref) <= HALF["bf16"] * np.abs(ref) + 2 * slack).all()
    elif dt == "fp8":
        scale = rows("%s_scale" % name).astype(np.float64)
        amax = np.abs(ref).max(-1)
        want = np.where(amax > 0, amax / 448, 1.0)
        assert (np.abs(scale - want) <= 2.0 ** -23 * want + 2 * slack.max(-1) / 448).all()
        v = O.e4m3_value(x) * scale[..., None]
        # half a step of e4m3 (of its subnormals below 2^-6), the scale's and the quotient's roundings
        tol = HALF["fp8"] * np.abs(ref) + 2.0 ** -10 * scale[..., None] + 2 * slack + 2.0 ** -21 * np.abs(ref)
        assert (np.abs(v - ref) <= tol).all()
    else:
        sf = O.e4m3_value(rows("%s_sf" % name))
        amax = np.abs(ref).reshape(ref.shape[:-1] + (8, 16)).max(-1)
        want = np.minimum(amax / (6 * g), 448)
        sl = slack.reshape(amax.shape + (16,)).max(-1) / (6 * g)
        assert (np.abs(sf - want) <= HALF["fp8"] * want + 2.0 ** -10 + 2 * sl + 2.0 ** -21 * want).all()
        den = np.repeat(sf * g, 16, axis=-1)
        v = O.e2m1_value(O.unpack_e2m1(x)) * den
        z = np.abs(ref) / np.where(den > 0, den, 1)
        half = np.where(z <= 2, 0.25, np.where(z <= 4, 0.5, 1.0)) + np.maximum(z - 6, 0)
        tol = np.where(den > 0, half * den * (1 + 2.0 ** -20), np.abs(ref)) + 2 * slack
        assert (np.abs(v - ref) <= tol).all()


def _run(T, Hq, H, kv="bf16", idx="bf16", rotary=128, sections=None, layout="halves", q_fp8=False, norm=(), seed=0, strided=True,
         index=True, far=100000, padding=0, in_place=False, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    total = Hq + 3 * H + 1
    qkv = (torch.randn((T, total, 128), generator=gen) * torch.exp(torch.randn((T, total, 1), generator=gen))).bfloat16().cuda()
    parts = qkv.split([Hq, H, H, H, 1], dim=1)
    q, k, v, iq, ik = parts if strided else [x.contiguous() for x in parts]
    ik = ik.squeeze(1)
    sections = [rotary // 2] if sections is None else sections
    pos = torch.randint(-far, far, (len(sections), T), generator=gen, dtype=torch.int64).int()
    pool = -(-T // 128) + 2
    slots = torch.randperm(pool * 128, generator=gen)[:T].int()
    if padding:
        slots[torch.randperm(T, generator=gen)[:padding]] = -1
    cache, bufs = _cache(kv, idx, pool, H)
    rope = msa.msa_rope_init(rotary, THETA, sections, layout)
    w = {n: (0.3 * torch.randn(128, generator=gen)).bfloat16().cuda() for n in norm}
    qk = msa.QkNorm(eps=1e-6, offset=offset, **w) if norm else None
    dt, kind, scale = (torch.uint8, "fp8", 2.0 ** -5) if q_fp8 else (torch.bfloat16, "bf16", 1.0)
    hq = q.cpu().clone()
    q_out = msa.Query(q if in_place else torch.zeros((T, Hq, 128), dtype=dt, device="cuda"), kind, scale)
    iq_out = msa.Query(torch.zeros((T, H, 128), dtype=dt, device="cuda"), kind, scale) if index else None
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_rope_insert(cache, rope, pos.cuda(), slots.cuda(), q, q_out, iq if index else None, iq_out, k, v,
                        ik if index else None, qk, ws)
    assert msa.msa_read_device_status(ws)[1] == 0
    p = pos.numpy()

    def want(x, name):
        x = x.float().cpu().numpy()
        x = x[:, None] if x.ndim == 2 else x
        ref = plain_rope(x, None if name == "v" else p, rotary, THETA, sections, layout,
                         w[name].float().cpu().numpy() if name in w else None, 1e-6, offset)
        # fp32 before the rounding: sine and cosine to 4e-7 (the angle 2^-23 of a half turn, sincospif
        # two steps), two products and a sum; the norm's sum, root and two products to 12 roundings
        size = np.sqrt((ref ** 2).sum(-1, keepdims=True)) if name != "v" else 0 * ref[..., :1]
        pairs = np.abs(ref)  # |a| + |b| <= 2 max of the turned pair's length; bounded by the row's norm
        return ref, (6e-7 * np.minimum(size, 2 * np.abs(ref).max(-1, keepdims=True)) + (12 * 2.0 ** -24 if name in w else 0) * pairs) * np.ones_like(ref)

    ref, slack = want(hq, "q")
    _check_query(q_out.data, q_fp8, scale, ref, slack)
    s = slots.tolist()
    if index:
        _check_query(iq_out.data, q_fp8, scale, *want(iq, "index_q"))
        _check_rows(bufs, "idx", idx, s, *want(ik, "index_k"))
    _check_rows(bufs, "k", kv, s, *want(k, "k"))
    _check_rows(bufs, "v", kv, s, *want(v, "v"))
    # rows that no token maps to are as they were
    dead = torch.ones(pool * 128, dtype=torch.bool)
    dead[slots[slots >= 0].long()] = False
    for name, x in bufs.items():
        if name.startswith("idx") and not index:
            assert (x == 0).all()
            continue
        flat = x.cpu().movedim(2, 1).flatten(0, 1) if not name.startswith("idx") else x.cpu().flatten(0, 1)
        assert (flat[dead] == 0).all(), name
    return bufs


@pytest.mark.parametrize("kv,idx", [("bf16", "bf16"), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("fp8", "bf16"), ("nvfp4", "fp8")])
@pytest.mark.parametrize("T", [1, 2, 33, 300])
def test_formats(kv, idx, T):
    _run(T, 8, 2, kv, idx, norm=("q", "k", "index_q", "index_k"), seed=T)


@pytest.mark.parametrize("rotary,sections,layout", [(128, [64], "adjacent"), (64, [32], "halves"), (96, [24, 12, 12], "halves"),
                                                    (32, [8, 4, 4], "adjacent"), (16, [8], "halves"), (128, [16, 24, 24, 0], "halves"),
                                                    (128, [0, 64], "adjacent")])
def test_rotations(rotary, sections, layout):
    _run(70, 5, 1, rotary=rotary, sections=sections, layout=layout, seed=rotary)


@pytest.mark.parametrize("layout", ["halves", "adjacent"])
def test_four_axes(layout):
    _run(45, 4, 2, "fp8", "fp8", rotary=128, sections=[7, 21, 13, 23], layout=layout, far=100000, seed=12)


@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (7, 7), (64, 4), (16, 8)])
def test_head_counts(Hq, H):
    _run(40, Hq, H, "fp8", "fp8", seed=Hq)


def test_far_positions_lose_no_precision():
    _run(64, 4, 2, far=2 ** 31 - 1, seed=3)


def test_e4m3_queries_and_no_index():
    _run(50, 6, 2, "nvfp4", "nvfp4", q_fp8=True, norm=("q",), seed=4)
    _run(50, 6, 2, "fp8", "fp8", index=False, seed=5)


def test_many_tokens_with_padding():
    _run(6001, 4, 1, "fp8", "fp8", padding=1000, norm=("q", "k"), seed=6)


def test_queries_in_place():
    _run(90, 4, 2, strided=False, in_place=True, seed=7)


def test_zero_rotation_is_the_cache_insert():
    # positions 0, no norm: the caches get msa_cache_insert's bytes
    for kv in ("bf16", "fp8", "nvfp4"):
        gen = torch.Generator().manual_seed(8)
        T, H = 200, 4
        k, v, q = ((torch.randn((T, H, 128), generator=gen)).bfloat16().cuda() for _ in range(3))
        ik = torch.randn((T, 128), generator=gen).bfloat16().cuda()
        slots = torch.randperm(3 * 128, generator=gen)[:T].int().cuda()
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        a, ab = _cache(kv, kv, 3, H)
        b, bb = _cache(kv, kv, 3, H)
        msa.msa_cache_insert(a, slots, k, v, ik, ws)
        out = msa.Query(torch.empty_like(q))
        msa.msa_rope_insert(b, msa.msa_rope_init(128, THETA), torch.zeros((1, T), dtype=torch.int32, device="cuda"), slots, q, out,
                            None, None, k, v, ik, None, ws)
        assert msa.msa_read_device_status(ws)[1] == 0
        assert torch.equal(out.data, q)
        for name in ab:
            assert torch.equal(ab[name].view(torch.uint8), bb[name].view(torch.uint8)), (kv, name)


def test_slot_outside_the_pool_is_flagged_and_skipped():
    gen = torch.Generator().manual_seed(9)
    T, H = 5, 2
    q, k, v = (torch.randn((T, H, 128), generator=gen).bfloat16().cuda() for _ in range(3))
    cache, bufs = _cache("fp8", "fp8", 2, H)
    slots = torch.tensor([1, 256, -1, 2 ** 31 - 1, 130], dtype=torch.int32, device="cuda")
    out = msa.Query(torch.zeros_like(q))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    msa.msa_rope_insert(cache, msa.msa_rope_init(64, 1e4), pos, slots, q, out, None, None, k, v, None, None, ws)
    assert msa.msa_read_device_status(ws) == (5, 1)
    written = (bufs["k_scale"] != 0).any(1).flatten().nonzero().flatten().tolist()
    assert written == [1, 130]
    assert (out.data != 0).any(-1).all()  # the queries are written all the same


def test_custom_frequencies():
    # a caller's own table: every pair a quarter turn a position, the second half the other way round
    rope = msa.msa_rope_init(128, THETA)
    for i in range(64):
        rope.turns[i] = 1 << 62 if i < 32 else (1 << 64) - (1 << 62)
    x = torch.randn((4, 1, 128), generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    cache, _ = _cache("bf16", "bf16", 1, 1)
    out = msa.Query(torch.empty_like(x))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pos = torch.tensor([0, 1, 2, -1], dtype=torch.int32, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    msa.msa_rope_insert(cache, rope, pos, slots, x, out, None, None, x, x, None, None, ws)
    a, b = x[:, 0, :64].float(), x[:, 0, 64:].float()
    sign = torch.ones(64, device="cuda")
    sign[32:] = -1
    y0, y1 = out.data[:, 0, :64].float(), out.data[:, 0, 64:].float()
    for t, quarter in enumerate((0, 1, 2, -1)):
        c = [1.0, 0.0, -1.0, 0.0][quarter % 4]
        s = [0.0, 1.0, 0.0, -1.0][quarter % 4] * sign
        assert torch.equal(y0[t], a[t] * c - b[t] * s) and torch.equal(y1[t], a[t] * s + b[t] * c)
