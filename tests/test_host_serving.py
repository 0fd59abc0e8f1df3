"""Refusals of the serving entry points, before any launch (no GPU is touched)."""

import ctypes
import math

import pytest

ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_03_gb300 import _build
    import block_sparse_attention_03_gb300 as msa
    _build.build()
    return msa.lib()


def _structs(**over):
    import block_sparse_attention_03_gb300 as msa
    c = msa.MsaCacheT(1, 1, 100, 128, 4, 128, 128, 16, 32, None, None, 48, 64, 80, None, 96, 0, 0, 0)
    b = msa.MsaBatchT(2, 1, 50, 16, 32)
    f = msa.MsaConfigT(16, 0, 0, 128 ** -0.5, 128 ** -0.5, 0)
    for k, v in over.items():
        obj, field = k.split("__")
        setattr({"c": c, "b": b, "f": f}[obj], field, v)
    return c, b, f


def test_dense_refusals(lib):
    import block_sparse_attention_03_gb300 as msa
    ws, big = ctypes.c_void_p(4096), 1 << 30

    def call(q=None, hq=16, out=16, ws=ws, size=big, **over):
        c, b, f = _structs(**over)
        q = msa.MsaQueryT(16, 0, 1.0) if q is None else q
        return lib.msa_dense_attend(ref(c), ref(b), ref(f), ref(q), hq, out, None, ws, size, None)

    c, b, f = _structs()
    need = lib.msa_dense_workspace_size(ref(c), ref(b), 16)
    assert need > 256
    assert call(size=need - 1) == 3
    assert call(hq=15) == 1 and call(hq=0) == 1
    assert call(hq=4 * 65) == 2 and call(b__q_per_seq=9) == 2
    assert call(out=None) == 1 and call(out=24) == 1 and call(ws=None) == 1 and call(ws=ctypes.c_void_p(4100)) == 1
    assert call(q=msa.MsaQueryT(None, 0, 1.0)) == 1 and call(q=msa.MsaQueryT(16, 2, 1.0)) == 2
    assert call(q=msa.MsaQueryT(16, 1, 0.0)) == 1
    assert call(c__k=None) == 1 and call(c__v=17) == 1 and call(c__k_scale=None) == 1 and call(c__kv_dtype=3) == 2
    assert call(f__sm_scale=math.inf) == 1 and call(b__num_seqs=0) == 1 and call(b__seq_lens=None) == 1
    assert lib.msa_dense_attend(None, ref(b), ref(f), None, 16, 16, None, ws, big, None) == 1
    # the workspace does not grow with the batch or the length, and 0 is an invalid description
    c2, b2, _ = _structs(b__num_seqs=500, b__max_blocks_per_seq=4000)
    assert lib.msa_dense_workspace_size(ref(c2), ref(b2), 16) == need
    assert lib.msa_dense_workspace_size(ref(c), ref(b), 15) == 0
    c3, b3, _ = _structs(b__q_per_seq=9)
    assert lib.msa_dense_workspace_size(ref(c3), ref(b3), 16) == 0


def test_rope_init(lib):
    import block_sparse_attention_03_gb300 as msa
    r = msa.msa_rope_init(128, 1e4, [16, 24, 24])
    assert list(r.axis) == [0] * 16 + [1] * 24 + [2] * 24 and r.axes == 3
    for i in (0, 1, 17, 63):  # turns a position x 2^64, to double precision
        assert abs(r.turns[i] / 2.0 ** 64 - 1e4 ** (-2 * i / 128) / (2 * math.pi)) <= 2.0 ** -50 * 1e4 ** (-2 * i / 128)
    for bad in (dict(rotary_dim=120), dict(rotary_dim=144), dict(rotary_dim=0), dict(theta=0.0), dict(theta=math.nan),
                dict(sections=[32]), dict(sections=[70, -6]), dict(sections=[65]), dict(sections=[16, 16, 16, 8, 8]),
                dict(sections=[]), dict(layout="other")):
        args = dict(rotary_dim=128, theta=1e4, sections=[64], layout="halves")
        args.update(bad)
        with pytest.raises(msa.MsaError):
            msa.msa_rope_init(**args)


def test_rope_refusals(lib):
    import block_sparse_attention_03_gb300 as msa
    ws = ctypes.c_void_p(4096)

    def call(rope=None, tokens=4, pos=16, slots=16, hq=16, q=(16, 4096), qo=(16, 0, 1.0), iq=(16, 4096), iqo=(16, 0, 1.0),
             k=(16, 4096), v=(16, 4096), ik=(16, 4096), norm=None, ws=ws, size=256, **over):
        c, _, _ = _structs(**over)
        rope = msa.msa_rope_init(128, 1e4) if rope is None else rope
        rows = [None if x is None else ref(msa.MsaRowsT(*x)) for x in (q, iq, k, v, ik)]
        out = [None if x is None else ref(msa.MsaQueryT(*x)) for x in (qo, iqo)]
        n = None if norm is None else ref(norm)
        return lib.msa_rope_insert(ref(c), ref(rope), tokens, pos, slots, hq, rows[0], out[0], rows[1], out[1], rows[2], rows[3],
                                   rows[4], n, ws, size, None)

    assert call(tokens=0) == 0
    assert call(tokens=-1) == 1 and call(pos=None) == 1 and call(slots=None) == 1 and call(hq=0) == 2
    assert call(q=None) == 1 and call(q=(None, 8)) == 1 and call(q=(24, 4096)) == 1 and call(q=(16, 4100)) == 1
    assert call(k=(16, -8)) == 1 and call(v=None) == 1
    assert call(iq=None) == 1 and call(iqo=None) == 1  # one of the two without the other
    assert call(qo=(16, 2, 1.0)) == 2 and call(qo=(16, 1, 0.0)) == 1 and call(qo=(16, 1, 1e-39)) == 1 and call(qo=(20, 0, 1.0)) == 1
    assert call(ws=None) == 1 and call(size=255) == 3
    assert call(c__idx=None) == 1 and call(c__v_scale=None) == 1
    bad = msa.msa_rope_init(128, 1e4)
    bad.axis[5] = 1
    assert call(rope=bad) == 1
    bad = msa.msa_rope_init(128, 1e4)
    bad.rotary_dim = 24
    assert call(rope=bad) == 2
    assert call(norm=msa.MsaQkNormT(17, None, None, None, 1e-6, 0.0)) == 1
    assert call(norm=msa.MsaQkNormT(16, None, None, None, -1.0, 0.0)) == 1
    assert call(norm=msa.MsaQkNormT(16, None, None, None, math.nan, 0.0)) == 1


def test_tables_refusals(lib):
    ws = ctypes.c_void_p(4096)
    names = ("num_seqs", "num_blocks", "cached", "new", "max_nb", "table", "cap", "free", "count", "count_out", "lens", "offsets",
             "max_tokens", "slots", "positions", "ws", "size", "stream")
    base = dict(zip(names, (4, 100, 16, 32, 10, 48, 100, 64, 80, 96, 112, 128, 50, 144, 160, ws, 256, None)))

    def call(**over):
        return lib.msa_build_tables(*[{**base, **over}[n] for n in names])

    for bad in (dict(num_seqs=0), dict(num_blocks=0), dict(max_nb=0), dict(cap=-1), dict(max_tokens=-1), dict(cached=None),
                dict(new=None), dict(table=None), dict(free=None), dict(count=None), dict(count_out=None), dict(lens=None),
                dict(offsets=None), dict(slots=None), dict(positions=None), dict(ws=None), dict(count_out=80), dict(lens=16),
                dict(lens=32), dict(offsets=16), dict(offsets=32)):
        assert call(**bad) == 1, bad
    assert call(num_seqs=8193) == 2 and call(num_blocks=1 << 24) == 2 and call(max_nb=(1 << 23) + 1) == 2
    assert call(max_tokens=1 << 30) == 2 and call(size=255) == 3


class _Elsewhere:
    """A tensor that says it is on device `at`."""

    def __init__(self, t, at=0):
        self._t, self._at = t, at

    def get_device(self):
        return self._at

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def on_device_0(monkeypatch):
    """The binding takes device 0 for the current one; no call may reach the library."""
    import block_sparse_attention_03_gb300 as msa

    def never(*a):
        raise AssertionError("the call was not refused")

    msa._torch_names()
    monkeypatch.setattr(msa, "_device", lambda: 0)
    monkeypatch.setattr(msa, "_lib_handle", type("Lib", (), {n: staticmethod(never) for n in msa.EXPORTS})())
    return msa


def _refused(msa, call, good, bad):
    for name, value in bad:
        with pytest.raises(msa.MsaError):
            call(**{**good, name: value})
    with pytest.raises(AssertionError):  # and as it is, it would have gone through
        call(**good)


def test_python_refuses_what_the_kernels_would_misread(on_device_0):
    import torch
    msa = on_device_0
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    z = lambda *s, dt=bf, at=0: _Elsewhere(torch.zeros(s, dtype=dt), at)  # noqa: E731
    cut = lambda *s, dt=i32: _Elsewhere(torch.zeros((*s, 2), dtype=dt)[..., 0])  # noqa: E731  not dense
    cache = msa.PagedCache("bf16", "bf16", 2, 2, z(2, 2, 128, 128), z(2, 2, 128, 128), None)
    ws = z(4096, dt=u8)

    def dense(lens, table, q, out, lse, k=cache.k):
        c = msa.PagedCache("bf16", "bf16", 2, 2, k, cache.v, None)
        msa.msa_dense_attend(c, msa.Batch(lens, table, 2), msa.Config(), msa.Query(q), 4, out, lse, ws, stream=0)

    _refused(msa, dense, dict(lens=z(3, dt=i32), table=z(3, 5, dt=i32), q=z(6, 4, 128), out=z(6, 4, 128),
                              lse=z(6, 4, dt=torch.float32)),
             [("lens", z(3, dt=torch.int64)), ("lens", cut(3)), ("lens", z(3, dt=i32, at=1)), ("table", z(2, 5, dt=i32)),
              ("table", z(15, dt=i32)), ("table", cut(3, 5)), ("table", z(3, 5, dt=torch.int64)), ("q", z(3, 4, 128)),
              ("q", z(6, 4, 128, dt=torch.float32)), ("q", z(6, 4, 128, at=-1)), ("out", z(6, 4, 64)),
              ("out", z(6, 4, 128, dt=torch.float32)), ("out", cut(6, 4, 128, dt=bf)), ("lse", z(6, 4)),
              ("lse", z(3, 4, dt=torch.float32)), ("lse", z(6, 4, dt=torch.float32, at=-1)),
              ("k", z(2, 2, 128, 128, at=1)), ("k", z(2, 2, 128, 128, at=-1))])

    rope = msa.MsaRopeT()
    rope.axes = 2

    def insert(pos, slots, q, qo, k, v, w):
        msa.msa_rope_insert(cache, rope, pos, slots, q, msa.Query(qo), None, None, k, v, None, msa.QkNorm(q=w), ws, stream=0)

    _refused(msa, insert, dict(pos=z(2, 3, dt=i32), slots=z(3, dt=i32), q=z(3, 4, 128), qo=z(3, 4, 128),
                               k=z(3, 2, 128), v=z(3, 2, 128), w=z(128)),
             [("pos", z(2, 3, dt=torch.int64)), ("pos", cut(2, 3)), ("slots", cut(3)), ("slots", z(3, dt=torch.int64)),
              ("slots", z(3, dt=i32, at=1)), ("q", z(3, 4, 128, dt=torch.float16)), ("qo", z(3, 4, 128, dt=u8)),
              ("qo", cut(3, 4, 128, dt=bf)), ("k", z(3, 2, 128, dt=torch.float32)), ("v", z(3, 2, 128, at=1)),
              ("qo", z(3, 4, 128, at=1)), ("k", z(3, 2, 128, at=-1)), ("w", z(64)), ("w", z(128, at=-1)),
              ("w", z(128, dt=torch.float32)), ("w", cut(128, dt=bf))])

    names = ("cached_lens", "new_lens", "block_table", "free_blocks", "free_count", "seq_lens", "token_offsets", "slot_mapping",
             "positions", "free_count_out")
    sizes = ((3,), (3,), (3, 5), (9,), (1,), (3,), (4,), (7,), (7,), (1,))
    good = {n: z(*s, dt=i32) for n, s in zip(names, sizes)}
    _refused(msa, lambda **a: msa.msa_build_tables(10, workspace=ws, stream=0, **a), good,
             [(n, z(*s, dt=torch.int64)) for n, s in zip(names, sizes)] +
             [(n, z(*s, dt=i32, at=-1)) for n, s in zip(names, sizes)] +
             [(n, cut(*s)) for n, s in zip(names, sizes) if s != (1,)] +
             [("block_table", z(3, 5, dt=i32, at=1)), ("block_table", z(3, 5, dt=i32, at=-1)), ("block_table", z(2, 5, dt=i32)),
              ("seq_lens", z(2, dt=i32)), ("token_offsets", z(3, dt=i32)), ("positions", z(6, dt=i32)), ("new_lens", z(4, dt=i32))])


def test_python_checks_shapes():
    import torch
    import block_sparse_attention_03_gb300 as msa
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    cache = msa.PagedCache("bf16", "bf16", 2, 2, z(2, 2, 128, 128), z(2, 2, 128, 128), None)
    rope = msa.msa_rope_init(128, 1e4)
    pos, slots, ws = z(1, 3, dt=torch.int32), z(3, dt=torch.int32), z(256, dt=torch.uint8)
    good = dict(q=z(3, 4, 128), q_out=msa.Query(z(3, 4, 128)), k=z(3, 2, 128), v=z(3, 2, 128))
    for bad in (dict(k=z(3, 1, 128)), dict(v=z(2, 2, 128)), dict(k=z(3, 2, 256)[..., ::2]), dict(q_out=msa.Query(z(3, 3, 128))),
                dict(q=z(3, 128))):
        a = {**good, **bad}
        with pytest.raises(msa.MsaError):
            msa.msa_rope_insert(cache, rope, pos, slots, a["q"], a["q_out"], None, None, a["k"], a["v"], None, None, ws, stream=0)
    with pytest.raises(msa.MsaError):
        msa.msa_rope_insert(cache, rope, z(2, 3, dt=torch.int32), slots, good["q"], good["q_out"], None, None, good["k"], good["v"],
                            None, None, ws, stream=0)
