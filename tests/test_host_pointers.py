"""Pointers that the serving entry points refuse before any launch (no GPU is touched)."""

import ctypes

import pytest

from test_host_serving import _structs, lib  # noqa: F401  (a fixture)

ref = ctypes.byref


def test_misaligned_words_are_refused(lib):  # noqa: F811
    import block_sparse_attention_03_gb300 as msa

    def dense(lse=None, **over):
        c, b, f = _structs(**over)
        q = msa.MsaQueryT(16, 0, 1.0)
        return lib.msa_dense_attend(ref(c), ref(b), ref(f), ref(q), 16, 16, lse, ctypes.c_void_p(4096), 1 << 30, None)

    for off in (1, 2, 3):
        assert dense(lse=64 + off) == 1 and dense(b__seq_lens=64 + off) == 1 and dense(b__block_table=64 + off) == 1

    def rope(tokens=0, pos=16, slots=16, ws=4096):
        c, _, _ = _structs()
        r = msa.msa_rope_init(128, 1e4)
        row, out = msa.MsaRowsT(16, 4096), msa.MsaQueryT(16, 0, 1.0)
        return lib.msa_rope_insert(ref(c), ref(r), tokens, pos, slots, 16, ref(row), ref(out), None, None, ref(row), ref(row), None,
                                   None, ctypes.c_void_p(ws), 256, None)

    def insert(tokens=0, slots=16, ws=4096):
        c, _, _ = _structs()
        return lib.msa_cache_insert(ref(c), tokens, slots, 16, 16, None, ctypes.c_void_p(ws), 256, None)

    assert rope() == 0 and insert() == 0
    for tokens in (0, 5):
        for off in (1, 2, 3):
            assert rope(tokens, pos=64 + off) == 1 and rope(tokens, slots=64 + off) == 1 and rope(tokens, ws=4096 + off) == 1
            assert insert(tokens, slots=64 + off) == 1 and insert(tokens, ws=4096 + off) == 1


# arguments of msa_build_tables, in its order, none of the arrays near another
NAMES = ("num_seqs", "num_blocks", "cached", "new", "max_nb", "table", "cap", "free", "count", "count_out", "lens", "offsets",
         "max_tokens", "slots", "positions", "ws", "size", "stream")
ARRAYS = ("cached", "new", "table", "free", "count", "count_out", "lens", "offsets", "slots", "positions")


def _tables(lib, **over):  # noqa: F811
    base = dict(num_seqs=4, num_blocks=100, max_nb=10, cap=100, max_tokens=50, ws=ctypes.c_void_p(4096), size=256, stream=None)
    base.update({n: 65536 * (i + 1) for i, n in enumerate(ARRAYS)})
    return lib.msa_build_tables(*[{**base, **over}[n] for n in NAMES])


@pytest.mark.parametrize("name", ARRAYS)
def test_misaligned_words_of_the_tables(lib, name):  # noqa: F811
    for off in (1, 2, 3):
        assert _tables(lib, **{name: 1 << 20 | off}) == 1
        assert _tables(lib, ws=ctypes.c_void_p(4096 + off)) == 1


SIZES = dict(zip(ARRAYS, (4, 4, 40, 100, 1, 1, 4, 5, 50, 50)))  # words
INPUTS = ("cached", "new", "count")


@pytest.mark.parametrize("a", [n for n in ARRAYS if n not in INPUTS])
@pytest.mark.parametrize("b", ARRAYS)
def test_what_the_tables_write_overlaps_nothing(lib, a, b):  # noqa: F811
    if a == b:
        return
    at = 1 << 20
    for off in {0, SIZES[b] - 1, 1 - SIZES[a]}:  # the same place, the last word, the first word
        assert _tables(lib, **{b: at, a: at + 4 * off}) == 1, off
    assert _tables(lib, **{a: 4096 + 4}) == 1  # the workspace's status word is written too
