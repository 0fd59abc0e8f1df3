"""The launches of a batch that has more units than one of the dense attend's counts: which sequences each takes, and
where their parts of the call's arrays begin, for lists of keys and for whole sequences (host code alone)."""

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "msa_cut.h"
int main(int, char** a) {
  long v[9];
  for (int i = 0; i < 8; ++i) v[i] = atol(a[i + 1]);
  for (long s0 = 0; s0 < v[0];) {
    const msa::DenseCut c = msa::dense_cut(s0, v[0], v[1], v[2], v[3], (int)v[4], (int)v[5], (int)v[6], (int)v[7]);
    printf("%ld %ld %ld %ld %ld\n", c.s0, c.n, c.table, c.lists, c.row);
    if (c.n < 1) return 1;
    s0 += c.n;
  }
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("cut")
    (at / "main.cc").write_text(MAIN)
    include = os.path.join(ROOT, "block_sparse_attention_03_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-I", include, str(at / "main.cc"), "-o", str(at / "main")], check=True)

    def run(*v):
        r = subprocess.run([str(at / "main"), *map(str, v)], capture_output=True, text=True, check=True)
        return [tuple(map(int, x.split())) for x in r.stdout.splitlines()]

    return run


@pytest.mark.parametrize("seqs,per", [(1, 1), (7, 1), (7, 2), (7, 3), (7, 7), (7, 9), (64, 5)])
@pytest.mark.parametrize("tokens,hq,max_nb,G,topk", [(1, 4, 5, 4, 16), (3, 12, 7, 2, 8), (8, 64, 2, 1, 32)])
@pytest.mark.parametrize("lists", [False, True])
def test_parts_are_where_their_sequences_lie(cut, seqs, per, tokens, hq, max_nb, G, topk, lists):
    units = tokens * G * (topk + 1) if lists else G * (2 * max_nb + 4)
    table = np.arange(seqs * max_nb).reshape(seqs, max_nb)
    idx = np.arange(seqs * tokens * G * topk).reshape(seqs, tokens, G, topk)
    rows = np.arange(seqs * tokens * hq).reshape(seqs, tokens, hq)
    for limit in (per * units, per * units + units - 1):
        got = cut(seqs, units, limit, tokens, hq, max_nb, G, topk)
        assert [c[0] for c in got] == list(range(0, seqs, per)) and sum(c[1] for c in got) == seqs
        for s0, n, at, li, row in got:
            assert n * units <= limit
            assert (at, li, row) == (table[s0, 0], idx[s0, 0, 0, 0], rows[s0, 0, 0])


def test_offsets_pass_32_bits(cut):
    # 2^27 tokens' lists of 32, 4 heads, in launches of 2^32 - 1 units
    seqs, tokens, hq, max_nb, G, topk = 1 << 24, 8, 64, 300, 4, 32
    units = tokens * G * (topk + 1)
    got = cut(seqs, units, (1 << 32) - 1, tokens, hq, max_nb, G, topk)
    assert len(got) > 1 and got[-1][0] + got[-1][1] == seqs
    s0 = got[-1][0]
    assert got[-1][2:] == (s0 * max_nb, s0 * tokens * G * topk, s0 * tokens * hq) and got[-1][3] > 1 << 32
