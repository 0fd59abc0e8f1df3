"""Rows of the dense attend that see no key: out 0 and lse -inf whatever their
query holds, beside rows that do see keys."""

import numpy as np
import pytest
import torch

from _serving import check_dense, paged_case, plain_dense, run_dense

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("r", [1, 4, 8])
def test_a_query_that_is_not_finite_where_no_key_is_seen(kv, r, bad):
    # sequences shorter than the five new tokens: the first tokens sit at negative positions
    Q, lens = 5, [3, 0, 1, 200]
    c = paged_case(lens, kv, Q=Q, Hq=r, H=1, seed=51)
    clean = plain_dense(c)
    see = np.array([max(0, T - Q + i + 1) for T in lens for i in range(Q)])
    rows = torch.tensor(np.flatnonzero(see == 0)).cuda()
    c["q"][rows, :, 3] = bad
    c["q"][17] = bad  # and one that sees 198 keys
    out, lse = run_dense(c)
    assert torch.isnan(out[17].float()).all() and torch.isnan(lse[17]).all()
    keep = np.array([i for i in range(len(see)) if i != 17])
    check_dense(c, out, lse, clean, rows=keep)
