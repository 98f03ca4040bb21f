"""Queries that are not finite, in both attention kernels and every type: their rows are NaN, as the fp64
definition has them, and no other row changes by a bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attention_ref as R
from tests import gpu_util as U
from tests.test_kv_attn_gpu import queries, run

pytestmark = pytest.mark.gpu


# 6 rows of a key/value head, 48 and 600 of several row tiles
@pytest.mark.parametrize("new", [3, 24, 300])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_rows_of_nonfinite_queries_are_nan(io, d, new):
    c = R.Cache([300 + new], 2, 64, d, new=[new], seed=80)
    q = queries(new, 4, d, io, "thd", 81)
    clean, clean_lse = run(c, q)
    q[1, 2, 7] = float("inf")           # (a key's 0 times infinity is a NaN)
    q[2, 0, 9] = float("nan")
    q[new - 1, 3, d - 1] = float("-inf")
    with np.errstate(invalid="ignore"):
        want, want_lse = c.reference(U.f64(q), d ** -0.5, True, 0)[:2]
    bad = torch.zeros(new, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = bad[new - 1, 3] = True
    assert np.array_equal(np.isnan(want).all(-1), bad.cpu().numpy())
    assert np.array_equal(np.isnan(want_lse), bad.cpu().numpy())
    o, lse = run(c, q)
    assert o[2, 0].isnan().all()
    assert o[1, 2].isnan().all()
    assert o[new - 1, 3].isnan().all()
    assert lse[bad].isnan().all()
    assert torch.equal(o[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])
