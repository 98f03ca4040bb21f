"""gdn_kv8_attn with 17 to 32 rows a key/value head: they go by the kernel for few rows, in two or three
eights, and meet attention_ref's tolerance without what the kernel for many rows may lose."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attention8_ref as R8
from tests import attention_ref as R
from tests import gpu_util as U
from tests.test_kv8_attn_gpu import queries, run

pytestmark = pytest.mark.gpu


def check(c, q, causal=True, window=0, scale=None):
    o, lse = run(c, q, causal, window, scale)
    ref = c.reference(U.f64(q), c.d ** -0.5 if scale is None else scale, causal, window)
    assert np.all(np.abs(U.f64(o) - ref[0]) <= R.tolerance(ref, q.dtype))
    empty = np.isneginf(ref[1])
    assert np.array_equal(empty, np.isneginf(U.f64(lse)))


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("lens", [[700, 33, 0], [2600, 1025, 3], [9000, 17, 20011]])
@pytest.mark.parametrize("G,new", [(1, 17), (12, 2), (5, 5), (4, 7), (8, 4)])
def test_matches_definition(G, new, lens, d, page):
    c = R8.Cache8(lens, 2, page, d, new=[new] * 3, head_scale=G == 8, seed=G + new)
    check(c, queries(c.tokens, 2 * G, d, torch.bfloat16, "thd", d + new))
    check(c, queries(c.tokens, 2 * G, d, torch.bfloat16, "thd", d + new), False, 40)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [17, 24, 32])
def test_weights_far_apart(rows, d):
    # keys that grow along the sequence or shrink, and values that are zero where weights are large
    page, n = 16, 1408
    for zero in (False, True):
        c = R8.Cache8([n], 1, page, d, new=[1], seed=9)
        for p in range(n // page):
            blk = c.table[0, p]
            c.np_pages[blk, 0, :page * d] = 0x38                              # every element 1 ...
            c.np_pages[blk, 0, R8.exponent_at(page, d, 0, 0)] = p // 4        # ... times 2^(p/4 - 15)
            if zero and (p < 8 or p >= n // page - 8):
                c.np_pages[blk, 0, page * d:2 * page * d] = 0
        c.upload()
        q = torch.ones(1, rows, d, dtype=torch.bfloat16, device="cuda")
        q[:, 1::3] = -1
        q[:, 2::5] = 0.01
        check(c, q, scale=0.02)
