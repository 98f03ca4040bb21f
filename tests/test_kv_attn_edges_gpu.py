"""gdn_kv_attn where its arguments or its pieces of work change the form of a call: windows as large
as an int next to rows before place 0, pieces with one and with two row tiles in turn."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from tests import attention_ref as R
from tests.test_kv_attn_gpu import check, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31, 2 ** 32 + 3, sys.maxsize])
@pytest.mark.parametrize("lens,new", [([300, 3, 0], 7), ([3, 150], 40), ([300, 1], 4)])
def test_window_as_large_as_can_be(lens, new, window, causal, io):
    # "no window" as it is often spelled, where a sequence has fewer places than new tokens: rows
    # that see something share a row tile with rows that see nothing (tiles of 8 rows: the last
    # case; of 256: the second, in bf16)
    c = R.Cache(lens, 1, 16, 64, new=[new] * len(lens), seed=40 + new)
    q = queries(c.tokens, 2, 64, io, "thd", 41)
    o = check(c, q, causal, window)
    assert (o == check(c, q, causal, 0)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_at_the_end_of_pieces_with_one_and_two_row_tiles(d):
    # sequences of 200 and of 20 rows in turn, several in every CTA: the second row tile's warps
    # have nothing to do in every other piece.  A NaN among the last values of every third
    # sequence is found by the rows that see it, and by nobody else.
    page, B = 64, 301
    new = [100 if b % 2 == 0 else 10 for b in range(B)]
    lens = [150 + (37 * b) % 700 for b in range(B)]
    c = R.Cache(lens, 1, page, d, new=new, seed=42)
    q = queries(c.tokens, 2, d, torch.bfloat16, "thd", 43)
    clean, _ = run(c, q)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    code, scale = page * d // 2, page * d // 16
    for b in range(0, B, 3):
        back = 1 + b % 5                                       # places before the end
        where = lens[b] - back
        row, block = where % page, b % (d // 16)
        c.np_pages[c.table[b, where // page], 0, 2 * code + scale + row * (d // 16) + block] = 0x7F
        bad[c.at[b + 1] - back:c.at[b + 1], :, 16 * block:16 * block + 16] = True
    c.pages = torch.from_numpy(np.ascontiguousarray(c.np_pages)).cuda()
    for _ in range(5):
        o, _ = run(c, q)
        assert torch.equal(o.isnan(), bad)
        assert torch.equal(o[~bad], clean[~bad])
