"""gdn_kv_attn at the ends of its arguments' ranges: windows as large as an int next to rows before
place 0."""
from __future__ import annotations

import sys

import pytest
import torch

from tests import attention_ref as R
from tests.test_kv_attn_gpu import check, queries

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
