"""Packed offsets of the cache's entry points that leave tokens to no sequence."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests.test_kv_attn_gpu import queries

pytestmark = pytest.mark.gpu

# (offsets, tokens of the call)
BAD = [([2, 3, 5], 5), ([0, 3, 4], 5), ([0, 0, 0], 5), ([5, 5, 5], 5), ([1, 3, 5], 5)]
GOOD = [([0, 3, 5], 5), ([0, 0, 5], 5), ([0, 5, 5], 5)]


@pytest.mark.parametrize("entry", ["append", "read", "attn few", "attn many"])
@pytest.mark.parametrize("cu,n", BAD + GOOD)
def test_offsets_have_to_pack_the_tokens(cu, n, entry):
    c = R.Cache([40, 20], 2, 16, 64, new=[3, 2], seed=50)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    at = (c.pages, c.table_t, c.len_t)
    q = queries(n, 16 if entry == "attn many" else 4, 64, torch.bfloat16, "thd", 51)
    gdn.sync_check()

    def call():
        if entry == "append":
            gdn.gdn_kv_append(c.pages, q[:, :2], q[:, 2:], *at[1:], cu_seqlens=off, check=True)
        elif entry == "read":
            gdn.gdn_kv_read(*at, n, 64, cu_seqlens=off, check=True)
        else:
            gdn.gdn_kv_attn(q, *at, cu_seqlens=off, check=True)

    if (cu, n) in GOOD:
        call()
        return
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()      # reported once
