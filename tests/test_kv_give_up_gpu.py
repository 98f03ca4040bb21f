"""The bounded waits of the attention kernels over the cache, where they run out: every lane of a
warp learns the same, the host reads a timeout, and the context stays usable."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests.test_kv_attn_gpu import check, queries

pytestmark = pytest.mark.gpu


def status():
    return gdn.load().gdn_sync_check(gdn._stream(None))


def test_completed_waits_succeed_in_every_lane():
    status()
    assert gdn.selftest_ring(True, 1000)[:2] == (256, 256)
    assert status() == gdn.GDN_OK


@pytest.mark.parametrize("limit", [1, 64])
def test_waits_that_nothing_completes_give_up_in_every_lane(limit):
    status()
    assert gdn.selftest_ring(False, limit)[:2] == (0, 0)
    assert status() == gdn.GDN_ERR_DEVICE_TIMEOUT
    assert status() == gdn.GDN_OK                # cleared once read
    c = R.Cache([300, 70], 2, 16, 64, new=[3, 3], seed=60)
    check(c, queries(6, 4, 64, torch.bfloat16, "thd", 61))


def test_refusals():
    for args in ((True, 0), (True, -1), (False, 1 << 23)):
        with pytest.raises(gdn.GdnError):
            gdn.selftest_ring(*args)
