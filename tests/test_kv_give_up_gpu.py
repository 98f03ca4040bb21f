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


@pytest.mark.parametrize("complete,limit", [(True, 1000), (False, 1), (False, 64)])
def test_copies_that_nobody_waited_for_are_drained(complete, limit):
    # by the drain's own bound, not the one that has run out
    for _ in range(20):
        assert gdn.selftest_ring(complete, limit)[2] == 2048
    status()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("limit", [1, 2, 8])
def test_short_limits_end_in_a_status(limit, io):
    # whether or not a wait runs out at so few polls, the call ends, says so, and the next one
    # is right (8 rows of a head at most: the kernel whose tiles arrive by bulk copies)
    c = R.Cache([9000, 77, 0, 4000, 12001], 2, 16, 64, seed=62)
    q = queries(5, 8, 64, io, "thd", 63)
    want = check(c, q)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    prev = gdn.get_option(gdn.GDN_OPT_WAIT_LIMIT)
    gdn.set_option(gdn.GDN_OPT_WAIT_LIMIT, limit)
    try:
        for _ in range(5):
            flush.zero_()
            o = gdn.gdn_kv_attn(q, c.pages, c.table_t, c.len_t)
            s = status()
            assert s in (gdn.GDN_OK, gdn.GDN_ERR_DEVICE_TIMEOUT)
            if s == gdn.GDN_OK:
                assert (o.double().cpu().numpy() == want).all()
    finally:
        gdn.set_option(gdn.GDN_OPT_WAIT_LIMIT, prev)
    assert (check(c, q) == want).all()


def test_refusals():
    for args in ((True, 0), (True, -1), (False, 1 << 23)):
        with pytest.raises(gdn.GdnError):
            gdn.selftest_ring(*args)
