"""The cache's entry points through the debug bounds-check build (csrc/gdn_check.cuh): small cases of
both attention kernels, every width and type, match the fp64 definition with no check failed."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import _build
from tests import attention_ref as R
from tests.test_kv_attn_gpu import check, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked_lib():
    lib = gdn.load(_build.build_variant("check"))
    prev = gdn._lib
    gdn._lib = lib   # the binding's calls go through the checked library
    try:
        assert lib.gdn_bounds_violation(1) == 0   # a checked build, nothing recorded yet
        yield lib
    finally:
        gdn._lib = prev


def clean(lib):
    assert lib.gdn_sync_check(gdn._stream(None)) == gdn.GDN_OK
    line = lib.gdn_bounds_violation(1)
    assert line == 0, "bounds check failed at source line %d" % line


# lens, new, Hq, H, d, page, causal, window: up to 16 rows of a head, or any rows in fp32 or at d = 256
FEW = [
    ([0, 1, 15, 16, 17, 255, 256, 300], [1] * 8, 8, 2, 128, 64, True, 0),
    ([5000, 77], [1, 1], 4, 2, 64, 16, True, 0),
    ([700, 513, 40], [5, 5, 5], 4, 2, 128, 256, True, 100),
    ([300, 3, 0], [7, 7, 7], 2, 2, 64, 32, False, 5),
    ([2500, 700], [9, 2], 4, 2, 256, 64, True, 0),
]
MANY = [
    ([700, 513, 40], [5, 3, 40], 8, 2, 64, 64, True, 0),
    ([400, 257], [100, 100], 8, 2, 128, 16, False, 60),
    ([3000], [300], 7, 1, 128, 128, True, 0),
    ([20000, 900], [5, 5], 4, 1, 64, 256, True, 0),
    ([130, 0, 260], [2, 0, 130], 6, 2, 128, 32, True, 0),
]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window", FEW)
def test_few_rows(checked_lib, lens, new, Hq, H, d, page, causal, window, io):
    c = R.Cache(lens, H, page, d, new=new, head_scale=d == 64, seed=70 + d)
    check(c, queries(c.tokens, Hq, d, io, "thd", 71), causal, window)
    clean(checked_lib)


@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window", MANY)
def test_many_rows(checked_lib, lens, new, Hq, H, d, page, causal, window):
    c = R.Cache(lens, H, page, d, new=new, head_scale=d == 64, seed=72 + d)
    check(c, queries(c.tokens, Hq, d, torch.bfloat16, "htd", 73), causal, window)
    clean(checked_lib)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_append_and_read(checked_lib, io):
    new, lens, d = [3, 0, 17], [40, 5, 17], 64
    c = R.Cache(lens, 2, 16, d, new=new, seed=74)
    k = queries(20, 2, d, io, "thd", 75)
    cos, sin = gdn.gdn_rope_table(64, d)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    at = (c.pages, c.table_t, c.len_t)
    gdn.gdn_kv_append(c.pages, k, k, *at[1:], cu_seqlens=c.cu, cos=cos, sin=sin, pos=pos, check=True)
    got = gdn.gdn_kv_read(*at, 20, d, cu_seqlens=c.cu, dtype=io, check=True)
    clean(checked_lib)
    gdn._lib = None
    try:
        want = gdn.gdn_kv_read(*at, 20, d, cu_seqlens=c.cu, dtype=io, check=True)
    finally:
        gdn._lib = checked_lib
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_page_outside_the_pool_is_no_access(checked_lib):
    # the host's mistake is reported as ever, and no check fails behind it
    for new, Hq in (([1, 1], 4), ([9, 9], 8)):
        c = R.Cache([140, 20], 2, 16, 64, new=new, seed=76)
        table = c.table_t.clone()
        table[0, 3] = c.pages.shape[0]
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_kv_attn(queries(c.tokens, Hq, 64, torch.bfloat16, "thd", 77), c.pages, table, c.len_t,
                            check=True)
        assert e.value.status == gdn.GDN_ERR_INVALID_ARG
        clean(checked_lib)
