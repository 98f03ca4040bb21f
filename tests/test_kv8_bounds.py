"""The 8-bit cache in the debug bounds-check build (csrc/gdn_check.cuh): its unit compiles there, and
small cases of append, read and both attention kernels, every width and type, match the fp64
definition with no check failed."""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import _build
from tests import attention8_ref as R8


@pytest.mark.skipif(shutil.which(_build.NVCC) is None, reason="nvcc not available")
def test_unit_compiles_with_checks():
    with tempfile.TemporaryDirectory() as tmp:
        cmd = [_build.NVCC] + _build._flags() + _build.VARIANTS["check"] + [
            "-c", os.path.join(_build.CSRC, "gdn_kv8.cu"), "-o", os.path.join(tmp, "kv8.o")]
        r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


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


# lens, new, Hq, H, d, page, causal, window
CASES = [
    ([0, 1, 15, 16, 17, 255, 256, 300], [1] * 8, 8, 2, 128, 64, True, 0),
    ([5000, 77], [1, 1], 4, 2, 64, 16, True, 0),
    ([700, 513, 40], [5, 5, 5], 4, 2, 128, 256, True, 100),
    ([300, 3, 0], [7, 7, 7], 2, 2, 64, 32, False, 5),
    ([2500, 700], [9, 2], 4, 2, 256, 64, True, 0),
    ([700, 513, 40], [5, 3, 40], 8, 2, 64, 256, True, 0),
    ([400, 257], [100, 100], 8, 2, 128, 16, False, 60),
    ([3000], [300], 7, 1, 128, 128, True, 0),
    ([130, 0, 260], [2, 0, 130], 6, 2, 128, 32, True, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window", CASES)
def test_attention(checked_lib, lens, new, Hq, H, d, page, causal, window, io):
    from tests.test_kv8_attn_gpu import check, queries
    c = R8.Cache8(lens, H, page, d, new=new, head_scale=d == 64, seed=70 + d)
    check(c, queries(c.tokens, Hq, d, io, "thd", 71), causal, window)
    clean(checked_lib)


@pytest.mark.gpu
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 256), (256, 64)])
def test_append_and_read(checked_lib, d, page, io):
    from tests.test_kv8_attn_gpu import queries
    new, lens = [3, 0, 17], [40, 5, 17]
    c = R8.Cache8(lens, 2, page, d, new=new, seed=74)
    k = queries(20, 2, d, io, "thd", 75)
    cos, sin = gdn.gdn_rope_table(64, d)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    at = (c.pages, c.table_t, c.len_t)
    gdn.gdn_kv8_append(c.pages, k, k, *at[1:], q=k, cu_seqlens=c.cu, cos=cos, sin=sin, pos=pos,
                       check=True)
    got = gdn.gdn_kv8_read(*at, 20, d, cu_seqlens=c.cu, dtype=io, check=True)
    clean(checked_lib)
    gdn._lib = None
    try:
        want = gdn.gdn_kv8_read(*at, 20, d, cu_seqlens=c.cu, dtype=io, check=True)
    finally:
        gdn._lib = checked_lib
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_a_page_outside_the_pool_is_no_access(checked_lib):
    from tests.test_kv8_attn_gpu import queries
    for new, Hq in (([1, 1], 4), ([9, 9], 8)):
        c = R8.Cache8([140, 20], 2, 16, 64, new=new, seed=76)
        table = c.table_t.clone()
        table[0, 8] = c.pages.shape[0]
        q = queries(c.tokens, Hq, 64, torch.bfloat16, "thd", 77)
        for call in (lambda: gdn.gdn_kv8_attn(q, c.pages, table, c.len_t, check=True),
                     lambda: gdn.gdn_kv8_append(c.pages, q[:, :2], q[:, 2:4], table, c.len_t, check=True)):
            with pytest.raises(gdn.GdnError) as e:
                call()
            assert e.value.status == gdn.GDN_ERR_INVALID_ARG
            clean(checked_lib)


@pytest.mark.gpu
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [10, 20])
def test_attention_of_several_eights_of_rows(checked_lib, new, d, io):
    from tests.test_kv8_attn_gpu import check, queries
    c = R8.Cache8([1800, 0, 1025, 7], 2, 32, d, new=[new] * 4, seed=78)
    check(c, queries(c.tokens, 2, d, io, "thd", 79))
    clean(checked_lib)
