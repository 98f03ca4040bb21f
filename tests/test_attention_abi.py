"""Host-side refusals of the attention layer's entry points (CPU): they answer
before any CUDA call, so made-up device addresses are fine."""
import ctypes

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import _build
from gated_deltanet_recurrence_gdn_gb300 import attention as A

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def rows(heads=4, data=FAKE, tok=512, head=128, seq=0):
    return A._Rows(data, seq, head, tok, heads)


def rotary(**kw):
    x = dict(cos=FAKE, sin=FAKE, pos=FAKE, axes=None, stride_axis=0, stride_seq=0, table_len=8,
             d_rot=128, n_axes=1, flags=0)
    x.update(kw)
    return A._Rotary(*x.values())


def kv(**kw):
    x = dict(pages=FAKE, head_scale=None, page_table=FAKE, kv_len=FAKE, cu_seqlens=None, n_pages=4,
             page_size=64, heads=2, d=128, N=2, max_pages=3, n_tokens=2, table_stride=3)
    x.update(kw)
    return A._Kv(*x.values())


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_page_bytes(lib):
    assert gdn.gdn_kv_page_bytes(64, 128) == 64 * 144
    assert gdn.gdn_kv_page_bytes(16, 64) == 16 * 72
    for page, d in ((48, 128), (8, 128), (512, 128), (0, 64), (64, 96), (64, 512), (-16, 64)):
        assert gdn.gdn_kv_page_bytes(page, d) == 0


def test_rope_refusals(lib):
    def f(q=rows(), qo=rows(), k=None, ko=None, B=1, T=2, d=128, rot=rotary(), dt=1):
        return lib.gdn_rope(ref(q), ref(qo), ref(k), ref(ko), B, T, d, ref(rot), dt, None)

    bad, un, al = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_ALIGNMENT
    assert f(T=0) == gdn.GDN_OK and f(B=0) == gdn.GDN_OK
    assert f(B=-1) == bad and f(dt=3) == bad and f(rot=None) == bad and f(q=None) == bad
    assert f(k=rows()) == bad                                  # no place for its result
    assert f(qo=rows(heads=5)) == bad and f(q=rows(data=None)) == bad and f(q=rows(heads=0)) == bad
    assert f(d=120) == un and f(d=272) == un and f(d=0) == un
    assert f(q=rows(data=FAKE + 8)) == al and f(q=rows(tok=516)) == al and f(q=rows(head=4)) == al
    assert f(q=rows(tok=516), dt=0, B=0) == gdn.GDN_OK
    assert f(rot=rotary(d_rot=24)) == un and f(rot=rotary(d_rot=144)) == bad
    assert f(rot=rotary(n_axes=0)) == bad and f(rot=rotary(n_axes=5)) == un
    assert f(rot=rotary(flags=4)) == bad and f(rot=rotary(cos=None)) == bad
    assert f(rot=rotary(table_len=0)) == bad and f(rot=rotary(pos=FAKE + 2)) == al
    assert f(rot=rotary(axes=bytes([0] * 63 + [2]), n_axes=2)) == bad
    assert f(rot=rotary(sin=FAKE + 4)) == al


def test_cache_refusals(lib):
    bad, un, al = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_ALIGNMENT

    def append(c=kv(), k=rows(2), v=rows(2), q=None, qo=None, rot=None, dt=1):
        return lib.gdn_kv_append(ref(c), ref(k), ref(v), ref(q), ref(qo), ref(rot), dt, None)

    def read(c=kv(), k=rows(2), v=rows(2), dt=1):
        return lib.gdn_kv_read(ref(c), ref(k), ref(v), dt, None)

    def attn(c=kv(), q=rows(4), o=rows(4), max_len=9, max_new=1, window=0, flags=1, dt=1, lse=None):
        return lib.gdn_kv_attn(ref(c), ref(q), ref(o), lse, max_len, max_new, 1.0, window, flags,
                               dt, None)

    for f in (append, read, attn):
        assert f(kv(n_tokens=0)) == gdn.GDN_OK
        assert f(None) == bad and f(kv(N=-1)) == bad and f(kv(n_tokens=-1)) == bad
        assert f(kv(N=0)) == bad and f(kv(n_tokens=3)) == bad   # not the same number each
        assert f(kv(pages=None)) == bad and f(kv(kv_len=None)) == bad and f(kv(page_table=None)) == bad
        assert f(kv(n_pages=0)) == bad and f(kv(max_pages=0)) == bad and f(kv(heads=0)) == bad
        assert f(kv(page_size=48)) == un and f(kv(d=96)) == un and f(kv(max_pages=1 << 26)) == un
        assert f(kv(pages=FAKE + 8)) == al and f(kv(kv_len=FAKE + 2)) == al
        assert f(dt=7) == bad
    for f in (append, read):
        assert f(k=None) == bad and f(v=rows(3)) == bad and f(k=rows(2, tok=132)) == al
    assert append(q=rows(4)) == bad and append(q=rows(4), qo=rows(5)) == bad
    assert append(rot=rotary(d_rot=48)) == un                    # halves of 24: a block lies across
    assert append(rot=rotary(flags=2)) == bad                    # turns forward only
    assert attn(q=rows(3), o=rows(3)) == bad                     # not a multiple of the heads
    assert attn(o=rows(2)) == bad and attn(flags=2) == bad and attn(window=-1) == bad
    assert attn(max_len=-1) == bad and attn(max_new=-1) == bad and attn(lse=FAKE + 1) == al


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    x = torch.zeros(2, 2, 64)
    pages = torch.zeros(1, 2, 16 * 72, dtype=torch.uint8)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append(pages, x, x, i, i[:, 0])
    with pytest.raises(ValueError):
        gdn.gdn_kv_attn(x, pages, i, i[:, 0])
    with pytest.raises(ValueError):
        gdn.gdn_rope(x[None], None, x[0], x[0], i[0])
    with pytest.raises(ValueError):
        gdn.gdn_kv_pages(1, 1, 24, 64)


def test_rope_axes():
    assert gdn.gdn_rope_axes((2, 3, 1)) == bytes([0, 0, 1, 1, 1, 2])
    assert gdn.gdn_rope_axes((2, 3, 1), interleave=True) == bytes([0, 1, 2, 0, 1, 1])
