"""Host-side refusals of the 8-bit cache's entry points and of their binding (CPU): they answer before
any CUDA call, so made-up device addresses are fine."""
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import attention as A
from tests.test_attention_abi import FAKE, kv, lib, ref, rotary, rows  # noqa: F401
from tests.test_attention_devices import On, bf, i32


def test_page_bytes(lib):  # noqa: F811
    assert gdn.gdn_kv8_page_bytes(64, 128) == 64 * 256 + 16
    assert gdn.gdn_kv8_page_bytes(16, 64) == 16 * 128 + 16
    assert gdn.gdn_kv8_page_bytes(128, 64) == 128 * 128 + 16
    assert gdn.gdn_kv8_page_bytes(256, 256) == 256 * 512 + 32
    for page, d in ((48, 128), (8, 128), (512, 128), (0, 64), (64, 96), (64, 512), (-16, 64)):
        assert gdn.gdn_kv8_page_bytes(page, d) == 0
    for page in (16, 32, 64, 128, 256):
        for d in (64, 128, 256):
            size = gdn.gdn_kv8_page_bytes(page, d)
            assert size % 16 == 0 and A._page_size8(size, d) == page
            for wrong in (size + 16, size - 16, size - 1, size + 2 * d // 2):
                assert A._page_size8(wrong, d) == 0
    assert A._page_size8(0, 64) == 0 and A._page_size8(16, 64) == 0 and A._page_size8(2064, 0) == 0


def test_refusals(lib):  # noqa: F811
    bad, un, al = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_ALIGNMENT

    def append(c=kv(), k=rows(2), v=rows(2), q=None, qo=None, rot=None, dt=1):
        return lib.gdn_kv8_append(ref(c), ref(k), ref(v), ref(q), ref(qo), ref(rot), dt, None)

    def read(c=kv(), k=rows(2), v=rows(2), dt=1):
        return lib.gdn_kv8_read(ref(c), ref(k), ref(v), dt, None)

    def attn(c=kv(), q=rows(4), o=rows(4), max_len=9, max_new=1, window=0, flags=1, dt=1, lse=None):
        return lib.gdn_kv8_attn(ref(c), ref(q), ref(o), lse, max_len, max_new, 1.0, window, flags,
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
        for n in (2 ** 31 - 1, 2 ** 31 - 255):
            assert f(kv(n_tokens=n, N=1, heads=2)) == un
    for f in (append, read):
        assert f(k=None) == bad and f(v=rows(3)) == bad and f(k=rows(2, tok=132)) == al
    assert append(q=rows(4)) == bad and append(q=rows(4), qo=rows(5)) == bad
    assert append(rot=rotary(d_rot=48)) == un                    # halves of 24: a block lies across
    assert append(rot=rotary(flags=2)) == bad                    # turns forward only
    assert attn(q=rows(3), o=rows(3)) == bad                     # not a multiple of the heads
    assert attn(o=rows(2)) == bad and attn(flags=2) == bad and attn(window=-1) == bad
    assert attn(max_len=-1) == bad and attn(max_new=-1) == bad and attn(lse=FAKE + 1) == al


def cache(m, **more):
    x = dict(pages=torch.zeros(5, 2, 16 * 128 + 16, dtype=torch.uint8),
             table=torch.zeros(2, 3, dtype=i32), length=torch.zeros(2, dtype=i32),
             cu=torch.zeros(3, dtype=i32), scale=torch.zeros(2, 2), **more)
    return {n: m(n, t) for n, t in x.items()}


def append(m):
    x = cache(m, k=torch.zeros(4, 2, 64, dtype=bf), v=torch.zeros(4, 2, 64, dtype=bf),
              q=torch.zeros(4, 4, 64, dtype=bf), out=torch.zeros(4, 4, 64, dtype=bf),
              cos=torch.zeros(8, 32), sin=torch.zeros(8, 32), pos=torch.zeros(4, dtype=i32))
    return list(x), lambda: gdn.gdn_kv8_append(
        x["pages"], x["k"], x["v"], x["table"], x["length"], q=x["q"], cu_seqlens=x["cu"],
        kv_scale=x["scale"], cos=x["cos"], sin=x["sin"], pos=x["pos"], out=x["out"])


def read(m):
    x = cache(m, k=torch.zeros(4, 2, 64, dtype=bf), v=torch.zeros(4, 2, 64, dtype=bf))
    return list(x), lambda: gdn.gdn_kv8_read(x["pages"], x["table"], x["length"], 4, 64,
                                             cu_seqlens=x["cu"], kv_scale=x["scale"],
                                             out=(x["k"], x["v"]))


def attn(m):
    x = cache(m, q=torch.zeros(4, 4, 64, dtype=bf), out=torch.zeros(4, 4, 64, dtype=bf))
    return list(x), lambda: gdn.gdn_kv8_attn(x["q"], x["pages"], x["table"], x["length"],
                                             cu_seqlens=x["cu"], kv_scale=x["scale"], out=x["out"])


@pytest.mark.parametrize("make", [append, read, attn])
def test_tensors_of_a_call_share_a_device(make, monkeypatch):
    calls = []
    monkeypatch.setattr(A, "_call", lambda *a: calls.append(a))
    names, call = make(lambda n, t: On(t, 3))
    call()
    assert len(calls) == 1 and calls[0][1] == "gdn_kv8_" + make.__name__
    for other in names:
        for at in (0, -1):
            _, call = make(lambda n, t: On(t, at if n == other else 3))
            with pytest.raises(ValueError):
                call()
    assert len(calls) == 1


def test_a_cache_in_4_bits_is_refused(monkeypatch):
    monkeypatch.setattr(A, "_call", lambda *a: pytest.fail("called"))
    for make in (append, read, attn):
        # (pages of 16 rows of 64 in 4 bits)
        _, call = make(lambda n, t: On(torch.zeros(5, 2, 16 * 72, dtype=torch.uint8) if n == "pages" else t, 0))
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        gdn.gdn_kv8_pages(1, 1, 24, 64)
