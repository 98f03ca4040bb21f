"""Host-side checks of the attention layer's entry points at the ends of their sizes (CPU: they answer
before any CUDA call)."""
import pytest

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests.test_attention_abi import kv, lib, ref, rotary, rows  # noqa: F401

un = gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("B,T", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 255), (2 ** 30, 2), (65536, 65536)])
def test_rope_tokens_of_the_last_block_fit_an_int(lib, B, T):  # noqa: F811
    # (d = 80 and 48: a block's 51 or 85 tokens do not divide 2^31)
    for d in (16, 48, 80, 128):
        assert lib.gdn_rope(ref(rows()), ref(rows()), None, None, B, T, d, ref(rotary(d_rot=16)), 1,
                            None) == un


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 255])
def test_cache_tokens_of_the_last_block_fit_an_int(lib, n):  # noqa: F811
    c = kv(n_tokens=n, N=1, heads=2)
    assert lib.gdn_kv_append(ref(c), ref(rows(2)), ref(rows(2)), None, None, None, 1, None) == un
    assert lib.gdn_kv_read(ref(c), ref(rows(2)), ref(rows(2)), 1, None) == un
    assert lib.gdn_kv_attn(ref(c), ref(rows(2)), ref(rows(2)), None, 9, 1, 1.0, 0, 1, 1, None) == un


def test_packed_tokens_have_no_stride_seq(lib):  # noqa: F811
    # (rows of packed tokens ignore it, so it may be anything; what else is wrong is still found)
    al, bad = gdn.GDN_ERR_ALIGNMENT, gdn.GDN_ERR_INVALID_ARG
    r, q3 = rows(2, seq=3), rows(3, seq=3)
    assert lib.gdn_kv_append(ref(kv()), ref(r), ref(r), ref(rows(4, seq=5)), ref(rows(5, seq=7)), None, 1,
                             None) == bad
    assert lib.gdn_kv_read(ref(kv()), ref(r), ref(q3), 1, None) == bad
    assert lib.gdn_kv_attn(ref(kv()), ref(q3), ref(q3), None, 9, 1, 1.0, 0, 1, 1, None) == bad
    assert lib.gdn_kv_read(ref(kv()), ref(rows(2, tok=132, seq=3)), ref(r), 1, None) == al
    assert lib.gdn_rope(ref(r), ref(r), None, None, 1, 2, 128, ref(rotary()), 1, None) == al
