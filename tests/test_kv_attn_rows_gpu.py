"""gdn_kv_attn where rows, tiles and pieces meet: on both sides of the row count that goes to
tcgen05 products, several row tiles, pieces cut over the CTAs, pools past 32 bits, repeats."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests import gpu_util as U
from tests.test_kv_attn_gpu import check, queries, run

pytestmark = pytest.mark.gpu

# lens, new, Hq, H, d, page, causal, window, head scales, layout
CASES = [
    ([700, 95, 8], [4, 4, 4], 8, 2, 128, 64, True, 0, True, "thd"),       # 16 rows of a head
    ([700, 95, 8], [5, 5, 5], 8, 2, 128, 64, True, 0, True, "thd"),       # 20
    ([700, 95, 8], [1, 17, 0], 2, 2, 64, 16, True, 0, False, "htd"),      # 1 to 17, planned as 17
    ([3000], [300], 7, 1, 128, 16, True, 0, False, "thd"),                # nine row tiles
    ([300, 1, 64, 65, 127, 128, 129], [300, 1, 64, 65, 127, 128, 129], 6, 2, 64, 256, True, 0, True,
     "thd"),                                                              # prompts from nothing
    ([900, 400], [130, 257], 3, 3, 64, 32, True, 1, False, "thd"),        # each sees itself only
    ([900, 400], [130, 257], 4, 2, 128, 128, False, 129, True, "htd"),
    ([20000, 900], [5, 5], 4, 1, 64, 64, True, 0, False, "thd"),          # one cut over many CTAs
    ([20000, 900], [5, 5], 4, 1, 64, 64, True, 4097, False, "thd"),
    ([2500, 700], [9, 2], 4, 2, 256, 64, True, 0, True, "thd"),           # several passes of 8 rows
]


@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window,head_scale,layout", CASES)
def test_rows_and_tiles(lens, new, Hq, H, d, page, causal, window, head_scale, layout):
    c = R.Cache(lens, H, page, d, new=new, head_scale=head_scale, seed=100 + len(lens) + d)
    check(c, queries(c.tokens, Hq, d, torch.bfloat16, layout, d + page), causal, window)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("most", [2, 9])
def test_many_short_sequences(most, io):
    # pieces of one tile and of none, several of them in every CTA
    rng = np.random.default_rng(most)
    lens = [int(x) for x in rng.integers(0, 400, 300)]
    new = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, most + 1, 300))]
    c = R.Cache(lens, 2, 16, 64, new=new, seed=20)
    check(c, queries(c.tokens, 8, 64, io, "thd", 21))


@pytest.mark.parametrize("new", [1, 12])
def test_pool_past_32_bits(new):
    # pages whose offset in the pool needs 33 bits
    H, page, d = 2, 64, 128
    c = R.Cache([1000, 77], H, page, d, new=[new, new], seed=22)
    q = queries(2 * new, 8, d, torch.bfloat16, "thd", 23)
    want, lse = run(c, q)
    far = (1 << 32) // (H * gdn.gdn_kv_page_bytes(page, d)) + 1
    pool = torch.empty(far + c.pages.shape[0], *c.pages.shape[1:], dtype=torch.uint8, device="cuda")
    pool[far:] = c.pages
    table = torch.where(c.table_t >= 0, c.table_t + far, c.table_t)
    o, l2 = gdn.gdn_kv_attn(q, pool, table, c.len_t, return_lse=True, check=True)
    assert torch.equal(o, want) and torch.equal(l2, lse)


@pytest.mark.parametrize("new,H,d", [(1, 8, 128), (2, 4, 256), (40, 2, 128), (300, 1, 64)])
def test_same_bits_again(new, H, d):
    # pieces of a cut are added in one order, whichever CTA ends first
    c = R.Cache([6000, 900, 2500], H, 64, d, new=[new] * 3, seed=24)
    q = queries(3 * new, 4 * H, d, torch.bfloat16, "thd", 25)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    want, lse = run(c, q)
    for _ in range(4):
        flush.zero_()
        o, l2 = run(c, q)
        assert torch.equal(o, want) and torch.equal(l2, lse)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 24])
def test_rows_do_not_depend_on_the_batch(new, io):
    # a sequence alone and among others, to the rounding of another division into pieces
    lens = [1500, 333, 4000]
    c = R.Cache(lens, 2, 32, 128, new=[new] * 3, seed=26)
    q = queries(3 * new, 4, 128, io, "thd", 27)
    whole, _ = run(c, q)
    for b in range(3):
        sl = slice(b * new, (b + 1) * new)
        one = gdn.gdn_kv_attn(q[sl], c.pages, c.table_t[b:b + 1], c.len_t[b:b + 1], check=True)
        k, v = R.cached(c.np_pages, c.table[b], lens[b], 2, 32, 128)
        ref = R.attention(U.f64(q[sl]), k, v, lens[b], 128 ** -0.5, True, 0)
        assert np.all(np.abs(U.f64(one) - U.f64(whole[sl])) <= 2 * R.tolerance(ref, io))
