"""gdn_kv8_attn where a key/value head has 9 to 32 rows, or where all its rows go by the kernel for few
(fp32 rows, d = 256): a piece then has one, two or three eights of rows.  Against the fp64 definition,
with test_kv8_attn_gpu's tolerances."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention8_ref as R8
from tests.test_kv8_attn_gpu import check, queries, run

pytestmark = pytest.mark.gpu
IO = [torch.bfloat16, torch.float32]


# sequences on both sides of 1024 places
@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("lens", [[700, 33, 0], [2600, 1025, 3]])
@pytest.mark.parametrize("G,new", [(1, 9), (8, 2), (16, 1), (1, 17), (12, 2), (5, 5), (8, 4)])
def test_matches_definition(G, new, lens, d, page, io):
    c = R8.Cache8(lens, 2, page, d, new=[new] * 3, head_scale=G == 8, seed=G + new)
    check(c, queries(c.tokens, 2 * G, d, io, "thd", d + new))


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 40), (False, 7), (True, 1)])
def test_masks_and_ragged_tokens(causal, window, d, io):
    # rows that see nothing, and eights with no row
    c = R8.Cache8([1500, 0, 20, 1100, 2], 1, 32, d, new=[20, 0, 3, 1, 9], seed=d)
    check(c, queries(c.tokens, 1, d, io, "htd", 90), causal, window, max_new=20)
    c = R8.Cache8([1500, 2, 700], 3, 256, d, new=[6, 5, 4], seed=d + 1)
    check(c, queries(c.tokens, 12, d, io, "thd", 91), causal, window, max_new=6)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [12, 20])
def test_long_sequences_cut_over_the_gpu(new, d, io):
    c = R8.Cache8([9000, 17, 0, 20011], 1, 64, d, new=[new] * 4, seed=5)
    q = queries(4 * new, 1, d, io, "thd", 1)
    check(c, q)
    check(c, q, max_len=20011, max_new=new)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [16, 24])
def test_nan_reaches_only_the_rows_that_see_it(new, d, io):
    page, L = 64, 1300
    c = R8.Cache8([L], 1, page, d, new=[new], seed=10)
    q = queries(new, 1, d, io, "thd", 5)
    clean, _ = run(c, q)
    for back in (1, 8, new - 1):                              # places before the end
        where = L - back
        at = (page + where % page) * d + 32
        blk = c.table[0, where // page]
        kept = c.np_pages[blk, 0, at:at + 16].copy()
        c.np_pages[blk, 0, at:at + 16] = 0x7F
        c.upload()
        o, _ = run(c, q)
        bad = torch.zeros_like(o, dtype=torch.bool)
        bad[new - back:, :, 32:48] = True
        assert torch.equal(o.isnan(), bad)
        assert torch.equal(o[~bad], clean[~bad])
        c.np_pages[blk, 0, at:at + 16] = kept


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [16, 24])
def test_scores_that_grow_and_weights_far_apart(rows, d, io):
    # keys that grow along the sequence (the maximum moves in every step), or shrink (every weight
    # after the first ones is small), in some rows and not in others
    page, n = 16, 1408
    c = R8.Cache8([n], 1, page, d, new=[1], seed=9)
    for p in range(n // page):
        c.np_pages[c.table[0, p], 0, :page * d] = 0x38                             # every element 1 ...
        c.np_pages[c.table[0, p], 0, R8.exponent_at(page, d, 0, 0)] = p // 4       # ... times 2^(p/4 - 15)
    c.upload()
    q = torch.ones(1, rows, d, dtype=io, device="cuda")
    q[:, 1::3] = -1
    q[:, 2::5] = 0.01
    check(c, q, scale=0.02)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("rows", [12, 20])
def test_same_bits_again_and_in_a_graph(rows, io):
    c = R8.Cache8([3000, 1200, 9], 2, 64, 128, seed=11)
    q = queries(3, 2 * rows, 128, io, "thd", 12)
    o, lse = run(c, q)
    out = torch.empty_like(q)
    call = lambda: gdn.gdn_kv8_attn(q, c.pages, c.table_t, c.len_t, out=out, return_lse=True)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, again = call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(again, lse)
