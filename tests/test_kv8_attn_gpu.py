"""gdn_kv8_attn against the fp64 definition: head layouts, lengths, masks that leave rows empty,
garbage where nothing is seen, exponents at both ends, and the refusals.  Tolerances are
attention_ref's: e4m3 * 2^(e - 15) enters the products exactly, as the 4-bit cache's numbers do."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention8_ref as R8
from tests import attention_ref as R
from tests import gpu_util as U
from tests.test_kv_attn_gpu import DT, queries
from tests.test_kv_attn_gpu import CASES as CASES4

pytestmark = pytest.mark.gpu


def run(c, q, causal=True, window=0, scale=None, **kw):
    uniform = min(c.new) == max(c.new)
    return gdn.gdn_kv8_attn(q, c.pages, c.table_t, c.len_t, cu_seqlens=None if uniform else c.cu,
                            kv_scale=c.scale_t, causal=causal, window=window, scale=scale,
                            return_lse=True, check=True, **kw)


def lost(c, q):
    """What the kernel for many rows may lose beyond attention_ref.tolerance: the largest weight of a
    row is at least 2^8 as it is held in fp16, whose least step is 2^-24, so a weight is off by
    2^-25 / 2^8 of the largest, and with the largest at most 1 the result by 2^-33 of the sum of
    the values' magnitudes.  (It shows where the largest weights meet zeros.)"""
    out = np.zeros(q.shape)
    if q.dtype != torch.bfloat16 or c.d > 128 or max(c.new) * q.shape[1] // c.H <= 16:
        return out
    for b, n in enumerate(c.lens):
        _, v = R8.cached(c.np_pages, c.table[b], n, c.H, c.page_size, c.d,
                         None if c.scale is None else c.scale.astype(np.float64))
        out[c.at[b]:c.at[b + 1]] = np.repeat(np.abs(v).sum(1), q.shape[1] // c.H, 0) * 2.0 ** -33
    return out


def check(c, q, causal=True, window=0, scale=None, **kw):
    o, lse = run(c, q, causal, window, scale, **kw)
    assert o.dtype == q.dtype and o.shape == q.shape
    ref = c.reference(U.f64(q), c.d ** -0.5 if scale is None else scale, causal, window)
    o, lse = U.f64(o), U.f64(lse)
    assert np.all(np.abs(o - ref[0]) <= R.tolerance(ref, q.dtype) + lost(c, q))
    empty = np.isneginf(ref[1])
    assert np.array_equal(empty, np.isneginf(lse))
    # the score's error, and the sum's and its logarithm's roundings
    tol = 2.0 ** -20 * (4 + ref[3] + np.abs(ref[1], where=~empty, out=np.zeros_like(ref[1])))
    assert np.all(np.abs(np.where(empty, 0, lse) - np.where(empty, 0, ref[1])) <= tol)
    return o


MORE = [
    # pages of 256 in tiles of 256 and of 128, their second exponents' group
    ([255, 256, 257, 640], [1] * 4, 8, 2, 64, 256, True, 0, True, "thd", "bf16"),
    ([255, 256, 257, 640], [3] * 4, 8, 2, 128, 256, True, 0, True, "thd", "f32"),
    ([255, 256, 257, 640], [30] * 4, 8, 2, 128, 256, True, 0, False, "htd", "bf16"),
    ([333, 129], [40, 7], 4, 2, 64, 16, True, 33, False, "thd", "bf16"),
]


@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window,head_scale,layout,io", CASES4 + MORE)
def test_matches_definition(lens, new, Hq, H, d, page, causal, window, head_scale, layout, io):
    c = R8.Cache8(lens, H, page, d, new=new, head_scale=head_scale, seed=len(lens) + d)
    check(c, queries(c.tokens, Hq, d, DT[io], layout, d + page), causal, window)


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_long_sequences_cut_over_the_gpu(io, new):
    c = R8.Cache8([9000, 17, 0, 20011], 1, 64, 64, new=[new] * 4, seed=5)
    q = queries(4 * new, 4, 64, DT[io], "thd", 1)
    check(c, q)
    # a tighter bound on the length plans another division
    check(c, q, max_len=20011, max_new=new)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_sequences(io):
    # more sequences than a CTA has threads to share them out
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    c = R8.Cache8(lens, 1, 16, 64, seed=6)
    check(c, queries(700, 2, 64, DT[io], "thd", 2))


@pytest.mark.parametrize("size", [1e-30, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_query_magnitudes(io, new, size):
    c = R8.Cache8([333, 70], 2, 32, 64, new=[new] * 2, seed=7)
    check(c, queries(2 * new, 4, 64, DT[io], "thd", 3, size), scale=0.125 / max(size, 1.0) * 4)


@pytest.mark.parametrize("exponents", [(0, 0), (0, 3), (20, 22), (0, 22)])
@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_exponents_at_both_ends(d, io, new, exponents):
    # down to 2^-24 and up to 57344: both ends of fp16
    c = R8.Cache8([333, 70], 2, 32, d, new=[new] * 2, seed=8, exponents=exponents)
    check(c, queries(2 * new, 4, d, DT[io], "thd", 4), scale=2.0 ** (8 - exponents[1]) / d)


def test_scale_sign_and_zero():
    c = R8.Cache8([333, 70], 2, 32, 64, seed=8)
    for scale in (-0.3, 0.0, 2.0):
        check(c, queries(2, 4, 64, torch.float32, "thd", 4), scale=scale)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_growing_scores_raise_the_maximum(io, new):
    # keys that grow along the sequence: the running maximum moves in every step
    d, page = 64, 16
    c = R8.Cache8([352], 1, page, d, new=[new], seed=9)
    for p in range(22):
        c.np_pages[c.table[0, p], 0, :page * d] = 0x38                        # every element 1 ...
        c.np_pages[c.table[0, p], 0, R8.exponent_at(page, d, 0, 0)] = p       # ... times 2^(p - 15)
    c.upload()
    q = torch.ones(new, 2, d, dtype=DT[io], device="cuda")
    check(c, q, scale=0.01)
    check(c, -q, scale=0.01)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,new", [(128, 64, 24), (64, 16, 24), (256, 32, 24), (128, 64, 300)])
def test_nan_reaches_only_the_rows_that_see_it(d, page, new, io):
    L = new + 200
    c = R8.Cache8([L], 1, page, d, new=[new], seed=10)
    q = queries(new, 2, d, DT[io], "thd", 5)
    clean, _ = run(c, q, window=150)
    where = L - new // 2                                      # half of the rows see this place
    blk, row = c.table[0, where // page], where % page
    at = (page + row) * d + 16
    # a NaN in 16 neighbours of the value, as the append leaves it: those dimensions of the rows
    # that see it
    kept = c.np_pages[blk, 0, at:at + 16].copy()
    c.np_pages[blk, 0, at:at + 16] = 0x7F
    c.upload()
    o, _ = run(c, q, window=150)
    bad = torch.zeros_like(o, dtype=torch.bool)
    first = where - (L - new)
    bad[first:min(new, first + 150), :, 16:32] = True
    assert torch.equal(o.isnan(), bad)
    assert torch.equal(o[~bad], clean[~bad])
    # in one element: within its 16 neighbours, its own at least
    c.np_pages[blk, 0, at:at + 16] = kept
    c.np_pages[blk, 0, at + 5] = 0xFF
    c.upload()
    o, _ = run(c, q, window=150)
    assert not o[~bad].isnan().any() and torch.equal(o[~bad], clean[~bad])
    assert o[first:min(new, first + 150), :, 21].isnan().all()
    # a NaN in the key: all of those rows
    c.np_pages[blk, 0, at + 5] = kept[5]
    c.np_pages[blk, 0, row * d + 40] = 0xFF
    c.upload()
    o, _ = run(c, q, window=150)
    bad[first:min(new, first + 150)] = True
    assert torch.equal(o.isnan(), bad)
    assert torch.equal(o[~bad], clean[~bad])


@pytest.mark.parametrize("new", [3, 24, 300])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_rows_of_nonfinite_queries_are_nan(io, d, new):
    c = R8.Cache8([300 + new], 2, 64, d, new=[new], seed=80)
    q = queries(new, 4, d, io, "thd", 81)
    clean, clean_lse = run(c, q)
    q[1, 2, 7] = float("inf")           # (infinities of both signs among the products)
    q[1, 2, 8] = float("-inf")
    q[2, 0, 9] = float("nan")
    bad = torch.zeros(new, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    o, lse = run(c, q)
    assert o[2, 0].isnan().all() and o[1, 2].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(o[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, sys.maxsize])
@pytest.mark.parametrize("lens,new", [([300, 3, 0], 7), ([3, 150], 40), ([300, 1], 4)])
def test_window_as_large_as_can_be(lens, new, window, causal, io):
    c = R8.Cache8(lens, 1, 16, 64, new=[new] * len(lens), seed=40 + new)
    q = queries(c.tokens, 2, 64, io, "thd", 41)
    o = check(c, q, causal, window)
    assert (o == check(c, q, causal, 0)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_nan_at_the_end_of_pieces_with_one_and_two_row_tiles(d):
    page, B = 64, 301
    new = [100 if b % 2 == 0 else 10 for b in range(B)]
    lens = [150 + (37 * b) % 700 for b in range(B)]
    c = R8.Cache8(lens, 1, page, d, new=new, seed=42)
    q = queries(c.tokens, 2, d, torch.bfloat16, "thd", 43)
    clean, _ = run(c, q)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    for b in range(0, B, 3):
        back = 1 + b % 5                                       # places before the end
        where = lens[b] - back
        row, block = where % page, b % (d // 16)
        at = (page + row) * d + 16 * block
        c.np_pages[c.table[b, where // page], 0, at:at + 16] = 0x7F
        bad[c.at[b + 1] - back:c.at[b + 1], :, 16 * block:16 * block + 16] = True
    c.upload()
    for _ in range(3):
        o, _ = run(c, q)
        assert torch.equal(o.isnan(), bad)
        assert torch.equal(o[~bad], clean[~bad])


@pytest.mark.parametrize("heads", [8, 64])
def test_same_bits_again_on_another_stream_and_in_a_graph(heads):
    c = R8.Cache8([5000, 77, 1234], 2, 64, 128, seed=12)
    q = queries(3, heads, 128, torch.bfloat16, "thd", 7)
    a, la = run(c, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = torch.zeros_like(q)
        for _ in range(20):
            x.add_(0)
        x.copy_(q)
        b, lb = gdn.gdn_kv8_attn(x, c.pages, c.table_t, c.len_t, return_lse=True)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv8_attn(q, c.pages, c.table_t, c.len_t, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)


def test_table_rows_apart_and_views():
    c = R8.Cache8([200, 90], 2, 64, 128, seed=14)
    q = queries(2, 4, 128, torch.bfloat16, "thd", 9)
    want, _ = run(c, q)
    wide = torch.full((2, 9), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table_t.shape[1]] = c.table_t
    lens = torch.cat([c.len_t[:1] * 0 - 5, c.len_t, c.len_t[:1] * 0 - 5])
    fused = torch.full((2, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:6] = q
    got = gdn.gdn_kv8_attn(fused[:, 2:6], c.pages, wide[:, 2:2 + c.table_t.shape[1]], lens[1:3],
                           check=True)
    assert torch.equal(want, got)


@pytest.mark.parametrize("what", ["page", "len", "max_len", "max_new"])
def test_bad_indices_are_reported(what):
    c = R8.Cache8([140, 20], 2, 16, 64, new=[3, 2], seed=15)
    q = queries(5, 4, 64, torch.bfloat16, "thd", 10)
    table, length, kw = c.table_t.clone(), c.len_t.clone(), {}
    if what == "page":
        table[0, 3] = -1
    elif what == "len":
        length[0] = -1
    elif what == "max_len":
        kw["max_len"] = 139
    else:
        kw["max_new"] = 2
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_kv8_attn(q, c.pages, table, length, cu_seqlens=c.cu, check=True, **kw)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()


def test_nothing_to_do():
    c = R8.Cache8([40], 2, 16, 64, new=[0], seed=16)
    q = queries(0, 4, 64, torch.bfloat16, "thd", 11)
    assert run(c, q)[0].shape == q.shape


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("limit", [1, 8])
def test_short_limits_end_in_a_status(limit, io):
    # whether or not a wait runs out at so few polls, the call ends, says so, and the next one
    # is right
    c = R8.Cache8([9000, 77, 0, 4000, 12001], 2, 16, 64, seed=62)
    q = queries(5, 8, 64, io, "thd", 63)
    want = check(c, q)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    prev = gdn.get_option(gdn.GDN_OPT_WAIT_LIMIT)
    gdn.set_option(gdn.GDN_OPT_WAIT_LIMIT, limit)
    try:
        for _ in range(5):
            flush.zero_()
            o = gdn.gdn_kv8_attn(q, c.pages, c.table_t, c.len_t)
            s = gdn.load().gdn_sync_check(gdn._stream(None))
            assert s in (gdn.GDN_OK, gdn.GDN_ERR_DEVICE_TIMEOUT)
            if s == gdn.GDN_OK:
                assert (o.double().cpu().numpy() == want).all()
    finally:
        gdn.set_option(gdn.GDN_OPT_WAIT_LIMIT, prev)
    assert (check(c, q) == want).all()


def test_the_append_and_the_attention_agree():
    """Prompts appended and attended to, against attention over the rows themselves: what differs is
    the cache's rounding, half a step of e4m3 each, 2^-4 of an element (or 2^-10 of the block's
    scale, whose largest element is above half of 448): of keys the scores, of values the result."""
    H, d, page, new = 2, 128, 32, [70, 33]
    n = sum(new)
    k, v, q = (queries(n, h, d, torch.float32, "thd", i) for i, h in enumerate((H, H, 4)))
    table = torch.tensor([[0, 3, 1], [2, 4, 5]], dtype=torch.int32, device="cuda")
    length = torch.tensor(new, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda")
    pages = gdn.gdn_kv8_pages(6, H, page, d)
    gdn.gdn_kv8_append(pages, k, v, table, length, cu_seqlens=cu)
    o = U.f64(gdn.gdn_kv8_attn(q, pages, table, length, cu_seqlens=cu, check=True))
    k, v, q = U.f64(k), U.f64(v), U.f64(q)
    for a, b in ((0, 70), (70, 103)):
        rows = [np.swapaxes(x[a:b], 0, 1) for x in (k, v)]
        want, _, mass, size = R.attention(q[a:b], *rows, b - a, d ** -0.5, True, 0)
        step = 2.0 ** -4 * np.abs(v[a:b]).max() + 2.0 ** -10
        # weights move by exp(2 * the largest score's error) - 1
        moved = np.expm1(2 * (2.0 ** -4 * size + 2.0 ** -10 * np.abs(q[a:b]).sum(-1) * d ** -0.5))[..., None]
        assert np.all(np.abs(o[a:b] - want) <= step + 2 * moved * (mass + step))
