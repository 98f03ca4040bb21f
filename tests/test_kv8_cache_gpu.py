"""gdn_kv8_append and gdn_kv8_read: what the 8-bit cache holds, where it lies, how a block's exponent
grows, and what stays untouched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention8_ref as R8
from tests import attention_ref as R
from tests import gpu_util as U
from tests.test_kv_cache_gpu import DT, tokens

pytestmark = pytest.mark.gpu

CASES = [
    # lens before, new, Hq, H, d, page, rot, axes, adjacent, head scales, layout, io
    ([0, 15, 16, 63, 130], [1, 1, 1, 1, 1], 8, 2, 128, 64, 128, 1, False, False, "thd", "bf16"),
    ([0, 3, 100], [37, 1, 65], 4, 4, 64, 16, 64, 3, False, True, "thd", "f32"),
    ([5, 0, 0, 31], [3, 0, 128, 2], 6, 3, 256, 32, 64, 2, False, True, "htd", "bf16"),
    ([7], [300], 2, 1, 128, 128, 48, 1, True, False, "htd", "f32"),
    ([250, 1], [10, 10], 3, 1, 64, 256, 0, 1, False, False, "thd", "bf16"),
    ([17, 40, 7], [17, 17, 17], 5, 5, 64, 32, 32, 1, False, False, "thd", "f32"),
    ([200, 127, 255], [130, 130, 130], 2, 2, 256, 256, 256, 4, True, True, "thd", "bf16"),
]


@pytest.mark.parametrize("had,new,Hq,H,d,page,rot,axes,adjacent,head_scale,layout,io", CASES)
@pytest.mark.parametrize("exponents", [(3, 9), (14, 20)])
def test_append_and_read(had, new, Hq, H, d, page, rot, axes, adjacent, head_scale, layout, io, exponents):
    """Blocks that had rows under small exponents grow (the tokens are normal numbers of size 1 to
    10, which want 6 to 10), those under large ones stay."""
    dt = DT[io]
    lens = [a + b for a, b in zip(had, new)]
    c = R8.Cache8(lens, H, page, d, new=new, head_scale=head_scale, seed=page, exponents=exponents)
    n = c.tokens
    # what lies at the new places before the call, and exponents of blocks that had no rows, is of no use
    for b in range(len(lens)):
        for p in range(had[b], lens[b]):
            for i in (0, 1):
                r = p % page
                c.np_pages[c.table[b, p // page], :, (i * page + r) * d:(i * page + r + 1) * d] = 0xFF
                if p % 16 == 0:
                    c.np_pages[c.table[b, p // page], :, R8.exponent_at(page, d, i, r)] = 0xFF
    c.upload()
    q, k, v = (tokens(n, h, d, dt, layout, 10 * i + d) for i, h in enumerate((Hq, H, H)))
    rng = np.random.default_rng(d)
    pos = rng.integers(0, 5000, (axes, n)).astype(np.int32)
    which = [i % axes for i in range(rot // 2)]
    kw = {}
    if rot:
        cos, sin = gdn.gdn_rope_table(5000, rot)
        kw = dict(cos=cos, sin=sin, pos=torch.from_numpy(pos).cuda(), axes=which, adjacent=adjacent)
    uniform = min(new) == max(new)
    cu = None if uniform else c.cu
    qo = gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, q=q, cu_seqlens=cu,
                            kv_scale=c.scale_t, check=True, **kw)
    got = c.pages.cpu().numpy()

    def turned(x):
        x = U.f64(x)
        if rot:
            x = np.swapaxes(R.rotate(np.swapaxes(x, 0, 1), U.f64(cos), U.f64(sin), pos, which,
                                     adjacent), 0, 1)
        return x

    # q: two products and a sum in fp32, then dt
    want = turned(q)
    tol = 8 * 2.0 ** -24 * np.abs(U.f64(q)).max(-1, keepdims=True) + (
        np.abs(want) * 2.0 ** -8 if io == "bf16" else 0)
    assert np.all(np.abs(U.f64(qo) - want) <= tol)

    ones = np.ones((2, H))
    gs = ones if c.scale is None else c.scale.astype(np.float64)
    expect = c.np_pages.copy()
    held = [np.zeros((n, H, d)), np.zeros((n, H, d))]
    rows = turned(k), U.f64(v)
    grew = 0
    for b in range(len(lens)):
        for first in range(had[b] // 16 * 16, lens[b], 16):
            lo, hi = max(first, had[b]), min(first + 16, lens[b])
            if lo >= hi:
                continue
            blk, t = c.table[b, first // page], c.at[b] + lo - had[b]
            for i in (0, 1):
                x = rows[i][t:t + hi - lo] / gs[i][:, None]                  # [new, H, d]
                # a turned element is two products and a sum of the row's numbers (8 roundings,
                # doubled), the quotient by the head's scale two more
                off = 16 * 2.0 ** -24 * np.abs(U.f64(k[t:t + hi - lo])).max((0, 2)) / gs[i] if i == 0 else np.zeros(H)
                m = np.abs(x).max((0, 2))
                at = R8.exponent_at(page, d, i, first % page)
                e = got[blk, :, at].astype(np.int64)
                slack = off + 4 * 2.0 ** -24 * m
                had_rows = lo > first
                was = c.np_pages[blk, :, at].astype(np.int64) if had_rows else np.zeros(H, dtype=np.int64)
                low, high = (np.maximum(was, R8.least_exponent(y)) for y in (m - slack, m + slack))
                assert np.all((e == low) | (e == high))
                expect[blk, :, at] = e
                for r in range(first % page, first % page + lo - first):     # rows that were there
                    a = (i * page + r) * d
                    y = c.np_pages[blk, :, a:a + d]
                    code = R8.nearest(R.e4m3(y) * 2.0 ** (was - e)[:, None]) | (y & 128)
                    expect[blk, :, a:a + d] = np.where((e > was)[:, None], code, y)
                    grew += int((e > was).sum())
                for j in range(hi - lo):
                    a = (i * page + first % page + lo - first + j) * d
                    codes = got[blk, :, a:a + d]
                    h = R.e4m3(codes)
                    y = x[j] * 2.0 ** (15.0 - e)[:, None]
                    best = np.abs(R8.GRID[R8.nearest(y)] - np.abs(y))
                    assert np.all(np.abs(h - y) <= best + 2 * (slack * 2.0 ** (15.0 - e))[:, None])
                    held[i][t + j] = h * 2.0 ** (e - 15.0)[:, None] * gs[i][:, None]
                    expect[blk, :, a:a + d] = codes
    assert np.array_equal(got, expect)           # nothing else was written
    if exponents[1] < 10 and any(h % 16 and n for h, n in zip(had, new)):
        assert grew > 0

    rk, rv = gdn.gdn_kv8_read(c.pages, c.table_t, c.len_t, n, d, cu_seqlens=cu, kv_scale=c.scale_t,
                              dtype=dt, check=True)
    for x, y in ((rk, held[0]), (rv, held[1])):
        assert np.all(np.abs(U.f64(x) - y) <= np.abs(y) * (2.0 ** -8 if io == "bf16" else 2.0 ** -23))


def test_tokens_one_by_one_end_in_the_exponents_of_all_at_once():
    """A block's last exponent is that of its largest token, however the tokens came; the codes differ
    by a second rounding at most, a step of the numbers below 2^-6 of the block's scale."""
    H, d, page, L = 2, 64, 32, 45
    k, v = (tokens(L, H, d, torch.float32, "thd", i) for i in (1, 2))
    grow = torch.exp(0.2 * torch.arange(L, device="cuda"))[:, None, None]
    k, v = k * grow, v * grow
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    length = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    whole, steps = gdn.gdn_kv8_pages(2, H, page, d), gdn.gdn_kv8_pages(2, H, page, d)
    gdn.gdn_kv8_append(whole, k, v, table, length(L), check=True)
    for i in range(L):
        gdn.gdn_kv8_append(steps, k[i:i + 1], v[i:i + 1], table, length(i + 1))
    gdn.sync_check()
    a, b = whole.cpu().numpy(), steps.cpu().numpy()
    assert np.array_equal(a[:, :, 2 * page * d:], b[:, :, 2 * page * d:])
    x, y = R.e4m3(a[:, :, :2 * page * d]), R.e4m3(b[:, :, :2 * page * d])
    # both within half a step of the same number, one after a further half step (or several, of
    # halving size: growth by growth) of what it was: steps are 2^-9 below 2^-6, 1/8 of a binade above
    step = np.maximum(2.0 ** -9, np.exp2(np.floor(np.log2(np.maximum(np.maximum(np.abs(x), np.abs(y)), 2.0 ** -9)))) / 8)
    assert np.all(np.abs(x - y) <= 1.5 * step)


def test_idle_slots_are_left_alone():
    c = R8.Cache8([0, 40, 0], 2, 16, 64, new=[1, 1, 1], seed=1)
    k, v = (tokens(3, 2, 64, torch.bfloat16, "thd", i) for i in (1, 2))
    before = c.pages.clone()
    q = tokens(3, 4, 64, torch.bfloat16, "thd", 3)
    qo = gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, q=q, check=True)
    assert torch.equal(q, qo)                    # no rotation asked for
    changed = (c.pages != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(c.table[1, 2])]       # place 39 of the one live sequence
    rk, rv = gdn.gdn_kv8_read(c.pages, c.table_t, c.len_t, 3, 64, check=True)
    for x in (rk, rv):
        assert not x[0].any() and x[1].any() and not x[2].any()


@pytest.mark.parametrize("lens,new", [([3, 20], [7, 7]), ([3, 20], [7, 2]), ([0, 17], [20, 20])])
def test_more_new_tokens_than_the_sequence_has(lens, new):
    """The first of them lie before place 0: they are not written, the others are."""
    c = R8.Cache8(lens, 2, 16, 64, new=new, seed=2)
    n = sum(new)
    k, v, q = (tokens(n, h, 64, torch.bfloat16, "thd", i) for i, h in enumerate((2, 2, 4)))
    cu = c.cu if new[0] != new[1] else None
    qo = gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, q=q, cu_seqlens=cu, check=True)
    assert torch.equal(q, qo)
    rk, rv = gdn.gdn_kv8_read(c.pages, c.table_t, c.len_t, n, 64, cu_seqlens=cu, check=True)
    at = 0
    for L, m in zip(lens, new):
        for x, y in ((rk, k), (rv, v)):
            dead = max(0, m - L)
            assert not x[at:at + dead].any()
            # half a step of e4m3, 2^-4, and below 2^-6 of the block's scale 2^-10 of it
            top = y[at:at + m].abs().max().float() if m else 0
            live = slice(at + dead, at + m)
            assert torch.all((x[live].float() - y[live].float()).abs() <= 2.0 ** -4 * y[live].float().abs() + 2.0 ** -16 * top)
        at += m


def test_extremes():
    d, page = 64, 32
    x = torch.zeros(32, 1, d)
    x[0, 0, :16] = 1e30                          # saturates at 448 * 2^7
    x[1, 0, 3] = float("inf")
    x[1, 0, 4] = 1.0
    x[2, 0, 20] = float("nan")                   # its 16 neighbours, nothing else
    x[2, 0, 0] = -6.0
    x[16, 0, 20] = float("nan")                  # does not count for the second block's exponent
    x[16, 0, 21] = 1e20
    x[17, 0, :] = 2.0 ** -25                     # half of the least number under the least exponent: a tie
    x[18, 0, :] = 2.0 ** -24
    x[19, 0, 0] = -0.0
    x[20, 0, 0] = 448 * 2.0 ** -15               # all that the least exponent holds
    x = x.cuda()
    c = R8.Cache8([32], 1, page, d, new=[32], seed=2)
    gdn.gdn_kv8_append(c.pages, x, x, c.table_t, c.len_t, check=True)
    rk, rv = gdn.gdn_kv8_read(c.pages, c.table_t, c.len_t, 32, d, dtype=torch.float32, check=True)
    raw = c.pages[int(c.table[0, 0]), 0].cpu()
    for i, y in enumerate((rk[:, 0], rv[:, 0])):
        assert raw[R8.exponent_at(page, d, i, 0)] == 22 and raw[R8.exponent_at(page, d, i, 16)] == 0
        assert torch.all(y[0, :16] == 57344) and not y[0, 16:].any()
        assert y[1, 3] == 57344 and y[1, 4] == 1.0
        bad = torch.zeros(d, dtype=torch.bool, device="cuda")
        bad[16:32] = True
        assert torch.equal(y[2].isnan(), bad) and y[2, 0] == -6.0
        assert torch.equal(y[16].isnan(), bad) and not y[16, ~bad].any()
        assert not y[17].any() and torch.all(y[18] == 2.0 ** -24)
        assert y[19, 0] == 0 and y[20, 0] == 448 * 2.0 ** -15
        assert torch.signbit(y[19, 0])


@pytest.mark.parametrize("turn", ["no", "halves", "adjacent"])
def test_nan_takes_its_neighbours_after_the_turn(turn):
    # in halves a NaN reaches both elements of its pair, 32 apart, and both blocks
    d = 64
    x = torch.ones(3, 1, d, device="cuda")
    x[1, 0, 5] = float("nan")
    kw = {}
    if turn != "no":
        cos, sin = gdn.gdn_rope_table(8, d)
        kw = dict(cos=cos, sin=sin, pos=torch.arange(3, dtype=torch.int32, device="cuda"),
                  adjacent=turn == "adjacent")
    c = R8.Cache8([3], 1, 16, d, new=[3], seed=3)
    gdn.gdn_kv8_append(c.pages, x, x, c.table_t, c.len_t, check=True, **kw)
    rk, rv = gdn.gdn_kv8_read(c.pages, c.table_t, c.len_t, 3, d, dtype=torch.float32, check=True)
    bad = torch.zeros(3, d, dtype=torch.bool, device="cuda")
    bad[1, :16] = True
    assert torch.equal(rv[:, 0].isnan(), bad)
    if turn == "halves":
        bad[1, 32:48] = True
    assert torch.equal(rk[:, 0].isnan(), bad)


@pytest.mark.parametrize("what", ["page", "len", "cu", "pos"])
def test_bad_indices_are_reported(what):
    c = R8.Cache8([40, 20], 2, 16, 64, new=[3, 2], seed=4)
    k = tokens(5, 2, 64, torch.bfloat16, "thd", 1)
    cos, sin = gdn.gdn_rope_table(8, 64)
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    table, length, cu = c.table_t.clone(), c.len_t.clone(), c.cu.clone()
    if what == "page":
        table[0, 2] = c.pages.shape[0]
    elif what == "len":
        length[1] = 16 * table.shape[1] + 1
    elif what == "cu":
        cu[1] = 9
    else:
        pos[4] = 8
    before = c.pages.clone()
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_kv8_append(c.pages, k, k, table, length, cu_seqlens=cu, cos=cos, sin=sin, pos=pos,
                           check=True)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    if what == "page":      # the tokens of that page were left out, the others written
        assert torch.equal(c.pages[int(c.table[0, 2])], before[int(c.table[0, 2])])
        assert not torch.equal(c.pages[int(c.table[1, 1])], before[int(c.table[1, 1])])
    gdn.sync_check()


# (offsets, tokens of the call)
BAD = [([2, 3, 5], 5), ([0, 3, 4], 5), ([0, 0, 0], 5), ([5, 5, 5], 5), ([1, 3, 5], 5), ([0, -3, 5], 5),
       ([0, 1 << 30, 5], 5), ([-(1 << 30), 3, 5], 5)]
GOOD = [([0, 3, 5], 5), ([0, 0, 5], 5), ([0, 5, 5], 5)]


@pytest.mark.parametrize("entry", ["append", "read", "attn few", "attn many"])
@pytest.mark.parametrize("cu,n", BAD + GOOD)
def test_offsets_have_to_pack_the_tokens(cu, n, entry):
    c = R8.Cache8([40, 20], 2, 16, 64, new=[3, 2], seed=50)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    at = (c.pages, c.table_t, c.len_t)
    q = tokens(n, 16 if entry == "attn many" else 4, 64, torch.bfloat16, "thd", 51)
    gdn.sync_check()

    def call():
        if entry == "append":
            gdn.gdn_kv8_append(c.pages, q[:, :2], q[:, 2:], *at[1:], cu_seqlens=off, check=True)
        elif entry == "read":
            gdn.gdn_kv8_read(*at, n, 64, cu_seqlens=off, check=True)
        else:
            gdn.gdn_kv8_attn(q, *at, cu_seqlens=off, check=True)

    if (cu, n) in GOOD:
        call()
        return
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()      # reported once


def test_pool_past_32_bits():
    # a page whose offset in the pool needs 33 bits
    H, page, d = 8, 64, 128
    size = gdn.gdn_kv8_page_bytes(page, d)
    n = (1 << 32) // (H * size) + 40
    pages = torch.empty((n, H, size), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n - 1], [3]], dtype=torch.int32, device="cuda")
    length = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    k, v = (tokens(2, H, d, torch.bfloat16, "thd", i) for i in (1, 2))
    gdn.gdn_kv8_append(pages, k, v, table, length, check=True)
    rk, rv = gdn.gdn_kv8_read(pages, table, length, 2, d, check=True)
    small = gdn.gdn_kv8_pages(2, H, page, d)
    order = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(small, k, v, order, length, check=True)
    sk, sv = gdn.gdn_kv8_read(small, order, length, 2, d, check=True)
    assert torch.equal(rk, sk) and torch.equal(rv, sv)
    for heads in (2 * H, 32 * H):                # a few rows and many
        q = tokens(2, heads, d, torch.bfloat16, "thd", 3)
        a = gdn.gdn_kv8_attn(q, pages, table, length, check=True)
        b = gdn.gdn_kv8_attn(q, small, order, length, check=True)
        assert torch.equal(a, b)


def test_captured_in_a_graph_and_on_another_stream():
    c = R8.Cache8([33, 100], 2, 32, 64, new=[2, 2], seed=6)
    k, v, q = (tokens(4, h, 64, torch.bfloat16, "thd", i) for i, h in enumerate((2, 2, 4)))
    cos, sin = gdn.gdn_rope_table(128, 64)
    kw = dict(q=q, cos=cos, sin=sin, pos=torch.tensor([31, 32, 98, 99], dtype=torch.int32, device="cuda"))
    start = c.pages.clone()
    want_q = gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, check=True, **kw)
    want = c.pages.clone()
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, out=out, **kw)
    side = torch.cuda.Stream()
    for run in (g.replay, lambda: gdn.gdn_kv8_append(c.pages, k, v, c.table_t, c.len_t, out=out, **kw)):
        c.pages.copy_(start)
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(c.pages, want) and torch.equal(out, want_q)
