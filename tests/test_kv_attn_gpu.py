"""gdn_kv_attn against the fp64 definition: head layouts, lengths, masks that
leave rows empty, garbage where nothing is seen, and the refusals."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def queries(n, H, d, dt, layout, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (size * torch.randn(n, H, d, generator=g, device="cuda")).to(dt)
    return x.transpose(0, 1).contiguous().transpose(0, 1) if layout == "htd" else x


def run(c, q, causal=True, window=0, scale=None, **kw):
    uniform = min(c.new) == max(c.new)
    return gdn.gdn_kv_attn(q, c.pages, c.table_t, c.len_t, cu_seqlens=None if uniform else c.cu,
                           kv_scale=c.scale_t, causal=causal, window=window, scale=scale,
                           return_lse=True, check=True, **kw)


def check(c, q, causal=True, window=0, scale=None, **kw):
    o, lse = run(c, q, causal, window, scale, **kw)
    assert o.dtype == q.dtype and o.shape == q.shape
    ref = c.reference(U.f64(q), c.d ** -0.5 if scale is None else scale, causal, window)
    o, lse = U.f64(o), U.f64(lse)
    assert np.all(np.abs(o - ref[0]) <= R.tolerance(ref, q.dtype))
    empty = np.isneginf(ref[1])
    assert np.array_equal(empty, np.isneginf(lse))
    # the score's error, and the sum's and its logarithm's roundings
    tol = 2.0 ** -20 * (4 + ref[3] + np.abs(ref[1], where=~empty, out=np.zeros_like(ref[1])))
    assert np.all(np.abs(lse - ref[1])[~empty] <= tol[~empty])
    return o


# lens, new, Hq, H, d, page, causal, window, head scales, layout, io
CASES = [
    ([77], [1], 16, 2, 64, 16, True, 0, False, "thd", "f32"),
    ([1], [1], 1, 1, 128, 64, True, 0, False, "thd", "bf16"),
    ([0, 1, 15, 16, 17, 127, 128, 129, 300], [1] * 9, 8, 2, 128, 64, True, 0, True, "thd", "bf16"),
    ([0, 1, 15, 16, 17, 127, 128, 129, 300], [1] * 9, 8, 2, 128, 16, True, 0, True, "htd", "f32"),
    ([1000, 2100, 3], [1] * 3, 12, 4, 128, 32, True, 0, False, "thd", "bf16"),
    ([2049], [1], 9, 1, 256, 128, True, 0, True, "thd", "bf16"),
    ([2049, 500], [1, 1], 9, 3, 256, 16, True, 0, True, "htd", "f32"),
    ([600, 33], [1, 1], 16, 16, 64, 256, True, 0, False, "thd", "bf16"),
    ([700, 513, 40], [5, 5, 5], 8, 2, 128, 16, True, 100, False, "thd", "bf16"),
    ([700, 513, 40], [5, 3, 40], 8, 2, 64, 64, True, 0, True, "htd", "bf16"),
    ([700, 513, 40], [5, 3, 40], 4, 1, 128, 64, False, 0, True, "thd", "f32"),
    ([130, 0, 260], [2, 0, 130], 6, 2, 128, 32, True, 0, False, "thd", "bf16"),
    ([400, 257], [100, 100], 8, 2, 128, 64, False, 60, False, "htd", "bf16"),
    ([300, 3, 0], [7, 7, 7], 2, 2, 64, 16, True, 0, False, "thd", "f32"),      # rows before place 0
    ([300, 3, 0], [7, 7, 7], 2, 2, 128, 16, False, 5, False, "thd", "bf16"),
    ([1500], [1], 4, 2, 128, 64, True, 1, False, "thd", "bf16"),               # sees itself only
    ([5000], [1], 2, 1, 128, 128, True, 17, True, "thd", "f32"),
]


@pytest.mark.parametrize("lens,new,Hq,H,d,page,causal,window,head_scale,layout,io", CASES)
def test_matches_definition(lens, new, Hq, H, d, page, causal, window, head_scale, layout, io):
    c = R.Cache(lens, H, page, d, new=new, head_scale=head_scale, seed=len(lens) + d)
    check(c, queries(c.tokens, Hq, d, DT[io], layout, d + page), causal, window)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_long_sequences_cut_over_the_gpu(io):
    # many tiles a CTA and many CTAs a sequence, at lengths around the cuts
    c = R.Cache([9000, 17, 0, 20011], 1, 64, 64, seed=5)
    check(c, queries(4, 4, 64, DT[io], "thd", 1))
    # a tighter bound on the length plans another division
    check(c, queries(4, 4, 64, DT[io], "thd", 1), max_len=20011, max_new=1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_sequences(io):
    # more sequences than a CTA has threads to share them out
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    c = R.Cache(lens, 1, 16, 64, seed=6)
    check(c, queries(700, 2, 64, DT[io], "thd", 2))


@pytest.mark.parametrize("size", [1e-30, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_query_magnitudes(io, size):
    # scores from all alike to one winner; queries far outside fp16's range
    c = R.Cache([333, 70], 2, 32, 64, seed=7)
    check(c, queries(2, 4, 64, DT[io], "thd", 3, size), scale=0.125 / max(size, 1.0) * 4)


def test_scale_sign_and_zero():
    c = R.Cache([333, 70], 2, 32, 64, seed=8)
    for scale in (-0.3, 0.0, 2.0):
        check(c, queries(2, 4, 64, torch.float32, "thd", 4), scale=scale)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_growing_scores_raise_the_maximum(io):
    # keys that grow along the sequence: the running maximum moves in every step
    d, page = 64, 16
    c = R.Cache([1024], 1, page, d, seed=9)
    at = 2 * (page * d // 2)
    for p in range(64):
        c.np_pages[c.table[0, p], 0, at:at + page * d // 16] = 0x18 + p
        c.np_pages[c.table[0, p], 0, :page * d // 2] = 0x22      # every element 1
    c.pages = torch.from_numpy(c.np_pages).cuda()
    q = torch.ones(1, 2, d, dtype=DT[io], device="cuda")
    check(c, q, scale=0.01)
    check(c, -q, scale=0.01)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,new", [(128, 64, 24), (64, 16, 24), (256, 32, 24), (128, 64, 300)])
def test_nan_reaches_only_the_rows_that_see_it(d, page, new, io):
    L = new + 200
    c = R.Cache([L], 1, page, d, new=[new], seed=10)
    q = queries(new, 2, d, DT[io], "thd", 5)
    clean, _ = run(c, q, window=150)
    where = L - new // 2                                      # half of the rows see this place
    blk, row = c.table[0, where // page], where % page
    code, scale = page * d // 2, page * d // 16
    # a NaN in one block of the value: those 16 dimensions of the rows that see it
    c.np_pages[blk, 0, 2 * code + scale + row * (d // 16) + 1] = 0x7F
    c.pages = torch.from_numpy(c.np_pages).cuda()
    o, _ = run(c, q, window=150)
    bad = torch.zeros_like(o, dtype=torch.bool)
    first = where - (L - new)
    bad[first:min(new, first + 150), :, 16:32] = True
    assert torch.equal(o.isnan(), bad)
    assert torch.equal(o[~bad], clean[~bad])
    # a NaN in the key: all of those rows
    c.np_pages[blk, 0, 2 * code + scale + row * (d // 16) + 1] = 0x30
    c.np_pages[blk, 0, 2 * code + row * (d // 16) + 2] = 0xFF
    c.pages = torch.from_numpy(c.np_pages).cuda()
    o, _ = run(c, q, window=150)
    bad[first:min(new, first + 150)] = True
    assert torch.equal(o.isnan(), bad)
    assert torch.equal(o[~bad], clean[~bad])


def test_nonfinite_queries_stay_in_their_rows():
    c = R.Cache([300], 2, 64, 128, new=[3], seed=11)
    q = queries(3, 4, 128, torch.bfloat16, "thd", 6)
    clean, _ = run(c, q)
    q[1, 2, 7] = float("inf")
    q[2, 0, 9] = float("nan")
    o, _ = run(c, q)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[1, 2] = bad[2, 0] = True
    assert o[bad].isnan().all() or not o[1, 2].isfinite().all()
    assert torch.equal(o[~bad], clean[~bad])


def test_same_bits_again_and_on_another_stream():
    c = R.Cache([5000, 77, 1234], 2, 64, 128, seed=12)
    q = queries(3, 8, 128, torch.bfloat16, "thd", 7)
    a, la = run(c, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = torch.zeros_like(q)
        for _ in range(20):
            x.add_(0)
        x.copy_(q)
        b, lb = gdn.gdn_kv_attn(x, c.pages, c.table_t, c.len_t, return_lse=True)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_captured_in_a_graph():
    c = R.Cache([900, 40], 2, 64, 128, seed=13)
    q = queries(2, 8, 128, torch.bfloat16, "thd", 8)
    want, _ = run(c, q)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    gdn.gdn_kv_attn(q, c.pages, c.table_t, c.len_t, out=out)
    torch.cuda.synchronize()
    out.zero_()
    with torch.cuda.graph(g):
        gdn.gdn_kv_attn(q, c.pages, c.table_t, c.len_t, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_table_rows_apart_and_views():
    # a persistent page table wider than this call's, lengths in the middle of an array,
    # queries inside a fused projection
    c = R.Cache([200, 90], 2, 64, 128, seed=14)
    q = queries(2, 4, 128, torch.bfloat16, "thd", 9)
    want, _ = run(c, q)
    wide = torch.full((2, 9), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.table_t.shape[1]] = c.table_t
    lens = torch.cat([c.len_t[:1] * 0 - 5, c.len_t, c.len_t[:1] * 0 - 5])
    fused = torch.full((2, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:6] = q
    got = gdn.gdn_kv_attn(fused[:, 2:6], c.pages, wide[:, 2:2 + c.table_t.shape[1]], lens[1:3],
                          check=True)
    assert torch.equal(want, got)


@pytest.mark.parametrize("what", ["page", "len", "max_len", "max_new", "cu"])
def test_bad_indices_are_reported(what):
    c = R.Cache([140, 20], 2, 16, 64, new=[3, 2], seed=15)
    q = queries(5, 4, 64, torch.bfloat16, "thd", 10)
    table, length, cu, kw = c.table_t.clone(), c.len_t.clone(), c.cu.clone(), {}
    if what == "page":
        table[0, 3] = -1
    elif what == "len":
        length[0] = -1
    elif what == "max_len":
        kw["max_len"] = 139
    elif what == "max_new":
        kw["max_new"] = 2
    else:
        cu[1] = 9
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_kv_attn(q, c.pages, table, length, cu_seqlens=cu, check=True, **kw)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()


def test_nothing_to_do():
    c = R.Cache([40], 2, 16, 64, new=[0], seed=16)
    q = queries(0, 4, 64, torch.bfloat16, "thd", 11)
    assert run(c, q)[0].shape == q.shape
