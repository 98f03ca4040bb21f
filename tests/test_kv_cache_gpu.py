"""gdn_kv_append and gdn_kv_read: what the 4-bit cache holds, where it lies, and
what stays untouched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention_ref as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tokens(n, H, d, dt, layout, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, H, d, generator=g, device="cuda")
    x = (x * torch.exp(torch.randn(1, H, d, generator=g, device="cuda"))).to(dt)
    return x.transpose(0, 1).contiguous().transpose(0, 1) if layout == "htd" else x


def nearest_scale(m, slack):
    """The e4m3 numbers next to m / 6 (at most 448): the nearest, or both where m / 6 is within
    fp32's rounding of their middle."""
    grid = R.e4m3(np.arange(127))
    t = np.minimum(m / 6, 448.0)
    off = np.abs(grid - t[..., None])
    best = off.min(-1)
    return off <= (best + 8 * 2.0 ** -24 * t + 2 * slack / 6)[..., None]


def check_held(x, codes, scales, g, off):
    """x fp64 [..., d] against its codes and scale bytes: the scale is the e4m3 number nearest a
    sixth of the largest magnitude of 16, and each element the nearest it can be held as, both to
    within fp32's rounding (4 roundings, 2^-24 each, doubled) and twice `off`, what x itself may
    be off by."""
    y = x.reshape(*x.shape[:-1], -1, 16) / g[:, None, None]
    slack = (off / g)[:, None]
    ok = nearest_scale(np.abs(y).max(-1), slack)
    assert np.all(np.take_along_axis(ok, scales[..., None].astype(np.int64), -1))
    s = R.e4m3(scales)[..., None]
    e = np.stack([codes & 15, codes >> 4], -1).reshape(y.shape)
    held = R.E2M1[e] * s
    best = np.abs(R.E2M1 * s[..., None] - y[..., None]).min(-1)
    assert np.all(np.abs(held - y) <= best + 8 * 2.0 ** -24 * np.abs(y) + 2 * slack[..., None])
    return (held * g[:, None, None]).reshape(x.shape)


CASES = [
    # lens before, new, Hq, H, d, page, rot, axes, adjacent, head scales, layout, io
    ([0, 15, 16, 63, 130], [1, 1, 1, 1, 1], 8, 2, 128, 64, 128, 1, False, False, "thd", "bf16"),
    ([0, 3, 100], [37, 1, 65], 4, 4, 64, 16, 64, 3, False, True, "thd", "f32"),
    ([5, 0, 0, 31], [3, 0, 128, 2], 6, 3, 256, 32, 64, 2, False, True, "htd", "bf16"),
    ([7], [300], 2, 1, 128, 128, 48, 1, True, False, "htd", "f32"),
    ([250, 1], [10, 10], 3, 1, 64, 256, 0, 1, False, False, "thd", "bf16"),
]


@pytest.mark.parametrize("had,new,Hq,H,d,page,rot,axes,adjacent,head_scale,layout,io", CASES)
def test_append_and_read(had, new, Hq, H, d, page, rot, axes, adjacent, head_scale, layout, io):
    dt = DT[io]
    lens = [a + b for a, b in zip(had, new)]
    c = R.Cache(lens, H, page, d, new=new, head_scale=head_scale, seed=page)
    n = c.tokens
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
    qo = gdn.gdn_kv_append(c.pages, k, v, c.table_t, c.len_t, q=q, cu_seqlens=cu,
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

    ones = np.ones(H)
    gs = (ones, ones) if c.scale is None else c.scale.astype(np.float64)
    expect = c.np_pages.copy()
    held = [np.zeros((n, H, d)), np.zeros((n, H, d))]
    all_k, all_v = turned(k), U.f64(v)
    code, scale = page * d // 2, page * d // 16
    for b in range(len(lens)):
        for j in range(new[b]):
            p, t = had[b] + j, c.at[b] + j
            blk, row = c.table[b, p // page], p % page
            for i, x in ((0, all_k[t]), (1, all_v[t])):
                a, s = i * code + row * (d // 2), 2 * code + i * scale + row * (d // 16)
                codes, scales = got[blk, :, a:a + d // 2], got[blk, :, s:s + d // 16]
                # a turned element is two products and a sum of the row's numbers
                off = 8 * 2.0 ** -24 * np.abs(U.f64(k[t])).max(-1) if i == 0 else np.zeros(H)
                held[i][t] = check_held(x, codes.astype(np.int64), scales, gs[i], off)
                expect[blk, :, a:a + d // 2], expect[blk, :, s:s + d // 16] = codes, scales
    assert np.array_equal(got, expect)           # nothing else was written

    rk, rv = gdn.gdn_kv_read(c.pages, c.table_t, c.len_t, n, d, cu_seqlens=cu, kv_scale=c.scale_t,
                             dtype=dt, check=True)
    for x, y in ((rk, held[0]), (rv, held[1])):
        assert np.all(np.abs(U.f64(x) - y) <= np.abs(y) * (2.0 ** -8 if io == "bf16" else 2.0 ** -23))


def test_idle_slots_are_left_alone():
    c = R.Cache([0, 40, 0], 2, 16, 64, new=[1, 1, 1], seed=1)
    k, v = (tokens(3, 2, 64, torch.bfloat16, "thd", i) for i in (1, 2))
    before = c.pages.clone()
    q = tokens(3, 4, 64, torch.bfloat16, "thd", 3)
    qo = gdn.gdn_kv_append(c.pages, k, v, c.table_t, c.len_t, q=q, check=True)
    assert torch.equal(q, qo)                    # no rotation asked for
    changed = (c.pages != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(c.table[1, 2])]       # place 39 of the one live sequence
    rk, rv = gdn.gdn_kv_read(c.pages, c.table_t, c.len_t, 3, 64, check=True)
    for x in (rk, rv):
        assert not x[0].any() and x[1].any() and not x[2].any()


def test_extremes():
    d, page = 64, 16
    x = torch.zeros(6, 1, d)
    x[0, 0, :16] = 1e30                          # saturates at 6 * 448
    x[1, 0, 3] = float("inf")
    x[1, 0, 4] = 1.0
    x[2, 0, 20] = float("nan")                   # its 16 neighbours, nothing else
    x[2, 0, 0] = 6.0
    x[3, 0, :] = 2.0 ** -13                      # below the smallest scale's half: zero
    x[4, 0, :16] = torch.linspace(-6, 6, 16)
    x[5, 0, 0] = -0.0
    x = x.cuda()
    c = R.Cache([6], 1, page, d, new=[6], seed=2)
    gdn.gdn_kv_append(c.pages, x, x, c.table_t, c.len_t, check=True)
    rk, rv = gdn.gdn_kv_read(c.pages, c.table_t, c.len_t, 6, d, dtype=torch.float32, check=True)
    for y in (rk[:, 0], rv[:, 0]):
        assert torch.all(y[0, :16] == 2688) and not y[0, 16:].any()
        assert y[1, 3] == 2688 and y[1, 4] == 0
        bad = torch.zeros(d, dtype=torch.bool, device="cuda")
        bad[16:32] = True
        assert torch.equal(y[2].isnan(), bad) and y[2, 0] == 6.0
        assert not y[3].any() and not y[5].any()
        grid = torch.tensor(R.E2M1, device="cuda").float()
        assert torch.isin(y[4, :16], grid).all()
        assert torch.all((y[4, :16] - x[4, 0, :16]).abs() <= 1.0)


def test_ties_go_to_even():
    d = 64
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    even = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    x = torch.zeros(1, 1, d)
    x[0, 0, :8] = torch.tensor([6.0] + mid)
    x[0, 0, 8:15] = -torch.tensor(mid)
    c = R.Cache([1], 1, 16, d, new=[1], seed=3)
    gdn.gdn_kv_append(c.pages, x.cuda(), x.cuda(), c.table_t, c.len_t, check=True)
    rk, _ = gdn.gdn_kv_read(c.pages, c.table_t, c.len_t, 1, d, dtype=torch.float32)
    assert rk[0, 0, :8].tolist() == [6.0] + even
    assert rk[0, 0, 8:15].tolist() == [-e for e in even]


@pytest.mark.parametrize("what", ["page", "len", "cu", "pos"])
def test_bad_indices_are_reported(what):
    c = R.Cache([40, 20], 2, 16, 64, new=[3, 2], seed=4)
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
        gdn.gdn_kv_append(c.pages, k, k, table, length, cu_seqlens=cu, cos=cos, sin=sin, pos=pos,
                          check=True)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    if what == "page":      # the tokens of that page were left out, the others written
        assert torch.equal(c.pages[int(c.table[0, 2])], before[int(c.table[0, 2])])
        assert not torch.equal(c.pages[int(c.table[1, 1])], before[int(c.table[1, 1])])
    gdn.sync_check()


def test_pool_past_32_bits():
    # a page whose offset in the pool needs 33 bits
    H, page, d = 8, 64, 128
    size = gdn.gdn_kv_page_bytes(page, d)
    n = (1 << 32) // (H * size) + 40
    pages = torch.empty((n, H, size), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n - 1], [3]], dtype=torch.int32, device="cuda")
    length = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    k, v = (tokens(2, H, d, torch.bfloat16, "thd", i) for i in (1, 2))
    gdn.gdn_kv_append(pages, k, v, table, length, check=True)
    rk, rv = gdn.gdn_kv_read(pages, table, length, 2, d, check=True)
    small = gdn.gdn_kv_pages(2, H, page, d)
    order = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(small, k, v, order, length, check=True)
    sk, sv = gdn.gdn_kv_read(small, order, length, 2, d, check=True)
    assert torch.equal(rk, sk) and torch.equal(rv, sv)
    q = tokens(2, 2 * H, d, torch.bfloat16, "thd", 3)
    a = gdn.gdn_kv_attn(q, pages, table, length, check=True)
    b = gdn.gdn_kv_attn(q, small, order, length, check=True)
    assert torch.equal(a, b)
