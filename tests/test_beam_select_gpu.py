"""gdn_beam_select against its definition in fp64: ties, banned tokens, finished and dead beams, rows at
any address, and logits that are not finite.

Beams and tokens have to be equal.  The kernel's logarithm of a row's sum is within 2^-20 of the
definition's (a relative error of the sum below 2^-20: exponentials 2^-21 each, at most a few fp32
additions of 2^-24 on every level), so inputs here are drawn with no two beams' candidates nearer
than that at a border, which is checked; equal rows give equal scores.  Scores: that and fp32's
rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn

from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NEAR = 2.0 ** -20


def logsum(x):
    top = np.max(x, -1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return top, np.log(np.sum(np.exp(x - top), -1, keepdims=True))


def definition(logits, scores, n, done=None, eos=0, apart=True):
    """(scores, beam, token) [B, n] of fp64 logits [B, W, V]."""
    B, W, V = logits.shape
    with np.errstate(invalid="ignore"):
        top, rest = logsum(logits)
        x = scores[..., None] + ((logits - top) - rest)
    x[np.isneginf(logits)] = -np.inf
    x = np.where((np.isnan(logits) | np.isposinf(logits)).any(-1, keepdims=True), np.nan, x)
    x[np.isneginf(scores)] = -np.inf
    if done is not None:
        only = np.full(x.shape, -np.inf)
        only[..., eos] = scores
        x = np.where(done[..., None], only, x)
    out = [np.zeros((B, n)), np.zeros((B, n), dtype=np.int64), np.zeros((B, n), dtype=np.int64)]
    for b in range(B):
        y = x[b].ravel()
        order = np.lexsort((np.arange(W * V), -np.where(np.isnan(y), np.inf, y)))
        best = order[:n + 1]
        v = y[best]
        if apart:
            gap = np.abs(np.diff(v))
            other = np.diff(best // V) != 0
            assert not np.any(other & (gap < 4 * NEAR) & (gap > 0)), "inputs too near each other"
        out[0][b], out[1][b], out[2][b] = v[:n], best[:n] // V, best[:n] % V
    return out


def check(logits, scores, n=None, done=None, eos=None, **kw):
    got = gdn.gdn_beam_select(logits, scores, n, done=done, eos=eos, check=True, **kw)
    B, W = scores.shape
    n = W if n is None else n
    V = logits.shape[-1]
    want = definition(U.f64(logits).reshape(B, W, V), U.f64(scores), n,
                      None if done is None else done.cpu().numpy().astype(bool), eos)
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[2].cpu().numpy(), want[2])
    a, b = U.f64(got[0]), want[0]
    finite = np.isfinite(b)
    assert np.array_equal(a[~finite], b[~finite], equal_nan=True)
    assert np.all(np.abs(a - b)[finite] <= NEAR + 2.0 ** -24 * np.abs(b[finite]))
    return got


def inputs(B, W, V, dt, seed, size=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = size * torch.randn(B, W, V, generator=g, device="cuda")
    return x.to(DT[dt]), -10 * torch.rand(B, W, generator=g, device="cuda")


CASES = [
    (1, 1, 1, 1), (1, 1, 2, 1), (2, 3, 1, 3), (1, 2, 7, 14), (3, 4, 31, 32), (2, 5, 257, 10),
    (1, 4, 1000, 4), (2, 31, 600, 20), (5, 3, 4095, 6), (2, 2, 4097, 32), (1, 32, 513, 32), (7, 8, 8191, 16),
    (2, 4, 32000, 8), (1, 5, 50257, 5), (40, 8, 32003, 16), (3, 16, 65536, 32), (1, 1, 300001, 20),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,n", CASES)
def test_matches_definition(B, W, V, n, dt):
    x, s = inputs(B, W, V, dt, V + n)
    check(x, s, n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 5000, 40001])
def test_all_alike_goes_by_index(V, dt):
    """Every number equal: the lowest beam, its lowest tokens; also at fp32's ends."""
    for value in (0.0, -1.5, 3.0e38, -3.0e38):
        x = torch.full((2, 3, V), value, device="cuda").to(DT[dt])
        s = torch.zeros(2, 3, device="cuda")
        got = check(x, s, 7)
        assert got[2].tolist() == [list(range(7))] * 2 and not got[1].any()
    # zeros of both signs are equal
    x = torch.zeros(1, 1, V, device="cuda").to(DT[dt])
    x[..., ::2] = -0.0
    assert check(x, torch.zeros(1, 1, device="cuda"), 9)[2].tolist() == [list(range(9))]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4096, 50257])
def test_equal_beams_give_equal_scores_wherever_their_rows_lie(V, dt):
    # (50257 numbers of 2 bytes: each row begins at another address modulo 16)
    x, _ = inputs(2, 1, V, dt, 3)
    x[:, :, 1234] = 20.0
    x = x.expand(2, 9, V).contiguous()
    s = torch.full((2, 9), -2.5, device="cuda")
    scores, beam, token = check(x, s, 27)
    # the best token of every beam first, in the beams' order, at one score
    assert beam[:, :9].tolist() == [list(range(9))] * 2
    for b in range(2):
        assert scores[b, :9].unique().numel() == 1 and token[b, :9].unique().numel() == 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_ties_in_rows(dt):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-3, 4, (3, 4, 20011), generator=g, device="cuda").to(DT[dt])
    s = -torch.rand(3, 4, generator=g, device="cuda")
    check(x, s, 32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["ascending", "descending", "few", "block"])
def test_orders_that_defeat_a_bound(kind, dt):
    """Sorted rows, rows with all but a few numbers banned, and the largest numbers side by side."""
    V, n = 30000, 24
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(2, 3, V, generator=g, device="cuda")
    if kind == "ascending":
        x = x.sort(-1).values
    elif kind == "descending":
        x = x.sort(-1, descending=True).values
    elif kind == "few":
        keep = torch.randint(0, V, (5,), generator=g, device="cuda")
        y = torch.full_like(x, -float("inf"))
        y[..., keep] = x[..., keep]
        x = y
    else:
        x[..., 12345:12345 + 100] += 10
    check(x.to(DT[dt]), -5 * torch.rand(2, 3, generator=g, device="cuda"), n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lowest", [False, True])
def test_banned_tokens(dt, lowest):
    """-infinity, or the type's lowest number, in some places, in all but one, and in all of a row."""
    V = 9000
    x, s = inputs(3, 4, V, dt, 7)
    off = torch.finfo(DT[dt]).min if lowest else -float("inf")
    x[0, :, 1000:8000] = off
    x[1, 1] = off
    x[1, 1, 77] = 1.0
    x[2, 2] = off
    for n in (4, 20):
        check(x, s, n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("W", [3, 31, 32])
def test_fewer_tokens_left_than_wanted(dt, W):
    """All but two tokens at the type's lowest number: the rest goes by index (in fp64 too a score
    next to that number is lost)."""
    x, s = inputs(2, W, 700, dt, 17)
    y = torch.full_like(x, torch.finfo(DT[dt]).min)
    y[..., 50] = x[..., 50]
    y[..., 600] = x[..., 600]
    s[:, 3:] = -float("inf")
    check(y, s, 20)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_first_step(dt):
    """One beam of a group counts; with all dead, the lowest continuations come, at -infinity."""
    x, s = inputs(2, 4, 3001, dt, 8)
    s[:, 1:] = -float("inf")
    s[1, 0] = -float("inf")
    got = check(x, s, 8)
    assert got[0][1].isneginf().all() and got[2][1].tolist() == list(range(8))
    # (a dead beam's logits are not looked at)
    x[:, 1:] = float("nan")
    check_same = gdn.gdn_beam_select(x, s, 8, check=True)
    assert all(torch.equal(a, b) for a, b in zip(got, check_same))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("eos", [0, 2, 1500])
def test_finished_beams(dt, eos):
    V = 1501
    x, s = inputs(5, 6, V, dt, 9)
    done = torch.zeros(5, 6, dtype=torch.bool, device="cuda")
    done[1, 2] = done[2, :] = done[3, 0] = done[3, 5] = done[4, 1] = True
    s[4, 1] = -float("inf")
    x[3, 0] = float("nan")                    # (nor are a finished one's)
    for n in (6, 12):
        check(torch.where(done[..., None], torch.zeros((), dtype=x.dtype, device="cuda"), x), s, n, done, eos)
        a = gdn.gdn_beam_select(x, s, n, done=done, eos=eos, check=True)
        b = gdn.gdn_beam_select(x, s, n, done=done.to(torch.uint8), eos=eos, check=True)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    # fewer tokens than continuations wanted
    check(x[..., :2].contiguous(), s, 12, done, min(eos, 1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite_show(dt, bad):
    x, s = inputs(2, 3, 5000, dt, 10)
    clean = check(x, s, 6)
    x[1, 1, 4321] = bad
    got = check(x, s, 6)
    assert got[0][1].isnan().all() and (got[1][1] == 1).all()
    assert all(torch.equal(a[0], b[0]) for a, b in zip(clean, got))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("at", [5, 30000])
def test_a_nan_among_the_lowest_numbers_is_not_lost(dt, at):
    # (before and after the numbers that the sum is about)
    x = torch.full((1, 2, 40000), torch.finfo(DT[dt]).min, device="cuda").to(DT[dt])
    x[0, :, 20000] = 1.0
    s = torch.zeros(1, 2, device="cuda")
    check(x, s, 3)
    x[0, 1, at] = float("nan")
    got = check(x, s, 3)
    assert got[0].isnan().all() and (got[1] == 1).all()


def test_views_streams_graphs_and_outputs():
    V = 5003
    x, s = inputs(4, 3, V, "bf16", 11)
    want = check(x, s, 5)
    # the last position of a longer run of logits, and of a padded vocabulary
    wide = torch.full((4, 3, 2, V + 9), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :, 1, 3:3 + V] = x
    view = wide[:, :, 1, 3:3 + V]
    for y in (view, view.flatten(0, 1), x.view(12, V)):
        assert all(torch.equal(a, b) for a, b in zip(want, gdn.gdn_beam_select(y, s, 5, check=True)))
    out = tuple(torch.zeros_like(t) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_beam_select(view, s, 5, out=out)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    other = tuple(torch.zeros_like(t) for t in want)
    with torch.cuda.graph(g):
        gdn.gdn_beam_select(view, s, 5, out=out)
    with torch.cuda.graph(h):
        gdn.gdn_beam_select(x, s, 5, out=other)
    for _ in range(3):
        for t in out + other:
            t.zero_()
        g.replay()
        h.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        assert all(torch.equal(a, b) for a, b in zip(want, other))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("far", [False, True])
def test_the_largest_vocabulary(dt, far):
    # equal numbers: the largest sum that there is; and one number far above the others
    V = 1 << 22
    x = torch.full((1, 2, V), -1.0, device="cuda").to(DT[dt])
    if far:
        x[0, 0, V - 1] = x[0, 1, 0] = 30.0
    check(x, torch.tensor([[-1.0, -1.5]], device="cuda"), 32)


def test_rows_past_32_bits():
    # rows more than 2^31 elements apart
    V, far = 1000, (1 << 31) + 8
    store = torch.zeros(far + 2 * V, dtype=torch.bfloat16, device="cuda")
    x, s = inputs(1, 2, V, "bf16", 12)
    view = torch.as_strided(store, (2, V), (far, 1))
    view.copy_(x[0])
    a, b = gdn.gdn_beam_select(view, s, 2, check=True), check(x, s, 2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_nothing_to_do():
    x = torch.zeros(0, 4, 10, device="cuda")
    assert [t.shape for t in gdn.gdn_beam_select(x, torch.zeros(0, 4, device="cuda"), 3)] == [(0, 3)] * 3
