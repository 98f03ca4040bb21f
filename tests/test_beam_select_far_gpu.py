"""gdn_beam_select with finite logits of large magnitude: vocabularies masked with a number far below the
others, beams whose tokens are all masked, and rows that lie far from 0 as a whole.

Against the definition in fp64 with test_beam_select_gpu's tolerance: a logarithm is off by no more here,
as it is formed from differences of logits, and exponentials of differences below -104 are 0 in fp32."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests.test_beam_select_gpu import DT, check, inputs

pytestmark = pytest.mark.gpu

# on both sides of where products with log2(e) lose what the sum is about, and where they overflow
FAR = [-9.9e3, -1.2e4, -1e4, -1e5, -1e6, 1e6, -1e7, -1e9, 1e10, -1e10, -1e12, -1e15, -1e20, -1e30, 1e30, -1e32,
       -1e36, -2e38, 2.5e38]
MASKS = [x for x in FAR if x < 0]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 50257])
@pytest.mark.parametrize("value", FAR)
def test_rows_of_one_value(value, V, dt):
    x = torch.full((2, 3, V), value, device="cuda").to(DT[dt])
    s = torch.tensor([[-0.25, 0.0, -1.5], [-3.0, -3.5, -0.5]], device="cuda")
    got = check(x, s, 7)
    assert got[2].tolist() == [list(range(7))] * 2 and got[1][:, 0].tolist() == [1, 2]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 50257])
@pytest.mark.parametrize("mask", MASKS)
def test_all_but_neighbouring_tokens_masked(mask, V, dt):
    """Threads that see the mask alone, before, behind and beside those that do not."""
    for at in (0, V // 2 + 3, V - 30):
        x, s = inputs(2, 3, V, dt, V + at)
        y = torch.full_like(x, mask)
        y[..., at:at + 30] = x[..., at:at + 30]
        check(y, s, 24)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [700, 50257])
@pytest.mark.parametrize("mask", MASKS)
def test_part_of_the_vocabulary_masked(mask, V, dt):
    # whole batches of a thread before the others, behind them, and here and there
    x, s = inputs(4, 2, V, dt, V + 1)
    x[0, :, :4 * V // 5] = mask
    x[1, :, V // 5:] = mask
    g = torch.Generator(device="cuda").manual_seed(V)
    hit = torch.rand(V, generator=g, device="cuda") < 0.99
    hit[77:177] = False
    x[2, :, hit] = mask
    x[3, :, 1:] = mask                              # one token is left
    check(x[:3].contiguous(), s[:3].contiguous(), 20)
    # (a beam's one token; what else there is of one beam goes by index)
    check(x[3:].contiguous(), s[3:].contiguous(), 2)
    got = check(x[3:, :1].contiguous(), s[3:, :1].contiguous(), 9)
    assert got[2].tolist() == [list(range(9))]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", MASKS)
def test_a_beam_whose_tokens_are_all_masked(mask, dt):
    """Next to ordinary ones: it has the score of any row of equal logits, not infinity, nor NaN."""
    x, s = inputs(2, 4, 32003, dt, 21)
    x[0, 1] = mask
    x[1, 0] = x[1, 2] = mask
    s[0, 1] = s[1, 2] = 3.0
    check(x, s, 12)


@pytest.mark.parametrize("offset", [9.9e3, 1.1e4, 1e5, 1e6, 1e7, -9.9e3, -1.1e4, -1e5, -1e6, -1e7])
@pytest.mark.parametrize("V", [700, 50257])
def test_rows_with_an_offset(offset, V):
    x, s = inputs(2, 3, V, "f32", 22)
    check(x + offset, s, 10)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [-1e5, -1e10, -1e30, -2e38])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_shows_among_masked_tokens(bad, mask, dt):
    for V, at in ((700, 5), (50257, 9), (50257, 30000), (50257, 50256)):
        x = torch.full((1, 2, V), mask, device="cuda").to(DT[dt])
        x[0, :, V // 2] = 1.0
        s = torch.zeros(1, 2, device="cuda")
        x[0, 1, at] = bad
        got = check(x, s, 3)
        assert got[0].isnan().all() and (got[1] == 1).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_at_any_address_gives_equal_scores(dt):
    # (50257 numbers of 2 bytes: each row begins at another address modulo 16)
    x, _ = inputs(1, 1, 50257, dt, 23)
    x[..., 100:50000] = -1e10
    x[..., 20000] = 20.0
    x = x.expand(1, 9, -1).contiguous()
    scores, beam, token = check(x, torch.full((1, 9), -2.5, device="cuda"), 27)
    assert beam[0, :9].tolist() == list(range(9))
    assert scores[0, :9].unique().numel() == 1 and (token[0, :9] == 20000).all()


def test_ordinary_rows_keep_their_bits_beside_masked_ones():
    x, s = inputs(2, 3, 30000, "bf16", 24)
    want = gdn.gdn_beam_select(x[:, :1].contiguous(), s[:, :1].contiguous(), 8, check=True)
    x[:, 1:] = -1e10
    s[:, 1:] = -100.0
    got = gdn.gdn_beam_select(x, s, 8, check=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
