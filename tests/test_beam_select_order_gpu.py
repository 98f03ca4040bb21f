"""gdn_beam_select where the sums that scores are compared as do not fall with the logits: a sum of two
fp32 numbers is rounded, and of two neighbouring logits the smaller one's may come out larger.  Every
place of the result is written all the same, and a beam's tokens come in the order of their logits."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at,low,high", [(-25, 0.5, 0.75), (-23, 2.2, 3.8)])
@pytest.mark.parametrize("V", [40, 3000])
@pytest.mark.parametrize("W", [1, 2])
def test_neighbouring_logits(W, V, at, low, high):
    """Rows whose second and third numbers are -2^at and the next one below it, the first somewhere in
    [low, high]: 1 to 35 of 10^4 scores in that range turn the two sums around (in numpy's fp32)."""
    B = 1 << 15
    g = torch.Generator(device="cuda").manual_seed(V - at)
    second = torch.tensor(-2.0 ** at, device="cuda")
    third = torch.nextafter(second, second - 1)
    x = third - 1e-3 * torch.rand(1, W, V, generator=g, device="cuda") - 1e-6
    x = x.repeat(B // W, 1, 1)
    x[..., 5] = low + (high - low) * torch.rand(B // W, W, generator=g, device="cuda")
    x[..., 7] = second
    x[..., 31] = third
    s = -60 * torch.rand(B // W, W, generator=g, device="cuda")
    if W == 2:
        s[:, 1] = s[:, 0] - 40                       # its candidates are no match for the first beam's
    for n in (2, 3):
        out = (torch.zeros(B // W, n, device="cuda"),) + tuple(
            torch.full((B // W, n), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        gdn.gdn_beam_select(x, s, n, out=out, check=True)
        assert (out[1] == 0).all()
        want = torch.tensor([5, 7, 31][:n], dtype=torch.int32, device="cuda")
        assert torch.equal(out[2], want.expand(B // W, n))
        assert (out[0][:, 1:] <= out[0][:, :-1]).all()
