"""The hybrid decoder of examples/: rope, append and attention next to the gated delta rule, as a
user runs them.

Tolerances (fp32 rows).  Chunks and single tokens of the same sequence differ by the kernels' fp32
rounding (1e-5 of a row at most); such a difference moves a cached number by one of its steps only
where it lies that close to a boundary: about 1e-4 of the numbers, each by a third of its size at
most, sqrt(1e-4) / 3 = 3e-3 of a row; three layers and the projections: 2e-2.  Against the pass
without a cache: e2m1 steps are 1/2 to 1 wide over [1, 6] with the largest of 16 at 6, an error of
about 10 % of a row in the keys (so in the scores, which are of order 1, and the weights) and in the
values: sqrt(2) * 0.1, next to the residual stream: 0.25.
"""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu
COUNTS = [3, 130, 1, 64]


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples",
                        "hybrid_decoder.py")
    spec = importlib.util.spec_from_file_location("hybrid_decoder", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _tokens(n, seed):
    return torch.randint(0, 256, (n,), generator=torch.Generator().manual_seed(seed))


def _apart(x, y):
    return ((x - y).norm(dim=-1) / y.norm(dim=-1)).max().item()


@pytest.mark.parametrize("layers", ["gag", "a"])
def test_tokens_match_chunks(ex, layers):
    """Prompts in one pass, then tokens one by one (the step replayed from a graph), against all
    of it in one pass and in two."""
    model = ex.Decoder(layers=layers, dtype=torch.float32)
    more = 9
    seqs = [_tokens(n + more, 10 + n).cuda() for n in COUNTS]
    whole = ex.Serving(model, len(COUNTS))
    full = whole.extend(torch.cat(seqs), [n + more for n in COUNTS])
    full = full.split([n + more for n in COUNTS])

    one = ex.Serving(model, len(COUNTS))
    got = one.extend(torch.cat([s[:n] for s, n in zip(seqs, COUNTS)]), COUNTS).split(COUNTS)
    for b, n in enumerate(COUNTS):
        assert _apart(got[b], full[b][:n]) < 2e-2
    for j in range(more):
        got = one.step(torch.stack([s[n + j] for s, n in zip(seqs, COUNTS)]))
        assert _apart(got, torch.stack([f[n + j] for f, n in zip(full, COUNTS)])) < 2e-2
    assert one.len.tolist() == whole.len.tolist()

    two = ex.Serving(model, len(COUNTS))
    two.extend(torch.cat([s[:n] for s, n in zip(seqs, COUNTS)]), COUNTS)
    rest = two.extend(torch.cat([s[n:] for s, n in zip(seqs, COUNTS)]), [more] * len(COUNTS))
    assert _apart(rest, torch.cat([f[n:] for f, n in zip(full, COUNTS)])) < 2e-2
    gdn.sync_check()


def test_serving_matches_training_pass(ex):
    model = ex.Decoder(dtype=torch.float32)
    x = _tokens(200, 5).cuda()
    got = ex.Serving(model, 1).extend(x, [200])
    with torch.no_grad():
        want = model(x[None])[0]
    assert _apart(got, want) < 0.25
    gdn.sync_check()


def test_training_learns(ex):
    """Gradients reach every weight, and the loss falls."""
    model = ex.Decoder()
    losses = ex.train(model, 12, T=128)
    assert losses[-1] < losses[0] - 0.3
    assert all(p.grad.abs().max() > 0 for p in model.parameters())
    gdn.sync_check()
