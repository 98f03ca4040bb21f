"""The hybrid decoder of examples/ served from a cache in 8 bits and by beam search: append,
attention, gdn_decode, selection and reordering together, as a user runs them.

Tolerances (fp32 rows).  An e4m3 number is off by at most 2^-4 of itself, so a cached row by
2^-4 / sqrt(3) = 3.6 % where errors are spread evenly; keys (so scores, of order 1, and weights) and
values: sqrt(2) * 0.036 = 5 %, next to the residual stream: 0.09 against the pass without a cache
(0.25 there is in 4 bits, for 10 % of a row).  Chunks and single tokens of the same sequence differ
by fp32's rounding, which moves a cached number by a step where it lies that close to a boundary
(1e-4 of the numbers, an eighth of their size at most: 1.3e-3 of a row), and by second roundings of
what lies below 2^-14 of its block's largest (2^-10 / 448 of that at most): 2e-2, as in 4 bits."""
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
def test_tokens_match_chunks_in_8_bits(ex, layers):
    model = ex.Decoder(layers=layers, dtype=torch.float32)
    more = 9
    seqs = [_tokens(n + more, 10 + n).cuda() for n in COUNTS]
    full = ex.Serving(model, len(COUNTS), bits=8).extend(torch.cat(seqs), [n + more for n in COUNTS])
    full = full.split([n + more for n in COUNTS])
    one = ex.Serving(model, len(COUNTS), bits=8)
    got = one.extend(torch.cat([s[:n] for s, n in zip(seqs, COUNTS)]), COUNTS).split(COUNTS)
    for b, n in enumerate(COUNTS):
        assert _apart(got[b], full[b][:n]) < 2e-2
    for j in range(more):
        got = one.step(torch.stack([s[n + j] for s, n in zip(seqs, COUNTS)]))
        assert _apart(got, torch.stack([f[n + j] for f, n in zip(full, COUNTS)])) < 2e-2
    gdn.sync_check()


def test_8_bits_match_the_training_pass(ex):
    model = ex.Decoder(dtype=torch.float32)
    x = _tokens(200, 5).cuda()
    got = ex.Serving(model, 1, bits=8).extend(x, [200])
    with torch.no_grad():
        want = model(x[None])[0]
    assert _apart(got, want) < 0.09
    gdn.sync_check()


@pytest.mark.parametrize("layers,bits,eos", [("gag", 8, None), ("gag", 4, None), ("aga", 8, 7)])
def test_beams_are_their_own_sequences(ex, layers, bits, eos):
    """After a search of many steps every beam's next logits and its score are those of its tokens
    run through a cache of their own in one pass: states, tables and pages went with it."""
    W, steps = 5, 21
    model = ex.Decoder(layers=layers, dtype=torch.float32)
    prompts = [_tokens(n, 20 + n).cuda() for n in COUNTS]
    search = ex.BeamServing(model, len(COUNTS), W, bits, eos)
    search.start(torch.cat(prompts), COUNTS)
    for _ in range(steps - 1):
        search.step()
    gdn.sync_check()
    seqs, scores = search.sequences(), search.scores.clone()
    assert torch.all(scores[:, :-1] >= scores[:, 1:])
    assert len({tuple(x) for b in seqs.tolist() for x in b}) > len(COUNTS)      # beams differ
    with torch.no_grad():
        got = search._token()                                               # the next logits
    whole = [torch.cat([p, seqs[b, w]]) for b, p in enumerate(prompts) for w in range(W)]
    counts = [len(x) for x in whole]
    ref = ex.Serving(model, len(whole), bits=bits)
    logits = ref.extend(torch.cat(whole), counts).split(counts)
    assert _apart(got, torch.stack([x[-1] for x in logits])) < 2e-2
    for i, x in enumerate(logits):
        n = COUNTS[i // W]
        each = x[n - 1:n - 1 + steps].log_softmax(-1).gather(1, seqs[i // W, i % W][:, None])[:, 0]
        if eos is not None:      # (a finished beam goes on for nothing)
            end = (seqs[i // W, i % W] == eos).cumsum(0)
            each = torch.where((end == 0) | ((end == 1) & (seqs[i // W, i % W] == eos)), each, 0.0)
        # each term is off by twice what its logits are, 2e-2 of their root mean square (below 2 here)
        bound = steps * 2 * 2e-2 * x.pow(2).mean(-1).sqrt().max().item()
        assert abs(each.sum().item() - scores[i // W, i % W].item()) < bound
    gdn.sync_check()
