"""The 8-bit cache's and the beam search's calls on two streams at once, and in two graphs whose
replays take turns: each has scratch of its own, and gives the same bits as alone."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from tests import attention8_ref as R8
from tests.test_kv8_attn_gpu import queries

pytestmark = pytest.mark.gpu


def attention(seed, heads):
    c = R8.Cache8([5000, 77, 1234 + seed], 2, 64, 128, seed=seed)
    q = queries(3, heads, 128, torch.bfloat16, "thd", seed)
    out = torch.zeros_like(q)
    return lambda: gdn.gdn_kv8_attn(q, c.pages, c.table_t, c.len_t, out=out), (out,)


def select(seed, V):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(6, 5, V, generator=g, device="cuda").bfloat16()
    s = -torch.rand(6, 5, generator=g, device="cuda")
    out = tuple(torch.zeros(6, 7, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
    return lambda: gdn.gdn_beam_select(x, s, 7, out=out), out


def reorder(seed, n):
    g = torch.Generator(device="cuda").manual_seed(seed)
    start = torch.randn(12, n, generator=g, device="cuda")
    state, out = start.clone(), torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    slots = torch.randperm(12, generator=g, device="cuda").int().view(3, 4)
    parent = torch.randint(0, 4, (3, 4), generator=g, device="cuda").int()

    def call():
        state.copy_(start)
        gdn.gdn_beam_reorder(parent, slots, states=[state], out=out)
    return call, (state, out)


def append(seed, n):
    c = R8.Cache8([n + 9, n + 40], 2, 32, 64, new=[n, n], seed=seed)
    k = queries(2 * n, 2, 64, torch.float32, "thd", seed)
    start = c.pages.clone()

    def call():
        c.pages.copy_(start)
        gdn.gdn_kv8_append(c.pages, k, k, c.table_t, c.len_t)
    return call, (c.pages,)


PAIRS = [(attention, (1, 8), (2, 8)), (attention, (3, 64), (4, 64)), (attention, (5, 8), (6, 64)),
         (select, (1, 50257), (2, 32000)), (select, (3, 1000), (4, 128256)), (reorder, (1, 4096), (2, 65536)),
         (append, (1, 1), (2, 70))]


@pytest.mark.parametrize("make,a,b", PAIRS)
def test_two_at_once(make, a, b):
    calls = [make(*a), make(*b)]
    want = []
    for call, outs in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (call, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        assert all(torch.equal(x, y) for x, y in zip(outs, w))
    graphs = []
    for call, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _, outs in calls:
        for t in outs:
            t.zero_()
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        assert all(torch.equal(x, y) for x, y in zip(outs, w))
    gdn.sync_check()
