"""gdn_beam_reorder against a plain form of its definition: lanes, states, page tables and pages, all
bit for bit, and what it leaves alone."""
from __future__ import annotations

import random

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def definition(parent, slots, lens=None, table=None, own=None, page=0):
    """New slots and table as lists, and the copies: lanes (from, to), pages (from, to)."""
    B, W = len(parent), len(parent[0])
    new, lanes, pages = [list(s) for s in slots], [], []
    rows = None if table is None else [list(r) for r in table]
    for b in range(B):
        free = [slots[b][i] for i in range(W) if i not in parent[b]]
        seen = set()
        for i, p in enumerate(parent[b]):
            if rows is not None:
                rows[b * W + i] = list(table[b * W + p])
            if p not in seen:
                seen.add(p)
                new[b][i] = slots[b][p]
                continue
            new[b][i] = free.pop(0)
            lanes.append((slots[b][p], new[b][i]))
            if rows is not None:
                at, part = divmod(lens[b * W + p], page)
                rows[b * W + i][at:] = own[new[b][i]][at:]
                if part:
                    pages.append((table[b * W + p][at], own[new[b][i]][at]))
    return new, rows, lanes, pages


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Beams:
    def __init__(self, B, W, spare, seed, max_pages=0, page=16, lens=None):
        r = random.Random(seed)
        self.B, self.W, self.lanes = B, W, B * W + spare
        lanes = r.sample(range(self.lanes), B * W)
        self.slots = [lanes[b * W:(b + 1) * W] for b in range(B)]
        self.page, self.table, self.own, self.lens = page, None, None, None
        if max_pages:
            ids = r.sample(range(self.lanes * max_pages + 5), self.lanes * max_pages)
            self.n_pages = self.lanes * max_pages + 5
            self.own = [ids[i * max_pages:(i + 1) * max_pages] for i in range(self.lanes)]
            self.table = [list(self.own[s]) for row in self.slots for s in row]
            each = lens if lens is not None else [r.randrange(0, max_pages * page + 1) for _ in range(B)]
            self.lens = [n for n in each for _ in range(W)]


def parents(B, W, kind, seed):
    r = random.Random(seed)
    if kind == "same":
        return [list(range(W))] * B
    if kind == "swap":
        return [list(range(W))[::-1]] * B
    if kind == "one":
        return [[r.randrange(W)] * W for _ in range(B)]
    return [[r.randrange(W) for _ in range(W)] for _ in range(B)]


def run(x, parent, states, caches, **kw):
    """One reorder of x, checked; x then holds the new slots and table."""
    new, rows, lanes, pages = definition(parent, x.slots, x.lens, x.table, x.own, x.page)
    want_s, want_c = [s.clone() for s in states], [c.clone() for c in caches]
    for s, old in zip(want_s, states):
        for a, b in lanes:
            s[b] = old[a]
    for c, old in zip(want_c, caches):
        for a, b in pages:
            c[b] = old[a]
    if x.table is not None:
        kw.update(page_table=i32(x.table), own_pages=i32(x.own), kv_len=i32(x.lens), page_size=x.page,
                  caches=caches)
    got = gdn.gdn_beam_reorder(i32(parent), i32(x.slots), states=states, check=True, **kw)
    slots, table = got if x.table is not None else (got, None)
    assert slots.tolist() == new
    if table is not None:
        assert table.tolist() == rows
    assert all(torch.equal(a, b) for a, b in zip(states + caches, want_s + want_c))
    x.slots, x.table = new, rows
    return slots


def pool(n, shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(n, *shape, generator=g, device="cuda").to(dtype)
    return torch.randint(0, 100, (n, *shape), generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("kind", ["same", "swap", "one", "mixed"])
@pytest.mark.parametrize("B,W", [(1, 1), (1, 4), (3, 32), (17, 5), (300, 3), (1, 2)])
def test_lanes_and_states(B, W, kind):
    x = Beams(B, W, 3, B + W)
    states = [pool(x.lanes, (2, 8, 8), torch.float32, 1), pool(x.lanes, (24,), torch.bfloat16, 2),
              pool(x.lanes, (16,), torch.uint8, 3)]
    for step in range(2):
        run(x, parents(B, W, kind, 10 * B + step), states, [])


@pytest.mark.parametrize("kind", ["same", "one", "mixed"])
@pytest.mark.parametrize("B,W,max_pages,page", [(1, 4, 6, 16), (5, 6, 40, 64), (9, 3, 1, 256), (2, 32, 33, 32)])
def test_tables_and_pages(B, W, max_pages, page, kind):
    x = Beams(B, W, 2, 7 * B + W, max_pages, page)
    caches = [gdn_pages(x.n_pages, 2, 64, 4), pool(x.n_pages, (1, 528), torch.uint8, 5)]
    run(x, parents(B, W, kind, B), [pool(x.lanes, (64,), torch.float32, 6)], caches)


def gdn_pages(n, heads, size, seed):
    return pool(n, (heads, size), torch.uint8, seed)


@pytest.mark.parametrize("n", [0, 15, 16, 17, 95, 96])
def test_lengths_at_page_borders(n):
    # (a full page and an empty one are not copied; at 96 there is no page left)
    x = Beams(2, 4, 1, n, 6, 16, [n, n])
    run(x, [[0, 0, 1, 1], [3, 3, 3, 3]], [], [gdn_pages(x.n_pages, 1, 80, 8)])


def test_a_search_of_many_steps():
    """Tokens written one a step, each by the beam that has them: after every reorder a beam reads its
    own history through its table, and no beam writes to a page that another one reads."""
    B, W, page, steps = 3, 5, 4, 30
    x = Beams(B, W, 2, 1, -(-steps // page), page, [0] * B)
    cache = torch.zeros(x.n_pages, page, 2, dtype=torch.int64, device="cuda")     # a token: 16 bytes
    state = torch.zeros(x.lanes, 4, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(B * W)]
    r = random.Random(2)
    for t in range(steps):
        writes = set()
        for i in range(B * W):
            at = x.table[i][t // page]
            assert at not in writes
            writes.add(at)
            cache[at, t % page] = 1000 * t + i
            history[i].append(1000 * t + i)
            state[x.slots[i // W][i % W]] = history[i][-1]
        x.lens = [t + 1] * (B * W)
        parent = parents(B, W, r.choice(["same", "swap", "one", "mixed"]), t)
        run(x, parent, [state], [cache])
        history = [list(history[b * W + parent[b][w]]) for b in range(B) for w in range(W)]
        for i in range(B * W):
            rows = cache[i32(x.table[i]).long()].flatten(0, 1)[:t + 1, 0]
            assert rows.tolist() == history[i]
            assert int(state[x.slots[i // W][i % W], 0]) == history[i][-1]


def test_a_prompt_is_shared_by_its_beams():
    """All beams go on from the first: its full pages are in every table, its last one is copied."""
    x = Beams(2, 3, 0, 3, 4, 16, [40, 33])
    cache = gdn_pages(x.n_pages, 2, 32, 9)
    first = [x.table[0][:2], x.table[3][:2]]
    run(x, [[0] * 3] * 2, [pool(x.lanes, (4,), torch.float32, 1)], [cache])
    for b in range(2):
        for w in range(3):
            row = x.table[3 * b + w]
            assert row[:2] == first[b] and row[2] == x.own[x.slots[b][w]][2]
            assert torch.equal(cache[row[2]], cache[x.table[3 * b][2]])


@pytest.mark.parametrize("n", [1, 63, 64, 65, 130])
def test_many_layers(n):
    # more pools than one launch takes
    x = Beams(4, 4, 0, n, 3, 16)
    states = [pool(x.lanes, (4 * (1 + i % 5),), torch.float32, i) for i in range(n)]
    caches = [gdn_pages(x.n_pages, 1, 16 * (1 + i % 3), i) for i in range(n // 2)]
    run(x, parents(4, 4, "mixed", n), states, caches)


def test_many_groups():
    # more groups than one launch takes
    x = Beams(5000, 2, 0, 4, 2, 16)
    run(x, parents(5000, 2, "mixed", 5), [pool(x.lanes, (4,), torch.float32, 1)],
        [gdn_pages(x.n_pages, 1, 16, 2)])


def test_large_states_and_a_lane_past_32_bits():
    # 8 lanes of 768 MB: offsets past 2^32, many pieces of a lane
    x = Beams(1, 3, 5, 5)
    x.slots = [[7, 6, 0]]
    state = torch.zeros(8, 3 << 26, dtype=torch.float32, device="cuda")
    for lane in (7, 6, 0):
        state[lane, ::4097] = lane + 1
        state[lane, -1] = -lane
    slots = gdn.gdn_beam_reorder(i32([[0, 0, 1]]), i32(x.slots), states=[state], check=True)
    assert slots.tolist() == [[7, 0, 6]]
    assert torch.equal(state[0], state[7]) and state[0, -1] == -7 and state[6, -1] == -6


def test_outputs_streams_and_graphs():
    x = Beams(4, 4, 0, 6, 5, 16)
    parent = parents(4, 4, "mixed", 7)
    state, cache = pool(x.lanes, (64, 64), torch.float32, 1), gdn_pages(x.n_pages, 2, 64, 2)
    new, rows, lanes, pages = definition(parent, x.slots, x.lens, x.table, x.own, x.page)
    start = state.clone(), cache.clone()
    want = state.clone(), cache.clone()
    for a, b in lanes:
        want[0][b] = start[0][a]
    for a, b in pages:
        want[1][b] = start[1][a]
    # a table that is part of a wider one
    wide = torch.full((16, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:7] = i32(x.table)
    out = torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.full((16, 8), -5, dtype=torch.int32, device="cuda")
    args = dict(states=[state], caches=[cache], page_table=wide[:, 2:7], own_pages=i32(x.own),
                kv_len=i32(x.lens), page_size=16, out=(out[0], out[1][:, 1:6]))
    at = i32(parent), i32(x.slots)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()

    def on_side():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            gdn.gdn_beam_reorder(*at, **args)
        torch.cuda.current_stream().wait_stream(side)

    with torch.cuda.graph(g):
        gdn.gdn_beam_reorder(*at, **args)
    for call in (on_side, g.replay, g.replay):
        state.copy_(start[0])
        cache.copy_(start[1])
        out[0].zero_()
        out[1].fill_(-5)
        call()
        torch.cuda.synchronize()
        assert torch.equal(state, want[0]) and torch.equal(cache, want[1])
        assert out[0].tolist() == new and out[1][:, 1:6].tolist() == rows
        assert (out[1][:, 0] == -5).all() and (out[1][:, 6:] == -5).all()
    gdn.sync_check()


@pytest.mark.parametrize("what", ["parent", "parent<0", "slot", "page", "own", "len", "len<0", "lens differ"])
def test_bad_indices_are_reported(what):
    x = Beams(2, 3, 0, 8, 3, 16, [20, 20])
    parent = [[0, 0, 0], [1, 1, 2]]
    if what == "parent":
        parent[0][1] = 3
    elif what == "parent<0":
        parent[0][1] = -1
    elif what == "slot":
        x.slots[0][1] = x.lanes
    elif what == "page":
        x.table[0][1] = x.n_pages
    elif what == "own":
        x.own[x.slots[0][1]][1] = -1
    elif what == "len":
        x.lens[:3] = [49] * 3
    elif what == "len<0":
        x.lens[:3] = [-16] * 3
    else:
        x.lens[1] = 21
    state, cache = pool(x.lanes, (8,), torch.float32, 1), gdn_pages(x.n_pages, 1, 32, 2)
    before = state.clone()
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_beam_reorder(i32(parent), i32(x.slots), states=[state], caches=[cache],
                             page_table=i32(x.table), own_pages=i32(x.own), kv_len=i32(x.lens),
                             page_size=16, check=True)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    gdn.sync_check()
    # the other group went on
    a, b = x.slots[1][1], x.slots[1][0]
    assert torch.equal(state[b], before[a])


def test_nothing_to_do():
    empty = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert gdn.gdn_beam_reorder(empty, empty, states=[torch.zeros(1, 4, device="cuda")]).shape == (0, 4)
