"""The binding's native part (csrc/gdn_bind.cpp) against its Python part: the same calls give the same
bits by either, the usual ones go by the native part alone, and whatever Python refuses is refused
before anything is written."""
from __future__ import annotations

import itertools

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import attention, beams

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float32]


@pytest.fixture
def native_only(monkeypatch):
    def never(*a):
        raise AssertionError("the Python part made the call")
    monkeypatch.setattr(attention, "_call", never)
    monkeypatch.setattr(beams, "_call", never)


def python_only(monkeypatch):
    class No:
        def __getattr__(self, name):
            return lambda *a: NotImplemented
    monkeypatch.setattr(attention, "_native", No)
    monkeypatch.setattr(beams, "_native", No)


class Cache:
    """3 sequences of 2 new tokens each, in pages of 32."""

    def __init__(self, bits, dt, d=64, H=2, Hq=4, layout="thd"):
        g = torch.Generator(device="cuda").manual_seed(7)
        self.kind = "gdn_kv8_" if bits == 8 else "gdn_kv_"
        self.pages = getattr(gdn, self.kind + "pages")(12, H, 32, d)
        self.table = torch.randperm(12, generator=g, device="cuda").int().view(3, 4)
        self.len = torch.tensor([100, 2, 33], dtype=torch.int32, device="cuda")
        self.cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
        self.scale = torch.rand(2, H, generator=g, device="cuda") + 0.5

        def rows(heads):
            x = torch.randn(6, heads, d, generator=g, device="cuda").to(dt)
            return x if layout == "thd" else x.transpose(0, 1).contiguous().transpose(0, 1)
        self.q, self.k, self.v = rows(Hq), rows(H), rows(H)
        self.cos, self.sin = gdn.gdn_rope_table(128, d)
        self.pos = torch.tensor([98, 99, 0, 1, 31, 32], dtype=torch.int32, device="cuda")
        self.pos3 = torch.stack([self.pos, self.pos + 1, self.pos + 2])
        self.axes = gdn.gdn_rope_axes([d // 4, d // 8, d // 8])
        self.d = d

    def call(self, what, *args, **kw):
        return getattr(gdn, self.kind + what)(*args, **kw)

    def all(self):
        """What appends, reads back and attends, with every argument in some call."""
        out = []
        at = (self.table, self.len)
        turns = [dict(), dict(cos=self.cos, sin=self.sin, pos=self.pos),
                 dict(cos=self.cos, sin=self.sin, pos=self.pos3, axes=self.axes, adjacent=True),
                 dict(cos=self.cos, sin=self.sin, pos=self.pos3, axes=list(self.axes))]
        for turn, cu, scale, q in itertools.product(turns, (None, self.cu), (None, self.scale),
                                                    (None, self.q)):
            o = None if q is None or cu is None else torch.zeros_like(q)
            r = self.call("append", self.pages, self.k, self.v, *at, q=q, cu_seqlens=cu,
                          kv_scale=scale, out=o, **turn)
            assert (r is None) == (q is None) and (o is None or r is o)
            out += [self.pages.clone()] + ([] if r is None else [r])
        for dt, cu, scale in itertools.product(DT, (None, self.cu), (None, self.scale)):
            o = None if cu is None else tuple(torch.zeros(6, self.k.shape[1], self.d, dtype=dt, device="cuda")
                                              for _ in range(2))
            r = self.call("read", self.pages, *at, 6, self.d, cu_seqlens=cu, kv_scale=scale, dtype=dt,
                          out=o)
            assert o is None or (r[0] is o[0] and r[1] is o[1])
            out += list(r)
        for cu, scale, more in itertools.product((None, self.cu), (None, self.scale), (
                dict(), dict(causal=False, window=5, scale=0.25), dict(max_len=100, max_new=2),
                dict(max_len=1 << 70, max_new=1 << 40, window=1 << 33), dict(return_lse=True))):
            o = None if cu is None else torch.zeros_like(self.q)
            r = self.call("attn", self.q, self.pages, *at, cu_seqlens=cu, kv_scale=scale, out=o, **more)
            first = r[0] if more.get("return_lse") else r
            assert first.stride() == self.q.stride() and (o is None or first is o)
            out += list(r) if isinstance(r, tuple) else [r]
        return out


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride()
        assert torch.equal(x, y)


@pytest.mark.parametrize("layout", ["thd", "htd"])
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bits", [4, 8])
def test_cache_calls(bits, dt, layout, native_only, monkeypatch):
    got = Cache(bits, dt, layout=layout).all()
    monkeypatch.undo()
    python_only(monkeypatch)
    same(got, Cache(bits, dt, layout=layout).all())


def selections():
    g = torch.Generator(device="cuda").manual_seed(8)
    out = []
    for dt in DT:
        x = torch.randn(3, 4, 1000, generator=g, device="cuda").to(dt)
        s = -torch.rand(3, 4, generator=g, device="cuda")
        done = torch.rand(3, 4, generator=g, device="cuda") < 0.3
        wide = torch.randn(12, 1024, generator=g, device="cuda").to(dt)
        for args, kw in (((x, s), {}), ((x, s, 7), {}), ((wide[:, :999], s, 1), {}),
                         ((x, s, 5), dict(done=done, eos=3)),
                         ((x, s), dict(done=done.byte(), eos=0)),
                         ((x[:, :1], s[:, :1].contiguous(), 4), {})):
            r = gdn.gdn_beam_select(*args, **kw)
            o = tuple(torch.zeros_like(t) for t in r)
            assert gdn.gdn_beam_select(*args, out=o, **kw) is o
            same(r, o)
            out += list(r)
    return out


def reorders():
    g = torch.Generator(device="cuda").manual_seed(9)
    out = []
    parent = torch.randint(0, 4, (2, 4), generator=g, device="cuda").int()
    slots = torch.randperm(8, generator=g, device="cuda").int().view(2, 4)
    own = torch.arange(24, dtype=torch.int32, device="cuda").view(8, 3)
    length = torch.tensor([40] * 4 + [70] * 4, dtype=torch.int32, device="cuda")
    table = own[slots.view(-1).long()].contiguous()
    for kind in (list, tuple):
        states = kind([torch.randn(8, 3, 16, generator=g, device="cuda"), torch.rand(8, 4, device="cuda", generator=g).double()])
        caches = kind([gdn.gdn_kv8_pages(24, 2, 32, 64).random_(generator=g)])
        for given in (False, True):
            r = gdn.gdn_beam_reorder(parent, slots, states=states, out=torch.zeros_like(slots) if given else None)
            kw = dict(page_table=table, own_pages=own, kv_len=length, page_size=32)
            o = (torch.zeros_like(slots), torch.zeros_like(table)) if given else None
            s, t = gdn.gdn_beam_reorder(parent, slots, states=states, caches=caches, out=o, **kw)
            u, w = gdn.gdn_beam_reorder(parent, slots, **kw)
            assert not given or (s is o[0] and t is o[1])
            out += [r, s, t, u, w] + [x.clone() for x in states] + [x.clone() for x in caches]
    return out


@pytest.mark.parametrize("calls", [selections, reorders])
def test_beam_calls(calls, native_only, monkeypatch):
    got = calls()
    monkeypatch.undo()
    python_only(monkeypatch)
    same(got, calls())


def refused(monkeypatch, fn, kw):
    """That both parts refuse, with the same words."""
    with pytest.raises((ValueError, gdn.GdnError)) as a:
        fn(**kw)
    with monkeypatch.context() as m:
        python_only(m)
        with pytest.raises((ValueError, gdn.GdnError)) as b:
            fn(**kw)
    assert a.type is b.type and str(a.value) == str(b.value)


def test_refusals_of_the_cache(monkeypatch):
    c = Cache(8, torch.bfloat16)
    before = c.pages.clone()
    at = dict(page_table=c.table, kv_len=c.len)
    short, wrong = c.table[:2], c.table.long()
    good = dict(pages=c.pages, k=c.k, v=c.v, **at)
    for bad in (dict(page_table=short), dict(page_table=wrong), dict(page_table=c.table.t()),
                dict(kv_len=c.len.float()), dict(kv_len=c.len[:2]), dict(kv_len=c.len.cpu()),
                dict(v=c.v.float()), dict(v=c.v[:5]), dict(k=c.k[:, :1]), dict(k=c.k.half(), v=c.v.half()),
                dict(k=c.k[..., :32], v=c.v[..., :32]), dict(k=c.k.cpu(), v=c.v.cpu()),
                dict(pages=c.pages.int()), dict(pages=c.pages[..., :-1]), dict(pages=c.pages.cpu()),
                dict(cu_seqlens=c.cu[:3]), dict(cu_seqlens=c.cu.long()), dict(kv_scale=c.scale[:1]),
                dict(kv_scale=c.scale.double()), dict(kv_scale=c.scale.t().contiguous().t()),
                dict(q=c.q.float()), dict(q=c.q[:, :, ::2]), dict(q=c.q, out=c.q[:3]), dict(out=c.q),
                dict(cos=c.cos), dict(cos=c.cos, sin=c.sin), dict(adjacent=True), dict(axes=c.axes),
                dict(cos=c.cos, sin=c.sin[:5], pos=c.pos), dict(cos=c.cos.double(), sin=c.sin, pos=c.pos),
                dict(cos=c.cos, sin=c.sin, pos=c.pos[:4]), dict(cos=c.cos, sin=c.sin, pos=c.pos.long()),
                dict(cos=c.cos, sin=c.sin, pos=c.pos3), dict(cos=c.cos, sin=c.sin, pos=c.pos3, axes=c.axes[:5]),
                dict(cos=c.cos, sin=c.sin, pos=c.pos3, axes=[0, 256] * 16),
                dict(cos=c.cos, sin=c.sin, pos=c.pos3, axes=[7] * 32)):
        refused(monkeypatch, gdn.gdn_kv8_append, {**good, **bad})
    assert torch.equal(c.pages, before)
    good = dict(pages=c.pages, n_tokens=6, d=64, **at)
    for bad in (dict(n_tokens=5), dict(n_tokens=-3), dict(d=96), dict(d=0), dict(dtype=torch.float16),
                dict(out=(c.k, c.v.float())), dict(out=(c.k[:5], c.v)), dict(page_table=short)):
        refused(monkeypatch, gdn.gdn_kv8_read, {**good, **bad})
    good = dict(q=c.q, pages=c.pages, **at)
    for bad in (dict(q=c.q.half()), dict(q=c.q[0]), dict(q=c.q[:5]), dict(out=c.q.float()),
                dict(out=c.q[:3]), dict(pages=gdn.gdn_kv_pages(12, 2, 32, 64)), dict(page_table=wrong)):
        refused(monkeypatch, gdn.gdn_kv8_attn, {**good, **bad})
    for bad in (dict(window=-1), dict(max_len=-1), dict(max_new=-1), dict(q=c.q[:, :3])):
        refused(monkeypatch, gdn.gdn_kv8_attn, {**good, **bad})      # (by the library)


def test_refusals_of_the_beams(monkeypatch):
    x, s = torch.zeros(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    done = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    good = dict(logits=x, scores=s)
    outs = tuple(torch.zeros(2, 3, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32))
    for bad in (dict(logits=x.half()), dict(logits=x[:1]), dict(logits=x[..., ::2]), dict(logits=x.cpu()),
                dict(scores=s.double()), dict(scores=s.view(-1)), dict(scores=s.t().contiguous().t()),
                dict(n=0), dict(n=151), dict(done=done), dict(eos=1), dict(done=done, eos=50),
                dict(done=done, eos=-1), dict(done=done.int(), eos=1), dict(done=done[:1], eos=1),
                dict(out=(outs[0], outs[1], outs[0])), dict(n=2, out=outs),
                dict(logits=torch.zeros(2, 4, 50, device="cuda")[:, :3])):
        refused(monkeypatch, gdn.gdn_beam_select, {**good, **bad})
    refused(monkeypatch, gdn.gdn_beam_select, dict(logits=x, scores=s, n=33))
    parent = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    state = torch.rand(6, 8, device="cuda")
    own = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    length = torch.full((6,), 20, dtype=torch.int32, device="cuda")
    good = dict(parent=parent, slots=slots, states=[state])
    paged = dict(page_table=own.clone(), own_pages=own, kv_len=length, page_size=16)
    kept = state.clone()
    for bad in (dict(parent=parent.long()), dict(slots=slots[:1]), dict(slots=slots.cpu()), dict(states=[]),
                dict(states=[state, state[:5]]), dict(states=[state.cpu()]), dict(states=[state[:, ::2]]),
                dict(page_table=own), dict(caches=[own]), dict(out=slots), dict(out=parent),
                dict(out=slots.long()), {**paged, "own_pages": own[:5]}, {**paged, "own_pages": own[:, :1]},
                {**paged, "kv_len": length[:5]}, {**paged, "page_table": own[:5]},
                {**paged, "out": (slots.clone(), own)}, {**paged, "out": (slots.clone(), own[:5].clone())},
                {**paged, "caches": [own.t()]}):
        refused(monkeypatch, gdn.gdn_beam_reorder, {**good, **bad})
    refused(monkeypatch, gdn.gdn_beam_reorder, {**good, **paged, "page_size": 17})
    assert torch.equal(state, kept)


def test_what_is_rarer_goes_by_python():
    c = Cache(8, torch.bfloat16)
    c.call("append", c.pages, c.k, c.v, c.table, c.len)
    want = c.call("attn", c.q, c.pages, c.table, c.len, scale=1.0)
    assert torch.equal(c.call("attn", c.q, c.pages, c.table, c.len, scale=1), want)
    k, v = c.call("read", c.pages, c.table, c.len, 6, 64)
    o = [torch.zeros_like(k), torch.zeros_like(v)]
    c.call("read", c.pages, c.table, c.len, 6, 64, out=o)
    assert torch.equal(o[0], k) and torch.equal(o[1], v)
    x = torch.rand(6, 8, device="cuda")
    parent = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    gdn.gdn_beam_reorder(parent, slots, states=(t for t in [x]))
    assert torch.equal(x[1], x[0]) and torch.equal(x[5], x[3])
    w = torch.nn.Parameter(c.q.float())        # rows that want a gradient: the result does not
    c4 = Cache(8, torch.float32)
    assert not c4.call("attn", w, c4.pages, c4.table, c4.len).requires_grad


def test_another_stream_and_a_graph():
    c = Cache(8, torch.bfloat16)
    c.call("append", c.pages, c.k, c.v, c.table, c.len)
    want = c.call("attn", c.q, c.pages, c.table, c.len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.call("attn", c.q, c.pages, c.table, c.len)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.call("attn", c.q, c.pages, c.table, c.len)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
