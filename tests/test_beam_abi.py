"""Host-side refusals of the beam search's entry points and of their binding (CPU)."""
import ctypes

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import beams as Bm
from tests.test_attention_abi import FAKE, lib, ref  # noqa: F401
from tests.test_attention_devices import On, bf, i32

bad, un, al = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_ALIGNMENT


def test_select_refusals(lib):  # noqa: F811
    def f(logits=FAKE, stride=100, scores=FAKE, done=None, eos=0, outs=(FAKE, FAKE, FAKE), B=2, W=3,
          V=100, n=4, dt=1):
        return lib.gdn_beam_select(logits, stride, scores, done, eos, *outs, B, W, V, n, dt, None)

    assert f(B=0) == gdn.GDN_OK
    assert f(B=-1) == bad and f(W=0) == bad and f(V=0) == bad and f(n=0) == bad and f(dt=2) == bad
    assert f(W=33) == un and f(n=33) == un and f(B=1 << 24) == un and f(V=(1 << 22) + 1) == un
    assert f(V=1, n=4) == bad                                   # three continuations in all
    assert f(done=FAKE, eos=100) == bad and f(done=FAKE, eos=-1) == bad
    assert f(logits=None) == bad and f(scores=None) == bad
    for i in range(3):
        assert f(outs=[None if j == i else FAKE for j in range(3)]) == bad
        assert f(outs=[FAKE + 2 if j == i else FAKE for j in range(3)]) == al
    assert f(logits=FAKE + 1) == al and f(logits=FAKE + 2, dt=0) == al and f(scores=FAKE + 1) == al


def pools(*x):
    return (Bm._Pool * len(x))(*[Bm._Pool(*p) for p in x])


def tables(**kw):
    x = dict(page_table=FAKE, table_out=FAKE, own_pages=FAKE, kv_len=FAKE, max_pages=4, page_size=16,
             table_stride=4, out_stride=4, own_stride=4)
    x.update(kw)
    return Bm._Tables(*x.values())


def test_reorder_refusals(lib):  # noqa: F811
    def f(parent=FAKE, slots=FAKE, out=FAKE, B=2, W=3, lanes=6, states=((FAKE, 64, 6),), t=None,
          caches=()):
        return lib.gdn_beam_reorder(parent, slots, out, B, W, lanes, pools(*states), len(states),
                                    ref(t), pools(*caches), len(caches), None)

    page = (FAKE, 32, 9)
    assert f(B=0) == gdn.GDN_OK and f(B=0, t=tables(), caches=(page,)) == gdn.GDN_OK
    assert f(B=-1) == bad and f(W=0) == bad and f(lanes=0) == bad
    assert f(W=33) == un and f(B=(1 << 20) + 1) == un and f(states=((FAKE, 64, 6),) * 4097) == un
    assert f(parent=None) == bad and f(slots=None) == bad and f(out=None) == bad
    assert f(parent=FAKE + 2) == al and f(slots=FAKE + 1) == al and f(out=FAKE + 3) == al
    assert f(states=((FAKE, 64, 5),)) == bad                    # not a row per lane
    assert f(states=((None, 64, 6),)) == bad and f(states=((FAKE, -16, 6),)) == bad
    assert f(states=((FAKE + 8, 64, 6),)) == al and f(states=((FAKE, 24, 6),)) == al
    assert f(states=((FAKE, 1 << 50, 6),)) == un
    assert f(caches=(page,)) == bad                             # no table to go by
    for name in ("page_table", "table_out", "own_pages", "kv_len"):
        assert f(t=tables(**{name: None})) == bad and f(t=tables(**{name: FAKE + 2})) == al
    assert f(t=tables(max_pages=0)) == bad and f(t=tables(page_size=24)) == bad
    assert f(t=tables(page_size=0)) == bad and f(t=tables(max_pages=1 << 28)) == un
    assert f(t=tables(), caches=((FAKE, 20, 9),)) == al
    assert lib.gdn_beam_reorder(FAKE, FAKE, FAKE, 2, 3, 6, None, 1, None, None, 0, None) == bad
    assert lib.gdn_beam_reorder(FAKE, FAKE, FAKE, 2, 3, 6, None, 0, ref(tables()), None, 1, None) == bad
    assert ctypes.sizeof(Bm._Pool) == 24 and ctypes.sizeof(Bm._Tables) == 64


def select(m, **kw):
    x = dict(logits=torch.zeros(2, 3, 50, dtype=bf), scores=torch.zeros(2, 3),
             done=torch.zeros(2, 3, dtype=torch.bool), o0=torch.zeros(2, 4),
             o1=torch.zeros(2, 4, dtype=i32), o2=torch.zeros(2, 4, dtype=i32))
    x.update(kw)
    x = {n: m(n, t) for n, t in x.items()}
    return list(x), lambda: gdn.gdn_beam_select(x["logits"], x["scores"], 4, done=x["done"], eos=1,
                                                out=(x["o0"], x["o1"], x["o2"]))


def reorder(m, **kw):
    x = dict(parent=torch.zeros(2, 3, dtype=i32), slots=torch.zeros(2, 3, dtype=i32),
             state=torch.zeros(7, 4), cache=torch.zeros(9, 2, 16, dtype=torch.uint8),
             table=torch.zeros(6, 5, dtype=i32), own=torch.zeros(7, 5, dtype=i32),
             length=torch.zeros(6, dtype=i32), o0=torch.zeros(2, 3, dtype=i32),
             o1=torch.zeros(6, 5, dtype=i32))
    x.update(kw)
    x = {n: m(n, t) for n, t in x.items()}
    return list(x), lambda: gdn.gdn_beam_reorder(
        x["parent"], x["slots"], states=[x["state"]], caches=[x["cache"]], page_table=x["table"],
        own_pages=x["own"], kv_len=x["length"], page_size=16, out=(x["o0"], x["o1"]))


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(Bm, "_call", lambda *a: made.append(a))
    return made


@pytest.mark.parametrize("make", [select, reorder])
def test_tensors_of_a_call_share_a_device(make, calls):
    names, call = make(lambda n, t: On(t, 3))
    call()
    assert len(calls) == 1
    for other in names:
        for at in (0, -1):
            _, call = make(lambda n, t: On(t, at if n == other else 3))
            with pytest.raises(ValueError):
                call()
    _, call = make(lambda n, t: On(t, -1))
    with pytest.raises(ValueError):
        call()
    assert len(calls) == 1


on = lambda n, t: On(t, 0)  # noqa: E731


@pytest.mark.parametrize("kw", [
    dict(logits=torch.zeros(2, 3, 50, dtype=torch.float16)), dict(logits=torch.zeros(2, 2, 50)),
    dict(logits=torch.zeros(5, 50)), dict(logits=torch.zeros(6)), dict(logits=torch.zeros(2, 50, 3).transpose(1, 2)),
    dict(logits=torch.zeros(2, 5, 50)[:, :3]), dict(logits=torch.zeros(2, 3, 1)),
    dict(scores=torch.zeros(6)), dict(scores=torch.zeros(2, 3, dtype=bf)), dict(scores=torch.zeros(3, 2).t()),
    dict(done=torch.zeros(2, 3)), dict(done=torch.zeros(6, dtype=torch.bool)), dict(o0=torch.zeros(2, 3)),
    dict(o1=torch.zeros(2, 4)), dict(o2=torch.zeros(2, 4, dtype=torch.int64)),
], ids=lambda k: next(iter(k)))
def test_select_binding_refuses(calls, kw):
    with pytest.raises(ValueError):
        select(on, **kw)[1]()
    assert not calls


def test_select_binding_takes_and_refuses_the_rest(calls):
    x, s, d = On(torch.zeros(2, 3, 50), 0), On(torch.zeros(2, 3), 0), On(torch.zeros(2, 3, dtype=torch.uint8), 0)
    gdn.gdn_beam_select(x, s)
    gdn.gdn_beam_select(On(torch.zeros(6, 50), 0), s, 150 // 5)
    gdn.gdn_beam_select(On(torch.zeros(2, 3, 4, 50)[:, :, 1], 0), s, 1, done=d, eos=49)
    assert len(calls) == 3 and calls[2][5] == 200                # rows 200 apart
    for args, kw in (((0,), {}), ((151,), {}), ((-1,), {}), ((1,), dict(done=d)), ((1,), dict(eos=1)),
                     ((1,), dict(done=d, eos=50)), ((1,), dict(done=d, eos=-1))):
        with pytest.raises(ValueError):
            gdn.gdn_beam_select(x, s, *args, **kw)
    assert len(calls) == 3


@pytest.mark.parametrize("kw", [
    dict(parent=torch.zeros(6, dtype=i32)), dict(parent=torch.zeros(2, 3, dtype=torch.int64)),
    dict(slots=torch.zeros(2, 4, dtype=i32)), dict(state=torch.zeros(6, 4)), dict(state=torch.zeros(7, 8)[:, ::2]),
    dict(state=torch.zeros(())), dict(cache=torch.zeros(9, 4)[:, ::2]), dict(table=torch.zeros(5, 5, dtype=i32)),
    dict(table=torch.zeros(6, 4, dtype=i32)), dict(own=torch.zeros(6, 5, dtype=i32)),
    dict(own=torch.zeros(7, 4, dtype=i32)), dict(own=torch.zeros(7, 5)), dict(length=torch.zeros(2, dtype=i32)),
    dict(o0=torch.zeros(6, dtype=i32)), dict(o1=torch.zeros(6, 6, dtype=i32)),
], ids=lambda k: next(iter(k)))
def test_reorder_binding_refuses(calls, kw):
    with pytest.raises(ValueError):
        reorder(on, **kw)[1]()
    assert not calls


def test_reorder_binding_takes_and_refuses_the_rest(calls):
    p, s, state = On(torch.zeros(2, 3, dtype=i32), 0), On(torch.zeros(2, 3, dtype=i32), 0), On(torch.zeros(7, 4), 0)
    table, own, n = On(torch.zeros(6, 5, dtype=i32), 0), On(torch.zeros(7, 5, dtype=i32), 0), On(torch.zeros(6, dtype=i32), 0)
    gdn.gdn_beam_reorder(p, s, states=[state])
    gdn.gdn_beam_reorder(p, s, page_table=table, own_pages=own, kv_len=n, page_size=16)
    assert len(calls) == 2
    for kw in (dict(), dict(states=[state], caches=[state]), dict(page_table=table),
               dict(page_table=table, own_pages=own, kv_len=n), dict(states=[state], page_size=16),
               dict(states=[state], out=s), dict(states=[state], out=p),
               dict(page_table=table, own_pages=own, kv_len=n, page_size=16,
                    out=(On(torch.zeros(2, 3, dtype=i32), 0), table))):
        with pytest.raises(ValueError):
            gdn.gdn_beam_reorder(p, s, **kw)
    assert len(calls) == 2
