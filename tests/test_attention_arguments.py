"""What the attention layer's binding refuses by itself (CPU: tensors that say they lie on a GPU, and the
call itself left out)."""
import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import attention as A
from tests.test_attention_devices import On, bf, i32


def on(*shape, dtype=bf):
    return On(torch.zeros(*shape, dtype=dtype), 0)


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(A, "_call", lambda *a: made.append(a))
    return made


def cache():
    return (on(5, 2, 16 * 72, dtype=torch.uint8), on(2, 3, dtype=i32), on(2, dtype=i32))


def append(**kw):
    pages, table, length = cache()
    return gdn.gdn_kv_append(pages, on(4, 2, 64), on(4, 2, 64), table, length, **kw)


TURN = dict(cos=on(8, 32, dtype=torch.float32), sin=on(8, 32, dtype=torch.float32), pos=on(4, dtype=i32))


def test_append_turns_or_is_not_asked_to(calls):
    append()
    append(**TURN)
    append(q=on(4, 4, 64), out=on(4, 4, 64), **TURN)
    append(axes=bytes(32), **dict(TURN, pos=on(1, 4, dtype=i32)))
    assert len(calls) == 4 and [c[9] is None for c in calls] == [True, False, False, False]


@pytest.mark.parametrize("left", [("cos",), ("sin",), ("pos",), ("cos", "sin"), ("cos", "pos"), ("sin", "pos")])
def test_append_refuses_half_a_turn(calls, left):
    # (keys would be stored as they are, and read as if turned)
    with pytest.raises(ValueError):
        append(**{n: t for n, t in TURN.items() if n not in left})
    assert not calls


@pytest.mark.parametrize("kw", [dict(axes=bytes(32)), dict(adjacent=True), dict(out=on(4, 4, 64))])
def test_append_refuses_what_it_has_no_use_for(calls, kw):
    with pytest.raises(ValueError):
        append(**kw)
    assert not calls


def test_rope_writes_both_or_one(calls):
    q, k, pos = on(2, 4, 3, 64), on(2, 2, 3, 64), on(3, dtype=i32)
    at = (TURN["cos"], TURN["sin"], pos)
    gdn.gdn_rope(q, k, *at, out=(q, k))
    gdn.gdn_rope(q, None, *at, out=(q, None))
    for a, b in ((k, None), (None, k)):
        with pytest.raises(ValueError):
            gdn.gdn_rope(q, a, *at, out=(q, b))
    assert len(calls) == 2


@pytest.mark.parametrize("call", [
    lambda: gdn.gdn_kv_read(*cache(), 4, 0),
    lambda: gdn.gdn_kv_read(*cache(), 4, -64),
    lambda: gdn.gdn_kv_read(*cache(), -2, 64),
    lambda: gdn.gdn_kv_read(*cache(), 4, 64, dtype=torch.float16),
    lambda: gdn.gdn_kv_attn(on(4, 4, 0), *cache()),
    lambda: gdn.gdn_kv_attn(on(4, 4, 64), on(5, 2, 0, dtype=torch.uint8), *cache()[1:]),
    lambda: append(q=on(4), out=on(4)),
    lambda: append(q=on(4, 4, 1, 64), out=on(4, 4, 1, 64)),
    lambda: gdn.gdn_rope(on(2, 4, 3, 64), on(3), *(TURN["cos"], TURN["sin"], on(3, dtype=i32)),
                         out=(on(2, 4, 3, 64), on(3))),
    lambda: gdn.gdn_rope_table(4, 63, device="cpu"),
    lambda: gdn.gdn_rope_table(4, -2, device="cpu"),
    lambda: gdn.gdn_rope_table(-1, 64, device="cpu"),
    lambda: gdn.gdn_rope_axes((8, -1, 8)),
], ids=lambda c: None)
def test_refusals_are_value_errors(calls, call):
    with pytest.raises(ValueError):
        call()
    assert not calls


def test_negative_sections_dealt_out_end():
    # (dealing out in turn never came to an end: nothing was left to run out)
    with pytest.raises(ValueError):
        gdn.gdn_rope_axes((2, -1), interleave=True)
