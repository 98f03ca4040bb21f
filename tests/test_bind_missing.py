"""Without the binding's native part (_bind.so) the calls that it makes are Python's (CPU: tensors that
say they lie on a GPU, and the call itself left out)."""
from __future__ import annotations

import sys

import pytest
import torch

import gated_deltanet_recurrence_gdn_gb300 as gdn
from gated_deltanet_recurrence_gdn_gb300 import attention, beams
from tests import test_attention_devices as D
from tests import test_beam_abi as B


@pytest.fixture
def without(monkeypatch):
    monkeypatch.setitem(sys.modules, gdn.__name__ + "._bind", None)      # (an import of it fails)
    monkeypatch.delattr(gdn, "_bind", raising=False)
    monkeypatch.setattr(attention, "_native_kept", None)


@pytest.mark.parametrize("make", [D.append, D.read, D.attn, B.select, B.reorder])
def test_calls_are_made_and_refused_without_it(make, without, monkeypatch):
    calls = []
    for module in (attention, beams):
        monkeypatch.setattr(module, "_call", lambda *a: calls.append(a))
    _, call = make(lambda n, t: D.On(t, 0))
    with pytest.warns(RuntimeWarning, match="native part"):
        call()
    assert len(calls) == 1
    call()                                              # (it says so once)
    assert len(calls) == 2
    names, _ = make(lambda n, t: D.On(t, 0))
    for other in names:
        _, call = make(lambda n, t: D.On(t, -1 if n == other else 0))
        with pytest.raises(ValueError):
            call()
    assert len(calls) == 2


def test_host_tensors_are_refused_without_it(without):
    with pytest.warns(RuntimeWarning, match="native part"), pytest.raises(ValueError):
        gdn.gdn_beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2))
