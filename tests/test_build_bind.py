"""The library is built without what only the binding's native part needs (CPU: a compiler that fails,
no PyTorch)."""
from __future__ import annotations

import os
import shutil
import sys

import pytest

from gated_deltanet_recurrence_gdn_gb300 import _build

pytestmark = pytest.mark.skipif(shutil.which(_build.NVCC) is None, reason="nvcc not available")


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """Another _bind.so than the tree's; the library is built as it is."""
    _build.build()
    bind = str(tmp_path / "_bind.so")
    monkeypatch.setattr(_build, "BIND", bind)
    return bind


@pytest.mark.parametrize("there", [False, True])
@pytest.mark.parametrize("job", [[sys.executable, "-c", "raise SystemExit('no header')"], ["no-such-compiler"]])
def test_without_a_compiler_for_it(job, there, elsewhere, monkeypatch):
    if there:                                   # one that is out of date is not left to be loaded
        open(elsewhere, "w").close()
        os.utime(elsewhere, (1, 1))
    monkeypatch.setattr(_build, "_bind_job", lambda *a: job)
    with pytest.warns(RuntimeWarning, match="native part is not built"):
        assert _build.build() == _build.LIB
    assert os.listdir(os.path.dirname(elsewhere)) == [] and os.path.exists(_build.LIB)


def test_without_pytorch(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "_torch", lambda: None)
    with pytest.warns(RuntimeWarning, match="no PyTorch"):
        assert _build.build() == _build.LIB
    assert not os.path.exists(elsewhere)
