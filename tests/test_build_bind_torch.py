"""The binding's native part is built again for another PyTorch, Python or compiler, whatever their files'
dates say (CPU: a PyTorch that is a version.py, and a compiler that writes an empty file)."""
from __future__ import annotations

import os
import shutil
import sys

import pytest

from gated_deltanet_recurrence_gdn_gb300 import _build

pytestmark = pytest.mark.skipif(shutil.which(_build.NVCC) is None, reason="nvcc not available")


def test_another_pytorch_is_another_build(monkeypatch, tmp_path):
    _build.build()
    bind, at = str(tmp_path / "_bind.so"), tmp_path / "torch"
    at.mkdir()
    version = at / "version.py"
    version.write_text("__version__ = '1'")
    os.utime(version, (1, 1))
    monkeypatch.setattr(_build, "BIND", bind)
    monkeypatch.setattr(_build, "BIND_MADE_OF", str(tmp_path / "bind.txt"), raising=False)
    monkeypatch.setattr(_build, "_torch", lambda: str(at))
    flags = ["-O2"]
    monkeypatch.setattr(_build, "_bind_job", lambda *a: [
        sys.executable, "-c", "open(%r, 'a').close()" % a[-1]] + flags)

    def built():
        if os.path.exists(bind):
            os.utime(bind, (2 ** 31, 2 ** 31))       # (newer than everything)
        before = os.path.getmtime(bind) if os.path.exists(bind) else None
        assert _build.build() == _build.LIB
        return os.path.getmtime(bind) != before

    assert built() and not built()
    version.write_text("__version__ = '2'")
    os.utime(version, (1, 1))                        # another PyTorch, older in time
    assert built() and not built()
    flags.append("-O3")
    assert built() and not built()
    os.remove(bind)
    assert built() and not built()
