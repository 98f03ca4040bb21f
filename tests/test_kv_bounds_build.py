"""The cache's translation units compile in the debug bounds-check build, and keep their barriers where
it looks for them: in dynamic shared memory (CPU)."""
import os
import re
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from gated_deltanet_recurrence_gdn_gb300 import _build

UNITS = ["gdn_kv.cu", "gdn_kv_attn.cu", "gdn_kv_attn_tc.cu", "gdn_rope.cu", "gdn_selftest.cu"]


@pytest.mark.skipif(shutil.which(_build.NVCC) is None, reason="nvcc not available")
def test_units_compile_with_checks():
    with tempfile.TemporaryDirectory() as tmp:
        def compile_one(name):
            cmd = [_build.NVCC] + _build._flags() + _build.VARIANTS["check"] + [
                "-c", os.path.join(_build.CSRC, name), "-o", os.path.join(tmp, name + ".o")]
            r = subprocess.run(cmd, capture_output=True, text=True)
            return name, r.returncode, r.stdout + r.stderr

        with ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
            results = list(ex.map(compile_one, UNITS))
    failed = [(n, out[-2000:]) for n, rc, out in results if rc != 0]
    assert not failed, failed


@pytest.mark.parametrize("name", ["gdn_kv_attn.cu", "gdn_kv_attn_tc.cu"])
def test_barriers_lie_in_dynamic_shared_memory(name):
    # (the checks accept no other; a static one would never be initialised there)
    with open(os.path.join(_build.CSRC, name)) as f:
        text = f.read()
    assert not re.search(r"(?<!extern )__shared__[^;]*\buint64_t\b", text)
