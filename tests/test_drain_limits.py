"""Waits for products and copies in flight at a CTA's end (CPU, by reading the sources): none of
them may be cut short by GDN_OPT_WAIT_LIMIT, which may just have run out in the same CTA."""
import glob
import os
import re

from gated_deltanet_recurrence_gdn_gb300 import _build

WAIT = re.compile(r"mbar_wait\(([^;]*)\);")


def test_drains_have_a_bound_of_their_own():
    seen = 0
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu*")):
        with open(path) as f:
            for args in WAIT.findall(f.read()):
                if "DRAIN" in args or "armed" in args:
                    seen += 1
                    assert args.endswith("kDrainLimit"), (os.path.basename(path), args)
    assert seen >= 11
