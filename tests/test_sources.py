"""What the kernels' sources keep to, whatever a program does with the library."""
import glob
import os

from top_hs2_fa_gb300 import build


def test_no_multicast():
    """No load and no arrival goes to several CTAs at once: the one library is what every rank of a
    program on several devices loads, over pools that the caller chooses."""
    files = sorted(f for f in glob.glob(os.path.join(build.CSRC, "*")) if f.endswith((".cu", ".cuh", ".h")))
    assert len(files) > 20
    for f in files:
        with open(f, encoding="utf-8") as fh:
            assert "multicast" not in fh.read(), f
