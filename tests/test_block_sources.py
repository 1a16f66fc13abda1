"""Properties of the kernels' sources that no run on one GPU can show (CPU)."""

import glob
import os
import re

from tensor_core_dense_fp16_gb300 import build as tcbuild

CSRC = os.path.join(os.path.dirname(tcbuild.__file__), "csrc")


def sources():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")))
    assert files
    return {os.path.basename(f): open(f, encoding="utf-8").read() for f in files}


def code(text):
    """The text without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_load_is_multicast():
    """An operand may be memory of another GPU, where a multicast load is not
    safe: every CTA loads for itself (commits may be multicast)."""
    for name, text in sources().items():
        for call in re.findall(r"asm volatile\((.*?)\);", code(text), flags=re.S):
            assert not ("cp.async.bulk" in call and "multicast" in call), name
