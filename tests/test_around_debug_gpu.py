"""The operators around the feed-forward block under the -DHGEMM_DEBUG build,
in a process of its own (the library variant is chosen when it is loaded)."""

import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.gpu
def test_operators_in_the_debug_build():
    env = dict(os.environ, HGEMM_LIBRARY_VARIANT="debug")
    r = subprocess.run([sys.executable, os.path.join(HERE, "around_debug_cases.py")], env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, f"{r.stdout[-2000:]}\n{r.stderr[-4000:]}"
    assert "the operators around the block clean" in r.stdout
