"""examples/tp_layer.py: prompts, then decode steps, through projection,
rotation and append, attention, output projection and the fused norms, on 2
and 8 ranks, against the same block in fp64."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("ranks", [2, 8])
def test_the_example_agrees_with_the_plain_block(ranks):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "tp_layer.py"), "--ranks", str(ranks), "--check"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("relative error") == 4
