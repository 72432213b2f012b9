"""Attention with a form of the scores, norms around a block, rotation by axes
and AdamW under the checked build (liblin_checked.so): the tests of these
operators run again on it, each of which ends with the device status, so that a
failed check fails its test."""

import os
import subprocess
import sys

import pytest

from tests.test_checked_step_gpu import CHILD, ROOT

pytestmark = pytest.mark.gpu

SUITES = {
    "attention with scores": ["tests/test_attention_scores_gpu.py"],
    "block norms and rotation by axes": ["tests/test_block_norms_gpu.py", "tests/test_rope_axes_gpu.py"],
    "adamw": ["tests/test_adamw_gpu.py"],
    "a step": ["tests/test_gated_block_example_gpu.py"],
}


@pytest.mark.parametrize("suite", SUITES)
def test_under_the_checked_build(suite):
    files = [os.path.join(ROOT, f) for f in SUITES[suite]]
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *files],
                       env=dict(os.environ, LIN_CHECKED="1"), cwd=ROOT, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " passed" in r.stdout
