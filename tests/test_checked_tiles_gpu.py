"""Attention with a form of the scores in two tiles to a CTA, and over documents,
under the checked build (liblin_checked.so): some of these tests run again on it,
each of which ends with the device status, so that a failed check fails its test."""

import os
import subprocess
import sys

import pytest

from tests.test_checked_step_gpu import CHILD, ROOT

pytestmark = pytest.mark.gpu


def test_under_the_checked_build():
    files = [os.path.join(ROOT, "tests", f"test_attention_score_{f}_gpu.py") for f in ("tiles", "documents")]
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *files, "-k", "ranges or nobodys or 64"],
                       env=dict(os.environ, LIN_CHECKED="1"), cwd=ROOT, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " passed" in r.stdout
