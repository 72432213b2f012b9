"""Attention, norms and rotation, and distillation under the checked build
(liblin_checked.so: rows, heads, ring stages, parts and units checked before
each access): the tests of these operators run again on it, each of which ends
with the device status, so that a failed check fails its test."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import os, sys
import pytest
sys.path.insert(0, sys.argv[1])
from transformer_linear_layer_tcgen05_gb300 import build, lin
build.build_library(checked=True)
build.build_calls()
assert lin.LIB_PATH == build.CHECKED_LIB_PATH, lin.LIB_PATH
status = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *sys.argv[2:]])
assert lin.lin_get_device_status() == lin.LIN_SUCCESS, lin.lin_last_device_check()
with open("/proc/self/maps") as f:
    assert "liblin_checked.so" in f.read()
sys.exit(status)
"""

SUITES = {
    "attention": ["tests/test_attention_gpu.py", "tests/test_attention_edges_gpu.py"],
    "norms and rotation": ["tests/test_qk_norm_rope_gpu.py"],
    "distillation": ["tests/test_distill_gpu.py", "tests/test_distill_rows_gpu.py"],
    "a step": ["tests/test_decoder_block_example_gpu.py"],
}


@pytest.mark.parametrize("suite", SUITES)
def test_under_the_checked_build(suite):
    files = [os.path.join(ROOT, f) for f in SUITES[suite]]
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, *files],
                       env=dict(os.environ, LIN_CHECKED="1"), cwd=ROOT, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:]
    assert " passed" in r.stdout
