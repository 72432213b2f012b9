"""How the distillation kernel lays rows out over CTAs and shared memory
(lin_distill.h), compiled for the CPU with the host C++ compiler and checked
over its whole range (tests/distill_layout_check.cpp): rows covered, and within
the shared memory of a CTA for every number of entries. No GPU."""

import os
import shutil
import subprocess

import pytest

from tests.test_host_logic import ROOT, _cuda_include


def test_rows_fit_shared_memory(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    inc = _cuda_include()
    if not cxx or not inc:
        pytest.skip("needs a host C++ compiler and the CUDA headers")
    exe = tmp_path / "distill_layout_check"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I",
                    os.path.join(ROOT, "transformer_linear_layer_tcgen05_gb300", "csrc"),
                    "-I", inc, os.path.join(ROOT, "tests", "distill_layout_check.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
