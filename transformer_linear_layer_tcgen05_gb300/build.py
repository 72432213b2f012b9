"""Build ``liblin.so`` (the C-ABI library of include/lin.h) in-tree with nvcc.

Every translation unit is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, then linked as a
shared library next to this file. Object files go to ``_build/`` at the
repository root. A rebuild happens only when a source or header is newer than
the library.

``build_calls()`` builds ``_lin_calls``, the Python extension module of the
short calls' marshalling (csrc/lin_calls.cpp), with the host compiler, for the
running interpreter and its torch (the file's name carries the interpreter's
tag). ``build_library()`` builds it beside the library where torch is installed;
the library itself needs neither torch nor Python's headers, and stands whether
the module could be built or not.

``build_library(checked=True)`` builds the same sources with
``-DLIN_DEVICE_CHECKS=1`` into ``liblin_checked.so`` (objects in
``_build/checked/``): the checked build, whose kernels check their shared
memory, TMEM, TMA-coordinate and global indices (include/lin.h).
"""

from __future__ import annotations

import importlib.metadata
import importlib.util
import json
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "liblin.so")
CHECKED_LIB_PATH = os.path.join(PKG_DIR, "liblin_checked.so")
CALLS_PATH = os.path.join(PKG_DIR, "_lin_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
CALLS_SOURCE = os.path.join(CSRC, "lin_calls.cpp")

SOURCES = ["lin_api.cu", "lin_kernels_tf32.cu", "lin_kernels_f16.cu",
           "lin_kernels_cluster_swiglu.cu", "lin_kernels_cluster_cvt.cu",
           "lin_kernels_cluster_bt.cu", "lin_kernels_cluster_dual.cu", "lin_loss.cu",
           "lin_noalloc.cu", "lin_host.cu", "lin_attn_fwd.cu", "lin_attn_bwd.cu",
           "lin_attn_api.cu", "lin_rope.cu", "lin_distill.cu", "lin_step_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build liblin.so")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "lin.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(checked: bool = False) -> bool:
    lib = CHECKED_LIB_PATH if checked else LIB_PATH
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _calls_made_for() -> dict:
    """What the extension module is built for, beside its sources."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # (a torch without a record of its own)
        version = "unknown"
    return {"python": sys.version, "torch": version}


def _calls_record() -> str:
    return os.path.join(BUILD_DIR, os.path.basename(CALLS_PATH) + ".json")


def calls_up_to_date() -> bool:
    try:
        with open(_calls_record()) as f:
            if json.load(f) != _calls_made_for():
                return False
        t = os.path.getmtime(CALLS_PATH)
    except (OSError, ValueError):
        return False
    return all(os.path.getmtime(f) <= t for f in (
        CALLS_SOURCE, os.path.join(INCLUDE, "lin.h"), os.path.abspath(__file__)))


def _calls_command(out: str, nvcc: str) -> list[str]:
    """The host compiler's command for the extension module."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), CALLS_SOURCE,
            "-o", out, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda"]


def _start_calls():
    """The extension module's compilation, begun; _finish_calls() ends it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    return subprocess.Popen(_calls_command(CALLS_PATH + ".tmp", _nvcc()), stdout=subprocess.PIPE,
                            stderr=subprocess.STDOUT, text=True)


def _finish_calls(proc) -> None:
    out, _ = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError("compilation failed:\nlin_calls.cpp:\n" + out)
    os.replace(CALLS_PATH + ".tmp", CALLS_PATH)
    with open(_calls_record(), "w") as f:
        json.dump(_calls_made_for(), f)


def build_calls(force: bool = False) -> str:
    """Compile the extension module _lin_calls; return its path. Raises on any
    failure."""
    if force or not calls_up_to_date():
        _finish_calls(_start_calls())
    return CALLS_PATH


def build_library(force: bool = False, verbose: bool = False, extra_flags=(),
                  checked: bool = False) -> str:
    """Compile and link liblin.so (or, ``checked``, liblin_checked.so); return
    its path. Raises on any failure. The extension module _lin_calls is built
    beside liblin.so where torch is installed; a failure of that is a warning
    (the calls that need the module raise)."""
    calls = problem = None
    if not checked and importlib.util.find_spec("torch") and (force or not calls_up_to_date()):
        try:
            calls = _start_calls()
        except Exception as e:  # noqa: BLE001  (whatever ails torch or the compiler)
            problem = e
    try:
        path = _build_library(force, verbose, extra_flags, checked)
    except BaseException:
        if calls:
            calls.kill()
            calls.communicate()
        raise
    if calls:
        try:
            _finish_calls(calls)
        except Exception as e:  # noqa: BLE001
            problem = e
    if problem:
        warnings.warn(f"the extension module _lin_calls was not built: {problem}", stacklevel=2)
    return path


def _build_library(force: bool, verbose: bool, extra_flags, checked: bool) -> str:
    lib_path = CHECKED_LIB_PATH if checked else LIB_PATH
    if not force and up_to_date(checked):
        return lib_path
    nvcc = _nvcc()
    build_dir = os.path.join(BUILD_DIR, "checked") if checked else BUILD_DIR
    os.makedirs(build_dir, exist_ok=True)
    if checked:
        extra_flags = (*extra_flags, "-DLIN_DEVICE_CHECKS=1")
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *ARCH, *CFLAGS, *extra_flags, *os.environ.get("LIN_NVCC_FLAGS", "").split(),
               "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose and out:
            print(out, file=sys.stderr)
        if p.returncode != 0:
            failed.append(f"{src}:\n{out}")
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(failed))
    tmp = lib_path + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(link), file=sys.stderr)
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout)
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv,
                        checked="--checked" in sys.argv))
