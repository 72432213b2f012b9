"""What builds what: the library without torch or with a host compiler that
fails, and the extension module for the running interpreter and torch only
(CPU; one small translation unit stands for the library's)."""

import json
import os
import sys

import pytest

from transformer_linear_layer_tcgen05_gb300 import build, lin


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's products in a folder of the test's own."""
    name = os.path.basename(build.CALLS_PATH)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "liblin.so"))
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / name))
    monkeypatch.setattr(build, "SOURCES", ["lin_noalloc.cu"])
    return tmp_path


def test_library_without_torch(elsewhere, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda n, *a: None if n == "torch" else find(n, *a))
    assert build.build_library() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)
    assert build.up_to_date()


def test_library_where_the_module_cannot_be_built(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.warns(UserWarning, match="_lin_calls was not built"):
        build.build_library()
    assert build.up_to_date() and not os.path.exists(build.CALLS_PATH)
    with pytest.raises(RuntimeError, match="lin_calls.cpp"):
        build.build_calls()
    monkeypatch.setenv("CXX", str(elsewhere / "no such compiler"))
    with pytest.warns(UserWarning, match="_lin_calls was not built"):
        build.build_library()


def test_the_module_is_of_one_interpreter_and_torch():
    build.build_library()
    assert build.calls_up_to_date()
    assert build.CALLS_PATH.endswith(build.sysconfig.get_config_var("EXT_SUFFIX"))
    record = build._calls_record()
    with open(record) as f:
        made_for = json.load(f)
    assert made_for == build._calls_made_for()
    for other in ({**made_for, "torch": "0.0.1"}, {**made_for, "python": "2.7"}, {}):
        try:
            with open(record, "w") as f:
                json.dump(other, f)
            assert not build.calls_up_to_date()
        finally:
            with open(record, "w") as f:
                json.dump(made_for, f)
    assert build.calls_up_to_date()


def test_the_binding_refuses_a_module_of_another_torch(monkeypatch):
    build.build_library()
    calls = lin._short_calls()
    monkeypatch.setattr(lin, "_calls", None)
    monkeypatch.setattr(calls, "torch_version", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch 0.0.1"):
        lin._short_calls()
    monkeypatch.delattr(calls, "torch_version")
    with pytest.raises(RuntimeError, match="an unknown one"):
        lin._short_calls()
