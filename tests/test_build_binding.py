"""The native binding is optional: the library is built, and its calls go
through ctypes, without it or with one of another torch."""
import os
import sys
import types

import pytest
import torch

from up_projection_b200 import _capi, build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The binding and its stamp in a folder of their own; the library as it is."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / os.path.basename(build.BINDING)))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "up_to_date", lambda: True)
    return tmp_path


def test_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with open(build.BINDING, "w") as f:
        f.write("of another torch")
    os.utime(build.BINDING, (1, 1))
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build() == build.LIB
    assert not os.path.exists(build.BINDING)       # nothing old is left to be imported


def test_library_is_built_before_the_binding(elsewhere, monkeypatch):
    order = []
    monkeypatch.setattr(build, "up_to_date", lambda: order.append("library") or True)
    monkeypatch.setattr(build, "build_binding", lambda force=False: order.append("binding"))
    build.build()
    assert order == ["library", "binding"]


def test_binding_of_another_torch_or_interpreter_is_not_current(monkeypatch):
    build.build_binding()
    assert build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert not build.binding_up_to_date()
    monkeypatch.undo()
    assert build.binding_up_to_date()
    # an interpreter's suffix, which no other interpreter imports
    assert build.BINDING.endswith(build.sysconfig.get_config_var("EXT_SUFFIX"))


def test_binding_of_another_torch_is_not_called(monkeypatch):
    handle = _capi.lib()
    bound = []
    other = types.SimpleNamespace(built_for="another torch", bind=lambda *a: bound.append(a))
    monkeypatch.setitem(sys.modules, "up_projection_b200._binding", other)
    monkeypatch.setattr("up_projection_b200._binding", other, raising=False)
    monkeypatch.setattr(_capi, "_native", None)
    _capi._bind(handle)
    assert _capi._native is None and not bound
    other.built_for = build.binding_stamp()
    _capi._bind(handle)
    assert _capi._native is other and len(bound) == 1
