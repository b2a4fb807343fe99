"""build.py where the binding's native half cannot be built: the library does not depend on it."""

from __future__ import annotations

import importlib.util
import os
import types

import pytest

import paged_kv_cache_330_b200 as pa

PKG = os.path.dirname(pa.__file__)


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """build.py with its outputs in tmp_path and a compiler that only leaves files."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name in ("LIB", "CALLS"):
        monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "obj"))

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(mod, "subprocess", types.SimpleNamespace(run=run))
    return mod


def test_both_halves_are_built(builder):
    assert builder.build() == builder.LIB
    assert os.path.exists(builder.LIB) and os.path.exists(builder.CALLS)


@pytest.mark.parametrize("kind", ["no torch", "no headers"])
def test_the_library_is_built_without_torch(builder, tmp_path, monkeypatch, capsys, kind):
    found = None if kind == "no torch" else types.SimpleNamespace(origin=str(tmp_path / "torch" / "__init__.py"))
    monkeypatch.setattr(builder, "importlib", types.SimpleNamespace(util=types.SimpleNamespace(find_spec=lambda n: found)))
    assert builder.build() == builder.LIB
    assert os.path.exists(builder.LIB) and not os.path.exists(builder.CALLS)
    assert "no torch with headers" in capsys.readouterr().err


def test_the_library_is_linked_where_the_other_half_fails(builder, monkeypatch):
    def broken():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(builder, "_build_calls", broken)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        builder.build()
    assert os.path.exists(builder.LIB)


def test_int4_calls_name_the_missing_module(monkeypatch):
    import sys
    monkeypatch.setattr(pa, "_NATIVE", None)
    monkeypatch.setitem(sys.modules, pa.__name__ + "._calls", None)  # import finds nothing
    with pytest.raises(ImportError, match="native module _calls.so"):
        pa._native()
