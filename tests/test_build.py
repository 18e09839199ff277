"""The in-tree build: the C library stands alone, the native module beside it needs Python's headers."""
import os
import sysconfig

import pytest

pytest.importorskip("torch")

import chain_gb300 as cg
from chain_gb300 import _build


def test_the_library_builds_without_pythons_headers(monkeypatch, tmp_path):
    _build.build()  # up to date
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {"include": str(tmp_path / "none")})
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.NATIVE)
    # the calls that need the module say what is missing
    monkeypatch.setattr(cg, "_calls", None)
    with pytest.raises(RuntimeError, match="Python.h"):
        cg._small()
