"""Building: the binding's short way belongs to one torch and one Python, and the library is built without it."""
import os
import sysconfig

import pytest
import torch

from serving_sd_verify_gb300 import build


@pytest.fixture(autouse=True)
def _built():
    build.build()


def test_another_torch_or_python_is_another_file(monkeypatch):
    here = build.fast_path()
    assert build.fast_up_to_date() and os.path.exists(here)
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    there = build.fast_path()
    assert there != here and not build.fast_up_to_date() and build.up_to_date()
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")
    assert build.fast_path() not in (here, there) and not build.fast_up_to_date()


@pytest.mark.parametrize("how", [ImportError("no torch"), FileNotFoundError("g++"), RuntimeError("cannot find -lc10_cuda")])
def test_the_library_is_built_without_it(monkeypatch, tmp_path, how):
    def fails():
        raise how
    monkeypatch.setattr(build, "fast_path", lambda: str(tmp_path / "missing.so"))
    monkeypatch.setattr(build, "_build_fast", fails)
    with pytest.warns(RuntimeWarning, match="short way"):
        assert build.build() == build.LIB


def test_it_alone_is_built_where_it_alone_is_missing(monkeypatch, tmp_path, recwarn):
    path = str(tmp_path / os.path.basename(build.fast_path()))
    monkeypatch.setattr(build, "fast_path", lambda: path)
    before = os.path.getmtime(build.LIB)
    build.build()
    assert os.path.exists(path) and build.fast_up_to_date() and os.path.getmtime(build.LIB) == before
    assert not [w for w in recwarn if issubclass(w.category, RuntimeWarning)]
