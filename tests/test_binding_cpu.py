"""Loading the library where the binding's short way is missing or does not load: a warning, and all calls as ever."""
import importlib.util
import os

import pytest

from serving_sd_verify_gb300 import build


@pytest.fixture()
def fresh():
    """The binding's module once more, not yet loaded."""
    build.build()
    path = os.path.join(build.PKG, "sd_verify.py")
    spec = importlib.util.spec_from_file_location("sd_verify_fresh", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_loads_with_the_short_way(fresh, recwarn):
    lib = fresh.load()
    assert fresh._fast is not None and fresh.load() is lib
    assert not [w for w in recwarn if issubclass(w.category, RuntimeWarning)]


@pytest.mark.parametrize("content", [None, b"", b"no shared object"])
def test_loads_without_it(fresh, tmp_path, monkeypatch, content):
    path = tmp_path / "_fast_calls.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(fresh, "FAST_PATH", str(path))
    with pytest.warns(RuntimeWarning, match="short way"):
        lib = fresh.load()
    assert fresh._fast is None and fresh.load() is lib
    assert fresh.load().sd_fault_word is not None
    with pytest.raises(ValueError):            # a call goes through the long way's checks
        fresh.sd_compact_tree_paged(*[__import__("torch").zeros(1)] * 6)


def test_the_library_itself_is_needed(fresh, tmp_path, monkeypatch):
    monkeypatch.setattr(fresh, "LIB_PATH", str(tmp_path / "libsdverify.so"))
    with pytest.raises(RuntimeError, match="missing"):
        fresh.load()
    assert fresh._lib is None
