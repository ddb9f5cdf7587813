"""The binding's short way lets go of the interpreter's lock while it is inside a C entry: a launch can wait there for
work that needs it.  The entries are stand-ins that answer whether the lock is held."""
import importlib.machinery
import importlib.util
import shutil
import subprocess

import pytest

from test_gpu_fast_calls import S, calls  # noqa: F401

pytestmark = pytest.mark.gpu

ENTRIES = ["sd_norm_rotary", "sd_norm_rotary_append_paged", "sd_paged_attention_e4m3", "sd_paged_tree_attention", "sd_compact_tree_paged"]


@pytest.fixture(scope="module")
def stand_in(S, tmp_path_factory):  # noqa: F811
    d = tmp_path_factory.mktemp("lock")
    (d / "entries.c").write_text("int PyGILState_Check(void);\n" + "".join(f"int {e}(void) {{ return PyGILState_Check(); }}\n" for e in ENTRIES))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(d / "entries.so"), str(d / "entries.c")], check=True)
    copy = str(d / "_fast_calls.so")           # a module of its own, with entry points of its own
    shutil.copy(S._fast.__file__, copy)
    loader = importlib.machinery.ExtensionFileLoader("_fast_calls", copy)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fast_calls", loader))
    loader.exec_module(module)
    module.bind(str(d / "entries.so"))
    return module


@pytest.mark.parametrize("name", ["norm", "append", "attend", "tree", "compact"])
def test_the_lock_is_free_inside_a_call(S, calls, stand_in, monkeypatch, name):  # noqa: F811
    fn, short, kw, _ = calls[name]
    answers = []

    class Short:
        def __getattr__(self, entry):
            def call(*a):
                answers.append((entry, getattr(stand_in, entry)(*a)))
                return S.SD_OK
            return call
    monkeypatch.setattr(S, "_fast", Short())
    fn(**kw)
    assert answers == [(short, 0)], "the lock was held"
