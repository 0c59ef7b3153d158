"""Building and loading the library and the binding's native module, in any order and without what the module needs."""
import os
import shutil
import subprocess
import sys

import pytest

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200 import build as b

PACKAGE = os.path.dirname(os.path.abspath(b.__file__))


@pytest.fixture(scope="module", autouse=True)
def _built():
    b.build()


@pytest.fixture
def checkout(tmp_path):
    """The package's Python files and libgbs.so under another root, without the native module."""
    to = tmp_path / "gated_block_sparse_gate_b200"
    to.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py") or name == "libgbs.so":
            shutil.copy(os.path.join(PACKAGE, name), to)
    return to


def _run(checkout, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=checkout.parent, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(checkout.parent)})
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()


def test_a_native_module_built_after_the_import_is_used(checkout):
    module = b.build_marshal()
    if module is None:
        pytest.skip("built without the headers")
    out = _run(checkout, f"""
import shutil
from gated_block_sparse_gate_b200 import binding as gb
print(gb._native is gb._NoCalls)
shutil.copy({module!r}, {str(checkout)!r})
gb.load_library()
print(gb._native is gb._marshal, gb._fits is gb._marshal.fits, gb._heads_of is gb._marshal.heads)
""")
    assert out == ["True"] * 4


def test_without_the_native_module_the_binding_loads(checkout):
    assert _run(checkout, """
from gated_block_sparse_gate_b200 import binding as gb
gb.load_library()
print(gb._native is gb._NoCalls, gb._marshal is None)
""") == ["True", "True"]


def test_the_native_module_is_the_one_loaded_here():
    assert b.build_marshal() is None or (gb.load_library() and gb._native is gb._marshal)


def test_the_library_builds_without_a_host_compiler(monkeypatch, tmp_path):
    """nvcc is stood in for; the module's compiler does not exist, or fails."""
    made = []
    run = subprocess.run

    def nvcc(cmd, **kw):
        if cmd[0] != "nvcc":
            return run(cmd, **kw)
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgbs.so"))
    module = str(tmp_path / "_marshal.so")
    monkeypatch.setattr(b, "marshal_path", lambda: module)
    monkeypatch.setattr(b.subprocess, "run", nvcc)
    monkeypatch.delenv("NVCC", raising=False)
    for compiler in (str(tmp_path / "no compiler"), "false"):
        monkeypatch.setenv("CXX", compiler)
        open(module, "w").close()  # made from other sources: not to be loaded
        with pytest.warns(UserWarning, match="marshal.cpp was not built"):
            assert b.build(force=True) == b.LIB
    assert len(made) == 2 and not os.path.exists(module)


def test_the_library_builds_without_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # an import of it raises ImportError
    assert b.build() == b.LIB and b.build_marshal() is None


def test_the_native_module_of_another_torch_is_not_loaded(checkout):
    """Its name tells which torch it was compiled against."""
    module = b.build_marshal()
    if module is None:
        pytest.skip("built without the headers")
    shutil.copy(module, checkout)
    for change in ("torch.__version__ = '9.9.9+other'", "torch.version.git_version = 'another commit'", ""):
        assert _run(checkout, f"""
import torch
{change}
from gated_block_sparse_gate_b200 import binding as gb
gb.load_library()
print(gb._native is gb._NoCalls)
""") == [str(bool(change))]
