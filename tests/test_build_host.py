"""The build as its callers make it: each in a process of its own, and on a tree
that is up to date, where nothing else has imported torch."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_build_twice_in_new_processes():
    pytest.importorskip("torch")
    for _ in range(2):
        r = run("import __graft_entry__ as g; g.build()")
        assert r.returncode == 0, r.stderr


def test_ops_without_torch_imported_first():
    pytest.importorskip("torch")
    from sparse_linear_layer_gb300 import build
    build.build()
    r = run("import sys; from sparse_linear_layer_gb300 import binding; assert 'torch' not in sys.modules; "
            "assert binding.ops().pack")
    assert r.returncode == 0, r.stderr


def test_ops_says_not_built_only_when_the_file_is_absent():
    pytest.importorskip("torch")
    from sparse_linear_layer_gb300 import build
    build.build()
    r = run("from sparse_linear_layer_gb300 import binding; binding.OPS_PATH += '.absent'; binding.ops()")
    assert r.returncode != 0 and "is not built" in r.stderr
    # a module that is there and cannot be loaded reports the loader's own error
    r = run("import sys; sys.modules['sparse_linear_layer_gb300._q8ops'] = None; "
            "from sparse_linear_layer_gb300 import binding; binding.ops()")
    assert r.returncode != 0 and ("ImportError" in r.stderr or "ModuleNotFoundError" in r.stderr)
    assert "is not built" not in r.stderr


@pytest.fixture
def fake_tree(tmp_path, monkeypatch):
    """build.py with its outputs in tmp_path and an nvcc that only creates the file
    it is asked for."""
    from sparse_linear_layer_gb300 import build
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho x > "$2"\n')
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    for name, path in (("LIB", "libsnk.so"), ("OPS", "_q8ops.so"), ("OBJ", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    return build


def test_library_is_linked_when_the_torch_module_does_not_compile(fake_tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="q8_ops.cpp"):
        fake_tree.build()
    assert os.path.exists(fake_tree.LIB) and not os.path.exists(fake_tree.OPS)
    with pytest.raises(RuntimeError, match="q8_ops.cpp"):   # still missing, still an error
        fake_tree.build()


def test_library_is_built_without_torch(fake_tree, monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)
    assert fake_tree.build() == fake_tree.LIB
    assert os.path.exists(fake_tree.LIB) and not os.path.exists(fake_tree.OPS)
    assert fake_tree.up_to_date()


def test_another_torch_rebuilds_the_torch_module(fake_tree, monkeypatch, tmp_path):
    """... and nothing else."""
    import importlib.machinery
    import importlib.util
    cxx = tmp_path / "g++"
    cxx.write_text((tmp_path / "nvcc").read_text())
    cxx.chmod(0o755)
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", str(cxx))
    fake_tree.build()
    assert fake_tree.up_to_date()
    times = os.stat(fake_tree.LIB).st_mtime_ns, os.stat(fake_tree.OPS).st_mtime_ns
    fake_tree.build()
    assert times == (os.stat(fake_tree.LIB).st_mtime_ns, os.stat(fake_tree.OPS).st_mtime_ns)
    other = tmp_path / "torch"
    other.mkdir()
    (other / "__init__.py").write_text("")
    (other / "version.py").write_text("__version__ = '0.0'\n")
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(other / "__init__.py"))
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    assert not fake_tree.up_to_date()
    fake_tree.build()
    assert fake_tree.up_to_date()
    assert os.stat(fake_tree.LIB).st_mtime_ns == times[0] and os.stat(fake_tree.OPS).st_mtime_ns != times[1]
