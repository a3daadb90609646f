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
