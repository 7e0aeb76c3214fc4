"""liblce.so is a C library: it builds without torch, and a binding that does not compile leaves it built.
The build runs in a process of its own, over one small source, into a folder of its own."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "memory_bounded_linear_gb300", "csrc", "build.py")

SCRIPT = """
import importlib.util, os, sys
{before}
spec = importlib.util.spec_from_file_location("lce_build", {path!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
tmp = sys.argv[1]
b.BUILD, b.LIB, b.NATIVE = tmp, os.path.join(tmp, "liblce.so"), os.path.join(tmp, "_native.so")
b.SOURCES = ["lce_static_scratch.cu"]
b.build()
"""


def _build(tmp_path, before, **env):
    return subprocess.run([sys.executable, "-c", SCRIPT.format(before=before, path=BUILD), str(tmp_path)],
                          capture_output=True, text=True, env=dict(os.environ, **env))


def test_without_torch(tmp_path):
    r = _build(tmp_path, "sys.modules['torch'] = None")
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "liblce.so").exists() and not (tmp_path / "_native.so").exists()
    assert "torch" in r.stderr                     # says what was left out


def test_binding_that_does_not_compile(tmp_path):
    r = _build(tmp_path, "", CXX="false")
    assert r.returncode != 0 and "py_binding.cpp" in r.stderr
    assert (tmp_path / "liblce.so").exists()
