"""Building and importing the package where torch is not installed."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# An interpreter that has no torch: neither `import torch` nor a search finds it.
WITHOUT_TORCH = """
import sys
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.partition(".")[0] == "torch":
            raise ModuleNotFoundError(f"No module named {name!r}", name=name)
sys.meta_path.insert(0, NoTorch())
import importlib.util
_find = importlib.util.find_spec
importlib.util.find_spec = lambda name, package=None: None if name == "torch" else _find(name, package)
"""

# build() with its compiler and linker replaced by programs that write what they
# would have made, in another folder than the package's
BUILD = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("hip_build", os.path.join({root!r}, "dense_gemm_11_amd", "build.py"))
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BUILD, b.LIB, b.BIND = (os.path.join({tmp!r}, n) for n in ("objects", "libdense_gemm.so", "_bind.so"))
ran = []
def run(cmd, **kw):
    ran.append(cmd[-1])
    open(cmd[-1], "w").close()
    import subprocess
    return subprocess.CompletedProcess(cmd, 0, "", "")
class Subprocess:
    pass
b.subprocess = Subprocess()
b.subprocess.run = run
open(b.BIND, "w").write("of an earlier build")
print(b.build())
print("library", os.path.exists(b.LIB), "module", os.path.exists(b.BIND) and os.path.getsize(b.BIND) == 0,
      "objects", len(os.listdir(b.BUILD)), "of", len(b.SOURCES))
"""


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_build_without_torch(tmp_path):
    """The library is built, the extension module is not, nor is an older one left."""
    p = python(WITHOUT_TORCH + BUILD.format(root=ROOT, tmp=str(tmp_path)))
    assert p.returncode == 0, p.stderr
    words = p.stdout.split()
    assert words[0] == str(tmp_path / "libdense_gemm.so") and words[1:5] == ["library", "True", "module", "False"]
    assert words[6] == words[8] and not (tmp_path / "_bind.so").exists()


def test_build_with_torch(tmp_path):
    pytest.importorskip("torch")
    p = python(BUILD.format(root=ROOT, tmp=str(tmp_path)))
    assert p.returncode == 0, p.stderr
    words = p.stdout.split()
    assert words[1:5] == ["library", "True", "module", "True"] and int(words[6]) == int(words[8]) + 1


def test_raw_calls_without_torch():
    p = python(WITHOUT_TORCH + """
import dense_gemm_11_amd as g
h = g.gemm_create()
print(g.gemm_route_workspace_bytes(100, 8) > 0, g.gemm_route(h, -1, 0, 8, 0, None, 0, 0, 0, 0, 0, 0, 0, 0))
g.gemm_destroy(h)
""")
    assert p.returncode == 0, p.stderr
    assert p.stdout.split() == ["True", "1"]
