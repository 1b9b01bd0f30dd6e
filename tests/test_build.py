"""The build of the library and of the Python module beside it, on a copy of
the sources with stand-ins for the compilers (nothing is compiled here)."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

PACKAGE = "nvfp4_moe_expert_topk_b200"


@pytest.fixture
def tree(tmp_path):
    shutil.copytree(os.path.join(ROOT, PACKAGE, "csrc"), tmp_path / PACKAGE / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copy(os.path.join(ROOT, PACKAGE, "build.py"), tmp_path / PACKAGE)
    compiler = tmp_path / "compiler"                     # writes its -o file, and nothing else
    compiler.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\n')
    compiler.chmod(0o755)
    return tmp_path


def build(tree, **env):
    env = dict(os.environ, NVCC=str(tree / "compiler"), CXX=str(tree / "compiler"), **env)
    p = subprocess.run([sys.executable, str(tree / PACKAGE / "build.py")], env=env, capture_output=True, text=True, timeout=300)
    return p, tree / PACKAGE / "libnvfp4moe.so", tree / PACKAGE / "_binding.so"


def test_both_are_built(tree):
    p, library, module = build(tree)
    assert p.returncode == 0 and library.exists() and module.exists(), p.stderr


def test_library_without_torch(tree):
    """The C library needs nvcc alone; the Python module is left out."""
    (tree / "no_torch").mkdir()
    (tree / "no_torch" / "torch.py").write_text("raise ImportError('no torch here')\n")
    p, library, module = build(tree, PYTHONPATH=str(tree / "no_torch"))
    assert p.returncode == 0 and library.exists() and not module.exists(), p.stderr
    assert "_binding.so" in p.stderr and "no torch here" in p.stderr


@pytest.mark.parametrize("cxx", ["false", "/nowhere/g++"])
def test_library_where_the_module_does_not_compile(tree, cxx):
    """The failure is the module's: the library is built, the failure is named,
    and no module of older sources stays behind."""
    module = tree / PACKAGE / "_binding.so"
    module.write_text("of older sources")
    os.utime(module, (1, 1))
    p = subprocess.run([sys.executable, str(tree / PACKAGE / "build.py")], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, NVCC=str(tree / "compiler"), CXX=cxx))
    assert p.returncode == 0 and (tree / PACKAGE / "libnvfp4moe.so").exists() and not module.exists(), p.stderr
    assert "_binding.so" in p.stderr
