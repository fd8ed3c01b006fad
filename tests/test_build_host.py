"""What the build needs, with a stand-in for nvcc (no GPU, nothing compiled)."""
import os
import shutil
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "causal_kernelized_linear_gb300"


@pytest.fixture
def tree(tmp_path):
    """A copy of the sources, and an nvcc that writes its output file."""
    ignore = shutil.ignore_patterns("_build*", "__pycache__")
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG, ignore=ignore)
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text(f"#!{sys.executable}\nimport sys\n"
                    "open(sys.argv[sys.argv.index('-o') + 1], 'w').write('built')\n")
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    return tmp_path


def run(tree, code=None, **env):
    cmd = [sys.executable, "-c", code] if code else [sys.executable, str(tree / PKG / "build.py")]
    full = {**os.environ, "NVCC": str(tree / "bin" / "nvcc"), "PYTHONPATH": str(tree), **env}
    return subprocess.run(cmd, env=full, cwd=tree, capture_output=True, text=True, timeout=300)


def test_library_without_pytorch(tree):
    (tree / "none").mkdir()
    (tree / "none" / "torch.py").write_text("raise ImportError('no PyTorch here')\n")
    r = run(tree, PYTHONPATH=str(tree / "none"))
    assert r.returncode == 0, r.stderr
    assert (tree / PKG / "_build" / "liblinattn.so").read_text() == "built"
    assert not (tree / PKG / "_build" / "la_block.so").exists()


def test_library_is_linked_before_the_extension_fails(tree):
    r = run(tree, CXX="/bin/false")
    assert r.returncode != 0 and "la_block" in r.stderr + r.stdout or "py_block" in r.stderr
    assert (tree / PKG / "_build" / "liblinattn.so").read_text() == "built"


def test_extension_of_another_pytorch_is_built_again_and_not_loaded(tree):
    """A stand-in compiler too: what counts is when it is called."""
    cxx = tree / "bin" / "cxx"
    cxx.write_text(f"#!{sys.executable}\nimport sys\n"
                   f"open({str(tree / 'calls')!r}, 'a').write('x')\n"
                   "open(sys.argv[sys.argv.index('-o') + 1], 'w').write('built')\n")
    cxx.chmod(cxx.stat().st_mode | stat.S_IXUSR)
    for want in ("x", "x"):          # built once; the second build has nothing to do
        r = run(tree, CXX=str(cxx))
        assert r.returncode == 0, r.stderr
        assert (tree / "calls").read_text() == want
    code = f"import torch; torch.__version__ = '9.9.9'; import {PKG} as la; "
    r = run(tree, code + f"from {PKG} import _block, _binding; _binding._lib = object(); _block._load_ext()",
            CXX=str(cxx))
    assert r.returncode != 0 and "9.9.9" in r.stderr and "built for" in r.stderr, r.stderr
    r = run(tree, code + "la.build()", CXX=str(cxx))
    assert r.returncode == 0, r.stderr
    assert (tree / "calls").read_text() == "xx"
