"""How the grouped products' Python calls are built and found, without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

from fp32_gemm_amd import build


def test_the_library_builds_without_torch(monkeypatch):
    # A user of the C ABI needs hipcc alone.
    monkeypatch.setattr(build, "_build_once", lambda verbose, jobs: {})
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build(verbose=False) == build.LIB


def test_the_command_says_what_it_left_out(monkeypatch, capsys):
    monkeypatch.setattr(build, "_build_once", lambda verbose, jobs: {})
    monkeypatch.setattr(shutil, "which", lambda name: None)
    build.main()
    assert "g++ not found" in capsys.readouterr().out
    with pytest.raises(RuntimeError, match="g\\+\\+ not found"):
        build.build_calls()


def run(code):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)


CALL = """
try:
    lib.gemm_grouped(None, None, None, None)
except ImportError as error:
    print(error)
"""


def test_calls_built_for_another_torch_say_so():
    p = run("import torch; torch.__version__ = '0.1'; import fp32_gemm_amd as lib" + CALL)
    assert p.returncode == 0, p.stderr
    assert "gemm_grouped: built for torch" in p.stdout and "this is torch 0.1" in p.stdout


def test_the_package_imports_without_the_calls():
    # As it did before there were any: the library's own calls need no more.
    p = run("import sys; sys.modules['fp32_gemm_amd._torch_calls'] = None\n"
            "from fp32_gemm_amd import *; import fp32_gemm_amd as lib\n"
            "assert num_configs() > 0 and lib.grouped.plan('nt', lib.grouped.torch.float32, 1, 8, 8, 8)" + CALL)
    assert p.returncode == 0, p.stderr
    assert "python -m fp32_gemm_amd.build" in p.stdout
