"""How the grouped products' Python calls are built and found, without a GPU."""
import shutil
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
