"""Compiles a C++ program that includes the library's plain C++ headers, runs it and returns what it
printed, so that host logic and index rules are tested on the CPU as they are built."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(source, tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "program.cpp", tmp_path / "program"
    src.write_text(source)
    csrc = os.path.join(ROOT, "rmsnorm_precision_activation_gb300", "csrc")
    built = subprocess.run([cxx, "-std=c++17", "-O1", "-I" + csrc, "-I" + os.path.join(ROOT, "include"),
                            str(src), "-o", str(exe)], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr[-4000:]
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0, (ran.stdout + ran.stderr)[-4000:]
    return ran.stdout
