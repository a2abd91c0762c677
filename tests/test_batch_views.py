"""What a batch refuses, on the CPU and under the sanitizers: views of token tensors that overlap, fuzzed against the bytes
they name, and sizes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_rotation_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"


def _build(tmp_path, name):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / name
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", CUDA_INCLUDE,
           os.path.join(ROOT, "tests", name + ".cpp"), os.path.join(CSRC, "leyline_batch_plan.cpp"),
           os.path.join(CSRC, "leyline_planner.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr:
        pytest.skip("the sanitizer runtimes are not installed: " + build.stderr.strip()[-200:])
    assert build.returncode == 0, build.stderr
    return exe


def _run(exe, *args):
    run = subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "0 failed checks" in run.stdout


def test_overlap_of_views_under_sanitizers(tmp_path):
    exe = _build(tmp_path, "batch_views_sanitize")
    for seed in ("1", "2"):
        _run(exe, "20000", seed)


def test_sizes_of_a_batch(tmp_path):
    _run(_build(tmp_path, "batch_sizes_sanitize"))
