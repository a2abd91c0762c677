"""The host side of a batch, on the CPU and under the sanitizers: views of token tensors that overlap, fuzzed against the
bytes they name, sizes, the split of the attention's work, and tensors that require a gradient."""
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


def test_split_of_the_work_with_both_item_costs(tmp_path):
    exe = _build(tmp_path, "batch_split_sanitize")
    for seed in ("1", "2"):
        _run(exe, "4000", seed)


def test_tensors_that_require_a_gradient():
    """There is no backward pass: the output would silently have no gradient.  No device is touched."""
    torch = pytest.importorskip("torch")
    from rope_rotation_gb300 import leyline as L
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16, requires_grad=True)
    rows, w = q.view(24, 64)[:4], torch.zeros(64, dtype=torch.bfloat16, requires_grad=True)
    plain = L.heads(q.detach(), "q", 4, 6, 64)
    for call in (lambda: L.heads(q, "q", 4, 6, 64), lambda: L.leyline_append(None, 0, rows),
                 lambda: L.leyline_append(None, 0, rows.detach(), latent_norm=w),
                 lambda: L.leyline_append(None, 0, rows.detach(), key_norm=w),
                 lambda: L.leyline_rotate(None, plain, plain, norm=w),
                 lambda: L.leyline_attention(None, 0, plain, plain, plain, torch.zeros(4, 6, requires_grad=True), 1.0)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        assert L.heads(q, "q", 4, 6, 64).token_stride == 384
