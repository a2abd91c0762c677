"""What the C ABI's host side enqueues, in which order, and which calls it takes: over a CUDA runtime of the test's own
(host_calls_fake.cpp), on the CPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_rotation_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"
HOST = ["leyline_pool.cpp", "leyline_evict.cpp", "leyline_batch.cpp", "leyline_batch_plan.cpp", "leyline_planner.cpp"]


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    out = tmp_path_factory.mktemp("host_calls") / "host_calls_fake"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", CUDA_INCLUDE,
           os.path.join(ROOT, "tests", "host_calls_fake.cpp")] + [os.path.join(CSRC, f) for f in HOST] + ["-ldl", "-o", str(out)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr:
        pytest.skip("the sanitizer runtimes are not installed: " + build.stderr.strip()[-200:])
    assert build.returncode == 0, build.stderr
    return str(out)


def run(exe, case):
    done = subprocess.run([exe, case], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stdout + done.stderr
    assert " 0 failed checks" in done.stdout


CASES = ["first_eviction", "freed_pages", "status_word", "empty_lists", "idle_step", "plan_copies", "lengths"]


@pytest.mark.parametrize("case", CASES)
def test_host_calls(exe, case):
    run(exe, case)
