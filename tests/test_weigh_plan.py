"""The plan of weighing rows, on the CPU: fuzzed under the sanitizers; the binding's argument checks of eviction."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_rotation_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"


def test_weigh_plan_fuzz_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "weigh_plan_sanitize"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", CUDA_INCLUDE,
           os.path.join(ROOT, "tests", "weigh_plan_sanitize.cpp"), os.path.join(CSRC, "leyline_batch_plan.cpp"),
           os.path.join(CSRC, "leyline_planner.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr:
        pytest.skip("the sanitizer runtimes are not installed: " + build.stderr.strip()[-200:])
    assert build.returncode == 0, build.stderr
    for seed in (1, 2):
        run = subprocess.run([str(exe), "3000", str(seed)], capture_output=True, text=True, timeout=300)
        assert run.returncode == 0, run.stdout + run.stderr
        assert " 0 failed checks" in run.stdout


def test_keep_records():
    from rope_rotation_gb300 import leyline
    a = leyline.keep_batch([(3, 100), (1, 5, 2, 1)])
    assert a.dtype.itemsize == 16 and [tuple(x) for x in a.tolist()] == [(3, 100, 0, 0), (1, 5, 2, 1)]
    assert leyline.keep_batch(a) is a and leyline.keep_batch([]).size == 0
    for bad in ([(1,)], [(1, 2, 3)], np.zeros((2, 2), dtype=leyline.KEEP_DTYPE), np.zeros(4, dtype=leyline.KEEP_DTYPE)[::2]):
        with pytest.raises(ValueError):
            leyline.keep_batch(bad)


def test_null_handles_are_refused():
    """No device is touched: every call names its fault before it looks at one."""
    import rope_rotation_gb300
    from rope_rotation_gb300 import leyline as L
    rope_rotation_gb300.build()
    lib = L.load()
    w = L.RowWeights(None, 0, 0, 0)
    bt = L.BlockTable()
    assert lib.leyline_attention_weights(None, 0, None, None, None, ctypes.byref(w), 1.0, 1.0, 0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_select_rows(None, ctypes.byref(bt), ctypes.byref(w), None, 0, None, 0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_evict(None, ctypes.byref(bt), None, 0, None, 0, None, None) == L.LEYLINE_ERR_INVALID_ARG
    assert "null" in L.leyline_last_error()


def test_views_of_weights_and_lists():
    torch = pytest.importorskip("torch")
    from rope_rotation_gb300 import leyline as L
    t = torch.zeros(3, 50)
    w = L.row_weights(t)
    assert (w.ptr, w.req_stride, w.rows, w.num_reqs) == (t.data_ptr(), 50, 50, 3)
    w = L.row_weights(t[1:, 4:20])
    assert (w.ptr, w.req_stride, w.rows, w.num_reqs) == (t.data_ptr() + 4 * 54, 50, 16, 2)
    assert L.row_weights(t[:1]).req_stride == 50
    for bad in (t.double(), t[0], t[:, ::2], t[:1].expand(3, 50), t.clone().requires_grad_()):
        with pytest.raises(ValueError):
            L.row_weights(bad)
    keeps = L.keep_batch([(0, 7), (1, 3)])
    kept = torch.zeros(2, 10, dtype=torch.int32)
    assert L._lists(kept, keeps) == (kept.data_ptr(), 10)
    for bad in (kept.long(), kept[:1], kept[:, :6], kept[:, ::2][:, :5], kept[:1].expand(2, 10), kept.view(-1)):
        with pytest.raises(ValueError):
            L._lists(bad, keeps)
