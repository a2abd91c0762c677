"""The host plan of a batch of new tokens, on the CPU: fuzzed under the sanitizers, and the
binding's argument checks ("Leyline: KV Cache Directives for Agentic Inference", section 2.3:
rows are prefilled into new slots)."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rope_rotation_gb300", "csrc")
CUDA_INCLUDE = "/usr/local/cuda/include"


def test_batch_plan_fuzz_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "batch_plan_sanitize"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", CUDA_INCLUDE,
           os.path.join(ROOT, "tests", "batch_plan_sanitize.cpp"), os.path.join(CSRC, "leyline_batch_plan.cpp"),
           os.path.join(CSRC, "leyline_planner.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "sanitize" in build.stderr:
        pytest.skip("the sanitizer runtimes are not installed: " + build.stderr.strip()[-200:])
    assert build.returncode == 0, build.stderr
    for seed in (1, 2):
        run = subprocess.run([str(exe), "4000", str(seed)], capture_output=True, text=True, timeout=300)
        assert run.returncode == 0, run.stdout + run.stderr
        assert "0 failed checks" in run.stdout


def test_chunk_records():
    from rope_rotation_gb300 import leyline
    a = leyline.chunk_batch([(3, 100, 7), (1, 5, 2, 40)])
    assert a.dtype.itemsize == 24
    assert [tuple(x) for x in a.tolist()] == [(3, 7, 100, 100), (1, 2, 5, 40)]
    assert leyline.chunk_batch(a) is a
    assert leyline.chunk_batch([]).size == 0
    with pytest.raises(ValueError):
        leyline.chunk_batch([(1, 2)])
    with pytest.raises(ValueError):
        leyline.chunk_batch(np.zeros((2, 2), dtype=leyline.CHUNK_DTYPE))


def test_null_handles_are_refused():
    """No device is touched: every call names its fault before it looks at one."""
    import ctypes

    import rope_rotation_gb300
    from rope_rotation_gb300 import leyline as L
    rope_rotation_gb300.build()
    lib = L.load()
    out = ctypes.c_void_p()
    assert lib.leyline_batch_create(None, 1, 1, 1, ctypes.byref(out)) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_batch_destroy(None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_batch_plan(None, None, None, 0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_append(None, 0, None, 576, None, None, 0.0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_rotate(None, None, None, None, 0.0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert lib.leyline_attention(None, 0, None, None, None, None, 1.0, 0, None) == L.LEYLINE_ERR_INVALID_ARG
    assert "batch" in L.leyline_last_error()


def test_heads_views():
    torch = pytest.importorskip("torch")
    from rope_rotation_gb300 import leyline as L
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    h = L.heads(q, "q", 4, 6, 64)
    assert (h.token_stride, h.head_stride) == (384, 64)
    h = L.heads(q.transpose(0, 1).contiguous().transpose(0, 1), "q", 4, 6, 64)
    assert (h.token_stride, h.head_stride) == (64, 256)
    h = L.heads(q[:1, :1], "q", 1, 1, 64)  # strides of axes of one entry are put right
    assert (h.token_stride, h.head_stride) == (64, 64)
    for t, tokens in ((q.float(), 4), (q, 5), (q[:, :5], 4), (q[..., :32], 4), (q[..., ::2], 4), (q[0], 1)):
        with pytest.raises(ValueError):
            L.heads(t, "q", tokens, 6, 64)
