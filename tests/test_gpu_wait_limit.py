"""A wait inside a kernel that nobody ends: it gives up after its limit, sets the CTA's flag, records the timeout in the
pool's status word, and the pool goes on."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Result(ctypes.Structure):
    _fields_ = [("complete", ctypes.c_int * 64), ("local", ctypes.c_int * 64), ("cluster", ctypes.c_int * 64),
                ("quit", ctypes.c_int), ("milliseconds", ctypes.c_int)]


def test_a_wait_that_nobody_ends_gives_up(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rope_rotation_gb300
    from rope_rotation_gb300 import _build
    from rope_rotation_gb300.leyline import LeylineError
    from rope_rotation_gb300.runtime import PagedCache
    rope_rotation_gb300.build()
    so = tmp_path / "wait_limit.so"
    cmd = [_build.nvcc()] + _build.ARCH + ["-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static",
                                          "--expt-relaxed-constexpr", "-I", _build.INCLUDE, "-I", _build.CSRC,
                                          os.path.join(ROOT, "tests", "wait_limit.cu"), "-o", str(so)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    lib = ctypes.CDLL(str(so))
    lib.wait_limit.restype = ctypes.c_int
    lib.wait_limit.argtypes = [ctypes.c_void_p, ctypes.POINTER(Result)]
    cache = PagedCache(1, 16, 8, 1, 4)
    cache.check_status()
    r = Result()
    assert lib.wait_limit(cache.pool, ctypes.byref(r)) == 0
    assert list(r.complete) == [1] * 64
    assert list(r.local) == [0] * 64 and list(r.cluster) == [0] * 64
    assert r.quit == 2 and r.milliseconds < 2000
    with pytest.raises(LeylineError, match="0x20") as e:
        cache.check_status()
    assert e.value.code == -8
    cache.check_status()  # cleared
    cache.add_request(0, 20)
    torch.cuda.synchronize()
    cache.close()
