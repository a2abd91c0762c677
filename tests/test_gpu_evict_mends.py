"""Eviction by attention weight, cases that went wrong or were not held by a test: the first eviction of a pool, lists of no
rows, steps without tokens, what reaches no other row where query tiles pass, and how near the weights come to 64 bits (see
batch_harness and test_gpu_evict for the formulas)."""
import math
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rope_rotation_gb300
    rope_rotation_gb300.build()


import batch_harness as BH  # noqa: E402  (needs torch)
from test_gpu_evict import check_evict, check_weigh, fresh_weights, pick, queries, weights64  # noqa: E402

LAZY, SPLIT = 2, 4
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------------------- evict --
@pytest.mark.parametrize("B", [16, 1])
def test_first_eviction_of_a_pool_leaves_the_legacy_stream_alone(B):
    """The states of the lists are there from the pool's creation on: a first eviction on a stream of its own neither waits
    for the legacy stream nor leaves work there that its kernels are not ordered after."""
    rng = np.random.default_rng(1)
    lists = [pick(rng, 300, 100)]
    kept = torch.tensor(lists, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    legacy = torch.cuda.default_stream()
    for turn in range(2):  # the first turn loads the kernels
        cache = BH.make_cache([300], seed=2, layers=1, B=B, latent=64, rope=16)
        rows = BH.logical(cache, 0, 0, 300)[0].clone()
        torch.cuda.synchronize()
        ended = torch.cuda.Event()
        with torch.cuda.stream(legacy):
            torch.cuda._sleep(600_000_000)  # some 0.3 s
            ended.record()
        t0 = time.monotonic()
        cache.evict([(0, 100)], kept, stream=stream)
        spent = time.monotonic() - t0
        running = not ended.query()
        torch.cuda.synchronize()
        cache.check_status()
        assert torch.equal(BH.logical(cache, 0, 0, 100)[0], rows[torch.tensor(lists[0], device="cuda")])
        cache.close()
    assert running, f"the call waited for the legacy stream, {spent:.3f} s"
