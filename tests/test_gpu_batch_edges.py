"""Batches of new tokens where they can go wrong: values that are not finite in masked rows, scores that rise late,
batches that share a pool, steps without tokens (see batch_harness for formulas and tolerances)."""
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

LAZY, SPLIT = 2, 4


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lat,rope,bands,heads,B,flags", [
    (512, 64, 1, 4, 16, 0), (512, 64, 1, 128, 16, 0), (512, 64, 1, 16, 5, 0), (512, 64, 1, 16, 16, LAZY),
    (512, 128, 4, 16, 16, 0), (384, 64, 2, 4, 16, SPLIT), (40, 48, 1, 3, 16, 0)])
@pytest.mark.parametrize("start", [0, 70, 9000])
def test_a_bad_token_does_not_reach_the_ones_before_it(bad, lat, rope, bands, heads, B, flags, start):
    """Token 5 of 9 brings a value (and key) that is not finite: tokens 0 to 4, and the other request's, are as
    without it.  A start of 9000 splits the row tiles, so pieces without any row of a token join in."""
    cache = BH.make_cache([start, 33], extra=16, layers=1, B=B, latent=lat, rope=rope, bands=bands, flags=flags)
    b = cache.batch(2, 16, heads)
    chunks = [(0, start, 9), (1, 33, 2)]
    b.plan(chunks)
    rows = BH.bf16(11, cache.row, seed=1)
    ql = BH.bf16(11, heads, lat, seed=2) if bands == 1 else None
    q = BH.bf16(11, heads, rope, seed=3)
    scale = rope ** -0.5 if bands > 1 else 0.07
    b.append(0, rows)
    want, wlse, tol, ltol = BH.attention64(cache, 0, chunks, ql, q, scale)
    rows[5, 3::lat // bands] = bad
    b.append(0, rows)
    out, lse = b.attention(0, ql, q, scale)
    for t in (0, 1, 2, 3, 4, 9, 10):
        assert bool(((out[t].double() - want[t]).abs() <= tol[t]).all()), t
        assert bool(((lse[t].double() - wlse[t]).abs() <= ltol[t]).all()), t
    if bad != bad:  # (an infinite key's score is -inf for a query of the other sign: that row is left out)
        assert not bool(out[5:9, :, 3].isfinite().any())
    cache.check_status()
    cache.close()


@pytest.mark.parametrize("start,n,heads", [(0, 200, 16), (700, 1, 128), (1000, 20, 128), (20000, 1, 128), (300, 3, 130),
                                           (20000, 3, 8)])
@pytest.mark.parametrize("peak", [127.0, -127.0, 24.0])
def test_scores_that_rise_late(start, n, heads, peak):
    """The rows' scores climb along the cache by up to 160, far past what a reference taken from its first rows
    can hold, fall by as much, or climb by 30."""
    cache = BH.make_cache([start], extra=n, layers=1)
    b = cache.batch(1, n, heads)
    b.plan([(0, start, n)])
    b.append(0, BH.bf16(n, 576, seed=1))
    end = start + n
    rows, flat = BH.logical(cache, 0, 0, end)
    rows = rows.clone()
    rows[:, 0] = (torch.arange(end, device="cuda") * (peak / end)).to(torch.bfloat16)
    cache.write_layer_rows(0, flat, rows)
    ql, q = BH.bf16(n, heads, 512, seed=2), BH.bf16(n, heads, 64, seed=3)
    ql[:, :, 0] = 18.0
    BH.check_attention(cache, b, 0, [(0, start, n)], ql, q, 0.07, f"rising to {peak}")
    if n > 1 and start:
        BH.check_attention(cache, b, 0, [(0, start, n)], ql, q, 0.07, f"rising to {peak}, prefix", prefix=True)
    cache.check_status()
    cache.close()


@pytest.mark.parametrize("lat,rope,bands", [(512, 64, 1), (512, 128, 4), (40, 48, 1)])
def test_large_values(lat, rope, bands):
    """Values near the end of bf16's range: their weighted sums stay in fp32's."""
    cache = BH.make_cache([500], extra=8, layers=1, latent=lat, rope=rope, bands=bands)
    b = cache.batch(1, 8, 16 if bands > 1 else 128)
    b.plan([(0, 500, 8)])
    b.append(0, BH.bf16(8, cache.row, seed=1))
    rows, flat = BH.logical(cache, 0, 0, 508)
    rows = rows.clone()
    rows[::3, 7] = 1e38
    cache.write_layer_rows(0, flat, rows)
    ql = BH.bf16(8, b.q_heads, lat, seed=2) if bands == 1 else None
    if bands == 1:
        ql[:, :, 7] = 0.0
    q = BH.bf16(8, b.q_heads, rope, seed=3)
    BH.check_attention(cache, b, 0, [(0, 500, 8)], ql, q, 0.07, "large values")
    cache.close()


def test_steps_without_tokens():
    cache = BH.make_cache([20], extra=8, layers=1)
    b = cache.batch(2, 8, 4)
    for chunks in ([], [(0, 20, 0)]):
        b.plan(chunks)
        before = cache.kv.clone()
        b.append(0, BH.bf16(0, 576))
        assert b.rotate(BH.bf16(0, 4, 64)).shape == (0, 4, 64)
        out, lse = b.attention(0, BH.bf16(0, 4, 512), BH.bf16(0, 4, 64), 0.07)
        assert out.shape == (0, 4, 512) and lse.shape == (0, 4)
        torch.cuda.synchronize()
        assert torch.equal(before.view(torch.int16), cache.kv.view(torch.int16))
    b.plan([(0, 20, 1)])  # and tensors of a padded batch: the rows past the plan's tokens stay
    out = torch.full((6, 4, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 4), 7.0, device="cuda")
    turned = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    b.append(0, BH.bf16(6, 576))
    b.rotate(BH.bf16(6, 4, 64, seed=2), out=turned)
    b.attention(0, BH.bf16(6, 4, 512, seed=1), turned, 0.07, out=out, lse=lse)
    assert bool((out[1:] == 7).all()) and bool((lse[1:] == 7).all()) and bool((turned[1:] == 7).all())
    assert bool((out[0] != 7).any())
    cache.check_status()
    cache.close()


def test_two_batches_of_a_pool_on_two_streams():
    """Each batch has its own plan and workspace; the library orders their calls on the pool."""
    cache = BH.make_cache([900, 20000, 300], extra=200, layers=1)
    one, two = cache.batch(2, 200, 16), cache.batch(2, 200, 128)
    plans = [(one, [(0, 900, 100), (2, 300, 1)]), (two, [(1, 20000, 2)])]
    streams = [torch.cuda.Stream() for _ in plans]
    data = []
    for k, (b, chunks) in enumerate(plans):
        n = sum(c[2] for c in chunks)
        data.append((BH.bf16(n, 576, seed=k), BH.bf16(n, b.q_heads, 512, seed=10 + k), BH.bf16(n, b.q_heads, 64, seed=20 + k)))
    torch.cuda.synchronize()
    outs = [[], []]
    for k, (b, chunks) in enumerate(plans):
        with torch.cuda.stream(streams[k]):
            b.plan(chunks)
    for _ in range(4):
        for k, (b, chunks) in enumerate(plans):
            with torch.cuda.stream(streams[k]):
                rows, ql, q = data[k]
                b.append(0, rows)
                outs[k].append(b.attention(0, ql, q, 0.07))
    torch.cuda.synchronize()
    for k, (b, chunks) in enumerate(plans):
        for out, lse in outs[k][1:]:
            assert torch.equal(out, outs[k][0][0]) and torch.equal(lse, outs[k][0][1])
        out, lse = BH.check_attention(cache, b, 0, chunks, data[k][1], data[k][2], 0.07, f"batch {k}")
        assert torch.equal(out, outs[k][0][0])
    cache.check_status()
    cache.close()


def test_outputs_that_overlap_are_refused():
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([40], extra=16, layers=1)
    b = cache.batch(1, 8, 4)
    b.plan([(0, 40, 3)])
    ql, q = BH.bf16(3, 4, 512), BH.bf16(3, 4, 64)
    flat = torch.empty(4 * 3 * 512, dtype=torch.bfloat16, device="cuda")
    for out in (ql, flat.as_strided((3, 4, 512), (512, 1024, 1)), flat.as_strided((3, 4, 512), (512, 512, 1))):
        with pytest.raises(LeylineError) as e:
            b.attention(0, ql, q, 0.07, out=out)
        assert e.value.code == -1
    b.attention(0, ql, q, 0.07, out=flat.as_strided((3, 4, 512), (512, 1536, 1)))  # heads outermost
    cache.check_status()
    cache.close()


@pytest.mark.parametrize("heads,reqs", [(128, 100), (20, 300)])
def test_many_short_tiles(heads, reqs):
    """Row tiles of one or two cache tiles (with a prefix: of none) one after another on a CTA."""
    rng = np.random.default_rng(heads)
    lens = rng.integers(0, 130, size=reqs)
    lens[:8] = 0
    chunks = [(r, int(n), int(rng.integers(1, 9))) for r, n in enumerate(lens)]
    cache = BH.make_cache(lens.tolist(), extra=8, layers=1)
    b = cache.batch(reqs, 8 * reqs, heads)
    b.plan(chunks)
    T = b.tokens
    b.append(0, BH.bf16(T, 576, seed=1))
    ql, q = BH.bf16(T, heads, 512, seed=2), BH.bf16(T, heads, 64, seed=3)
    for prefix in (False, True):
        first = BH.check_attention(cache, b, 0, chunks, ql, q, 0.07, "short tiles", prefix=prefix)
        for _ in range(20):
            out, lse = b.attention(0, ql, q, 0.07, prefix=prefix)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    cache.check_status()
    cache.close()
