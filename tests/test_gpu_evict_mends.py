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


@pytest.mark.parametrize("kw", [dict(), dict(B=1), dict(flags=LAZY), dict(flags=LAZY, B=1)])
def test_requests_that_keep_no_rows(kw):
    """Selections and evictions of nothing, alone, together and among others, with lists as select_rows makes them."""
    cache = BH.make_cache([50, 33, 0, 1], seed=3, layers=2, latent=64, rope=16, **kw)
    pages = cache.free_pages()
    if cache.pending() is not None:
        for r in (0, 1, 3):
            flat = torch.from_numpy(cache.slot_index(r, np.arange(int(cache.seq_lens_host[r])))).cuda()
            cache.pending().view(-1)[flat] = 9
    w = fresh_weights(cache, seed=1)
    behind = w.clone()
    kept = cache.select_rows(w, [(0, 0), (2, 0)])
    assert tuple(kept.shape) == (2, 0)
    cache.evict([(0, 0), (2, 0)], kept, weights=w)
    torch.cuda.synchronize()
    cache.check_status()
    assert cache.seq_lens_host.tolist() == [0, 33, 0, 1] and cache.seq_lens_dev.tolist() == [0, 33, 0, 1]
    assert cache.free_pages() == pages + -(-50 // cache.block_size) and bool((cache.table[0] == -1).all())
    assert int((w[0, :50] != 0).sum()) == 0 and torch.equal(w[0, 50:], behind[0, 50:]) and torch.equal(w[1:], behind[1:])
    kept = cache.select_rows(w, [(3, 0), (1, 7), (0, 0)])
    check_evict(cache, [(3, 0), (1, 7), (0, 0)], [[], kept[1, :7].tolist(), []], weights=w)
    cache.select_rows(w[:, :0], [(3, 0), (2, 0)])  # requests without rows have no weights
    kept = cache.select_rows(w, [(1, 0)])
    cache.evict([(1, 0)], kept)
    torch.cuda.synchronize()
    cache.check_status()
    assert cache.free_pages() == cache.num_pages and int(cache.seq_lens_host.sum()) == 0
    if cache.pending() is not None:
        assert int(cache.pending().abs().sum()) == 0
    cache.close()


# ------------------------------------------------------------------- weigh --
def test_a_step_without_tokens_takes_what_attention_returned():
    cache = BH.make_cache([100], seed=4, layers=1)
    b = cache.batch(2, 4, 8)
    w = fresh_weights(cache)
    want = w.clone()
    for chunks in ([], [(0, 100, 0)]):
        b.plan(chunks)
        ql, q = queries(cache, 0, 8)
        out, lse = b.attention(0, ql, q, 0.1)
        assert tuple(lse.shape) == (0, 8)
        b.attention_weights(0, ql, q, lse, 0.1, w)
        b.attention_weights(0, ql, q, lse, 0.1, w[:0])
    torch.cuda.synchronize()
    cache.check_status()
    assert torch.equal(w, want)
    b.close()
    cache.close()


PASSING = {  # more than 128 query rows a band, two chunks of one request, items that are cut and joined
    "mla": (dict(), 20), "mla b1": (dict(B=1), 20), "mla lazy": (dict(flags=LAZY), 20), "mla split": (dict(flags=SPLIT), 7),
    "mla lazy b1": (dict(flags=LAZY, B=1), 33), "mla 128 heads": (dict(), 128), "mla lazy 150 heads": (dict(flags=LAZY), 150),
    "grouped": (dict(rope=128, bands=4), 16), "grouped lazy": (dict(rope=128, bands=2, flags=LAZY), 20),
    "grouped 64 b1": (dict(rope=64, bands=2, B=1), 130), "grouped lazy 256": (dict(rope=256, bands=2, flags=LAZY), 12)}
CHUNKS = [(0, 200, 40), (1, 100, 30), (0, 250, 20)]  # of requests of 300 and 200 rows


def passing(shape):
    kw, per_band = PASSING[shape]
    cache = BH.make_cache([300, 200], seed=5, layers=1, **kw)
    heads = per_band * cache.rope_heads
    if cache.pending() is not None:
        cache.pending().random_(-300, 300)
    b = cache.batch(4, 90, heads)
    b.plan(CHUNKS)
    b.append(0, BH.bf16(90, cache.row, seed=8))
    ql, q = queries(cache, 90, heads, seed=9)
    lse = 2 + torch.rand(90, heads, device="cuda")
    return cache, b, heads, ql, q, lse


@pytest.mark.parametrize("shape", PASSING)
def test_rows_that_hold_nothing_where_queries_pass(shape):
    cache, b, heads, ql, q, lse = passing(shape)
    for req, n in ((0, 270), (1, 130)):  # rows behind the chunks
        flat = torch.from_numpy(cache.slot_index(req, np.arange(n, int(cache.seq_lens_host[req])))).cuda()
        bad = torch.full((len(flat), cache.row), NAN, device="cuda", dtype=torch.bfloat16)
        bad[::2] = INF
        cache.write_layer_rows(0, flat, bad)
    scale = 0.1
    for what in ("some heads", "a token", "a chunk"):
        holes = torch.zeros(90, heads, dtype=torch.bool, device="cuda")
        if what == "some heads":
            holes[::3, ::2] = True
        elif what == "a token":
            holes[[0, 39, 40, 89]] = True
        else:
            holes[40:70] = True
        x = lse.clone()
        x[holes] = -INF
        no = q.clone()  # queries that attend to nothing may hold anything
        no[holes] = NAN
        nol = None if ql is None else torch.where(holes[..., None], torch.full_like(ql, INF), ql)
        for decay, prefix in ((1.0, False), (0.0, True)):
            w = fresh_weights(cache, seed=1)
            if decay == 0.0:
                w.fill_(NAN)
            check_weigh(cache, b, 0, CHUNKS, nol, no, x, scale, w, decay, prefix, f"{shape} {what}")
            assert bool(w[0, :270].isfinite().all()) and bool(w[1, :130].isfinite().all())
        y = lse.clone()
        y[holes] = INF  # so high that nothing is left
        w1, w2 = fresh_weights(cache, seed=2), fresh_weights(cache, seed=2)
        b.attention_weights(0, ql, q, y, scale, w1)
        b.attention_weights(0, ql, q, x, scale, w2)
        assert torch.equal(w1, w2), what
    # attended rows that are not finite spoil their own weights alone
    rows = np.array([17, 255, 256, 269])
    flat = torch.from_numpy(cache.slot_index(0, rows)).cuda()
    cache.write_layer_rows(0, flat, torch.full((4, cache.row), NAN, device="cuda", dtype=torch.bfloat16))
    w3 = fresh_weights(cache, seed=2)
    b.attention_weights(0, ql, q, x, scale, w3)
    spoilt = torch.zeros_like(w3, dtype=torch.bool)
    spoilt[0, torch.from_numpy(rows).cuda()] = True
    assert bool(w3[spoilt].isnan().all()) and torch.equal(w3[~spoilt], w2[~spoilt])
    torch.cuda.synchronize()
    cache.check_status()
    b.close()
    cache.close()


@pytest.mark.parametrize("shape", PASSING)
def test_bad_pages_where_queries_pass(shape):
    """In a full tile of 256 rows and in a partial one: the rows of the page keep their weights, all others get theirs."""
    from rope_rotation_gb300.leyline import LeylineError
    cache, b, heads, ql, q, lse = passing(shape)
    B = cache.block_size
    old = fresh_weights(cache, seed=4)
    want = old.clone()
    b.attention_weights(0, ql, q, lse, 0.1, want)
    cache.check_status()
    for row in (48, 258):
        blk = row // B
        held = cache.table[0, blk].item()
        for page in (-1, cache.num_pages, 2 ** 31 - 1):
            cache.table[0, blk] = page
            got = old.clone()
            b.attention_weights(0, ql, q, lse, 0.1, got)
            with pytest.raises(LeylineError) as e:
                cache.check_status()
            assert e.value.code == -8
            gone = torch.zeros_like(got, dtype=torch.bool)
            gone[0, blk * B:(blk + 1) * B] = True
            assert torch.equal(got[gone], old[gone]) and torch.equal(got[~gone], want[~gone])
        cache.table[0, blk] = held
    got = old.clone()
    b.attention_weights(0, ql, q, lse, 0.1, got)
    torch.cuda.synchronize()
    cache.check_status()
    assert torch.equal(got, want)
    b.close()
    cache.close()


@pytest.mark.parametrize("shape", ["mla", "mla lazy b1", "grouped", "grouped 64 b1"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_a_table_entry_of_any_value_is_reported(shape, tokens):
    """The smallest number of all is a bad page like any other, where queries stay and where they pass."""
    from rope_rotation_gb300.leyline import LeylineError
    kw, per_band = PASSING[shape]
    cache = BH.make_cache([300], seed=6, layers=1, **kw)
    heads = min(per_band, 64) * cache.rope_heads
    b = cache.batch(1, tokens, heads)
    b.plan([(0, 300 - tokens, tokens)])
    b.append(0, BH.bf16(tokens, cache.row))
    ql, q = queries(cache, tokens, heads)
    lse = torch.ones(tokens, heads, device="cuda")
    w = fresh_weights(cache)
    b.attention_weights(0, ql, q, lse, 0.1, w)
    cache.check_status()
    held = cache.table[0, 3].item()
    cache.table[0, 3] = -2 ** 31
    b.attention_weights(0, ql, q, lse, 0.1, w)
    with pytest.raises(LeylineError) as e:
        cache.check_status()
    assert e.value.code == -8
    cache.table[0, 3] = held
    b.close()
    cache.close()


# ---------------------------------------------------------------- accuracy --
NEAR = {
    "mla": dict(), "mla b1": dict(B=1), "mla split": dict(flags=SPLIT), "mla lazy": dict(flags=LAZY),
    "mla lazy b1 pairs": dict(flags=LAZY, B=1, pair_layout=1), "mla lazy split": dict(flags=LAZY | SPLIT, B=8),
    "grouped 64": dict(rope=64, bands=4), "grouped 64 lazy": dict(rope=64, bands=4, flags=LAZY),
    "grouped 128": dict(rope=128, bands=4), "grouped 128 lazy": dict(rope=128, bands=4, flags=LAZY),
    "grouped 256": dict(rope=256, bands=2), "grouped 256 lazy pairs": dict(rope=256, bands=2, flags=LAZY, pair_layout=1),
    "odd": dict(latent=72, rope=48), "odd bands lazy": dict(latent=96, rope=96, bands=3, flags=LAZY)}


@pytest.mark.parametrize("shape", NEAR)
@pytest.mark.parametrize("per_band", [1, 16, 40, 72, 128])
def test_weights_are_near_those_of_64_bits(shape, per_band):
    """In the 2-norm over a request's rows, within 2^-16: keys of 1 to 10 blocks of 64 columns by 1 to 128 query rows a band,
    which stay, and by some more, which pass.

    Inputs are N(0, 1) and scores of standard deviation 1, so the largest weights, which the norm goes by, have scores up to
    5 and an lse of some 3.  An accumulator of the matrix unit that cuts its sum off at each of its up to 40 steps loses up to
    2^-23 of it a step; it grows from 0 to the score, so 40 * 2^-23 * 5 / 2 = 1.2e-5 at most, every step cut by a whole bit.  The
    exponent is rounded three times, 2^-24 of 8 each, 1.4e-6, the exponential and the sum add 2^-21.  A lazy band is the
    sum of two bf16 values, off by 2^-18 of a pair at most and with both signs: over 64 products of the band alone 8 *
    2^-18 / 8 = 3.8e-6 of a score's standard deviation, mostly averaged out over queries.  With one bf16 value instead it
    would be 2e-3 (where queries stay), and 1e-4 over 130 queries."""
    kw = NEAR[shape]
    lens = [1500, 700, 130]
    cache = BH.make_cache(lens, extra=0, seed=7, layers=1, **kw)
    heads = per_band * cache.rope_heads
    few = [(r, n - 1, 1) for r, n in enumerate(lens)]
    many = -(-130 // per_band)  # tokens of more than 128 query rows a band
    some = [(r, n - many, many) for r, n in enumerate(lens) if n > many]
    turns = torch.randint(-4000, 300, cache.pending().shape, device="cuda", dtype=torch.int32) if cache.pending() is not None else None
    for chunks in (few, some):
        n = sum(c[2] for c in chunks)
        b = cache.batch(3, n, heads)
        b.plan(chunks)
        if turns is not None:
            torch.cuda.synchronize()
            cache.pending().copy_(turns)
        for band_alone in (False, True):
            if cache.rope_heads > 1 and band_alone:
                continue
            ql, q = queries(cache, n, heads, seed=10)
            d = cache.rope_dim
            if ql is not None and band_alone:
                ql.zero_()
            elif ql is not None:
                d += cache.latent_dim
            scale = d ** -0.5
            lse = 3 + torch.rand(n, heads, device="cuda")
            w = torch.full((3, cache.table.shape[1] * cache.block_size), NAN, device="cuda")
            want, tol, written = weights64(cache, 0, chunks, ql, q, lse, scale, w, 0.0, pair_layout=kw.get("pair_layout", 0))
            b.attention_weights(0, ql, q, lse, scale, w, 0.0)
            torch.cuda.synchronize()
            cache.check_status()
            for req, start, m in chunks:
                on = written[req]
                got, ref = w[req][on].double(), want[req][on]
                off = float((got - ref).norm() / ref.norm())
                assert off <= 2.0 ** -16, f"{shape} {per_band} {m} tokens, request {req}, band alone {band_alone}: {off}"
                assert bool(((got - ref).abs() <= tol[req][on]).all())
        b.close()
    cache.close()


@pytest.mark.parametrize("kw,per_band,tokens", [
    (dict(), 20, 8), (dict(B=1), 128, 6), (dict(flags=LAZY), 20, 8), (dict(), 1, 1), (dict(), 16, 1), (dict(), 128, 1), (dict(B=1), 96, 1),
    (dict(rope=256, bands=2), 20, 8), (dict(rope=256, bands=2), 8, 1), (dict(rope=128, bands=4), 20, 8), (dict(rope=64, bands=4), 3, 1)])
def test_scores_are_not_biased(kw, per_band, tokens):
    """The logarithm of a weight that one query alone gives is its score x.  Over rows with scores of many sizes and both signs,
    |x| above an eighth of the largest, x is off by less than 2^-22 of itself in the mean.

    An accumulator of the matrix unit cuts off half of its last bit a step on average, 0.72 * 2^-24 of what it holds; over n steps
    that add up to x evenly (n + 1) / 2 times that at most, 8e-7 x for the 36 of an MLA key.  The kernels make up for 1.75e-8 (n - 1),
    6.1e-7 x.  So x is 1.9e-7 too small at most, and if nothing were cut off in the first half of the steps 1.5e-7 too large.
    2^-22 is 2.4e-7.  The factor's rounding adds 2^-25, and what differs from row to row averages out.  (One accumulator for MLA keys was
    6.7e-7 too small, two 3.2e-7.)"""
    n = 4096
    cache = BH.make_cache([n], seed=1, layers=1, **kw)
    heads, lat, d = per_band * cache.rope_heads, cache.latent_dim, cache.rope_dim
    mla = cache.rope_heads == 1
    b = cache.batch(1, tokens, heads)
    b.plan([(0, n - tokens, tokens)])
    g = torch.Generator(device="cuda").manual_seed(5)
    width = d + (lat if mla else 0)
    query = torch.randn(width, generator=g, device="cuda").bfloat16()
    keys = (torch.linspace(-1.5, 1.5, n, device="cuda")[:, None] * query.float()
            + 0.7 * torch.randn(n, width, generator=g, device="cuda")).bfloat16()
    flat = torch.from_numpy(cache.slot_index(0, np.arange(n))).cuda()
    rows = BH.bf16(n, cache.row, seed=2)
    rows[:, 0 if mla else lat:(0 if mla else lat) + width] = keys
    cache.write_layer_rows(0, flat, rows)
    ql, q = queries(cache, tokens, heads, seed=3)
    if mla:
        ql[0, 0] = query[:lat]
    q[0, 0] = query[-d:]
    lse = torch.full((tokens, heads), INF, device="cuda")
    lse[0, 0] = 0.0
    scale = 2.0 ** -5  # exact
    w = torch.zeros(1, cache.table.shape[1] * cache.block_size, device="cuda")
    b.attention_weights(0, ql, q, lse, scale, w, 0.0)
    torch.cuda.synchronize()
    cache.check_status()
    seen = n - tokens + 1
    want = (keys.double() @ query.double())[:seen]
    got = w[0, :seen].double().log() / scale
    on = want.abs() > want.abs().max() / 8
    off = float(((got - want) / want)[on].mean())
    assert abs(off) < 2.0 ** -22, f"{kw} {per_band} {tokens}: {off}"
    b.close()
    cache.close()
