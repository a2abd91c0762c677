"""Eviction by attention weight on the GPU: the weights that queries give to rows, the choice of the rows to keep, the
removal of the others, and a run of them together, against plain forms in 64 bits (see batch_harness)."""
import math

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

LAZY, SPLIT, REINDEX = 2, 4, 1
NAN = float("nan")


# ------------------------------------------------------------------- weigh --
def weights64(cache, layer, chunks, q_latent, q_rope, lse, scale, weights, decay, prefix=False, pair_layout=0):
    """(weights, tolerance) in fp64, and which of them the call writes.  The tolerance follows from the arithmetic: a
    score is off by dx as in batch_harness.attention64 (an fp32 sum of d products, the turn of a lazy key), the exponent
    x - lse by three roundings of terms of their sizes (2^-22 of |x| + |lse|), the exponential by 2^-21, a sum of n
    positive terms in any order by n * 2^-24 of itself, and decay * w + sum by two roundings."""
    out = weights.double().clone()
    tol = torch.zeros_like(out)
    written = torch.zeros_like(out, dtype=torch.bool)
    H, G, lat, t0 = q_rope.shape[1], cache.rope_heads, cache.latent_dim, 0
    sums, errs, ends = {}, {}, {}
    for req, start, n in [c[:3] for c in chunks]:
        if n == 0:
            continue
        end = start + n
        got = torch.zeros(end, dtype=torch.float64, device="cuda")
        err = torch.zeros_like(got)
        rows, flat = BH.logical(cache, req, layer, end)
        rows = rows.double()
        keys = rows[:, lat:].view(end, G, -1)
        lazy = cache.pending() is not None
        if lazy:
            keys = BH.turn64(keys, cache.pending().view(-1)[flat][:, None].expand(end, G), pair_layout=pair_layout)
        seen = torch.arange(end, device="cuda") <= (start - 1 if prefix else start + torch.arange(n, device="cuda")[:, None])
        seen = seen.expand(n, end)
        for h in range(H):
            k = keys[:, h * G // H]
            q = q_rope[t0:t0 + n, h].double()
            x, mag, d = q @ k.T, q.abs() @ k.abs().T, k.shape[1]
            turn = q.abs() @ BH.pair_norm(k, pair_layout).T * (2.0 ** -17 + 2.0 ** -20) if lazy else 0.0
            if G == 1:
                ql = q_latent[t0:t0 + n, h].double()
                x, mag, d = x + ql @ rows[:, :lat].T, mag + ql.abs() @ rows[:, :lat].abs().T, d + lat
            s = lse[t0:t0 + n, h].double()[:, None]
            on = seen & (s > -math.inf)
            p = torch.where(on, torch.exp(x * scale - s), 0.0)
            dx = abs(scale) * (mag * d * 2.0 ** -23 + turn) + 2.0 ** -22 * ((x * scale).abs() + s.abs())
            got += p.sum(0)
            err += torch.where(on, p * (dx + 2.0 ** -21 + n * H * 2.0 ** -24), 0.0).sum(0)
        sums.setdefault(req, torch.zeros(out.shape[1], dtype=torch.float64, device="cuda"))[:end] += got
        errs.setdefault(req, torch.zeros(out.shape[1], dtype=torch.float64, device="cuda"))[:end] += err
        ends[req] = max(ends.get(req, 0), end)
        t0 += n
    for req, end in ends.items():
        old = out[req, :end] * decay if decay else torch.zeros_like(out[req, :end])
        out[req, :end] = old + sums[req][:end]
        tol[req, :end] = errs[req][:end] + 2.0 ** -23 * (old.abs() + sums[req][:end])
        written[req, :end] = True
    return out, tol, written


def check_weigh(cache, batch, layer, chunks, q_latent, q_rope, lse, scale, weights, decay=1.0, prefix=False, what="",
                pair_layout=0):
    want, tol, written = weights64(cache, layer, chunks, q_latent, q_rope, lse, scale, weights, decay, prefix, pair_layout)
    before = weights.clone()
    got = batch.attention_weights(layer, q_latent, q_rope, lse, scale, weights, decay, prefix)
    assert got is weights
    torch.cuda.synchronize()
    cache.check_status()
    off = (got.double() - want).abs()
    assert bool((off[written] <= tol[written]).all()), \
        f"{what}: off by {float((off[written] / tol[written].clamp_min(1e-300)).nan_to_num(1e9).max())} of its tolerance"
    assert torch.equal(got[~written].view(torch.int32), before[~written].view(torch.int32)), f"{what}: other rows changed"


def queries(cache, tokens, heads, seed=0, scale=1.0):
    ql = BH.bf16(tokens, heads, cache.latent_dim, seed=seed, scale=scale) if cache.rope_heads == 1 else None
    return ql, BH.bf16(tokens, heads, cache.rope_dim, seed=seed + 1, scale=scale)


def fresh_weights(cache, seed=0, rows=None, nan_from=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(cache.table.shape[0], rows or cache.table.shape[1] * cache.block_size, generator=g, device="cuda")
    if nan_from is not None:
        w[:, nan_from:] = NAN
    return w


SHAPES = {
    "mla": dict(), "mla b1": dict(B=1), "mla b5": dict(B=5), "mla b8": dict(B=8), "mla b64": dict(B=64),
    "mla split": dict(flags=SPLIT), "mla lazy": dict(flags=LAZY), "mla lazy b1": dict(flags=LAZY, B=1),
    "mla lazy split b8": dict(flags=LAZY | SPLIT, B=8), "mla lazy pairs": dict(flags=LAZY, pair_layout=1),
    "grouped": dict(rope=128, bands=4), "grouped b1": dict(rope=128, bands=4, B=1),
    "grouped lazy": dict(rope=128, bands=4, flags=LAZY), "grouped split 64": dict(rope=64, bands=8, flags=SPLIT),
    "grouped lazy pairs 256": dict(rope=256, bands=2, flags=LAZY, pair_layout=1),
    "grouped lazy b5 64": dict(rope=64, bands=4, flags=LAZY, B=5), "grouped 256": dict(rope=256, bands=2),
    "odd": dict(latent=64, rope=16), "odd lazy": dict(latent=72, rope=48, flags=LAZY), "odd bands": dict(latent=48, rope=32, bands=3),
    "wide": dict(latent=1024, rope=256), "odd bands lazy": dict(latent=96, rope=96, bands=3, flags=LAZY, pair_layout=1),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("per_band", [1, 5, 16])
def test_weigh_matches_the_formula(shape, per_band):
    kw = SHAPES[shape]
    lens = [1, 130, 700, 0, 64, 257]
    cache = BH.make_cache(lens, extra=160, seed=3, **kw)
    if cache.pending() is not None:
        turns = torch.randint(-4000, 300, cache.pending().shape, device="cuda", dtype=torch.int32)
        turns[torch.rand(cache.pending().shape, device="cuda") < 0.4] = 0
        cache.pending()[:, :] = turns
        cache.pending()[::3] = 77  # and pages that share one
    heads = per_band * cache.rope_heads
    chunk_sets = [[(1, 129, 1), (2, 699, 1), (4, 63, 1), (0, 0, 1), (5, 256, 1)],
                  [(2, 640, 60), (5, 257, 40), (3, 0, 9), (1, 0, 0)],
                  [(2, 300, 20), (4, 64, 150), (2, 700, 3)]]
    b = cache.batch(8, 400, heads)
    scale = (cache.rope_dim + (128 if cache.rope_heads == 1 else 0)) ** -0.5
    for i, chunks in enumerate(chunk_sets):
        b.plan(chunks)
        n = sum(c[2] for c in chunks)
        for layer in range(2):  # the chunks' rows, which hold nothing yet
            b.append(layer, BH.bf16(n, cache.row, seed=40 + i))
        ql, q = queries(cache, n, heads, seed=50 + i)
        lse = 3 + torch.randn(n, heads, device="cuda")
        for decay, prefix in ((1.0, False), (0.9, True), (0.0, False)):
            w = fresh_weights(cache, seed=i)
            if decay == 0.0:
                w.fill_(NAN)
            check_weigh(cache, b, 1, chunks, ql, q, lse, scale, w, decay, prefix, f"{shape} {i} {decay}",
                        kw.get("pair_layout", 0))
    b.close()
    cache.close()


@pytest.mark.parametrize("heads,tokens,length,kw", [
    (128, 1, 5000, {}), (128, 9, 3000, {}), (130, 2, 1000, {}), (200, 1, 700, {}), (300, 3, 400, {}), (20, 33, 2000, {}),
    (40, 4, 4100, dict(B=1)), (16, 200, 1500, dict(flags=LAZY)), (128, 5, 900, dict(flags=LAZY, B=1)),
    (64, 100, 1300, dict(rope=128, bands=4)), (32, 7, 6000, dict(rope=128, bands=4, flags=LAZY)),
    (32, 1, 3000, dict(rope=128, bands=32)), (512, 2, 600, dict(rope=64, bands=2)), (1024, 1, 300, {}),
    (16, 1, 1, {}), (16, 2, 2, {}), (3, 17, 17, {}), (64, 300, 300, {})])
def test_weigh_many_query_rows(heads, tokens, length, kw):
    """Chunks at the end of requests, one of them alone and beside shorter ones."""
    if kw.get("bands") == 32:
        kw = dict(kw, latent=2048 // 2)
    cache = BH.make_cache([length, max(length // 3, tokens), length], layers=1, seed=4, **kw)
    if cache.pending() is not None:
        cache.pending().random_(-300, 300)
    b = cache.batch(3, 3 * tokens, heads)
    ql, q = queries(cache, 3 * tokens, heads, seed=6, scale=0.7)
    scale = 192 ** -0.5
    for reqs in ((0,), (2, 1, 0)):
        chunks = [(r, int(cache.seq_lens_host[r]) - tokens, tokens) for r in reqs]
        b.plan(chunks)
        n = tokens * len(reqs)
        rows = BH.bf16(n, cache.row, seed=7)
        b.append(0, rows)
        _, lse = b.attention(0, ql, q, scale)
        w = torch.zeros(3, cache.table.shape[1] * cache.block_size, device="cuda")
        check_weigh(cache, b, 0, chunks, ql, q, lse, scale, w, what=f"{heads} {tokens} {length} {reqs}")
        # every query row gives 1 in all
        total = w.double().sum(1)
        want = torch.tensor([float(tokens * heads) if r in reqs else 0.0 for r in range(3)], dtype=torch.float64, device="cuda")
        assert bool(((total - want).abs() <= 2.0 ** -9 * want).all())
    b.close()
    cache.close()


@pytest.mark.parametrize("latent", [64, 128, 192, 256, 320, 448, 512])
@pytest.mark.parametrize("rope,flags", [(64, 0), (128, 0), (64, LAZY), (128, LAZY)])
def test_weigh_keys_of_few_columns(latent, rope, flags):
    """Keys of 2 to 12 blocks of 64 columns, by 16 to 128 query rows."""
    lens = [300, 31, 1]
    cache = BH.make_cache(lens, seed=21, layers=1, latent=latent, rope=rope, flags=flags)
    if cache.pending() is not None:
        cache.pending().random_(-300, 300)
    for heads in (16, 40, 72, 128):
        b = cache.batch(3, 3, heads)
        chunks = [(r, n - 1, 1) for r, n in enumerate(lens)]
        b.plan(chunks)
        ql, q = queries(cache, 3, heads, seed=22)
        lse = 3 + torch.randn(3, heads, device="cuda")
        check_weigh(cache, b, 0, chunks, ql, q, lse, 0.07, fresh_weights(cache, seed=1), 0.5, what=f"{latent} {rope} {heads}")
        b.close()
    cache.close()


@pytest.mark.parametrize("kw", [{}, dict(B=1), dict(flags=LAZY), dict(rope=128, bands=4), dict(latent=64, rope=16)])
def test_weigh_rows_that_hold_nothing(kw):
    """NaN and infinities in rows that no token attends to reach no other row's weight; a query row without an lse adds
    nothing; the largest and the most negative lse neither."""
    cache = BH.make_cache([300, 200], seed=5, layers=1, **kw)
    heads = 4 * cache.rope_heads
    b = cache.batch(2, 16, heads)
    chunks = [(0, 290, 5), (1, 0, 7)]  # rows behind both chunks
    b.plan(chunks)
    b.append(0, BH.bf16(12, cache.row, seed=8))
    for req, n in ((0, 295), (1, 7)):
        flat = torch.from_numpy(cache.slot_index(req, np.arange(n, int(cache.seq_lens_host[req])))).cuda()
        bad = torch.full((len(flat), cache.row), NAN, device="cuda", dtype=torch.bfloat16)
        bad[::2] = float("inf")
        cache.write_layer_rows(0, flat, bad)
    ql, q = queries(cache, 12, heads, seed=9)
    lse = 2 + torch.rand(12, heads, device="cuda")
    lse[3] = -math.inf
    lse[7, ::2] = -math.inf
    w = fresh_weights(cache, seed=1)
    check_weigh(cache, b, 0, chunks, ql, q, lse, 0.1, w, what="holes")
    assert bool(w[0, :295].isfinite().all()) and bool(w[1, :7].isfinite().all())
    # one attended row that is not finite spoils its own weight alone
    flat = torch.from_numpy(cache.slot_index(0, np.array([17]))).cuda()
    cache.write_layer_rows(0, flat, torch.full((1, cache.row), NAN, device="cuda", dtype=torch.bfloat16))
    w2 = fresh_weights(cache, seed=1)
    b.attention_weights(0, ql, q, lse, 0.1, w2)
    assert bool(w2[0, 17].isnan()) and torch.equal(torch.cat((w2[0, :17], w2[0, 18:295])), torch.cat((w[0, :17], w[0, 18:295])))
    # negative and zero scales; lse so high that nothing is left
    for scale in (-0.2, 0.0):
        w = fresh_weights(cache, seed=2)
        b.plan([(1, 0, 7)])
        check_weigh(cache, b, 0, [(1, 0, 7)], None if ql is None else ql[:7], q[:7], lse[:7], scale, w, what=f"scale {scale}")
    b.plan(chunks)
    w = fresh_weights(cache, seed=2)
    want = w.clone()
    b.attention_weights(0, ql, q, torch.full_like(lse, math.inf), 0.1, w)
    assert torch.equal(torch.cat((w[0, :17], w[0, 18:])), torch.cat((want[0, :17], want[0, 18:])))
    cache.check_status()
    b.close()
    cache.close()


@pytest.mark.parametrize("kw", [dict(), dict(rope=128, bands=4), dict(latent=64, rope=16), dict(B=1, pair_layout=1)])
def test_weigh_turns_of_any_count(kw):
    """Counts up to the ends of their type.  Angles of 2^31 radians in fp64, here and in the formula, are off by 2^-21."""
    cache = BH.make_cache([900, 300], seed=25, layers=1, flags=LAZY, **kw)
    ends = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 26, -2 ** 26 - 1, 2 ** 20 + 1, 0, -1], dtype=torch.int32, device="cuda")
    cache.pending().copy_(ends[torch.randint(0, 7, cache.pending().shape, device="cuda")])
    heads = 16 * cache.rope_heads
    b = cache.batch(2, 80, heads)
    for chunks in ([(0, 899, 1), (1, 299, 1)], [(0, 840, 60)]):
        was = cache.pending().clone()
        b.plan(chunks)
        torch.cuda.synchronize()
        cache.pending().copy_(was)
        tokens = sum(c[2] for c in chunks)
        ql, q = queries(cache, tokens, heads, seed=26)
        lse = 3 + torch.randn(tokens, heads, device="cuda")
        check_weigh(cache, b, 0, chunks, ql, q, lse, 0.07, fresh_weights(cache, seed=1), what=f"{kw}",
                    pair_layout=kw.get("pair_layout", 0))
    b.close()
    cache.close()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("lat,rope,bands", [(512, 64, 1), (512, 128, 4), (512, 64, 8), (512, 256, 2), (72, 48, 1), (96, 96, 3)])
def test_weigh_lazy_naive_pools(lat, rope, bands, layout):
    """With the naive rounding a turned band is a bf16 value: a lazy pool's rows weigh what those of an eager pool do that
    holds what a gather returns."""
    lens = [1234, 77]
    kw = dict(extra=8, precision=1, latent=lat, rope=rope, bands=bands, pair_layout=layout)
    lazy, eager = BH.make_cache(lens, flags=LAZY, **kw), BH.make_cache(lens, **kw)
    for r, n in enumerate(lens):
        flat = torch.from_numpy(lazy.slot_index(r, np.arange(n))).cuda()
        turns = torch.from_numpy(np.random.default_rng(r).integers(-9000, 9000, n // 10 + 1).astype(np.int32)).cuda()
        lazy.pending().view(-1)[flat] = turns[torch.arange(n, device="cuda") // 10]
        flat_e = torch.from_numpy(eager.slot_index(r, np.arange(n))).cuda()
        for layer in range(2):
            eager.write_layer_rows(layer, flat_e, lazy.gather(r, layer, 0, n))
    heads = 8 * bands
    b = lazy.batch(2, 120, heads)
    for chunks in ([(0, 1233, 1), (1, 75, 2)], [(0, 1100, 110), (1, 70, 7)]):
        tokens = sum(c[2] for c in chunks)
        was = lazy.pending().clone()
        b.plan(chunks)  # clears the counts of the chunks' rows, which are to be written: here they stay
        torch.cuda.synchronize()
        lazy.pending().copy_(was)
        ql, q = queries(lazy, tokens, heads, seed=24)
        lse = 3 + torch.randn(tokens, heads, device="cuda")
        w = fresh_weights(lazy, seed=2)
        want, tol, written = weights64(eager, 1, chunks, ql, q, lse, 0.07, w, 0.5)
        b.attention_weights(1, ql, q, lse, 0.07, w, 0.5)
        torch.cuda.synchronize()
        lazy.check_status()
        assert bool(((w.double() - want).abs()[written] <= tol[written]).all())
    b.close()
    lazy.close()
    eager.close()


def test_weigh_strided_tensors_and_same_bits():
    cache = BH.make_cache([900, 70], seed=6, layers=2)
    b = cache.batch(2, 40, 24)
    chunks = [(0, 880, 20), (1, 60, 10)]
    b.plan(chunks)
    for layer in range(2):
        b.append(layer, BH.bf16(30, cache.row, seed=3))
    wide = BH.bf16(30, 24, 1152, seed=4)
    ql, q = wide[..., 64:576], wide[..., 1024:1088]
    lse = 2 + torch.rand(30, 24, device="cuda")
    w = fresh_weights(cache, seed=3, rows=1500)[:, 100:1100]  # rows of a wider tensor
    check_weigh(cache, b, 1, chunks, ql, q, lse, 0.07, w, what="strided")
    heads_first = BH.bf16(24, 30, 576, seed=5).transpose(0, 1)
    w1, w2 = fresh_weights(cache, seed=3), fresh_weights(cache, seed=3)
    check_weigh(cache, b, 0, chunks, heads_first[..., :512], heads_first[..., 512:], lse, 0.07, w1, what="heads first")
    b.attention_weights(0, heads_first[..., :512], heads_first[..., 512:], lse, 0.07, w2)
    assert torch.equal(w1, w2)
    one = BH.bf16(1, 1, 576, seed=5).expand(30, 24, 576)  # broadcast queries
    check_weigh(cache, b, 0, chunks, one[..., :512], one[..., 512:], lse, 0.07, w1, what="broadcast")
    stream = torch.cuda.Stream()
    w3 = w1.clone()
    torch.cuda.synchronize()
    b.attention_weights(0, one[..., :512], one[..., 512:], lse, 0.07, w1)
    b.attention_weights(0, one[..., :512], one[..., 512:], lse, 0.07, w3, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(w1, w3)
    b.close()
    cache.close()


@pytest.mark.parametrize("kw", [{}, dict(flags=LAZY, B=1), dict(rope=128, bands=4), dict(latent=64, rope=16)])
def test_weigh_captured_and_replayed(kw):
    """A graph of attention and its weights is replayed after plans of other shapes."""
    lens = [3000, 500, 40]
    cache = BH.make_cache(lens, extra=600, seed=7, layers=1, **kw)
    heads = 8 * cache.rope_heads
    b = cache.batch(4, 300, heads)
    ql, q = queries(cache, 300, heads, seed=10)
    w = torch.zeros(3, cache.table.shape[1] * cache.block_size, device="cuda")
    b.plan([(0, 2999, 1)])
    out, lse = b.attention(0, ql, q, 0.05)
    b.attention_weights(0, ql, q, lse, 0.05, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attention(0, ql, q, 0.05, out=out, lse=lse)
        b.attention_weights(0, ql, q, lse, 0.05, w, decay=0.5)
    for chunks in ([(0, 2999, 1), (1, 499, 1)], [(0, 2800, 200), (2, 40, 90)], [(1, 0, 290)], [],
                   [(2, 0, 1), (1, 450, 50), (2, 1, 3), (0, 0, 1)]):
        b.plan(chunks)
        n = sum(c[2] for c in chunks)
        if n:
            b.append(0, BH.bf16(n, cache.row, seed=11))
        w0 = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        cache.check_status()
        if n:
            _, lse1 = b.attention(0, ql, q, 0.05)
            b.attention_weights(0, ql, q, lse1, 0.05, w0, decay=0.5)
        assert torch.equal(w, w0), chunks
    # under capture the weights need room for any plan
    from rope_rotation_gb300.leyline import LeylineError
    b.plan([(2, 0, 2)])
    x = torch.zeros(1, device="cuda")
    for small in (torch.full((3, 64), 0.25, device="cuda"), torch.full((2, w.shape[1]), 0.25, device="cuda")):
        with pytest.raises(LeylineError):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                x += 1
                b.attention_weights(0, ql, q, lse, 0.05, small)
    b.close()
    cache.close()


@pytest.mark.parametrize("kw,heads", [({}, 16), (dict(flags=LAZY, B=1), 16), (dict(rope=128, bands=4), 32), ({}, 128)])
def test_weigh_steps_of_decodes_and_a_chunk(kw, heads):
    """Plans whose requests go to two kernels: many decoded tokens beside chunks of a prompt."""
    lens = [4200] * 20 + [700, 3, 1500]
    cache = BH.make_cache(lens, seed=18, layers=1, **kw)
    if cache.pending() is not None:
        cache.pending().random_(-300, 300)
    b = cache.batch(40, 600, heads)
    scale = 0.06
    w = fresh_weights(cache, seed=1)
    graph = None
    for chunks in ([(r, 4199 - r, 1) for r in range(20)] + [(20, 500, 200)],
                   [(22, 0, 300), (20, 0, 0)] + [(r, 4199, 1) for r in (5, 3, 7)] + [(21, 2, 1)],
                   [(20, 690, 10)] + [(r, 4100, 2) for r in reversed(range(20))] + [(22, 1499, 1), (20, 600, 3)]):
        b.plan(chunks)
        n = sum(c[2] for c in chunks)
        b.append(0, BH.bf16(n, cache.row, seed=19))
        ql, q = queries(cache, 600, heads, seed=20)
        lse = 3 + torch.randn(600, heads, device="cuda")
        check_weigh(cache, b, 0, chunks, ql, q, lse, scale, w, 0.5, what=f"{chunks[0]}")
        if graph is None:
            ql0, q0, lse0, w0 = ql, q, lse, torch.zeros_like(w)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                b.attention_weights(0, ql0, q0, lse0, scale, w0)
        w0.zero_()
        graph.replay()
        torch.cuda.synchronize()
        cache.check_status()
        one = torch.zeros_like(w)
        b.attention_weights(0, ql0, q0, lse0, scale, one)
        assert torch.equal(w0, one)  # a replay gives what a call does
    b.close()
    cache.close()


@pytest.mark.parametrize("kw", [{}, dict(rope=128, bands=4), dict(latent=64, rope=16)])
@pytest.mark.parametrize("tokens", [1, 80])
def test_weigh_replayed_for_another_table(kw, tokens):
    """Weights that do not hold a replayed plan's requests or rows: those requests' are left as they were."""
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([400, 90], extra=200, seed=17, layers=1, **kw)
    heads = 8 * cache.rope_heads
    b = cache.batch(4, 300, heads)
    ql, q = queries(cache, 300, heads, seed=10)
    lse = 3 + torch.randn(300, heads, device="cuda")
    rows = cache.table.shape[1] * cache.block_size
    w = torch.rand(3, rows, device="cuda")  # the last row is not the weights'
    view = w[:2]
    b.plan([(0, 399, 1)])
    b.attention_weights(0, ql, q, lse, 0.05, view)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attention_weights(0, ql, q, lse, 0.05, view)
    # of the same pool, with longer requests and more of them: their pages are those of the first table, again and again
    blocks = cache.table.shape[1]
    more = leyline.Tables(torch.cat([cache.table, cache.table[:1].expand(2, -1)]).repeat(1, 2).contiguous(),
                          torch.zeros(4, dtype=torch.int32, device="cuda"), np.array([400, 90, 300, 300], dtype=np.int64))
    more.table[:, blocks:] = cache.table[0, :1]
    more.table[:, :blocks][more.table[:, :blocks] < 0] = cache.table[0, 0]
    more.seq_lens_host[0] = rows + 50
    chunks = [(0, rows + 50 - tokens, tokens), (2, 300 - tokens, tokens), (1, 90 - tokens, tokens)]
    leyline.leyline_batch_plan(b.handle, more, leyline.chunk_batch(chunks), leyline.current_stream_ptr(0))
    want = w.clone()
    graph.replay()
    torch.cuda.synchronize()
    with pytest.raises(LeylineError) as e:
        cache.check_status()
    assert e.value.code == -8
    assert torch.equal(w[[0, 2]], want[[0, 2]]) and torch.equal(w[1, 90:], want[1, 90:])
    assert bool((w[1, :90] > want[1, :90]).any())
    b.close()
    cache.close()


def test_weigh_refusals():
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([100, 30], seed=8, layers=1)
    b = cache.batch(2, 4, 8)
    ql, q = queries(cache, 4, 8)
    lse = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(2, 160, device="cuda")
    with pytest.raises(LeylineError):  # no plan
        b.attention_weights(0, ql, q, lse, 0.1, w)
    b.plan([(0, 98, 2), (1, 28, 2)])
    good = w.clone()
    calls = [
        lambda: b.attention_weights(1, ql, q, lse, 0.1, w), lambda: b.attention_weights(-1, ql, q, lse, 0.1, w),
        lambda: b.attention_weights(0, ql, q, lse, float("nan"), w),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w, decay=-1.0),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w, decay=float("inf")),
        lambda: b.attention_weights(0, None, q, lse, 0.1, w), lambda: b.attention_weights(0, ql, q[:3], lse, 0.1, w),
        lambda: b.attention_weights(0, ql, q, lse[:3], 0.1, w), lambda: b.attention_weights(0, ql, q, lse.double(), 0.1, w),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w[:1]), lambda: b.attention_weights(0, ql, q, lse, 0.1, w[:, :99]),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w.double()), lambda: b.attention_weights(0, ql, q, lse, 0.1, w[0]),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w[:, ::2]), lambda: b.attention_weights(0, ql, q, lse, 0.1, w.cpu()),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w[:1].expand(2, 160)),
        lambda: b.attention_weights(0, ql, q, w.view(-1)[:32].view(4, 8), 0.1, w),
        lambda: b.attention_weights(0, ql, q.view(torch.float32).view(-1)[:1024].view(4, 256)[:, :32].view(torch.bfloat16)
                                    .view(4, 1, 64).expand(4, 8, 64), lse, 0.1, q.view(torch.float32).view(4, 256)),
        lambda: b.attention_weights(0, ql, q, lse, 0.1, w.clone().requires_grad_()),
        lambda: b.attention_weights(0, ql, q, lse.clone().requires_grad_(), 0.1, w),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((LeylineError, ValueError)):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert torch.equal(w, good)
    # a plan that an eviction has outdated
    kept = cache.select_rows(w, [(0, 50)])
    cache.evict([(0, 50)], kept)
    with pytest.raises(LeylineError):
        b.attention_weights(0, ql, q, lse, 0.1, w)
    b.plan([])
    b.attention_weights(0, ql, q, lse, 0.1, w)  # no tokens: nothing
    torch.cuda.synchronize()
    cache.check_status()
    assert torch.equal(w, good)
    b.close()
    cache.close()


def test_weigh_skips_bad_pages():
    from rope_rotation_gb300.leyline import LeylineError
    for kw in ({}, dict(B=1), dict(flags=LAZY), dict(latent=64, rope=16)):
        cache = BH.make_cache([200], seed=9, layers=1, **kw)
        b = cache.batch(1, 1, 4)
        b.plan([(0, 199, 1)])
        b.append(0, BH.bf16(1, cache.row))
        ql, q = queries(cache, 1, 4)
        lse = torch.zeros(1, 4, device="cuda")
        want = fresh_weights(cache, seed=4)
        w = want.clone()
        b.attention_weights(0, ql, q, lse, 0.02, want)
        cache.check_status()
        B = cache.block_size
        held = cache.table[0, 3].item()
        for page in (-1, cache.num_pages, 2 ** 31 - 1):
            cache.table[0, 3] = page
            got = w.clone()
            b.attention_weights(0, ql, q, lse, 0.02, got)
            with pytest.raises(LeylineError) as e:
                cache.check_status()
            assert e.value.code == -8
            assert torch.equal(got[0, 3 * B:4 * B], w[0, 3 * B:4 * B])
            assert torch.equal(got[0, :3 * B], want[0, :3 * B]) and torch.equal(got[0, 4 * B:], want[0, 4 * B:])
        cache.table[0, 3] = held
        b.close()
        cache.close()


# ------------------------------------------------------------------ select --
def greatest(w, length, n_keep, first, last):
    """What is kept, by a sort of Python numbers."""
    v = w[:length].double().cpu().tolist()
    middle = sorted(range(first, length - last), key=lambda t: (-v[t] if v[t] == v[t] else math.inf, t))
    middle = middle[:n_keep - first - last]
    # a NaN lies below minus infinity: keys of both are inf above, so order them again
    if any(v[t] != v[t] for t in range(length)):
        middle = sorted(range(first, length - last), key=lambda t: (v[t] != v[t], -v[t] if v[t] == v[t] else 0.0, t))
        middle = middle[:n_keep - first - last]
    return sorted([*range(first), *middle, *range(length - last, length)])


def select_pool(lens, B=16):
    """A cache whose tables hold nothing: a selection reads lengths and weights alone."""
    from rope_rotation_gb300.runtime import PagedCache
    cache = PagedCache(1, B, 4, max(len(lens), 1), max([1] + [-(-n // B) for n in lens]), 64, 16)
    cache.seq_lens_host[:len(lens)] = lens
    return cache


def check_select(cache, w, keeps, what=""):
    longest = max([k[1] for k in keeps] + [1])
    kept = torch.full((len(keeps) + 1, longest + 5), -7, dtype=torch.int32, device="cuda")
    out = cache.select_rows(w, keeps, out=kept)
    assert out is kept
    torch.cuda.synchronize()
    cache.check_status()
    got = kept.cpu().numpy()
    for k, (req, n, first, last) in enumerate(keeps):
        want = greatest(w[req], int(cache.seq_lens_host[req]), n, first, last)
        assert got[k, :n].tolist() == want, f"{what}: entry {k} of {keeps[k]}"
        assert (got[k, n:] == -7).all(), f"{what}: behind the list"
    assert (got[-1] == -7).all()


@pytest.mark.parametrize("length", [0, 1, 2, 31, 32, 33, 255, 1023, 1024, 1025, 4096, 10007, 70001, 140000])
def test_select_matches_a_sort(length):
    cache = select_pool([length, length // 2])
    g = torch.Generator(device="cuda").manual_seed(length)
    w = (3 * torch.randn(2, length + 3, generator=g, device="cuda")).exp()
    w[:, ::7] = 0.0
    sets = [(n, f, l) for n in sorted({0, 1, length // 3, length // 2, length - 1, length})
            for f, l in ((0, 0), (1, 0), (0, 2), (4, 64), (n // 2, n - n // 2)) if 0 <= n <= length and f + l <= n]
    for n, f, l in sets:
        check_select(cache, w, [(0, n, f, l)], f"{length}")
    check_select(cache, w, [(1, length // 4, 0, 0), (0, length // 2, 0, 0)], "two")
    cache.close()


@pytest.mark.parametrize("kind", ["equal", "two values", "tiny steps", "signs", "special", "ascending", "descending", "ints"])
def test_select_ties_and_special_values(kind):
    length = 9000
    cache = select_pool([length])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(length, generator=g, device="cuda")
    if kind == "equal":
        x.fill_(0.37)
    elif kind == "two values":
        x = (x > 0.5).float()
    elif kind == "tiny steps":  # keys that differ in their last bits alone
        x = (torch.full((length,), 0x3F800000, dtype=torch.int32, device="cuda")
             + torch.randint(0, 9, (length,), generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    elif kind == "special":
        pick = torch.randint(0, 8, (length,), generator=g, device="cuda")
        values = torch.tensor([NAN, -NAN, 0.0, -0.0, math.inf, -math.inf, 1e-45, -1e-45], device="cuda")
        x = values[pick]
    elif kind == "ascending":
        x = torch.arange(length, device="cuda").float()
    elif kind == "descending":
        x = -torch.arange(length, device="cuda").float()
    elif kind == "ints":
        x = torch.randint(-3, 4, (length,), generator=g, device="cuda").float()
    w = x[None].clone()
    for n, f, l in ((1, 0, 0), (17, 0, 0), (1000, 4, 64), (4500, 0, 0), (8200, 100, 33), (8999, 0, 0), (9000, 0, 0)):
        check_select(cache, w, [(0, n, f, l)], kind)
    cache.close()


def test_select_many_requests_and_strides():
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 3000, 70)]
    cache = select_pool(lens)
    w = torch.rand(80, 3333, device="cuda")[5:, 133:]  # rows of a wider tensor, not 16-byte aligned
    keeps = []
    for r in rng.permutation(70):
        n = int(rng.integers(0, lens[r] + 1))
        f = int(rng.integers(0, n + 1)) if rng.random() < 0.5 else 0
        keeps.append((int(r), n, f, int(rng.integers(0, n - f + 1)) if rng.random() < 0.5 else 0))
    check_select(cache, w, keeps, "many")
    from rope_rotation_gb300 import leyline
    a = leyline.keep_batch(keeps)
    out = cache.select_rows(w, a)  # makes its output
    assert out.shape == (70, max(k[1] for k in keeps)) and out.dtype == torch.int32
    for k, (req, n, f, l) in enumerate(keeps):
        assert out[k, :n].tolist() == greatest(w[req], lens[req], n, f, l) and bool((out[k, n:] == -1).all())
    assert cache.select_rows(w, []).shape == (0, 0)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = cache.select_rows(w, a, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    cache.close()


def test_select_refusals():
    from rope_rotation_gb300.leyline import LeylineError
    cache = select_pool([100, 50])
    w = torch.rand(2, 112, device="cuda")
    out = torch.full((2, 100), -7, dtype=torch.int32, device="cuda")
    bad = [[(2, 1)], [(-1, 1)], [(0, 101)], [(0, -1)], [(0, 10, 6, 5)], [(0, 10, -1, 0)], [(0, 10, 0, -1)], [(0, 10), (0, 5)],
           [(0, 10, 2 ** 31 - 1, 2 ** 31 - 1)]]
    for keeps in bad:
        with pytest.raises((LeylineError, ValueError)) as e:  # (the binding refuses a list longer than its row)
            cache.select_rows(w, keeps, out=out)
        assert getattr(e.value, "code", -1) == -1
    calls = [
        lambda: cache.select_rows(w, [(0, 1, 2)], out=out), lambda: cache.select_rows(w[:, :99], [(0, 10)], out=out),
        lambda: cache.select_rows(w[:1], [(1, 10)], out=out), lambda: cache.select_rows(w.half(), [(0, 10)], out=out),
        lambda: cache.select_rows(w, [(0, 10)], out=out.long()), lambda: cache.select_rows(w, [(0, 10)], out=out[:0]),
        lambda: cache.select_rows(w, [(0, 10)], out=out[:, :9]), lambda: cache.select_rows(w, [(0, 10)], out=out[:, ::2]),
        lambda: cache.select_rows(w, [(0, 10), (1, 10)], out=out[:1].expand(2, 100)),
        lambda: cache.select_rows(w, [(0, 10)], out=out.cpu()), lambda: cache.select_rows(w.cpu(), [(0, 10)], out=out),
        lambda: cache.select_rows(w, [(0, 10)], out=w.view(torch.int32)),
        lambda: cache.select_rows(w.clone().requires_grad_(), [(0, 10)], out=out),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((LeylineError, ValueError)):
            call()
            pytest.fail(f"call {i} was taken")
    x = torch.zeros(1, device="cuda")
    with pytest.raises(LeylineError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            x += 1
            cache.select_rows(w, [(0, 10)], out=out)
    torch.cuda.synchronize()
    assert bool((out == -7).all())
    cache.close()


# ------------------------------------------------------------------- evict --
def snapshot(cache):
    views = [v.clone() for v in cache.page_views()]
    pending = None if cache.pending() is None else cache.pending().clone()
    return views, cache.table.clone(), cache.seq_lens_host.copy(), pending, cache.free_pages()


def rows_of(cache, req, layer, n):
    rows, flat = BH.logical(cache, req, layer, n)
    return rows.view(torch.int16).clone(), flat


def free_ids(cache):
    """The free list in hand-out order (taken and given back in that order)."""
    from rope_rotation_gb300 import leyline
    ids = leyline.leyline_alloc_pages(cache.pool, cache.free_pages())
    leyline.leyline_free_pages(cache.pool, ids)
    return ids.tolist()


def check_evict(cache, keeps, lists, weights=None, what=""):
    """lists: ascending rows of each entry.  Everything that an eviction may and may not change."""
    B, layers = cache.block_size, cache.num_layers
    reqs = [k[0] for k in keeps]
    before = {r: ([rows_of(cache, r, l, int(cache.seq_lens_host[r]))[0] for l in range(layers)],
                  cache.slot_index(r, np.arange(int(cache.seq_lens_host[r])))) for r in reqs if cache.seq_lens_host[r]}
    free = free_ids(cache)
    views, table, lens, pending, n_free = snapshot(cache)
    w = None if weights is None else weights.clone()
    longest = max([len(x) for x in lists] + [1])
    kept = torch.full((len(keeps), longest + 3), -5, dtype=torch.int32)
    for k, rows in enumerate(lists):
        kept[k, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
    kept = kept.cuda()
    cache.evict(keeps, kept, weights=weights)
    torch.cuda.synchronize()
    cache.check_status()
    after = cache.table.cpu().numpy()
    old_table = table.cpu().numpy()
    returned, owned = [], set()
    want_lens = lens.copy()
    for k, rows in enumerate(lists):
        want_lens[reqs[k]] = len(rows)
    assert np.array_equal(cache.seq_lens_host, want_lens)
    assert np.array_equal(cache.seq_lens_dev.cpu().numpy(), want_lens), what
    for r in range(len(lens)):
        n_old, n_new = -(-int(lens[r]) // B), -(-int(want_lens[r]) // B)
        if r not in reqs:
            assert np.array_equal(after[r], old_table[r]), what
            continue
        owned |= set(old_table[r, :n_old].tolist())
        assert (after[r, n_new:] == -1).all(), what
        rows = lists[reqs.index(r)]
        assert after[r, :n_new].tolist() == (old_table[r, rows].tolist() if B == 1 else old_table[r, :n_new].tolist()), what
    for k, r in enumerate(reqs):  # pages go back in the order of the entries and of their blocks
        n_old, n_new = -(-int(lens[r]) // B), -(-int(want_lens[r]) // B)
        dropped = sorted(set(range(n_old)) - set(lists[k])) if B == 1 else range(n_new, n_old)
        returned += old_table[r, list(dropped)].tolist() if len(dropped) else []
    assert cache.free_pages() == n_free + len(returned)
    assert free_ids(cache) == free + returned, what
    for k, r in enumerate(reqs):
        if not lens[r]:
            continue
        old, slots = before[r]
        rows = torch.tensor(lists[k], dtype=torch.long, device="cuda")
        for l in range(layers):
            got, flat = rows_of(cache, r, l, len(lists[k]))
            assert torch.equal(got, old[l][rows]), f"{what}: rows of request {r} layer {l}"
        if pending is not None:
            want = pending.view(-1)[torch.from_numpy(slots).cuda()][rows]
            assert torch.equal(cache.pending().view(-1)[flat], want), f"{what}: pending turns of request {r}"
            gone = torch.from_numpy(np.setdiff1d(slots, flat.cpu().numpy())).cuda()
            assert int(cache.pending().view(-1)[gone].abs().sum()) == 0, f"{what}: turns left behind"
        if weights is not None:
            assert torch.equal(weights[r, :len(rows)].view(torch.int32), w[r][rows].view(torch.int32)), what
            if len(rows) < lens[r]:
                assert bool((weights[r, len(rows):int(lens[r])] == 0).all()), what
            assert torch.equal(weights[r, int(lens[r]):].view(torch.int32), w[r, int(lens[r]):].view(torch.int32)), what
    if weights is not None:
        others = [r for r in range(w.shape[0]) if r not in reqs]
        assert torch.equal(weights[others].view(torch.int32), w[others].view(torch.int32)), what
    # pages that no listed request held are as they were, and with one row a page all of them
    others = torch.tensor([p for p in range(cache.num_pages) if B == 1 or p not in owned], dtype=torch.long,
                          device="cuda")
    for now, was in zip(cache.page_views(), views):
        assert torch.equal(now[:, others].view(torch.int16), was[:, others].view(torch.int16)), f"{what}: other pages"
    if pending is not None and B > 1:
        assert torch.equal(cache.pending()[others], pending[others]), what


def pick(rng, length, n):
    return sorted(rng.choice(length, n, replace=False).tolist()) if n else []


EVICT_SHAPES = {
    "b16": dict(), "b5": dict(B=5), "b64": dict(B=64), "b1": dict(B=1), "lazy": dict(flags=LAZY),
    "lazy b1": dict(flags=LAZY, B=1), "lazy split b5": dict(flags=LAZY | SPLIT, B=5), "split": dict(flags=SPLIT),
    "reindex b1": dict(flags=REINDEX, B=1), "grouped": dict(rope=128, bands=4, B=8),
    "grouped lazy split": dict(rope=64, bands=2, flags=LAZY | SPLIT), "odd": dict(latent=64, rope=16, B=3),
    "odd wide": dict(latent=1000, rope=240, B=7),
}


@pytest.mark.parametrize("shape", EVICT_SHAPES)
def test_evict_moves_what_is_kept(shape):
    rng = np.random.default_rng(5)
    lens = [0, 1, 2, 16, 17, 333, 1500, 64, 700]
    cache = BH.make_cache(lens, seed=11, layers=3, **EVICT_SHAPES[shape])
    if cache.pending() is not None:
        cache.pending()[:, :] = torch.randint(-50, 50, cache.pending().shape, device="cuda", dtype=torch.int32)
        from rope_rotation_gb300 import leyline  # free pages carry no turns
        ids = leyline.leyline_alloc_pages(cache.pool, cache.free_pages())
        leyline.leyline_free_pages(cache.pool, ids)
    w = fresh_weights(cache, seed=2)
    w[:, ::5] = -0.0
    w[3, 2] = NAN
    for what, choose in (
            ("random", lambda n: pick(rng, n, int(rng.integers(0, n + 1)))),
            ("half", lambda n: pick(rng, n, n // 2)),
            ("one gone", lambda n: [t for t in range(n) if t != n // 3]),
            ("prefix", lambda n: list(range(n - n // 4))),
            ("suffix", lambda n: list(range(n // 4, n))),
            ("all", lambda n: list(range(n))),
            ("none of some", lambda n: [] if n % 2 else list(range(0, n, 2))),
            ("none", lambda n: [])):
        reqs = [int(r) for r in rng.permutation(len(lens)) if what == "none" or rng.random() < 0.7]
        lists = [choose(int(cache.seq_lens_host[r])) for r in reqs]
        check_evict(cache, [(r, len(x)) for r, x in zip(reqs, lists)], lists, w if what != "half" else None, f"{shape} {what}")
    cache.close()


def test_evict_many_requests_in_a_full_pool():
    """More requests than a launch takes; no page is free, and none is needed."""
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 120, 75)]
    cache = BH.make_cache(lens, seed=12, layers=2, B=8, latent=64, rope=16, slack=0)
    assert cache.free_pages() == 0
    w = fresh_weights(cache, seed=3)
    reqs = [int(r) for r in rng.permutation(75)]
    lists = [pick(rng, lens[r], int(rng.integers(0, lens[r] + 1))) for r in reqs]
    check_evict(cache, [(r, len(x)) for r, x in zip(reqs, lists)], lists, w, "many")
    cache.close()


def test_evict_long_request():
    rng = np.random.default_rng(7)
    for B, flags in ((16, 0), (16, LAZY), (1, 0)):
        cache = BH.make_cache([40000, 100], seed=13, layers=2, B=B, flags=flags)
        w = fresh_weights(cache, seed=3)
        lists = [pick(rng, 40000, 31000)]
        check_evict(cache, [(0, 31000)], lists, w, f"long {B}")
        cache.close()


def test_evict_refusals_and_bad_lists():
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    for B in (16, 1):
        cache = BH.make_cache([100, 50], seed=14, layers=2, B=B, latent=64, rope=16)
        w = fresh_weights(cache, seed=4)
        kept = torch.arange(100, dtype=torch.int32, device="cuda").repeat(2, 1)
        state = snapshot(cache)
        for keeps in ([(2, 1)], [(-1, 1)], [(0, 101)], [(0, -1)], [(0, 10), (0, 5)]):
            with pytest.raises(LeylineError) as e:
                cache.evict(keeps, torch.zeros(2, 200, dtype=torch.int32, device="cuda"))
            assert e.value.code == -1
        calls = [
            lambda: cache.evict([(0, 10)], kept.long()), lambda: cache.evict([(0, 10)], kept[:, :9]),
            lambda: cache.evict([(0, 10), (1, 5)], kept[:1]), lambda: cache.evict([(0, 10)], kept[:, ::2]),
            lambda: cache.evict([(0, 10)], kept.cpu()), lambda: cache.evict([(0, 10)], kept, weights=w[:, :99]),
            lambda: cache.evict([(1, 10)], kept, weights=w[:1]), lambda: cache.evict([(0, 10)], kept, weights=w.cpu()),
            lambda: cache.evict([(0, 10)], w.view(torch.int32), weights=w),
        ]
        for i, call in enumerate(calls):
            with pytest.raises((LeylineError, ValueError)):
                call()
                pytest.fail(f"call {i} was taken")
        x = torch.zeros(1, device="cuda")
        with pytest.raises(LeylineError):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                x += 1
                cache.evict([(0, 10)], kept)
        cache.evict([], kept[:0])
        torch.cuda.synchronize()
        now = snapshot(cache)
        for a, b in zip(state[0], now[0]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(state[1], now[1]) and np.array_equal(state[2], now[2]) and state[4] == now[4]
        # lists that do not ascend within the request: its first rows are kept, and the status says so
        for bad in ([3, 2, 5], [0, 0, 1], [-1, 0, 1], [5, 6, 100], [2 ** 31 - 1, 0, 1], [0, 1, -2 ** 31]):
            cache2 = BH.make_cache([100, 50], seed=14, layers=2, B=B, latent=64, rope=16)
            rows = [rows_of(cache2, 0, l, 3)[0] for l in range(2)]
            w2 = fresh_weights(cache2, seed=4)
            want = w2[0, :3].clone()
            lists = torch.tensor([bad], dtype=torch.int32, device="cuda")
            cache2.evict([(0, 3)], lists, weights=w2)
            with pytest.raises(LeylineError) as e:
                cache2.check_status()
            assert e.value.code == -8
            for l in range(2):
                assert torch.equal(rows_of(cache2, 0, l, 3)[0], rows[l])
            assert torch.equal(w2[0, :3], want) and int(cache2.seq_lens_dev[0]) == 3
            ids = free_ids(cache2)
            held = cache2.table.cpu().numpy()
            held = held[held >= 0].tolist()
            assert sorted(ids + held) == list(range(cache2.num_pages))
            cache2.close()
        # requests with more pages than the pool can take back
        full = BH.make_cache([64], seed=1, layers=1, B=B, latent=64, rope=16, slack=0)
        ids = leyline.leyline_alloc_pages(full.pool, full.free_pages())
        leyline.leyline_free_pages(full.pool, np.arange(full.num_pages, dtype=np.int32)[:full.num_pages])
        with pytest.raises(LeylineError):
            full.evict([(0, 1)], kept)
        assert len(ids) == 0
        full.close()
        cache.close()


@pytest.mark.parametrize("kw", [dict(), dict(flags=LAZY), dict(B=1), dict(B=1, flags=LAZY | REINDEX), dict(flags=SPLIT, B=5)])
def test_evict_among_other_work(kw):
    """Splices that overlap, evictions, steps of a batch and selections in flight at once, on two streams: the same state as
    of a pool that waits after every call."""
    from rope_rotation_gb300 import leyline
    rng = np.random.default_rng(10)
    lens = [900, 700, 800, 600, 500, 40]
    repl = BH.bf16(2, 7, 576, seed=31)
    x, ql, q = BH.bf16(9, 576, seed=32), BH.bf16(9, 4, 512, seed=33), BH.bf16(9, 4, 64, seed=34)
    wide = torch.zeros(6, 1000, dtype=torch.int32, device="cuda")
    plans = []
    for turn in range(3):
        span, n = ((300, 200), (180, 150), (140, 100))[turn]
        rows = {r: pick(rng, span, n) for r in (turn, 3, 4)}
        for k, r in enumerate(rows):
            wide[3 * (turn % 2) + k, 10:10 + len(rows[r])] = torch.tensor(rows[r], dtype=torch.int32)
        plans.append(([(r, len(v)) for r, v in rows.items()], wide.clone()[3 * (turn % 2):3 * (turn % 2) + 3, 10:500]))
    ends = []
    for wait in (True, False):
        cache = BH.make_cache(lens, extra=100, seed=30, slack=8000, **kw)
        w = fresh_weights(cache, seed=35)
        b = cache.batch(3, 9, 4)
        out = []
        torch.cuda.synchronize()
        first, second = torch.cuda.Stream(), torch.cuda.Stream()

        def done():
            if wait:
                torch.cuda.synchronize()

        for turn, (keeps, kept) in enumerate(plans):
            with torch.cuda.stream(first):
                for r in range(3):
                    cache.splice([leyline.directive(r, 20 + turn, 60, repl)], first)
                    done()
            cache.evict(keeps, kept, weights=w, stream=second)
            done()
            first.wait_stream(second)  # (weights are the caller's to order)
            with torch.cuda.stream(first):
                n = [int(v) for v in cache.seq_lens_host]
                b.plan([(3, n[3], 4), (turn, n[turn] - 2, 3), (5, n[5], 2)])
                done()
                for layer in range(2):
                    b.append(layer, x)
                    done()
                _, lse = b.attention(1, ql, q, 0.05)
                b.attention_weights(1, ql, q, lse, 0.05, w, 0.9)
                done()
                out.append(cache.select_rows(w, [(5, 30), (3, 100, 1, 2)]))
            second.wait_stream(first)
        torch.cuda.synchronize()
        cache.check_status()
        out += [cache.gather(r, layer, 0, int(cache.seq_lens_host[r])).view(torch.int16) for r in range(6) for layer in range(2)]
        out += [w.view(torch.int32), cache.table.clone(), torch.tensor(free_ids(cache)), torch.from_numpy(cache.seq_lens_host.copy())]
        ends.append([t.clone() for t in out])
        torch.cuda.synchronize()
        b.close()
        cache.close()
    for one, other in zip(*ends):
        assert torch.equal(one, other)


@pytest.mark.parametrize("B", [16, 1])
def test_evict_after_bad_lists(B):
    """What is found of a call's lists says nothing of the next ones', of fewer requests or of more."""
    from rope_rotation_gb300.leyline import LeylineError
    rng = np.random.default_rng(9)
    lens = [60] * 40
    cache = BH.make_cache(lens, seed=16, layers=1, B=B, latent=64, rope=16)
    lists = torch.zeros(40, 50, dtype=torch.int32, device="cuda")  # none of them ascends
    cache.evict([(r, 50) for r in range(40)], lists)
    with pytest.raises(LeylineError):
        cache.check_status()
    for reqs, n in (([3], 45), (range(40), 40), ([7, 8], 30), (range(20), 25), ([5], 20), (range(40), 15)):
        reqs = [int(r) for r in reqs if cache.seq_lens_host[r] >= n]
        check_evict(cache, [(r, n) for r in reqs], [pick(rng, int(cache.seq_lens_host[r]), n) for r in reqs], what=f"{B} {n}")
    cache.close()


def test_evict_and_the_page_accounting():
    """Checkpoint and rollback around an eviction, and plans that it outdates."""
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    rng = np.random.default_rng(8)
    for B, flags in ((16, 0), (1, 0), (1, LAZY), (16, LAZY)):
        cache = BH.make_cache([300, 80], seed=15, layers=2, B=B, flags=flags, latent=64, rope=16)
        if cache.pending() is not None:
            slots = torch.from_numpy(cache.slot_index(0, np.arange(300))).cuda()
            cache.pending().view(-1)[slots] = torch.arange(300, dtype=torch.int32, device="cuda") - 100
        other = cache.batch(1, 1, 1)
        other.plan([(1, 79, 1)])
        leyline.leyline_pool_checkpoint(cache.pool)
        state = snapshot(cache)
        rows = [rows_of(cache, 0, l, 300)[0] for l in range(2)]
        kept = torch.tensor([pick(rng, 300, 100)], dtype=torch.int32, device="cuda")
        cache.evict([(0, 100)], kept)
        other.append(0, BH.bf16(1, 80))  # a plan of another request still holds
        torch.cuda.synchronize()
        cache.check_status()
        if B == 1:  # rows stayed where they were: all of it comes back
            leyline.leyline_pool_rollback(cache.pool)
        else:
            with pytest.raises(LeylineError):
                leyline.leyline_pool_rollback(cache.pool)
            leyline.leyline_pool_rollback(cache.pool, leyline.LEYLINE_ROLLBACK_ACCEPT_TURNED)
        cache.table.copy_(state[1])
        cache.seq_lens_host[:] = state[2]
        cache.seq_lens_dev.copy_(torch.from_numpy(state[2]).to(torch.int32))
        torch.cuda.synchronize()
        assert cache.free_pages() == state[4]
        if state[3] is not None:
            assert torch.equal(cache.pending(), state[3])
        if B == 1:
            for l in range(2):
                assert torch.equal(rows_of(cache, 0, l, 300)[0], rows[l])
        other.close()
        cache.close()


def test_pending_view_keeps_its_cache():
    """The counts are the pool's memory: a tensor over them keeps the pool that its cache would free."""
    import gc
    import weakref
    cache = BH.make_cache([40], seed=1, layers=1, B=16, latent=64, rope=16, flags=LAZY)
    seen = weakref.ref(cache)
    counts = cache.pending().view(-1)[3:]
    del cache
    gc.collect()
    assert seen() is not None
    assert int(counts.abs().sum()) == 0
    del counts
    gc.collect()
    assert seen() is None


# ---------------------------------------------------------------- together --
@pytest.mark.parametrize("kw", [dict(), dict(B=1, flags=LAZY), dict(rope=128, bands=4, B=8), dict(flags=LAZY | SPLIT),
                                dict(B=1, flags=REINDEX)])
def test_a_run_within_a_budget(kw):
    """Requests decode, weigh, and are cut to their budget again and again, with a splice between: what attention sees in
    the end are the rows that the policy kept, at the positions they were encoded at."""
    from rope_rotation_gb300 import leyline
    layers, heads_per = 2, 4
    lens = [150, 40, 90]
    budget = 64
    cache = BH.make_cache(lens, extra=200, seed=16, layers=layers, **kw)
    heads = heads_per * cache.rope_heads
    b = cache.batch(3, 64, heads)
    room = cache.table.shape[1] * cache.block_size
    w = torch.zeros(3, room, device="cuda")
    # a model of each request: its rows as read (turned), by layer, and the next position
    rows = {r: [cache.gather(r, l, 0, n).clone() for l in range(layers)] for r, n in enumerate(lens)}
    pos = list(lens)
    scale = 0.06
    rng = np.random.default_rng(9)
    for step in range(6):
        new = [int(rng.integers(1, 20)) for _ in lens]
        chunks = [(r, int(cache.seq_lens_host[r]), n, pos[r]) for r, n in enumerate(new)]
        b.plan(chunks)
        n = sum(new)
        want = w.double().clone()
        for l in range(layers):
            x = BH.bf16(n, cache.row, seed=100 + 10 * step + l)
            b.append(l, x)
            ql, q = queries(cache, n, heads, seed=200 + 10 * step + l)
            q = b.rotate(q)
            out, lse = b.attention(l, ql, q, scale)
            b.attention_weights(l, ql, q, lse, scale, w, decay=0.9 if l == 0 else 1.0)
            t0 = 0
            for r, m in enumerate(new):
                band = x[t0:t0 + m, cache.latent_dim:].double().view(m, cache.rope_heads, -1)
                p = pos[r] + torch.arange(m, device="cuda")
                band = BH.turn64(band, p[:, None].expand(m, cache.rope_heads)).flatten(1).to(torch.bfloat16)
                rows[r][l] = torch.cat((rows[r][l], torch.cat((x[t0:t0 + m, :cache.latent_dim], band), 1)))
                t0 += m
            chk, tol, _ = weights64(cache, l, chunks, ql, q, lse, scale, torch.zeros_like(w), 0.0)
            want = want * (0.9 if l == 0 else 1.0) + chk
            assert bool(((w.double() - want).abs() <= tol * 2 + 2.0 ** -20 * want.abs() + 1e-30).all()), step
        pos = [p + m for p, m in zip(pos, new)]
        keeps = [(r, budget, 2, 8) for r in range(3) if cache.seq_lens_host[r] > budget]
        kept = cache.select_rows(w, keeps)
        lists = [greatest(w[k[0]], int(cache.seq_lens_host[k[0]]), *k[1:]) for k in keeps]
        for k, x in enumerate(lists):
            assert kept[k, :len(x)].tolist() == x
        before = w.clone()
        cache.evict(keeps, kept, weights=w)
        for k, x in enumerate(lists):
            r = keeps[k][0]
            idx = torch.tensor(x, device="cuda")
            rows[r] = [v[idx] for v in rows[r]]
            assert torch.equal(w[r, :len(x)], before[r][idx]) and int((w[r, len(x):] != 0).sum()) == 0
        if step == 2:  # a directive on the shortened request: its weights are the caller's to move
            repl = BH.bf16(layers, 5, cache.row, seed=77)
            cache.splice([leyline.directive(0, 10, 30, repl, mode=leyline.LEYLINE_EVICT)])
            rows[0] = [torch.cat((v[:10], repl[l], v[30:])) for l, v in enumerate(rows[0])]
            w[0] = torch.cat((w[0, :10], torch.zeros(5, device="cuda"), w[0, 30:], torch.zeros(15, device="cuda")))
        for r in range(3):
            assert int(cache.seq_lens_host[r]) == len(rows[r][0])
            for l in range(layers):
                got = cache.gather(r, l, 0, len(rows[r][l])).double()
                off = (got - rows[r][l].double()).abs()
                # latents bit for bit; bands within a rounding (appended ones are turned in fp32)
                assert torch.equal(got[:, :cache.latent_dim], rows[r][l][:, :cache.latent_dim].double())
                assert bool((off <= 2.0 ** -7 * rows[r][l].double().abs() + 2.0 ** -16).all())
    torch.cuda.synchronize()
    cache.check_status()
    b.close()
    cache.close()
