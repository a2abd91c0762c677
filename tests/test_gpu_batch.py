"""Batches of new tokens on the GPU: rows appended through the block table, queries turned,
attention over the cache, against the formulas in 64 bits (see batch_harness)."""
import itertools

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


# -------------------------------------------------------------------- plan --
@pytest.mark.parametrize("B", [1, 5, 16])
@pytest.mark.parametrize("flags", [0, LAZY | SPLIT])
def test_plan_extends_requests(B, flags):
    """Lengths, table and free list after plans; old entries stay, new pages are distinct and were free."""
    lens = [0, 37, 16, 1]
    cache = BH.make_cache(lens, extra=400, B=B, flags=flags, latent=64, rope=16)
    b = cache.batch(8, 600, 1)
    lens = np.array(lens)
    for chunks in ([(0, 0, 1), (1, 37, 70), (3, 0, 3)], [(1, 100, 7), (2, 16, 33), (2, 49, 1), (0, 1, 0)],
                   [(0, 0, 300)], []):
        before = cache.table.cpu().numpy().copy()
        free = cache.free_pages()
        b.plan(chunks)
        new = lens.copy()
        for r, start, n in chunks:
            new[r] = max(new[r], start + n)
        torch.cuda.synchronize()
        cache.check_status()
        after = cache.table.cpu().numpy()
        assert np.array_equal(cache.seq_lens_host, new)
        assert np.array_equal(cache.seq_lens_dev.cpu().numpy(), new)
        old_blocks, new_blocks = -(-lens // B), -(-new // B)
        assert free - cache.free_pages() == int((new_blocks - old_blocks).sum())
        held = []
        for r in range(len(lens)):
            assert np.array_equal(after[r, :old_blocks[r]], before[r, :old_blocks[r]])
            assert (after[r, new_blocks[r]:] == -1).all()
            held += after[r, :new_blocks[r]].tolist()
        assert len(set(held)) == len(held) and min(held) >= 0 and max(held) < cache.num_pages
        lens = new
    b.close()
    cache.close()


def test_plan_refuses_and_changes_nothing():
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([40, 7], extra=0, B=8, latent=64, rope=16, slack=2, spare_blocks=8)
    b = cache.batch(3, 64, 4)
    with pytest.raises(LeylineError):  # no plan yet
        b.append(0, BH.bf16(1, 80))
    b.plan([(0, 39, 1)])
    table = cache.table.clone()
    for chunks, code in (
            ([(2, 0, 1)], -1), ([(-1, 0, 1)], -1), ([(0, -1, 1)], -1), ([(0, 41, 1)], -1), ([(0, 40, -1)], -1),
            ([(0, 40, 65)], -1), ([(0, 0, 1)] * 4, -1), ([(0, 10, 5), (0, 14, 2)], -1),
            ([(0, 10, 9), (0, 12, 0), (0, 15, 2)], -1), ([(0, 40, 1, -3)], -1), ([(1, 7, 60)], -4),
            ([(0, 40, 1), (0, 42, 1)], -1)):
        with pytest.raises(LeylineError) as e:
            b.plan(chunks)
        assert e.value.code == code, chunks
    big = cache.batch(1, 200, 4)
    with pytest.raises(LeylineError) as e:  # past the table's room
        big.plan([(0, 40, 200)])
    assert e.value.code == -7
    torch.cuda.synchronize()
    assert cache.free_pages() == 2 and cache.seq_lens_host.tolist() == [40, 7]
    assert torch.equal(table, cache.table)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(1, device="cuda")
    with pytest.raises(LeylineError) as e:
        with torch.cuda.graph(graph, stream=stream):
            x += 1
            b.plan([(0, 39, 1)])
    assert e.value.code == -1
    b.close()
    big.close()
    cache.close()


def test_refusals_of_the_calls():
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([40], extra=16, B=16)
    with pytest.raises(LeylineError):
        cache.batch(0, 1, 1)
    with pytest.raises(LeylineError):
        cache.batch(1, 0, 1)
    with pytest.raises(LeylineError):
        cache.batch(1, 1, 1025)
    b = cache.batch(2, 8, 4)
    with pytest.raises(LeylineError):  # a pool outlives its batches
        leyline.leyline_pool_destroy(cache.pool)
    b.plan([(0, 40, 3)])
    rows, q, ql = BH.bf16(3, 576), BH.bf16(3, 4, 64), BH.bf16(3, 4, 512)
    out = torch.empty(3, 4, 512, dtype=torch.bfloat16, device="cuda")
    for call in (
            lambda: b.append(2, rows), lambda: b.append(-1, rows), lambda: b.append(0, rows, eps=-1.0),
            lambda: b.append(0, rows, eps=float("nan")),
            lambda: b.append(0, BH.bf16(3, 580)[:, 2:578]),  # rows not 16-byte aligned
            lambda: b.attention(2, ql, q, 1.0), lambda: b.attention(0, ql, q, float("inf")),
            lambda: leyline.leyline_attention(b.handle, 0, None, leyline.heads(q, "q", 3, 4, 64),
                                              leyline.heads(out, "o", 3, 4, 512), None, 1.0),
            lambda: leyline.leyline_attention(b.handle, 0, leyline.heads(ql, "q", 3, 4, 512),
                                              leyline.heads(q, "q", 3, 4, 64), leyline.heads(out, "o", 3, 4, 512),
                                              None, 1.0, flags=2),
            lambda: b.rotate(q, out=q.as_strided((3, 4, 64), (64, 64, 1))),  # heads and tokens overlap
            lambda: b.rotate(q, out=q, eps=-0.5)):
        with pytest.raises(LeylineError) as e:
            call()
        assert e.value.code == -1
    for call in (
            lambda: b.append(0, rows.float()), lambda: b.append(0, rows[:2]), lambda: b.append(0, rows[:, :512]),
            lambda: b.append(0, rows, latent_norm=BH.bf16(64)), lambda: b.append(0, rows.cpu(), key_norm=BH.bf16(8)),
            lambda: b.attention(0, None, q, 1.0), lambda: b.attention(0, ql, q.float(), 1.0),
            lambda: b.attention(0, ql[:, :3], q, 1.0), lambda: b.attention(0, ql, q, 1.0, lse=torch.empty(3, 4)),
            lambda: b.attention(0, ql, q, 1.0, lse=torch.empty(3, 4, dtype=torch.float64, device="cuda")),
            lambda: b.rotate(q.cpu())):
        with pytest.raises((ValueError, LeylineError)):
            call()
    with pytest.raises(LeylineError):  # pageable host rows
        b.append(0, rows.cpu())
    grouped = BH.make_cache([4], B=16, latent=256, rope=64, bands=4)
    uneven = grouped.batch(1, 1, 6)  # heads that do not go over the bands: for append and rotate alone
    uneven.plan([(0, 3, 1)])
    uneven.append(0, BH.bf16(1, 512))
    uneven.rotate(BH.bf16(1, 6, 64))
    with pytest.raises(LeylineError):
        uneven.attention(0, None, BH.bf16(1, 6, 64), 1.0)
    gb = grouped.batch(1, 4, 8)
    gb.plan([(0, 0, 4)])
    with pytest.raises(LeylineError):
        gb.append(0, BH.bf16(4, 512), latent_norm=BH.bf16(256))
    with pytest.raises(ValueError):
        gb.attention(0, BH.bf16(4, 8, 64), BH.bf16(4, 8, 64), 1.0)
    for c in (cache, grouped):
        c.check_status()
        c.close()


# ------------------------------------------------------------------ append --
SHAPES = {  # latent, rope, bands
    "mla": (512, 64, 1),
    "grouped": (512, 128, 4),
    "grouped-64": (256, 64, 4),
    "grouped-256": (512, 256, 2),
    "grouped-192": (384, 64, 2),  # values of 192
    "odd": (40, 48, 1),
    "odd-grouped": (72, 16, 3),
    "wide": (1024, 256, 2),
}


@pytest.mark.parametrize("shape,B,flags,pairs,norms", [
    ("mla", 16, 0, 0, True), ("mla", 16, 0, 0, False), ("mla", 1, LAZY, 1, True), ("mla", 5, SPLIT, 0, True),
    ("grouped", 16, 0, 0, True), ("grouped", 1, LAZY | SPLIT, 1, True), ("odd", 7, 0, 0, True),
    ("odd", 16, SPLIT, 1, False), ("odd-grouped", 3, LAZY, 0, True), ("wide", 16, 0, 0, True)])
def test_append(shape, B, flags, pairs, norms):
    lat, rope, bands = SHAPES[shape]
    lens = [50, 0, 333]
    cache = BH.make_cache(lens, extra=700, B=B, latent=lat, rope=rope, bands=bands, flags=flags, pair_layout=pairs)
    if flags & LAZY:  # rows written again lose their pending turn, the others keep it
        cache.pending().fill_(0)
        for r, n in enumerate(lens):
            flat = torch.from_numpy(cache.slot_index(r, np.arange(n))).cuda()
            cache.pending().view(-1)[flat] = 7
    b = cache.batch(4, 1000, bands)
    # a chunk over old and new rows with a rotary position of its own, a first row, a long one, none
    chunks = [(0, 45, 9, 100045), (1, 0, 1), (2, 333, 600), (2, 0, 0)]
    b.plan(chunks)
    T = b.tokens
    wide = BH.bf16(T, cache.row + 24, seed=3)
    rows = wide[:, 8:8 + cache.row]  # a slice of wider rows
    lw = (1 + BH.bf16(lat, seed=4, scale=0.1).float()).to(torch.bfloat16) if norms and bands == 1 else None
    kw = (1 + BH.bf16(rope, seed=5, scale=0.1).float()).to(torch.bfloat16) if norms else None
    before = [v.clone() for v in cache.page_views()]
    layer = 1
    b.append(layer, rows, latent_norm=lw, key_norm=kw, eps=1e-5)
    torch.cuda.synchronize()
    cache.check_status()
    x = rows.double()
    t0, written = 0, []
    for c in chunks:
        r, start, n = c[:3]
        if n == 0:
            continue
        rope0 = c[3] if len(c) == 4 else start
        got, flat = BH.logical(cache, r, layer, start + n)
        got, flat = got[start:], flat[start:]
        written.append(flat)
        wl = x[t0:t0 + n, :lat]
        if lw is None:
            assert torch.equal(got[:, :lat], rows[t0:t0 + n, :lat])
        else:
            BH.check_normed(got[:, :lat], BH.norm64(wl, lw, 1e-5), "latent")
        wb = x[t0:t0 + n, lat:].reshape(n, bands, rope)
        if kw is not None:
            wb = BH.norm64(wb, kw, 1e-5)
        pos = torch.arange(rope0, rope0 + n, device="cuda")[:, None].expand(n, bands)
        BH.check_turned(got[:, lat:].reshape(n, bands, rope), BH.turn64(wb, pos, pair_layout=pairs), "band", pairs,
                        kw is not None)
        t0 += n
    # every other slot, and the other layer, as they were
    keep = torch.ones(cache.num_pages * B, dtype=torch.bool, device="cuda")
    keep[torch.cat(written)] = False
    for old, new in zip(before, cache.page_views()):
        old = old.view(torch.int16).view(cache.num_layers, cache.num_pages * B, -1)
        new = new.view(torch.int16).view(cache.num_layers, cache.num_pages * B, -1)
        assert torch.equal(old[0], new[0])
        assert torch.equal(old[1][keep], new[1][keep])
    if flags & LAZY:
        pend = cache.pending().view(-1)
        assert int(pend[torch.cat(written)].abs().sum()) == 0
        flat = torch.from_numpy(cache.slot_index(2, np.arange(333))).cuda()
        assert bool((pend[flat] == 7).all())
    cache.close()


def test_append_rows_in_pinned_host_memory():
    cache = BH.make_cache([0], extra=40, B=16)
    b = cache.batch(1, 40, 1)
    b.plan([(0, 0, 33)])
    rows = BH.bf16(33, 576, seed=1)
    from rope_rotation_gb300 import leyline
    leyline.leyline_append(b.handle, 0, rows.cpu().pin_memory())
    b.append(1, rows)
    torch.cuda.synchronize()
    a0, a1 = BH.logical(cache, 0, 0, 33)[0], BH.logical(cache, 0, 1, 33)[0]
    assert torch.equal(a0.view(torch.int16), a1.view(torch.int16))
    cache.close()


def test_naive_rounding_pool():
    """LEYLINE_ROTATE_BF16_NAIVE: cos, sin and the products rounded to bf16, as a splice's turn."""
    cache = BH.make_cache([0], extra=64, B=16, precision=1)
    b = cache.batch(1, 64, 2)
    b.plan([(0, 0, 50)])
    rows = BH.bf16(50, 576, seed=1)
    q = rows[:, None, 512:].expand(50, 2, 64)
    b.append(0, rows)
    out = b.rotate(q, out=torch.empty(50, 2, 64, dtype=torch.bfloat16, device="cuda"))

    def r(v):
        return v.to(torch.bfloat16).double()
    j = torch.arange(32, dtype=torch.float64, device="cuda")
    a = torch.arange(50, device="cuda").double()[:, None] * 10000.0 ** (-j / 32)
    c, s = a.cos().to(torch.bfloat16).double(), a.sin().to(torch.bfloat16).double()
    x, y = rows[:, 512:544].double(), rows[:, 544:].double()
    want = torch.cat((r(x * c) - r(y * s), r(x * s) + r(y * c)), -1).to(torch.bfloat16)
    got = BH.logical(cache, 0, 0, 50)[0][:, 512:]
    assert torch.equal(got, want)
    assert torch.equal(out[:, 0], want) and torch.equal(out[:, 1], want)
    cache.close()


# ------------------------------------------------------------------ rotate --
@pytest.mark.parametrize("rope,heads,pairs,norm", [(64, 16, 0, False), (64, 5, 1, True), (128, 32, 0, True),
                                                   (48, 3, 0, True), (16, 128, 1, False), (256, 1, 0, True)])
@pytest.mark.parametrize("layout", ["plain", "head-major", "in place", "slice"])
def test_rotate(rope, heads, pairs, norm, layout):
    cache = BH.make_cache([10, 900], extra=300, B=16, latent=64, rope=rope, pair_layout=pairs)
    b = cache.batch(2, 300, heads)
    b.plan([(0, 10, 1, 131071), (1, 850, 211)])
    T = b.tokens
    q = BH.bf16(T, heads, rope, seed=2)
    if layout == "head-major":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "slice":
        q = BH.bf16(T, heads, rope + 40, seed=2)[..., 8:8 + rope]
    w = (1 + BH.bf16(rope, seed=6, scale=0.1).float()).to(torch.bfloat16) if norm else None
    x = q.double()
    if norm:
        x = BH.norm64(x, w, 1e-6)
    pos = torch.cat((torch.tensor([131071]), torch.arange(850, 850 + 211))).cuda()[:, None].expand(T, heads)
    out = b.rotate(q, out=q if layout == "in place" else None, norm=w)
    BH.check_turned(out, BH.turn64(x, pos, pair_layout=pairs), "query", pairs, norm)
    cache.close()


# --------------------------------------------------------------- attention --
def _attend(lens, chunks, heads, shape="mla", B=16, flags=0, pairs=0, prefix=False, scale=None, layer=1, seed=0,
            strided=False, pend=None):
    lat, rope, bands = SHAPES[shape]
    cache = BH.make_cache(lens, extra=max([c[2] for c in chunks] + [1]), B=B, latent=lat, rope=rope, bands=bands,
                          flags=flags, pair_layout=pairs, seed=seed)
    b = cache.batch(max(len(chunks), 1), max(sum(c[2] for c in chunks), 1), heads)
    b.plan(chunks)
    T = b.tokens
    rows = BH.bf16(T, cache.row, seed=seed + 1)
    for k in range(2):
        b.append(k, rows)
    if flags & LAZY:  # turns of the rows before the chunks, in runs
        g = np.random.default_rng(seed)
        for r in range(len(lens)):
            n = min([int(cache.seq_lens_host[r])] + [c[1] for c in chunks if c[0] == r])
            if n:
                flat = torch.from_numpy(cache.slot_index(r, np.arange(n))).cuda()
                turns = g.choice(pend or [0, -5988, 48, 3, -100000], size=n // 37 + 1)
                cache.pending().view(-1)[flat] = torch.from_numpy(turns[np.arange(n) // 37].astype(np.int32)).cuda()
    ql = BH.bf16(T, heads, lat, seed=seed + 2) if bands == 1 else None
    q = BH.bf16(T, heads, rope, seed=seed + 3)
    if strided:
        ql = BH.bf16(heads, T, lat + 8, seed=seed + 2).transpose(0, 1)[..., 8:] if bands == 1 else None
        q = BH.bf16(T, heads, rope + 128, seed=seed + 3)[..., 128:]
    if scale is None:
        scale = (192 if bands == 1 else rope) ** -0.5
    BH.check_attention(cache, b, layer, chunks, ql, q, scale, f"{shape} {chunks}", prefix, pairs)
    torch.cuda.synchronize()
    cache.check_status()
    cache.close()


@pytest.mark.parametrize("ctx", [1, 2, 15, 63, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("heads", [1, 16, 20, 64, 128])
def test_attention_decode(ctx, heads):
    _attend([ctx - 1], [(0, ctx - 1, 1)], heads, seed=ctx)


@pytest.mark.parametrize("B", [1, 3, 5, 8, 16, 24, 64, 100])
@pytest.mark.parametrize("flags", [0, LAZY, SPLIT, LAZY | SPLIT])
@pytest.mark.parametrize("shape", ["mla", "grouped"])
def test_attention_blocks_and_pools(B, flags, shape):
    _attend([700, 0, 129, 64], [(0, 700, 1), (1, 0, 70), (2, 100, 29), (3, 64, 3)], 16, shape, B=B, flags=flags, seed=B)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 17, 64, 100, 257])
@pytest.mark.parametrize("heads", [1, 5, 16, 40])
def test_attention_chunks(n, heads):
    """Chunks from one token on, at the start of a request, after its rows, and inside them."""
    _attend([0, 333, 400], [(0, 0, n), (1, 333, n), (2, 20, n)], heads, seed=n)


@pytest.mark.parametrize("shape", ["grouped", "grouped-64", "grouped-256", "grouped-192", "odd", "odd-grouped", "wide"])
@pytest.mark.parametrize("flags,pairs", [(0, 0), (LAZY, 0), (LAZY, 1), (SPLIT, 0)])
@pytest.mark.parametrize("per", [1, 4, 7])
def test_attention_row_shapes(shape, flags, pairs, per):
    heads = per * SHAPES[shape][2]
    _attend([130, 0, 1000], [(0, 130, 1), (1, 0, 33), (2, 1000, 5)], heads, shape, B=16, flags=flags, pairs=pairs)


@pytest.mark.parametrize("shape", ["mla", "grouped"])
def test_attention_prefix_and_rows_without_keys(shape):
    _attend([0, 64, 500], [(0, 0, 5), (1, 64, 9), (2, 63, 2), (2, 300, 100)], 16, shape, prefix=True)


@pytest.mark.parametrize("shape", ["mla", "grouped"])
def test_attention_strided_tensors(shape):
    _attend([100, 300], [(0, 100, 3), (1, 300, 40)], 8, shape, strided=True)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_attention_scales(scale):
    """Equal weights, the smallest score first, and nearly one-hot weights (scores near +-100)."""
    _attend([1000], [(0, 1000, 2)], 16, scale=scale)


def test_attention_interleaved_lazy():
    _attend([900], [(0, 900, 20)], 16, flags=LAZY, pairs=1, B=1)


@pytest.mark.parametrize("shape", ["mla", "grouped", "grouped-64", "grouped-256", "odd"])
def test_lazy_naive_pool_attends_to_the_gathered_rows(shape):
    """With the naive rounding a turned band is a bf16 value: attention over a lazy pool gives the same bits as over
    an eager pool that holds what leyline_gather returns."""
    lat, rope, bands = SHAPES[shape]
    lens = [1234, 77]
    kw = dict(extra=8, B=16, precision=1, latent=lat, rope=rope, bands=bands)
    lazy = BH.make_cache(lens, flags=LAZY, **kw)
    eager = BH.make_cache(lens, **kw)
    for r, n in enumerate(lens):
        flat = torch.from_numpy(lazy.slot_index(r, np.arange(n))).cuda()
        turns = torch.from_numpy(np.random.default_rng(r).integers(-9000, 9000, n // 10 + 1).astype(np.int32)).cuda()
        lazy.pending().view(-1)[flat] = turns[torch.arange(n, device="cuda") // 10]
        flat_e = torch.from_numpy(eager.slot_index(r, np.arange(n))).cuda()
        for layer in range(2):
            eager.write_layer_rows(layer, flat_e, lazy.gather(r, layer, 0, n))
    chunks = [(0, 1234, 3), (1, 77, 1)]
    ql, q = BH.bf16(4, 16, lat) if bands == 1 else None, BH.bf16(4, 16, rope, seed=1)
    rows = BH.bf16(4, lazy.row, seed=2)
    got = []
    for cache in (lazy, eager):
        b = cache.batch(2, 4, 16)
        b.plan(chunks)
        b.append(1, rows)
        got.append(b.attention(1, ql, q, 0.07))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    lazy.close()
    eager.close()


def test_attention_repeats_bit_for_bit_and_between_streams():
    lens = [5000, 3, 700]
    cache = BH.make_cache(lens, extra=8, B=16)
    b = cache.batch(3, 16, 16)
    chunks = [(0, 5000, 1), (1, 3, 5), (2, 700, 8)]
    b.plan(chunks)
    T = b.tokens
    rows, ql, q = BH.bf16(T, 576), BH.bf16(T, 16, 512, seed=1), BH.bf16(T, 16, 64, seed=2)
    for layer in range(2):
        b.append(layer, rows)
    first = [t.clone() for t in b.attention(1, ql, q, 0.07)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for k in range(10):  # calls of one batch share its workspace: the library orders them
        with torch.cuda.stream(streams[k % 2]):
            outs.append(b.attention(1, ql, q, 0.07))
            b.attention(0, ql, q, 0.5)
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    cache.close()


def test_bad_pages_are_reported_not_followed():
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([300], extra=4, B=16)
    b = cache.batch(1, 4, 16)
    b.plan([(0, 300, 1)])
    b.append(0, BH.bf16(1, 576))
    cache.check_status()
    cache.table[0, 3] = cache.num_pages
    cache.table[0, 7] = -5
    out, lse = b.attention(0, BH.bf16(1, 16, 512), BH.bf16(1, 16, 64), 0.07)
    torch.cuda.synchronize()
    with pytest.raises(LeylineError) as e:
        cache.check_status()
    assert e.value.code == -8
    assert bool(out.isfinite().all())
    cache.check_status()
    cache.table[0, 18] = -1  # the page of the row that the next plan writes
    b.plan([(0, 299, 1)])
    b.append(0, BH.bf16(1, 576))
    with pytest.raises(LeylineError):
        cache.check_status()
    cache.close()


# ------------------------------------------------------------ as it is used --
def _step(cache, b, layer, rows, q, ql, lw, scale):
    b.append(layer, rows[layer], latent_norm=lw)
    return b.attention(layer, ql[layer], b.rotate(q[layer]), scale)


@pytest.mark.parametrize("flags,B", [(0, 16), (REINDEX, 1), (LAZY | REINDEX, 1), (LAZY | SPLIT, 16)])
def test_splice_then_prefill_of_r_and_decode(flags, B):
    """A splice drops a span and opens room for R; the rows of R are then prefilled in place, layer by layer,
    together with a decoded token at the end; then the request decodes on."""
    from rope_rotation_gb300 import leyline
    cache = BH.make_cache([900, 250], extra=64, B=B, flags=flags, slack=1000)
    n_r, s, e = 13, 400, 650
    blank = torch.zeros(2, n_r, 576, dtype=torch.bfloat16, device="cuda")
    b = cache.batch(4, 64, 16)
    cache.splice([leyline.directive(0, s, e, blank)])
    n0 = 900 - (e - s) + n_r
    for step, chunks in enumerate([[(0, s, n_r), (0, n0, 1), (1, 250, 4)], [(0, n0 + 1, 1), (1, 254, 1)]]):
        b.plan(chunks)
        T = b.tokens
        rows = [BH.bf16(T, 576, seed=10 * step + k) for k in range(2)]
        ql = [BH.bf16(T, 16, 512, seed=20 + 10 * step + k) for k in range(2)]
        q = [BH.bf16(T, 16, 64, seed=30 + 10 * step + k) for k in range(2)]
        lw = BH.bf16(512, seed=9)
        for layer in range(2):
            out, lse = _step(cache, b, layer, rows, q, ql, lw, 0.07)
            pos = torch.cat([torch.arange(c[1], c[1] + c[2]) for c in chunks]).cuda()[:, None].expand(T, 16)
            want_q = BH.turn64(q[layer].double(), pos)
            turned = b.rotate(q[layer])
            BH.check_turned(turned, want_q, "query")
            want, wlse, tol, ltol = BH.attention64(cache, layer, chunks, ql[layer], turned, 0.07)
            assert bool(((out.double() - want).abs() <= tol).all())
            assert bool(((lse.double() - wlse).abs() <= ltol).all())
    torch.cuda.synchronize()
    cache.check_status()
    assert cache.seq_lens_host.tolist() == [n0 + 2, 255]
    # and the next splice finds the cache as any other
    cache.splice([leyline.directive(0, 5, 40), leyline.directive(1, 100, 200)])
    torch.cuda.synchronize()
    cache.check_status()
    assert cache.seq_lens_host.tolist() == [n0 + 2 - 35, 155]
    cache.close()


def test_captured_step_replays_with_new_plans():
    """One graph of a step's layers, replayed after each plan, against eager calls on a twin cache."""
    caches = [BH.make_cache([700, 64, 0], extra=200, B=16, seed=3) for _ in range(2)]
    room = 128
    batches = [c.batch(3, room, 16) for c in caches]
    rows = [torch.zeros(room, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ql = [torch.zeros(room, 16, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = [torch.zeros(room, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lw = BH.bf16(512, seed=9)
    outs = [(torch.zeros(room, 16, 512, dtype=torch.bfloat16, device="cuda"),
             torch.zeros(room, 16, device="cuda")) for _ in range(2)]
    turned = torch.zeros_like(q[0])
    plans = [[(0, 700, 1), (1, 64, 1)], [(0, 701, 100), (2, 0, 3)], [(1, 65, 1), (0, 801, 1), (2, 3, 1)], []]
    batches[0].plan([(0, 699, 1)])
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for layer in range(2):
            batches[0].append(layer, rows[layer], latent_norm=lw)
            batches[0].rotate(q[layer], out=turned)
            batches[0].attention(layer, ql[layer], turned, 0.07, out=outs[layer][0], lse=outs[layer][1])
    for k, plan in enumerate(plans):
        T = sum(c[2] for c in plan)
        for layer in range(2):
            rows[layer][:T] = BH.bf16(T, 576, seed=10 * k + layer)
            ql[layer][:T] = BH.bf16(T, 16, 512, seed=100 + 10 * k + layer)
            q[layer][:T] = BH.bf16(T, 16, 64, seed=200 + 10 * k + layer)
        for o in outs:
            o[0].fill_(7.0)
            o[1].fill_(7.0)
        batches[0].plan(plan)
        graph.replay()
        batches[1].plan(plan)
        for layer in range(2):
            batches[1].append(layer, rows[layer], latent_norm=lw)
            if T:
                out, lse = batches[1].attention(layer, ql[layer], batches[1].rotate(q[layer]), 0.07)
                assert torch.equal(outs[layer][0][:T], out[:T]) and torch.equal(outs[layer][1][:T], lse[:T])
            assert bool((outs[layer][0][T:] == 7.0).all()) and bool((outs[layer][1][T:] == 7.0).all())
        torch.cuda.synchronize()
        for r in range(3):
            n = int(caches[0].seq_lens_host[r])
            for layer in range(2):
                x, y = (BH.logical(c, r, layer, n)[0].view(torch.int16) for c in caches)
                assert torch.equal(x, y)
    for c in caches:
        c.check_status()
        c.close()


def test_plan_and_rollback():
    """A rollback gives back the pages a plan took; rows written again ask for the flag."""
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([100], extra=100, B=16)
    b = cache.batch(1, 64, 4)
    table, free = cache.table.clone(), cache.free_pages()
    leyline.leyline_pool_checkpoint(cache.pool)
    b.plan([(0, 100, 50)])
    assert cache.free_pages() == free - 3
    leyline.leyline_pool_rollback(cache.pool)
    cache.table.copy_(table)
    cache.seq_lens_dev[0] = 100
    cache.seq_lens_host[0] = 100
    assert cache.free_pages() == free
    b.plan([(0, 99, 2)])
    with pytest.raises(LeylineError):
        leyline.leyline_pool_rollback(cache.pool)
    leyline.leyline_pool_rollback(cache.pool, leyline.LEYLINE_ROLLBACK_ACCEPT_TURNED)
    assert cache.free_pages() == free
    cache.close()


def test_rows_and_slots_past_32_bits():
    """A pool whose rows start past 2^31 elements: 1.9 M slots of 576 in each of two layers."""
    pages = 120000
    cache = BH.PagedCache(2, 16, pages, 1, 300)
    cache.kv.zero_()
    ids = np.arange(pages - 300, pages, dtype=np.int32)[::-1].copy()  # the last pages of the pool
    cache.table[0].copy_(torch.from_numpy(ids))
    cache.seq_lens_dev[0] = 4000
    cache.seq_lens_host[0] = 4000
    flat = torch.from_numpy(cache.slot_index(0, np.arange(4000))).cuda()
    cache.write_layer_rows(1, flat, BH.bf16(4000, 576, seed=5))
    b = cache.batch(1, 8, 16)
    chunks = [(0, 3992, 8)]
    b.plan(chunks)
    b.append(1, BH.bf16(8, 576, seed=6))
    BH.check_attention(cache, b, 1, chunks, BH.bf16(8, 16, 512, seed=7), BH.bf16(8, 16, 64, seed=8), 0.07, "far rows")
    assert int((cache.kv_view()[0] != 0).sum()) == 0
    cache.close()


def test_many_random_batches():
    """Random lengths, chunks and pools, the plan's work split in many ways."""
    rng = np.random.default_rng(11)
    for k, (flags, B, shape) in enumerate(itertools.product((0, LAZY | SPLIT), (1, 16), ("mla", "grouped"))):
        lens = rng.integers(0, 1500, size=9).tolist()
        chunks = [(r, int(rng.integers(0, n + 1)) if rng.random() < 0.3 else n, int(rng.integers(0, 40)))
                  for r, n in enumerate(lens)]
        _attend(lens, chunks, int(rng.choice([4, 16, 32])), shape, B=B, flags=flags, seed=k)
