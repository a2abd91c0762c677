"""Batches of new tokens, cases that once went wrong: outputs whose weights are rounded, streams, captures, views that
overlap, plans that no longer hold (see batch_harness for formulas and tolerances)."""
import gc

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


@pytest.mark.parametrize("lat,rope,bands,heads,n,start,flags,B", [
    (512, 64, 1, 128, 40, 1000, 0, 16), (512, 64, 1, 128, 40, 1000, SPLIT, 5), (512, 64, 1, 128, 1, 9000, 0, 16),
    (512, 64, 1, 16, 1, 900, 0, 16), (512, 64, 1, 16, 3, 900, LAZY, 16), (512, 64, 1, 20, 30, 200, 0, 1),
    (512, 128, 4, 32, 4, 1500, 0, 16), (512, 128, 4, 32, 4, 1500, LAZY, 1), (384, 64, 2, 8, 5, 300, 0, 16),
    (512, 256, 2, 8, 5, 300, 0, 16), (40, 48, 1, 3, 5, 300, 0, 16)])
@pytest.mark.parametrize("scale", [0.125, 1.0])
def test_equal_values_come_back_as_they_are(lat, rope, bands, heads, n, start, flags, B, scale):
    """Where all rows hold one value, its weighted mean is that value, whatever the weights: whichever way the weights are
    rounded, their sum must be that of the rounded ones.  The sums' fp32 errors are under (end + 2) * 2^-23 < 2^-9.8 of the
    value (end <= 9001; equal signs in a dimension), a bf16 half step is at least 2^-9 of it, so the output has its bits."""
    cache = BH.make_cache([start], extra=n, layers=1, B=B, latent=lat, rope=rope, bands=bands, flags=flags)
    b = cache.batch(1, n, heads)
    chunks = [(0, start, n)]
    b.plan(chunks)
    rows = BH.bf16(start + n, cache.row, seed=1)
    rows[:, :lat] = BH.bf16(1, lat, seed=2)
    flat = torch.from_numpy(cache.slot_index(0, np.arange(start + n))).cuda()
    cache.write_layer_rows(0, flat, rows)
    ql = torch.zeros(n, heads, lat, dtype=torch.bfloat16, device="cuda") if bands == 1 else None
    q = BH.bf16(n, heads, rope, seed=3)
    out, lse = BH.check_attention(cache, b, 0, chunks, ql, q, scale, "equal values")
    want = rows[0, :lat].view(bands, lat // bands).repeat_interleave(heads // bands, 0).expand(n, heads, lat // bands)
    assert torch.equal(out, want), f"{int((out != want).sum())} of {out.numel()} values differ"
    cache.check_status()
    cache.close()


def _stream_of(t):
    """The stream that torch's allocator keeps a tensor's block for."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


class _ForeignStream:
    """Another library's stream: an object with the address."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("kind", ["torch", "address", "foreign"])
def test_outputs_belong_to_the_stream_of_their_call(kind):
    """Made for the current stream, they could be blocks that its kernels still read, or be handed out again while the
    call's stream writes them."""
    cache = BH.make_cache([100], extra=8, layers=1)
    b = cache.batch(1, 8, 16)
    b.plan([(0, 100, 3)])
    rows, ql, q = BH.bf16(3, 576), BH.bf16(3, 16, 512, seed=1), BH.bf16(3, 16, 64, seed=2)
    b.append(0, rows)
    want = (b.rotate(q), *b.attention(0, ql, q, 0.07), cache.gather(0, 0, 0, 103))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = {"torch": side, "address": side.cuda_stream, "foreign": _ForeignStream(side)}[kind]
    got = (b.rotate(q, stream=s), *b.attention(0, ql, q, 0.07, stream=s), cache.gather(0, 0, 0, 103, stream=s))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
        assert _stream_of(y) == side.cuda_stream and _stream_of(x) != side.cuda_stream
    cache.check_status()
    cache.close()


def _refused_under_capture(call, error):
    """The code of the error that `call` raises under capture.  A graph of an earlier capture that is collected during a
    capture ends it, so they go before."""
    gc.collect()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    x = torch.zeros(1, device="cuda")
    refused = None
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        x += 1
        try:
            call()
        except error as e:
            refused = getattr(e, "code", 0)
    assert refused is not None
    return refused


@pytest.mark.parametrize("given", [False, True])
def test_a_capture_asks_for_room_for_every_plan(given):
    """Captured calls go over the tokens of the plan that is current at a replay, up to max_tokens: tensors of the tokens of
    the plan at the capture would be read and written out of range.  (Nothing is replayed here.)"""
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([100], extra=16, layers=1)
    b = cache.batch(1, 8, 4)
    b.plan([(0, 100, 2)])

    def tensors(n):
        return (BH.bf16(n, 576), BH.bf16(n, 4, 512), BH.bf16(n, 4, 64), torch.empty(n, 4, 512, dtype=torch.bfloat16, device="cuda"),
                torch.empty(n, 4, device="cuda"))
    rows, ql, q, out, lse = tensors(2)
    big_rows, big_ql, big_q, big_out, big_lse = tensors(8)
    flat = torch.empty(8 * 4 * 512, dtype=torch.bfloat16, device="cuda")
    one = leyline.heads(flat.as_strided((2, 4, 512), (512, 2 * 512, 1)), "out", 2, 4, 512)  # heads outermost, 2 tokens each
    turned = leyline.heads(flat.as_strided((2, 4, 64), (64, 2 * 64, 1)), "out", 2, 4, 64)
    kw = lambda: {"stream": torch.cuda.current_stream()} if given else {}  # noqa: E731
    for call in (
            lambda: b.append(0, rows, **kw()), lambda: b.rotate(q, **kw()), lambda: b.rotate(big_q, out=q, **kw()),
            lambda: b.attention(0, ql, big_q, 0.07, out=big_out, lse=big_lse, **kw()),
            lambda: b.attention(0, big_ql, q, 0.07, out=big_out, lse=big_lse, **kw()),
            lambda: b.attention(0, big_ql, big_q, 0.07, out=out, lse=big_lse, **kw()),
            lambda: b.attention(0, big_ql, big_q, 0.07, out=big_out, lse=lse, **kw())):
        _refused_under_capture(call, ValueError)
    h = [leyline.heads(t, "q", 8, 4, d) for t, d in ((big_ql, 512), (big_q, 64))]
    assert _refused_under_capture(lambda: leyline.leyline_rotate(b.handle, h[1], turned), LeylineError) == -1
    assert _refused_under_capture(lambda: leyline.leyline_attention(b.handle, 0, *h, one, None, 0.07), LeylineError) == -1
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):  # with the room it asks for
        b.append(0, big_rows)
        b.attention(0, big_ql, b.rotate(big_q), 0.07, out=big_out, lse=big_lse)
    del graph
    b.append(0, rows)  # and outside a capture the plan's tokens do
    b.attention(0, ql, b.rotate(q), 0.07, out=out, lse=lse)
    cache.check_status()
    cache.close()


def test_views_that_overlap_the_queries_are_refused():
    """Outputs a head, a token or a part of a head off the queries, lse over them: other CTAs would read what one has
    written.  Parts of one wider tensor that share no byte are taken, and give what tensors of their own do."""
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([40], extra=16, layers=1)
    b = cache.batch(1, 8, 4)
    b.plan([(0, 40, 3)])
    b.append(0, BH.bf16(3, 576, seed=4))
    flat = BH.bf16(8 * 4 * 1100, seed=5)

    def at(first, dim, token=4 * 512, head=512, dtype=torch.bfloat16):
        return flat.as_strided((3, 4, dim), (token, head, 1), first)
    ql, q = BH.bf16(3, 4, 512), BH.bf16(3, 4, 64, seed=1)
    ql2 = at(0, 512)
    for call in (
            lambda: b.attention(0, ql2, q, 0.07, out=at(512, 512)), lambda: b.attention(0, ql2, q, 0.07, out=at(2048, 512)),
            lambda: b.attention(0, ql2, q, 0.07, out=at(2048 * 3 - 8, 512)),
            lambda: b.attention(0, ql, at(8, 64), 0.07, out=at(0, 512)),
            lambda: b.attention(0, ql2, q, 0.07, lse=flat[8:32].view(torch.float32).view(3, 4)),
            lambda: b.attention(0, ql, q, 0.07, out=at(0, 512), lse=flat[2048:2072].view(torch.float32).view(3, 4)),
            lambda: b.rotate(at(0, 64), out=at(8, 64)), lambda: b.rotate(at(0, 64), out=at(512, 64)),
            lambda: b.rotate(at(2048, 64), out=at(0, 64))):
        before = flat.clone()
        with pytest.raises(LeylineError) as e:
            call()
        assert e.value.code == -1
        assert torch.equal(before.view(torch.int16), flat.view(torch.int16))
    # a token's row as [head][latent 512 | band 64 | turned band 64 | output 512]
    wide = torch.zeros(3, 4, 1152, dtype=torch.bfloat16, device="cuda")
    wide[..., :512], wide[..., 512:576] = ql, q
    turned = b.rotate(wide[..., 512:576], out=wide[..., 576:640])
    out, lse = b.attention(0, wide[..., :512], turned, 0.07, out=wide[..., 640:])
    want = b.attention(0, ql, b.rotate(q), 0.07)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(wide[..., :512], ql) and torch.equal(wide[..., 512:576], q)
    b.rotate(at(0, 64), out=at(64, 64))
    cache.check_status()
    cache.close()


@pytest.mark.parametrize("noalloc", [False, True])
def test_plans_that_an_edit_has_outdated_are_refused(noalloc):
    """After a splice of one of its requests a plan's slots may be another request's, after a rollback free ones."""
    from rope_rotation_gb300 import leyline
    from rope_rotation_gb300.leyline import LeylineError
    cache = BH.make_cache([100, 80, 60], extra=64, layers=1, slack=50)
    b, other = cache.batch(3, 16, 4), cache.batch(1, 16, 4)
    rows, ql, q = BH.bf16(3, 576), BH.bf16(3, 4, 512), BH.bf16(3, 4, 64)

    def splice(req):
        dirs = [leyline.directive(req, 10, 30)]
        if noalloc:
            leyline.leyline_splice_noalloc(cache.pool, cache.tables, dirs)
        else:
            cache.splice(dirs)

    def calls(batch=b):
        batch.append(0, rows)
        batch.rotate(q)
        batch.attention(0, ql, q, 0.07)

    def refused():
        torch.cuda.synchronize()
        before = cache.kv.clone()
        for call in (lambda: b.append(0, rows), lambda: b.rotate(q), lambda: b.attention(0, ql, q, 0.07)):
            with pytest.raises(LeylineError) as e:
                call()
            assert e.value.code == -1
        assert torch.equal(before.view(torch.int16), cache.kv.view(torch.int16))
    b.plan([(0, 100, 2), (2, 60, 1), (1, 80, 0)])
    calls()
    splice(1)  # no new tokens of this one
    calls()
    splice(2)
    refused()
    other.plan([(1, 60, 3)])  # another batch's plan does not make this one's good
    calls(other)
    refused()
    b.plan([(2, 30, 3)])
    calls()
    table, lens = cache.table.clone(), cache.seq_lens_host.copy()
    leyline.leyline_pool_checkpoint(cache.pool)
    other.plan([(1, 63, 1)])
    calls(other)
    leyline.leyline_pool_rollback(cache.pool)
    cache.table.copy_(table)
    cache.seq_lens_dev.copy_(torch.from_numpy(lens).to(torch.int32))
    cache.seq_lens_host[:] = lens
    calls()  # made before the checkpoint
    with pytest.raises(LeylineError):
        other.append(0, rows)
    b.plan([(0, 100, 1), (2, 10, 2)])
    calls()
    with pytest.raises(LeylineError):  # rows were written again
        leyline.leyline_pool_rollback(cache.pool)
    leyline.leyline_pool_rollback(cache.pool, leyline.LEYLINE_ROLLBACK_ACCEPT_TURNED)
    refused()
    b.plan([])
    b.append(0, rows[:0])  # nothing to do
    cache.check_status()
    cache.close()
