"""Caches filled for the tests of batches of new tokens, and their operators in 64 bits.

The formulas ("Leyline: KV Cache Directives for Agentic Inference", section 2.2: the band of position
p is R(p) applied to the position-free band):
    norm       x * w / sqrt(mean(x^2) + eps)
    turn       x' = x cos - y sin, y' = x sin + y cos with angle p * theta^(-2j/d)
    attention  out = sum_s softmax(scale <q, k_s>) v_s over the rows s <= the token's own
Slots that no table entry names, and rows past a request's length, hold NaN.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from rope_rotation_gb300 import leyline
from rope_rotation_gb300.runtime import PagedCache

HALF = 2.0 ** -8  # half a bf16 step, relative to the value


def make_cache(lens, extra=0, layers=2, B=16, latent=512, rope=64, bands=1, flags=0, pair_layout=0, precision=0,
               theta=10000.0, slack=5, seed=0, spare_blocks=4):
    """A cache of the given lengths with N(0, 1) rows on pages in a random order; `extra` rows of room each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    room = sum(-(-(n + extra) // B) for n in lens)
    max_blocks = max(-(-(n + extra) // B) for n in lens) + spare_blocks if lens else 1
    cache = PagedCache(layers, B, room + slack, max(len(lens), 1), max_blocks, latent, rope, theta, pair_layout,
                       precision, flags, bands)
    # a shuffled free list: take every page and give them back in another order
    n = room + slack
    pages = leyline.leyline_alloc_pages(cache.pool, n)
    order = np.random.default_rng(seed).permutation(pages)
    leyline.leyline_free_pages(cache.pool, order)
    cache.kv.fill_(float("nan"))
    for r, length in enumerate(lens):
        cache.add_request(r, length)
        if not length:
            continue
        flat = torch.from_numpy(cache.slot_index(r, np.arange(length))).cuda()
        for layer in range(layers):
            rows = torch.randn(length, cache.row, generator=g, device="cuda").to(torch.bfloat16)
            cache.write_layer_rows(layer, flat, rows)
    torch.cuda.synchronize()
    return cache


def bf16(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def norm64(x, w, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def turn64(x, pos, theta=10000.0, pair_layout=0):
    """x [..., d] fp64 turned by pos [...] (broadcast over leading axes)."""
    d = x.shape[-1]
    j = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    a = pos.double()[..., None] * theta ** (-2.0 * j / d)
    c, s = a.cos(), a.sin()
    if pair_layout == 0:
        u, v = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((u * c - v * s, u * s + v * c), -1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)


def pair_norm(x, pair_layout=0):
    """Norm of each element's pair, same shape."""
    d = x.shape[-1]
    if pair_layout == 0:
        n = torch.hypot(x[..., :d // 2], x[..., d // 2:])
        return torch.cat((n, n), -1)
    n = torch.hypot(x[..., 0::2], x[..., 1::2])
    return torch.stack((n, n), -1).flatten(-2)


def check_turned(got, want, what, layout=0, normed=False):
    """A turned band, rounded once: half a bf16 step of the value, and of the pair's norm an fp32 error of
    the turn (two products, a sum, cos and sin rounded: under 4 * 2^-24, taken 2^-20) and of the norm
    (a sum of at most 1024 squares, halved by the root, and three products: under 2^-14)."""
    fp32 = 2.0 ** -20 + (2.0 ** -14 if normed else 0.0)
    tol = HALF * want.abs() + (1 + HALF) * fp32 * pair_norm(want, layout) + 2.0 ** -133
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()) and not bool(got.isnan().any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(((got.double() - want).abs() / tol).max())}"


def check_normed(got, want, what):
    tol = (HALF + (1 + HALF) * 2.0 ** -14) * want.abs() + 2.0 ** -133
    assert bool(((got.double() - want).abs() <= tol).all()), what


def logical(cache, req, layer, n):
    """Rows [0, n) as stored, through the table (no pending turn applied)."""
    flat = torch.from_numpy(cache.slot_index(req, np.arange(n))).cuda()
    page, slot = flat // cache.block_size, flat % cache.block_size
    return cache.read_rows(torch.full_like(page, layer), page, slot), flat


def attention64(cache, layer, chunks, q_latent, q_rope, scale, prefix=False, pair_layout=0, theta=10000.0):
    """(out, lse, tol_out, tol_lse) in fp64; the tolerances follow from the arithmetic:

    a score's error dx: an fp32 sum of d products is off by at most d * 2^-24 of the sum of their magnitudes
    (taken twice, for any order inside the matrix unit), a lazily turned key by an fp32 error of the turn (2^-20 of its
    pair) and by what two bf16 values leave of it (2^-17);
    the weights exp(x - m) by dx and 2^-21, and by half a bf16 step in the product with the values; their sum by
    2^-23 for each of n / 64 + 64 additions in a row.  So out is off by
    (HALF + 2 dx + ...) * sum p |v| / l and the final rounding, lse by dx and the sum's error."""
    outs, lses, tols, ltols, t0 = [], [], [], [], 0
    H = q_rope.shape[1]
    G = cache.rope_heads
    lat = cache.latent_dim
    for req, start, n in [c[:3] for c in chunks]:
        end = start if prefix else start + n
        dv = lat // G
        out = torch.zeros(n, H, dv, dtype=torch.float64, device="cuda")
        lse = torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        ltol = torch.zeros_like(lse)
        if n and end:
            rows, flat = logical(cache, req, layer, end)
            rows = rows.double()
            keys = rows[:, lat:].view(end, G, -1)
            turned = None
            if cache.pending() is not None:
                turned = cache.pending().view(-1)[flat]
                keys = turn64(keys, turned[:, None].expand(end, G), theta, pair_layout)
            seen = torch.arange(end, device="cuda") <= (start - 1 if prefix else start +
                                                         torch.arange(n, device="cuda")[:, None])
            seen = seen.expand(n, end)
            for h in range(H):
                k = keys[:, h * G // H]
                v = rows[:, :lat] if G == 1 else rows[:, :lat].view(end, G, dv)[:, h * G // H]
                q = q_rope[t0:t0 + n, h].double()
                x = q @ k.T
                mag = q.abs() @ k.abs().T
                lazy = q.abs() @ pair_norm(k, pair_layout).T * (2.0 ** -17 + 2.0 ** -20) if turned is not None else 0.0
                d = k.shape[1]
                if G == 1:
                    ql = q_latent[t0:t0 + n, h].double()
                    x = x + ql @ v.T
                    mag = mag + ql.abs() @ v.abs().T
                    d += lat
                x = torch.where(seen, x * scale, -math.inf)
                dx = torch.where(seen, abs(scale) * (mag * d * 2.0 ** -23 + lazy) + x.abs() * 2.0 ** -22, 0.0).amax(1)
                lse[:, h] = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[:, h:h + 1])
                out[:, h] = p @ v
                sums = (end / 64 + 64) * 2.0 ** -23 + 2.0 ** -21
                tol[:, h] = HALF * out[:, h].abs() + ((1 + HALF) * (HALF + 2 * dx + 2 * sums))[:, None] * (p @ v.abs())
                ltol[:, h] = dx + sums + 2.0 ** -22 * lse[:, h].abs()
        outs.append(out)
        lses.append(lse)
        tols.append(tol)
        ltols.append(ltol)
        t0 += n
    return tuple(torch.cat(x) for x in (outs, lses, tols, ltols))


def check_attention(cache, batch, layer, chunks, q_latent, q_rope, scale, what, prefix=False, pair_layout=0,
                    theta=10000.0):
    out, lse = batch.attention(layer, q_latent, q_rope, scale, prefix=prefix)
    want, wlse, tol, ltol = attention64(cache, layer, chunks, q_latent, q_rope, scale, prefix, pair_layout, theta)
    n = want.shape[0]
    got, glse = out[:n].double(), lse[:n].double()
    empty = wlse == -math.inf
    assert bool((glse[empty] == -math.inf).all()) and bool((got[empty] == 0).all()), f"{what}: rows without keys"
    off = (glse - wlse).abs()
    assert bool((off[~empty] <= ltol[~empty]).all()), \
        f"{what}: lse off by {float((off[~empty] / ltol[~empty]).max())} of its tolerance"
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                                 f"{float(((got - want).abs() / tol.clamp_min(1e-300)).nan_to_num(1e9).max())}")
    return out, lse
