"""The operators of a decoding step over a paged cache, as cases to be timed and compared.

A serving step hands the cache one chunk of new tokens per request (one token when it decodes,
more when it reads a prompt, re-encodes a replacement or checks drafted tokens).  In every layer it

  append     norms the latent (or each key head), turns the keys by their positions and writes the
             rows through the block table;
  rotate     norms each query head and turns it by its position;
  attention  attends with the chunk's queries over all rows of their request up to their own.

Rows are as in the pool: [latent 512 | key band 64] for MLA (values are the latent), or
[values of 4 heads x 128 | keys of 4 heads x 128] for grouped heads.
"""
import math
import random

import torch

own = False

THETA = 10000.0
EPS = 1e-6
LAYERS = 2  # rows of one layer lie among those of others, as in a pool
LAYER = 1

#: Row layouts: latent (or values of all heads), key band, bands per row, softmax scale.
LAYOUTS = {
    "mla": {"latent": 512, "rope": 64, "bands": 1, "scale": 192 ** -0.5},
    "grouped": {"latent": 512, "rope": 128, "bands": 4, "scale": 128 ** -0.5},
}


def listed():
    return [
        # one new token of one request: the smallest call, latency alone
        _append("append: one token", reqs=1, tokens=1, ctx=4096),
        # a long prompt chunk of one request
        _append("append: prompt chunk", reqs=1, tokens=8192, ctx=32768),
        # ragged chunks of 16 requests, grouped key heads with a norm for each, one row a page
        _append("append: grouped, ragged", reqs=16, tokens=509, ctx=8000, layout="grouped", block=1, ragged=True),
        # the queries of one decoding step
        _rotate("rotate: decode", reqs=16, tokens=1, ctx=24000, heads=16),
        # the query bands of a prompt chunk with 128 heads
        _rotate("rotate: prompt chunk", reqs=1, tokens=4096, ctx=8192, heads=128),
        # normed query heads of a ragged batch
        _rotate("rotate: normed heads, ragged", reqs=7, tokens=301, ctx=5000, heads=32, layout="grouped", ragged=True),
        # one request decodes over a 32k context (27-layer, 16-head shape)
        _attention("attention: decode 1 x 32k", reqs=1, tokens=1, ctx=32768, heads=16),
        # 16 requests of the concurrency sweep decode (61-layer, 128-head shape)
        _attention("attention: decode sweep", reqs=16, tokens=1, ctx=24000, heads=128, ragged=True),
        # 64 short requests after splices in a lazy pool with one row a page
        _attention("attention: decode lazy", reqs=64, tokens=1, ctx=4001, heads=16, block=1, lazy=True, ragged=True),
        # a prompt chunk, 128 heads: the largest product
        _attention("attention: prompt chunk", reqs=1, tokens=512, ctx=8192, heads=128),
        # replacements and drafts of several requests at once, split-rope pool
        _attention("attention: ragged chunks", reqs=8, tokens=61, ctx=15000, heads=16, split=True, ragged=True),
        # grouped heads: four drafted tokens of each of 16 requests
        _attention("attention: grouped drafts", reqs=16, tokens=4, ctx=8000, heads=32, layout="grouped", ragged=True),
    ]


def _case(op, name, reqs, tokens, ctx, heads, layout, block, lazy, split, ragged, shape):
    c = {"name": name, "op": op, "reqs": reqs, "tokens": tokens, "ctx": ctx, "heads": heads, "layout": layout,
         "block": block, "lazy": lazy, "split": split, "ragged": ragged, "shape": shape}
    if name is None:
        del c["name"]
    return c


def _append(name, reqs, tokens, ctx, layout="mla", block=16, lazy=False, split=False, ragged=False, shape=1):
    return _case("append", name, reqs, tokens, ctx, 1, layout, block, lazy, split, ragged, shape)


def _rotate(name, reqs, tokens, ctx, heads, layout="mla", ragged=False, shape=2):
    return _case("rotate", name, reqs, tokens, ctx, heads, layout, 16, False, False, ragged, shape)


def _attention(name, reqs, tokens, ctx, heads, layout="mla", block=16, lazy=False, split=False, ragged=False, shape=3):
    return _case("attention", name, reqs, tokens, ctx, heads, layout, block, lazy, split, ragged, shape)


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    shape = rng.randrange(1 << 20)
    block = rng.choice([1, 5, 16, 16, 64])
    lazy, split, ragged = rng.random() < 0.3, rng.random() < 0.3, rng.random() < 0.7
    layout = "mla" if rng.random() < 0.7 else "grouped"
    op = rng.choice(["append", "rotate", "attention", "attention"])
    if op == "append":
        reqs = _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, 8192 // reqs)
        return _append(None, reqs, tokens, tokens + _log_int(rng, 1, 20000), layout, block, lazy, split, ragged, shape)
    if op == "rotate":
        heads = _log_int(rng, 1, 128 if layout == "mla" else 64)
        reqs = _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, max(1, 4096 // reqs))
        return _rotate(None, reqs, tokens, tokens + _log_int(rng, 1, 20000), heads, layout, ragged, shape)
    heads = rng.choice([4, 8, 12, 20, 32, 64]) if layout == "grouped" else rng.choice([1, 5, 16, 16, 20, 40, 64, 128])
    reqs = _log_int(rng, 1, 64)
    tokens = _log_int(rng, 1, 512)
    ctx = _log_int(rng, 1, 32768)
    # no dearer than the listed ones: fewer requests, then fewer tokens
    while (reqs * tokens * heads * (tokens + ctx) > 2 ** 28 or reqs * (tokens + ctx) > 2 ** 18
           or reqs * tokens * heads > 2 ** 16):
        if reqs > 1:
            reqs = (reqs + 1) // 2
        else:
            tokens = (tokens + 1) // 2
    return _attention(None, reqs, tokens, tokens + ctx, heads, layout, block, lazy, split, ragged, shape)


def _lengths(c):
    """(total length, chunk length) of each request; they follow from the case alone."""
    r = random.Random(c["shape"])
    out = []
    for _ in range(c["reqs"]):
        n, total = c["tokens"], c["ctx"]
        if c["ragged"]:  # lengths of both spread around their middle, never past 2.5 times it
            n = max(1, min(n, round(n * r.uniform(0.3, 1.0))))
            total = max(n, round(total * min(2.5, math.exp(r.gauss(0.0, 0.6)))))
        out.append((max(total, n), n))
    return out


def work(c):
    lay = LAYOUTS[c["layout"]]
    row = lay["latent"] + lay["bands"] * lay["rope"]
    lens = _lengths(c)
    t = sum(n for _, n in lens)
    if c["op"] == "append":
        return {"bytes": 4 * row * t, "flops": 8 * row * t}  # rows read and written
    if c["op"] == "rotate":
        e = t * c["heads"] * lay["rope"]
        return {"bytes": 4 * e, "flops": 8 * e}
    pairs = sum(n * (total - n) + n * (n + 1) // 2 for total, n in lens)  # (query token, row) pairs
    value = lay["latent"] // lay["bands"]
    key = value + lay["rope"] if c["layout"] == "mla" else lay["rope"]
    kv = sum(total for total, _ in lens) * row * 2
    q_out = t * c["heads"] * (2 * key + 2 * value + 4)
    return {"bytes": kv + q_out, "flops": 2 * pairs * c["heads"] * (key + value)}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    lay = LAYOUTS[c["layout"]]
    lat, band, bands, B = lay["latent"], lay["rope"], lay["bands"], c["block"]
    row = lat + bands * band
    lens = _lengths(c)
    blocks = [-(-total // B) for total, _ in lens]
    pages = sum(blocks) + 7
    t = sum(n for _, n in lens)
    s = {"case": c, "lens": lens}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    # pages in a random order, as a pool hands them out after a while
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["reqs"], max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(blocks):
        table[r, :n] = order[at:at + n]
        at += n
    s["table"] = table
    if c["op"] == "rotate":  # needs no rows: a pool of a page for each request
        kv = torch.zeros(LAYERS * pages * B * row, dtype=torch.bfloat16, device="cuda")
    else:
        kv = normal(LAYERS * pages * B * row)
    pending = None
    if c["lazy"]:  # after splices: runs of rows that share a turn, most of them without one
        runs = [host.choice([0, 0, -host.randrange(1, 6000), host.randrange(1, 200)]) for _ in range(16)]
        pending = torch.zeros(pages * B, dtype=torch.int32, device="cuda")
        for r, (total, n) in enumerate(lens):
            rows = torch.arange(total - n, device="cuda")  # the chunk's own rows carry none
            turn = torch.tensor(runs, device="cuda", dtype=torch.int32)[rows * 16 // max(total, 1)]
            pending[_slots(table[r], rows, B)] = turn
    s["pages"], s["pending"] = pages, pending
    chunks = [(r, total - n, n) for r, (total, n) in enumerate(lens)]
    if own:
        from rope_rotation_gb300 import leyline
        from rope_rotation_gb300.runtime import PagedCache
        flags = (leyline.LEYLINE_POOL_LAZY if c["lazy"] else 0) | (leyline.LEYLINE_POOL_SPLIT_ROPE if c["split"] else 0)
        cache = PagedCache(LAYERS, B, pages, c["reqs"], max(blocks), lat, band, rope_theta=THETA, flags=flags,
                           rope_heads=bands)
        cache.kv.copy_(kv)
        cache.table.copy_(table)
        cache.seq_lens_host[:] = [total for total, _ in lens]
        cache.seq_lens_dev.copy_(torch.tensor([total for total, _ in lens], dtype=torch.int32))
        if pending is not None:
            cache.pending().copy_(pending.view(pages, B))
        kv = cache.kv
        batch = cache.batch(max_chunks=c["reqs"], max_tokens=t, q_heads=c["heads"])
        batch.plan(chunks)  # once a step, for the calls of all its layers
        s["cache"], s["batch"] = cache, batch
    s["kv"] = kv

    # the step's positions and slots, which its layers share
    pos = torch.cat([torch.arange(total - n, total, device="cuda") for total, n in lens])
    req = torch.cat([torch.full((n,), r, device="cuda") for r, (_, n) in enumerate(lens)])
    s["pos"] = pos
    s["slot"] = table[req, pos // B].long() * B + pos % B
    if c["op"] == "append":
        s["rows"] = normal(t, row)
        s["latent_norm"] = (1 + 0.1 * normal(lat).float()).to(torch.bfloat16) if c["layout"] == "mla" else None
        s["key_norm"] = (1 + 0.1 * normal(band).float()).to(torch.bfloat16) if c["layout"] == "grouped" else None
    elif c["op"] == "rotate":
        s["q"] = normal(t, c["heads"], band)
        s["norm"] = (1 + 0.1 * normal(band).float()).to(torch.bfloat16) if c["layout"] == "grouped" else None
        s["out"] = torch.empty_like(s["q"])
    else:
        s["q_latent"] = normal(t, c["heads"], lat) if c["layout"] == "mla" else None
        s["q_rope"] = normal(t, c["heads"], band)
        s["out"] = torch.empty(t, c["heads"], lat // bands, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(t, c["heads"], dtype=torch.float32, device="cuda")
        # padded [request][token] places for the plain form: rows of the cache, and of the chunk's tokens
        longest, most = max(total for total, _ in lens), max(n for _, n in lens)
        rows = torch.arange(longest, device="cuda")
        s["kv_slot"] = table[:, :1].long() * B + torch.zeros_like(rows)
        for r, (total, _) in enumerate(lens):
            s["kv_slot"][r, :total] = _slots(table[r], rows[:total], B)
        tok = torch.arange(most, device="cuda")
        first = torch.tensor([0] + [n for _, n in lens], device="cuda").cumsum(0)[:-1]
        count = torch.tensor([n for _, n in lens], device="cuda")
        start = torch.tensor([total - n for total, n in lens], device="cuda")
        s["tok_ok"] = tok < count[:, None]
        s["tok"] = torch.minimum(first[:, None] + tok, first[:, None] + count[:, None] - 1)
        s["last"] = torch.where(s["tok_ok"], start[:, None] + tok, 0)  # last row a token attends to
    return s


def _slots(table_row, rows, B):
    return table_row[rows // B].long() * B + rows % B


def run(s):
    c = s["case"]
    if own:
        b = s["batch"]
        if c["op"] == "append":
            b.append(LAYER, s["rows"], latent_norm=s["latent_norm"], key_norm=s["key_norm"], eps=EPS)
            return s["kv"]
        if c["op"] == "rotate":
            return b.rotate(s["q"], out=s["out"], norm=s["norm"], eps=EPS)
        return b.attention(LAYER, s["q_latent"], s["q_rope"], LAYOUTS[c["layout"]]["scale"], out=s["out"], lse=s["lse"])
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "rotate":
        q = s["q"].float()
        if s["norm"] is not None:
            q = _rms(q, s["norm"])
        s["out"].copy_(_turn(q, s["pos"][:, None]))
        return s["out"]
    return _plain_attention(s)


def _rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _turn(x, pos):
    """Half-split pairs of the last axis turned by pos * theta_j; the angles in 64 bits."""
    half = x.shape[-1] // 2
    theta = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    a = pos.double()[..., None] * theta
    cos, sin = a.cos().to(x.dtype), a.sin().to(x.dtype)
    x, y = x[..., :half], x[..., half:]
    return torch.cat((x * cos - y * sin, x * sin + y * cos), -1)


def _arrays(c, kv, pages):
    """[layer][slot][...] views of the latents and of the bands."""
    lay = LAYOUTS[c["layout"]]
    lat, bw, slots = lay["latent"], lay["bands"] * lay["rope"], pages * c["block"]
    if c["split"]:
        n = LAYERS * slots * lat
        return kv[:n].view(LAYERS, slots, lat), kv[n:].view(LAYERS, slots, bw)
    rows = kv.view(LAYERS, slots, lat + bw)
    return rows[..., :lat], rows[..., lat:]


def _plain_append(s):
    c = s["case"]
    lay = LAYOUTS[c["layout"]]
    lat, bands = s["rows"][:, :lay["latent"]].float(), s["rows"][:, lay["latent"]:].float()
    if s["latent_norm"] is not None:
        lat = _rms(lat, s["latent_norm"])
    bands = bands.view(-1, lay["bands"], lay["rope"])
    if s["key_norm"] is not None:
        bands = _rms(bands, s["key_norm"])
    bands = _turn(bands, s["pos"][:, None])
    a, b = _arrays(c, s["kv"], s["pages"])
    a[LAYER, s["slot"]] = lat.to(torch.bfloat16)
    b[LAYER, s["slot"]] = bands.flatten(1).to(torch.bfloat16)
    return s["kv"]


def _plain_attention(s):
    c = s["case"]
    lay = LAYOUTS[c["layout"]]
    a, b = _arrays(c, s["kv"], s["pages"])
    n, longest = s["kv_slot"].shape
    lat = a[LAYER][s["kv_slot"]].float()
    band = b[LAYER][s["kv_slot"]].float().view(n, longest, lay["bands"], lay["rope"])
    if s["pending"] is not None:
        band = _turn(band, s["pending"][s["kv_slot"]][..., None])
    group = c["heads"] // lay["bands"]
    if c["layout"] == "mla":  # every head attends to the one key [latent | band]; its value is the latent
        key = torch.cat((lat, band[:, :, 0]), -1)[:, None]
        value = lat[:, None]
        q = torch.cat((s["q_latent"], s["q_rope"]), -1)[s["tok"]].float()
    else:
        key = band.transpose(1, 2)
        value = lat.view(n, longest, lay["bands"], -1).transpose(1, 2)
        q = s["q_rope"][s["tok"]].float()
    most = s["tok"].shape[1]
    q = q.view(n, most, lay["bands"], group, -1).transpose(1, 2).flatten(2, 3)  # [request][key head][token, group][...]
    x = q @ key.transpose(-1, -2) * lay["scale"]
    hidden = torch.arange(longest, device=x.device) > s["last"][..., None]
    x.view(n, lay["bands"], most, group, longest).masked_fill_(hidden[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ value) / total
    lse = (top + total.log())[..., 0]
    out = out.view(n, lay["bands"], most, group, -1).transpose(1, 2).flatten(2, 3)
    lse = lse.view(n, lay["bands"], most, group).transpose(1, 2).flatten(2, 3)
    s["out"].copy_(out[s["tok_ok"]])
    s["lse"].copy_(lse[s["tok_ok"]])
    return s["out"], s["lse"]


def exact(c, seed):
    """From the definitions in 64 bits, request by request; turns as products of complex numbers."""
    s = prepare(c, seed)
    lay = LAYOUTS[c["layout"]]
    L, R, H, B = lay["latent"], lay["rope"], lay["bands"], c["block"]
    slots = s["pages"] * B

    def spun(v, positions):  # v [..., rope], positions broadcast over its leading axes
        z = torch.complex(v[..., :R // 2].contiguous(), v[..., R // 2:].contiguous())
        j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
        w = torch.exp(-2 * j / R * math.log(THETA))
        z = z * torch.polar(torch.ones_like(w), positions.double()[..., None] * w)
        return torch.cat((z.real, z.imag), -1)

    def normed(v, weight):
        return v / (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt() * weight.double()

    if c["op"] == "rotate":
        q = s["q"].double()
        return spun(q if s["norm"] is None else normed(q, s["norm"]), s["pos"][:, None].expand(q.shape[:2]))
    kv = s["kv"].double()
    if c["op"] == "append":
        x = s["rows"].double()
        lat, keys = x[:, :L], x[:, L:].reshape(-1, H, R)
        if s["latent_norm"] is not None:
            lat = normed(lat, s["latent_norm"])
        if s["key_norm"] is not None:
            keys = normed(keys, s["key_norm"])
        keys = spun(keys, s["pos"][:, None].expand(keys.shape[:2])).reshape(-1, H * R)
        at = (LAYER * slots + s["slot"])[:, None]
        if c["split"]:
            kv[at * L + torch.arange(L, device="cuda")] = lat
            kv[LAYERS * slots * L + at * H * R + torch.arange(H * R, device="cuda")] = keys
        else:
            kv[at * (L + H * R) + torch.arange(L + H * R, device="cuda")] = torch.cat((lat, keys), 1)
        return kv
    outs, lses, t0 = [], [], 0
    for r, (total, n) in enumerate(s["lens"]):
        place = torch.arange(total, device="cuda")
        slot = s["table"][r][place // B].long() * B + place % B
        at = (LAYER * slots + slot)[:, None]
        if c["split"]:
            lat = kv[at * L + torch.arange(L, device="cuda")]
            keys = kv[LAYERS * slots * L + at * H * R + torch.arange(H * R, device="cuda")]
        else:
            lat = kv[at * (L + H * R) + torch.arange(L, device="cuda")]
            keys = kv[at * (L + H * R) + L + torch.arange(H * R, device="cuda")]
        keys = keys.view(total, H, R)
        if s["pending"] is not None:
            keys = spun(keys, s["pending"][slot][:, None].expand(total, H))
        seen = place <= (total - n + torch.arange(n, device="cuda"))[:, None]  # [token][row]
        out = torch.empty(n, c["heads"], L // H, dtype=torch.float64, device="cuda")
        lse = torch.empty(n, c["heads"], dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            k = h * H // c["heads"]
            logit = s["q_rope"][t0:t0 + n, h].double() @ keys[:, k].T
            if c["layout"] == "mla":
                logit += s["q_latent"][t0:t0 + n, h].double() @ lat.T
            logit = torch.where(seen, logit * lay["scale"], -math.inf)
            lse[:, h] = torch.logsumexp(logit, 1)
            value = lat if c["layout"] == "mla" else lat.view(total, H, L // H)[:, k]
            out[:, h] = torch.exp(logit - lse[:, h:h + 1]) @ value
        outs.append(out)
        lses.append(lse)
        t0 += n
    return torch.cat(outs), torch.cat(lses)
