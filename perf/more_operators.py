"""The operators of eviction by attention weight over a paged cache, as cases to be timed and compared.

A serving step that has to stay within a budget of rows per request

  weigh      adds to each row's weight what the step's queries gave it: the sum over tokens and heads of
             exp(scale <q, k_s> - lse), with the lse that attention returned (in every layer);
  select     picks the rows a request keeps: its first and its last few, and of the others those of the
             greatest weight (equal weights: the lowest rows);
  evict      drops the other rows in all layers: kept row i of the list becomes row i, its bands stay at the
             positions they were encoded at, its weight and its pending turn move along, and the pages past
             the new length go back.  With one row a page only table entries move.

Rows are as in the pool: [latent 512 | key band 64] for MLA, or [values of 4 heads x 128 | keys of 4 heads x
128] for grouped heads.
"""
import math
import random

import torch

own = False

THETA = 10000.0
LAYERS = 2  # weigh: rows of one layer lie among those of others, as in a pool
LAYER = 1

#: Row layouts: latent (or values of all heads), key band, bands per row, softmax scale.
LAYOUTS = {
    "mla": {"latent": 512, "rope": 64, "bands": 1, "scale": 192 ** -0.5},
    "grouped": {"latent": 512, "rope": 128, "bands": 4, "scale": 128 ** -0.5},
}


def listed():
    return [
        # one new token of one request (27-layer, 16-head shape): the smallest call, latency alone
        _weigh("weigh: one token", reqs=1, tokens=1, ctx=4096, heads=16),
        # 16 requests of the concurrency sweep decode (61-layer, 128-head shape)
        _weigh("weigh: decode sweep", reqs=16, tokens=1, ctx=24000, heads=128, ragged=True),
        # the last 64 tokens of a 32k prompt vote on its rows
        _weigh("weigh: last window of a prompt", reqs=1, tokens=64, ctx=32768, heads=16, decay=0.0),
        # a prompt chunk, 128 heads: the largest product
        _weigh("weigh: prompt chunk", reqs=1, tokens=512, ctx=8192, heads=128),
        # grouped heads: four drafted tokens of each of 16 requests, older weight fading
        _weigh("weigh: grouped drafts", reqs=16, tokens=4, ctx=8000, heads=32, layout="grouped", decay=0.9, ragged=True),
        # 64 short requests after splices in a lazy pool with one row a page
        _weigh("weigh: decode lazy", reqs=64, tokens=1, ctx=4001, heads=16, block=1, lazy=True, ragged=True),
        # one request is cut to a quarter: the smallest call
        _select("select: one request", reqs=1, ctx=4096, keep=0.25),
        # 16 requests of the concurrency sweep are cut to half
        _select("select: sweep", reqs=16, ctx=24000, keep=0.5, ragged=True),
        # long requests lose a few per cent of their rows
        _select("select: long requests", reqs=8, ctx=131072, keep=0.95),
        # the rows of a 32k request in 27 layers are cut to half
        _evict("evict: 27 x 32k to half", reqs=1, ctx=32768, layers=27, keep=0.5),
        # 16 requests in a lazy pool lose a tenth
        _evict("evict: lazy, ragged", reqs=16, ctx=8000, layers=4, keep=0.9, lazy=True, ragged=True),
        # one row a page: only table entries, weights and counts move
        _evict("evict: one row a page", reqs=16, ctx=24000, layers=1, keep=0.5, block=1, lazy=True, ragged=True),
    ]


def _case(op, name, **fields):
    c = {"op": op, "heads": 16, "tokens": 1, "layout": "mla", "block": 16, "lazy": False, "split": False,
         "ragged": False, "shape": 5, "layers": LAYERS, "decay": 1.0, "keep": 1.0, "first": 0, "last": 0}
    c.update(fields)
    if name is not None:
        c["name"] = name
    return c


def _weigh(name, **fields):
    return _case("weigh", name, **fields)


def _select(name, **fields):
    return _case("select", name, **{"first": 4, "last": 64, **fields})


def _evict(name, **fields):
    return _case("evict", name, **{"first": 4, "last": 64, **fields})


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    common = {"shape": rng.randrange(1 << 20), "ragged": rng.random() < 0.7}
    op = rng.choice(["weigh", "weigh", "select", "evict"])
    pool = {"block": rng.choice([1, 5, 16, 16, 64]), "lazy": rng.random() < 0.3, "split": rng.random() < 0.3,
            "layout": "mla" if rng.random() < 0.7 else "grouped"}
    if op == "weigh":
        heads = rng.choice([4, 8, 12, 20, 32, 64]) if pool["layout"] == "grouped" else rng.choice([1, 5, 16, 16, 20, 40, 64, 128])
        reqs, tokens, ctx = _log_int(rng, 1, 64), _log_int(rng, 1, 512), _log_int(rng, 1, 32768)
        # no dearer than the listed ones: fewer requests, then fewer tokens
        while (reqs * tokens * heads * (tokens + ctx) > 2 ** 28 or reqs * (tokens + ctx) > 2 ** 18
               or reqs * tokens * heads > 2 ** 16):
            if reqs > 1:
                reqs = (reqs + 1) // 2
            else:
                tokens = (tokens + 1) // 2
        return _weigh(None, reqs=reqs, tokens=tokens, ctx=tokens + ctx, heads=heads, decay=rng.choice([1.0, 1.0, 0.9, 0.0]),
                      **common, **pool)
    keep = rng.choice([0.02, 0.25, 0.5, 0.5, 0.9, 0.99])
    ends = {"first": rng.choice([0, 1, 4, 37]), "last": rng.choice([0, 1, 64, 333])}
    if op == "select":
        reqs, ctx = _log_int(rng, 1, 64), _log_int(rng, 100, 131072)
        while reqs * ctx > 2 ** 19:
            reqs = (reqs + 1) // 2
        return _select(None, reqs=reqs, ctx=ctx, keep=keep, **ends, **common)
    reqs, ctx, layers = _log_int(rng, 1, 32), _log_int(rng, 100, 32768), _log_int(rng, 1, 27)
    while reqs * ctx * layers > 2 ** 19:
        if reqs > 1:
            reqs = (reqs + 1) // 2
        else:
            layers = (layers + 1) // 2
    return _evict(None, reqs=reqs, ctx=ctx, layers=layers, keep=keep, **ends, **common, **pool)


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


def _keeps(c):
    """(request, rows kept, first rows kept, last rows kept) of each request: the weights always have a say."""
    out = []
    for r, (total, _) in enumerate(_lengths(c)):
        first, last = min(c["first"], total // 8), min(c["last"], total // 8)
        out.append((r, max(min(round(total * c["keep"]), total - 2), first + last + 2), first, last))
    return out


def work(c):
    lay = LAYOUTS[c["layout"]]
    row = lay["latent"] + lay["bands"] * lay["rope"]
    lens = _lengths(c)
    rows = sum(total for total, _ in lens)
    if c["op"] == "select":  # weights read, rows of the list written
        return {"bytes": 4 * rows + 4 * sum(k[1] for k in _keeps(c)), "flops": rows}
    if c["op"] == "evict":  # rows behind the first dropped one read and written, list, weights and counts
        kept, moved = sum(k[1] for k in _keeps(c)), sum(k[1] - k[2] for k in _keeps(c))
        b = 4 * kept + 8 * kept + (8 * kept if c["lazy"] else 0)
        return {"bytes": b + (8 * kept if c["block"] == 1 else 4 * row * c["layers"] * moved), "flops": rows}
    t = sum(n for _, n in lens)
    pairs = sum(n * (total - n) + n * (n + 1) // 2 for total, n in lens)  # (query token, row) pairs
    key = row if c["layout"] == "mla" else lay["rope"]
    key_bytes = 2 * (row if c["layout"] == "mla" else lay["bands"] * lay["rope"])
    return {"bytes": rows * (key_bytes + 8) + t * c["heads"] * (2 * key + 4), "flops": 2 * pairs * c["heads"] * key}


def _slots(table_row, rows, B):
    return table_row[rows // B].long() * B + rows % B


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    lay = LAYOUTS[c["layout"]]
    lat, band, bands, B, layers = lay["latent"], lay["rope"], lay["bands"], c["block"], c["layers"]
    row = lat + bands * band
    lens = _lengths(c)
    blocks = [-(-total // B) for total, _ in lens]
    longest = max(blocks) * B
    s = {"case": c, "lens": lens, "keeps": _keeps(c)}

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    # weights of earlier steps, of about this step's size: a few rows have most of them, some were never attended to
    weights = (2 * normal(c["reqs"], longest)).exp_() * (0.1 * c["heads"] * c["tokens"] / c["ctx"])
    weights[uniform(c["reqs"], longest) < 0.1] = 0.0
    for r, (total, _) in enumerate(lens):
        weights[r, total:] = 0.0
    s["weights"] = weights
    cache_rows = 0 if c["op"] == "select" else sum(blocks) + 7
    pages = max(cache_rows, 1)
    # pages in a random order, as a pool hands them out after a while
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["reqs"], max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(blocks):
        table[r, :n] = order[at:at + n] if cache_rows else 0
        at += n
    kv = normal(layers * pages * B * row).to(torch.bfloat16)
    pending = None
    if c["lazy"]:  # after splices: runs of rows that share a turn, most of them without one
        runs = [host.choice([0, 0, -host.randrange(1, 6000), host.randrange(1, 200)]) for _ in range(16)]
        pending = torch.zeros(pages * B, dtype=torch.int32, device="cuda")
        for r, (total, n) in enumerate(lens):
            rows = torch.arange(total - n, device="cuda")  # the chunk's own rows carry none
            turn = torch.tensor(runs, device="cuda", dtype=torch.int32)[rows * 16 // max(total, 1)]
            pending[_slots(table[r], rows, B)] = turn
    lens_dev = torch.tensor([total for total, _ in lens], dtype=torch.int32, device="cuda")
    s["pages"] = pages
    s["kept"] = torch.full((c["reqs"], max(k[1] for k in s["keeps"])), -1, dtype=torch.int32, device="cuda")
    if c["op"] == "evict":  # the lists that a policy made: of the weights' greatest
        for r, n, first, last in s["keeps"]:
            s["kept"][r, :n] = _greatest(weights[r], lens[r][0], n, first, last)
    s["kv"], s["table"], s["seq_lens"], s["pending"] = kv, table, lens_dev, pending
    if c["op"] == "weigh":
        t = sum(n for _, n in lens)
        s["q_latent"] = normal(t, c["heads"], lat).to(torch.bfloat16) if c["layout"] == "mla" else None
        s["q_rope"] = normal(t, c["heads"], band).to(torch.bfloat16)
        # padded [request][token] places for the plain form: rows of the cache, and of the chunk's tokens
        most, longest = max(n for _, n in lens), max(total for total, _ in lens)
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
        s["total"] = lens_dev.long()
        # what attention over the same rows returned
        x = _scores(s)
        n, bands_, most, group, longest = x.shape
        lse = torch.logsumexp(x, -1)
        s["lse"] = lse.transpose(1, 2).flatten(2, 3)[s["tok_ok"]].contiguous()
    if own:
        from rope_rotation_gb300 import leyline
        from rope_rotation_gb300.runtime import PagedCache
        flags = (leyline.LEYLINE_POOL_LAZY if c["lazy"] else 0) | (leyline.LEYLINE_POOL_SPLIT_ROPE if c["split"] else 0)
        cache = PagedCache(layers, B, pages, c["reqs"], max(blocks), lat, band, rope_theta=THETA, flags=flags,
                           rope_heads=bands)
        leyline.leyline_alloc_pages(cache.pool, pages)  # every page is in use; evictions give some back
        cache.kv.copy_(kv)
        cache.table.copy_(table)
        cache.seq_lens_host[:] = [total for total, _ in lens]
        cache.seq_lens_dev.copy_(lens_dev)
        if pending is not None:
            cache.pending().copy_(pending.view(pages, B))
            s["pending"] = cache.pending().view(-1)
        s["kv"], s["cache"] = cache.kv, cache
        s["table"], s["seq_lens"] = cache.table, cache.seq_lens_dev
        if c["op"] == "weigh":
            s["batch"] = cache.batch(max_chunks=c["reqs"], max_tokens=sum(n for _, n in lens), q_heads=c["heads"])
            s["batch"].plan([(r, total - n, n) for r, (total, n) in enumerate(lens)])  # once a step, for all its layers
        elif c["op"] == "evict":
            leyline.leyline_pool_checkpoint(cache.pool)
    if c["op"] == "evict":  # what a pass starts from
        s["before"] = (s["table"].clone(), s["seq_lens"].clone(), None if pending is None else s["pending"].clone())
    return s


def run(s):
    c = s["case"]
    if c["op"] == "weigh":
        if own:
            s["batch"].attention_weights(LAYER, s["q_latent"], s["q_rope"], s["lse"], LAYOUTS[c["layout"]]["scale"],
                                         s["weights"], decay=c["decay"])
            return s["weights"]
        return _plain_weigh(s)
    if c["op"] == "select":
        if own:
            return s["cache"].select_rows(s["weights"], s["keeps"], out=s["kept"])
        for r, n, first, last in s["keeps"]:
            s["kept"][r, :n] = _greatest(s["weights"][r], s["lens"][r][0], n, first, last)
        return s["kept"]
    # the eviction before is dropped, as a program drops one that it does not want: its rows stay as they were moved
    table, seq_lens, pending = s["before"]
    s["table"].copy_(table)
    s["seq_lens"].copy_(seq_lens)
    if own:
        from rope_rotation_gb300 import leyline
        cache = s["cache"]
        leyline.leyline_pool_rollback(cache.pool, leyline.LEYLINE_ROLLBACK_ACCEPT_TURNED)
        cache.seq_lens_host[:] = [total for total, _ in s["lens"]]
        cache.evict(s["keeps"], s["kept"], weights=s["weights"])
    else:
        if pending is not None:
            s["pending"].copy_(pending)
        _plain_evict(s)
    moved = [] if c["block"] == 1 else [s["kv"]]  # with one row a page no row moves
    return moved + [s["table"], s["seq_lens"], s["weights"]] + ([] if pending is None else [s["pending"]])


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
        n = c["layers"] * slots * lat
        return kv[:n].view(c["layers"], slots, lat), kv[n:].view(c["layers"], slots, bw)
    rows = kv.view(c["layers"], slots, lat + bw)
    return rows[..., :lat], rows[..., lat:]


def _scores(s):
    """[request][key head][token][group][row] scores in 32 bits, -inf where a token does not attend."""
    c = s["case"]
    lay = LAYOUTS[c["layout"]]
    a, b = _arrays(c, s["kv"], s["pages"])
    n, longest = s["kv_slot"].shape
    band = b[LAYER][s["kv_slot"]].float().view(n, longest, lay["bands"], lay["rope"])
    if s["pending"] is not None:
        band = _turn(band, s["pending"][s["kv_slot"]][..., None])
    if c["layout"] == "mla":  # every head attends to the one key [latent | band]
        key = torch.cat((a[LAYER][s["kv_slot"]].float(), band[:, :, 0]), -1)[:, None]
        q = torch.cat((s["q_latent"], s["q_rope"]), -1)[s["tok"]].float()
    else:
        key = band.transpose(1, 2)
        q = s["q_rope"][s["tok"]].float()
    most, group = s["tok"].shape[1], c["heads"] // lay["bands"]
    q = q.view(n, most, lay["bands"], group, -1).transpose(1, 2).flatten(2, 3)  # [request][key head][token, group][...]
    x = (q @ key.transpose(-1, -2)).mul_(lay["scale"]).view(n, lay["bands"], most, group, longest)
    hidden = torch.arange(longest, device=x.device) > s["last"][..., None]
    return x.masked_fill_(hidden[:, None, :, None], -math.inf)


def _plain_weigh(s):
    c, lay, w = s["case"], LAYOUTS[s["case"]["layout"]], s["weights"]
    x = _scores(s)
    n, bands, most, group, longest = x.shape
    lse = torch.full((n, most, c["heads"]), math.inf, device=x.device)  # places without a token get nothing
    lse[s["tok_ok"]] = s["lse"]
    p = x.sub_(lse.view(n, most, bands, group).transpose(1, 2)[..., None]).exp_()
    new = w[:, :longest] * c["decay"] + p.sum((1, 2, 3))
    inside = torch.arange(longest, device=x.device) < s["total"][:, None]
    w[:, :longest] = torch.where(inside, new, w[:, :longest])
    return w


def _greatest(w, total, n, first, last):
    """Ascending rows that a request of `total` rows keeps."""
    rows = torch.arange(total, device=w.device)
    order = w[first:total - last].sort(descending=True, stable=True).indices[:n - first - last] + first
    return torch.cat((rows[:first], order.sort().values, rows[total - last:])).to(torch.int32)


def _plain_evict(s):
    c, w = s["case"], s["weights"]
    B = c["block"]
    for r, n, _, _ in s["keeps"]:
        total = s["lens"][r][0]
        old = _slots(s["table"][r], torch.arange(total, device=w.device), B)
        kept = s["kept"][r, :n].long()
        turns = None if s["pending"] is None else s["pending"][old[kept]]
        w[r, :n] = w[r, kept]
        w[r, n:total] = 0.0
        if B == 1:
            if turns is not None:
                s["pending"][old] = 0
                s["pending"][old[kept]] = turns
            s["table"][r, :n] = s["table"][r, kept]
        else:
            if turns is not None:
                s["pending"][old[:n]] = turns
                s["pending"][old[n:]] = 0
            for part in _arrays(c, s["kv"], s["pages"]):
                part[:, old[:n]] = part[:, old[kept]]
        s["table"][r, -(-n // B):] = -1
        s["seq_lens"][r] = n
    return s


def exact(c, seed):
    """From the definitions, in 64 bits where something is computed, request by request."""
    s = prepare(c, seed)
    lay = LAYOUTS[c["layout"]]
    L, R, H, B = lay["latent"], lay["rope"], lay["bands"], c["block"]
    slots = s["pages"] * B
    if c["op"] == "select":
        kept = s["kept"].clone()
        w = s["weights"].cpu()
        for r, n, first, last in s["keeps"]:
            total = s["lens"][r][0]
            middle = sorted(range(first, total - last), key=lambda t, v=w[r].tolist(): (-v[t], t))[:n - first - last]
            rows = sorted(list(range(first)) + middle + list(range(total - last, total)))
            kept[r, :n] = torch.tensor(rows, dtype=torch.int32)
        return kept
    if c["op"] == "evict":
        kv, table, weights = s["kv"].clone(), s["table"].clone(), s["weights"].clone()
        seq = s["seq_lens"].clone()
        pending = None if s["pending"] is None else s["pending"].clone()
        place = lambda r, t: int(hosts[r][t // B]) * B + t % B
        hosts = s["table"].cpu().tolist()
        row = L + H * R
        for r, n, _, _ in s["keeps"]:
            total, rows = s["lens"][r][0], s["kept"][r, :n].cpu().tolist()
            src = torch.tensor([place(r, t) for t in rows], device="cuda", dtype=torch.long)
            every = torch.tensor([place(r, t) for t in range(total)], device="cuda", dtype=torch.long)
            weights[r, :total] = 0.0
            weights[r, :n] = s["weights"][r].index_select(0, torch.tensor(rows, device="cuda", dtype=torch.long))
            seq[r] = n
            table[r] = -1
            if pending is not None:
                pending[every] = 0
            if B == 1:
                table[r, :n] = src.to(torch.int32)
                if pending is not None:
                    pending[src] = s["pending"][src]
                continue
            table[r, :-(-n // B)] = s["table"][r, :-(-n // B)]
            dst = every[:n]
            if pending is not None:
                pending[dst] = s["pending"][src]
            for layer in range(c["layers"]):
                base = layer * slots
                for width, start in ((L, 0), (H * R, c["layers"] * slots * L)) if c["split"] else ((row, 0),):
                    size = c["layers"] * slots * width
                    kv[start:start + size].view(-1, width)[base + dst] = s["kv"][start:start + size].view(-1, width)[base + src]
        moved = [] if B == 1 else [kv]
        return moved + [table, seq, weights.double()] + ([] if pending is None else [pending])

    def spun(v, positions):  # v [..., rope], positions broadcast over its leading axes
        z = torch.complex(v[..., :R // 2].contiguous(), v[..., R // 2:].contiguous())
        j = torch.arange(R // 2, dtype=torch.float64, device="cuda")
        w = torch.exp(-2 * j / R * math.log(THETA))
        z = z * torch.polar(torch.ones_like(w), positions.double()[..., None] * w)
        return torch.cat((z.real, z.imag), -1)

    out, t0 = s["weights"].double(), 0
    for r, (total, n) in enumerate(s["lens"]):
        place = torch.arange(total, device="cuda")
        slot = s["table"][r][place // B].long() * B + place % B
        at = (LAYER * slots + slot)[:, None]
        if c["split"]:
            lat = s["kv"][at * L + torch.arange(L, device="cuda")].double()
            keys = s["kv"][c["layers"] * slots * L + at * H * R + torch.arange(H * R, device="cuda")].double()
        else:
            lat = s["kv"][at * (L + H * R) + torch.arange(L, device="cuda")].double()
            keys = s["kv"][at * (L + H * R) + L + torch.arange(H * R, device="cuda")].double()
        keys = keys.view(total, H, R)
        if s["pending"] is not None:
            keys = spun(keys, s["pending"][slot][:, None].expand(total, H))
        seen = place <= (total - n + torch.arange(n, device="cuda"))[:, None]  # [token][row]
        got = torch.zeros(total, dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            logit = s["q_rope"][t0:t0 + n, h].double() @ keys[:, h * H // c["heads"]].T
            if c["layout"] == "mla":
                logit += s["q_latent"][t0:t0 + n, h].double() @ lat.T
            got += torch.where(seen, torch.exp(logit * lay["scale"] - s["lse"][t0:t0 + n, h].double()[:, None]), 0.0).sum(0)
        out[r, :total] = out[r, :total] * c["decay"] + got
        t0 += n
    return out
