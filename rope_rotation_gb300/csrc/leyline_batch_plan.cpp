// leyline_batch_plan.cpp -- host planning of a batch of new tokens: the chunks' validation, the
// pages they take, and the split of the attention's work over the CTAs.  Touches no device.
#include <algorithm>
#include <climits>
#include <cstdio>

#include "leyline_batch.h"

namespace leyline {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int bad(const char* msg) { return set_error(LEYLINE_ERR_INVALID_ARG, msg); }

// Whether [a, a + wa) and [b + d * stride, ... + wb) meet for some d with -below <= d <= above.
bool meet(int64_t a, int64_t wa, int64_t b, int64_t wb, int64_t stride, int64_t below, int64_t above)
{
    if (stride == 0) return a < b + wb && b < a + wa;
    // a - wb < b + d * stride < a + wa
    auto floor_div = [](int64_t x, int64_t y) { return x >= 0 ? x / y : -ceil_div(-x, y); };
    const int64_t lo = floor_div(a - wb - b, stride) + 1, hi = floor_div(a + wa - 1 - b, stride);
    return std::max(lo, -below) <= std::min(hi, above);
}

}  // namespace

bool overlap(Extent a, Extent b)
{
    if (a.tokens <= 0 || b.tokens <= 0 || a.heads <= 0 || b.heads <= 0) return false;
    for (Extent* x : {&a, &b}) {  // the stride of an axis of one entry says nothing
        if (x->heads == 1) x->head_stride = 0;
        if (x->tokens == 1) x->token_stride = 0;
    }
    const int64_t shift = (int64_t)(b.address - a.address);
    auto length = [](const Extent& x) { return (x.tokens - 1) * x.token_stride + (x.heads - 1) * x.head_stride + x.width; };
    if (shift >= length(a) || -shift >= length(b)) return false;
    // Along an axis whose stride they share (or that has one entry in one of them), `n` entries, only the distance of two
    // entries matters; the other axis, `m` entries, is taken as one piece first, then entry by entry.
    enum Answer { kNo, kYes, kUnknown };
    constexpr int64_t kMostPairs = 1 << 16;
    using Field = int64_t Extent::*;
    auto along = [&](Field n, Field stride, Field m, Field other) {
        if (a.*stride != b.*stride && a.*n > 1 && b.*n > 1) return kUnknown;
        const int64_t s = a.*n > 1 ? a.*stride : b.*stride, below = a.*n - 1, above = b.*n - 1;
        if (!meet(0, (a.*m - 1) * (a.*other) + a.width, shift, (b.*m - 1) * (b.*other) + b.width, s, below, above)) return kNo;
        if (a.*other == b.*other || a.*m == 1 || b.*m == 1) {
            if (a.*m + b.*m > kMostPairs) return kUnknown;
            const int64_t o = a.*m > 1 ? a.*other : b.*other;
            for (int64_t d = 1 - a.*m; d < b.*m; ++d)
                if (meet(0, a.width, shift + d * o, b.width, s, below, above)) return kYes;
            return kNo;
        }
        if (a.*m * (b.*m) > kMostPairs) return kUnknown;
        for (int64_t i = 0; i < a.*m; ++i)
            for (int64_t j = 0; j < b.*m; ++j)
                if (meet(i * (a.*other), a.width, shift + j * (b.*other), b.width, s, below, above)) return kYes;
        return kNo;
    };
    Answer x = along(&Extent::tokens, &Extent::token_stride, &Extent::heads, &Extent::head_stride);
    if (x == kUnknown) x = along(&Extent::heads, &Extent::head_stride, &Extent::tokens, &Extent::token_stride);
    return x != kNo;
}

int check_sizes(const Geometry& g, int32_t max_chunks, int32_t max_tokens, int32_t q_heads)
{
    const int32_t bands = std::max(g.rope_heads, 1);
    if (max_chunks < 1 || max_chunks > (1 << 16)) return bad("max_chunks must be in [1, 65536]");
    if (max_tokens < 1 || max_tokens > (1 << 22)) return bad("max_tokens must be in [1, 4194304]");
    if (q_heads < 1 || q_heads > 1024) return bad("q_heads must be in [1, 1024]");
    if (g.latent_dim < 8 || g.latent_dim > kAttnMaxValue || g.latent_dim % (8 * bands) != 0)
        return bad("attention needs a latent_dim in [8, 1024], a multiple of 8 * rope_heads");
    if (g.rope_dim > kAttnMaxRope) return bad("attention needs rope_dim <= 256");
    // the kernels count a chunk's query rows of a band in 32 bits
    if (q_heads % bands == 0 && (int64_t)max_tokens * (q_heads / bands) > INT32_MAX - kPairRows)
        return bad("max_tokens * q_heads / rope_heads must be below 2^31 - 128");
    return LEYLINE_OK;
}

int check_chunks(const Geometry& g, const leyline_block_table_t& bt, const leyline_chunk_t* chunks, int32_t n,
                 int64_t max_tokens, int64_t free_pages, int64_t pop_base, ChunkPlan* out)
{
    char msg[192];
    const int64_t cap = (int64_t)bt.max_blocks * g.block_size;
    struct Req {
        int64_t old_len, len, pop, last_run;
    };
    std::vector<int32_t> order(n);
    std::vector<int32_t> req_of;  // requests of the plan, sorted
    for (int32_t k = 0; k < n; ++k) {
        const leyline_chunk_t& c = chunks[k];
        order[k] = k;
        if (c.req < 0 || c.req >= bt.num_reqs || c.n < 0 || c.start < 0 || c.rope_start < 0 ||
            c.rope_start > ((int64_t)1 << 40)) {
            snprintf(msg, sizeof msg, "chunk %d: request, n, start or rope_start out of range", k);
            return bad(msg);
        }
        out->tokens += c.n;
        if (out->tokens > max_tokens) return bad("more tokens than the batch holds");
        req_of.push_back(c.req);
    }
    std::sort(req_of.begin(), req_of.end());
    req_of.erase(std::unique(req_of.begin(), req_of.end()), req_of.end());
    std::vector<Req> reqs(req_of.size());
    auto find = [&](int32_t req) -> Req& {
        return reqs[std::lower_bound(req_of.begin(), req_of.end(), req) - req_of.begin()];
    };
    for (size_t i = 0; i < reqs.size(); ++i) {
        const int64_t len = bt.seq_lens_host[req_of[i]];
        if (len < 0 || len > cap) return bad("seq_lens_host entry outside [0, max_blocks * block_size]");
        reqs[i] = Req{len, len, -1, -1};
    }
    for (int32_t k = 0; k < n; ++k) {
        const leyline_chunk_t& c = chunks[k];
        Req& r = find(c.req);
        if (c.start > r.len) {
            snprintf(msg, sizeof msg, "chunk %d: start %lld is past the request's length %lld", k, (long long)c.start,
                     (long long)r.len);
            return bad(msg);
        }
        if (c.start + c.n > cap)
            return set_error(LEYLINE_ERR_CAPACITY, "a chunk ends past max_blocks * block_size");
        if (c.start + c.n > INT32_MAX - kAttnKeys) return set_error(LEYLINE_ERR_CAPACITY, "a length above 2^31 - 65");
        if (c.n > 0 && c.start < r.old_len) out->rewrites = true;
        r.len = std::max(r.len, c.start + c.n);
    }
    // rows of one request's chunks may not overlap
    std::sort(order.begin(), order.end(), [&](int32_t x, int32_t y) {
        const leyline_chunk_t &a = chunks[x], &c = chunks[y];
        return a.req != c.req ? a.req < c.req : a.start != c.start ? a.start < c.start : a.n < c.n;
    });
    int32_t before = -1;  // the last chunk with rows
    for (int32_t k : order) {
        const leyline_chunk_t& c = chunks[k];
        if (c.n == 0) continue;
        if (before >= 0 && chunks[before].req == c.req && c.start < chunks[before].start + chunks[before].n) {
            snprintf(msg, sizeof msg, "chunks %d and %d share rows of request %d", before, k, c.req);
            return bad(msg);
        }
        before = k;
    }
    for (size_t i = 0; i < reqs.size(); ++i) {
        Req& r = reqs[i];
        r.pop = pop_base + out->pages;
        out->pages += ceil_div(r.len, g.block_size) - ceil_div(r.old_len, g.block_size);
        if (r.len != r.old_len) out->new_len.emplace_back(req_of[i], r.len);
    }
    if (out->pages > free_pages) return set_error(LEYLINE_ERR_NO_PAGES, "not enough free pages for the chunks' rows");
    int32_t tok = 0;
    for (int32_t k = 0; k < n; ++k) {
        const leyline_chunk_t& c = chunks[k];
        Req& r = find(c.req);
        out->chunks.push_back(ChunkDev{c.req, c.n, tok, 0, c.start});
        for (int32_t t = 0; t < c.n; t += kPlanRun) {
            r.last_run = (int64_t)out->runs.size();
            out->runs.push_back(PlanRun{c.req, std::min(kPlanRun, c.n - t), tok + t,
                                        (int32_t)ceil_div(r.old_len, g.block_size), c.start + t, c.rope_start + t,
                                        r.pop, -1});
        }
        tok += c.n;
    }
    for (const Req& r : reqs)
        if (r.last_run >= 0 && r.len != r.old_len) out->runs[r.last_run].new_len = r.len;
    return LEYLINE_OK;
}

// The split of the attention's work over the CTAs.  A row tile costs its key tiles plus item_cost;
// the tiles form one list, which the CTAs take in contiguous runs of equal cost, so a tile may end
// in one CTA and go on in the next.  A CTA never starts or leaves less than kMinKeyTiles of a tile
// that has more.  split_by cuts by a given share and returns the last CTA's cost.
constexpr int64_t kMinKeyTiles = 2;

static int64_t split_by(const WorkShape& w, const std::vector<ChunkDev>& chunks, int64_t quota, Split* out)
{
    int64_t used = 0;  // of the current CTA's quota
    int32_t cta = 0;
    out->cta_begin[0] = 0;
    auto next_cta = [&] {
        if (cta + 1 < w.ctas) {
            out->cta_begin[++cta] = out->n_items;
            used = 0;
        }
    };
    for (size_t k = 0; k < chunks.size(); ++k) {
        const ChunkDev& c = chunks[k];
        const int64_t rows = (int64_t)c.n * w.group;
        for (int32_t band = 0; band < w.bands; ++band)
            for (int64_t r0 = 0; r0 < rows; r0 += w.rows) {
                const int32_t n_rows = (int32_t)std::min<int64_t>(w.rows, rows - r0);
                const int64_t end = c.start + (r0 + n_rows - 1) / w.group + 1;
                const int64_t tiles = ceil_div(end, kAttnKeys);
                int64_t done = 0;
                int32_t first_item = out->n_items;
                while (done < tiles) {
                    const bool last_cta = cta + 1 == w.ctas;
                    const int64_t left = tiles - done;
                    int64_t take = last_cta ? left : std::min(left, quota - used - w.item_cost);
                    if (take < left && (take < kMinKeyTiles || left - take < kMinKeyTiles)) {
                        // too little room here, or too little left over: all of it or none
                        if (used > 0 && take < kMinKeyTiles) {
                            next_cta();
                            continue;
                        }
                        take = std::min(left, std::max(take, kMinKeyTiles));
                        if (left - take < kMinKeyTiles) take = left;
                    }
                    AttnItem& it = out->items[out->n_items++];
                    it = AttnItem{(int32_t)k, band, (int32_t)r0, n_rows, (int32_t)(done * kAttnKeys),
                                  (int32_t)std::min(end, (done + take) * kAttnKeys), -1, 0};
                    done += take;
                    used += take + w.item_cost;
                    if (used + w.item_cost >= quota) next_cta();
                }
                const int32_t parts = out->n_items - first_item;
                if (parts > 1) {
                    out->joins[out->n_joins++] =
                        AttnJoin{(int32_t)k, band, (int32_t)r0, n_rows, out->n_parts, parts, {0, 0}};
                    for (int32_t i = first_item; i < out->n_items; ++i) out->items[i].part = out->n_parts++;
                }
            }
    }
    while (cta < w.ctas) out->cta_begin[++cta] = out->n_items;
    return used;
}

void split_work(const WorkShape& w, const std::vector<ChunkDev>& chunks, Split* out)
{
    int64_t total = 0, pieces = 0;
    for (const ChunkDev& c : chunks) {
        const int64_t rows = (int64_t)c.n * w.group;
        for (int64_t r0 = 0; r0 < rows; r0 += w.rows) {
            const int64_t last = (std::min(r0 + w.rows, rows) - 1) / w.group;
            total += w.bands * ceil_div(c.start + last + 1, kAttnKeys);
            pieces += w.bands;
        }
    }
    // Cutting tiles adds pieces, and borders leave some of a CTA's share unused: the last CTA takes
    // what is left, so the share grows until that is no more than a share.
    const Split empty = *out;
    int64_t quota = ceil_div(total + w.item_cost * pieces, w.ctas) + 1;
    while (split_by(w, chunks, quota, out) > quota) {
        *out = empty;
        quota += std::max<int64_t>(1, quota / 64);
    }
}

// Whether the work goes to pairs of CTAs: by an estimate of either kernel's cycles.  A cache tile of 64 rows takes a CTA
// 3800 cycles and 10 for each query row, a pair 1900 for up to 128; an item costs a pair more at its ends, and the call
// 4000 cycles more to start.  16 requests decode over 24000 rows: 16 heads 111 us by CTAs, 107 by pairs, 64 heads 124,
// 113, 128 heads 206, 123; 64 over 4000 rows: 16 heads 78, 81, 64 heads 92, 90; one over 32768: 16 heads 18, 21, 128 heads
// 28, 25; 300 over 130 rows: 64 heads 36, 40.  Rows that are copied one by one (`copied`: block sizes that 8 does not
// divide) take a pair 2450 a tile, a CTA no more than the others: 16 over 24000 rows, 64 heads 129, 140, 128 heads 213, 143.
bool pairs_are_faster(const WorkShape& w, const std::vector<ChunkDev>& chunks, bool copied)
{
    constexpr int64_t kTile = 3800, kTileRow = 10, kTileItem = 8400, kPairItem = 12000, kPairStart = 4000;
    const int64_t pair_tile = copied ? 2450 : 1900;
    const int64_t pairs = w.ctas / 2;
    int64_t single = kTileItem * w.ctas, pair = kPairItem * pairs;  // as many items are cut
    for (const ChunkDev& c : chunks) {
        const int64_t rows = (int64_t)c.n * w.group, keys = ceil_div(c.start + c.n, kAttnKeys);
        const int64_t tiles = ceil_div(rows, kAttnRows), pair_tiles = ceil_div(rows, kPairRows);
        single += tiles * (keys * kTile + kTileItem) + rows * keys * kTileRow;
        pair += pair_tiles * (keys * pair_tile + kPairItem);
    }
    return single * pairs > (pair + kPairStart * pairs) * w.ctas;
}

}  // namespace leyline
