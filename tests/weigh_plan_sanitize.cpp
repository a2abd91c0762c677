// weigh_plan_sanitize.cpp -- a fuzz driver for the plan of weighing rows (weigh_work in leyline_batch_plan.cpp), built by
// tests/test_weigh_plan.py with AddressSanitizer and UndefinedBehaviorSanitizer.
//
// Seeded random chunks and head layouts.  Of every plan it checks that
//   - each request's chunks are linked in the order of their rows, and its rows end where the last one does;
//   - requests whose queries stay come first, each kind in the order of the requests;
//   - the work, decoded as the kernels decode it, covers each row (queries that stay, rows of any shape), or each pair of a
//     tile of cache rows and a query tile (keys that stay), exactly once;
//   - what stays and what passes fit a CTA's shared memory;
//   - the sums of cut query tiles have places of their own within their buffer, and the second kernel finds them.
// Exit code 0: every check held.  Usage: weigh_plan_sanitize <iterations> <seed>
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "leyline_batch.h"

using namespace leyline;

namespace {

uint64_t g_state = 0;

uint64_t next_u64()
{
    uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

int64_t uniform(int64_t lo, int64_t hi) { return lo + (int64_t)(next_u64() % (uint64_t)(hi - lo + 1)); }
bool chance(int percent) { return uniform(0, 99) < percent; }

int failures = 0;
long iter = 0;

void check(bool ok, const char* what)
{
    if (ok) return;
    if (failures < 20) std::fprintf(stderr, "iteration %ld: %s\n", iter, what);
    ++failures;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The last request whose work begins at or before x, as the kernels look it up.
const WeighReq& find(const WeighReq* reqs, int n, int64_t x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].begin <= x) lo = mid;
        else hi = mid - 1;
    }
    return reqs[lo];
}

}  // namespace

int main(int argc, char** argv)
{
    const long iters = argc > 1 ? std::atol(argv[1]) : 2000;
    g_state = argc > 2 ? (uint64_t)std::atoll(argv[2]) : 1;
    long modes[4] = {};
    for (iter = 0; iter < iters; ++iter) {
        Geometry g{};
        g.block_size = (int32_t)uniform(1, 40);
        g.num_pages = 1 << 24;
        leyline_block_table_t bt{};
        bt.num_reqs = (int32_t)uniform(1, 30);
        bt.max_blocks = 4000;
        std::vector<int64_t> lens((size_t)bt.num_reqs);
        for (int64_t& l : lens) l = chance(20) ? 0 : uniform(0, chance(20) ? 60000 : 900);
        for (int64_t& l : lens) l = std::min(l, (int64_t)bt.max_blocks * g.block_size);
        bt.seq_lens_host = lens.data();
        std::vector<leyline_chunk_t> chunks;
        const bool decode = chance(40);
        for (int32_t r = 0; r < bt.num_reqs; ++r) {
            if (chance(30)) continue;
            int64_t at = decode ? std::max<int64_t>(lens[r] - 1, 0) : uniform(0, lens[r]);
            for (int k = 0; k < (decode ? 1 : (int)uniform(1, 3)) && at <= lens[r]; ++k) {
                const int32_t n = decode ? 1 : (int32_t)(chance(20) ? 0 : uniform(1, chance(10) ? 3000 : 60));
                if (at + n > (int64_t)bt.max_blocks * g.block_size) break;
                chunks.push_back(leyline_chunk_t{r, n, at, at});
                at += n + uniform(0, 5);
            }
        }
        // in any order that keeps a request's own
        if (chance(50)) std::stable_sort(chunks.begin(), chunks.end(), [](auto& a, auto& b) { return a.req % 5 < b.req % 5; });
        ChunkPlan plan;
        if (check_chunks(g, bt, chunks.data(), (int32_t)chunks.size(), 1 << 20, 1 << 24, 0, &plan) != LEYLINE_OK) continue;
        std::set<int32_t> named;
        for (const auto& c : chunks)
            if (c.n > 0) named.insert(c.req);
        check(plan.weigh.size() == named.size(), "a request with tokens has work");
        int32_t before = -1;
        size_t linked = 0;
        for (const WeighReq& r : plan.weigh) {
            check(r.req > before && named.count(r.req), "requests ascend");
            before = r.req;
            int64_t last = -1, end = 0;
            for (int32_t c = r.chunk; c >= 0; c = plan.chunks[c].next) {
                check(plan.chunks[c].req == r.req && plan.chunks[c].n > 0 && plan.chunks[c].start > last, "chunks in order");
                last = plan.chunks[c].start;
                end = last + plan.chunks[c].n;
                ++linked;
            }
            check(end == r.end, "end of the rows");
        }
        check(linked == (size_t)std::count_if(chunks.begin(), chunks.end(), [](auto& c) { return c.n > 0; }), "every chunk is linked");

        const int32_t keys[3] = {1, 2, 4};
        const bool mla = chance(50);
        WeighShape w{chance(85), mla ? 1 : (int32_t)uniform(2, 9), (int32_t)(chance(30) ? uniform(1, 400) : uniform(1, 32)),
                     mla ? 9 : keys[uniform(0, 2)], (int32_t)uniform(1, 200),
                     keys[uniform(0, 2)], chance(50)};
        BatchHeader h{};
        std::vector<WeighReq> reqs = plan.weigh;
        weigh_work(w, plan.chunks, &reqs, &h);
        const int n = (int)reqs.size(), stay = h.weigh_stay;
        ++modes[!w.tiles ? 0 : stay == n ? 1 : stay == 0 ? 2 : 3];
        check(h.weigh_reqs == n && stay >= 0 && stay <= n && (w.tiles || stay == 0), "header");
        const int32_t tokens = weigh_tokens(w.group), blocks = (int32_t)ceil_div(w.group, kWeighCols);
        check(tokens * std::min(w.group, kWeighCols) <= kWeighCols, "query tiles fit");
        std::set<int32_t> reqs_of;
        for (int k = 0; k < n; ++k) {
            check(k == 0 || k == stay || reqs[k].req > reqs[k - 1].req, "requests ascend within their kind");
            reqs_of.insert(reqs[k].req);
        }
        check(reqs_of == named, "every request is there");
        // rows: of requests whose queries stay, or of all where the tensor cores do not take them
        const int by_rows = w.tiles ? stay : n;
        const int64_t step = w.tiles ? 32 : 1;
        int64_t at = 0, stay_tiles = 0;
        for (int k = 0; k < by_rows; ++k) {
            const WeighReq& r = reqs[k];
            check(r.begin == at, "work in order");
            at += ceil_div(r.end, step);
            stay_tiles += ceil_div(r.end, kPairKeys);
            const ChunkDev& c = plan.chunks[r.chunk];
            if (w.tiles) check(c.next < 0 && c.n * w.group <= h.weigh_cols && h.weigh_cols <= kWeighCols, "one query tile");
        }
        check(at == (w.tiles ? h.weigh_stay_work : h.weigh_work), "all of it");
        for (int k = 0; k < 20 && at > 0; ++k) {
            const int64_t x = uniform(0, at - 1);
            const WeighReq& r = find(reqs.data(), by_rows, x);
            check(x >= r.begin && x < r.begin + ceil_div(r.end, step), "its request is found");
        }
        if (stay > 0)
            check(stay_bytes(w.bands, w.q_chunks, h.weigh_cols) + 2 * weigh_stage_planes(h.weigh_box, w.bands == 1, w.lazy, w.band_chunks) *
                                                                          kWeighKeys * 128 <= kWeighSmem, "shared memory");
        check(stay == 0 || stay == n || stay_tiles >= kWeighSplit * w.pairs, "two kernels where it is worth it");
        if (!w.tiles) continue;
        // items: of the others
        const WeighReq* others = reqs.data() + stay;
        const int m = n - stay;
        int64_t parts = 0, tiles_before = 0;
        at = 0;
        for (int k = 0; k < m; ++k) {
            const WeighReq& r = others[k];
            const int64_t tiles = ceil_div(r.end, kPairKeys);
            int64_t units = 0;  // products of two query tiles
            for (int32_t c = r.chunk; c >= 0; c = plan.chunks[c].next) units += ceil_div(ceil_div(plan.chunks[c].n, tokens) * blocks, 2);
            check(r.units == units * w.bands && r.begin == at, "units");
            check((int64_t)r.segs * h.weigh_seg >= r.units && (int64_t)(r.segs - 1) * h.weigh_seg < r.units, "segments cover them");
            at += tiles * r.segs;
            if (r.segs > 1) {
                check(r.part == parts && r.tile == tiles_before, "places of cut query tiles");
                parts += tiles * r.segs;
                for (int64_t i : {tiles_before, tiles_before + tiles - 1}) {  // as the second kernel looks them up
                    int lo = 0, hi = m - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (others[mid].tile <= i) lo = mid;
                        else hi = mid - 1;
                    }
                    check(&others[lo] == &r, "a cut tile's request is found");
                }
                tiles_before += tiles;
            }
            for (int64_t i : {r.begin, r.begin + tiles * r.segs - 1}) check(&find(others, m, i) == &r, "an item's request is found");
        }
        check(at == h.weigh_work && tiles_before == h.weigh_tiles, "all of it");
        check(parts <= 2 * (int64_t)kWeighItems * w.pairs, "sums fit their buffer");
    }
    std::printf("%ld plans by rows, %ld with queries that stay, %ld with keys that stay, %ld of both, %d failed checks\n", modes[0],
                modes[1], modes[2], modes[3], failures);
    return failures == 0 && modes[0] > 0 && modes[1] > 0 && modes[2] > 0 && modes[3] > 0 ? 0 : 1;
}
