// batch_split_sanitize.cpp -- the split of the attention's work (split_work, leyline_batch_plan.cpp) with the item costs of
// both kinds of kernel, built by tests/test_batch_views.py with the sanitizers.
//
// Seeded random chunks.  Pieces cover each row tile's cache rows once, in order and on key-tile borders, CTAs take
// contiguous runs of them, and partial results and joins fit their arrays and name each other.  No CTA has more work than
//   (even + 2 * item_cost + kLeast) * 65 / 64 + 2 * kLeast,   even = cost without cuts / CTAs, kLeast = 2:
// a CTA stops at most item_cost + kLeast - 1 short of its share, and starts at most one piece that another began, which
// costs item_cost again, so a share of even + 2 * item_cost + kLeast goes round; shares grow by 1/64 until one does; and a
// CTA goes past its share by less than a piece that may not be cut smaller.
// Exit code 0: every check held.  Usage: batch_split_sanitize <iterations> <seed>
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "leyline_batch.h"

using namespace leyline;

namespace {
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
}  // namespace

int main(int argc, char** argv)
{
    const long iters = argc > 1 ? std::atol(argv[1]) : 4000;
    std::mt19937_64 rng(argc > 2 ? std::atoll(argv[2]) : 1);
    auto uniform = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    int failures = 0;
    long iter = 0;
    auto check = [&](bool ok, const char* what) {
        if (ok) return;
        if (failures++ < 20) std::fprintf(stderr, "iteration %ld: %s\n", iter, what);
    };
    for (iter = 0; iter < iters; ++iter) {
        const bool pairs = uniform(0, 1) != 0;
        const int32_t ctas = (int32_t)(uniform(0, 1) ? (pairs ? 76 : 152) : uniform(1, 200));
        const WorkShape w{(int32_t)uniform(1, pairs ? 1 : 4), (int32_t)uniform(1, 128), ctas,
                          pairs ? kPairRows : uniform(0, 1) ? kAttnRows : kAttnRowsLazy, pairs ? kItemCostPairs : kItemCost};
        std::vector<ChunkDev> chunks((size_t)uniform(0, 40));
        int32_t tok = 0;
        const int64_t most = uniform(0, 1) ? 30000 : 300;
        for (size_t k = 0; k < chunks.size(); ++k) {
            const int32_t n = (int32_t)uniform(0, uniform(0, 1) ? 3 : 100);
            chunks[k] = ChunkDev{(int32_t)k, n, tok, 0, uniform(0, most)};
            tok += n;
        }
        int64_t tiles = 0, whole = 0;
        for (const ChunkDev& c : chunks)
            for (int64_t r0 = 0; r0 < (int64_t)c.n * w.group; r0 += w.rows) {
                const int64_t last = std::min<int64_t>(r0 + w.rows, (int64_t)c.n * w.group) - 1;
                tiles += w.bands;
                whole += w.bands * (ceil_div(c.start + last / w.group + 1, kAttnKeys) + w.item_cost);
            }
        // exact sizes, so that the sanitizer sees any entry too many
        std::vector<AttnItem> items((size_t)(tiles + ctas));
        std::vector<int32_t> begin(ctas + 1);
        std::vector<AttnJoin> joins(ctas);
        Split sp{items.data(), begin.data(), joins.data()};
        split_work(w, chunks, &sp);
        check(sp.n_items <= tiles + ctas && sp.n_joins <= ctas && sp.n_parts <= 2 * ctas, "array bounds");
        check(begin[0] == 0 && begin[ctas] == sp.n_items, "CTA ranges");
        constexpr int64_t kLeast = 2;
        const int64_t even = ceil_div(whole, ctas);
        for (int32_t i = 0; i < ctas; ++i) {
            check(begin[i] <= begin[i + 1], "CTA ranges out of order");
            int64_t cost = 0;
            for (int32_t k = begin[i]; k < begin[i + 1]; ++k)
                cost += ceil_div(items[k].key1 - items[k].key0, kAttnKeys) + w.item_cost;
            check(cost <= (even + 2 * w.item_cost + kLeast) * 65 / 64 + 2 * kLeast, "an uneven split");
        }
        int32_t at = 0, join = 0, part = 0;
        for (size_t k = 0; k < chunks.size(); ++k)
            for (int32_t band = 0; band < w.bands; ++band)
                for (int64_t r0 = 0; r0 < (int64_t)chunks[k].n * w.group; r0 += w.rows) {
                    const int32_t rows = (int32_t)std::min<int64_t>(w.rows, (int64_t)chunks[k].n * w.group - r0);
                    const int64_t end = chunks[k].start + (r0 + rows - 1) / w.group + 1;
                    int64_t key = 0;
                    const int32_t first = at;
                    while (key < end && at < sp.n_items) {
                        const AttnItem& it = items[at++];
                        check(it.chunk == (int32_t)k && it.band == band && it.row0 == r0 && it.rows == rows && it.key0 == key &&
                                  it.key1 > it.key0 && (it.key1 == end || it.key1 % kAttnKeys == 0),
                              "item fields");
                        key = it.key1;
                    }
                    check(key == end, "a row tile is not covered");
                    if (at - first == 1) {
                        check(items[first].part == -1, "a whole tile has a part");
                        continue;
                    }
                    check(join < sp.n_joins, "a split tile has no join");
                    if (join >= sp.n_joins) break;
                    const AttnJoin& j = joins[join++];
                    check(j.chunk == (int32_t)k && j.band == band && j.row0 == r0 && j.rows == rows && j.part0 == part &&
                              j.parts == at - first,
                          "join fields");
                    for (int32_t i = first; i < at; ++i) check(items[i].part == part++, "parts out of order");
                }
        check(at == sp.n_items && join == sp.n_joins && part == sp.n_parts, "items, joins or parts left over");
    }
    std::printf("%d failed checks\n", failures);
    return failures == 0 ? 0 : 1;
}
