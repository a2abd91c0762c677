// batch_plan_sanitize.cpp -- a fuzz driver for the host plan of a batch of new tokens
// (leyline_batch_plan.cpp), built by tests/test_batch_plan.py with AddressSanitizer and
// UndefinedBehaviorSanitizer.
//
// Seeded random lengths and chunks, valid and invalid.  Of every accepted plan it checks that
//   - the runs cover each chunk's rows once, in token order, and the pages taken are those the
//     new lengths need;
//   - the split covers each row tile's cache rows once, in order, in pieces on key-tile borders;
//     every CTA's range lies in the item list; partial results and joins fit their arrays
//     (2 * CTAs and CTAs) and name each other;
//   - no CTA has much more work than an even share.
// Exit code 0: every check held.  Usage: batch_plan_sanitize <iterations> <seed>
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
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

}  // namespace

int main(int argc, char** argv)
{
    const long iters = argc > 1 ? std::atol(argv[1]) : 20000;
    g_state = argc > 2 ? (uint64_t)std::atoll(argv[2]) : 1;
    long accepted = 0, refused = 0;
    for (iter = 0; iter < iters; ++iter) {
        Geometry g{};
        g.block_size = (int32_t)(chance(30) ? 1 : uniform(2, 40));
        const int32_t num_reqs = (int32_t)uniform(1, 20);
        const int32_t max_blocks = (int32_t)uniform(1, 4000);
        const int64_t cap = (int64_t)max_blocks * g.block_size;
        std::vector<int64_t> lens(num_reqs);
        for (auto& x : lens) x = uniform(0, chance(50) ? cap : std::min<int64_t>(cap, 200));
        leyline_block_table_t bt{};
        bt.seq_lens_host = lens.data();
        bt.num_reqs = num_reqs;
        bt.max_blocks = max_blocks;
        const int32_t n = (int32_t)uniform(0, 2 * num_reqs);
        std::vector<leyline_chunk_t> chunks(n);
        std::vector<int64_t> cur = lens;
        for (auto& c : chunks) {
            c.req = (int32_t)uniform(chance(3) ? -1 : 0, num_reqs - (chance(3) ? 0 : 1));
            const int64_t len = c.req >= 0 && c.req < num_reqs ? cur[c.req] : 0;
            c.n = (int32_t)uniform(chance(3) ? -1 : 0, chance(50) ? 3 : 700);
            c.start = chance(70) ? len : uniform(chance(3) ? -1 : 0, len + (chance(3) ? 1 : 0));
            c.rope_start = chance(90) ? std::max<int64_t>(c.start, 0) : uniform(-1, 100000);
            if (c.req >= 0 && c.req < num_reqs) cur[c.req] = std::max(len, c.start + c.n);
        }
        const int64_t free_pages = chance(80) ? 1 << 20 : uniform(0, 50);
        const int64_t max_tokens = chance(80) ? 1 << 20 : uniform(1, 500);
        const int64_t pop_base = uniform(0, 1000);
        ChunkPlan plan;
        const int rc = check_chunks(g, bt, chunks.data(), n, max_tokens, free_pages, pop_base, &plan);
        // an independent statement of what is valid
        bool valid = true;
        int64_t tokens = 0, pages = 0;
        std::vector<int64_t> len = lens;
        std::map<int32_t, std::vector<std::pair<int64_t, int64_t>>> rows;
        for (const auto& c : chunks) {
            if (c.req < 0 || c.req >= num_reqs || c.n < 0 || c.start < 0 || c.rope_start < 0 || c.start > len[c.req] ||
                c.start + c.n > cap) {
                valid = false;
                break;
            }
            len[c.req] = std::max(len[c.req], c.start + c.n);
            tokens += c.n;
            for (const auto& x : rows[c.req])
                if (c.n > 0 && c.start < x.second && x.first < c.start + c.n) valid = false;
            if (c.n > 0) rows[c.req].emplace_back(c.start, c.start + c.n);
        }
        if (valid)
            for (int32_t r = 0; r < num_reqs; ++r) pages += ceil_div(len[r], g.block_size) - ceil_div(lens[r], g.block_size);
        valid = valid && tokens <= max_tokens && pages <= free_pages;
        check((rc == LEYLINE_OK) == valid, "accepted and valid differ");
        if (rc != LEYLINE_OK) {
            ++refused;
            continue;
        }
        ++accepted;
        check(plan.tokens == tokens && plan.pages == pages, "token or page count");
        check((int32_t)plan.chunks.size() == n, "chunk count");
        size_t run = 0;
        std::map<int32_t, int64_t> stored;
        std::vector<char> taken((size_t)pages, 0);
        for (int32_t k = 0; k < n; ++k) {
            const ChunkDev& c = plan.chunks[k];
            check(c.req == chunks[k].req && c.n == chunks[k].n && c.start == chunks[k].start, "chunk fields");
            int64_t at = 0;
            while (at < c.n && run < plan.runs.size()) {
                const PlanRun& r = plan.runs[run++];
                check(r.req == c.req && r.start == c.start + at && r.tok0 == c.tok0 + at && r.n > 0 && r.n <= kPlanRun &&
                          r.rope_start == chunks[k].rope_start + at,
                      "run fields");
                check(r.old_blocks == ceil_div(lens[c.req], g.block_size), "old blocks");
                if (r.new_len >= 0) {
                    check(stored.emplace(c.req, r.new_len).second, "a length is stored twice");
                }
                for (int64_t t = r.start; t < r.start + r.n; ++t)
                    if (t / g.block_size >= r.old_blocks && t % g.block_size == 0) {
                        const int64_t p = r.pop + t / g.block_size - r.old_blocks - pop_base;
                        check(p >= 0 && p < pages && !taken[(size_t)p], "a page is taken twice or out of range");
                        if (p >= 0 && p < pages) taken[(size_t)p] = 1;
                    }
                at += r.n;
            }
            check(at == c.n, "runs do not cover a chunk");
        }
        check(run == plan.runs.size(), "runs left over");
        check(std::count(taken.begin(), taken.end(), 1) == pages, "a page taken has no row");
        for (int32_t r = 0; r < num_reqs; ++r)
            check((len[r] != lens[r]) == (stored.count(r) != 0) && (!stored.count(r) || stored[r] == len[r]),
                  "stored length");

        WorkShape w{(int32_t)uniform(1, 4), (int32_t)uniform(1, 64), (int32_t)(chance(50) ? 152 : uniform(1, 200)),
                    chance(50) ? kAttnRows : chance(50) ? kAttnRowsLazy : kPairRows};
        (void)pairs_are_faster(w, plan.chunks);
        int64_t tiles = 0, work = 0;
        for (const ChunkDev& c : plan.chunks) tiles += w.bands * ceil_div((int64_t)c.n * w.group, w.rows);
        // exact sizes, so that the sanitizer sees any entry too many
        std::vector<AttnItem> items((size_t)(tiles + w.ctas));
        std::vector<int32_t> begin(w.ctas + 1);
        std::vector<AttnJoin> joins(w.ctas);
        Split sp{items.data(), begin.data(), joins.data()};
        split_work(w, plan.chunks, &sp);
        check(sp.n_items <= tiles + w.ctas && sp.n_joins <= w.ctas && sp.n_parts <= 2 * w.ctas, "array bounds");
        check(begin[0] == 0 && begin[w.ctas] == sp.n_items, "CTA ranges");
        int64_t heaviest = 0;
        for (int32_t i = 0; i < w.ctas; ++i) {
            check(begin[i] <= begin[i + 1], "CTA ranges out of order");
            int64_t cost = 0;
            for (int32_t k = begin[i]; k < begin[i + 1]; ++k) cost += ceil_div(items[k].key1 - items[k].key0, kAttnKeys) + 2;
            heaviest = std::max(heaviest, cost);
            work += cost;
        }
        check(heaviest <= ceil_div(work, w.ctas) * 33 / 32 + 8, "an uneven split");
        int32_t at = 0, join = 0, part = 0;
        for (int32_t k = 0; k < n; ++k)
            for (int32_t band = 0; band < w.bands; ++band)
                for (int64_t r0 = 0; r0 < (int64_t)plan.chunks[k].n * w.group; r0 += w.rows) {
                    const int64_t left = (int64_t)plan.chunks[k].n * w.group - r0;
                    const int32_t n_rows = (int32_t)std::min<int64_t>(w.rows, left);
                    const int64_t end = plan.chunks[k].start + (r0 + n_rows - 1) / w.group + 1;
                    int64_t key = 0;
                    const int32_t first = at;
                    while (key < end && at < sp.n_items) {
                        const AttnItem& it = items[at++];
                        check(it.chunk == k && it.band == band && it.row0 == r0 && it.rows == n_rows && it.key0 == key &&
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
                    check(j.chunk == k && j.band == band && j.row0 == r0 && j.rows == n_rows && j.part0 == part &&
                              j.parts == at - first,
                          "join fields");
                    for (int32_t i = first; i < at; ++i) check(items[i].part == part++, "parts out of order");
                }
        check(at == sp.n_items && join == sp.n_joins && part == sp.n_parts, "items, joins or parts left over");
    }
    std::printf("%ld accepted, %ld refused, %d failed checks\n", accepted, refused, failures);
    return failures == 0 ? 0 : 1;
}
