// weigh_sizes_sanitize.cpp -- the plan of weighing rows (weigh_work in leyline_batch_plan.cpp) at the largest sizes that a batch
// takes: query rows of a band up to 2^31 - 128, cache rows up to 2^31 - 65.  Built by tests/test_weigh_sizes.py with the
// sanitizers.  Exit code 0: query tiles are cut into segments that cover them, and their sums fit their buffer.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "leyline_batch.h"

using namespace leyline;

int main()
{
    int failures = 0, plans = 0;
    for (int32_t group : {1, 3, 16, 128, 129, 512, 1024})
        for (int32_t bands : {1, 2, 8})
            for (int32_t pairs : {1, 76})
                for (int64_t rows : {1000ll, 1000000ll, 2147483583ll})
                    for (int32_t requests : {1, 2, 50}) {
                        const int64_t most = std::min<int64_t>({(INT32_MAX - 128) / group, 1 << 22, rows * requests});
                        const int32_t n = (int32_t)std::max<int64_t>(1, most / requests);
                        std::vector<ChunkDev> chunks;
                        std::vector<WeighReq> reqs;
                        for (int32_t r = 0; r < requests; ++r) {
                            chunks.push_back(ChunkDev{r, n, r * n, -1, rows - n});
                            reqs.push_back(WeighReq{r, r, rows, 0, 0, 0, 0, 0});
                        }
                        const WeighShape w{true, bands, group, bands == 1 ? 9 : 2, pairs, bands == 1 ? 1 : 2, false};
                        BatchHeader h{};
                        weigh_work(w, chunks, &reqs, &h);
                        ++plans;
                        const int64_t tokens = weigh_tokens(group), blocks = (group + kWeighCols - 1) / kWeighCols;
                        int64_t parts = 0, items = 0;
                        bool ok = h.weigh_seg > 0;
                        for (size_t k = h.weigh_stay; k < reqs.size(); ++k) {
                            const WeighReq& r = reqs[k];
                            const int64_t tiles = (r.end + kPairKeys - 1) / kPairKeys;
                            const int64_t units = ((n + tokens - 1) / tokens * blocks + 1) / 2 * bands;
                            ok = ok && r.units == units && r.segs > 0 && r.begin == items && (int64_t)r.segs * h.weigh_seg >= units &&
                                 (int64_t)(r.segs - 1) * h.weigh_seg < units;
                            items += tiles * r.segs;
                            if (r.segs > 1) parts += tiles * r.segs;
                        }
                        ok = ok && items == h.weigh_work && parts <= 2ll * kWeighItems * pairs;
                        if (!ok && failures++ < 10)
                            std::fprintf(stderr, "group %d, %d bands, %d pairs, %lld rows, %d requests of %d tokens: segments of %d\n", group,
                                         bands, pairs, (long long)rows, requests, n, h.weigh_seg);
                    }
    std::printf("%d plans, %d failed checks\n", plans, failures);
    return failures == 0 ? 0 : 1;
}
