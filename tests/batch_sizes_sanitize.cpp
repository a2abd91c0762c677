// batch_sizes_sanitize.cpp -- the sizes a batch takes (check_sizes, leyline_batch_plan.cpp), built by
// tests/test_batch_views.py.  The items of the attention's work number a chunk's query rows (token, head of a band) in 32
// bits, with room for a whole tile past the last.  Exit code 0: every check held.
#include <climits>
#include <cstdio>

#include "leyline_batch.h"

using namespace leyline;

int main()
{
    int failures = 0;
    auto takes = [&](int32_t latent, int32_t rope, int32_t bands, int32_t chunks, int32_t tokens, int32_t heads, bool want) {
        Geometry g{};
        g.latent_dim = latent;
        g.rope_dim = rope;
        g.rope_heads = bands;
        if ((check_sizes(g, chunks, tokens, heads) == LEYLINE_OK) != want) {
            std::fprintf(stderr, "latent %d, rope %d, bands %d, chunks %d, tokens %d, heads %d: %s\n", latent, rope, bands, chunks,
                         tokens, heads, want ? "refused" : "taken");
            ++failures;
        }
    };
    takes(512, 64, 1, 1, 1, 1, true);
    takes(512, 64, 1, 1 << 16, 1 << 20, 1024, true);
    takes(512, 64, 1, 1, 1 << 21, 1024, false);  // 2^31 rows
    takes(512, 64, 1, 1, (1 << 21) - 1, 1024, true);
    takes(512, 64, 1, 1, 1 << 22, 1024, false);
    takes(512, 64, 1, 1, 1 << 22, 512, false);
    takes(512, 64, 1, 1, 1 << 22, 511, true);
    takes(512, 64, 4, 1, 1 << 22, 1024, true);   // 256 heads a band
    takes(512, 64, 2, 1, 1 << 22, 1024, false);
    takes(512, 64, 2, 1, 1 << 22, 1023, true);   // for append and rotate alone
    takes(512, 64, 1, 0, 1, 1, false);
    takes(512, 64, 1, (1 << 16) + 1, 1, 1, false);
    takes(512, 64, 1, 1, (1 << 22) + 1, 1, false);
    takes(512, 64, 1, 1, 1, 1025, false);
    takes(0, 64, 1, 1, 1, 1, false);
    takes(1032, 64, 1, 1, 1, 1, false);
    takes(512, 272, 1, 1, 1, 1, false);
    takes(520, 64, 2, 1, 1, 2, false);
    std::printf("%d failed checks\n", failures);
    return failures == 0 ? 0 : 1;
}
