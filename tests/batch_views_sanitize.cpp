// batch_views_sanitize.cpp -- overlap() of two views of token tensors (leyline_batch_plan.cpp) against the bytes that they
// name, one by one, on seeded random views; built by tests/test_batch_views.py with the sanitizers.
// Exit code 0: it never misses a shared byte, and tells views apart wherever they share a stride.
// Usage: batch_views_sanitize <iterations> <seed>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>

#include "leyline_batch.h"

using namespace leyline;

int main(int argc, char** argv)
{
    const long iters = argc > 1 ? std::atol(argv[1]) : 20000;
    std::mt19937_64 rng(argc > 2 ? std::atoll(argv[2]) : 1);
    auto uniform = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
    long met = 0, apart = 0, failures = 0;
    for (long iter = 0; iter < iters; ++iter) {
        auto view = [&] {
            Extent x{};
            x.address = 1000 + uniform(0, 60);
            x.tokens = uniform(0, 6);
            x.heads = uniform(0, 5);
            x.width = uniform(1, 8);
            x.token_stride = uniform(0, 40);
            x.head_stride = uniform(0, 40);
            return x;
        };
        const Extent a = view();
        Extent b = view();
        const int kind = (int)uniform(0, 4);  // parts of one tensor, mostly
        if (kind >= 2) b.token_stride = a.token_stride;
        if (kind == 1 || kind >= 3) b.head_stride = a.head_stride;
        std::set<uintptr_t> bytes;
        for (int64_t t = 0; t < a.tokens; ++t)
            for (int64_t h = 0; h < a.heads; ++h)
                for (int64_t i = 0; i < a.width; ++i) bytes.insert(a.address + t * a.token_stride + h * a.head_stride + i);
        bool shared = false;
        for (int64_t t = 0; t < b.tokens; ++t)
            for (int64_t h = 0; h < b.heads; ++h)
                for (int64_t i = 0; i < b.width; ++i) shared |= bytes.count(b.address + t * b.token_stride + h * b.head_stride + i) > 0;
        (shared ? met : apart) += 1;
        const bool got = overlap(a, b);
        if (got != overlap(b, a) || (shared && !got) || (!shared && got && kind > 0)) {
            if (++failures < 20)
                std::fprintf(stderr, "iteration %ld: kind %d, shared %d, got %d\n", iter, kind, shared, got);
        }
    }
    // large ones: a token's row of 128 heads as [query 64 | output 512], and head after head of a long chunk
    const int64_t T = 1 << 22, H = 1024;
    const Extent q{1 << 20, T, H, 2 * H * 576, 2 * 576, 128}, out{(1 << 20) + 128, T, H, 2 * H * 576, 2 * 576, 1024};
    Extent shifted = out;
    shifted.address -= 16;
    const Extent rows{1 << 20, T, H, 128, T * 256, 128}, halves{(1 << 20) + T * 128, T, H, 128, T * 256, 128};
    if (overlap(q, out) || !overlap(q, shifted) || overlap(rows, halves)) ++failures;
    std::printf("%ld met, %ld apart, %ld failed checks\n", met, apart, failures);
    return failures == 0 ? 0 : 1;
}
