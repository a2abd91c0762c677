// leyline_attention.cuh -- what the tensor-core attention kernels share (leyline_attention_tile.cu,
// leyline_attention_pair.cu).
#pragma once

#include "leyline_attention_any.cuh"
#include "leyline_tcgen05.cuh"

namespace leyline {
namespace {

constexpr int kAtomBytes = 1024;  // 8 rows x 128 bytes
constexpr unsigned long long kDrainTime = 1000000ull;  // 1 ms: longer than any load in flight takes

// The item as every role sees it.
struct Work {
    AttnItem it;
    ChunkDev ch;
    int tiles;      // cache tiles
    long long end;  // cache rows [key0, end) are loaded
};

__device__ __forceinline__ Work load_work(const AttnArgs& a, int i)
{
    Work w;
    w.it = a.items[i];
    w.ch = a.chunks[w.it.chunk];
    w.end = min((long long)w.it.key1, a.prefix ? (long long)w.ch.start : (long long)w.it.key1);
    w.tiles = w.end > w.it.key0 ? (int)((w.end - w.it.key0 + kAttnKeys - 1) / kAttnKeys) : 0;
    return w;
}

// The stages in turn, and the parity of their current use.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ void advance(int stages)
    {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// False (for the whole warp) when the CTA has given up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* quit, int32_t* status)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, quit, status));
}

// A cache row's page (as the table has it) and its row in the page; nothing is loaded past `end`.
struct PageOf {
    int page, off;
    bool in;
};

__device__ __forceinline__ PageOf page_of(const AttnArgs& a, const TileMaps& maps, const Work& w, const int32_t* table_row,
                                          long long pos)
{
    const unsigned u = (unsigned)pos, B = (unsigned)a.g.block_size;
    const unsigned blk = maps.shift >= 0 ? u >> maps.shift : u / B;
    PageOf p{-1, (int)(u - blk * B), pos < w.end};
    if (p.in) p.page = table_row[blk];
    return p;
}

// Its slot; -1 past the end and for a bad page.
__device__ __forceinline__ long long slot_of(const AttnArgs& a, const PageOf& p)
{
    if (p.page >= 0 && p.page < a.g.num_pages) return (long long)p.page * a.g.block_size + p.off;
    if (p.in) raise_status(a.status, ST_BAD_PAGE);
    return -1;
}

// Whether TMA takes the tile at `key` (its values, in a lazy pool).
__device__ __forceinline__ bool by_box(const TileMaps& maps, const Work& w, long long key)
{
    return maps.box > 0 && key + kAttnKeys <= w.end;
}

// Where the CTA gives up, what is still in flight must land before it ends.  A stage's barrier may lack arrivals then,
// so the loads are waited for by time.
__device__ __forceinline__ void let_loads_land(int* quit)
{
    if (!*(volatile int*)quit) return;  // every load has been waited for by the MMAs
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < kDrainTime) {
    }
}

// Named barriers of the four softmax warps.
__device__ __forceinline__ bool any_of_softmax(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// The driver's encoder of tensor maps, looked up at run time (the library links no driver library).
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled()
{
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace
}  // namespace leyline
