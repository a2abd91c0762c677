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

// Scale and write the outputs of an item's rows [row, row + 16) that it has: of block b (of `blocks`) a lane holds the
// dimension first + step * b + lane of each (blocks past value_dim: none), in columns of TMEM `pitch` apart; factor: of
// all 16 rows.  kRows: rows of a partial result; scratch: 1 KB of shared memory of this warp's.  Returns whether some
// value is not finite.
// Outputs go through shared memory in 16-byte vectors, their rows' addresses formed once for all blocks: with a 2-byte
// store and an address for each value, the end of an item of 128 rows took 38500 cycles, a fifth of all for 8000 cache rows.
template <int kRows>
__device__ __forceinline__ bool put_rows(const AttnArgs& a, const Work& w, int group, int value_dim, int row, int first,
                                         int step, int blocks, uint32_t tmem, int pitch, const float* factor,
                                         uint32_t scratch)
{
    const int lane = threadIdx.x & 31;
    float f[16];
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(factor + k);
        f[k] = x.x;
        f[k + 1] = x.y;
        f[k + 2] = x.z;
        f[k + 3] = x.w;
    }
    __nv_bfloat16* to[2];  // of rows lane / 4 and 8 + lane / 4, 16 bytes a lane
    bool on[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = row + 8 * i + lane / 4, q = w.it.row0 + r, tok = q / group;
        on[i] = r < w.it.rows;
        to[i] = static_cast<__nv_bfloat16*>(a.out.ptr) + (w.ch.tok0 + tok) * a.out.token_stride +
                (w.it.band * group + q - tok * group) * a.out.head_stride + 8 * (lane % 4);
    }
    const uint32_t sel = lane & 1 ? 0x3276 : 0x5410;
    float bad[2] = {0.f, 0.f};  // 0, or NaN once a value is not finite
#pragma unroll 2
    for (int b = 0; b < blocks; ++b) {
        const int dim = first + step * b;
        if (dim >= value_dim) break;
        uint32_t v[16] = {};
        if (w.tiles > 0) {
            tmem_ld16(tmem + b * pitch, v);
            tmem_wait_ld();
        }
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            o[k] = __uint_as_float(v[k]) * f[k];
            bad[k & 1] = fmaf(o[k], 0.f, bad[k & 1]);
        }
        if (w.it.part >= 0) {
            float* part = a.part_out + ((long long)w.it.part * kRows + row) * value_dim + dim + lane;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (row + k < w.it.rows) part[k * value_dim] = o[k];
            continue;
        }
        // a word of two neighbouring dimensions: even lanes of the even row, odd lanes of the odd one
        uint32_t words[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t x = pack_bf16x2(o[2 * k], o[2 * k + 1]);
            words[k] = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 1), sel);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(scratch + 128 * k + 64 * (lane & 1) + 4 * (lane >> 1)), "r"(words[k])
                         : "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 x;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(scratch + 512 * i + 16 * lane)
                         : "memory");
            if (on[i]) *reinterpret_cast<uint4*>(to[i] + dim) = x;
        }
        __syncwarp();
    }
    return bad[0] + bad[1] != 0.f;
}

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
