// leyline_attention.cu -- attention of a batch's tokens over the paged cache (sm_103a): the
// kernel for any row shape, and the join of split row tiles.
#include "leyline_attention_any.cuh"

namespace leyline {
namespace {

// ------------------------------------------------------------- any row shape --
__global__ void __launch_bounds__(kAnyThreads) attend_any_kernel(const __grid_constant__ AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    wait_for_previous_grid();
    allow_next_grid();
    for (int it = a.cta_begin[blockIdx.x]; it < a.cta_begin[blockIdx.x + 1]; ++it)
        attend_rows<kAnyThreads>(a, a.items[it], 0, a.items[it].rows, kAttnRows, smem);
}

// -------------------------------------------------------------------- join --
// Partial results k of a row: out = sum w_k out_k with w_k = exp(lse_k - max) / sum of these, lse = max + ln of that sum.
// A warp takes kSlices times 128 value dimensions of a query row: its lanes form the weights of 32 parts at a time, then
// read the parts eight loads at a time (a row split over 128 CTAs took 73 us with one dependent load after another).
// Bound by the latency of these steps: with 4 slices a warp and a row's 512 dimensions in one, a quarter as many warps
// go through them (62 tiles of 128 rows in 2 or 3 parts: 26 -> 12 us).  Where a plan splits tiles into many parts, kSplit = 4
// warps share a row's parts: 12 -> 6 us for that row; with two or three parts the other warps would have nothing to do.
// The parts are added in a fixed order, so the result does not depend on which CTA finished first.
constexpr int kJoinThreads = 128;
constexpr int kJoinSlice = 128;

template <int kSplit, int kSlices>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnArgs a, int groups, int per_join)
{
    __shared__ float4 sum_s[kSlices][kJoinThreads];
    wait_for_previous_grid();
    // the next kernel is not let in early: its CTAs, one per SM, would crowd onto the SMs that are free first
    constexpr int kUnits = kJoinThreads / 32 / kSplit;  // of a CTA: (row, group of slices)
    constexpr int kAtOnce = 8 / kSlices;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, sub = warp % kSplit;
    const int j = blockIdx.x / per_join, unit = (blockIdx.x - j * per_join) * kUnits + warp / kSplit;
    const int r = unit / groups, first = (unit - r * groups) * kSlices * kJoinSlice + 4 * lane;
    const AttnJoin jn = a.joins[j];
    // (with kSplit > 1 a CTA has one unit, so it leaves as a whole)
    if (j >= a.header->n_joins || r >= jn.rows) return;
    const int pitch = a.header->pairs ? kPairRows : kAttnRows;
    const ChunkDev ch = a.chunks[jn.chunk];
    const Geometry& g = a.g;
    const bool mla = g.rope_heads <= 1;
    const int group = a.q_heads / (mla ? 1 : g.rope_heads);
    const int vdim = g.latent_dim / (mla ? 1 : g.rope_heads);
    const float* lse = a.part_lse + (long long)jn.part0 * pitch + r;
    float top = -INFINITY;
    for (int k = lane; k < jn.parts; k += 32) top = fmaxf(top, lse[(long long)k * pitch]);
    for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    // a part without rows: lse -inf, weight 0 (it wrote zeros)
    auto weight = [&](int k) {
        const float x = k < jn.parts ? lse[(long long)k * pitch] : -INFINITY;
        return x == -INFINITY ? 0.f : exp2f((x - top) * kLog2e);
    };
    float total = 0.f;
    for (int k = lane; k < jn.parts; k += 32) total += weight(k);
    for (int m = 16; m > 0; m /= 2) total += __shfl_xor_sync(0xffffffffu, total, m);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const float* part = a.part_out + ((long long)jn.part0 * pitch + r) * vdim + first;
    float4 o[kSlices];
#pragma unroll
    for (int s = 0; s < kSlices; ++s) o[s] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 32 * sub; k0 < jn.parts; k0 += 32 * kSplit) {
        const int n = min(32, jn.parts - k0);
        const float mine = weight(k0 + lane) * inv;
        for (int k = 0; k < n; k += kAtOnce) {
            float4 v[kAtOnce][kSlices];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                for (int s = 0; s < kSlices; ++s)
                    v[u][s] = k + u < n && first + s * kJoinSlice < vdim
                                  ? __ldcg(reinterpret_cast<const float4*>(part + (long long)(k0 + k + u) * pitch * vdim +
                                                                           s * kJoinSlice))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const float w = __shfl_sync(0xffffffffu, mine, k + u);
#pragma unroll
                for (int s = 0; s < kSlices; ++s) {
                    o[s].x = fmaf(w, v[u][s].x, o[s].x);
                    o[s].y = fmaf(w, v[u][s].y, o[s].y);
                    o[s].z = fmaf(w, v[u][s].z, o[s].z);
                    o[s].w = fmaf(w, v[u][s].w, o[s].w);
                }
            }
        }
    }
    if (kSplit > 1) {
#pragma unroll
        for (int s = 0; s < kSlices; ++s) sum_s[s][threadIdx.x] = o[s];
        __syncthreads();
        if (sub != 0) return;
        for (int k = 1; k < kSplit; ++k)
#pragma unroll
            for (int s = 0; s < kSlices; ++s) {
                const float4 v = sum_s[s][threadIdx.x + 32 * k];
                o[s].x += v.x;
                o[s].y += v.y;
                o[s].z += v.z;
                o[s].w += v.w;
            }
    }
    const int row = jn.row0 + r, tok = row / group;
    const long long t = ch.tok0 + tok, head = jn.band * group + row - tok * group;
    __nv_bfloat16* to =
        static_cast<__nv_bfloat16*>(a.out.ptr) + t * a.out.token_stride + head * a.out.head_stride + first;
#pragma unroll
    for (int s = 0; s < kSlices; ++s)
        if (first + s * kJoinSlice < vdim)
            *reinterpret_cast<uint2*>(to + s * kJoinSlice) =
                make_uint2(pack_bf16x2(o[s].x, o[s].y), pack_bf16x2(o[s].z, o[s].w));
    if (first == 0 && a.lse)
        a.lse[t * a.q_heads + head] = total > 0.f ? top + log2f(total) * kLn2 : (total == 0.f ? -INFINITY : total);
}

}  // namespace

int attention_prepare(const Geometry& g, const void* kv, TileMaps* maps)
{
    if (attention_takes_tiles(g)) return attention_tile_prepare(g, kv, maps);
    return (int)cudaFuncSetAttribute(attend_any_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)any_shape(g).bytes);
}

int launch_attention(const AttnArgs& a, const TileMaps& maps, int ctas, void* stream)
{
    if (attention_takes_tiles(a.g)) return launch_attention_tile(a, maps, ctas, stream);
    return (int)launch_dependent_smem(attend_any_kernel, ctas, kAnyThreads, any_shape(a.g).bytes,
                                      (cudaStream_t)stream, a);
}

int launch_join(const AttnArgs& a, int joins, int rows, bool many_parts, void* stream)
{
    const int vdim = a.g.latent_dim / std::max(a.g.rope_heads, 1);
    const int slices = many_parts ? 1 : 4, groups = (vdim + slices * kJoinSlice - 1) / (slices * kJoinSlice);
    const int units = kJoinThreads / 32 / (many_parts ? 4 : 1);
    const int per_join = (rows * groups + units - 1) / units;
    cudaStream_t s = (cudaStream_t)stream;
    return (int)(many_parts ? launch_dependent(join_kernel<4, 1>, joins * per_join, kJoinThreads, s, a, groups, per_join)
                            : launch_dependent(join_kernel<1, 4>, joins * per_join, kJoinThreads, s, a, groups, per_join));
}

}  // namespace leyline
