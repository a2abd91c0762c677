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
// Partial results k of a row: out = sum w_k out_k / sum w_k with w_k = exp(lse_k - max),
// lse = max + ln sum w_k.  A warp per query row and 128 value dimensions: its lanes form the weights of 32 parts at a
// time, then read the parts eight loads at a time (a row split over 128 CTAs took 73 us with one dependent load after
// another).  Where a plan splits tiles into many parts, kSplit = 4 warps share a row's: 12 -> 6 us for that row; with
// two or three parts a row the other three would have nothing to do.  The parts are added in a fixed order, so
// the result does not depend on which CTA finished first.
constexpr int kJoinThreads = 128;

template <int kSplit>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnArgs a, int slices, int rows)
{
    __shared__ float4 sum_s[kJoinThreads];
    __shared__ float total_s[kJoinThreads / 32];
    wait_for_previous_grid();
    // the next kernel is not let in early: its CTAs, one per SM, would crowd onto the SMs that are free first
    constexpr int kUnits = kJoinThreads / 32 / kSplit;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, sub = warp % kSplit;
    const long long unit = blockIdx.x * (long long)kUnits + warp / kSplit;
    const int slice = (int)(unit % slices);
    const int j = (int)(unit / slices / rows), r = (int)(unit / slices % rows);
    // (with kSplit > 1 a CTA has one unit, so it leaves as a whole)
    if (j >= a.header->n_joins) return;
    const AttnJoin jn = a.joins[j];
    if (r >= jn.rows) return;
    const int pitch = a.header->pairs ? kPairRows : kAttnRows;
    const Geometry& g = a.g;
    const bool mla = g.rope_heads <= 1;
    const int group = a.q_heads / (mla ? 1 : g.rope_heads);
    const int vdim = g.latent_dim / (mla ? 1 : g.rope_heads);
    const float* lse = a.part_lse + (long long)jn.part0 * pitch + r;
    float top = -INFINITY;
    for (int k = lane; k < jn.parts; k += 32) top = fmaxf(top, lse[(long long)k * pitch]);
    for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const int d = 128 * slice + 4 * lane;
    const bool on = d < vdim;
    const float* part = a.part_out + ((long long)jn.part0 * pitch + r) * vdim + (on ? d : 0);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    for (int k0 = 32 * sub; k0 < jn.parts; k0 += 32 * kSplit) {
        const int n = min(32, jn.parts - k0);
        const float x = lane < n ? lse[(long long)(k0 + lane) * pitch] : -INFINITY;
        const float mine = x == -INFINITY ? 0.f : exp2f((x - top) * kLog2e);
        total += mine;
        for (int k = 0; k < n; k += 8) {
            float4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = k + u < n ? __ldcg(reinterpret_cast<const float4*>(part + (long long)(k0 + k + u) * pitch * vdim))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float w = __shfl_sync(0xffffffffu, mine, k + u);  // 0 for a part without rows, which wrote zeros
                o.x = fmaf(w, v[u].x, o.x);
                o.y = fmaf(w, v[u].y, o.y);
                o.z = fmaf(w, v[u].z, o.z);
                o.w = fmaf(w, v[u].w, o.w);
            }
        }
    }
    for (int m = 16; m > 0; m /= 2) total += __shfl_xor_sync(0xffffffffu, total, m);
    if (kSplit > 1) {
        sum_s[threadIdx.x] = o;
        if (lane == 0) total_s[warp] = total;
        __syncthreads();
        if (sub != 0) return;
        for (int k = 1; k < kSplit; ++k) {
            const float4 v = sum_s[threadIdx.x + 32 * k];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
            total += total_s[warp + k];
        }
    }
    const float inv = total > 0.f ? 1.f / total : total;
    const ChunkDev ch = a.chunks[jn.chunk];
    const int row = jn.row0 + r;
    const long long tok = ch.tok0 + row / group, head = jn.band * group + row % group;
    if (on)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out.ptr) + tok * a.out.token_stride +
                                  head * a.out.head_stride + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (slice == 0 && lane == 0 && a.lse)
        a.lse[tok * a.q_heads + head] = total > 0.f ? top + log2f(total) * kLn2 : (total == 0.f ? -INFINITY : total);
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
    const int slices = (vdim + 127) / 128;
    const long long units = (long long)joins * rows * slices;
    cudaStream_t s = (cudaStream_t)stream;
    return (int)(many_parts ? launch_dependent(join_kernel<4>, (int)units, kJoinThreads, s, a, slices, rows)
                            : launch_dependent(join_kernel<1>, (int)((units + 3) / 4), kJoinThreads, s, a, slices, rows));
}

}  // namespace leyline
