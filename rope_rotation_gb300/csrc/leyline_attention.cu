// leyline_attention.cu -- attention of a batch's tokens over the paged cache (sm_103a): the
// kernel for any row shape, and the join of split row tiles.
//
// Per query row (token, head), with x_s = scale * <q, k_s> over the rows s it attends to:
//   m = max x_s,  l = sum exp(x_s - m),  out = sum exp(x_s - m) v_s / l,  lse = m + ln l.
// One pass over the rows keeps m, l and the output, multiplying l and the output by
// exp(m_old - m_new) when a tile raises m.
#include "leyline_batch.h"
#include "leyline_device.cuh"

namespace leyline {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// Slot of cache row `row` of a table row; -1 (with the status bit) when its page is bad.
__device__ __forceinline__ long long row_slot(const int32_t* table_row, const Geometry& g, long long row,
                                              int32_t* status)
{
    const long long blk = row / g.block_size;
    const int page = table_row[blk];
    if (page < 0 || page >= g.num_pages) {
        raise_status(status, ST_BAD_PAGE);
        return -1;
    }
    return (long long)page * g.block_size + (row - blk * g.block_size);
}

// ------------------------------------------------------------- any row shape --
// A CTA takes its items' query rows 16 at a time and the cache rows 16 at a time through
// shared memory; one thread per (query row, cache row) score, the output in shared memory.  The output is kept as the
// mean by the weights so far, which is finite wherever the values are.
constexpr int kAnyThreads = 256;
constexpr int kAnyTile = 16;

struct AnyShape {
    int key_vecs, value_vecs, stage_vecs;  // 16-byte vectors of a key, a value and a staged row
    int q_pitch, s_pitch;                  // padded pitches (vectors) of the query and cache rows
    size_t q_off, s_off, o_off, bytes;
};

__host__ __device__ inline AnyShape any_shape(const Geometry& g)
{
    AnyShape s;
    const bool mla = g.rope_heads <= 1;
    s.value_vecs = g.latent_vecs / (mla ? 1 : g.rope_heads);
    s.key_vecs = g.head_vecs + (mla ? g.latent_vecs : 0);
    s.stage_vecs = s.value_vecs + g.head_vecs;  // [value | key band]; MLA: the whole row is the key
    s.q_pitch = s.key_vecs + 1;
    // lazy pools: and the low part of the turned band, which bf16 alone would round away
    s.s_pitch = s.stage_vecs + ((g.flags & LEYLINE_POOL_LAZY) ? g.head_vecs : 0) + 1;
    s.q_off = 0;
    s.s_off = s.q_off + (size_t)16 * kAnyTile * s.q_pitch;
    s.o_off = s.s_off + (size_t)16 * kAnyTile * s.s_pitch;
    s.bytes = s.o_off + sizeof(float) * kAnyTile * s.value_vecs * 8;
    return s;
}

// kRedo: only the items that a tensor-core kernel marked.  It marks those whose output is not finite, since a weight of
// 0 does not keep an infinity or a NaN of a masked row out of a matrix product, and (by pairs) those whose scores left
// its range.  Here a weight of 0 leaves its row out.
template <bool kRedo>
__global__ void __launch_bounds__(kAnyThreads) attend_any_kernel(const __grid_constant__ AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float p_s[kAnyTile][kAnyTile + 1];
    __shared__ float m_s[kAnyTile], l_s[kAnyTile], corr_s[kAnyTile];
    __shared__ long long slot_s[kAnyTile];
    const Geometry& g = a.g;
    const AnyShape sh = any_shape(g);
    uint4* q_s = reinterpret_cast<uint4*>(smem + sh.q_off);
    uint4* kv_s = reinterpret_cast<uint4*>(smem + sh.s_off);
    float* o_s = reinterpret_cast<float*>(smem + sh.o_off);
    const int tid = threadIdx.x;
    const int qi = tid / kAnyTile, ki = tid % kAnyTile;
    const bool mla = g.rope_heads <= 1;
    const int group = a.q_heads / (mla ? 1 : g.rope_heads);
    const int vdim = sh.value_vecs * 8;
    const bool bf16 = g.precision == LEYLINE_ROTATE_BF16_NAIVE;
    const float scale2 = a.scale * kLog2e;
    wait_for_previous_grid();
    allow_next_grid();
    const int pitch = a.header->pairs ? kPairRows : kAttnRows;
    // the CTA's items of the plan, or all items in turn
    const int it0 = kRedo ? blockIdx.x : a.cta_begin[blockIdx.x];
    const int it1 = kRedo ? a.header->n_items : a.cta_begin[blockIdx.x + 1];
    for (int it = it0; it < it1; it += kRedo ? gridDim.x : 1) {
        if (kRedo && a.redo[2 * it] == 0 && a.redo[2 * it + 1] == 0) continue;
        const AttnItem item = a.items[it];
        const ChunkDev ch = a.chunks[item.chunk];
        const int32_t* table_row = a.header->table + (long long)ch.req * a.header->max_blocks;
        for (int r0 = 0; r0 < item.rows; r0 += kAnyTile) {
            const int rows = min(kAnyTile, item.rows - r0);
            __syncthreads();
            for (int i = tid; i < rows * sh.key_vecs; i += kAnyThreads) {
                const int r = i / sh.key_vecs, c = i - r * sh.key_vecs;
                const int row = item.row0 + r0 + r;
                const long long tok = ch.tok0 + row / group, head = item.band * group + row % group;
                const int lat = sh.key_vecs - g.head_vecs;
                const HeadsView& v = c < lat ? a.q_latent : a.q_rope;
                q_s[r * sh.q_pitch + c] =
                    static_cast<const uint4*>(v.ptr)[(tok * v.token_stride + head * v.head_stride) / 8 +
                                                     (c < lat ? c : c - lat)];
            }
            for (int i = tid; i < kAnyTile * vdim; i += kAnyThreads) o_s[i] = 0.f;
            if (tid < kAnyTile) {
                m_s[tid] = -INFINITY;
                l_s[tid] = 0.f;
            }
            const int my_tok = (item.row0 + r0 + min(qi, rows - 1)) / group;
            const long long my_end = a.prefix ? ch.start : ch.start + my_tok + 1;  // rows [0, my_end)
            const int last_tok = (item.row0 + r0 + rows - 1) / group;
            const long long end = min((long long)item.key1, (long long)(a.prefix ? ch.start : ch.start + last_tok + 1));
            for (long long s0 = item.key0; s0 < end; s0 += kAnyTile) {
                const int keys = (int)min((long long)kAnyTile, end - s0);
                __syncthreads();
                if (tid < kAnyTile) slot_s[tid] = tid < keys ? row_slot(table_row, g, s0 + tid, a.status) : -1;
                __syncthreads();
                for (int i = tid; i < kAnyTile * sh.stage_vecs; i += kAnyThreads) {
                    const int r = i / sh.stage_vecs, c = i - r * sh.stage_vecs;
                    const long long slot = slot_s[r];
                    uint4 v = {};
                    if (slot >= 0)
                        v = c < sh.value_vecs ? a.kv[lat_off(g, a.layer, slot) + item.band * sh.value_vecs + c]
                                              : a.kv[band_off(g, a.layer, slot) + item.band * g.head_vecs +
                                                     (c - sh.value_vecs)];
                    kv_s[r * sh.s_pitch + c] = v;
                }
                __syncthreads();
                if (a.pending) {  // turn the bands by their rows' pending counts, into high and low parts
                    const int half = g.rope_dim / 2;
                    for (int i = tid; i < kAnyTile * half; i += kAnyThreads) {
                        const int r = i / half, j = i - r * half;
                        const int pend = slot_s[r] >= 0 ? a.pending[slot_s[r]] : 0;
                        __nv_bfloat16* band = reinterpret_cast<__nv_bfloat16*>(kv_s + r * sh.s_pitch + sh.value_vecs);
                        __nv_bfloat16* low = band + g.rope_dim;
                        const bool split = g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
                        const int e0 = split ? j : 2 * j, e1 = split ? j + half : 2 * j + 1;
                        const float x0 = __bfloat162float(band[e0]), x1 = __bfloat162float(band[e1]);
                        float y0 = x0, y1 = x1;
                        if (pend != 0) {
                            float c, s;
                            pending_trig(pend, a.turn, half, j, bf16, c, s);
                            if (bf16) turn_bf16(x0, x1, c, s, y0, y1);
                            else turn_fp32(x0, x1, c, s, y0, y1);
                        }
                        band[e0] = __float2bfloat16_rn(y0);
                        band[e1] = __float2bfloat16_rn(y1);
                        // the naive arm's result is the rounded one
                        low[e0] = __float2bfloat16_rn(bf16 ? 0.f : y0 - __bfloat162float(band[e0]));
                        low[e1] = __float2bfloat16_rn(bf16 ? 0.f : y1 - __bfloat162float(band[e1]));
                    }
                    __syncthreads();
                }
                float x = -INFINITY;
                if (qi < rows && s0 + ki < my_end && ki < keys) {  // a bad page's row counts as zeros
                    const uint4* qv = q_s + qi * sh.q_pitch;
                    const uint4* kvv = kv_s + ki * sh.s_pitch + (sh.stage_vecs - sh.key_vecs);
                    float acc = 0.f;
                    const int low_vecs = a.pending ? g.head_vecs : 0;
                    for (int c = 0; c < sh.key_vecs + low_vecs; ++c) {
                        // the query's band meets the low part too
                        const uint4 u = qv[c < sh.key_vecs ? c : c - g.head_vecs], w = kvv[c];
                        const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = bf2(uw[e]), h = bf2(ww[e]);
                            acc = fmaf(f.x, h.x, acc);
                            acc = fmaf(f.y, h.y, acc);
                        }
                    }
                    x = acc * scale2;
                }
                // the 16 lanes of a query row
                float top = x;
                for (int m = kAnyTile / 2; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                const float m_old = m_s[qi];
                const float m_new = fmaxf(m_old, top);
                const float p = x == -INFINITY ? 0.f : exp2f(x - m_new);  // a NaN score stays NaN
                float sum = p;
                for (int m = kAnyTile / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                const float l_old = m_new == -INFINITY ? 0.f : l_s[qi] * exp2f(m_old - m_new);
                const float l_new = l_old + sum;
                p_s[qi][ki] = l_new == 0.f ? 0.f : p / l_new;
                __syncwarp();
                if (ki == 0) {
                    corr_s[qi] = l_new == 0.f ? 0.f : l_old / l_new;
                    m_s[qi] = m_new;
                    l_s[qi] = l_new;
                }
                __syncthreads();
                const __nv_bfloat16* val = reinterpret_cast<const __nv_bfloat16*>(kv_s);
                for (int d = tid; d < vdim; d += kAnyThreads) {
                    float v[kAnyTile];
#pragma unroll
                    for (int k = 0; k < kAnyTile; ++k) v[k] = __bfloat162float(val[k * sh.s_pitch * 8 + d]);
                    for (int r = 0; r < rows; ++r) {
                        float o = o_s[r * vdim + d] * corr_s[r];
#pragma unroll
                        for (int k = 0; k < kAnyTile; ++k) o = p_s[r][k] == 0.f ? o : fmaf(p_s[r][k], v[k], o);
                        o_s[r * vdim + d] = o;
                    }
                }
            }
            __syncthreads();
            for (int i = tid; i < rows * vdim; i += kAnyThreads) {
                const int r = i / vdim, d = i - r * vdim;
                const float o = o_s[i];
                const int row = item.row0 + r0 + r;
                if (item.part >= 0) {
                    a.part_out[((long long)item.part * pitch + r0 + r) * vdim + d] = o;
                } else {
                    const long long tok = ch.tok0 + row / group, head = item.band * group + row % group;
                    static_cast<__nv_bfloat16*>(a.out.ptr)[tok * a.out.token_stride + head * a.out.head_stride + d] =
                        __float2bfloat16_rn(o);
                }
            }
            if (tid < rows) {
                const int row = item.row0 + r0 + tid;
                const float lse = l_s[tid] == 0.f ? -INFINITY : (m_s[tid] + log2f(l_s[tid])) * kLn2;
                if (item.part >= 0) {
                    a.part_lse[(long long)item.part * pitch + r0 + tid] = lse;
                } else if (a.lse) {
                    const long long tok = ch.tok0 + row / group, head = item.band * group + row % group;
                    a.lse[tok * a.q_heads + head] = lse;
                }
            }
        }
    }
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
    if (attention_takes_tiles(g)) {
        // the kernel that computes marked items again
        cudaError_t e = cudaFuncSetAttribute(attend_any_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)any_shape(g).bytes);
        return e != cudaSuccess ? (int)e : attention_tile_prepare(g, kv, maps);
    }
    return (int)cudaFuncSetAttribute(attend_any_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)any_shape(g).bytes);
}

int launch_attention_redo(const AttnArgs& a, int ctas, void* stream)
{
    return (int)launch_dependent_smem(attend_any_kernel<true>, ctas, kAnyThreads, any_shape(a.g).bytes,
                                      (cudaStream_t)stream, a);
}

int launch_attention(const AttnArgs& a, const TileMaps& maps, int ctas, void* stream)
{
    if (attention_takes_tiles(a.g)) return launch_attention_tile(a, maps, ctas, stream);
    return (int)launch_dependent_smem(attend_any_kernel<false>, ctas, kAnyThreads, any_shape(a.g).bytes,
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
