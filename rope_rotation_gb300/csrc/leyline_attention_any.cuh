// leyline_attention_any.cuh -- attention of a row tile of any row shape: the kernel of the rows that the tensor-core
// kernels do not take (leyline_attention.cu), and what those call for an item that they cannot finish.
//
// Per query row (token, head), with x_s = scale * <q, k_s> over the rows s it attends to:
//   m = max x_s,  l = sum exp(x_s - m),  out = sum exp(x_s - m) v_s / l,  lse = m + ln l.
// One pass over the rows keeps m, l and the output as the mean by the weights so far, which is finite wherever the
// values are.  A weight of 0 leaves its row out, whatever it holds.  On the CUDA cores, bound by instructions: 16 decodes of 32
// heads over 4000 rows of 8 bands of 96 take 723 us (0.3 TB/s).
#pragma once

#include "leyline_batch.h"
#include "leyline_device.cuh"

namespace leyline {
namespace {

__device__ __forceinline__ float2 bf2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// cos and sin of pending * theta_j, as a read of a lazy pool forms them (leyline_read.cu): in fp64, rounded once.  Below
// kTurnSpan^2 by R(a) R(b) = R(a + b) from the pool's two turn tables, past it by sincos.
__device__ __forceinline__ void pending_trig(int pend, const double* turn, int half, int j, bool bf16, float& c, float& s)
{
    const long long n = llabs((long long)pend);
    double sd, cd;
    if (n < (long long)kTurnSpan * kTurnSpan) {
        const double2* tables = reinterpret_cast<const double2*>(turn + (half + 1) / 2 * 2) + (size_t)j * kTurnSpan;
        const double2 x = tables[n % kTurnSpan], y = tables[(size_t)half * kTurnSpan + n / kTurnSpan];
        cd = fma(y.x, x.x, -(y.y * x.y));
        sd = copysign(1.0, (double)pend) * fma(y.y, x.x, y.x * x.y);
    } else {
        sincos((double)pend * turn[j], &sd, &cd);
    }
    c = bf16 ? __bfloat162float(__double2bfloat16(cd)) : (float)cd;
    s = bf16 ? __bfloat162float(__double2bfloat16(sd)) : (float)sd;
}

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

// Query rows and cache rows are taken 16 at a time through shared memory; one thread per (query row, cache row) score,
// the output in shared memory.
constexpr int kAnyThreads = 256;
constexpr int kAnyTile = 16;

struct AnyScratch {
    float p[kAnyTile][kAnyTile + 1];
    float m[kAnyTile], l[kAnyTile], corr[kAnyTile];
    long long slot[kAnyTile];
};

struct AnyShape {
    int key_vecs, value_vecs, stage_vecs;  // 16-byte vectors of a key, a value and a staged row
    int q_pitch, s_pitch;                  // padded pitches (vectors) of the query and cache rows
    size_t q_off, s_off, o_off, scratch, bytes;
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
    s.scratch = s.o_off + sizeof(float) * kAnyTile * s.value_vecs * 8;
    s.bytes = s.scratch + sizeof(AnyScratch);
    return s;
}

// Rows [from, to) of an item, by the `kThreads` threads of a CTA; pitch: rows of a partial result.
template <int kThreads>
__device__ __noinline__ void attend_rows(const AttnArgs& a, const AttnItem item, int from, int to, int pitch,
                                         unsigned char* smem)
{
    static_assert(kThreads >= kAnyThreads, "a thread per score");
    const Geometry& g = a.g;
    const AnyShape sh = any_shape(g);
    uint4* q_s = reinterpret_cast<uint4*>(smem + sh.q_off);
    uint4* kv_s = reinterpret_cast<uint4*>(smem + sh.s_off);
    float* o_s = reinterpret_cast<float*>(smem + sh.o_off);
    AnyScratch& s = *reinterpret_cast<AnyScratch*>(smem + sh.scratch);
    const int tid = threadIdx.x;
    const int qi = tid / kAnyTile % kAnyTile, ki = tid % kAnyTile;
    const bool mla = g.rope_heads <= 1;
    const int group = a.q_heads / (mla ? 1 : g.rope_heads);
    const int vdim = sh.value_vecs * 8;
    const bool bf16 = g.precision == LEYLINE_ROTATE_BF16_NAIVE;
    const float scale2 = a.scale * kLog2e;
    const ChunkDev ch = a.chunks[item.chunk];
    const int32_t* table_row = a.header->table + (long long)ch.req * a.header->max_blocks;
    for (int r0 = from; r0 < to; r0 += kAnyTile) {
        const int rows = min(kAnyTile, to - r0);
        __syncthreads();
        for (int i = tid; i < rows * sh.key_vecs; i += kThreads) {
            const int r = i / sh.key_vecs, c = i - r * sh.key_vecs;
            const int row = item.row0 + r0 + r;
            const long long tok = ch.tok0 + row / group, head = item.band * group + row % group;
            const int lat = sh.key_vecs - g.head_vecs;
            const HeadsView& v = c < lat ? a.q_latent : a.q_rope;
            q_s[r * sh.q_pitch + c] =
                static_cast<const uint4*>(v.ptr)[(tok * v.token_stride + head * v.head_stride) / 8 +
                                                 (c < lat ? c : c - lat)];
        }
        for (int i = tid; i < kAnyTile * vdim; i += kThreads) o_s[i] = 0.f;
        if (tid < kAnyTile) {
            s.m[tid] = -INFINITY;
            s.l[tid] = 0.f;
        }
        const int my_tok = (item.row0 + r0 + min(qi, rows - 1)) / group;
        const long long my_end = a.prefix ? ch.start : ch.start + my_tok + 1;  // rows [0, my_end)
        const int last_tok = (item.row0 + r0 + rows - 1) / group;
        const long long end = min((long long)item.key1, (long long)(a.prefix ? ch.start : ch.start + last_tok + 1));
        for (long long s0 = item.key0; s0 < end; s0 += kAnyTile) {
            const int keys = (int)min((long long)kAnyTile, end - s0);
            __syncthreads();
            if (tid < kAnyTile) s.slot[tid] = tid < keys ? row_slot(table_row, g, s0 + tid, a.status) : -1;
            __syncthreads();
            for (int i = tid; i < kAnyTile * sh.stage_vecs; i += kThreads) {
                const int r = i / sh.stage_vecs, c = i - r * sh.stage_vecs;
                const long long slot = s.slot[r];
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
                for (int i = tid; i < kAnyTile * half; i += kThreads) {
                    const int r = i / half, j = i - r * half;
                    const int pend = s.slot[r] >= 0 ? a.pending[s.slot[r]] : 0;
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
            if (tid < kAnyThreads) {
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
                const float m_old = s.m[qi];
                const float m_new = fmaxf(m_old, top);
                const float p = x == -INFINITY ? 0.f : exp2f(x - m_new);  // a NaN score stays NaN
                float sum = p;
                for (int m = kAnyTile / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                const float l_old = m_new == -INFINITY ? 0.f : s.l[qi] * exp2f(m_old - m_new);
                const float l_new = l_old + sum;
                s.p[qi][ki] = l_new == 0.f ? 0.f : p / l_new;
                __syncwarp();
                if (ki == 0) {
                    s.corr[qi] = l_new == 0.f ? 0.f : l_old / l_new;
                    s.m[qi] = m_new;
                    s.l[qi] = l_new;
                }
            }
            __syncthreads();
            const __nv_bfloat16* val = reinterpret_cast<const __nv_bfloat16*>(kv_s);
            for (int d = tid; d < vdim; d += kThreads) {
                float v[kAnyTile];
#pragma unroll
                for (int k = 0; k < kAnyTile; ++k) v[k] = __bfloat162float(val[k * sh.s_pitch * 8 + d]);
                for (int r = 0; r < rows; ++r) {
                    float o = o_s[r * vdim + d] * s.corr[r];
#pragma unroll
                    for (int k = 0; k < kAnyTile; ++k) o = s.p[r][k] == 0.f ? o : fmaf(s.p[r][k], v[k], o);
                    o_s[r * vdim + d] = o;
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < rows * vdim; i += kThreads) {
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
            const float lse = s.l[tid] == 0.f ? -INFINITY : (s.m[tid] + log2f(s.l[tid])) * kLn2;
            if (item.part >= 0) {
                a.part_lse[(long long)item.part * pitch + r0 + tid] = lse;
            } else if (a.lse) {
                const long long tok = ch.tok0 + row / group, head = item.band * group + row % group;
                a.lse[tok * a.q_heads + head] = lse;
            }
        }
    }
    __syncthreads();
}

}  // namespace
}  // namespace leyline
