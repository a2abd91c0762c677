// leyline_append.cu -- the elementwise side of a batch of new tokens (sm_103a): installing a
// plan, appending rows to the cache and turning queries.
//
// "Leyline: KV Cache Directives for Agentic Inference", section 2.3: prefill writes the rows of
// R into new slots, encoded at their final positions; section 2.2: the RoPE band of position p is
// R(p) applied to the position-free band.
//
// All three kernels are bound by memory (or, for a few tokens, by one launch): a row or a
// band is read once, kept in registers while its norm's sum is formed, and written once.  Calls back to back: append of one
// row 6 us and of 8192 MLA rows 7 (2.7 TB/s, in L2; 10 from a cold start), the host's time of a call; rotate of 4096 x 128
// bands of 64 25 us (5.4 TB/s, 0.80 of measured copies).  A plan of 8192 tokens installs in 21 us, once a step, most of it
// the fp64 sines.
#include "leyline_batch.h"
#include "leyline_device.cuh"

namespace leyline {
namespace {

// ----------------------------------------------------------------- install --
// One CTA per run of up to kPlanRun tokens of a chunk, and CTAs that copy the plan from the
// pinned staging buffer.  cos and sin of position * theta_j are formed in fp64 and rounded
// once to the rotation's arithmetic, as the host does for a splice's turns.
constexpr int kInstallThreads = 256;

__global__ void __launch_bounds__(kInstallThreads) install_plan_kernel(const __grid_constant__ InstallArgs a)
{
    wait_for_previous_grid();
    allow_next_grid();
    if ((int)blockIdx.x >= a.n_runs) {
        const long long ctas = gridDim.x - a.n_runs;
        for (long long i = (blockIdx.x - a.n_runs) * (long long)blockDim.x + threadIdx.x; i < a.plan_vecs;
             i += ctas * blockDim.x)
            a.plan[i] = a.staged[i];
        return;
    }
    const PlanRun r = a.runs[blockIdx.x];
    const Geometry& g = a.g;
    const long long B = g.block_size;
    if (threadIdx.x < r.n) {
        const long long row = r.start + threadIdx.x;
        const long long blk = row / B;
        int32_t* entry = a.table + (long long)r.req * a.max_blocks + blk;
        const bool fresh = blk >= r.old_blocks;
        const int page = fresh ? a.free_q[ring(r.pop + (blk - r.old_blocks), a.q_cap)] : *entry;
        long long slot = -1;
        if (page < 0 || page >= g.num_pages) {
            raise_status(a.status, fresh ? ST_BAD_FRESH : ST_BAD_PAGE);
        } else {
            slot = (long long)page * B + (row - blk * B);
            // a fresh block's first row is a row of this chunk: its token installs the page
            if (fresh && row == blk * B) *entry = page;
            if (a.pending) a.pending[slot] = 0;
        }
        a.slot[r.tok0 + threadIdx.x] = slot;
    }
    if (threadIdx.x == 0 && r.new_len >= 0) a.seq_lens_dev[r.req] = (int32_t)r.new_len;
    const int half = g.rope_dim / 2;
    for (int i = threadIdx.x; i < r.n * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        double s, c;
        sincos((double)(r.rope_start + t) * a.theta[j], &s, &c);
        float2 v = make_float2((float)c, (float)s);
        if (g.precision == LEYLINE_ROTATE_BF16_NAIVE)
            v = make_float2(__bfloat162float(__double2bfloat16(c)), __bfloat162float(__double2bfloat16(s)));
        a.trig[(long long)(r.tok0 + t) * half + j] = v;
    }
}

// ------------------------------------------------------------------- bands --
// A lane holds 8 pairs of a band, pairs 8q .. 8q + 7, as two 16-byte vectors: half-split the
// vectors q and q + head_vecs / 2 (x and y), interleaved 2q and 2q + 1.
template <int kLayout>
__device__ __forceinline__ void band_vecs(int q, int hv, int& v0, int& v1)
{
    v0 = kLayout == 0 ? q : 2 * q;
    v1 = kLayout == 0 ? q + hv / 2 : 2 * q + 1;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f)
{
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float* f)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float sum_squares(const uint4& v)
{
    float f[8], s = 0.f;
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
    return s;
}

// Scale by inv and the weights: x * inv * w.
__device__ __forceinline__ void norm8(float* f, float inv, const uint4& weight)
{
    float w[8];
    unpack8(weight, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
}

// Norm (inv > 0: by inv and the weights w0, w1) and turn the 8 pairs of (a, b) by trig[8q ..].
template <int kLayout>
__device__ __forceinline__ void encode_pairs(uint4& a, uint4& b, bool normed, float inv, const uint4& w0,
                                             const uint4& w1, const float2* trig, bool bf16)
{
    float x[8], y[8];
    unpack8(a, x);
    unpack8(b, y);
    if (normed) {
        norm8(x, inv, w0);
        norm8(y, inv, w1);
    }
    const float4* t4 = reinterpret_cast<const float4*>(trig);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = t4[i];
        c[2 * i] = t.x;
        s[2 * i] = t.y;
        c[2 * i + 1] = t.z;
        s[2 * i + 1] = t.w;
    }
    float* f[2] = {x, y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // pair i: half-split (x[i], y[i]); interleaved elements 2i, 2i + 1 of x then y
        float& p = kLayout == 0 ? x[i] : f[i / 4][2 * (i % 4)];
        float& r = kLayout == 0 ? y[i] : f[i / 4][2 * (i % 4) + 1];
        float po, ro;
        if (bf16) turn_bf16(round_bf16(p), round_bf16(r), c[i], s[i], po, ro);
        else turn_fp32(p, r, c[i], s[i], po, ro);
        p = po;
        r = ro;
    }
    a = pack8(x);
    b = pack8(y);
}

// Lanes that hold one band: head_vecs / 2 of a power-of-two group.
__device__ __forceinline__ int band_group(int hv)
{
    int w = 1;
    while (w < hv / 2) w *= 2;
    return w;  // <= 16: rope_dim <= 256
}

__device__ __forceinline__ float group_sum(float v, int width)
{
    for (int m = width / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// ------------------------------------------------------------------ append --
// A warp per token: the latent's vectors lie in its lanes' registers while the norm's sum is
// formed; then the bands, 32 / group of them at a time.
constexpr int kAppendThreads = 128;
constexpr int kLatentVecsPerLane = kAttnMaxValue / 8 / 32;

template <int kLayout>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a)
{
    wait_for_previous_grid();
    allow_next_grid();
    const Geometry& g = a.g;
    const int lane = threadIdx.x & 31;
    const bool bf16 = g.precision == LEYLINE_ROTATE_BF16_NAIVE;
    const int lv = g.latent_vecs, hv = g.head_vecs, half = g.rope_dim / 2;
    const int width = band_group(hv);
    const int q = lane % width;
    const long long n = a.header->n_tokens;
    const long long warps = (long long)gridDim.x * (kAppendThreads / 32);
    for (long long t = blockIdx.x * (long long)(kAppendThreads / 32) + threadIdx.x / 32; t < n; t += warps) {
        const long long slot = a.slot[t];
        if (slot < 0) continue;  // a bad page, recorded when the plan was installed
        const uint4* src = a.rows + t * a.row_stride;
        uint4* dst = a.kv + lat_off(g, a.layer, slot);
        uint4 v[kLatentVecsPerLane];
#pragma unroll
        for (int k = 0; k < kLatentVecsPerLane; ++k)
            if (lane + 32 * k < lv) v[k] = src[lane + 32 * k];
        if (a.latent_norm) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kLatentVecsPerLane; ++k)
                if (lane + 32 * k < lv) s += sum_squares(v[k]);
            s = group_sum(s, 32);
            const float inv = rsqrtf(s / (float)g.latent_dim + a.eps);
#pragma unroll
            for (int k = 0; k < kLatentVecsPerLane; ++k)
                if (lane + 32 * k < lv) {
                    float f[8];
                    unpack8(v[k], f);
                    norm8(f, inv, a.latent_norm[lane + 32 * k]);
                    v[k] = pack8(f);
                }
        }
#pragma unroll
        for (int k = 0; k < kLatentVecsPerLane; ++k)
            if (lane + 32 * k < lv) dst[lane + 32 * k] = v[k];
        const uint4* bands = src + lv;
        uint4* dbands = a.kv + band_off(g, a.layer, slot);
        int v0, v1;
        band_vecs<kLayout>(q, hv, v0, v1);
        for (int h0 = 0; h0 < g.rope_heads; h0 += 32 / width) {
            const int h = h0 + lane / width;
            const bool on = h < g.rope_heads && q < hv / 2;
            uint4 x = {}, y = {}, w0 = {}, w1 = {};
            if (on) {
                x = bands[h * hv + v0];
                y = bands[h * hv + v1];
            }
            float inv = 0.f;
            if (a.key_norm) {
                const float s = group_sum(sum_squares(x) + sum_squares(y), width);
                inv = rsqrtf(s / (float)g.rope_dim + a.eps);
                if (on) {
                    w0 = a.key_norm[v0];
                    w1 = a.key_norm[v1];
                }
            }
            if (on) {
                encode_pairs<kLayout>(x, y, a.key_norm != nullptr, inv, w0, w1, a.trig + t * half + 8 * q, bf16);
                dbands[h * hv + v0] = x;
                dbands[h * hv + v1] = y;
            }
        }
    }
}

// ------------------------------------------------------------------ rotate --
// A lane has two bands in flight: 32 KB on each SM with one, too little for the latency of memory (4096 tokens of 128
// bands of 64: 28 us with one, 25 with two at the same 32 warps per SM, 28 with four; 26 with one at 64 warps).
constexpr int kAtOnce = 2;

template <int kLayout>
__global__ void __launch_bounds__(kAppendThreads) rotate_kernel(const __grid_constant__ RotateArgs a)
{
    wait_for_previous_grid();
    allow_next_grid();
    const Geometry& g = a.g;
    const int lane = threadIdx.x & 31;
    const bool bf16 = g.precision == LEYLINE_ROTATE_BF16_NAIVE;
    const int hv = g.head_vecs, half = g.rope_dim / 2;
    const int width = band_group(hv);
    const int q = lane % width;
    int v0, v1;
    band_vecs<kLayout>(q, hv, v0, v1);
    const long long bands = (long long)a.header->n_tokens * a.q_heads;
    const long long per = 32 / width;  // bands of a warp at a time
    const long long warps = (long long)gridDim.x * (kAppendThreads / 32);
    for (long long b0 = (blockIdx.x * (long long)(kAppendThreads / 32) + threadIdx.x / 32) * per * kAtOnce; b0 < bands;
         b0 += warps * per * kAtOnce) {
        uint4 x[kAtOnce], y[kAtOnce];
        long long t[kAtOnce], h[kAtOnce];
        bool on[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const long long b = b0 + k * per + lane / width;
            on[k] = b < bands && q < hv / 2;
            t[k] = (unsigned)b / (unsigned)a.q_heads;  // bands <= 2^32
            h[k] = b - t[k] * a.q_heads;
            const uint4* src = static_cast<const uint4*>(a.q.ptr) + (t[k] * a.q.token_stride + h[k] * a.q.head_stride) / 8;
            x[k] = y[k] = make_uint4(0, 0, 0, 0);
            if (on[k]) {
                x[k] = src[v0];
                y[k] = src[v1];
            }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            uint4 w0 = {}, w1 = {};
            float inv = 0.f;
            if (a.norm) {
                const float s = group_sum(sum_squares(x[k]) + sum_squares(y[k]), width);
                inv = rsqrtf(s / (float)g.rope_dim + a.eps);
                if (on[k]) {
                    w0 = a.norm[v0];
                    w1 = a.norm[v1];
                }
            }
            if (on[k]) {
                uint4* dst = static_cast<uint4*>(a.out.ptr) + (t[k] * a.out.token_stride + h[k] * a.out.head_stride) / 8;
                encode_pairs<kLayout>(x[k], y[k], a.norm != nullptr, inv, w0, w1, a.trig + t[k] * half + 8 * q, bf16);
                dst[v0] = x[k];
                dst[v1] = y[k];
            }
        }
    }
}

}  // namespace

int launch_install(const InstallArgs& a, void* stream)
{
    const int copy = grid_for(a.plan_vecs, kInstallThreads, 64);
    return (int)launch_dependent(install_plan_kernel, a.n_runs + copy, kInstallThreads, (cudaStream_t)stream, a);
}

int launch_append(const AppendArgs& a, int64_t tokens, int sm_count, void* stream)
{
    const int grid = grid_for(tokens, kAppendThreads / 32, sm_count * 8);
    return (int)(a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT
                     ? launch_dependent(append_kernel<0>, grid, kAppendThreads, (cudaStream_t)stream, a)
                     : launch_dependent(append_kernel<1>, grid, kAppendThreads, (cudaStream_t)stream, a));
}

int launch_rotate(const RotateArgs& a, int64_t tokens, int sm_count, void* stream)
{
    const int grid = grid_for((tokens * a.q_heads * (a.g.rope_dim / 16) + kAtOnce - 1) / kAtOnce, kAppendThreads, sm_count * 8);
    return (int)(a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT
                     ? launch_dependent(rotate_kernel<0>, grid, kAppendThreads, (cudaStream_t)stream, a)
                     : launch_dependent(rotate_kernel<1>, grid, kAppendThreads, (cudaStream_t)stream, a));
}

}  // namespace leyline
