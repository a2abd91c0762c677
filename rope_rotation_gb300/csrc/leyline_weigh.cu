// leyline_weigh.cu -- the weight that a batch's queries give to each cache row (sm_103a): the kernel for any row shape.
//
// Row s of a request gets, over the plan's tokens t of that request that attend to it and their heads h,
//   w_s <- decay * w_s + sum exp(scale * <q_th, k_s> - lse_th),
// its column sum of the softmax's weights, whose normaliser lse is known by now: no maximum is needed.  A query row with
// lse -inf attends to nothing and adds nothing.
//
// A warp takes a cache row, whose key lies in its lanes' registers, and meets the query rows one after another, so the
// sum has one order.  The products on the CUDA cores bound it: one token each of 16 requests over 4000 rows takes 640 us with
// 8 bands of 96 and 32 heads, 445 with 16 heads over latents of 448 and a band of 96 (and 22 on the tensor cores with 512 + 64).
#include "leyline_attention_any.cuh"

namespace leyline {
namespace {

constexpr int kWeighThreads = 128;
constexpr int kKeyVecs = (kAttnMaxValue + kAttnMaxRope) / 8;
constexpr int kLaneVecs = kKeyVecs / 32;
constexpr int kAtOnce = 2;  // query rows in flight

__global__ void __launch_bounds__(kWeighThreads) weigh_any_kernel(const __grid_constant__ WeighArgs a)
{
    __shared__ float key_s[kWeighThreads / 32][8 * kKeyVecs];
    wait_for_previous_grid();
    allow_next_grid();
    const Geometry& g = a.g;
    const int lane = threadIdx.x & 31;
    float* key = key_s[threadIdx.x / 32];
    const bool mla = g.rope_heads <= 1, bf16 = g.precision == LEYLINE_ROTATE_BF16_NAIVE;
    const int bands = mla ? 1 : g.rope_heads, group = a.q_heads / bands;
    const int lat = mla ? g.latent_vecs : 0, vecs = lat + g.head_vecs, half = g.rope_dim / 2;
    const float scale2 = a.scale * kLog2e;
    const long long warps = (long long)gridDim.x * (kWeighThreads / 32), work = a.header->weigh_work;
    const int n_reqs = a.header->weigh_reqs;
    for (long long x = blockIdx.x * (long long)(kWeighThreads / 32) + threadIdx.x / 32; x < work; x += warps) {
        int lo = 0, hi = n_reqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.reqs[mid].begin <= x) lo = mid;
            else hi = mid - 1;
        }
        const WeighReq r = a.reqs[lo];
        if (r.req >= a.num_reqs || r.end > a.rows) {  // (a replayed plan)
            raise_status(a.status, ST_BAD_ROW);
            continue;
        }
        const long long row = x - r.begin;
        const long long slot = row_slot(a.header->table + (long long)r.req * a.header->max_blocks, g, row, a.status);
        if (slot < 0) continue;
        float sum = 0.f;
        for (int b = 0; b < bands; ++b) {
            __syncwarp();
            for (int c = lane; c < vecs; c += 32) {
                const uint4 v = c < lat ? a.kv[lat_off(g, a.layer, slot) + c]
                                        : a.kv[band_off(g, a.layer, slot) + b * g.head_vecs + (c - lat)];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    key[8 * c + 2 * e] = bf16_lo(w[e]);
                    key[8 * c + 2 * e + 1] = bf16_hi(w[e]);
                }
            }
            __syncwarp();
            const int pend = a.pending ? a.pending[slot] : 0;
            if (pend != 0) {
                float* band = key + 8 * lat;
                const bool split = g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
                for (int j = lane; j < half; j += 32) {
                    float& p = band[split ? j : 2 * j];
                    float& q = band[split ? j + half : 2 * j + 1];
                    float c, s, y0, y1;
                    pending_trig(pend, a.turn, half, j, bf16, c, s);
                    if (bf16) turn_bf16(p, q, c, s, y0, y1);
                    else turn_fp32(p, q, c, s, y0, y1);
                    p = bf16 ? round_bf16(y0) : y0;
                    q = bf16 ? round_bf16(y1) : y1;
                }
                __syncwarp();
            }
            float k[kLaneVecs][8];
#pragma unroll
            for (int i = 0; i < kLaneVecs; ++i)
                if (lane + 32 * i < vecs)
#pragma unroll
                    for (int e = 0; e < 8; ++e) k[i][e] = key[8 * (lane + 32 * i) + e];
            for (int at = r.chunk; at >= 0; at = a.chunks[at].next) {
                const ChunkDev ch = a.chunks[at];
                if (a.prefix && row >= ch.start) continue;
                const long long first = a.prefix ? 0 : max(0ll, row - (long long)ch.start);  // token that attends to the row
                const long long q_end = (long long)ch.n * group;
                for (long long q0 = first * group; q0 < q_end; q0 += kAtOnce) {
                    float dot[kAtOnce], norm[kAtOnce];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        dot[u] = 0.f;
                        norm[u] = -INFINITY;
                        if (q0 + u >= q_end) continue;
                        const long long tok = ch.tok0 + (q0 + u) / group, head = b * group + (q0 + u) % group;
                        norm[u] = a.lse[tok * a.q_heads + head];
                        const uint4* ql = static_cast<const uint4*>(a.q_latent.ptr) +
                                          (tok * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8;
                        const uint4* qr = static_cast<const uint4*>(a.q_rope.ptr) +
                                          (tok * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8;
#pragma unroll
                        for (int i = 0; i < kLaneVecs; ++i) {
                            const int c = lane + 32 * i;
                            if (c >= vecs) continue;
                            const uint4 v = c < lat ? ql[c] : qr[c - lat];
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                dot[u] = fmaf(bf16_lo(w[e]), k[i][2 * e], dot[u]);
                                dot[u] = fmaf(bf16_hi(w[e]), k[i][2 * e + 1], dot[u]);
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        for (int m = 16; m > 0; m /= 2) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], m);
                        if (norm[u] != -INFINITY) sum += exp2f(fmaf(dot[u], scale2, -norm[u] * kLog2e));
                    }
                }
            }
        }
        if (lane == 0) {
            float* w = a.weights + r.req * a.req_stride + row;
            *w = a.decay == 0.f ? sum : fmaf(a.decay, *w, sum);
        }
    }
}

}  // namespace

int launch_weigh(const WeighArgs& a, int sm_count, void* stream)
{
    return (int)launch_dependent(weigh_any_kernel, sm_count * 8, kWeighThreads, (cudaStream_t)stream, a);
}

}  // namespace leyline
