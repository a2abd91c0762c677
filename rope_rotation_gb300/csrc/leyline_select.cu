// leyline_select.cu -- the rows a request keeps, by their weights (sm_103a).
//
// Of the rows [first, len - last) the m = n_keep - first - last of greatest weight, equal weights from the lowest row
// up, and the rows at both ends: an ascending list.  Weights are compared as numbers: -0 equals 0, a NaN lies below
// everything.
//
// Weights become 32-bit keys in their order.  The m-th greatest key is found digit by digit, from the top: a histogram
// of the digit over the rows that share the digits found so far, and a sum over its bins from the greatest down.
#include "leyline_device.cuh"
#include "leyline_evict.h"

namespace leyline {
namespace {

// Keys in the order of the weights: 0 for a NaN, one key for both zeros.
__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w) return 0;
    const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024;

// Exclusive sum of x over the CTA's threads, and the total; scratch: 33 words.
__device__ __forceinline__ int block_scan(int x, int* scratch, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int incl = x;
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();  // scratch is free
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int s = lane < kSelectThreads / 32 ? scratch[lane] : 0;
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        scratch[lane] = s;
    }
    __syncthreads();
    total = scratch[kSelectThreads / 32 - 1];
    return incl - x + (warp > 0 ? scratch[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectArgs a,
                                                                const __grid_constant__ EvictSet set)
{
    __shared__ int bins[256];
    __shared__ int scratch[33];
    __shared__ int found[2];
    wait_for_previous_grid();
    allow_next_grid();
    const EvictReq r = set.req[blockIdx.x];
    const float* w = a.weights + r.req * a.req_stride;
    int32_t* kept = a.kept + (long long)r.list * a.kept_stride;
    const int tid = threadIdx.x, end = r.len - r.last, m = r.n_keep - r.first - r.last;
    uint32_t prefix = 0, mask = 0;
    int want = m;  // rows still to be taken among those that share the prefix
    for (int shift = 24; shift >= 0 && m > 0; shift -= 8) {
        if (tid < 256) bins[tid] = 0;
        __syncthreads();
        for (int i = r.first + tid; i < end; i += kSelectThreads) {
            const uint32_t k = order_key(w[i]);
            if ((k & mask) == prefix) atomicAdd(&bins[k >> shift & 255], 1);
        }
        __syncthreads();
        int total;
        const int mine = tid < 256 ? bins[255 - tid] : 0;
        const int above = block_scan(mine, scratch, total);
        if (tid < 256 && above < want && above + mine >= want) {
            found[0] = 255 - tid;
            found[1] = above;
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= 255u << shift;
        want -= found[1];
        __syncthreads();
    }
    // `want` of the rows whose key is the m-th greatest, and all above it
    for (int i = tid; i < r.first; i += kSelectThreads) kept[i] = i;
    int taken = r.first, equal = 0;
    for (int i0 = r.first; i0 < end && m > 0; i0 += kSelectThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < end ? order_key(w[i]) : 0;
        const bool eq = i < end && k == prefix;
        int n_eq, n_take;
        const int before = block_scan(eq, scratch, n_eq);
        const bool take = i < end && (k > prefix || (eq && equal + before < want));
        const int at = block_scan(take, scratch, n_take);
        if (take) kept[taken + at] = i;
        taken += n_take;
        equal += n_eq;
    }
    for (int i = tid; i < r.last; i += kSelectThreads) kept[r.n_keep - r.last + i] = end + i;
}

}  // namespace

int launch_select(const SelectArgs& a, const EvictSet& set, void* stream)
{
    return (int)launch_dependent(select_kernel, set.n, kSelectThreads, (cudaStream_t)stream, a, set);
}

}  // namespace leyline
