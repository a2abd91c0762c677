// leyline_select.cu -- the rows a request keeps, by their weights (sm_103a).
//
// Of the rows [first, len - last) the m = n_keep - first - last of greatest weight, equal weights from the lowest row
// up, and the rows at both ends: an ascending list.  Weights are compared as numbers: -0 equals 0, a NaN lies below
// everything.
//
// Weights become 32-bit keys in their order.  The m-th greatest key is found by its digits of 8 bits, from the top: a histogram of the
// digit over the rows that share the digits found so far, and a sum over its bins from the greatest down.  A cluster of CTAs
// takes a request, each of them a run of its rows, which a thread holds in registers, 16 in a row; the histograms meet
// through distributed shared memory, and the CTAs' counts of rows taken give each the place of its part of the list.
//
// What bounds it is latency, the barriers of up to four digits and of the list: one request of 4096 rows 8 us, 16 of some
// 30000 rows 23, 8 of 131072 rows 32, where a pass over the weights takes 0.6.  From 4 rows a thread on a request gets more
// CTAs.
#include <cooperative_groups.h>

#include "leyline_device.cuh"
#include "leyline_evict.h"

namespace leyline {
namespace {

namespace cg = cooperative_groups;

// Keys in the order of the weights: 0 for a NaN, one key for both zeros.
__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w) return 0;
    const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kHeld = 16;  // rows of a thread
constexpr int kSegment = kSelectThreads * kHeld;
constexpr int kMostCtas = 8;  // of a cluster
constexpr int kBins = 256;    // digits of 8 bits
constexpr int kDigits = 4;

struct SelectShared {
    alignas(16) uint32_t bins[kDigits][kBins];
    alignas(16) uint32_t total[kBins];  // over the cluster
    uint32_t scratch[33];
    uint32_t found[3];  // digit, rows of greater ones, rows of this one
    uint2 taken;  // rows above the m-th greatest key, and of that key, of this CTA
};

// *p if `on`, else NaN.  Without a branch: behind one a load waited for the one before it to be used.
__device__ __forceinline__ float load_if(bool on, const float* p)
{
    float x = __int_as_float(0x7fffffff);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.f32 %0, [%1];\n\t}" : "+f"(x) : "l"(p), "r"((uint32_t)on) : "memory");
    return x;
}

// Inclusive sum of x over the CTA's threads; scratch[31] holds the total afterwards.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();  // scratch is free
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = scratch[lane];
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        scratch[lane] = s;
    }
    __syncthreads();
    return x + (warp > 0 ? scratch[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectArgs a,
                                                                const __grid_constant__ EvictSet set)
{
    __shared__ SelectShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ctas = cluster.num_blocks(), tid = threadIdx.x;
    const EvictReq& r = set.req[blockIdx.x / ctas];
    const float* w = a.weights + r.req * a.req_stride + r.first;
    int32_t* kept = a.kept + (long long)r.list * a.kept_stride;
    const int rows = r.len - r.last - r.first, m = r.n_keep - r.first - r.last;
    // this CTA's rows [begin, end) of them, a thread's 16 (or as many as give every thread some) in a row
    const int per = (rows + ctas - 1) / ctas, begin = min(rows, rank * per), end = min(rows, begin + per);
    const int segments = (per + kSegment - 1) / kSegment;
    const int held = segments > 1 ? kHeld : (per + kSelectThreads - 1) / kSelectThreads;
    (&s.bins[0][0])[tid] = 0;
    static_assert(kDigits * kBins == kSelectThreads, "a bin for each thread");
    wait_for_previous_grid();
    allow_next_grid();
    uint32_t key[kHeld];
    auto load = [&](int segment) {
        const int at = begin + segment * kSegment + tid * held;
        float x[kHeld];
#pragma unroll
        for (int k = 0; k < kHeld; ++k) x[k] = load_if(k < held && at + k < end, w + at + k);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) key[k] = order_key(x[k]);
    };
    auto count = [&](int segment) { return max(0, min(held, end - begin - segment * kSegment - tid * held)); };
    load(0);
    __syncthreads();
    uint32_t prefix = 0, mask = 0;
    uint32_t want = m;  // rows still to be taken among those that share the prefix
    for (int d = 0; d < kDigits && m > 0; ++d) {
        const int shift = 24 - 8 * d;
        for (int g = 0; g < segments; ++g) {
            if (segments > 1) load(g);
            const int n = count(g);
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                if (k >= held) break;
                const bool on = k < n && (key[k] & mask) == prefix;
                const uint32_t bin = on ? key[k] >> shift & 255u : kBins;
                if (d == 0) {
                    // the first digits of most weights are few: one count for the lanes that share a bin, where an atomic of
                    // each of them took turns
                    const unsigned same = __match_any_sync(0xffffffffu, bin);
                    if (on && (same & ((1u << (tid & 31)) - 1)) == 0) atomicAdd(&s.bins[0][bin], __popc(same));
                } else if (on) {
                    atomicAdd(&s.bins[d][bin], 1u);
                }
            }
        }
        const uint32_t* sums = s.bins[d];
        if (ctas > 1) {
            cluster.sync();
            if (tid < kBins) {  // (a lane's 8 bins of each CTA in turn, by the warp below, took a round trip for each CTA)
                uint32_t x[kMostCtas], all = 0;
#pragma unroll
                for (int c = 0; c < kMostCtas; ++c) x[c] = *cluster.map_shared_rank(&s.bins[d][tid], c < ctas ? c : 0);
#pragma unroll
                for (int c = 0; c < kMostCtas; ++c) all += c < ctas ? x[c] : 0;
                s.total[tid] = all;
            }
            sums = s.total;
        }
        __syncthreads();
        if (tid < 32) {  // 8 bins a lane from the greatest down
            const int first = kBins - 8 - 8 * tid;
            const uint4 x = *reinterpret_cast<const uint4*>(sums + first), y = *reinterpret_cast<const uint4*>(sums + first + 4);
            const uint32_t bin[8] = {y.w, y.z, y.y, y.x, x.w, x.z, x.y, x.x};
            uint32_t mine = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) mine += bin[k];
            uint32_t upto = mine;
            for (int e = 1; e < 32; e *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, e);
                if (tid >= e) upto += x;
            }
            uint32_t before = upto - mine;
            if (before < want && upto >= want) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (before < want && before + bin[k] >= want) {
                        s.found[0] = first + 7 - k;
                        s.found[1] = before;
                        s.found[2] = bin[k];
                    }
                    before += bin[k];
                }
            }
        }
        __syncthreads();
        prefix |= s.found[0] << shift;
        mask |= 255u << shift;
        want -= s.found[1];
        if (s.found[2] == want) break;  // all rows of these digits are taken
        __syncthreads();
    }
    // `want` of the rows with the digits of the m-th greatest, the lowest ones, and all above them
    uint32_t above = 0, equal = 0;
    for (int g = 0; g < segments && m > 0; ++g) {
        if (segments > 1) load(g);
        const int n = count(g);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            above += k < n && (key[k] & mask) > prefix;
            equal += k < n && (key[k] & mask) == prefix;
        }
    }
    if (segments > 1) {  // (totals of the CTA; each segment's are found again below)
        block_scan(above, s.scratch);
        const uint32_t all = s.scratch[31];
        block_scan(equal, s.scratch);
        if (tid == 0) s.taken = make_uint2(all, s.scratch[31]);
    } else {
        const uint32_t both = block_scan(above << 16 | equal, s.scratch);  // (16384 rows of a CTA at most)
        if (tid == 0) s.taken = make_uint2(s.scratch[31] >> 16, s.scratch[31] & 0xffff);
        above = (both >> 16) - above;
        equal = (both & 0xffff) - equal;
    }
    uint32_t above0 = 0, equal0 = 0;  // of the CTAs before
    if (ctas > 1) {
        cluster.sync();
        uint2 x[kMostCtas - 1];
#pragma unroll
        for (int c = 0; c < kMostCtas - 1; ++c) x[c] = *cluster.map_shared_rank(&s.taken, c < rank ? c : rank);
#pragma unroll
        for (int c = 0; c < kMostCtas - 1; ++c) {
            above0 += c < rank ? x[c].x : 0;
            equal0 += c < rank ? x[c].y : 0;
        }
    }
    for (int g = 0; g < segments && m > 0; ++g) {
        const int n = count(g);
        if (segments > 1) {
            load(g);
            uint32_t x = 0, y = 0;
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                x += k < n && (key[k] & mask) > prefix;
                y += k < n && (key[k] & mask) == prefix;
            }
            const uint32_t both = block_scan(x << 16 | y, s.scratch), all = s.scratch[31];
            above = above0 + (both >> 16) - x;
            equal = equal0 + (both & 0xffff) - y;
            above0 += all >> 16;
            equal0 += all & 0xffff;
        } else {
            above += above0;
            equal += equal0;
        }
        const int at = r.first + begin + g * kSegment + tid * held;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            if (k >= n) break;
            const bool is_above = (key[k] & mask) > prefix, is_equal = (key[k] & mask) == prefix;
            if (is_above || (is_equal && equal < want)) kept[r.first + above + min(equal, want)] = at + k;
            above += is_above;
            equal += is_equal;
        }
    }
    for (int i = rank * kSelectThreads + tid; i < r.first; i += ctas * kSelectThreads) kept[i] = i;
    for (int i = rank * kSelectThreads + tid; i < r.last; i += ctas * kSelectThreads) kept[r.n_keep - r.last + i] = r.len - r.last + i;
    if (ctas > 1) cluster.sync();  // no CTA leaves while another may read its counts
}

}  // namespace

int launch_select(const SelectArgs& a, const EvictSet& set, void* stream)
{
    int longest = 0;
    for (int k = 0; k < set.n; ++k) longest = std::max(longest, set.req[k].len);
    // CTAs of a request: as few as leave a thread no more than 4 rows
    int ctas = 1;
    while (ctas < kMostCtas && longest > 4 * kSelectThreads * ctas) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(set.n * ctas));
    cfg.blockDim = dim3((unsigned)kSelectThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, select_kernel, a, set);
}

}  // namespace leyline
