// leyline_evict_rows.cu -- dropping the rows of a request that a list does not keep (sm_103a).
//
// Row i of the edited request is row kept[i] of the one before, in every layer; its bands stay at the positions they
// were encoded at ("Leyline: KV Cache Directives for Agentic Inference" has this as the compaction of the KV-streams
// page: evict without resetting positions), its pending turn and its weight move with it.
//
// One row a page: the rows stay where they are and their table entries move.  Else rows move within the request's own
// pages, so that a full pool can be edited: kept[i] >= i, and a CTA that takes the rows in order may write row i once
// it has read row kept[i], since every row it has still to read lies behind.  Such a chain of rows is kept to one CTA
// for each (request, layer, slice of a row's columns), and the chains run side by side.
//
// What bounds it is HBM with pieces of 128 bytes: half of 32768 rows of 27 layers kept in 176 us for one request and 686 for
// four, 90% of 16 requests of some 10000 rows of 4 layers, lazy, in 237 (0.86, 0.88 and 0.84 of the measured copy rate, with
// the two small kernels around it).  With few layers it is a chain's latency, 1.4 us a batch of rows whatever its size: one
// layer of the first 100 us.  Slices of 64 bytes then take 10% less, but 30% more in 27 layers, and so do 256 bytes.  One row
// a page, 16 requests of some 30000 rows: 17 us, the latency of two kernels.
#include "leyline_device.cuh"
#include "leyline_evict.h"

namespace leyline {
namespace {

// ------------------------------------------------------------------- stage --
__device__ __forceinline__ int page_at(const EvictArgs& a, const EvictReq& r, int blk)
{
    const int page = a.table[(long long)r.req * a.max_blocks + blk];
    if (page >= 0 && page < a.g.num_pages) return page;
    raise_status(a.status, ST_BAD_PAGE);
    return -1;
}

// The request of block `block` of kStageRows rows.
__device__ __forceinline__ int req_of(const EvictSet& set, int block)
{
    int lo = 0, hi = set.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (set.req[mid].block_begin <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The first of kept[0, n) that is not below `row`, by a warp: each step asks for 32 places at once.
__device__ __forceinline__ int lower_bound(const int32_t* kept, int n, int row)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;  // what is below lo is below row, from hi on it is not
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && kept[at] < row);
        const int count = below == 0 ? 0 : 32 - __clz(below);  // (of a list that does not ascend: any of them)
        if (count == 0) return lo;
        lo += (count - 1) * step + 1;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// A CTA for each kStageRows rows before the call.  The request's list is checked: whether it ascends within [0, len), and
// where its first row is that moves.  What moves of a kept row beside its rows goes to the staging arrays, and with one row a
// page a dropped row's page to the ring.  Nothing else is changed: after a bad list the commit does without all of it.
__global__ void __launch_bounds__(kStageRows) stage_kernel(const __grid_constant__ EvictArgs a,
                                                           const __grid_constant__ EvictSet set)
{
    __shared__ int mark[kStageRows], bounds[2], before[kStageRows / 32], hole;
    wait_for_previous_grid();
    allow_next_grid();
    const int q = req_of(set, blockIdx.x), tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const EvictReq& r = set.req[q];
    const int32_t* kept = a.kept + (long long)r.list * a.kept_stride;
    const int row0 = (blockIdx.x - r.block_begin) * kStageRows, row = row0 + tid, B = a.g.block_size;
    // this row's entry of the list
    const int k = row < r.n_keep ? kept[row] : 0, last = row > 0 && row < r.n_keep ? kept[row - 1] : -1;
    const bool bad = row < r.n_keep && (k < 0 || k >= r.len || last >= k);
    if (tid == 0) hole = r.n_keep;
    mark[tid] = -1;
    if (B == 1 && warp < 2) {
        const int bound = lower_bound(kept, r.n_keep, row0 + warp * kStageRows);
        if (lane == 0) bounds[warp] = bound;
    }
    __syncthreads();
    if (row < r.n_keep && k != row) atomicMin(&hole, row);
    if (B == 1) {
        const int at = bounds[0] + tid;
        if (at < bounds[1]) {
            const int place = kept[at] - row0;
            if (place >= 0 && place < kStageRows) mark[place] = at;
        }
    }
    const bool any_bad = __syncthreads_or(bad);
    if (tid == 0) {
        if (any_bad) atomicOr(&a.state[q].bad, 1);
        if (hole < r.n_keep) atomicMin(&a.state[q].hole, hole);
    }
    if (B > 1) {
        if (row >= r.n_keep || bad) return;
        if (a.weights) a.stage_w[r.stage + row] = a.weights[r.req * a.req_stride + k];
        if (a.pending) {
            const int blk = k / B, page = page_at(a, r, blk);
            a.stage_i[r.stage + row] = page < 0 ? 0 : a.pending[(long long)page * B + (k - blk * B)];
        }
        return;
    }
    const bool on = row < r.len;
    const int at = on ? mark[tid] : -1;
    const unsigned keeps = __ballot_sync(0xffffffffu, at >= 0);
    if (lane == 0) before[warp] = __popc(keeps);
    __syncthreads();
    if (!on) return;
    const int page = a.table[(long long)r.req * a.max_blocks + row];
    if (page < 0 || page >= a.g.num_pages) raise_status(a.status, ST_BAD_PAGE);
    if (at >= 0) {
        a.stage_i[r.stage + at] = page;
        if (a.weights) a.stage_w[r.stage + at] = a.weights[r.req * a.req_stride + row];
        return;
    }
    int kept_before = bounds[0] + __popc(keeps & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) kept_before += before[w];
    const int dropped = row - kept_before;  // (in range for a list that ascends)
    if (dropped >= 0 && dropped < r.len - r.n_keep) a.free_q[ring(r.push + dropped, a.q_cap)] = page;
}

// -------------------------------------------------------------------- move --
constexpr int kChainThreads = 256;
constexpr int kVecs = 8;                  // 16-byte vectors of a thread in a batch
constexpr int kBatchRows = kChainThreads;  // of a batch, at most: a thread looks up one
constexpr int kAhead = 2;                 // batches that are read before one is written
constexpr int kDstLists = 4;
static_assert(kAhead + 2 <= kDstLists, "slots are there from their look-up until they are written");

struct ChainShared {
    uint4 rows[kAhead][kVecs][kChainThreads];  // each thread's own vectors
    long long src[2][kBatchRows], dst[kDstLists][kBatchRows];  // slots of a batch's rows, -1: none
};

// One chain: `slice` vectors of each row of one request in one layer, in batches of as many rows as the CTA's threads
// hold.  Batches are read ahead (cp.async: a barrier waits for plain loads on their way): what a batch writes lies before
// the sources of all later ones.  The barrier between a batch's reads and its writes orders them over the CTA.
__global__ void __launch_bounds__(kChainThreads) move_rows_kernel(const __grid_constant__ EvictArgs a,
                                                                  const __grid_constant__ EvictSet set, int slices,
                                                                  int slice)
{
    extern __shared__ __align__(16) unsigned char smem[];
    ChainShared& sh = *reinterpret_cast<ChainShared*>(smem);
    wait_for_previous_grid();
    allow_next_grid();
    const Geometry& g = a.g;
    const int per_req = g.num_layers * slices;
    const int q = blockIdx.x / per_req, c = blockIdx.x - q * per_req;
    const int layer = c / slices, first = (c - layer * slices) * slice;  // of the row's vectors
    const EvictReq& r = set.req[q];
    const ListState st{a.state[q].bad, a.state[q].bad ? r.n_keep : min(a.state[q].hole, r.n_keep)};
    const int32_t* kept = a.kept + (long long)r.list * a.kept_stride;  // (a bad list moves nothing)
    const int32_t* table = a.table + (long long)r.req * a.max_blocks;
    const int width = min(slice, g.row_vecs - first), B = g.block_size, tid = threadIdx.x;
    const int batch = min(kChainThreads * kVecs / width, kBatchRows);
    const int batches = (r.n_keep - st.hole + batch - 1) / batch;
    // A thread looks up one row of each batch, each step a batch ahead of the next one: its place in the list, the pages of
    // its source and of itself, their slots.
    auto row_of = [&](int b) { return st.hole + b * batch + tid; };
    auto has = [&](int b) { return tid < batch && row_of(b) < r.n_keep; };
    auto ask_source = [&](int b) { return has(b) ? kept[row_of(b)] : 0; };
    auto ask_pages = [&](int b, int k, int& from, int& to) {
        if (!has(b)) return;
        from = table[k / B];
        to = table[row_of(b) / B];
    };
    auto settle = [&](int b, int k, int from_page, int to_page) {
        if (tid >= batch) return;
        long long from = -1, to = -1;
        if (has(b)) {
            if (from_page >= 0 && from_page < g.num_pages && to_page >= 0 && to_page < g.num_pages) {
                from = (long long)from_page * B + k % B;
                to = (long long)to_page * B + row_of(b) % B;
            } else {
                raise_status(a.status, ST_BAD_PAGE);
            }
        }
        sh.src[b & 1][tid] = from;
        sh.dst[b % kDstLists][tid] = to;
    };
    // A thread's vectors: of row `row[k]` of a batch the vector at `base[k]`, `pitch[k]` vectors from one slot to the next.
    int row[kVecs], pitch[kVecs];
    uint4* base[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int e = tid + k * kChainThreads, i = e / width, v = first + e - i * width;
        const bool latent = v < g.latent_vecs;
        row[k] = i < batch ? i : -1;
        base[k] = a.kv + (latent ? lat_off(g, layer, 0) + v : band_off(g, layer, 0) + (v - g.latent_vecs));
        pitch[k] = latent ? g.lat_row_vecs : g.rope_row_vecs;
    }
    auto read = [&](int b) {
        if (b < batches) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const long long from = row[k] >= 0 ? sh.src[b & 1][row[k]] : -1;
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(&sh.rows[b % kAhead][k][tid]);
                if (from >= 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(base[k] + from * pitch[k]) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto write = [&](int b) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const long long to = row[k] >= 0 ? sh.dst[b % kDstLists][row[k]] : -1;
            if (to >= 0) st_stream(base[k] + to * pitch[k], sh.rows[b % kAhead][k][tid]);
        }
    };
    int from, to;
    {  // the look-ups of the first batches side by side (one after another, 188 us for 176 above)
        int ks[kAhead + 1], fs[kAhead + 1], ts[kAhead + 1];
#pragma unroll
        for (int b = 0; b <= kAhead; ++b) ks[b] = ask_source(b);
#pragma unroll
        for (int b = 0; b <= kAhead; ++b) ask_pages(b, ks[b], fs[b], ts[b]);
#pragma unroll
        for (int b = 0; b <= kAhead; ++b) {
            settle(b, ks[b], fs[b], ts[b]);
            __syncthreads();
            if (b < kAhead) read(b);
        }
    }
    int k1 = ask_source(kAhead + 1);
    ask_pages(kAhead + 1, k1, from, to);
    int k2 = ask_source(kAhead + 2);
    for (int b = 0; b < batches; ++b) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        __syncthreads();
        write(b);
        read(b + kAhead);
        settle(b + kAhead + 1, k1, from, to);
        k1 = k2;
        ask_pages(b + kAhead + 2, k1, from, to);
        k2 = ask_source(b + kAhead + 3);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ commit --
__global__ void __launch_bounds__(kStageRows) commit_evict_kernel(const __grid_constant__ EvictArgs a,
                                                                  const __grid_constant__ EvictSet set)
{
    wait_for_previous_grid();
    allow_next_grid();
    if (blockIdx.x == 0 && threadIdx.x < kEvictReqs) a.next_state[threadIdx.x] = ListState{0, INT32_MAX};
    const int q = req_of(set, blockIdx.x), B = a.g.block_size;
    const EvictReq& r = set.req[q];
    const int row = (blockIdx.x - r.block_begin) * kStageRows + threadIdx.x;
    if (row >= r.len) return;
    const bool bad = a.state[q].bad != 0;
    int32_t* table = a.table + (long long)r.req * a.max_blocks;
    if (row == 0) {
        a.seq_lens_dev[r.req] = r.n_keep;
        if (bad) raise_status(a.status, ST_BAD_ROW);
    }
    if (a.weights && (row >= r.n_keep || !bad))
        a.weights[r.req * a.req_stride + row] = row < r.n_keep ? a.stage_w[r.stage + row] : 0.f;
    if (B == 1) {
        if (row >= r.n_keep) {  // of the pages that go back one each: those in the ring, or after a bad list the last ones
            int32_t* back = a.free_q + ring(r.push + (row - r.n_keep), a.q_cap);
            if (bad) *back = table[row];
            const int page = *back;
            if (a.pending && page >= 0 && page < a.g.num_pages) a.pending[page] = 0;
            table[row] = -1;
        } else if (!bad) {
            table[row] = a.stage_i[r.stage + row];
        }
        return;
    }
    const int blk = row / B, keep_blocks = (r.n_keep + B - 1) / B;
    if (row < r.n_keep && a.pending && !bad) {
        const int page = page_at(a, r, blk);
        if (page >= 0) a.pending[(long long)page * B + (row - blk * B)] = a.stage_i[r.stage + row];
    }
    // the first row of a block clears its dropped rows' turns, and gives its page back if all of them are
    if (row != blk * B || (blk + 1) * (long long)B <= r.n_keep) return;
    const int page = page_at(a, r, blk);
    if (a.pending && page >= 0)
        for (int i = max(r.n_keep - row, 0); i < min(B, r.len - row); ++i) a.pending[(long long)page * B + i] = 0;
    if (blk >= keep_blocks) {
        a.free_q[ring(r.push + (blk - keep_blocks), a.q_cap)] = page;
        table[blk] = -1;
    }
}

}  // namespace

int evict_prepare()
{
    return (int)cudaFuncSetAttribute(move_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ChainShared));
}

int launch_evict(const EvictArgs& a, const EvictSet& set, void* stream)
{
    cudaStream_t s = (cudaStream_t)stream;
    const EvictReq& back = set.req[set.n - 1];
    const int blocks = back.block_begin + (back.len + kStageRows - 1) / kStageRows;
    cudaError_t e = launch_dependent(stage_kernel, blocks, kStageRows, s, a, set);
    if (e == cudaSuccess && a.g.block_size > 1) {
        const int slice = 8, slices = (a.g.row_vecs + slice - 1) / slice;
        e = launch_dependent_smem(move_rows_kernel, set.n * a.g.num_layers * slices, kChainThreads, sizeof(ChainShared), s, a, set,
                                  slices, slice);
    }
    if (e == cudaSuccess) e = launch_dependent(commit_evict_kernel, blocks, kStageRows, s, a, set);
    return (int)e;
}

}  // namespace leyline
