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
#include "leyline_device.cuh"
#include "leyline_evict.h"

namespace leyline {
namespace {

constexpr int kCheckThreads = 1024;

// ------------------------------------------------------------------- check --
// One CTA a request: whether its list ascends within [0, len), and the first row that moves.
__global__ void __launch_bounds__(kCheckThreads) check_lists_kernel(const __grid_constant__ EvictArgs a,
                                                                    const __grid_constant__ EvictSet set)
{
    __shared__ int hole;
    wait_for_previous_grid();
    allow_next_grid();
    const EvictReq& r = set.req[blockIdx.x];
    const int32_t* kept = a.kept + (long long)r.list * a.kept_stride;
    if (threadIdx.x == 0) hole = r.n_keep;
    __syncthreads();
    bool bad = false;
    int mine = r.n_keep;
    for (int i = threadIdx.x; i < r.n_keep; i += kCheckThreads) {
        const int k = kept[i];
        bad |= k < 0 || k >= r.len || (i > 0 && kept[i - 1] >= k);
        if (k != i) mine = min(mine, i);
    }
    if (mine < r.n_keep) atomicMin(&hole, mine);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.state[blockIdx.x] = ListState{bad, bad ? r.n_keep : hole};
        if (bad) raise_status(a.status, ST_BAD_ROW);
    }
}

// ------------------------------------------------------------------- stage --
struct List {
    const int32_t* kept;
    bool bad;
    __device__ __forceinline__ int operator[](int i) const { return bad ? i : kept[i]; }
};

__device__ __forceinline__ List list_of(const EvictArgs& a, const EvictReq& r, const ListState& s)
{
    return List{a.kept + (long long)r.list * a.kept_stride, s.bad != 0};
}

// The request of row `row` of the launch's rows.
__device__ __forceinline__ int req_of(const EvictSet& set, long long row)
{
    int lo = 0, hi = set.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (set.req[mid].row_begin <= row) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int page_at(const EvictArgs& a, const EvictReq& r, int blk)
{
    const int page = a.table[(long long)r.req * a.max_blocks + blk];
    if (page >= 0 && page < a.g.num_pages) return page;
    raise_status(a.status, ST_BAD_PAGE);
    return -1;
}

constexpr int kStageThreads = 256;

// A thread for each row before the call: what moves of a kept row beside its rows goes to the staging arrays; with one
// row a page, a dropped row's page goes back.
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const __grid_constant__ EvictArgs a,
                                                              const __grid_constant__ EvictSet set, long long rows)
{
    wait_for_previous_grid();
    allow_next_grid();
    const int B = a.g.block_size;
    for (long long x = blockIdx.x * (long long)kStageThreads + threadIdx.x; x < rows; x += (long long)gridDim.x * kStageThreads) {
        const int q = req_of(set, x);
        const EvictReq& r = set.req[q];
        const List kept = list_of(a, r, a.state[q]);
        const int row = (int)(x - r.row_begin);
        if (B > 1) {
            if (row >= r.n_keep) continue;
            const int from = kept[row];
            if (a.weights) a.stage_w[r.stage + row] = a.weights[r.req * a.req_stride + from];
            if (a.pending) {
                const int blk = from / B, page = page_at(a, r, blk);
                a.stage_i[r.stage + row] = page < 0 ? 0 : a.pending[(long long)page * B + (from - blk * B)];
            }
            continue;
        }
        // kept rows before this one
        int lo = 0, hi = r.n_keep;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (kept[mid] < row) lo = mid + 1;
            else hi = mid;
        }
        const int page = a.table[(long long)r.req * a.max_blocks + row];
        if (lo < r.n_keep && kept[lo] == row) {
            a.stage_i[r.stage + lo] = page;
            if (a.weights) a.stage_w[r.stage + lo] = a.weights[r.req * a.req_stride + row];
            continue;
        }
        a.free_q[ring(r.push + (row - lo), a.q_cap)] = page;
        if (page < 0 || page >= a.g.num_pages) raise_status(a.status, ST_BAD_PAGE);
        else if (a.pending) a.pending[page] = 0;
    }
}

// -------------------------------------------------------------------- move --
constexpr int kChainThreads = 256;
constexpr int kVecs = 8;                  // 16-byte vectors of a thread in a batch
constexpr int kBatchRows = kChainThreads;  // of a batch, at most: a thread looks up one
constexpr int kAhead = 2;                 // batches that are read before one is written
constexpr int kDstLists = 8;
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
    const ListState st = a.state[q];
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
    for (int b = 0; b < kAhead; ++b) {
        const int k = ask_source(b);
        ask_pages(b, k, from, to);
        settle(b, k, from, to);
        __syncthreads();
        read(b);
    }
    {
        const int k = ask_source(kAhead);
        ask_pages(kAhead, k, from, to);
        settle(kAhead, k, from, to);
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
__global__ void __launch_bounds__(kCommitThreads) commit_evict_kernel(const __grid_constant__ EvictArgs a,
                                                                      const __grid_constant__ EvictSet set, long long rows)
{
    wait_for_previous_grid();
    allow_next_grid();
    const int B = a.g.block_size;
    for (long long x = blockIdx.x * (long long)kCommitThreads + threadIdx.x; x < rows;
         x += (long long)gridDim.x * kCommitThreads) {
        const int q = req_of(set, x);
        const EvictReq& r = set.req[q];
        const int row = (int)(x - r.row_begin);
        int32_t* table = a.table + (long long)r.req * a.max_blocks;
        if (row == 0) a.seq_lens_dev[r.req] = r.n_keep;
        if (a.weights) a.weights[r.req * a.req_stride + row] = row < r.n_keep ? a.stage_w[r.stage + row] : 0.f;
        if (B == 1) {
            table[row] = row < r.n_keep ? a.stage_i[r.stage + row] : -1;
            continue;
        }
        const int blk = row / B, keep_blocks = (r.n_keep + B - 1) / B;
        if (row < r.n_keep && a.pending) {
            const int page = page_at(a, r, blk);
            if (page >= 0) a.pending[(long long)page * B + (row - blk * B)] = a.stage_i[r.stage + row];
        }
        // the first row of a block clears its dropped rows' turns, and gives its page back if all of them are
        if (row != blk * B || (blk + 1) * (long long)B <= r.n_keep) continue;
        const int page = page_at(a, r, blk);
        if (a.pending && page >= 0)
            for (int i = max(r.n_keep - row, 0); i < min(B, r.len - row); ++i) a.pending[(long long)page * B + i] = 0;
        if (blk >= keep_blocks) {
            a.free_q[ring(r.push + (blk - keep_blocks), a.q_cap)] = page;
            table[blk] = -1;
        }
    }
}

}  // namespace

int launch_evict(const EvictArgs& a, const EvictSet& set, int sm_count, void* stream)
{
    cudaStream_t s = (cudaStream_t)stream;
    const EvictReq& back = set.req[set.n - 1];
    const long long rows = back.row_begin + back.len;
    cudaError_t e = launch_dependent(check_lists_kernel, set.n, kCheckThreads, s, a, set);
    if (e != cudaSuccess) return (int)e;
    if (a.g.block_size == 1 || a.weights || a.pending)
        e = launch_dependent(stage_kernel, grid_for(rows, kStageThreads, sm_count * 8), kStageThreads, s, a, set, rows);
    if (e == cudaSuccess && a.g.block_size > 1) {
        const int slice = 8, slices = (a.g.row_vecs + slice - 1) / slice;
        e = cudaFuncSetAttribute(move_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(ChainShared));
        if (e == cudaSuccess)
            e = launch_dependent_smem(move_rows_kernel, set.n * a.g.num_layers * slices, kChainThreads, sizeof(ChainShared), s, a,
                                      set, slices, slice);
    }
    if (e == cudaSuccess)
        e = launch_dependent(commit_evict_kernel, grid_for(rows, kCommitThreads, sm_count * 16), kCommitThreads, s, a, set, rows);
    return (int)e;
}

}  // namespace leyline
