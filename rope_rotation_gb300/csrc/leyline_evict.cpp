// leyline_evict.cpp -- eviction of rows by their weights: the C ABI entry points (leyline_select_rows, leyline_evict).
//
// Lengths, and with them the pages that go back, are known on the host from the counts of rows kept; which rows these
// are stays on the device.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <new>
#include <vector>

#include "leyline_batch.h"
#include "leyline_evict.h"
#include "leyline_pool_state.h"

using namespace leyline;

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int bad(const char* msg) { return set_error(LEYLINE_ERR_INVALID_ARG, msg); }

// What both calls check of a request's counts.
int check_keeps(const Geometry& g, const leyline_block_table_t& bt, const leyline_keep_t* keeps, int32_t n,
                int64_t kept_stride, bool ends)
{
    char msg[160];
    std::vector<int32_t> seen;
    seen.reserve(n);
    for (int32_t k = 0; k < n; ++k) {
        const leyline_keep_t& e = keeps[k];
        if (e.req < 0 || e.req >= bt.num_reqs) {
            snprintf(msg, sizeof msg, "entry %d: request out of range", k);
            return bad(msg);
        }
        const int64_t len = bt.seq_lens_host[e.req];
        if (len < 0 || len > (int64_t)bt.max_blocks * g.block_size)
            return bad("seq_lens_host entry outside [0, max_blocks * block_size]");
        if (len > kMostRows) return bad("a request of more than 2^31 - 2^16 rows");
        if (e.n_keep < 0 || e.n_keep > len) {
            snprintf(msg, sizeof msg, "entry %d: n_keep %d is not within the request's %lld rows", k, e.n_keep, (long long)len);
            return bad(msg);
        }
        if (ends && (e.first < 0 || e.last < 0 || (int64_t)e.first + e.last > e.n_keep)) {
            snprintf(msg, sizeof msg, "entry %d: first and last must be non-negative, and n_keep hold both", k);
            return bad(msg);
        }
        if (e.n_keep > kept_stride && n > 1) return bad("kept_stride is shorter than a list");
        seen.push_back(e.req);
    }
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return bad("a request appears twice");
    return LEYLINE_OK;
}

int64_t longest_list(const leyline_keep_t* keeps, int32_t n)
{
    int64_t longest = 0;
    for (int32_t k = 0; k < n; ++k) longest = std::max<int64_t>(longest, keeps[k].n_keep);
    return longest;
}

// The rows' weights, for requests up to the longest of `keeps`.  Requests without rows need no memory.
int check_weights(const leyline_row_weights_t& w, const leyline_block_table_t& bt, const leyline_keep_t* keeps, int32_t n,
                  int device, float** alias)
{
    if ((reinterpret_cast<uintptr_t>(w.ptr) & 3) != 0) return bad("weights must be a 4-byte aligned device pointer");
    if (w.num_reqs < 0 || w.rows < 0 || (w.num_reqs > 1 && w.req_stride < w.rows))
        return bad("weights: a request's stride is at least its rows");
    bool rows = false;
    for (int32_t k = 0; k < n; ++k) {
        const int64_t len = bt.seq_lens_host[keeps[k].req];
        if (keeps[k].req >= w.num_reqs || len > w.rows) return bad("weights do not hold every row of the requests");
        rows |= len > 0;
    }
    *alias = nullptr;
    if (!rows) return LEYLINE_OK;
    if (!w.ptr) return bad("weights must be a 4-byte aligned device pointer");
    void* a;
    bool host;
    int rc = resolve_access(w.ptr, device, "weights", &a, &host);
    *alias = static_cast<float*>(a);
    return rc;
}

// Lists without rows need no memory.
int check_lists(const int32_t* kept, int64_t kept_stride, int64_t longest, int device, int32_t** alias)
{
    if (kept_stride < 0) return bad("kept_stride must not be negative");
    *alias = nullptr;
    if (longest == 0) return LEYLINE_OK;
    if (!kept || (reinterpret_cast<uintptr_t>(kept) & 3) != 0) return bad("kept must be a 4-byte aligned device pointer");
    void* a;
    bool host;
    int rc = resolve_access(kept, device, "kept", &a, &host);
    *alias = static_cast<int32_t*>(a);
    return rc;
}

// Whether the lists share a byte with the weights.
bool lists_over_weights(const int32_t* kept, int64_t kept_stride, int64_t longest, int32_t n, const float* w,
                        const leyline_row_weights_t& view)
{
    if (longest == 0 || view.rows == 0) return false;
    const Extent lists{reinterpret_cast<uintptr_t>(kept), n, 1, 4 * kept_stride, 0, 4 * longest};
    const Extent rows{reinterpret_cast<uintptr_t>(w), view.num_reqs, 1, 4 * view.req_stride, 0, 4 * view.rows};
    return overlap(lists, rows);
}

int enter(leyline_pool_t* p, const leyline_block_table_t* bt, const leyline_keep_t* keeps, int32_t n, cudaStream_t stream,
          const char* what)
{
    if (!bt || !bt->table || !bt->seq_lens_dev || !bt->seq_lens_host || bt->num_reqs < 0 || bt->max_blocks < 0)
        return bad("incomplete block table");
    if (n < 0 || (n > 0 && !keeps)) return bad("bad keeps");
    return refuse_capture(stream, what);
}

int select_rows(leyline_pool_t* p, const leyline_block_table_t* bt, const leyline_row_weights_t* w,
                const leyline_keep_t* keeps, int32_t n, int32_t* kept, int64_t kept_stride, cudaStream_t stream)
{
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    int rc = enter(p, bt, keeps, n, stream, "leyline_select_rows");
    if (rc == LEYLINE_OK) rc = check_keeps(p->g, *bt, keeps, n, kept_stride, true);
    if (rc != LEYLINE_OK || n == 0) return rc;
    SelectArgs a{};
    float* weights = nullptr;
    const int64_t longest = longest_list(keeps, n);
    rc = check_weights(*w, *bt, keeps, n, p->device, &weights);
    if (rc == LEYLINE_OK) rc = check_lists(kept, kept_stride, longest, p->device, &a.kept);
    if (rc == LEYLINE_OK && lists_over_weights(a.kept, kept_stride, longest, n, weights, *w))
        rc = bad("kept must not lie over the weights");
    if (rc != LEYLINE_OK || longest == 0) return rc;
    a.weights = weights;
    a.req_stride = w->req_stride;
    a.kept_stride = kept_stride;
    p->window_open = false;  // other work on the pool ends the window of overlapping splices
    rc = order_after_previous(p, stream);
    if (rc != LEYLINE_OK) return rc;
    for (int32_t k0 = 0; k0 < n; k0 += kEvictReqs) {
        EvictSet set{};
        for (int32_t k = k0; k < std::min(n, k0 + kEvictReqs); ++k)
            set.req[set.n++] = EvictReq{keeps[k].req, keeps[k].n_keep, keeps[k].first, keeps[k].last,
                                        (int32_t)bt->seq_lens_host[keeps[k].req], k, 0, 0, 0, 0};
        int err = launch_select(a, set, stream);
        if (err != 0) return cuda_error((cudaError_t)err, "launching the selection kernel");
    }
    return mark_done(p, stream);
}

int evict(leyline_pool_t* p, leyline_block_table_t* bt, const leyline_keep_t* keeps, int32_t n, const int32_t* kept,
          int64_t kept_stride, const leyline_row_weights_t* w, cudaStream_t stream)
{
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    const Geometry& g = p->g;
    int rc = enter(p, bt, keeps, n, stream, "leyline_evict");
    if (rc == LEYLINE_OK) rc = check_keeps(g, *bt, keeps, n, kept_stride, false);
    if (rc != LEYLINE_OK || n == 0) return rc;
    EvictArgs a{};
    int32_t* lists = nullptr;
    const int64_t longest = longest_list(keeps, n);
    rc = check_lists(kept, kept_stride, longest, p->device, &lists);
    if (rc == LEYLINE_OK && w) rc = check_weights(*w, *bt, keeps, n, p->device, &a.weights);
    if (rc == LEYLINE_OK && w && lists_over_weights(lists, kept_stride, longest, n, a.weights, *w))
        rc = bad("kept must not lie over the weights");
    if (rc != LEYLINE_OK) return rc;

    std::vector<EvictReq> reqs;  // that lose rows
    int64_t pages = 0, launch_stage = 0, most_stage = 0;
    for (int32_t k = 0; k < n; ++k) {
        const int32_t len = (int32_t)bt->seq_lens_host[keeps[k].req];
        if (keeps[k].n_keep == len) continue;
        reqs.push_back(EvictReq{keeps[k].req, keeps[k].n_keep, 0, 0, len, k, 0, 0, 0, p->q_tail + pages});
        pages += ceil_div(len, g.block_size) - ceil_div(keeps[k].n_keep, g.block_size);
    }
    if (reqs.empty()) return LEYLINE_OK;
    // the longest first: a request's chains of rows take as long as its rows, whatever runs beside them
    std::stable_sort(reqs.begin(), reqs.end(), [](const EvictReq& x, const EvictReq& y) { return x.n_keep > y.n_keep; });
    for (size_t k = 0; k < reqs.size(); ++k) {
        if (k % kEvictReqs == 0) launch_stage = 0;
        else reqs[k].block_begin = reqs[k - 1].block_begin + (int32_t)ceil_div(reqs[k - 1].len, kStageRows);
        reqs[k].stage = launch_stage;
        launch_stage += reqs[k].n_keep;
        most_stage = std::max(most_stage, launch_stage);
    }
    if (p->q_tail - p->q_head + pages > g.num_pages)
        return bad("the requests hold more pages than the pool has free slots for: their tables were not filled from this pool");
    const int64_t half = ceil_div(most_stage, 4) * 4;
    rc = grow_stage(p, (size_t)(2 * half));
    if (rc == LEYLINE_OK) rc = order_after_previous(p, stream);
    if (rc != LEYLINE_OK) return rc;
    p->window_open = false;  // other work on the pool ends the window of overlapping splices
    a.kv = static_cast<uint4*>(p->kv);
    a.table = bt->table;
    a.seq_lens_dev = bt->seq_lens_dev;
    a.free_q = p->d_queue;
    a.q_cap = p->q_cap;
    a.kept = lists;
    a.kept_stride = kept_stride;
    a.req_stride = w ? w->req_stride : 0;
    a.pending = p->d_pending;
    a.stage_i = p->d_stage;
    a.stage_w = reinterpret_cast<float*>(p->d_stage + half);
    a.status = p->d_status;
    a.max_blocks = bt->max_blocks;
    a.g = g;
    for (size_t k0 = 0; k0 < reqs.size(); k0 += kEvictReqs) {
        EvictSet set{};
        set.n = (int32_t)std::min<size_t>(kEvictReqs, reqs.size() - k0);
        std::copy(reqs.begin() + k0, reqs.begin() + k0 + set.n, set.req);
        a.state = p->d_lists + p->lists_turn * kEvictReqs;
        a.next_state = p->d_lists + (1 - p->lists_turn) * kEvictReqs;
        p->lists_turn = 1 - p->lists_turn;
        int err = launch_evict(a, set, stream);
        if (err != 0) return cuda_error((cudaError_t)err, "launching the eviction kernels");
    }
    rc = mark_done(p, stream);
    if (rc != LEYLINE_OK) return rc;
    for (const EvictReq& r : reqs) {
        bt->seq_lens_host[r.req] = r.n_keep;
        outdate_plans(p, bt->table, r.req);
    }
    p->q_tail += pages;
    if (g.block_size > 1) p->ckpt_turned = true;  // rows moved within their pages
    return LEYLINE_OK;
}

template <typename F>
int guarded(F&& f)
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return bad("out of host memory");
    } catch (...) {
        return bad("unexpected host error");
    }
}

}  // namespace

extern "C" {

int leyline_select_rows(leyline_pool_t* pool, const leyline_block_table_t* bt, const leyline_row_weights_t* weights,
                        const leyline_keep_t* keeps, int32_t n, int32_t* kept, int64_t kept_stride, void* stream)
{
    NvtxRange range("leyline_select_rows");
    clear_error();
    if (!pool || !weights) return bad("null argument");
    return guarded([&] { return select_rows(pool, bt, weights, keeps, n, kept, kept_stride, (cudaStream_t)stream); });
}

int leyline_evict(leyline_pool_t* pool, leyline_block_table_t* bt, const leyline_keep_t* keeps, int32_t n,
                  const int32_t* kept, int64_t kept_stride, const leyline_row_weights_t* weights, void* stream)
{
    NvtxRange range("leyline_evict");
    clear_error();
    if (!pool) return bad("null pool");
    return guarded([&] { return evict(pool, bt, keeps, n, kept, kept_stride, weights, (cudaStream_t)stream); });
}

}  // extern "C"
