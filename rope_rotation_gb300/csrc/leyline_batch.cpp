// leyline_batch.cpp -- batches of new tokens: the host plan and the C ABI entry points.
//
// "Leyline: KV Cache Directives for Agentic Inference", section 2.3: prefill writes rows into
// new slots.  A plan is made once a step, on the host, for the lengths as they stand; the calls of
// the step's layers read it from the batch's device memory (see leyline_batch.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "leyline_batch.h"
#include "leyline_pool_state.h"

using namespace leyline;

// State of one batch (opaque to callers as leyline_batch_t).
struct leyline_batch {
    leyline_pool* pool = nullptr;
    int32_t max_chunks = 0;
    int32_t max_tokens = 0;
    int32_t q_heads = 0;
    int32_t value_dim = 0;
    WorkShape shape{};
    WorkShape pair_shape{};  // ctas 0: the pool's rows are not for pairs
    int64_t max_tiles = 0;
    BatchLayout layout{};
    TileMaps maps{};
    size_t stage_bytes = 0;  // plan + runs
    char* d_plan = nullptr;
    int64_t* d_slot = nullptr;
    float2* d_trig = nullptr;
    double* d_theta = nullptr;
    float* d_part_out = nullptr;
    float* d_part_lse = nullptr;
    int32_t* d_redo = nullptr;
    // pinned staging, used in turn: the host rewrites a slot once the install that read it is done
    static constexpr int kSlots = 4;
    char* h_stage[kSlots] = {};
    cudaEvent_t installed[kSlots] = {};
    bool slot_used[kSlots] = {};
    int next_slot = 0;
    bool planned = false;
    PlanMark mark;
    int32_t n_tokens = 0;
    int32_t n_joins = 0;
    bool pairs = false;  // the plan is for pairs
    bool many_parts = false;  // it splits a tile into more than kFewParts
};

namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The plan's device buffer: header, chunks, per-CTA ranges and joins, and last the items, of which a plan copies its own.
BatchLayout make_layout(int32_t max_chunks, int64_t max_tiles, int32_t ctas)
{
    BatchLayout l;
    l.chunks = align_up(sizeof(BatchHeader), 16);
    l.cta_begin = align_up(l.chunks + sizeof(ChunkDev) * (size_t)max_chunks, 16);
    l.joins = align_up(l.cta_begin + sizeof(int32_t) * (size_t)(ctas + 1), 16);
    l.items = align_up(l.joins + sizeof(AttnJoin) * (size_t)ctas, 16);
    l.bytes = align_up(l.items + sizeof(AttnItem) * (size_t)(max_tiles + ctas), 16);
    return l;
}

int bad(const char* msg) { return set_error(LEYLINE_ERR_INVALID_ARG, msg); }

// A heads view of `heads` heads of `dim` elements; resolves the pointer.
int check_heads(const leyline_heads_t* h, int device, const char* what, HeadsView* out)
{
    char msg[128];
    if (!h || !h->ptr || (reinterpret_cast<uintptr_t>(h->ptr) & 15) != 0) {
        snprintf(msg, sizeof msg, "%s must be a 16-byte aligned device pointer", what);
        return bad(msg);
    }
    if (h->token_stride % 8 != 0 || h->head_stride % 8 != 0 || h->token_stride < 0 || h->head_stride < 0) {
        snprintf(msg, sizeof msg, "%s: strides must be non-negative multiples of 8 elements", what);
        return bad(msg);
    }
    void* alias;
    bool host;
    int rc = resolve_access(h->ptr, device, what, &alias, &host);
    if (rc != LEYLINE_OK) return rc;
    *out = HeadsView{alias, h->token_stride, h->head_stride};
    return LEYLINE_OK;
}

// A norm's weights: bf16, 16-byte aligned, or NULL.
int check_norm(const void** w, int device, const char* what)
{
    if (!*w) return LEYLINE_OK;
    char msg[96];
    if ((reinterpret_cast<uintptr_t>(*w) & 15) != 0) {
        snprintf(msg, sizeof msg, "%s must be 16-byte aligned", what);
        return bad(msg);
    }
    void* alias;
    bool host;
    int rc = resolve_access(*w, device, what, &alias, &host);
    *w = alias;
    return rc;
}

// The tokens a call's tensors hold: a captured call may be replayed with plans of up to max_tokens.
int64_t room_of(const leyline_batch* b, bool captured) { return captured ? b->max_tokens : b->n_tokens; }

// Head axes written to must hold distinct places, for `tokens` tokens.
int check_written(const HeadsView& v, int64_t tokens, int64_t heads, int64_t dim, const char* what)
{
    char msg[128];
    const int64_t lo = std::min(v.token_stride, v.head_stride), hi = std::max(v.token_stride, v.head_stride);
    const int64_t inner = v.head_stride <= v.token_stride ? heads : tokens;
    if ((heads > 1 && (lo < dim || hi < inner * lo)) || (heads == 1 && v.token_stride < dim)) {
        snprintf(msg, sizeof msg, "%s: its strides let heads or tokens overlap", what);
        return bad(msg);
    }
    return LEYLINE_OK;
}

Extent extent(const HeadsView& v, int64_t tokens, int64_t heads, int64_t dim)
{
    return Extent{reinterpret_cast<uintptr_t>(v.ptr), tokens, heads, 2 * v.token_stride, 2 * v.head_stride, 2 * dim};
}

// Common start of the calls of a step's layers.
int enter(leyline_batch* b, cudaStream_t stream, bool* captured)
{
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &st);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        if (e == cudaErrorStreamCaptureImplicit)
            return bad("the legacy default stream cannot be used while another stream is being captured");
        return cuda_error(e, "querying the stream's capture status");
    }
    *captured = st != cudaStreamCaptureStatusNone;
    if (!*captured && b->mark.stale && b->n_tokens > 0)
        return bad("the batch's plan no longer holds: a splice or a rollback has changed one of its requests");
    b->pool->window_open = false;  // other work on the pool ends the window of overlapping splices
    // a captured call is ordered by its graph; an event of other work cannot enter the capture
    return *captured ? LEYLINE_OK : order_after_previous(b->pool, stream);
}

int leave(leyline_batch* b, cudaStream_t stream, bool captured)
{
    return captured ? LEYLINE_OK : mark_done(b->pool, stream);
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

void free_batch(leyline_batch* b)
{
    for (int i = 0; i < leyline_batch::kSlots; ++i) {
        if (b->installed[i]) cudaEventDestroy(b->installed[i]);
        if (b->h_stage[i]) cudaFreeHost(b->h_stage[i]);
    }
    if (b->d_plan) cudaFree(b->d_plan);
    if (b->d_slot) cudaFree(b->d_slot);
    if (b->d_trig) cudaFree(b->d_trig);
    if (b->d_theta) cudaFree(b->d_theta);
    if (b->d_part_out) cudaFree(b->d_part_out);
    if (b->d_part_lse) cudaFree(b->d_part_lse);
    if (b->d_redo) cudaFree(b->d_redo);
    delete b;
}

int create_batch(leyline_pool_t* p, int32_t max_chunks, int32_t max_tokens, int32_t q_heads, leyline_batch_t** out)
{
    const Geometry& g = p->g;
    const int32_t bands = std::max(g.rope_heads, 1);
    const int checked = check_sizes(g, max_chunks, max_tokens, q_heads);
    if (checked != LEYLINE_OK) return checked;
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    leyline_batch* b = new leyline_batch();
    b->pool = p;
    b->max_chunks = max_chunks;
    b->max_tokens = max_tokens;
    b->q_heads = q_heads;
    b->value_dim = g.latent_dim / bands;
    // a head count that does not go over the key bands does for append and rotate alone
    b->shape = WorkShape{bands, q_heads % bands == 0 ? q_heads / bands : 0, p->sm_count,
                         bands == 1 && attention_takes_tiles(g) && p->d_pending ? kAttnRowsLazy : kAttnRows};
    // every chunk's rows are cut into tiles of their own
    b->max_tiles = (ceil_div((int64_t)max_tokens * b->shape.group, b->shape.rows) + max_chunks) * bands;
    if (b->max_tiles > INT32_MAX / 4) {
        free_batch(b);
        return bad("max_tokens * q_heads is too large");
    }
    b->layout = make_layout(max_chunks, b->max_tiles, b->shape.ctas);
    b->stage_bytes = b->layout.bytes + sizeof(PlanRun) * (size_t)(ceil_div(max_tokens, kPlanRun) + max_chunks);
    const int half = g.rope_dim / 2;
    std::vector<double> theta(half);
    for (int j = 0; j < half; ++j) theta[j] = std::pow(g.theta, -2.0 * j / g.rope_dim);
    const size_t parts = 2 * (size_t)b->shape.ctas;
    cudaError_t e = cudaMalloc(&b->d_plan, b->layout.bytes);
    if (e == cudaSuccess) e = cudaMalloc(&b->d_slot, sizeof(int64_t) * (size_t)max_tokens);
    if (e == cudaSuccess) e = cudaMalloc(&b->d_trig, sizeof(float2) * (size_t)max_tokens * half);
    if (e == cudaSuccess) e = cudaMalloc(&b->d_theta, sizeof(double) * half);
    if (e == cudaSuccess) e = cudaMalloc(&b->d_part_out, sizeof(float) * parts * kAttnRows * b->value_dim);
    if (e == cudaSuccess) e = cudaMalloc(&b->d_part_lse, sizeof(float) * parts * kAttnRows);
    if (e == cudaSuccess) e = cudaMemcpy(b->d_theta, theta.data(), sizeof(double) * half, cudaMemcpyHostToDevice);
    // an unplanned batch has no tokens
    if (e == cudaSuccess) e = cudaMemset(b->d_plan, 0, b->layout.bytes);
    for (int i = 0; i < leyline_batch::kSlots && e == cudaSuccess; ++i) {
        e = cudaEventCreateWithFlags(&b->installed[i], cudaEventDisableTiming);
        if (e == cudaSuccess) e = cudaHostAlloc((void**)&b->h_stage[i], b->stage_bytes, cudaHostAllocDefault);
    }
    if (e == cudaSuccess) e = (cudaError_t)attention_prepare(g, p->kv, &b->maps);
    if (e == cudaSuccess && attention_takes_tiles(g))
        e = cudaMalloc(&b->d_redo, sizeof(int32_t) * 2 * (size_t)(b->max_tiles + b->shape.ctas));
    if (e == cudaSuccess && bands == 1 && attention_takes_tiles(g) && !p->d_pending) {
        b->pair_shape = WorkShape{1, b->shape.group, p->sm_count / 2, kPairRows, kItemCostPairs};
        e = (cudaError_t)attention_pair_prepare(g, p->kv, &b->maps);
    }
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        free_batch(b);
        return cuda_error(e, "creating the batch");
    }
    try {
        p->batches.push_back(&b->mark);
    } catch (...) {
        free_batch(b);
        throw;
    }
    *out = b;
    return LEYLINE_OK;
}

int plan_batch(leyline_batch_t* b, leyline_block_table_t* bt, const leyline_chunk_t* chunks, int32_t n,
               cudaStream_t stream)
{
    leyline_pool* p = b->pool;
    if (!bt || !bt->table || !bt->seq_lens_dev || !bt->seq_lens_host || bt->num_reqs < 0 || bt->max_blocks < 0)
        return bad("incomplete block table");
    if (n < 0 || (n > 0 && !chunks)) return bad("bad chunks");
    if (n > b->max_chunks) return bad("more chunks than the batch holds");
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    int rc = refuse_capture(stream, "leyline_batch_plan");
    if (rc != LEYLINE_OK) return rc;
    ChunkPlan cp;
    rc = check_chunks(p->g, *bt, chunks, n, b->max_tokens, p->q_tail - p->q_head, p->q_head, &cp);
    if (rc != LEYLINE_OK) return rc;

    PlanMark mark;
    mark.table = bt->table;
    for (const ChunkDev& c : cp.chunks)
        if (c.n > 0) mark.reqs.push_back(c.req);
    std::sort(mark.reqs.begin(), mark.reqs.end());
    mark.since_checkpoint = true;

    const int slot = b->next_slot;
    if (b->slot_used[slot]) {  // the install that read this staging slot may still be in flight
        cudaError_t e = cudaEventSynchronize(b->installed[slot]);
        if (e != cudaSuccess) return cuda_error(e, "waiting for an earlier plan");
    }
    char* h = b->h_stage[slot];
    const BatchLayout& l = b->layout;
    if (!cp.chunks.empty()) memcpy(h + l.chunks, cp.chunks.data(), sizeof(ChunkDev) * cp.chunks.size());
    Split split{reinterpret_cast<AttnItem*>(h + l.items), reinterpret_cast<int32_t*>(h + l.cta_begin),
                reinterpret_cast<AttnJoin*>(h + l.joins)};
    const bool pairs = b->pair_shape.ctas > 0 && pairs_are_faster(b->shape, cp.chunks, b->maps.box == 0);
    split_work(pairs ? b->pair_shape : b->shape, cp.chunks, &split);
    BatchHeader hd{};
    hd.table = bt->table;
    hd.max_blocks = bt->max_blocks;
    hd.n_tokens = (int32_t)cp.tokens;
    hd.n_joins = split.n_joins;
    hd.pairs = pairs ? 1 : 0;
    memcpy(h, &hd, sizeof hd);
    if (!cp.runs.empty()) memcpy(h + l.bytes, cp.runs.data(), sizeof(PlanRun) * cp.runs.size());

    InstallArgs a{};
    a.staged = reinterpret_cast<const uint4*>(h);
    a.plan = reinterpret_cast<uint4*>(b->d_plan);
    a.runs = reinterpret_cast<const PlanRun*>(h + l.bytes);
    a.plan_vecs = (int64_t)((l.items + sizeof(AttnItem) * (size_t)split.n_items) / 16);
    a.n_runs = (int32_t)cp.runs.size();
    a.max_blocks = bt->max_blocks;
    a.table = bt->table;
    a.seq_lens_dev = bt->seq_lens_dev;
    a.free_q = p->d_queue;
    a.q_cap = p->q_cap;
    a.pending = p->d_pending;
    a.theta = b->d_theta;
    a.slot = b->d_slot;
    a.trig = b->d_trig;
    a.status = p->d_status;
    a.g = p->g;
    rc = order_after_previous(p, stream);
    if (rc != LEYLINE_OK) return rc;
    p->window_open = false;  // other work on the pool ends the window of overlapping splices
    cudaError_t e = (cudaError_t)launch_install(a, stream);
    if (e != cudaSuccess) return cuda_error(e, "launching the plan's install kernel");
    e = cudaEventRecord(b->installed[slot], stream);
    if (e != cudaSuccess) return cuda_error(e, "recording the plan's install");
    b->slot_used[slot] = true;
    b->next_slot = (slot + 1) % leyline_batch::kSlots;
    rc = mark_done(p, stream);
    if (rc != LEYLINE_OK) return rc;
    for (const auto& x : cp.new_len) bt->seq_lens_host[x.first] = x.second;
    p->q_head += cp.pages;
    if (cp.rewrites) p->ckpt_turned = true;
    b->planned = true;
    std::swap(b->mark, mark);
    b->n_tokens = (int32_t)cp.tokens;
    b->n_joins = split.n_joins;
    b->pairs = pairs;
    b->many_parts = false;
    for (int32_t j = 0; j < split.n_joins; ++j) b->many_parts |= split.joins[j].parts > kFewParts;
    return LEYLINE_OK;
}

}  // namespace

extern "C" {

int leyline_batch_create(leyline_pool_t* pool, int32_t max_chunks, int32_t max_tokens, int32_t q_heads,
                         leyline_batch_t** out)
{
    clear_error();
    if (!out) return bad("null output pointer");
    *out = nullptr;
    if (!pool) return bad("null pool");
    return guarded([&] { return create_batch(pool, max_chunks, max_tokens, q_heads, out); });
}

int leyline_batch_destroy(leyline_batch_t* b)
{
    clear_error();
    if (!b) return bad("null batch");
    DeviceGuard guard(b->pool->device);
    int rc = wait_pool(b->pool);
    std::vector<PlanMark*>& live = b->pool->batches;
    live.erase(std::find(live.begin(), live.end(), &b->mark));
    free_batch(b);
    return rc;
}

int leyline_batch_plan(leyline_batch_t* b, leyline_block_table_t* bt, const leyline_chunk_t* chunks, int32_t n,
                       void* stream)
{
    NvtxRange range("leyline_batch_plan");
    clear_error();
    if (!b) return bad("null batch");
    return guarded([&] { return plan_batch(b, bt, chunks, n, (cudaStream_t)stream); });
}

int leyline_append(leyline_batch_t* b, int32_t layer, const void* rows, int64_t row_stride, const void* latent_norm,
                   const void* key_norm, float eps, void* stream_v)
{
    NvtxRange range("leyline_append");
    clear_error();
    if (!b) return bad("null batch");
    leyline_pool* p = b->pool;
    const Geometry& g = p->g;
    if (layer < 0 || layer >= g.num_layers) return bad("layer out of range");
    if (!b->planned) return bad("the batch has no plan");
    if (row_stride % 8 != 0 || row_stride < g.row_elems) return bad("row_stride must be a multiple of 8, at least a row");
    if (latent_norm && g.rope_heads > 1) return bad("latent_norm is for rows with one band (MLA)");
    if (!(eps >= 0.f)) return bad("eps must not be negative");
    cudaStream_t stream = (cudaStream_t)stream_v;
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    bool host = false, captured = false;
    void* alias = nullptr;
    int rc = enter(b, stream, &captured);
    if (rc != LEYLINE_OK) return rc;
    if (b->n_tokens == 0 && !captured) return LEYLINE_OK;
    if (!rows || (reinterpret_cast<uintptr_t>(rows) & 15) != 0) return bad("rows must be a 16-byte aligned pointer");
    rc = resolve_access(rows, p->device, "rows", &alias, &host);
    if (rc == LEYLINE_OK) rc = check_norm(&latent_norm, p->device, "latent_norm");
    if (rc == LEYLINE_OK) rc = check_norm(&key_norm, p->device, "key_norm");
    if (rc != LEYLINE_OK) return rc;
    AppendArgs a{};
    a.kv = static_cast<uint4*>(p->kv);
    a.rows = static_cast<const uint4*>(alias);
    a.row_stride = row_stride / 8;
    a.latent_norm = static_cast<const uint4*>(latent_norm);
    a.key_norm = static_cast<const uint4*>(key_norm);
    a.eps = eps;
    a.layer = layer;
    a.header = reinterpret_cast<const BatchHeader*>(b->d_plan);
    a.slot = b->d_slot;
    a.trig = b->d_trig;
    a.g = g;
    int err = launch_append(a, captured ? b->max_tokens : b->n_tokens, p->sm_count, stream);
    if (err != 0) return cuda_error((cudaError_t)err, "launching the append kernel");
    return leave(b, stream, captured);
}

int leyline_rotate(leyline_batch_t* b, const leyline_heads_t* q, const leyline_heads_t* out, const void* norm, float eps,
                   void* stream_v)
{
    NvtxRange range("leyline_rotate");
    clear_error();
    if (!b) return bad("null batch");
    leyline_pool* p = b->pool;
    if (!b->planned) return bad("the batch has no plan");
    if (!(eps >= 0.f)) return bad("eps must not be negative");
    cudaStream_t stream = (cudaStream_t)stream_v;
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    RotateArgs a{};
    bool captured = false;
    int rc = enter(b, stream, &captured);
    if (rc != LEYLINE_OK) return rc;
    if (b->n_tokens == 0 && !captured) return LEYLINE_OK;
    rc = check_heads(q, p->device, "q", &a.q);
    if (rc == LEYLINE_OK) rc = check_heads(out, p->device, "out", &a.out);
    if (rc == LEYLINE_OK) rc = check_written(a.out, room_of(b, captured), b->q_heads, p->g.rope_dim, "out");
    if (rc == LEYLINE_OK && q->ptr == out->ptr &&
        (q->token_stride != out->token_stride || q->head_stride != out->head_stride))
        rc = bad("q and out start at one address with different strides");
    const int64_t room = room_of(b, captured);
    if (rc == LEYLINE_OK && q->ptr != out->ptr &&
        overlap(extent(a.q, room, b->q_heads, p->g.rope_dim), extent(a.out, room, b->q_heads, p->g.rope_dim)))
        rc = bad("out may be q itself, but not overlap it otherwise");
    if (rc == LEYLINE_OK) rc = check_norm(&norm, p->device, "norm");
    if (rc != LEYLINE_OK) return rc;
    a.norm = static_cast<const uint4*>(norm);
    a.eps = eps;
    a.q_heads = b->q_heads;
    a.header = reinterpret_cast<const BatchHeader*>(b->d_plan);
    a.trig = b->d_trig;
    a.g = p->g;
    int err = launch_rotate(a, captured ? b->max_tokens : b->n_tokens, p->sm_count, stream);
    if (err != 0) return cuda_error((cudaError_t)err, "launching the rotate kernel");
    return leave(b, stream, captured);
}

int leyline_attention(leyline_batch_t* b, int32_t layer, const leyline_heads_t* q_latent, const leyline_heads_t* q_rope,
                      const leyline_heads_t* out, float* lse, float scale, int32_t flags, void* stream_v)
{
    NvtxRange range("leyline_attention");
    clear_error();
    if (!b) return bad("null batch");
    leyline_pool* p = b->pool;
    const Geometry& g = p->g;
    const bool mla = g.rope_heads <= 1;
    if (layer < 0 || layer >= g.num_layers) return bad("layer out of range");
    if (!b->planned) return bad("the batch has no plan");
    if (b->shape.group == 0) return bad("attention needs q_heads to be a multiple of rope_heads");
    if ((flags & ~LEYLINE_ATTENTION_PREFIX) != 0) return bad("unknown flags");
    if (!std::isfinite(scale)) return bad("scale must be finite");
    if (!mla && q_latent) return bad("q_latent must be NULL for rows of several bands");
    if ((reinterpret_cast<uintptr_t>(lse) & 3) != 0) return bad("lse must be 4-byte aligned");
    cudaStream_t stream = (cudaStream_t)stream_v;
    DeviceGuard guard(p->device);
    if (!guard.ok) return set_error(LEYLINE_ERR_CUDA, "cannot select the pool's device");
    AttnArgs a{};
    bool captured = false, host = false;
    int rc = enter(b, stream, &captured);
    if (rc != LEYLINE_OK) return rc;
    if (b->n_tokens == 0 && !captured) return LEYLINE_OK;
    rc = check_heads(q_rope, p->device, "q_rope", &a.q_rope);
    if (rc == LEYLINE_OK && mla) rc = check_heads(q_latent, p->device, "q_latent", &a.q_latent);
    if (rc == LEYLINE_OK) rc = check_heads(out, p->device, "out", &a.out);
    if (rc == LEYLINE_OK) rc = check_written(a.out, room_of(b, captured), b->q_heads, b->value_dim, "out");
    void* lse_alias = lse;
    if (rc == LEYLINE_OK && lse) rc = resolve_access(lse, p->device, "lse", &lse_alias, &host);
    if (rc != LEYLINE_OK) return rc;
    // other CTAs read queries while one writes its outputs, and an item may be computed again from its queries
    const int64_t room = room_of(b, captured);
    const Extent to = extent(a.out, room, b->q_heads, b->value_dim), band = extent(a.q_rope, room, b->q_heads, g.rope_dim);
    const Extent latent = extent(a.q_latent, mla ? room : 0, b->q_heads, g.latent_dim);
    if (overlap(to, band) || overlap(to, latent)) return bad("out must not lie over the queries");
    const Extent sums{reinterpret_cast<uintptr_t>(lse_alias), lse ? 1 : 0, 1, 0, 0, 4 * room * b->q_heads};
    if (overlap(sums, band) || overlap(sums, latent) || overlap(sums, to)) return bad("lse must not lie over out or the queries");
    a.kv = static_cast<const uint4*>(p->kv);
    a.lse = static_cast<float*>(lse_alias);
    a.scale = scale;
    a.layer = layer;
    a.prefix = flags & LEYLINE_ATTENTION_PREFIX;
    a.q_heads = b->q_heads;
    a.header = reinterpret_cast<const BatchHeader*>(b->d_plan);
    a.chunks = reinterpret_cast<const ChunkDev*>(b->d_plan + b->layout.chunks);
    a.items = reinterpret_cast<const AttnItem*>(b->d_plan + b->layout.items);
    a.cta_begin = reinterpret_cast<const int32_t*>(b->d_plan + b->layout.cta_begin);
    a.joins = reinterpret_cast<const AttnJoin*>(b->d_plan + b->layout.joins);
    a.part_out = b->d_part_out;
    a.part_lse = b->d_part_lse;
    a.redo = b->d_redo;
    a.pending = p->d_pending;
    a.turn = p->d_theta_j;
    a.status = p->d_status;
    a.g = g;
    // a captured call may be replayed with plans for either kernel: both are launched, and the one the plan is not for
    // ends at once
    int err = 0;
    if (captured || !b->pairs) err = launch_attention(a, b->maps, b->shape.ctas, stream);
    if (err == 0 && b->pair_shape.ctas > 0 && (captured || b->pairs))
        err = launch_attention_pair(a, b->maps, b->pair_shape.ctas, stream);
    if (err != 0) return cuda_error((cudaError_t)err, "launching the attention kernel");
    // and with plans that split more tiles
    const int joins = captured ? b->shape.ctas : b->n_joins;
    const int rows = captured ? (b->pair_shape.ctas > 0 ? kPairRows : kAttnRows) : b->pairs ? kPairRows : kAttnRows;
    if (joins > 0) {
        err = launch_join(a, joins, rows, captured || b->many_parts, stream);
        if (err != 0) return cuda_error((cudaError_t)err, "launching the join kernel");
    }
    return leave(b, stream, captured);
}

}  // extern "C"
