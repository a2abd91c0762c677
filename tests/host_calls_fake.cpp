// host_calls_fake.cpp -- the host side of the C ABI over a CUDA runtime of its own, built by tests/test_host_calls.py with
// the sanitizers: what each call enqueues, and in which order.  No GPU is used and no kernel runs.
//
// The runtime here keeps device memory on the host.  As CUDA documents it, a copy from pageable memory to the device has
// left the host's buffer when cudaMemcpy returns but may not have arrived, and a cudaMemset may not have run: both are work of
// the legacy stream, which other streams made as non-blocking ones are not ordered after.  So such work has to be waited
// for before a call returns or launches a kernel on another stream.
// Exit code 0: every check of the named case held.  Usage: host_calls_fake <case>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "leyline_batch.h"
#include "leyline_pool_state.h"

using namespace leyline;

namespace {

std::map<uintptr_t, size_t> device_memory;
bool legacy_pending = false;  // work of the legacy stream may still run
int unordered = 0;            // kernels launched on another stream meanwhile
int64_t copied_vecs = 0;      // of the last plan
int64_t weighed_rows = 0;     // that the last weighing's kernels take of a request
int copies_in = 0, selects = 0, evictions = 0, weighings = 0;
std::vector<ListState> seen_state;  // of the last eviction, both arrays

int launched(void* stream)
{
    if (stream && legacy_pending) ++unordered;
    return 0;
}

bool on_device(const void* p)
{
    auto at = device_memory.upper_bound((uintptr_t)p);
    if (at == device_memory.begin()) return false;
    --at;
    return (uintptr_t)p < at->first + at->second;
}

int failures = 0;
void check(bool ok, const char* what)
{
    if (ok) return;
    std::fprintf(stderr, "failed: %s (last error: %s)\n", what, leyline_last_error());
    ++failures;
}

}  // namespace

extern "C" {

cudaError_t cudaMalloc(void** p, size_t n)
{
    *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
    std::memset(*p, 0xab, n);
    device_memory[(uintptr_t)*p] = n;
    return cudaSuccess;
}
cudaError_t cudaFree(void* p)
{
    if (p) device_memory.erase((uintptr_t)p);
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned)
{
    *p = std::malloc(n);
    return cudaSuccess;
}
cudaError_t cudaFreeHost(void* p)
{
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind kind)
{
    std::memcpy(to, from, n);
    legacy_pending = kind == cudaMemcpyHostToDevice;  // a copy to the host waits for the stream
    copies_in += kind == cudaMemcpyHostToDevice;
    return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t n)
{
    std::memset(p, v, n);
    legacy_pending = true;
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* to, const void* from, size_t n, cudaMemcpyKind, cudaStream_t)
{
    std::memcpy(to, from, n);
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize()
{
    legacy_pending = false;
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s)
{
    if (!s) legacy_pending = false;
    return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void* p)
{
    *a = cudaPointerAttributes{};
    a->type = on_device(p) ? cudaMemoryTypeDevice : cudaMemoryTypeUnregistered;
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* st)
{
    *st = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int)
{
    *v = 152;
    return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaEventCreate(cudaEvent_t* e)
{
    *e = nullptr;
    return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) { return cudaEventCreate(e); }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t)
{
    *ms = 0.f;
    return cudaSuccess;
}

}  // extern "C"

namespace leyline {

int launch_init_queue(int32_t* q, int64_t n, void* s)
{
    for (int64_t i = 0; i < n; ++i) q[i] = (int32_t)i;
    if (!s) legacy_pending = true;
    return launched(s);
}
int launch_clear_pending(int32_t*, const int32_t*, int64_t, int32_t, void* s)
{
    if (!s) legacy_pending = true;
    return launched(s);
}
int launch_upload_plan(const void*, void*, size_t, void* s) { return launched(s); }
int launch_splice(const SpliceArgs&, const ParamPlan*, int, void* s, cudaEvent_t, cudaEvent_t) { return launched(s); }
int launch_gather(const void*, const int32_t*, const Geometry&, int32_t, int64_t, int64_t, void*, int32_t*, void* s) { return launched(s); }
int launch_gather_lazy(const void*, const int32_t*, const Geometry&, int32_t, int64_t, int64_t, void*, const int32_t*, const double*,
                       int32_t*, void* s)
{
    return launched(s);
}
int launch_materialize(void*, const int32_t*, int32_t, const MaterializeSet&, const Geometry&, int32_t*, const double*, int32_t*,
                       const MaterializeScratch&, void* s)
{
    return launched(s);
}
int move_rotate_blocks_per_sm(int* n) { return *n = 1, 0; }
int rotate_in_place_blocks_per_sm(int* n) { return *n = 1, 0; }
int bulk_prepare(int32_t, int* n) { return *n = 1, 0; }
int launch_install(const InstallArgs& a, void* s)
{
    for (int64_t i = 0; i < a.plan_vecs; ++i) {
        const int64_t at = i < a.gap_at ? i : i + a.gap;
        a.plan[at] = a.staged[at];
    }
    copied_vecs = a.plan_vecs;
    return launched(s);
}
int launch_append(const AppendArgs&, int64_t, int, void* s) { return launched(s); }
int launch_rotate(const RotateArgs&, int64_t, int, void* s) { return launched(s); }
bool attention_takes_tiles(const Geometry&) { return false; }
int attention_prepare(const Geometry&, const void*, TileMaps*) { return 0; }
int attention_pair_prepare(const Geometry&, const void*, TileMaps*) { return 0; }
int launch_attention(const AttnArgs&, const TileMaps&, int, void* s) { return launched(s); }
int launch_attention_pair(const AttnArgs&, const TileMaps&, int, void* s) { return launched(s); }
int launch_join(const AttnArgs&, int, int, bool, void* s) { return launched(s); }
int weigh_tile_prepare(const Geometry&, const void*, WeighMaps*) { return 0; }
int weigh_pair_prepare(const Geometry&) { return 0; }
int launch_weigh(const WeighArgs& a, int, void* s) { return ++weighings, weighed_rows = a.rows, launched(s); }
int launch_weigh_tile(const WeighArgs&, const WeighMaps&, int, void* s) { return ++weighings, launched(s); }
int launch_weigh_pair(const WeighArgs&, const WeighMaps&, int64_t, int, int, void* s) { return ++weighings, launched(s); }
int launch_select(const SelectArgs&, const EvictSet&, void* s) { return ++selects, launched(s); }
int evict_prepare() { return 0; }
int launch_evict(const EvictArgs& a, const EvictSet&, void* s)
{
    ++evictions;
    seen_state.assign(a.state, a.state + kEvictReqs);
    seen_state.insert(seen_state.end(), a.next_state, a.next_state + kEvictReqs);
    return launched(s);
}

}  // namespace leyline

namespace {

// A pool with two requests of 40 and 9 rows, or of `len0` and `len1`.
struct Fixture {
    leyline_pool_t* pool = nullptr;
    void* kv = nullptr;
    int32_t *table = nullptr, *lens_dev = nullptr, *kept = nullptr;
    float* weights = nullptr;
    int64_t lens[2];
    leyline_block_table_t bt{};
    leyline_row_weights_t w{};
    void* stream = reinterpret_cast<void*>(0x1000);

    Fixture(uint32_t flags = 0, int64_t len0 = 40, int64_t len1 = 9) : lens{len0, len1}
    {
        leyline_pool_desc_t d{};
        d.num_layers = 1;
        d.latent_dim = 512;
        d.rope_dim = 64;
        d.block_size = 4;
        d.num_pages = 30;
        d.rope_theta = 10000.0;
        d.flags = flags;
        cudaMalloc(&kv, 30 * 4 * 576 * 2);
        check(leyline_pool_create(&d, kv, &pool) == LEYLINE_OK, "creating the pool");
        check(!legacy_pending, "a pool's creation waits for its work");
        cudaMalloc((void**)&table, 2 * 12 * 4);
        cudaMalloc((void**)&lens_dev, 2 * 4);
        cudaMalloc((void**)&kept, 2 * 40 * 4);
        cudaMalloc((void**)&weights, 2 * 48 * 4);
        std::vector<int32_t> pages(13);
        check(leyline_alloc_pages(pool, 13, pages.data()) == LEYLINE_OK, "taking pages");
        bt = leyline_block_table_t{table, lens_dev, lens, 2, 12};
        w = leyline_row_weights_t{weights, 48, 48, 2};
        legacy_pending = false;
        copies_in = unordered = 0;
    }
    ~Fixture()
    {
        leyline_pool_destroy(pool);
        for (void* p : {kv, (void*)table, (void*)lens_dev, (void*)kept, (void*)weights}) cudaFree(p);
    }
};

void first_eviction()
{
    Fixture f;
    const leyline_keep_t keep{0, 30, 0, 0};
    check(leyline_evict(f.pool, &f.bt, &keep, 1, f.kept, 40, &f.w, f.stream) == LEYLINE_OK, "evicting");
    check(evictions == 1 && f.lens[0] == 30, "the eviction is enqueued");
    check(copies_in == 0, "the first eviction copies nothing by the legacy stream");
    check(unordered == 0 && !legacy_pending, "no kernel runs beside work of the legacy stream");
    for (const ListState& s : seen_state) check(s.bad == 0 && s.hole == INT_MAX, "the lists' states are ready");
}

void freed_pages()
{
    for (uint32_t flags : {0u, (uint32_t)LEYLINE_POOL_LAZY}) {
        Fixture f(flags);
        const int32_t ids[3] = {2, 0, 1};
        check(leyline_free_pages(f.pool, 3, ids) == LEYLINE_OK, "returning pages");
        check(!legacy_pending, "returned pages are in the free list when the call returns");
    }
}

void status_word()
{
    Fixture f;
    *f.pool->d_status = 8;
    check(leyline_sync_status(f.pool) == LEYLINE_ERR_DEVICE_CHECK, "the status is reported");
    check(*f.pool->d_status == 0 && !legacy_pending, "the status word is clear when the call returns");
    check(leyline_sync_status(f.pool) == LEYLINE_OK, "and stays so");
}

void empty_lists()
{
    Fixture f;
    const leyline_keep_t none[2] = {{1, 0, 0, 0}, {0, 0, 0, 0}};
    check(leyline_select_rows(f.pool, &f.bt, &f.w, none, 2, nullptr, 0, f.stream) == LEYLINE_OK, "lists of no rows have no memory");
    check(selects == 0, "and nothing is enqueued for them");
    const leyline_keep_t some{0, 1, 0, 0};
    check(leyline_select_rows(f.pool, &f.bt, &f.w, &some, 1, nullptr, 40, f.stream) == LEYLINE_ERR_INVALID_ARG, "a list of one row has");
    check(leyline_evict(f.pool, &f.bt, &some, 1, nullptr, 40, &f.w, f.stream) == LEYLINE_ERR_INVALID_ARG, "a list of one row has");
    check(f.lens[0] == 40, "a refused call changes nothing");
    const int64_t free_pages = leyline_free_page_count(f.pool);
    check(leyline_evict(f.pool, &f.bt, none, 2, nullptr, 0, &f.w, f.stream) == LEYLINE_OK, "all rows of a request can be dropped");
    check(evictions == 1 && f.lens[0] == 0 && f.lens[1] == 0, "and are");
    check(leyline_free_page_count(f.pool) == free_pages + 13, "with their pages");
    // requests without rows have no weights either
    leyline_row_weights_t no_rows{nullptr, 0, 0, 2};
    check(leyline_select_rows(f.pool, &f.bt, &no_rows, none, 2, nullptr, 0, f.stream) == LEYLINE_OK, "no weights of no rows");
    check(leyline_evict(f.pool, &f.bt, none, 2, nullptr, 0, &no_rows, f.stream) == LEYLINE_OK, "no weights of no rows");
    f.lens[0] = 5;
    check(leyline_select_rows(f.pool, &f.bt, &no_rows, none, 2, nullptr, 0, f.stream) == LEYLINE_ERR_INVALID_ARG, "rows have weights");
    no_rows = leyline_row_weights_t{nullptr, 48, 48, 2};
    check(leyline_select_rows(f.pool, &f.bt, &no_rows, none, 2, nullptr, 0, f.stream) == LEYLINE_ERR_INVALID_ARG, "rows have weights");
    check(leyline_evict(f.pool, &f.bt, none, 2, nullptr, 0, &no_rows, f.stream) == LEYLINE_ERR_INVALID_ARG, "rows have weights");
}

void idle_step()
{
    Fixture f;
    leyline_batch_t* b = nullptr;
    check(leyline_batch_create(f.pool, 2, 8, 4, &b) == LEYLINE_OK, "creating the batch");
    check(leyline_batch_plan(b, &f.bt, nullptr, 0, f.stream) == LEYLINE_OK, "a plan without tokens");
    const leyline_heads_t empty{nullptr, 0, 0};
    check(leyline_attention(b, 0, &empty, &empty, &empty, nullptr, 1.f, 0, f.stream) == LEYLINE_OK, "attention of no tokens");
    check(leyline_attention_weights(b, 0, &empty, &empty, nullptr, &f.w, 1.f, 1.f, 0, f.stream) == LEYLINE_OK, "weights of no tokens");
    const leyline_row_weights_t none{nullptr, 0, 0, 0};
    check(leyline_attention_weights(b, 0, &empty, &empty, nullptr, &none, 1.f, 1.f, 0, f.stream) == LEYLINE_OK, "weights of no tokens");
    check(weighings == 0, "nothing is enqueued");
    const leyline_chunk_t chunk{0, 1, 39, 39};
    check(leyline_batch_plan(b, &f.bt, &chunk, 1, f.stream) == LEYLINE_OK, "a plan of one token");
    leyline_heads_t q{f.kv, 4 * 512, 512};
    check(leyline_attention_weights(b, 0, &q, &q, nullptr, &f.w, 1.f, 1.f, 0, f.stream) == LEYLINE_ERR_INVALID_ARG, "a token has an lse");
    leyline_row_weights_t null = f.w;
    null.ptr = nullptr;
    check(leyline_attention_weights(b, 0, &q, &q, (float*)f.table, &null, 1.f, 1.f, 0, f.stream) == LEYLINE_ERR_INVALID_ARG, "and weights");
    check(leyline_attention_weights(b, 0, &q, &q, (float*)f.table, &f.w, 1.f, 1.f, 0, f.stream) == LEYLINE_OK && weighings == 1, "weighing it");
    check(leyline_batch_destroy(b) == LEYLINE_OK, "destroying the batch");
}

void plan_copies()
{
    Fixture f;
    const leyline_chunk_t chunks[2] = {{0, 1, 39, 39}, {1, 1, 8, 8}};
    int64_t vecs[2];
    for (int32_t room : {2, 4096}) {
        leyline_batch_t* b = nullptr;
        check(leyline_batch_create(f.pool, room, 8, 4, &b) == LEYLINE_OK, "creating the batch");
        check(leyline_batch_plan(b, &f.bt, chunks, 2, f.stream) == LEYLINE_OK, "a plan of two tokens");
        vecs[room > 2] = copied_vecs;
        check(leyline_batch_destroy(b) == LEYLINE_OK, "destroying the batch");
    }
    check(16 * (vecs[1] - vecs[0]) <= (int64_t)sizeof(ChunkDev) * 4094 + 64, "a plan copies the work of its own requests");
}

void lengths()
{
    // rows are counted past a request's end in 32 bits: by 2^14 where they are selected, by 512 where they are weighed
    const int64_t most = (int64_t)INT32_MAX - 65535;
    Fixture f;
    f.bt.max_blocks = 1 << 29;  // of 4 rows; nothing reads a table or weights here
    float* weights = reinterpret_cast<float*>((uintptr_t)1 << 40);
    device_memory[(uintptr_t)weights] = (size_t)1 << 34;
    for (int64_t len : {most, most + 1, (int64_t)INT32_MAX - 64, (int64_t)INT32_MAX}) {
        const bool taken = len <= most;
        const int before = selects + evictions;
        f.lens[0] = len;
        f.w = leyline_row_weights_t{weights, INT32_MAX, INT32_MAX, 1};
        const leyline_keep_t keep{0, 7, 1, 1};
        check((leyline_select_rows(f.pool, &f.bt, &f.w, &keep, 1, f.kept, 40, f.stream) == LEYLINE_OK) == taken, "selecting");
        if (!taken)
            check(leyline_evict(f.pool, &f.bt, &keep, 1, f.kept, 40, &f.w, f.stream) == LEYLINE_ERR_INVALID_ARG, "evicting");
        check(selects + evictions == before + taken && f.lens[0] == len, "nothing of a refused call is enqueued");
    }
    leyline_batch_t* b = nullptr;
    check(leyline_batch_create(f.pool, 2, 8, 4, &b) == LEYLINE_OK, "creating the batch");
    for (int64_t end : {most, most + 1, (int64_t)INT32_MAX - 64}) {
        const int before = weighings;
        f.lens[0] = end;
        const leyline_chunk_t chunk{0, 1, end - 1, end - 1};
        check(leyline_batch_plan(b, &f.bt, &chunk, 1, f.stream) == LEYLINE_OK, "a plan of the last row");
        const leyline_heads_t q{f.kv, 4 * 512, 512};
        const bool ok = leyline_attention_weights(b, 0, &q, &q, (float*)f.table, &f.w, 1.f, 1.f, 0, f.stream) == LEYLINE_OK;
        check(ok == (end <= most) && weighings == before + ok, "weighing");
        if (ok) check(weighed_rows <= most, "replayed plans of longer requests are left out");
    }
    check(leyline_batch_destroy(b) == LEYLINE_OK, "destroying the batch");
}

}  // namespace

int main(int argc, char** argv)
{
    const std::string name = argc > 1 ? argv[1] : "";
    if (name == "first_eviction") first_eviction();
    else if (name == "freed_pages") freed_pages();
    else if (name == "status_word") status_word();
    else if (name == "empty_lists") empty_lists();
    else if (name == "idle_step") idle_step();
    else if (name == "plan_copies") plan_copies();
    else if (name == "lengths") lengths();
    else check(false, "a case's name");
    std::printf("%s: %d failed checks\n", name.c_str(), failures);
    return failures == 0 ? 0 : 1;
}
