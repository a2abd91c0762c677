// leyline_weigh_tile.cu -- the weight that a batch's queries give to each cache row, on the tensor cores of sm_103a, where
// every request's query rows of a band fit one tile of 128 (decoding): MLA rows and the grouped rows that attention takes
// in tiles.
//
//   S^T = K Q^T  [128 cache rows x up to 128 query rows],  w_s += sum over columns of exp2(S^T * scale * log2 e - lse * log2 e)
//
// lse is given, so tiles need no common maximum, and a row of the cache is read once.  The queries of all bands stay in
// shared memory while the keys pass through a ring of chunks of 64 columns, as they come from HBM: the rest of shared
// memory, 64 KB for 128 MLA query rows and 176 KB for 16.  The CTAs take equal shares of 16 rows, one CTA an SM.
//
// Roles: warps 0-3 sum, warp 4 issues the products, warps 5-12 load, 16 rows of a chunk each.
#include "leyline_weigh.cuh"

namespace leyline {
namespace {

constexpr int kSumWarps = 4, kMmaWarp = kSumWarps, kLoadWarp = kMmaWarp + 1, kLoadWarps = 8;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr uint32_t kTmemCols = 256;  // two buffers of S^T

struct Misc {
    unsigned long long full[kMaxStages], empty[kMaxStages];
    unsigned long long stay_full, stay_empty;
    unsigned long long s_full[2], s_empty[2];
    unsigned long long drained;
    uint32_t tmem;
    int quit;
    alignas(16) float neg[2][kWeighCols];
    alignas(16) int limit[2][kWeighCols];
};
constexpr int kSmemBytes = kWeighSmem + (int)sizeof(Misc) + kLoadWarps * 128 * (int)sizeof(float2) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

// Every role walks the CTA's work in the same order: stay(r, u): the query tile u of every band is to stay; unit(r, t, u,
// end): a product, of rows below `end`; flush(r, t): the tile's sums are complete; release(): the queries are no longer used.
template <class Role>
__device__ __forceinline__ void walk(const WeighArgs& a, const Shape& s, Role& role)
{
    const long long work = a.header->weigh_work, g1 = work * (blockIdx.x + 1) / gridDim.x;
    for (long long g = work * blockIdx.x / gridDim.x; g < g1;) {
        const WeighReq r = find_request(a, g);
        const long long g_end = min(g1, (long long)(r.begin + (r.end + 15) / 16));
        if (!weights_hold(a, r)) {
            role.refuse();
            g = g_end;
            continue;
        }
        const ChunkDev ch = a.chunks[r.chunk];
        Unit u{ch, 0, 0, ch.n, 0, s.group, ch.n * s.group};
        role.stay(r, u);
        const int end = (int)min((g_end - (long long)r.begin) * 16, (long long)r.end);
        for (int key0 = (int)(g - r.begin) * 16; key0 < end; key0 += kWeighKeys) {
            const Tile t{key0, min(kWeighKeys, end - key0)};
            for (u.band = 0; u.band < s.bands; ++u.band) role.unit(r, t, u, end);
            role.flush(r, t);
        }
        role.release();
        g = g_end;
    }
}

// --------------------------------------------------------------------- loads --
template <int kKeys>
struct Loader {
    KeyLoader<kLoadWarps, kKeys, false> keys;
    Misc* m;
    uint32_t smem;
    int q_rows;
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;
    int landing = 0;  // chunks of copied rows that have been asked for and not been arrived for

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = warp_wait(bar, parity, &m->quit, keys.a.status);
        return ok;
    }

    // Arrive for chunks that have landed: all but the last `kLeft` asked for, of which the next one goes to stage ring.stage.
    template <int kLeft>
    __device__ __forceinline__ void arrive_landed()
    {
        if (landing <= kLeft) return;
        cp_async_wait<kLeft>();
        __syncwarp();
        for (; landing > kLeft; --landing) {
            const int stage = ring.stage >= landing ? ring.stage - landing : ring.stage - landing + keys.s.stages;
            if (keys.lane == 0) mbar_arrive(smem_addr(&m->full[stage]));
        }
    }

    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&) {}
    __device__ __forceinline__ void release()
    {
        if (ok) arrive_landed<0>();
    }

    __device__ __forceinline__ void stay(const WeighReq&, Unit u)
    {
        const Shape& s = keys.s;
        if (!wait(smem_addr(&m->stay_empty), stay_phase ^ 1)) return;
        stay_phase ^= 1;
        const uint32_t pitch = q_rows * 128;
        const int tid = 32 * keys.warp + keys.lane;
        for (u.band = 0; u.band < s.bands; ++u.band)
            for (int row = tid / 8; row < q_rows; row += 4 * kLoadWarps)
                copy_query_row(keys.a, s, u, row, tid % 8, 0, s.q_chunks, smem + u.band * s.q_chunks * pitch, pitch);
        cp_async_wait_all();
        __syncwarp();
        if (keys.lane == 0) mbar_arrive(smem_addr(&m->stay_full));
    }

    __device__ __forceinline__ void unit(const WeighReq& r, const Tile& t, const Unit& u, int end)
    {
        if (!ok) return;
        const Shape& s = keys.s;
        keys.look_up(r, t);
        keys.read_bands(u.band);
        const int next = t.key0 + kWeighKeys;
        const bool ahead = u.band + 1 == s.bands && next < end;
        if (ahead) keys.ask_ahead(r, next, min(kWeighKeys, end - next));
        for (int c = 0; c < s.chunks; ++c) {
            // (a stage is not waited for while more chunks are still to be arrived for than leave one free)
            if (keys.copied(c)) arrive_landed<kWeighStages - 2>();
            else arrive_landed<0>();
            if (!wait(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1)) return;
            keys.key_chunk(u.band, c, smem + s.stay_bytes + ring.stage * kChunkBytes, smem_addr(&m->full[ring.stage]));
            if (keys.copied(c)) ++landing;
            ring.advance(s.stages);
            if (c == 0 && ahead) keys.prefetch_ahead();
        }
    }
};

// ------------------------------------------------------------------ products --
struct Issuer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t smem, tmem;
    int q_rows;
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;
    int index = 0;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = warp_wait(bar, parity, &m->quit, a.status);
        return ok;
    }
    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&) {}
    __device__ __forceinline__ void stay(const WeighReq&, const Unit&) { wait(smem_addr(&m->stay_full), stay_phase); }
    __device__ __forceinline__ void release()
    {
        if (ok && elect_lane()) mma_commit(smem_addr(&m->stay_empty));
        __syncwarp();
        stay_phase ^= 1;
    }
    __device__ __forceinline__ void unit(const WeighReq&, const Tile&, const Unit& u, int)
    {
        const int buf = index & 1;
        if (!wait(smem_addr(&m->s_empty[buf]), ((index >> 1) & 1) ^ 1)) return;
        ++index;
        const uint32_t d = tmem + buf * kWeighCols, desc = mma_desc(kWeighKeys, padded(u.cols), false, false);
        for (int c = 0; c < s.chunks; ++c) {
            if (!wait(smem_addr(&m->full[ring.stage]), ring.phase)) return;
            fence_async_smem();
            tcgen05_after_sync();
            if (elect_lane()) {
                const int qc = c < s.q_chunks ? c : c - s.low;  // a band's low part meets the same queries
                product<false>(d, smem + s.stay_bytes + ring.stage * kChunkBytes,
                               smem + (u.band * s.q_chunks + qc) * q_rows * 128, desc, c > 0);
                mma_commit(smem_addr(&m->empty[ring.stage]));
                if (c + 1 == s.chunks) mma_commit(smem_addr(&m->s_full[buf]));
            }
            __syncwarp();
            ring.advance(s.stages);
        }
    }
};

// ---------------------------------------------------------------------- sums --
// The warps meet at a named barrier, so when the CTA gives up they go through their units without waiting, and write
// nothing; the status word says that the weights are not valid.
struct Summer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t tmem;
    int warp, lane;
    int index = 0;
    int at_tok = -1, at_band = -1;  // the query tile whose column this thread has
    Column col;
    float sum = 0.f;

    __device__ __forceinline__ void refuse()
    {
        if (threadIdx.x == 0) raise_status(a.status, ST_BAD_ROW);
    }
    __device__ __forceinline__ void stay(const WeighReq&, const Unit&) {}
    __device__ __forceinline__ void release() {}

    __device__ __forceinline__ void unit(const WeighReq&, const Tile& t, const Unit& u, int)
    {
        const int buf = index & 1, c = threadIdx.x, n = padded(u.cols);
        if (u.ch.tok0 != at_tok || u.band != at_band) {
            col = column_of(a, s, u, c);
            at_tok = u.ch.tok0;
            at_band = u.band;
        }
        m->neg[buf][c] = col.neg();
        m->limit[buf][c] = col.rows();
        // (and the columns are there for all warps)
        const bool masked = any_of_warps<kSumWarps>(c < u.cols && col.rows() < t.key0 + t.keys);
        mbar_wait(smem_addr(&m->s_full[buf]), (index >> 1) & 1, &m->quit, a.status);
        tcgen05_after_sync();
        if (32 * warp < t.keys)
            sum += sum_columns(tmem + buf * kWeighCols + ((uint32_t)(32 * warp) << 16), n, u.cols, a.scale * kLog2e, m->neg[buf],
                               m->limit[buf], t.key0 + 32 * warp + lane, masked);
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&m->s_empty[buf]));
        ++index;
    }

    __device__ __forceinline__ void flush(const WeighReq& r, const Tile& t)
    {
        const int row = 32 * warp + lane;
        if (row < t.keys && !*(volatile int*)&m->quit) store_weight(a, r, t.key0 + row, sum);
        sum = 0.f;
    }
};

template <int kKeys>
__global__ void __launch_bounds__(kThreads, 1) weigh_tile_kernel(const __grid_constant__ WeighArgs a,
                                                              const __grid_constant__ WeighMaps maps)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    unsigned char* base = raw + (smem - smem_addr(raw));
    Misc* m = reinterpret_cast<Misc*>(base + kWeighSmem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    wait_for_previous_grid();
    if (a.header->weigh_mode != kQueriesStay) return;  // the plan is for the other kernel
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&m->full[i]), kLoadWarps);
            mbar_init(smem_addr(&m->empty[i]), 1);
        }
        mbar_init(smem_addr(&m->stay_full), kLoadWarps);
        mbar_init(smem_addr(&m->stay_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&m->s_full[i]), 1);
            mbar_init(smem_addr(&m->s_empty[i]), kSumWarps);
        }
        mbar_init(smem_addr(&m->drained), 1);
        m->quit = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&m->tmem), kTmemCols);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = m->tmem;
    Shape s = make_shape(a, kKeys > 0);
    const int q_rows = a.header->weigh_cols;
    s.stay_bytes = s.bands * s.q_chunks * q_rows * 128;
    s.stages = min(kMaxStages, (kWeighSmem - s.stay_bytes) / kChunkBytes);
    if (warp < kMmaWarp) {
        Summer role{a, s, m, tmem, warp, lane};
        walk(a, s, role);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        Issuer role{a, s, m, smem, tmem, q_rows};
        walk(a, s, role);
        // nothing is in flight when TMEM is freed
        if (elect_lane()) mma_commit(smem_addr(&m->drained));
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
        }
    } else {
        const int w = warp - kLoadWarp;
        float2* trig = reinterpret_cast<float2*>(base + kWeighSmem + sizeof(Misc)) + 128 * w;
        Loader<kKeys> role{{a, maps, s, trig, w, lane, 0}, m, smem, q_rows};
        walk(a, s, role);
        cp_async_wait_all();
    }
    __syncthreads();
    let_loads_land(&m->quit);
    if (warp == kMmaWarp) {
        tcgen05_after_sync();
        tmem_free(tmem, kTmemCols);
    }
}

using Kernel = void (*)(WeighArgs, WeighMaps);

Kernel kernel_of(const Geometry& g)
{
    if (!(g.flags & LEYLINE_POOL_LAZY)) return weigh_tile_kernel<0>;
    return g.rope_dim == 64 ? weigh_tile_kernel<1> : g.rope_dim == 128 ? weigh_tile_kernel<2> : weigh_tile_kernel<4>;
}

}  // namespace

int weigh_tile_prepare(const Geometry& g, const void* kv, WeighMaps* maps)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return (int)cudaErrorNotSupported;
    const uint4* base = static_cast<const uint4*>(kv);
    const int64_t rows = g.num_pages * g.block_size * g.num_layers;
    maps->whole = g.rope_heads <= 1 && !(g.flags & LEYLINE_POOL_SPLIT_ROPE);
    maps->box = g.block_size % 16 == 0 ? 16 : g.block_size % 8 == 0 ? 8 : 0;
    maps->shift = -1;
    for (int k = 0; k < 31; ++k)
        if (g.block_size == 1 << k) maps->shift = k;
    const int groups = maps->box / 8;
    if (maps->box &&
        (!make_map(encode, &maps->rows, base, rows, g.lat_row_vecs, (g.latent_dim + (maps->whole ? g.rope_dim : 0)) / 64, 1, groups) ||
         !make_map(encode, &maps->bands, base + g.rope_base_vecs, rows, g.rope_row_vecs, g.rope_vecs / 8, 1, groups)))
        return (int)cudaErrorInvalidValue;
    return (int)cudaFuncSetAttribute(kernel_of(g), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

int launch_weigh_tile(const WeighArgs& a, const WeighMaps& maps, int ctas, void* stream)
{
    return (int)launch_dependent_smem(kernel_of(a.g), ctas, kThreads, kSmemBytes, (cudaStream_t)stream, a, maps);
}

}  // namespace leyline
