// leyline_weigh_pair.cu -- the weight that a batch's queries give to each cache row by pairs of CTAs (sm_103a), for requests
// whose query rows of a band do not fit one tile of 128: prompt chunks, drafts of many heads.
//
// As leyline_weigh_tile.cu, but the keys of 256 cache rows stay, 128 in each CTA, while query tiles pass, two at a time, one
// through each CTA, in products that span both (cta_group::2):
//   S^T = K Q^T  [256 x up to 256]: a CTA holds 128 cache rows, one of the two query tiles, and its rows of S^T.
// A chunk of queries is thus read into one SM for a product over two: with a query tile for each CTA alone, 64 bytes a
// cycle of each SM from L2, L2 bound the kernel at 37% of the tensor cores' rate.
//
// An item is a tile of 256 cache rows and a segment of the request's query tiles, which a pair takes in turn; where a
// request's query tiles are cut into segments a second kernel adds their sums up, in order.  Query tiles whose tokens all
// lie before an item's cache rows are left out.
//
// What bounds it is the tensor cores: 512 tokens of 128 heads over 8192 rows in 365 us back to back, 397 a call whose queries
// come from HBM, 0.80 to 0.86 of cuBLAS's rate
// for what the causal mask leaves.  The exponentials, 128 a thread and product, take nearly as long as a product and run
// beside the next one, in the other half of TMEM: a product has one accumulator, and its weights are 5e-7 off 64 bits at most
// (2-norm, relative; 1.6e-6 if exponent_scale did not make up for what it cuts off).  Two accumulators for products of half as
// many columns: 595 us.
// 64 tokens of 16 heads over 32768 rows take 37 us, 20 of them at the tensor cores' rate: 128 items are two for some of the 76
// pairs and one for others (the tensor cores 30 to 61% active, SM by SM), and each waits for its keys.
// Narrow keys are bound by the sums: 512 tokens of 32 heads on 4 bands of 128 over 8192 rows take 89 us, 18 of them at the tensor
// cores' rate and 28 at the exponentials'; a product of 8 steps is done long before the 128 columns a thread of the one before.
//
// Roles in each CTA: warps 0-3 sum the first query tile's columns, warps 4-7 the second's, warp 8 issues the products (in
// the first CTA alone), warp 9 asks for the queries (TMA boxes, one lane), warps 10-13 bring the keys, 32 rows each, and
// copy queries whose strides TMA does not take.
#include "leyline_weigh.cuh"

namespace leyline {
namespace {

constexpr int kSumWarps = 8, kMmaWarp = kSumWarps, kQueryWarp = kMmaWarp + 1, kLoadWarp = kQueryWarp + 1, kLoadWarps = 4;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kCols = 2 * kWeighCols;
constexpr uint32_t kTmemCols = 512;  // two buffers of S^T

// Barriers marked (first) are used in the first CTA alone; the others in both.
struct Misc {
    unsigned long long full[kMaxStages];  // (first)
    unsigned long long empty[kMaxStages];
    unsigned long long stay_full[kMaxChunks];  // (first)
    unsigned long long stay_empty;
    unsigned long long s_full[2];
    unsigned long long s_empty[2];  // (first)
    unsigned long long drained;
    uint32_t tmem;
    int quit;
    alignas(16) float neg[2][kCols];
    alignas(16) int limit[2][kCols];
    float half[kWeighKeys];  // sums over the second query tile's columns
    double turns[128];
    int counts[kWeighKeys];
};
constexpr int kSmemBytes = kWeighSmem + (int)sizeof(Misc) + kLoadWarps * 128 * (int)sizeof(float2) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

// Every role of both CTAs walks the pair's work in the same order; t is the tile of this CTA, whose rows may all lie behind
// the request's end:
//   stay(r, t, band)     the keys of the tile and band are to stay; release(): they are no longer used
//   unit(r, t, u, next)  a product, of the query tiles u and next (which may have no columns)
//   flush(r, t, part)    the tile's sums are complete (part < 0), or those of a segment are
template <class Role>
__device__ __forceinline__ void walk(const WeighArgs& a, const Shape& s, uint32_t rank, Role& role)
{
    const long long work = a.header->weigh_work;
    const int seg = a.header->weigh_seg, pairs = gridDim.x / 2;
    for (long long i = blockIdx.x / 2; i < work; i += pairs) {
        const WeighReq r = find_request(a.reqs + a.header->weigh_stay, a.header->weigh_reqs - a.header->weigh_stay, i);
        if (!weights_hold(a, r)) {
            role.refuse();
            continue;
        }
        const int local = (int)(i - r.begin), tile = local / r.segs;
        const long long first = (long long)tile * kPairKeys;
        const int key0 = (int)first + (int)rank * kWeighKeys;
        const Tile t{key0, (int)max(0ll, min((long long)kWeighKeys, (long long)r.end - key0))};
        const int u0 = (local - tile * r.segs) * seg, u1 = min(u0 + seg, r.units);
        const int per_band = r.units / s.bands;
        for (int band = u0 / per_band; band * per_band < u1; ++band) {
            const int lo = max(u0 - band * per_band, 0), hi = min(u1 - band * per_band, per_band);
            bool loaded = false;
            int at = 0;  // units of the chunks before
            for (int c = r.chunk; c >= 0 && at < hi;) {
                const ChunkDev ch = a.chunks[c];
                const int tiles = (ch.n + s.tokens - 1) / s.tokens * s.blocks, units = (tiles + 1) / 2;
                // query tiles whose last token lies before the cache rows attend to none of them
                const int skip = a.prefix ? (first < ch.start ? 0 : units)
                                          : (int)min((long long)units, max(0ll, (first - (long long)ch.start) / s.tokens * s.blocks / 2));
                auto query_tile = [&](int x) {
                    if (x >= tiles) return Unit{ch, band, ch.n, 0, 0, s.heads, 0};
                    const int tok = x / s.blocks * s.tokens, toks = min(s.tokens, ch.n - tok);
                    const int head0 = x % s.blocks * kWeighCols, heads = min(s.heads, s.group - head0);
                    return Unit{ch, band, tok, toks, head0, heads, toks * heads};
                };
                for (int x = max(lo - at, skip); x < min(hi - at, units); ++x) {
                    if (!loaded) role.stay(r, t, band);
                    loaded = true;
                    role.unit(r, t, query_tile(2 * x), query_tile(2 * x + 1));
                }
                at += units;
                c = ch.next;
            }
            if (loaded) role.release();
        }
        role.flush(r, t, r.segs > 1 ? r.part + local : -1);
    }
}

// Columns of a product that each of its two query tiles has.
__device__ __forceinline__ int tile_cols(const Unit& u, const Unit& next) { return padded(max(u.cols, next.cols)); }

__device__ __forceinline__ bool pair_warp_wait(uint32_t bar, uint32_t parity, Misc* m, int32_t* status)
{
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, &m->quit, status));
}

// --------------------------------------------------------------------- loads --
// One lane, the queries of this CTA's query tile of each product: their bytes of both CTAs are counted in the first, whose
// lane alone arrives, for the warps that copy them otherwise.  It waits for the stages in turn and asks for each of them,
// so that a parity always means the use before.
struct QueryLoader {
    const WeighArgs& a;
    const QueryMaps& maps;
    const Shape& s;
    Misc* m;
    uint32_t smem, rank;
    bool ok = true;
    Ring ring;

    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void stay(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void release() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void unit(const WeighReq&, const Tile&, const Unit& u0, const Unit& u1)
    {
        if (!ok) return;
        const Unit& u = rank == 0 ? u0 : u1;
        const uint32_t bytes = s.heads * s.tokens * 128;
        for (int c = 0; c < s.q_chunks; ++c) {
            ok = mbar_wait_cluster(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1, &m->quit, a.status);
            if (!ok) return;
            const uint32_t full = smem_addr(&m->full[ring.stage]);
            if (rank == 0) {
                mbar_expect_tx(full, 2 * bytes);
                mbar_arrive_n(full, 2 * kLoadWarps - 1);
            }
            const bool latent = c < s.latent;
            pair_box3(smem + s.stay_bytes + ring.stage * kChunkBytes, latent ? &maps.latent : &maps.band,
                      64 * (latent ? c : c - s.latent), u.band * s.group + u.head0, u.ch.tok0 + u.tok, cluster_addr(full, 0));
            ring.advance(s.stages);
        }
    }
};

template <int kKeys>
struct Loader {
    KeyLoader<kLoadWarps, kKeys> keys;
    Misc* m;
    uint32_t smem;
    int* counts;  // lazy pools: pending turns of this warp's rows
    bool copies;  // queries as well
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = pair_warp_wait(bar, parity, m, keys.a.status);
        return ok;
    }
    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void release() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&, int) {}

    __device__ __forceinline__ void stay(const WeighReq& r, const Tile& t, int band)
    {
        const Shape& s = keys.s;
        if (!wait(smem_addr(&m->stay_empty), stay_phase ^ 1)) return;
        stay_phase ^= 1;
        keys.look_up(r, t);
        // the band's chunks lie behind the latent's, in the order in which they pass in leyline_weigh_tile.cu: two of them
        // (one, if it has no more) and their low parts, groups of 8 rows of all of these together
        const int stored = kKeys > 0 ? s.latent : s.chunks;
        constexpr bool kTwo = kKeys > 1;
        constexpr int kPlanes = turned_planes(kKeys > 0 ? kKeys : 1), kPitch = kPlanes * kAtomBytes;
        if (kKeys > 0)
            for (int c = 0; c < (kTwo ? kKeys / 2 : 1); ++c)
                keys.copy_bands(band, c, c + kKeys / 2, kTwo, smem + (s.latent + c * kPlanes) * kChunkBytes, kPitch, smem_addr(counts));
        for (int c = 0; c < stored; ++c) {
            const bool in_rows = c < s.latent || (kKeys == 0 && keys.maps.whole);
            const int plane = in_rows ? c : band * s.keys + c - s.latent;
            const uint32_t dst = smem + c * kChunkBytes;
            if (keys.copied()) keys.copy_planes(in_rows, plane, 1, plane + 1, dst);
            else keys.box_planes(in_rows, 0, plane, 1, dst, smem_addr(&m->stay_full[c]));
        }
        if (kKeys == 0 && !keys.copied()) return;
        cp_async_wait_all();
        __syncwarp();
        if (kKeys > 0)
            for (int c = 0; c < (kTwo ? kKeys / 2 : 1); ++c)
                keys.turn_bands(c, c + kKeys / 2, kTwo, smem + (s.latent + c * kPlanes) * kChunkBytes, kPitch, counts);
        else fence_async_smem();
        __syncwarp();
        if (keys.lane == 0)
            for (int c = keys.copied() ? 0 : stored; c < s.chunks; ++c) keys.arrive(smem_addr(&m->stay_full[c]));
    }

    __device__ __forceinline__ void unit(const WeighReq&, const Tile&, const Unit& u0, const Unit& u1)
    {
        if (!ok || !copies) return;
        const Shape& s = keys.s;
        const Unit& u = keys.rank == 0 ? u0 : u1;
        const int rows = tile_cols(u0, u1), tid = 32 * keys.warp + keys.lane;
        for (int c = 0; c < s.q_chunks; ++c) {
            if (!wait(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1)) return;
            for (int row = tid / 8; row < rows; row += 4 * kLoadWarps)
                copy_query_row(keys.a, s, u, row, row, tid % 8, c, c + 1, smem + s.stay_bytes + ring.stage * kChunkBytes, 0);
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (keys.lane == 0) keys.arrive(smem_addr(&m->full[ring.stage]));
            ring.advance(s.stages);
        }
    }
};

// ------------------------------------------------------------------ products --
struct Issuer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t smem, tmem;
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;
    bool stay_ready = false;
    int index = 0;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = pair_warp_wait(bar, parity, m, a.status);
        return ok;
    }
    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void stay(const WeighReq&, const Tile&, int) { stay_ready = false; }
    __device__ __forceinline__ void release()
    {
        if (ok && elect_lane()) pair_commit(smem_addr(&m->stay_empty));
        __syncwarp();
        stay_phase ^= 1;
    }
    __device__ __forceinline__ void unit(const WeighReq&, const Tile&, const Unit& u, const Unit& next)
    {
        const int buf = index & 1;
        if (!wait(smem_addr(&m->s_empty[buf]), ((index >> 1) & 1) ^ 1)) return;
        ++index;
        const uint32_t d = tmem + buf * kCols, desc = mma_desc(2 * kWeighKeys, 2 * tile_cols(u, next), false, false);
        for (int c = 0; c < s.q_chunks; ++c) {
            const bool band = s.low > 0 && c >= s.latent;
            // chunks of a band: c = latent + b is plane b / half of the pair of chunks b % half
            const int b = c - s.latent, half = max(s.low / 2, 1), planes = turned_planes(s.low);
            const uint32_t turned = smem + (s.latent + b % half * planes) * kChunkBytes + b / half * kAtomBytes;
            if (!stay_ready) {  // (a band's chunks and low parts become ready together)
                if (!wait(smem_addr(&m->stay_full[c]), stay_phase)) return;
                if (band && !wait(smem_addr(&m->stay_full[c + s.low]), stay_phase)) return;
            }
            if (!wait(smem_addr(&m->full[ring.stage]), ring.phase)) return;
            fence_async_smem();
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t at = smem + s.stay_bytes + ring.stage * kChunkBytes;
                if (band) {
                    product(d, turned, planes * kAtomBytes, at, desc, c > 0);
                    product(d, turned + planes / 2 * kAtomBytes, planes * kAtomBytes, at, desc, true);  // its low part
                } else {
                    product(d, smem + c * kChunkBytes, kAtomBytes, at, desc, c > 0);
                }
                pair_commit(smem_addr(&m->empty[ring.stage]));
                if (c + 1 == s.q_chunks) pair_commit(smem_addr(&m->s_full[buf]));
            }
            __syncwarp();
            ring.advance(s.stages);
        }
        stay_ready = true;
    }
};

// ---------------------------------------------------------------------- sums --
// A unit is summed when the next one comes, whose lse are on their way by then.  The warps meet at a named barrier, so
// when the CTA gives up they go through their units without waiting, and write nothing; the status word says that the
// weights are not valid.
struct Summer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t tmem, rank;
    int warp, lane;
    int index = 0;  // of the unit to be summed
    bool waiting = false, cut = false;
    int n = 0, cols = 0, key0 = 0, keys = 0;
    float sum = 0.f;

    __device__ __forceinline__ void refuse()
    {
        if (threadIdx.x == 0 && rank == 0) raise_status(a.status, ST_BAD_ROW);
    }
    __device__ __forceinline__ void stay(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void release() {}

    __device__ __forceinline__ void unit(const WeighReq&, const Tile& t, const Unit& u0, const Unit& u1)
    {
        const bool second = warp >= kSumWarps / 2;
        const int c = threadIdx.x % kWeighCols, width = tile_cols(u0, u1);
        const Unit& u = second ? u1 : u0;
        const Column col = column_of(a, s, u, c);
        if (waiting) add();
        if (c < width) {
            m->neg[index & 1][(second ? width : 0) + c] = col.neg();
            m->limit[index & 1][(second ? width : 0) + c] = col.rows();
        }
        n = width;
        cols = u.cols;
        key0 = t.key0;
        keys = t.keys;
        cut = c < u.cols && col.rows() < key0 + keys;  // rows of the tile that this thread's column does not attend to
        waiting = true;
    }

    __device__ __forceinline__ void add()
    {
        const int buf = index & 1, quarter = warp & 3, from = warp < kSumWarps / 2 ? 0 : n;
        const bool masked = any_of_warps<kSumWarps>(cut);  // (and the columns are there for all warps)
        mbar_wait_cluster(smem_addr(&m->s_full[buf]), (index >> 1) & 1, &m->quit, a.status);
        tcgen05_after_sync();
        if (32 * quarter < keys && cols > 0)
            sum += sum_columns(tmem + buf * kCols + ((uint32_t)(32 * quarter) << 16) + from, padded(cols), cols, a.scale2[2],
                               m->neg[buf] + from, m->limit[buf] + from, key0 + 32 * quarter + lane, masked);
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) cluster_arrive_smem(cluster_addr(smem_addr(&m->s_empty[buf]), 0));
        ++index;
        waiting = false;
    }

    __device__ __forceinline__ void flush(const WeighReq& r, const Tile& t, int part)
    {
        if (waiting) add();
        const int row = 32 * (warp & 3) + lane;
        if (warp >= kSumWarps / 2) m->half[row] = sum;
        any_of_warps<kSumWarps>(false);
        const float got = sum + (warp < kSumWarps / 2 ? m->half[row] : 0.f);
        sum = 0.f;
        any_of_warps<kSumWarps>(false);  // before the other halves are written again
        if (warp >= kSumWarps / 2 || row >= t.keys || *(volatile int*)&m->quit) return;
        if (part >= 0) a.part[(long long)part * kPairKeys + rank * kWeighKeys + row] = got;
        else store_weight(a, r, t.key0 + row, got);
    }
};

template <int kKeys>
__global__ void __launch_bounds__(kThreads, 1) weigh_pair_kernel(const __grid_constant__ WeighArgs a,
                                                              const __grid_constant__ WeighMaps maps,
                                                              const __grid_constant__ QueryMaps queries)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    unsigned char* base = raw + (smem - smem_addr(raw));
    Misc* m = reinterpret_cast<Misc*>(base + kWeighSmem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    wait_for_previous_grid();
    if (a.header->weigh_work == 0) return;  // no request of the plan is for this kernel (both CTAs see the same)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&m->full[i]), 2 * kLoadWarps);  // both CTAs' copying warps, or the asking lane for as many
            mbar_init(smem_addr(&m->empty[i]), 1);
        }
        for (int i = 0; i < kMaxChunks; ++i) mbar_init(smem_addr(&m->stay_full[i]), 2 * kLoadWarps);
        mbar_init(smem_addr(&m->stay_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&m->s_full[i]), 1);
            mbar_init(smem_addr(&m->s_empty[i]), 2 * kSumWarps);
        }
        mbar_init(smem_addr(&m->drained), 1);
        m->quit = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (kKeys > 0) load_turns(a, 32 * kKeys, m->turns);
    if (warp == kMmaWarp) pair_tmem_alloc(smem_addr(&m->tmem), kTmemCols);
    tcgen05_before_sync();
    __syncthreads();
    cluster_sync();
    tcgen05_after_sync();
    const uint32_t tmem = m->tmem;
    Shape s = make_shape(a, kKeys > 0);
    s.stay_bytes = s.chunks * kChunkBytes;
    s.stages = min(kMaxStages, (kWeighSmem - s.stay_bytes) / kChunkBytes);
    if (warp < kMmaWarp) {
        Summer role{a, s, m, tmem, rank, warp, lane};
        walk(a, s, rank, role);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            Issuer role{a, s, m, smem, tmem};
            walk(a, s, rank, role);
            // nothing is in flight when TMEM is freed
            if (elect_lane()) pair_commit(smem_addr(&m->drained));
            __syncwarp();
            const unsigned long long t0 = global_ns();
            while (!mbar_try_cluster(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
            }
        }
    } else if (warp == kQueryWarp) {
        if (queries.usable && elect_lane()) {
            QueryLoader role{a, queries, s, m, smem, rank};
            walk(a, s, rank, role);
        }
        __syncwarp();
    } else {
        const int w = warp - kLoadWarp;
        float2* trig = reinterpret_cast<float2*>(base + kWeighSmem + sizeof(Misc)) + 128 * w;
        Loader<kKeys> role{{a, maps, s, trig, m->turns, w, lane, rank}, m, smem, m->counts + 32 * w, !queries.usable};
        walk(a, s, rank, role);
        cp_async_wait_all();
    }
    __syncthreads();
    let_loads_land(&m->quit);
    // neither CTA leaves while the other may still reach its shared memory, or a product its TMEM
    cluster_sync();
    if (warp == kMmaWarp) {
        tcgen05_after_sync();
        pair_tmem_free(tmem, kTmemCols);
    }
}

// Sums of requests whose query tiles were cut into segments: a CTA for a tile of cache rows, the segments in order.
__global__ void __launch_bounds__(kPairKeys) join_weights_kernel(const __grid_constant__ WeighArgs a)
{
    wait_for_previous_grid();
    const int n = a.header->weigh_reqs - a.header->weigh_stay;
    const WeighReq* reqs = a.reqs + a.header->weigh_stay;
    for (int i = blockIdx.x; i < a.header->weigh_tiles; i += gridDim.x) {
        int lo = 0, hi = n - 1;  // the last request whose cut tiles begin at or before this one has it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (reqs[mid].tile <= i) lo = mid;
            else hi = mid - 1;
        }
        const WeighReq r = reqs[lo];
        const int tile = i - r.tile;
        const long long key = (long long)tile * kPairKeys + threadIdx.x;
        if (key >= r.end || !weights_hold(a, r)) continue;
        const float* p = a.part + ((long long)r.part + (long long)tile * r.segs) * kPairKeys + threadIdx.x;
        float sum = 0.f;
        for (int k = 0; k < r.segs; ++k) sum += p[k * kPairKeys];
        store_weight(a, r, (int)key, sum);
    }
}

using Kernel = void (*)(WeighArgs, WeighMaps, QueryMaps);

Kernel kernel_of(const Geometry& g)
{
    if (!(g.flags & LEYLINE_POOL_LAZY)) return weigh_pair_kernel<0>;
    return g.rope_dim == 64 ? weigh_pair_kernel<1> : g.rope_dim == 128 ? weigh_pair_kernel<2> : weigh_pair_kernel<4>;
}

// Map of the queries `q` of `tokens` tokens, in boxes of 64 columns, `box_heads` heads and box_tokens tokens.  False: it
// cannot be had (axes that stand still), and the queries are copied a row at a time.
bool query_map(CUtensorMap* map, const HeadsView& q, int dim, int heads, int64_t tokens, int box_heads, int box_tokens)
{
    static const EncodeTiled encode = encode_tiled();
    // the stride of an axis of one entry says nothing
    const cuuint64_t head = heads > 1 ? 2 * (cuuint64_t)q.head_stride : 2 * (cuuint64_t)dim;
    const cuuint64_t token = tokens > 1 ? 2 * (cuuint64_t)q.token_stride : head * heads;
    if (!encode || head == 0 || token == 0) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens}, strides[2] = {head, token};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, steps[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q.ptr, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int weigh_pair_prepare(const Geometry& g)
{
    return (int)cudaFuncSetAttribute(kernel_of(g), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

int launch_weigh_pair(const WeighArgs& a, const WeighMaps& maps, int64_t tokens, int pairs, int joins, void* stream)
{
    const Geometry& g = a.g;
    const int group = a.q_heads / std::max(g.rope_heads, 1), heads = std::min(group, kWeighCols), toks = weigh_tokens(group);
    QueryMaps queries{};
    queries.usable = query_map(&queries.band, a.q_rope, g.rope_dim, a.q_heads, tokens, heads, toks) &&
                     (g.rope_heads > 1 || query_map(&queries.latent, a.q_latent, g.latent_dim, a.q_heads, tokens, heads, toks));
    cudaError_t e = launch_pairs(kernel_of(g), pairs, kThreads, kSmemBytes, (cudaStream_t)stream, a, maps, queries);
    if (e == cudaSuccess && joins > 0) e = launch_dependent(join_weights_kernel, joins, kPairKeys, (cudaStream_t)stream, a);
    return (int)e;
}

}  // namespace leyline
