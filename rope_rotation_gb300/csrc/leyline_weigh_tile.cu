// leyline_weigh_tile.cu -- the weight that a batch's queries give to each cache row, on the tensor cores of sm_103a, for
// requests whose query rows of a band fit one tile of 128 (decoding): MLA rows and the grouped rows that attention takes
// in tiles.
//
//   S^T = K Q^T  [256 cache rows x up to 128 query rows],  w_s += sum over columns of exp2(S^T * scale * log2 e - lse * log2 e)
//
// lse is given, so tiles need no common maximum, and a row of the cache is read once.  By pairs of CTAs (cta_group::2): each
// has half of a tile's cache rows, of their S^T, and of the queries of all bands, which stay in shared memory while the keys
// pass through what is left of it as they come from HBM, some planes of 64 columns at a time.  With all of 128 MLA query rows
// in a CTA only 64 KB were left, too little in flight for HBM's latency; and an SM takes about 110 cycles for a TMA box
// whatever its size, so boxes of one plane of 16 rows, 72 for 128 MLA rows, bound the kernel.  The pairs take equal shares
// of 32 rows.
//
// What bounds it is HBM: 16 requests decode over some 30000 rows in 95 us with 16 heads, 97 with 64, 105 with 128 (0.88 to
// 0.79 of the measured copy rate; the products 40 us of it); rows that are copied one by one (one a page) 110.  With few rows
// it is the chain of waits of one tile, page, keys, products, sums: one request of 4096 rows 10 us, half of it the call's.
// Shares of few tiles are bound by their ends, the launch, the queries' and the first keys' arrival and the last tile's sums, some
// 20 us: 16 grouped requests of some 10000 rows, 4 bands of 128, 8 tiles a pair, 45 us, 0.55 of the copy rate, DRAM 44% busy and
// the exponentials' unit 6%; of 64000 rows 173 us (0.89), of 128000 327 (0.95), so more rows cost what a copy of them does.
// Lazy pools turn every band again: 64 decodes over some 5000 rows, one a page, 129 us.  Of 100 us over 64 x 3800 rows 10 are the turns
// (90 with counts of 0), and eager rows take 65: a tile's band comes by itself there, in a step of its own, and the warps that load wait
// for it.
//
// Roles in each CTA: warps 0-3 sum, warp 4 issues the products (in the first CTA alone), warps 5-12 load, 16 rows of a plane
// each.
#include "leyline_weigh.cuh"

namespace leyline {
namespace {

constexpr int kSumWarps = 4, kMmaWarp = kSumWarps, kLoadWarp = kMmaWarp + 1, kLoadWarps = 8;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kBuffers = 8;  // of S^T, at most

// Barriers marked (first) are used in the first CTA alone; the others in both.
struct Misc {
    unsigned long long full[kMaxStages];  // (first)
    unsigned long long empty[kMaxStages];
    unsigned long long stay_full;         // (first)
    unsigned long long stay_empty;
    unsigned long long s_full[kBuffers];
    unsigned long long s_empty[kBuffers];  // (first)
    unsigned long long drained;
    uint32_t tmem;
    int quit;
    int least[kSumWarps];
    double turns[128];
    int counts[4][kWeighKeys];  // lazy pools: pending turns of the rows whose bands are in flight
};
constexpr int kSmemBytes = kWeighSmem + (int)sizeof(Misc) + kLoadWarps * 128 * (int)sizeof(float2) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

__device__ __forceinline__ bool pair_warp_wait(uint32_t bar, uint32_t parity, Misc* m, int32_t* status)
{
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, &m->quit, status));
}

// The share of a CTA in the rows [key0, end) of a pair, the first kPairKeys of them: half, in groups of 16.
__device__ __forceinline__ Tile share_of(uint32_t rank, int key0, int end)
{
    const int keys = max(0, min(kPairKeys, end - key0)), half = min(keys, (keys + 31) / 32 * 16);
    return rank == 0 ? Tile{key0, half} : Tile{key0 + half, keys - half};
}

// Every role of both CTAs walks the pair's work in the same order (the loaders by a loop of their own): stay(u): the query
// tile u of every band is to stay; unit(t, u): a product, t of this CTA's rows, of which there may be none; tile(r, t), flush(r, t): the
// tile's sums begin, and are complete; release(): the queries are no longer used.
template <class Role>
__device__ __forceinline__ void walk(const WeighArgs& a, const Shape& s, uint32_t rank, Role& role)
{
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const long long work = a.header->weigh_stay_work, g1 = work * (pair + 1) / pairs;
    for (long long g = work * pair / pairs; g < g1;) {
        const WeighReq r = find_request(a.reqs, a.header->weigh_stay, g);
        const long long g_end = min(g1, (long long)(r.begin + (r.end + 31) / 32));
        if (!weights_hold(a, r)) {
            role.refuse();
            g = g_end;
            continue;
        }
        const ChunkDev ch = a.chunks[r.chunk];
        Unit u{ch, 0, 0, ch.n, 0, s.group, ch.n * s.group};
        role.stay(u);
        const int end = (int)min((g_end - (long long)r.begin) * 32, (long long)r.end);
        for (int key0 = (int)(g - r.begin) * 32; key0 < end; key0 += kPairKeys) {
            const Tile t = share_of(rank, key0, end);
            role.tile(r, t);
            for (u.band = 0; u.band < s.bands; ++u.band) role.unit(t, u);
            role.flush(r, t);
        }
        role.release();
        g = g_end;
    }
}

// How a tile's planes pass, a step a stage: those of the latents (whole MLA rows: and their band), then those of the bands
// of all heads, `planes` at a time; in a lazy pool the bands turned, two of a band's chunks with their low parts.
struct Steps {
    int planes, stage_bytes;
    int rows, bands;       // planes of either kind
    int row_steps, steps;  // of a tile
    int turned;            // planes of a turned step, 0: bands are not turned
    int keys;              // chunks of a band

    // Planes of step i, and the pitch of their groups of 8 rows.
    __device__ __forceinline__ int count(int i) const
    {
        if (i < row_steps) return min(planes, rows - i * planes);
        return turned > 0 ? turned : min(planes, bands - (i - row_steps) * planes);
    }
    __device__ __forceinline__ int pitch(int i) const { return (i >= row_steps && turned > 0 ? turned : planes) * kAtomBytes; }
    // Turned steps of a band, and the first of the chunks of one.
    __device__ __forceinline__ int band_steps() const { return keys > 1 ? keys / 2 : 1; }
};

__device__ __forceinline__ Steps make_steps(const WeighArgs& a, const WeighMaps& maps, const Shape& s)
{
    Steps t;
    const bool mla = a.g.rope_heads <= 1;
    t.planes = weigh_planes(a.header->weigh_box, mla);
    t.stage_bytes = weigh_stage_planes(a.header->weigh_box, mla, s.low > 0, s.keys) * kChunkBytes;
    t.keys = s.keys;
    t.turned = s.low > 0 ? turned_planes(s.keys) : 0;
    t.rows = s.latent + (maps.whole && s.low == 0 ? s.keys : 0);
    t.bands = maps.whole && s.low == 0 ? 0 : s.bands * s.keys;
    t.row_steps = (t.rows + t.planes - 1) / t.planes;
    t.steps = t.row_steps + (t.turned > 0 ? s.bands * t.band_steps() : (t.bands + t.planes - 1) / t.planes);
    return t;
}

// The buffers of S^T, used in turn: with two of them grouped rows, whose bands have a product each, waited for their sums.
// A buffer is of several accumulators, each for a part of the key's chunks: an accumulator's error grows with its steps and
// with what it has come to, most of it a loss that exponent_scale makes up for.  Before that the 36 steps of an MLA key in one took
// the weights of one token 1.2e-6 off 64 bits (2-norm, relative), next to 3 to 6e-7 in three; now three are 1.2e-7 off.  The time is
// the same: 16 decodes of 128 heads over some 30000 rows 104 us with one and with two.  A band alone, of at most 16
// steps, has one.
struct Buffers {
    int cols, chunks, parts, count;  // chunks: of a part
    int at = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ Buffers(int c, const Shape& s) : cols(c)
    {
        chunks = weigh_part(s.latent > 0, s.chunks, c);
        parts = (s.chunks + chunks - 1) / chunks;
        count = min(kBuffers, (int)kTmemCols / (c * parts));
    }
    __device__ __forceinline__ uint32_t column() const { return at * cols * parts; }
    __device__ __forceinline__ void advance()
    {
        if (++at == count) {
            at = 0;
            phase ^= 1;
        }
    }
};

// --------------------------------------------------------------------- loads --
// What a warp has asked for by cp.async (rows that TMA does not take, the bands that are to be turned) and has not arrived
// for: groups of copies, the oldest first.  They are waited for when the next ones are on their way.
constexpr int kLanding = 3;
constexpr int kQueries = 15;  // a group's kind: the queries

template <int kKeys>
struct Loader {
    KeyLoader<kLoadWarps, kKeys> keys;
    const Steps& t;
    Misc* m;
    uint32_t smem;
    int q_rows, box;
    bool ok = true;
    Ring ring;
    int uses = 0;  // of stages so far
    uint32_t stay_phase = 0;
    // (In registers, a byte for each group: what lies in local memory comes from L2, next to all of shared memory.)
    int landing = 0;
    uint32_t kinds = 0, gaps = 0;  // 16 * stage + (0: rows, 1 + 4 * first chunk + buffer of counts: bands), kQueries; uses to the next one
    int oldest_use = 0, newest_use = 0;
    int bands_read = 0;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = pair_warp_wait(bar, parity, m, keys.a.status);
        return ok;
    }

    __device__ __forceinline__ uint32_t stage_at(int stage) const { return smem + keys.s.stay_bytes + stage * t.stage_bytes; }

    // The oldest group: wait for its copies, turn them if they are bands, and arrive.
    __device__ __forceinline__ void arrive_oldest()
    {
        if (landing == 1) cp_async_wait<0>();
        else if (landing == 2) cp_async_wait<1>();
        else cp_async_wait<2>();
        __syncwarp();
        const int stage = (int)(kinds & 255) / 16, what = (int)(kinds & 15) - 1;
        const bool queries = (kinds & 15) == kQueries;
        if (what < 0 || queries) {
            fence_async_smem();
            __syncwarp();
        } else if constexpr (kKeys > 0) {
            const int c = what / 4;
            keys.turn_bands(c, c + kKeys / 2, kKeys > 1, stage_at(stage), t.turned * kAtomBytes, m->counts[what % 4] + 16 * keys.warp);
        }
        if (keys.lane == 0) keys.arrive(smem_addr(queries ? &m->stay_full : &m->full[stage]));
        --landing;
        kinds >>= 8;
        oldest_use += (int)(gaps & 255);
        gaps >>= 8;
    }
    __device__ __forceinline__ void land(int use, int what)
    {
        cp_async_commit();
        if (landing == 0) oldest_use = use;
        else gaps |= (uint32_t)(use - newest_use) << (8 * (landing - 1));
        newest_use = use;
        kinds |= (uint32_t)what << (8 * landing);
        ++landing;
    }
    __device__ __forceinline__ bool queries(Unit u)
    {
        const Shape& s = keys.s;
        if (!wait(smem_addr(&m->stay_empty), stay_phase ^ 1)) return false;
        stay_phase ^= 1;
        const uint32_t pitch = q_rows * 128;
        const int tid = 32 * keys.warp + keys.lane;
        for (u.band = 0; u.band < s.bands; ++u.band)
            for (int row = tid / 8; row < q_rows; row += 4 * kLoadWarps)
                copy_query_row(keys.a, s, u, (int)keys.rank * q_rows + row, row, tid % 8, 0, s.q_chunks,
                               smem + u.band * s.q_chunks * pitch, pitch);
        land(uses, kQueries);  // (the keys are asked for meanwhile)
        return true;
    }

    // The rows [key0, end) of a request, in the order in which the other roles walk them.
    __device__ __forceinline__ bool rows(const WeighReq& r, int key0, int end)
    {
        const Shape& s = keys.s;
        const bool eager = !keys.copied() && t.row_steps > 0;
        const int most = kKeys > 0 && keys.copied() ? 2 : kLanding;
        int step = 0;
        for (;;) {
            // Groups that are arrived for: all at the end, the oldest of `most` and those whose stages are next.  A product
            // waits for a tile's turned bands, the last of its planes, so these go on as soon as they can: where TMA brings
            // the other planes when the next tile's first are asked for (after two of them 128 us, after three 139, here 121:
            // 16 decodes of 16 heads over some 30000 rows), else one group after another while the next stage is not free
            // (64 decodes over some 5000 rows, one a page, 148 us without, here 129; rows that are not turned 84 without, 88
            // with it).
            const uint32_t empty = smem_addr(&m->empty[ring.stage]);
            while (landing > 0 && (key0 >= end || landing == most || uses - oldest_use >= s.stages ||
                                   (kKeys > 0 && (eager ? step == 1 : !__all_sync(0xffffffffu, mbar_test_cluster(empty, ring.phase ^ 1))))))
                arrive_oldest();
            if (key0 >= end) return true;
            if (step == 0) {
                keys.look_up(r, share_of(keys.rank, key0, end));
                keys.look_ahead(r, share_of(keys.rank, key0 + kPairKeys, end));
            }
            if (!wait(empty, ring.phase ^ 1)) return false;
            const uint32_t dst = stage_at(ring.stage);
            const int band_step = step - t.row_steps;
            if (kKeys > 0 && band_step >= 0) {
                const int c = band_step % t.band_steps(), band = band_step / t.band_steps(), buffer = bands_read++ & 3;
                keys.copy_bands(band, c, c + kKeys / 2, kKeys > 1, dst, t.turned * kAtomBytes, smem_addr(m->counts[buffer] + 16 * keys.warp));
                land(uses, 16 * ring.stage + 1 + 4 * c + buffer);
            } else {
                const bool in_rows = band_step < 0;
                const int p = (in_rows ? step : band_step) * t.planes;
                if (keys.copied()) {
                    keys.copy_planes(in_rows, p, t.planes, in_rows ? t.rows : t.bands, dst);
                    land(uses, 16 * ring.stage);
                } else {
                    keys.box_planes(in_rows, box, p, t.planes, dst, smem_addr(&m->full[ring.stage]));
                }
            }
            ring.advance(s.stages);
            ++uses;
            if (++step < t.steps) continue;
            step = 0;
            key0 += kPairKeys;
        }
    }

    __device__ __forceinline__ void run()
    {
        const WeighArgs& a = keys.a;
        const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
        const long long work = a.header->weigh_stay_work, g1 = work * (pair + 1) / pairs;
        for (long long g = work * pair / pairs; g < g1;) {
            const WeighReq r = find_request(a.reqs, a.header->weigh_stay, g);
            const long long g_end = min(g1, (long long)(r.begin + (r.end + 31) / 32));
            if (weights_hold(a, r)) {
                const ChunkDev ch = a.chunks[r.chunk];
                if (!queries(Unit{ch, 0, 0, ch.n, 0, keys.s.group, ch.n * keys.s.group})) return;
                if (!rows(r, (int)(g - r.begin) * 32, (int)min((g_end - (long long)r.begin) * 32, (long long)r.end))) return;
            }
            g = g_end;
        }
    }
};

// ------------------------------------------------------------------ products --
struct Issuer {
    const WeighArgs& a;
    const Shape& s;
    const Steps& t;
    Misc* m;
    uint32_t smem, tmem;
    int q_rows;
    Buffers buf;
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;
    int step = 0, plane = 0;  // of the tile: where the products have come to

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = pair_warp_wait(bar, parity, m, a.status);
        return ok;
    }
    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&) {}
    __device__ __forceinline__ void tile(const WeighReq&, const Tile&) {}
    __device__ __forceinline__ void stay(const Unit&) { wait(smem_addr(&m->stay_full), stay_phase); }
    __device__ __forceinline__ void release()
    {
        if (ok && elect_lane()) pair_commit(smem_addr(&m->stay_empty));
        __syncwarp();
        stay_phase ^= 1;
    }
    // The query chunk of a plane of a step.
    __device__ __forceinline__ int query_chunk(int at) const
    {
        if (step < t.row_steps) return step * t.planes + at;
        const int i = step - t.row_steps;
        if (t.turned == 0) return s.latent + (i * t.planes + at) % t.keys;
        // planes of a turned step: the chunks c and c + keys / 2, then their low parts, which meet the same queries
        return s.latent + i % t.band_steps() + (t.turned == 4 ? at % 2 * (t.keys / 2) : 0);
    }
    __device__ __forceinline__ void unit(const Tile&, const Unit& u)
    {
        if (!wait(smem_addr(&m->s_empty[buf.at]), buf.phase ^ 1)) return;
        uint32_t d = tmem + buf.column();  // the accumulator
        int summed = 0;                    // its chunks so far
        const uint32_t full = smem_addr(&m->s_full[buf.at]);
        buf.advance();
        const uint32_t desc = mma_desc(kPairKeys, 2 * q_rows, false, false);
        const uint32_t queries = smem + u.band * s.q_chunks * q_rows * 128;
        for (int done = 0; done < s.chunks;) {
            if (plane == 0) {
                if (!wait(smem_addr(&m->full[ring.stage]), ring.phase)) return;
                fence_async_smem();
                tcgen05_after_sync();
            }
            const int count = t.count(step), n = min(count - plane, s.chunks - done);
            if (elect_lane()) {
                const uint32_t at = smem + s.stay_bytes + ring.stage * t.stage_bytes;
                uint32_t to = d;
                for (int i = 0, c = summed; i < n; ++i) {
                    product(to, at + (plane + i) * kAtomBytes, t.pitch(step), queries + query_chunk(plane + i) * q_rows * 128, desc, c > 0);
                    if (++c < buf.chunks) continue;
                    c = 0;
                    to += buf.cols;
                }
                if (plane + n == count) pair_commit(smem_addr(&m->empty[ring.stage]));
                if (done + n == s.chunks) pair_commit(full);
            }
            __syncwarp();
            for (summed += n; summed >= buf.chunks; summed -= buf.chunks) d += buf.cols;
            done += n;
            plane += n;
            if (plane < count) continue;
            plane = 0;
            if (++step == t.steps) step = 0;
            ring.advance(s.stages);
        }
    }
};

// ---------------------------------------------------------------------- sums --
// What the columns of all bands are given lies in shared memory while their queries stay.  The warps meet at a named barrier
// then, so when the CTA gives up they go through their units without waiting, and write nothing; the status word says that
// the weights are not valid.
struct Summer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t tmem;
    float* neg;   // [bands][cols]
    int* limit;
    int cols;
    Buffers buf;
    uint32_t rank;
    int warp, lane;
    int open = 0;  // rows below it are attended to by every column
    float sum = 0.f;
    int page = -1;  // of this thread's row of the tile, and its weight before
    float before = 0.f;

    __device__ __forceinline__ void refuse()
    {
        if (threadIdx.x == 0 && rank == 0) raise_status(a.status, ST_BAD_ROW);
    }
    __device__ __forceinline__ void stay(Unit u)
    {
        const int c = threadIdx.x;
        any_of_warps<kSumWarps>(false);  // the columns before are no longer used
        int least = INT32_MAX;
        for (u.band = 0; u.band < s.bands; ++u.band) {
            const Column col = column_of(a, s, u, c);
            if (c >= cols) continue;
            neg[u.band * cols + c] = col.neg();
            limit[u.band * cols + c] = col.rows();
            if (c < u.cols) least = min(least, col.rows());
        }
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) m->least[warp] = least;
        any_of_warps<kSumWarps>(false);
        open = min(min(m->least[0], m->least[1]), min(m->least[2], m->least[3]));
    }
    __device__ __forceinline__ void release() {}

    __device__ __forceinline__ void tile(const WeighReq& r, const Tile& t)
    {
        const int row = 32 * warp + lane;
        page = -1;
        if (row >= t.keys) return;
        page = a.header->table[(long long)r.req * a.header->max_blocks + (t.key0 + row) / a.g.block_size];
        before = a.decay == 0.f ? 0.f : a.weights[r.req * a.req_stride + t.key0 + row];
    }
    __device__ __forceinline__ void unit(const Tile& t, const Unit& u)
    {
        mbar_wait_cluster(smem_addr(&m->s_full[buf.at]), buf.phase, &m->quit, a.status);
        tcgen05_after_sync();
        if (32 * warp < t.keys) {
            const uint32_t at = tmem + buf.column() + ((uint32_t)(32 * warp) << 16);
            const int n = padded(u.cols), key = t.key0 + 32 * warp + lane;
            const bool masked = t.key0 + t.keys > open;
            const float scale2 = cols > 64 ? a.scale2[1] : a.scale2[0], *l = neg + u.band * cols;
            const int* end = limit + u.band * cols;
            sum += buf.parts == 4   ? sum_columns<4>(at, n, u.cols, scale2, l, end, key, masked, cols)
                   : buf.parts == 3 ? sum_columns<3>(at, n, u.cols, scale2, l, end, key, masked, cols)
                   : buf.parts == 2 ? sum_columns<2>(at, n, u.cols, scale2, l, end, key, masked, cols)
                                    : sum_columns(at, n, u.cols, scale2, l, end, key, masked);
        }
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) cluster_arrive_smem(cluster_addr(smem_addr(&m->s_empty[buf.at]), 0));
        buf.advance();
    }

    __device__ __forceinline__ void flush(const WeighReq& r, const Tile& t)
    {
        const int row = 32 * warp + lane;
        // (the loads have raised the status for a bad page)
        if (row < t.keys && page >= 0 && page < a.g.num_pages && !*(volatile int*)&m->quit)
            a.weights[r.req * a.req_stride + t.key0 + row] = a.decay == 0.f ? sum : fmaf(a.decay, before, sum);
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
    const uint32_t rank = cluster_rank();
    wait_for_previous_grid();
    if (a.header->weigh_stay == 0) return;  // no request of the plan is for this kernel (both CTAs see the same)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&m->full[i]), 2 * kLoadWarps);
            mbar_init(smem_addr(&m->empty[i]), 1);
        }
        mbar_init(smem_addr(&m->stay_full), 2 * kLoadWarps);
        mbar_init(smem_addr(&m->stay_empty), 1);
        for (int i = 0; i < kBuffers; ++i) {
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
    const int cols = a.header->weigh_cols, q_rows = cols / 2;
    s.stay_bytes = (int)stay_bytes(s.bands, s.q_chunks, cols);
    const Steps t = make_steps(a, maps, s);
    s.stages = min(kMaxStages, (kWeighSmem - s.stay_bytes) / t.stage_bytes);
    if (warp < kMmaWarp) {
        float* columns = reinterpret_cast<float*>(base + s.bands * s.q_chunks * q_rows * 128);
        Summer role{a, s, m, tmem, columns, reinterpret_cast<int*>(columns + s.bands * cols), cols, Buffers(cols, s),
                    rank, warp, lane};
        walk(a, s, rank, role);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            Issuer role{a, s, t, m, smem, tmem, q_rows, Buffers(cols, s)};
            walk(a, s, rank, role);
            // nothing is in flight when TMEM is freed
            if (elect_lane()) pair_commit(smem_addr(&m->drained));
            __syncwarp();
            const unsigned long long t0 = global_ns();
            while (!mbar_try_cluster(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
            }
        }
    } else {
        const int w = warp - kLoadWarp;
        float2* trig = reinterpret_cast<float2*>(base + kWeighSmem + sizeof(Misc)) + 128 * w;
        Loader<kKeys> role{{a, maps, s, trig, m->turns, w, lane, rank}, t, m, smem, q_rows, a.header->weigh_box};
        role.run();
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
    const bool mla = g.rope_heads <= 1;
    for (int i = 0; maps->box > 0 && i < kWeighBoxes; ++i) {
        const int groups = maps->box / 8, planes = weigh_planes(i, mla);
        if (!make_map(encode, &maps->rows[i], base, rows, g.lat_row_vecs, (g.latent_dim + (maps->whole ? g.rope_dim : 0)) / 64, planes, groups) ||
            !make_map(encode, &maps->bands[i], base + g.rope_base_vecs, rows, g.rope_row_vecs, g.rope_vecs / 8, planes, groups))
            return (int)cudaErrorInvalidValue;
    }
    return (int)cudaFuncSetAttribute(kernel_of(g), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

int launch_weigh_tile(const WeighArgs& a, const WeighMaps& maps, int pairs, void* stream)
{
    return (int)launch_pairs(kernel_of(a.g), pairs, kThreads, kSmemBytes, (cudaStream_t)stream, a, maps);
}

}  // namespace leyline
