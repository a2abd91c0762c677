// leyline_attention_mla.cu -- attention over MLA rows (latent 512, one 64-wide band) on the tensor
// cores of sm_103a.
//
// Rows are shared by all heads, so the (token, head) pairs of a chunk form the rows of one matrix
// product: per tile of 64 query rows and 64 cache rows
//   S   = Q K^T   [64 x 64],   K = [latent | band], 576 wide
//   O^T = V^T P^T [512 x 64],  V = the latent, the same bytes of shared memory
// with P = exp2(S * scale * log2 e - m).  O is kept transposed: its 512 value dimensions lie in the
// 128 TMEM lanes, 4 blocks of 64 columns, so a cache tile is loaded once, as rows, and serves as
// the K-major operand of S and as the MN-major operand of O^T.
//
// One persistent CTA per SM takes the contiguous run of items the plan gave it.  Roles:
//   warps 0-3  softmax: S from TMEM, running maximum and sum (fp32), P to shared memory, output
//   warp 4     issues the MMAs (one lane)
//   warp 5     loads cache tiles through the block table (TMA, 16 or 8 rows of a page at a time)
//   warps 6-9  copy the queries (cp.async: any strides), the cache tiles that TMA does not take (block
//              sizes that 8 does not divide; tiles that end inside, whose other rows are zeroed, since
//              they meet weights of 0 in the product with V), and in a lazy pool turn the bands
// In a lazy pool the band of each row is turned by its pending count on the way, in fp32, and goes
// to shared memory as the sum of two bf16 values: the scores then carry the turn to 2^-17, not to the
// 2^-9 of one bf16 rounding, which the other rows do not have either.
//
// A cache tile in shared memory is 8 groups of 8 rows; a group holds the rows' 64-wide column chunks one
// after another (latent 0..7, band, lazy pools: the band's low part), 8 rows x 128 bytes each, swizzled.
// That is what one TMA box of whole rows writes (columns, rows of a group, chunks, groups), and its
// strides serve both operands.  Smaller boxes, a chunk of 16 rows at a time, took 100 cycles of issue each, 36
// a tile, and bound the kernel.
// The maximum is only raised (and O rescaled) when a row's scores exceed it by 2^8: until then the
// weights are at most 2^8, and sums and products are fp32.
#include "leyline_batch.h"
#include "leyline_tcgen05.cuh"

namespace leyline {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kSoftmaxWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kCopyWarps = 4;
constexpr int kCopyThreads = 32 * kCopyWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + 2 + kCopyWarps);

constexpr int kLatentChunks = 8;
constexpr int kAtomBytes = 1024;                     // 8 rows x 128 bytes
constexpr int kStages = 2;
constexpr int kSteps = kAttnKeys / 16;               // steps of 16 cache rows, in which PV frees a stage

// Shared memory of a pool kind: query rows of a tile, column chunks of a cache row.
template <bool kLazy>
struct Smem {
    static constexpr int rows = kLazy ? kAttnRowsLazy : kAttnRows;
    static constexpr int chunks = kLazy ? 10 : 9;
    static constexpr int group_bytes = chunks * kAtomBytes;
    static constexpr int stage_bytes = kAttnKeys / 8 * group_bytes;
    static constexpr int q_chunk_bytes = rows * 128;  // queries: 9 chunks of `rows` rows
    static constexpr int q = 0;
    static constexpr int stage = q + 9 * q_chunk_bytes;
    static constexpr int p = stage + kStages * stage_bytes;
    static constexpr int misc = p + rows * 128;
};

struct Misc {
    unsigned long long full[kStages];
    unsigned long long empty[kStages][kSteps];
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2];
    unsigned long long p_ready, pv_done, drained;
    uint32_t tmem;
    int quit;
    float factor[kAttnRows];              // rescale, then 1 / l
    float2 trig[kCopyWarps][32];          // lazy pools: cos, sin of the last pending count
};
template <bool kLazy>
constexpr int kSmemBytes = Smem<kLazy>::misc + (int)sizeof(Misc) + 1024;  // and room to align the start
static_assert(kSmemBytes<false> <= 232448 && kSmemBytes<true> <= 232448, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // 4 blocks of 64 columns
constexpr uint32_t kTmemS = 256;  // 2 buffers of 64 columns

constexpr float kRaise = 8.f;
constexpr unsigned long long kDrainTime = 1000000ull;  // 1 ms: longer than any copy in flight takes

// The item as every role sees it.
struct Work {
    AttnItem it;
    ChunkDev ch;
    int tiles;      // cache tiles
    long long end;  // cache rows [key0, end) are loaded
};

__device__ __forceinline__ Work load_work(const AttnArgs& a, int i)
{
    Work w;
    w.it = a.items[i];
    w.ch = a.chunks[w.it.chunk];
    w.end = min((long long)w.it.key1, a.prefix ? (long long)w.ch.start : (long long)w.it.key1);
    w.tiles = w.end > w.it.key0 ? (int)((w.end - w.it.key0 + kAttnKeys - 1) / kAttnKeys) : 0;
    return w;
}

__device__ __forceinline__ int padded_rows(int rows) { return (rows + 15) & ~15; }

// -------------------------------------------------------------------- loads --
// The stages in turn, and the parity of their current use.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ void advance()
    {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// A cache row's page (as the table has it) and its row in the page; nothing is loaded past `end`.
struct PageOf {
    int page, off;
    bool in;
};

__device__ __forceinline__ PageOf page_of(const AttnArgs& a, const MlaMaps& maps, const Work& w, const int32_t* table_row,
                                          long long pos)
{
    const unsigned u = (unsigned)pos, B = (unsigned)a.g.block_size;
    const unsigned blk = maps.shift >= 0 ? u >> maps.shift : u / B;
    PageOf p{-1, (int)(u - blk * B), pos < w.end};
    if (p.in) p.page = table_row[blk];
    return p;
}

// Its row in the tensor maps (of all layers' rows); -8 (a box there holds no row of the tensor and loads
// zeros) past the end and for a bad page.
__device__ __forceinline__ int map_row(const AttnArgs& a, const PageOf& p)
{
    if (p.page >= 0 && p.page < a.g.num_pages)
        return (int)(((long long)a.layer * a.g.num_pages + p.page) * a.g.block_size + p.off);
    if (p.in) raise_status(a.status, ST_BAD_PAGE);
    return -8;
}

// False (for the whole warp) when the CTA has given up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, Misc* m, int32_t* status)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, &m->quit, status));
}

// Whether TMA takes the tile at `key` (of its latents, in a lazy pool).
__device__ __forceinline__ bool by_box(const MlaMaps& maps, const Work& w, long long key)
{
    return maps.box > 0 && key + kAttnKeys <= w.end;
}

template <bool kLazy>
__device__ __forceinline__ void load_tiles(const AttnArgs& a, const MlaMaps& maps, Misc* m, uint32_t smem)
{
    using S = Smem<kLazy>;
    const int lane = threadIdx.x & 31;
    const bool split = (a.g.flags & LEYLINE_POOL_SPLIT_ROPE) != 0;
    const bool wide = maps.box == 16;  // lanes 0..3: the tile's boxes of 16 rows; else lanes 0..7: of 8
    const int my_row = wide ? 16 * (lane & 3) : 8 * (lane & 7);
    Ring ring;
    bool go = true;
    for (int i = a.cta_begin[blockIdx.x]; go && i < a.cta_begin[blockIdx.x + 1]; ++i) {
        const Work w = load_work(a, i);
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        const bool paged = maps.box > 0;
        // the tile's boxes as indices of groups of 8 rows, found while the tile before is loaded
        int y[8];
        PageOf next{};
        auto resolve = [&] {
            const int mine = map_row(a, next) >> 3;  // a box that is not loaded: -1, or -2 where it has two groups
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(0xffffffffu, mine < 0 && wide ? -2 : mine, k);
        };
        if (paged && by_box(maps, w, w.it.key0)) {
            next = page_of(a, maps, w, table_row, w.it.key0 + my_row);
            resolve();
        }
        for (int t = 0; go && t < w.tiles; ++t) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            const uint32_t full = smem_addr(&m->full[ring.stage]);
            const uint32_t dst = smem + S::stage + ring.stage * S::stage_bytes;
            const bool more = paged && t + 1 < w.tiles && by_box(maps, w, key + kAttnKeys);
            if (more) next = page_of(a, maps, w, table_row, key + kAttnKeys + my_row);  // in flight meanwhile
            if (!by_box(maps, w, key)) {  // the copy warps' tile: only this warp's arrival
                go = warp_wait(smem_addr(&m->empty[ring.stage][kSteps - 1]), ring.phase ^ 1, m, a.status);
                if (go && lane == 0) mbar_arrive(full);
                ring.advance();
                continue;
            }
#pragma unroll
            for (int step = 0; step < kSteps; ++step) {
                go = go && warp_wait(smem_addr(&m->empty[ring.stage][step]), ring.phase ^ 1, m, a.status);
                if (!go) break;
                if (elect_lane()) {
                    if (step == 0) mbar_expect_tx(full, 8 * (kLazy ? 8 : 9) * kAtomBytes);
                    const uint32_t at = dst + 2 * step * S::group_bytes;
                    if (wide && !split && !kLazy) {
                        tma_box4(at, &maps.rows, y[step], full);
                    } else if (wide) {
                        // a group's chunks are fewer than its room: a box for each group
                        for (int k = 0; k < 2; ++k) {
                            tma_box4(at + k * S::group_bytes, &maps.rows, y[step] + k, full);
                            if (split && !kLazy)
                                tma_box3(at + k * S::group_bytes + 8 * kAtomBytes, &maps.bands, y[step] + k, full);
                        }
                    } else {
                        for (int k = 0; k < 2; ++k) {
                            tma_box4(at + k * S::group_bytes, &maps.rows, y[2 * step + k], full);
                            if (split && !kLazy)
                                tma_box3(at + k * S::group_bytes + 8 * kAtomBytes, &maps.bands, y[2 * step + k], full);
                        }
                    }
                }
                __syncwarp();
            }
            if (more) resolve();
            ring.advance();
        }
    }
    if (go) return;  // every load has been waited for by the MMAs
    // The CTA gives up: what is still in flight must land before it ends.  A stage's barrier may lack the copy
    // warps' arrivals, so the loads are waited for by time: none takes as long as the limit.
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < kDrainTime) {
    }
}

// ------------------------------------------------------------------- copies --
__device__ __forceinline__ void store(uint32_t at, const uint4& y)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}

template <bool kLazy>
struct Copier {
    using S = Smem<kLazy>;
    const AttnArgs& a;
    const MlaMaps& maps;
    Misc* m;
    uint32_t smem;
    int tid, v, r0;  // 16-byte chunk of a 128-byte row segment, first row
    int trig_count;  // pending count whose cos / sin this warp's slice holds
    bool trig_valid;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, m, a.status); }

    // This lane's 8 values of a row's band, turned by the row's pending count, as hi + lo (all 32 lanes; the 8
    // lanes of a row share `pend`).
    __device__ __forceinline__ void turned(const uint4& x, int pend, uint4& hi, uint4& lo)
    {
        const bool bf16 = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        const int lane = tid & 31;
        unsigned todo = __ballot_sync(0xffffffffu, pend != 0);
        const uint4 other = shfl_xor_vec(x, 4);
        hi = x;
        lo = make_uint4(0, 0, 0, 0);
        while (todo) {  // once per distinct count among the warp's rows
            const int count = __shfl_sync(0xffffffffu, pend, __ffs(todo) - 1);
            float2* cs = m->trig[tid / 32];
            if (!trig_valid || trig_count != count) {
                __syncwarp();
                float c, s;
                pending_trig(count, a.turn, 32, lane, bf16, c, s);
                cs[lane] = make_float2(c, s);
                __syncwarp();
                trig_valid = true;
                trig_count = count;
            }
            if (pend == count) {
                const uint32_t *xw = reinterpret_cast<const uint32_t*>(&x), *ow = reinterpret_cast<const uint32_t*>(&other);
                uint32_t *hw = reinterpret_cast<uint32_t*>(&hi), *lw = reinterpret_cast<uint32_t*>(&lo);
                const bool half_split = a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = bf16_lo(xw[k]), x1 = bf16_hi(xw[k]);
                    float r0, r1;
                    if (half_split) {  // this lane's half of pairs 8 (v & 3) + 2k, + 1: x' for v < 4, else y'
                        const float2 t0 = cs[8 * (v & 3) + 2 * k], t1 = cs[8 * (v & 3) + 2 * k + 1];
                        const float sgn = v < 4 ? -1.f : 1.f;
                        const float y0 = bf16_lo(ow[k]), y1 = bf16_hi(ow[k]);
                        if (bf16) {
                            r0 = round_bf16(x0 * t0.x) + sgn * round_bf16(y0 * t0.y);
                            r1 = round_bf16(x1 * t1.x) + sgn * round_bf16(y1 * t1.y);
                        } else {
                            r0 = fmaf(x0, t0.x, sgn * (y0 * t0.y));
                            r1 = fmaf(x1, t1.x, sgn * (y1 * t1.y));
                        }
                    } else {  // pair 4v + k
                        const float2 t = cs[4 * v + k];
                        if (bf16) turn_bf16(x0, x1, t.x, t.y, r0, r1);
                        else turn_fp32(x0, x1, t.x, t.y, r0, r1);
                    }
                    hw[k] = pack_bf16x2(r0, r1);
                    // the naive arm's result is the rounded one
                    lw[k] = bf16 ? 0u : pack_bf16x2(r0 - bf16_lo(hw[k]), r1 - bf16_hi(hw[k]));
                }
            }
            todo &= ~__ballot_sync(0xffffffffu, pend == count);
        }
    }

    // This thread's 16 bytes of query row `row` / cache row `row` in a chunk.
    __device__ __forceinline__ uint32_t q_place(int chunk, int row) const
    {
        return smem + S::q + chunk * S::q_chunk_bytes + row * 128 + ((v ^ (row & 7)) << 4);
    }
    __device__ __forceinline__ uint32_t place(int stage, int chunk, int row) const
    {
        return smem + S::stage + stage * S::stage_bytes + (row / 8) * S::group_bytes + chunk * kAtomBytes + (row & 7) * 128 +
               ((v ^ (row & 7)) << 4);
    }

    __device__ __forceinline__ void run()
    {
        const Geometry& g = a.g;
        const int group = a.q_heads;
        Ring ring;
        uint32_t q_phase = 0;
        trig_valid = false;
        for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
            const Work w = load_work(a, i);
            if (w.tiles == 0) continue;
            if (!wait(smem_addr(&m->q_empty), q_phase ^ 1)) return;
            q_phase ^= 1;
#pragma unroll 1
            for (int r = r0; r < padded_rows(w.it.rows); r += 16) {
                const bool on = r < w.it.rows;
                const int row = w.it.row0 + (on ? r : 0);
                const long long tok = w.ch.tok0 + row / group, head = row % group;
                const uint4* lat =
                    static_cast<const uint4*>(a.q_latent.ptr) + (tok * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8;
                const uint4* band =
                    static_cast<const uint4*>(a.q_rope.ptr) + (tok * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8;
#pragma unroll
                for (int c = 0; c <= kLatentChunks; ++c)
                    cp_async16(q_place(c, r), c < kLatentChunks ? lat + 8 * c + v : band + v, on);
            }
            cp_async_arrive(smem_addr(&m->q_full));
            const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
            for (int t = 0; t < w.tiles; ++t) {
                const long long key = w.it.key0 + (long long)t * kAttnKeys;
                const bool box = by_box(maps, w, key);
                const uint32_t full = smem_addr(&m->full[ring.stage]);
                if (box && !kLazy) {  // the load warp's tile: only these warps' arrivals
                    if (!wait(smem_addr(&m->empty[ring.stage][kSteps - 1]), ring.phase ^ 1)) return;
                    if (tid % 32 == 0) mbar_arrive_n(full, 32);
                    ring.advance();
                    continue;
                }
                long long slot[4];  // of rows r0 + 16 k: < 0, not loaded
                const uint4* band[4];
                uint4 hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = map_row(a, page_of(a, maps, w, table_row, key + r0 + 16 * k));
                    slot[k] = row < 0 ? -1 : row - (long long)a.layer * g.num_pages * g.block_size;
                    band[k] = a.kv + band_off(g, a.layer, max(slot[k], 0ll)) + v;
                }
                if (kLazy) {
                    int pend[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        pend[k] = slot[k] >= 0 ? a.pending[slot[k]] : 0;
                        hi[k] = slot[k] >= 0 ? ld_stream(band[k]) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 x = hi[k];
                        turned(x, pend[k], hi[k], lo[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // rows r0 + 16 k are freed by PV's step k
                    const int r = r0 + 16 * k;
                    if (!wait(smem_addr(&m->empty[ring.stage][k]), ring.phase ^ 1)) return;
                    if (kLazy) {
                        store(place(ring.stage, 8, r), hi[k]);
                        store(place(ring.stage, 9, r), lo[k]);
                    } else {
                        cp_async16(place(ring.stage, 8, r), band[k], slot[k] >= 0);
                    }
                    if (!box) {
                        const uint4* lat = a.kv + lat_off(g, a.layer, max(slot[k], 0ll)) + v;
#pragma unroll
                        for (int c = 0; c < kLatentChunks; ++c)
                            cp_async16(place(ring.stage, c, r), lat + 8 * c, slot[k] >= 0);
                    }
                }
                if (kLazy) {
                    fence_async_smem();
                    mbar_arrive(full);
                }
                cp_async_arrive(full);  // when the copies have landed
                ring.advance();
            }
        }
    }
};

// --------------------------------------------------------------------- MMAs --
// The tiles of the CTA's items in order, as the issuing warp walks them.
struct TileCursor {
    int item, end_item;
    int tile, tiles, n;  // n: columns of O^T (query rows, padded)
    int index;           // tiles before this one

    __device__ __forceinline__ void settle(const AttnArgs& a)
    {
        while (item < end_item) {
            const Work w = load_work(a, item);
            tiles = w.tiles;
            n = padded_rows(w.it.rows);
            tile = 0;
            if (tiles > 0) return;
            ++item;
        }
    }
    __device__ __forceinline__ void start(const AttnArgs& a)
    {
        item = a.cta_begin[blockIdx.x];
        end_item = a.cta_begin[blockIdx.x + 1];
        index = 0;
        settle(a);
    }
    __device__ __forceinline__ bool done() const { return item >= end_item; }
    __device__ __forceinline__ void next(const AttnArgs& a)
    {
        ++index;
        if (++tile == tiles) {
            ++item;
            settle(a);
        }
    }
};

template <bool kLazy>
__device__ __forceinline__ void issue_mmas(const AttnArgs& a, Misc* m, uint32_t smem, uint32_t tmem)
{
    using S = Smem<kLazy>;
    constexpr uint32_t kDescS = mma_desc(kAttnRows, kAttnKeys, false, false);
    constexpr uint32_t kStage = S::stage_bytes / 16, kGroup = S::group_bytes / 16, kQChunk = S::q_chunk_bytes / 16;
    const uint64_t q_mat = smem_matrix(smem + S::q, 16, 1024);
    const uint64_t k_mat = smem_matrix(smem + S::stage, 16, S::group_bytes);
    const uint64_t v_mat = smem_matrix(smem + S::stage, kAtomBytes, S::group_bytes);
    const uint64_t p_mat = smem_matrix(smem + S::p, 16, 1024);
    // The whole warp walks the tiles, so that what the MMAs are given stays uniform; one lane issues.
    auto test = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)); };
    TileCursor s, pv;
    s.start(a);
    pv.start(a);
    uint32_t q_phase = 0;
    uint32_t idle = 0;
    unsigned long long t0 = 0;
    while (!pv.done()) {
        bool moved = false;
        if (!s.done() && s.index <= pv.index + 1 && test(smem_addr(&m->full[s.index % kStages]), (s.index / kStages) & 1) &&
            (s.tile > 0 || test(smem_addr(&m->q_full), q_phase))) {
            fence_async_smem();
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t d = tmem + kTmemS + (s.index & 1) * 64;
                const uint64_t k_at = k_mat + (uint64_t)(s.index % kStages * kStage);
#pragma unroll
                for (int c = 0; c < S::chunks; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // the band's low part meets the query's band too
                        mma_bf16(d, q_mat + (uint64_t)(min(c, 8) * kQChunk + 2 * k),
                                 k_at + (uint64_t)(c * (kAtomBytes / 16) + 2 * k), kDescS, c > 0 || k > 0);
                mma_commit(smem_addr(&m->s_full[s.index & 1]));
                if (s.tile + 1 == s.tiles) mma_commit(smem_addr(&m->q_empty));
            }
            __syncwarp();
            if (s.tile == 0) q_phase ^= 1;
            s.next(a);
            moved = true;
        }
        if (pv.index < s.index && test(smem_addr(&m->p_ready), pv.index & 1)) {
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t desc = mma_desc(128, pv.n, true, false);
                const uint64_t v_at = v_mat + (uint64_t)(pv.index % kStages * kStage);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        mma_bf16(tmem + kTmemO + b * 64, v_at + (uint64_t)(2 * k * kGroup + 2 * b * (kAtomBytes / 16)),
                                 p_mat + 2 * k, desc, pv.tile > 0 || k > 0);
                    mma_commit(smem_addr(&m->empty[pv.index % kStages][k]));
                }
                mma_commit(smem_addr(&m->pv_done));
            }
            __syncwarp();
            pv.next(a);
            moved = true;
        }
        if (moved) {
            idle = 0;
        } else if ((++idle & 1023) == 0) {  // the clock is read now and then only: reading it is slow
            if (idle == 1024) t0 = global_ns();
            const bool late = global_ns() - t0 > kWaitLimit;
            if (late) {
                *(volatile int*)&m->quit = 1;
                raise_status(a.status, ST_TIMEOUT);
            }
            if (__any_sync(0xffffffffu, late || *(volatile int*)&m->quit)) break;
        }
    }
}

// ------------------------------------------------------------------ softmax --
__device__ __forceinline__ bool any_of_softmax(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// The softmax warps meet at named barriers, so when the CTA gives up they go through their tiles
// without waiting instead of leaving; the status word says that the output is not valid.

// Multiply the `n` columns of the four blocks of O^T by m->factor.
__device__ __forceinline__ void scale_output(Misc* m, uint32_t tmem_o, int n)
{
    for (int b = 0; b < 4; ++b)
        for (int c = 0; c < n; c += 16) {
            uint32_t v[16];
            tmem_ld16(tmem_o + b * 64 + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * m->factor[c + k]);
            tmem_st16(tmem_o + b * 64 + c, v);
        }
    tmem_wait_st();
}

template <bool kLazy>
__device__ __forceinline__ void run_softmax(const AttnArgs& a, Misc* m, uint32_t smem, uint32_t tmem)
{
    using S = Smem<kLazy>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t tmem_o = tmem + kTmemO + lanes;
    const float scale2 = a.scale * kLog2e;
    const int group = a.q_heads;
    int index = 0;  // tiles before this one
    for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
        const Work w = load_work(a, i);
        // this thread's two rows, their limits, running maxima (log2) and its part of their sums
        int row[2];
        long long limit[2];
        float top[2], sum[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            row[h] = 16 * warp + lane / 4 + 8 * h;
            const int tok = (w.it.row0 + min(row[h], w.it.rows - 1)) / group;
            limit[h] = row[h] < w.it.rows ? (a.prefix ? w.ch.start : w.ch.start + tok + 1) : 0;
            top[h] = -INFINITY;
            sum[h] = 0.f;
        }
        const long long open = a.prefix ? w.ch.start : w.ch.start + w.it.row0 / group + 1;  // every row attends below this
        const int n = padded_rows(w.it.rows);
        for (int t = 0; t < w.tiles; ++t, ++index) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            mbar_wait(smem_addr(&m->s_full[index & 1]), (index >> 1) & 1, &m->quit, a.status);
            tcgen05_after_sync();
            uint32_t v[32];
            tmem_ld_16x64(tmem + kTmemS + lanes + (index & 1) * 64, v);
            tmem_wait_ld();
            float x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k]) * scale2;
            if (key + kAttnKeys > open || w.it.rows < kAttnRows) {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int col = 8 * (k / 4) + 2 * (lane % 4) + (k & 1);
                    if (key + col >= limit[(k >> 1) & 1]) x[k] = -INFINITY;
                }
            }
            float tile_top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 32; ++k) tile_top[(k >> 1) & 1] = fmaxf(tile_top[(k >> 1) & 1], x[k]);
            tile_top[0] = quad_max(tile_top[0]);
            tile_top[1] = quad_max(tile_top[1]);
            const bool raise = any_of_softmax(tile_top[0] > top[0] + kRaise || tile_top[1] > top[1] + kRaise);
            float factor[2] = {1.f, 1.f};
            if (raise) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float old = top[h];
                    top[h] = fmaxf(old, tile_top[h]);
                    factor[h] = top[h] == -INFINITY ? 1.f : exp2f(old - top[h]);
                    sum[h] *= factor[h];
                }
            }
            // weights, their sum in fp32, and the weights rounded to bf16 for the product with V
            const float base[2] = {top[0] == -INFINITY ? 0.f : top[0], top[1] == -INFINITY ? 0.f : top[1]};
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int h = k & 1;
                const float e0 = exp2_approx(x[2 * k] - base[h]), e1 = exp2_approx(x[2 * k + 1] - base[h]);
                sum[h] += e0 + e1;
                p[k] = pack_bf16x2(e0, e1);
            }
            // P and O are free when the product of the tile before has finished
            if (index > 0) mbar_wait(smem_addr(&m->pv_done), (index - 1) & 1, &m->quit, a.status);
            if (raise && t > 0) {
                tcgen05_after_sync();
                if (lane % 4 == 0) {
                    m->factor[row[0]] = factor[0];
                    m->factor[row[1]] = factor[1];
                }
                softmax_sync();
                scale_output(m, tmem_o, n);
                softmax_sync();  // before the next rescale's factors
            }
            if (16 * warp < n) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {  // value k: columns 8 (k / 2) + 2 (lane % 4), + 1 of row[k & 1]
                    const int r = row[k & 1];
                    const uint32_t at = smem + S::p + r * 128 + (((k / 2) ^ (r & 7)) << 4) + 4 * (lane % 4);
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(p[k]) : "memory");
                }
            }
            fence_async_smem();
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&m->p_ready));
        }
        // the tile's result
        float l[2] = {quad_sum(sum[0]), quad_sum(sum[1])};
        if (lane % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[h] >= w.it.rows) continue;
                m->factor[row[h]] = l[h] == 0.f ? 0.f : 1.f / l[h];
                const float lse = l[h] == 0.f ? -INFINITY : (top[h] + log2f(l[h])) * kLn2;
                if (w.it.part >= 0) {
                    a.part_lse[(long long)w.it.part * kAttnRows + row[h]] = lse;
                } else if (a.lse) {
                    const int r = w.it.row0 + row[h];
                    a.lse[(long long)(w.ch.tok0 + r / group) * a.q_heads + r % group] = lse;
                }
            }
        }
        softmax_sync();
        if (w.tiles > 0) {
            mbar_wait(smem_addr(&m->pv_done), (index - 1) & 1, &m->quit, a.status);
            tcgen05_after_sync();
        }
        for (int b = 0; b < 4; ++b)
            for (int c = 0; c < n; c += 16) {
                uint32_t v[16] = {};
                if (w.tiles > 0) {
                    tmem_ld16(tmem_o + b * 64 + c, v);
                    tmem_wait_ld();
                }
                const int dim = 128 * b + 32 * warp + lane;
                for (int k = 0; k < 16; ++k) {
                    const int r = c + k;
                    if (r >= w.it.rows) break;
                    const float o = __uint_as_float(v[k]) * m->factor[r];
                    if (w.it.part >= 0) {
                        a.part_out[((long long)w.it.part * kAttnRows + r) * 512 + dim] = o;
                    } else {
                        const int q = w.it.row0 + r;
                        const long long tok = w.ch.tok0 + q / group, head = q % group;
                        static_cast<__nv_bfloat16*>(
                            a.out.ptr)[tok * a.out.token_stride + head * a.out.head_stride + dim] = __float2bfloat16_rn(o);
                    }
                }
            }
        tcgen05_before_sync();
        softmax_sync();  // before the next item's factors
    }
}

template <bool kLazy>
__global__ void __launch_bounds__(kThreads, 1) attend_mla_kernel(const __grid_constant__ AttnArgs a,
                                                              const __grid_constant__ MlaMaps maps)
{
    extern __shared__ unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    Misc* m = reinterpret_cast<Misc*>(raw + (smem - smem_addr(raw)) + Smem<kLazy>::misc);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            // the load warp and every copy thread (lazy pools: and again for the turned bands)
            mbar_init(smem_addr(&m->full[s]), 1 + (kLazy ? 2 : 1) * kCopyThreads);
            for (int k = 0; k < kSteps; ++k) mbar_init(smem_addr(&m->empty[s][k]), 1);
        }
        mbar_init(smem_addr(&m->q_full), kCopyThreads);
        mbar_init(smem_addr(&m->q_empty), 1);
        mbar_init(smem_addr(&m->s_full[0]), 1);
        mbar_init(smem_addr(&m->s_full[1]), 1);
        mbar_init(smem_addr(&m->p_ready), kSoftmaxWarps);
        mbar_init(smem_addr(&m->pv_done), 1);
        mbar_init(smem_addr(&m->drained), 1);
        m->quit = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&m->tmem), kTmemCols);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = m->tmem;
    wait_for_previous_grid();
    allow_next_grid();
    if (warp < kSoftmaxWarps) {
        run_softmax<kLazy>(a, m, smem, tmem);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        issue_mmas<kLazy>(a, m, smem, tmem);
        // nothing is in flight when TMEM is freed
        if (elect_lane()) mma_commit(smem_addr(&m->drained));
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
        }
    } else if (warp == kLoadWarp) {
        load_tiles<kLazy>(a, maps, m, smem);
    } else {
        const int tid = threadIdx.x - 32 * (kLoadWarp + 1);
        Copier<kLazy> c{a, maps, m, smem, tid, tid % 8, tid / 8, 0, false};
        c.run();
        cp_async_wait_all();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tcgen05_after_sync();
        tmem_free(tmem, kTmemCols);
    }
}


// The driver's encoder of tensor maps, looked up at run time (the library links no driver library).
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled()
{
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeTiled>(f);
}

// Map of `rows` rows of row_vecs 16-byte vectors at `base`: 64 columns, 8 rows of a group, `planes` planes of 64
// columns (none: three dimensions), groups; boxes of `groups` groups.
bool make_map(EncodeTiled encode, CUtensorMap* map, const uint4* base, int64_t rows, int row_vecs, int planes, int groups)
{
    const cuuint64_t row = (cuuint64_t)row_vecs * 16, n = (cuuint64_t)(rows / 8);
    const cuuint64_t dims[4] = {64, 8, planes ? (cuuint64_t)planes : n, n};
    const cuuint64_t strides[3] = {row, planes ? 128 : 8 * row, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(planes ? planes : groups), (cuuint32_t)groups}, steps[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 4 : 3, const_cast<uint4*>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int attention_mla_prepare(const Geometry& g, const void* kv, MlaMaps* maps)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return (int)cudaErrorNotSupported;
    const uint4* base = static_cast<const uint4*>(kv);
    // rows of every layer follow one another, in whole rows and in the arrays of a split-rope pool alike
    const int64_t rows = g.num_pages * g.block_size * g.num_layers;
    const bool whole = !(g.flags & (LEYLINE_POOL_SPLIT_ROPE | LEYLINE_POOL_LAZY));
    maps->box = g.block_size % 16 == 0 ? 16 : g.block_size % 8 == 0 ? 8 : 0;
    if (rows > INT32_MAX) return (int)cudaErrorInvalidValue;
    maps->shift = -1;
    for (int k = 0; k < 31; ++k)
        if (g.block_size == 1 << k) maps->shift = k;
    // a box holds two groups where their chunks follow one another
    if (maps->box && (!make_map(encode, &maps->rows, base, rows, g.lat_row_vecs, whole ? 9 : 8, whole && maps->box == 16 ? 2 : 1) ||
                      !make_map(encode, &maps->bands, base + g.rope_base_vecs, rows, g.rope_row_vecs, 0, 1)))
        return (int)cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attend_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmemBytes<false>);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_mla_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<true>);
    return (int)e;
}

int launch_attention_mla(const AttnArgs& a, const MlaMaps& maps, int ctas, void* stream)
{
    return (int)(a.pending ? launch_dependent_smem(attend_mla_kernel<true>, ctas, kThreads, kSmemBytes<true>,
                                                   (cudaStream_t)stream, a, maps)
                           : launch_dependent_smem(attend_mla_kernel<false>, ctas, kThreads, kSmemBytes<false>,
                                                   (cudaStream_t)stream, a, maps));
}

}  // namespace leyline
