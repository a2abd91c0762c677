// leyline_attention_pair.cu -- attention over MLA rows by pairs of CTAs (sm_103a): the kernel for many query rows
// (prompt chunks, many heads), where the tensor cores and shared memory bound the work.
//
// As leyline_attention_tile.cu, per tile of 64 cache rows, but two CTAs on neighbouring SMs work on 128 query rows
// with products that span both (cta_group::2):
//   S   = Q K^T    [128 x 64]: a CTA holds 64 query rows and 32 cache rows;
//   O^T = V^T P^T  [512 x 128]: a CTA holds 256 value dimensions of all 64 cache rows, and P of its own 64 query rows.
// Each CTA thus reads half of the operands of both products (S takes 24 cycles of shared memory a product instead of
// 32 at half the tensor rate, O^T 48 for twice the work), and K and V lie in buffers of their own: K is free for the
// next but one tile as soon as S is done, before the softmax.
//
// The reference maximum of a row is that of its item's first tile and stays: weights are exp2(x - m0), in bf16 and
// fp32 as exact relative to their size as any.  A later score above m0 by more than 80 (as a power of 2) could leave
// fp32's range in the sums; the item is then marked, as is one whose output is not finite, and computed
// again at the end without the tensor cores (leyline_attention_any.cuh).  So O never has to be rescaled, which would
// take both CTAs to agree in the middle of every tile.  Marked items are far slower: with all of them marked a prompt
// chunk of 512 tokens of 128 heads over 8192 rows takes 143 ms instead of 0.73, 16 decodes of 128 heads over some 16000
// rows 9.2 ms instead of 0.079; one request of the 16 alone takes as long, since its pairs finish last.
//
// Roles in each CTA: warps 0-3 softmax and output, warp 4 issues the products (in the first CTA alone), warps 5-6 load
// K and 7-10 V (TMA, one lane each: a thread issues a TMA instruction in 100 to 170 cycles, whatever its size, and a
// thread alone bound the kernel; where 8 does not divide the block size they copy their rows, a warp each), warps
// 11-14 copy the queries and the tiles that end inside.
//
// Bounds and measurements (GB300; cuBLAS bf16 at 1875 TFLOP/s in a burst, 1674 under the power limit; calls back to back
// over four inputs in turn).  The products take 864 + 512 cycles a tile, all of it 1530, and an item's ends 13000.  A prompt
// chunk of 512 tokens of 128 heads over 8192 rows 780 us (1.45 PFLOP/s, 0.77 of the burst, 0.87 of the other; clocks at 1850
// to 1940 MHz), ragged chunks of 61 tokens of 16 heads 147 us (1.2), 16 decodes of 128 heads over 24000 rows 118 us (5.0 TB/s,
// 0.74 of measured copies; 1.2 PFLOP/s).  One row a page, copied: 867, 198 and 144 us.
#include "leyline_attention.cuh"

namespace leyline {
namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kMmaWarp = 4, kKeyWarp = 5, kValueWarp = 7, kCopyWarp = 11;
constexpr int kKeyWarps = 2, kCopyWarps = 4;
constexpr int kThreads = 32 * (kCopyWarp + kCopyWarps);

constexpr int kRows = 64;               // query rows of a CTA
constexpr int kHalfKeys = kAttnKeys / 2;  // cache rows whose keys a CTA holds
constexpr int kStages = 2;
constexpr int kSteps = kAttnKeys / 16;
constexpr int kScores = 4;              // S buffers: S runs up to that many tiles ahead of O
constexpr int kChunkBytes = kRows * 128;  // queries: 9 chunks
constexpr int kKeyBytes = kHalfKeys / 8 * 9 * kAtomBytes;      // whole rows: [group][9 chunks]; else 8, and the band's region
constexpr int kBandOff = kHalfKeys / 8 * 8 * kAtomBytes;
constexpr int kValueGroup = 4 * kAtomBytes;                    // chunks 2 r, 2 r + 1, 4 + 2 r, 5 + 2 r of CTA r
constexpr int kValueBytes = kAttnKeys / 8 * kValueGroup;
constexpr int kKeyOff = 9 * kChunkBytes;
constexpr int kValueOff = kKeyOff + kStages * kKeyBytes;
constexpr int kPOff = kValueOff + kStages * kValueBytes;       // two buffers
constexpr int kMiscOff = kPOff + 2 * kChunkBytes;

// Barriers marked (first) are used in the first CTA alone; the others in both.
struct Misc {
    unsigned long long k_full[kStages], v_full[kStages];  // (first)
    unsigned long long k_empty[kStages], v_empty[kStages][kSteps];
    unsigned long long q_full;                            // (first)
    unsigned long long q_empty;
    unsigned long long tail_k[kStages], tail_v[kStages];  // the stage is free for a tile that ends inside
    unsigned long long s_full[kScores];
    unsigned long long p_ready[2];                        // (first)
    unsigned long long pv_done[2];
    unsigned long long x_ready;                           // both CTAs' factors are there
    unsigned long long drained;
    uint32_t tmem;
    int quit;
    float half[2][kRows];        // a row's maximum over either half of a tile's columns; then the second half's two sums
    float redo;                  // not 0: some item is to be computed again
    // 1 / sum of weights of both CTAs' rows, for items in turn: one CTA may be an item ahead of the other's last step
    alignas(16) float factor[2][2 * kRows];
};
static_assert(offsetof(Misc, factor) % 16 == 0 && kMiscOff % 16 == 0, "read in vectors");
constexpr int kSmemBytes = kMiscOff + (int)sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // 2 blocks of 128 columns: 128 of the CTA's dimensions x both CTAs' rows
constexpr uint32_t kTmemS = 256;  // kScores buffers of 32 columns

constexpr float kRange = 80.f;

__device__ __forceinline__ bool pair_warp_wait(uint32_t bar, uint32_t parity, Misc* m, int32_t* status)
{
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, &m->quit, status));
}

// -------------------------------------------------------------------- loads --
// The keys' loaders ask for the next tile's rows in L2 before they wait for a free stage: two tiles in shared memory are
// too few bytes in flight for HBM's latency.  For chunks of few row tiles alone: the rows of a long chunk are in L2
// already, and asking costs the loaders time.  Without and with, us: 16 decodes of 128 heads, one tile each, 135, 124; 8
// requests over 8000 rows with 7, 12, 24 and 48 tiles each 120.5, 117; 170.5, 166.4; 313.2, 309.4; 617, 612; one over 8192
// rows with 8, 16, 32, 64 and 128 tiles 32.5, 32.7; 42.6, 42.9; 65.0, 65.1; 112.4, 113.0; 205.1, 205.9; with 512 747, 772.
// The border costs up to 2.5% between 9 and 48 tiles of several requests; past it one long chunk is what loses.
constexpr int kPrefetchTiles = 8;

// `n` rows at a page's row, whole.
__device__ __forceinline__ void prefetch_rows(const AttnArgs& a, const PageOf& p, int n)
{
    if (p.page < 0 || p.page >= a.g.num_pages) return;
    const Geometry& g = a.g;
    const long long slot = (long long)p.page * g.block_size + p.off;
    prefetch_l2(a.kv + lat_off(g, a.layer, slot), (uint32_t)(n * g.lat_row_vecs * 16));
    if (g.lat_row_vecs != g.row_vecs) prefetch_l2(a.kv + band_off(g, a.layer, slot), (uint32_t)(n * g.rope_row_vecs * 16));
}

// One lane of a warp each.  Keys (kValues false): loader `part` of two takes 16 of this CTA's 32 rows of a tile, whole;
// values: loader `part` of four takes this CTA's four chunks of 16 of the tile's 64 rows, those of PV's step `part`.
template <bool kValues>
__device__ __forceinline__ void load_tiles(const AttnArgs& a, const TileMaps& maps, Misc* m, uint32_t smem, uint32_t rank,
                                           int part)
{
    const int pair = blockIdx.x / 2;
    const bool wide = maps.box == 16;
    const int boxes = wide ? 1 : 2;  // of two groups of 8 rows, or one each
    const int first = (kValues ? 0 : (int)rank * kHalfKeys) + 16 * part;
    const int layer_groups = (int)((long long)a.layer * a.g.num_pages * a.g.block_size / 8);
    const int chunks = maps.whole ? 9 : 8;
    Ring ring;
    for (int i = a.cta_begin[pair]; i < a.cta_begin[pair + 1]; ++i) {
        const Work w = load_work(a, i);
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        const bool prefetch = !kValues && w.ch.n * a.q_heads <= kPrefetchTiles * kPairRows;
        PageOf at[2];
        auto look_up = [&](long long key) {
            if (!by_box(maps, w, key)) return;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k < boxes) at[k] = page_of(a, maps, w, table_row, key + first + 8 * k);
        };
        look_up(w.it.key0);
        for (int t = 0; t < w.tiles; ++t) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            const bool box = by_box(maps, w, key);
            int y[2] = {-2, -2};
            if (box) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k < boxes) {
                        const long long slot = slot_of(a, at[k]);
                        if (slot >= 0) y[k] = layer_groups + (int)(slot >> 3);
                    }
            }
            if (t + 1 < w.tiles) {
                look_up(key + kAttnKeys);
                if (prefetch && by_box(maps, w, key + kAttnKeys)) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (k < boxes) prefetch_rows(a, at[k], maps.box);
                }
            }
            const uint32_t empty = smem_addr(kValues ? &m->v_empty[ring.stage][part] : &m->k_empty[ring.stage]);
            if (!mbar_wait_cluster(empty, ring.phase ^ 1, &m->quit, a.status)) return;
            if (!box) {  // the copy warps' tile.  They do not follow the stages' uses, which a parity could not tell apart
                mbar_arrive(smem_addr(kValues ? &m->tail_v[ring.stage] : &m->tail_k[ring.stage]));
            } else {
                // Both CTAs' bytes are counted in the first, whose loader alone arrives, for all that are expected: an
                // arrival from the other CTA is a release at cluster scope, which took 1000 to 1600 cycles here
                const uint32_t bar = smem_addr(kValues ? &m->v_full[ring.stage] : &m->k_full[ring.stage]);
                const uint32_t full = cluster_addr(bar, 0);
                if (rank == 0) {
                    mbar_expect_tx(bar, 2 * (kValues ? kValueBytes / kSteps : kKeyBytes / kKeyWarps));
                    mbar_arrive_n(bar, 2 * kCopyWarps / (kValues ? kSteps : kKeyWarps) - 1);
                }
                if (!kValues) {
                    const uint32_t dst = smem + kKeyOff + ring.stage * kKeyBytes;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (k < boxes) {
                            const int group = 2 * part + k;
                            pair_box4(dst + group * chunks * kAtomBytes, &maps.pair_keys, 0, y[k], full);
                            if (!maps.whole) pair_box4(dst + kBandOff + group * kAtomBytes, &maps.bands, 0, y[k], full);
                        }
                } else {
                    const uint32_t dst = smem + kValueOff + ring.stage * kValueBytes;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (k < boxes)
                            pair_box5(dst + (2 * part + k) * kValueGroup, &maps.pair_values, 2 * (int)rank, y[k], full);
                }
            }
            ring.advance(kStages);
        }
    }
}

// Pools whose block size 8 does not divide: the same warps copy their 16 rows of every tile (zeros past the end), all lanes
// 16 bytes at a time; pages are looked up two tiles ahead, and lines asked into L2 one ahead.
template <bool kValues>
__device__ __forceinline__ void copy_rows(const AttnArgs& a, const TileMaps& maps, Misc* m, uint32_t smem, uint32_t rank,
                                          int part)
{
    const Geometry& g = a.g;
    const int pair = blockIdx.x / 2, lane = threadIdx.x & 31, v = lane % 8, r0 = 16 * part + lane / 8;
    const int first = kValues ? 0 : (int)rank * kHalfKeys;
    const int chunks = maps.whole ? 9 : 8;
    Ring ring;
    for (int i = a.cta_begin[pair]; i < a.cta_begin[pair + 1]; ++i) {
        const Work w = load_work(a, i);
        const bool prefetch = !kValues && w.ch.n * a.q_heads <= kPrefetchTiles * kPairRows;
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        PageOf at[4], next[4];
        auto look_up = [&](PageOf (&p)[4], long long key) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = page_of(a, maps, w, table_row, key + first + r0 + 4 * k);
        };
        look_up(at, w.it.key0);
        look_up(next, w.it.key0 + kAttnKeys);
        for (int t = 0; t < w.tiles; ++t) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            int slot[4];  // < 0: zeros
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                slot[k] = (int)slot_of(a, at[k]);
                at[k] = next[k];
            }
            look_up(next, key + 2 * kAttnKeys);
            if (!pair_warp_wait(smem_addr(kValues ? &m->v_empty[ring.stage][part] : &m->k_empty[ring.stage]), ring.phase ^ 1, m,
                                a.status))
                return;
            const uint32_t dst = smem + (kValues ? kValueOff + ring.stage * kValueBytes : kKeyOff + ring.stage * kKeyBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + 4 * k;
                const uint4* lat = a.kv + lat_off(g, a.layer, max(slot[k], 0)) + v;
                const uint32_t in = (r & 7) * 128 + ((v ^ (r & 7)) << 4);
                if (kValues) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        cp_async16(dst + (r / 8) * kValueGroup + c * kAtomBytes + in, lat + 8 * (4 * (c / 2) + 2 * (int)rank + c % 2),
                                   slot[k] >= 0);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        cp_async16(dst + ((r / 8) * chunks + c) * kAtomBytes + in, lat + 8 * c, slot[k] >= 0);
                    cp_async16(dst + (maps.whole ? ((r / 8) * 9 + 8) * kAtomBytes : kBandOff + (r / 8) * kAtomBytes) + in,
                               a.kv + band_off(g, a.layer, max(slot[k], 0)) + v, slot[k] >= 0);
                }
            }
            if (prefetch && t + 1 < w.tiles) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (at[k].page < 0 || at[k].page >= g.num_pages) continue;
                    const int s = at[k].page * (int)g.block_size + at[k].off;
                    prefetch_line(a.kv + lat_off(g, a.layer, s) + 8 * v);
                    if (v == 0) prefetch_line(a.kv + band_off(g, a.layer, s));
                }
            }
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            // as many arrivals as the copy warps of both CTAs
            if (lane < kCopyWarps / (kValues ? kSteps : kKeyWarps))
                cluster_arrive_smem(cluster_addr(smem_addr(kValues ? &m->v_full[ring.stage] : &m->k_full[ring.stage]), 0));
            ring.advance(kStages);
        }
    }
}

// Queries of this CTA's rows, and tiles that end inside (where TMA takes the others): 16-byte copies, zeros for rows past
// the end.
__device__ __forceinline__ void copy_tiles(const AttnArgs& a, const TileMaps& maps, Misc* m, uint32_t smem, uint32_t rank)
{
    const Geometry& g = a.g;
    const int pair = blockIdx.x / 2, group = a.q_heads;
    const int tid = threadIdx.x - 32 * kCopyWarp, v = tid % 8, r0 = tid / 8;
    const int chunks = maps.whole ? 9 : 8;
    // the copies of all four warps have landed when each has arrived
    auto arrive = [&](unsigned long long* bar) {
        cp_async_wait_all();
        fence_async_smem();
        __syncwarp();
        if (tid % 32 == 0) cluster_arrive(cluster_addr(smem_addr(bar), 0), 1);
    };
    int ring_tiles = 0;  // of the items before
    uint32_t q_phase = 0, tail_phase = 0;  // (a bit for each stage)
    for (int i = a.cta_begin[pair]; i < a.cta_begin[pair + 1]; ++i) {
        const Work w = load_work(a, i);
        if (w.tiles == 0) continue;
        if (!pair_warp_wait(smem_addr(&m->q_empty), q_phase ^ 1, m, a.status)) return;
        q_phase ^= 1;
#pragma unroll 1
        for (int r = r0; r < kRows; r += 16) {
            const bool on = (int)rank * kRows + r < w.it.rows;
            const int row = w.it.row0 + (on ? (int)rank * kRows + r : 0);
            const long long tok = w.ch.tok0 + row / group, head = row % group;
            const uint4* lat = static_cast<const uint4*>(a.q_latent.ptr) +
                               (tok * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8 + v;
            const uint4* band =
                static_cast<const uint4*>(a.q_rope.ptr) + (tok * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8 + v;
            const uint32_t to = smem + r * 128 + ((v ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < 9; ++c) cp_async16(to + c * kChunkBytes, c < 8 ? lat + 8 * c : band, on);
        }
        arrive(&m->q_full);
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        // the last tile, where it ends inside
        const int stage = (ring_tiles + w.tiles - 1) % kStages;
        ring_tiles += w.tiles;
        const long long key = w.it.key0 + (long long)(w.tiles - 1) * kAttnKeys;
        if (maps.box == 0 || by_box(maps, w, key)) continue;
        if (!pair_warp_wait(smem_addr(&m->tail_k[stage]), tail_phase >> stage & 1, m, a.status)) return;
        const uint32_t keys = smem + kKeyOff + stage * kKeyBytes, values = smem + kValueOff + stage * kValueBytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + 16 * k;
            const long long slot = slot_of(a, page_of(a, maps, w, table_row, key + rank * kHalfKeys + r));
            const uint4* lat = a.kv + lat_off(g, a.layer, max(slot, 0ll)) + v;
            const uint4* band = a.kv + band_off(g, a.layer, max(slot, 0ll)) + v;
            const uint32_t in = (r & 7) * 128 + ((v ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < 8; ++c) cp_async16(keys + ((r / 8) * chunks + c) * kAtomBytes + in, lat + 8 * c, slot >= 0);
            cp_async16(keys + (maps.whole ? ((r / 8) * 9 + 8) * kAtomBytes : kBandOff + (r / 8) * kAtomBytes) + in, band,
                       slot >= 0);
        }
        arrive(&m->k_full[stage]);
        if (!pair_warp_wait(smem_addr(&m->tail_v[stage]), tail_phase >> stage & 1, m, a.status)) return;
        tail_phase ^= 1u << stage;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = r0 + 16 * k;
            const long long slot = slot_of(a, page_of(a, maps, w, table_row, key + r));
            const uint4* lat = a.kv + lat_off(g, a.layer, max(slot, 0ll)) + v;
            const uint32_t in = (r / 8) * kValueGroup + (r & 7) * 128 + ((v ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                cp_async16(values + c * kAtomBytes + in, lat + 8 * (4 * (c / 2) + 2 * (int)rank + c % 2), slot >= 0);
        }
        arrive(&m->v_full[stage]);
    }
}

// --------------------------------------------------------------------- MMAs --
struct TileCursor {
    int item, end_item;
    int tile, tiles;
    int index;  // tiles before this one
    Ring ring;

    __device__ __forceinline__ void settle(const AttnArgs& a)
    {
        while (item < end_item) {
            tiles = load_work(a, item).tiles;
            tile = 0;
            if (tiles > 0) return;
            ++item;
        }
    }
    __device__ __forceinline__ void start(const AttnArgs& a)
    {
        item = a.cta_begin[blockIdx.x / 2];
        end_item = a.cta_begin[blockIdx.x / 2 + 1];
        index = 0;
        settle(a);
    }
    __device__ __forceinline__ bool done() const { return item >= end_item; }
    __device__ __forceinline__ void next(const AttnArgs& a)
    {
        ++index;
        ring.advance(kStages);
        if (++tile == tiles) {
            ++item;
            settle(a);
        }
    }
};

__device__ __forceinline__ void issue_mmas(const AttnArgs& a, const TileMaps& maps, Misc* m, uint32_t smem, uint32_t tmem)
{
    constexpr uint32_t kDescS = mma_desc(2 * kRows, kAttnKeys, false, false);
    constexpr uint32_t kDescO = mma_desc(256, 2 * kRows, true, false);
    constexpr int kAtom = kAtomBytes / 16;
    const int chunks = maps.whole ? 9 : 8;
    const uint64_t q_mat = smem_matrix(smem, 16, 1024);
    const uint64_t k_mat = smem_matrix(smem + kKeyOff, 16, chunks * kAtomBytes);
    const uint64_t band_mat = smem_matrix(smem + kKeyOff + (maps.whole ? 8 * kAtomBytes : kBandOff), 16,
                                          (maps.whole ? 9 : 1) * kAtomBytes);
    const uint64_t v_mat = smem_matrix(smem + kValueOff, kAtomBytes, kValueGroup);
    const uint64_t p_mat = smem_matrix(smem + kPOff, 16, 1024);
    auto test = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_cluster(bar, parity)); };
    TileCursor s, pv;
    s.start(a);
    pv.start(a);
    uint32_t q_phase = 0;
    uint32_t idle = 0;
    unsigned long long t0 = 0;
    while (!pv.done()) {
        bool moved = false;
        if (!s.done() && s.index < pv.index + kScores && test(smem_addr(&m->k_full[s.ring.stage]), s.ring.phase) &&
            (s.tile > 0 || test(smem_addr(&m->q_full), q_phase))) {
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t d = tmem + kTmemS + (s.index % kScores) * 32;
                const uint32_t at = s.ring.stage * (kKeyBytes / 16);
#pragma unroll
                for (int c = 0; c < 9; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        pair_mma_bf16(d, q_mat + (uint64_t)(c * (kChunkBytes / 16) + 2 * k),
                                      (c < 8 ? k_mat + (uint64_t)(at + c * kAtom + 2 * k) : band_mat + (uint64_t)(at + 2 * k)),
                                      kDescS, c > 0 || k > 0);
                pair_commit(smem_addr(&m->s_full[s.index % kScores]));
                pair_commit(smem_addr(&m->k_empty[s.ring.stage]));
                if (s.tile + 1 == s.tiles) pair_commit(smem_addr(&m->q_empty));
            }
            __syncwarp();
            if (s.tile == 0) q_phase ^= 1;
            s.next(a);
            moved = true;
        }
        if (pv.index < s.index && test(smem_addr(&m->p_ready[pv.index & 1]), (pv.index >> 1) & 1) &&
            test(smem_addr(&m->v_full[pv.ring.stage]), pv.ring.phase)) {
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t at = pv.ring.stage * (kValueBytes / 16);
                const uint64_t p_at = p_mat + (uint64_t)((pv.index & 1) * (kChunkBytes / 16));
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        pair_mma_bf16(tmem + kTmemO + b * 128,
                                      v_mat + (uint64_t)(at + k * (2 * kValueGroup / 16) + 2 * b * kAtom), p_at + 2 * k, kDescO,
                                      pv.tile > 0 || k > 0);
                    pair_commit(smem_addr(&m->v_empty[pv.ring.stage][k]));
                }
                pair_commit(smem_addr(&m->pv_done[pv.index & 1]));
            }
            __syncwarp();
            pv.next(a);
            moved = true;
        }
        if (moved) {
            idle = 0;
        } else if ((++idle & 1023) == 0) {
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

// A thread has one query row (TMEM lanes 0..63 and again 64..127) and one half of a tile's columns.  The warps meet at
// named barriers, so when the CTA gives up they go on without waiting; the status word says the output is not valid.
__device__ __forceinline__ void run_softmax(const AttnArgs& a, Misc* m, uint32_t smem, uint32_t tmem, uint32_t rank)
{
    const int pair = blockIdx.x / 2;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const int r = 32 * (warp & 1) + lane, half = warp >> 1;
    const float scale2 = a.scale * kLog2e, unit = scale2 > 0.f ? scale2 : 1.f;
    const int group = a.q_heads;
    int index = 0;
    uint32_t x_phase = 0;
    for (int i = a.cta_begin[pair]; i < a.cta_begin[pair + 1]; ++i) {
        const Work w = load_work(a, i);
        const int rows = min(max(w.it.rows - (int)rank * kRows, 0), kRows);  // of this CTA
        const int row0 = w.it.row0 + (int)rank * kRows;
        const long long limit =
            r < rows ? (a.prefix ? w.ch.start : w.ch.start + (row0 + r) / group + 1) : 0;  // this row's: [0, limit)
        const long long open = a.prefix ? w.ch.start : w.ch.start + row0 / group + 1;      // every row attends below this
        float top = -INFINITY;
        float2 sum = make_float2(0.f, 0.f), used = make_float2(0.f, 0.f);
        bool redo = false;
        for (int t = 0; t < w.tiles; ++t, ++index) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            mbar_wait(smem_addr(&m->s_full[index % kScores]), (index / kScores) & 1, &m->quit, a.status);
            tcgen05_after_sync();
            uint32_t v[32];
            tmem_ld32(tmem + kTmemS + lanes + (index % kScores) * 32, v);
            tmem_wait_ld();
            float x[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k]);
            if (scale2 <= 0.f) {  // (else the weights' exponents are formed in one step from the products)
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] *= scale2;
            }
            if (key + kAttnKeys > open || rows < kRows) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (key + 32 * half + k >= limit) x[k] = -INFINITY;
            }
            float most = x[0];
#pragma unroll
            for (int k = 1; k < 32; ++k) most = fmaxf(most, x[k]);
            most *= unit;
            if (t == 0) {
                m->half[half][r] = most;
                softmax_sync();
                top = fmaxf(m->half[0][r], m->half[1][r]);
            } else {
                redo |= most > top + kRange;
            }
            const float base = top == -INFINITY ? 0.f : top;
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(unit, unit), make_float2(-base, -base));
                e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                sum = add2(sum, e);
                p[k] = pack_bf16x2(e.x, e.y);
                // the output is divided by the sum of the weights as the product has them (leyline_attention_tile.cu)
                used = add2(used, make_float2(bf16_lo(p[k]), bf16_hi(p[k])));
            }
            if (index > 1) mbar_wait_cluster(smem_addr(&m->pv_done[index & 1]), ((index - 2) >> 1) & 1, &m->quit, a.status);
            const uint32_t at = smem + kPOff + (index & 1) * kChunkBytes + r * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((4 * half + k) ^ (r & 7)) << 4)),
                             "r"(p[4 * k]), "r"(p[4 * k + 1]), "r"(p[4 * k + 2]), "r"(p[4 * k + 3])
                             : "memory");
            fence_async_smem();
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) cluster_arrive_smem(cluster_addr(smem_addr(&m->p_ready[index & 1]), 0));
        }
        // the rows' sums, and 1 / sum of the used weights of both CTAs' rows in both
        softmax_sync();  // the maxima have been read
        if (half == 1) {
            m->half[0][r] = sum.x + sum.y;
            m->half[1][r] = used.x + used.y;
        }
        softmax_sync();
        if (half == 0) {
            const float l = sum.x + sum.y + m->half[0][r], weights = used.x + used.y + m->half[1][r];
            if (r < rows) {
                const float lse = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
                if (w.it.part >= 0) {
                    a.part_lse[(long long)w.it.part * kPairRows + rank * kRows + r] = lse;
                } else if (a.lse) {
                    const int q = row0 + r;
                    a.lse[(long long)(w.ch.tok0 + q / group) * a.q_heads + q % group] = lse;
                }
            }
            const float f = weights == 0.f ? 0.f : 1.f / weights;
            const uint32_t to = smem_addr(&m->factor[x_phase][rank * kRows + r]);
            cluster_store(cluster_addr(to, 0), f);
            cluster_store(cluster_addr(to, 1), f);
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                cluster_arrive(cluster_addr(smem_addr(&m->x_ready), 0), 1);
                cluster_arrive(cluster_addr(smem_addr(&m->x_ready), 1), 1);
            }
        }
        mbar_wait_cluster(smem_addr(&m->x_ready), x_phase, &m->quit, a.status);
        if (w.tiles > 0) {
            mbar_wait_cluster(smem_addr(&m->pv_done[(index - 1) & 1]), ((index - 1) >> 1) & 1, &m->quit, a.status);
            tcgen05_after_sync();
        }
        for (int c = 0; c < w.it.rows; c += 16)  // (P is free)
            redo |= put_rows<kPairRows>(a, w, group, 512, c, 128 * (int)rank + 32 * warp, 256, 2, tmem + kTmemO + lanes + c,
                                        128, m->factor[x_phase] + c, smem + kPOff + warp * 1024);
        x_phase ^= 1;
        tcgen05_before_sync();
        redo = any_of_softmax(redo);  // and before the next item's maxima
        if (threadIdx.x == 0) {
            a.redo[2 * i + rank] = redo;
            if (redo) {
                const uint32_t to = smem_addr(&m->redo);
                cluster_store(cluster_addr(to, 0), 1.f);
                cluster_store(cluster_addr(to, 1), 1.f);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) attend_pair_kernel(const __grid_constant__ AttnArgs a,
                                                               const __grid_constant__ TileMaps maps)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    Misc* m = reinterpret_cast<Misc*>(raw + (smem - smem_addr(raw)) + kMiscOff);
    const int warp = threadIdx.x / 32;
    const uint32_t rank = cluster_rank();
    wait_for_previous_grid();
    // (the next kernel is let in by this one's end: let in before, the join's waiting CTAs cost 15 us of a call of 26)
    if (a.header->pairs == 0) return;  // the plan is for the other kernel (both CTAs see the same)
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&m->k_full[s]), 2 * kCopyWarps);  // both CTAs' copy warps, or the loaders for as many
            mbar_init(smem_addr(&m->v_full[s]), 2 * kCopyWarps);
            mbar_init(smem_addr(&m->k_empty[s]), 1);
            mbar_init(smem_addr(&m->tail_k[s]), kKeyWarps);
            mbar_init(smem_addr(&m->tail_v[s]), kSteps);
            for (int k = 0; k < kSteps; ++k) mbar_init(smem_addr(&m->v_empty[s][k]), 1);
        }
        mbar_init(smem_addr(&m->q_full), 2 * kCopyWarps);
        mbar_init(smem_addr(&m->q_empty), 1);
        for (int b = 0; b < kScores; ++b) mbar_init(smem_addr(&m->s_full[b]), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&m->p_ready[b]), 2 * kSoftmaxWarps);
            mbar_init(smem_addr(&m->pv_done[b]), 1);
        }
        mbar_init(smem_addr(&m->x_ready), 4);  // the two warps of each CTA that hold the sums
        mbar_init(smem_addr(&m->drained), 1);
        m->quit = 0;
        m->redo = 0.f;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) pair_tmem_alloc(smem_addr(&m->tmem), kTmemCols);
    tcgen05_before_sync();
    __syncthreads();
    cluster_sync();
    tcgen05_after_sync();
    const uint32_t tmem = m->tmem;
    if (warp < kSoftmaxWarps) {
        run_softmax(a, m, smem, tmem, rank);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            issue_mmas(a, maps, m, smem, tmem);
            // nothing is in flight when TMEM is freed
            if (elect_lane()) pair_commit(smem_addr(&m->drained));
            __syncwarp();
            const unsigned long long t0 = global_ns();
            while (!mbar_try_cluster(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
            }
        }
    } else if (warp < kValueWarp) {
        if (maps.box == 0) copy_rows<false>(a, maps, m, smem, rank, warp - kKeyWarp);
        else if (elect_lane()) load_tiles<false>(a, maps, m, smem, rank, warp - kKeyWarp);
        __syncwarp();
    } else if (warp < kCopyWarp) {
        if (maps.box == 0) copy_rows<true>(a, maps, m, smem, rank, warp - kValueWarp);
        else if (elect_lane()) load_tiles<true>(a, maps, m, smem, rank, warp - kValueWarp);
        __syncwarp();
    } else {
        copy_tiles(a, maps, m, smem, rank);
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
    const bool redo = m->redo != 0.f && !m->quit;
    __syncthreads();  // before shared memory is written again
    if (redo) {       // marked by either CTA: each computes its own rows again
        for (int i = a.cta_begin[blockIdx.x / 2]; i < a.cta_begin[blockIdx.x / 2 + 1]; ++i) {
            if (__ldcg(a.redo + 2 * i) == 0 && __ldcg(a.redo + 2 * i + 1) == 0) continue;
            const AttnItem item = a.items[i];
            attend_rows<kThreads>(a, item, min((int)rank * kRows, item.rows), min((int)(rank + 1) * kRows, item.rows), kPairRows,
                                  raw);
        }
    }
}

}  // namespace

int attention_pair_prepare(const Geometry& g, const void* kv, TileMaps* maps)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return (int)cudaErrorNotSupported;
    uint4* base = static_cast<uint4*>(const_cast<void*>(kv));
    const int64_t rows = g.num_pages * g.block_size * g.num_layers;
    const cuuint64_t row = (cuuint64_t)g.lat_row_vecs * 16, n = (cuuint64_t)(rows / 8);
    const cuuint32_t groups = (cuuint32_t)(maps->box / 8), ones[5] = {1, 1, 1, 1, 1};
    const cuuint32_t planes = maps->whole ? 9 : 8;
    // keys: 64 columns, 8 rows of a group, the row's planes, groups
    const cuuint64_t k_dims[4] = {64, 8, planes, n}, k_strides[3] = {row, 128, 8 * row};
    const cuuint32_t k_box[4] = {64, 8, planes, groups};
    // values: 64 columns, 8 rows, planes of a half of the latent, halves, groups; a box takes two planes of both halves
    const cuuint64_t v_dims[5] = {64, 8, 4, 2, n}, v_strides[4] = {row, 128, 512, 8 * row};
    const cuuint32_t v_box[5] = {64, 8, 2, 2, groups};
    if (maps->box > 0 &&
        (encode(&maps->pair_keys, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, k_dims, k_strides, k_box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        encode(&maps->pair_values, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, v_dims, v_strides, v_box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS))
        return (int)cudaErrorInvalidValue;
    return (int)cudaFuncSetAttribute(attend_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

int launch_attention_pair(const AttnArgs& a, const TileMaps& maps, int pairs, void* stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, attend_pair_kernel, a, maps);
}

}  // namespace leyline
