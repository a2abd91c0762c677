// leyline_attention_tile.cu -- attention of a batch's tokens over the paged cache on the tensor cores of
// sm_103a: MLA rows (latent 512, one 64-wide band) and grouped rows whose key bands and value slices are
// 64, 128 or (values: also 192) 256 wide.
//
// The heads of a chunk that share a key band form the rows of one matrix product, with the chunk's tokens: per
// tile of 64 query rows and 64 cache rows
//   S   = Q K^T   [64 x 64]
//   O^T = V^T P^T [values x 64],  P = exp2(S * scale * log2 e - m).
// MLA: K = [latent | band], 576 wide, and V = the latent, the same bytes of shared memory.  O is kept transposed:
// its value dimensions lie in the 128 TMEM lanes, in blocks of 64 columns, so a cache tile is loaded once, as rows,
// and serves as the K-major operand of S and as the MN-major operand of O^T.
//
// One persistent CTA per SM takes the contiguous run of items the plan gave it.  Roles:
//   warps 0-3  softmax: S from TMEM, running maximum and sum (fp32), P to shared memory, output
//   warp 4     issues the MMAs (one lane)
//   warps 5-8  load cache tiles through the block table, 16 rows of a tile each (TMA, one lane: a thread issues a
//              TMA instruction in 100 to 170 cycles, whatever its size, and a thread alone bound the kernel)
//   warps 9-12 copy the queries (cp.async: any strides), the cache tiles that TMA does not take (block
//              sizes that 8 does not divide; tiles that end inside, whose other rows are zeroed, since
//              they meet weights of 0 in the product with V)
// In a lazy pool the load warps turn the band of each row by its pending count on the way, in fp32, and it goes
// to shared memory as the sum of two bf16 values: the scores then carry the turn to 2^-17, not to the
// 2^-9 of one bf16 rounding, which the other rows do not have either.
//
// A cache tile in shared memory is 8 groups of 8 rows; a group holds the rows' 64-wide column chunks one
// after another, 8 rows x 128 bytes each, swizzled: [latent 0..7, band] for whole MLA rows, else the values, then
// (a region of its own) the band, then its low part.  That is what one TMA box writes (columns, rows of a group,
// chunks, groups), and its strides serve both operands.  Smaller boxes, a chunk of 16 rows at a time, took 100
// cycles of issue each, 36 a tile, and bound the kernel.
//
// The maximum is only raised (and O rescaled) when a row's scores exceed it by 2^8: until then the
// weights are at most 2^8, and sums and products are fp32.
// An item whose output is not finite is computed again, without the tensor cores: there a weight of 0 keeps a masked
// row's infinity or NaN out of the sum, in a matrix product it does not.  That is far slower: one NaN in an attended row of
// one of 64 requests of 16 heads over 4000 rows 1.34 ms instead of 0.070, of one of 16 with grouped drafts 1.9 instead of 0.058.
//
// Bounds and measurements (GB300; HBM copies at 6782 GB/s; calls back to back over four inputs in turn).  MLA: shared memory carries 2500 cycles of operands a tile; a
// tile takes 3400 from L2 and 3800 to 4400 from HBM, two of them in flight.  One decode of 16 heads over 32768 rows 22 us
// (18 with one input over and over, in L2: 14 here, the rest the join), 64 over 4000 rows 77 us (4.8 TB/s).  Grouped: HBM; 4
// drafted tokens of 16 requests, 32 heads on 4 bands of 128, 73 us (4.8 TB/s, 0.71 of measured).  Lazy MLA rows one a page:
// 112 us for 64 requests over 4000 (3.3 TB/s), by the copies of single rows and the turns; 16 rows a page 92.
#include "leyline_attention.cuh"

namespace leyline {
namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps;
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kLoadWarps = 4;  // one for each of PV's steps
constexpr int kCopyWarps = 4;
constexpr int kCopyThreads = 32 * kCopyWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kLoadWarps + kCopyWarps);

constexpr int kRegionChunk = kAttnKeys / 8 * kAtomBytes;  // a chunk of a tile's 64 rows
constexpr int kSteps = kAttnKeys / 16;  // steps of 16 cache rows, in which PV frees a stage
constexpr int kMaxStages = 6;

struct Misc {
    unsigned long long full[kMaxStages];
    unsigned long long empty[kMaxStages][kSteps];
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2];
    unsigned long long p_ready, pv_done, drained;
    uint32_t tmem;
    int quit;
    int redo;  // some item is to be computed again
    alignas(16) float factor[kAttnRows];  // rescale, then 1 / sum of weights
};
static_assert(offsetof(Misc, factor) % 16 == 0 && sizeof(Misc) % 16 == 0, "read in vectors");

// Shared memory of a kind of rows (bytes, from a 1024-byte aligned start).
struct Layout {
    int rows;           // query rows of a tile
    int values;         // chunks of the values (MLA: of the latent)
    int keys;           // chunks of the band
    int row_chunks;     // chunks of the first region's groups
    int q_chunks;
    int q_chunk_bytes;
    int band, low;      // regions in a stage
    int stage, stage_bytes, stages;
    int p, misc;
    int trig;           // lazy pools: cos, sin of the last pending count of each load warp
    int bytes;
};

__host__ __device__ constexpr Layout make_layout(bool mla, bool lazy, bool whole, int keys, int values, int stages)
{
    Layout l{};
    l.rows = mla && lazy ? kAttnRowsLazy : kAttnRows;
    l.values = values;
    l.keys = keys;
    l.row_chunks = whole ? values + keys : values;
    l.q_chunks = mla ? values + keys : keys;
    l.q_chunk_bytes = l.rows * 128;
    l.band = whole ? values * kAtomBytes : l.row_chunks * kRegionChunk;
    l.low = l.row_chunks * kRegionChunk + (whole ? 0 : keys * kRegionChunk);
    l.stage = l.q_chunks * l.q_chunk_bytes;
    l.stage_bytes = l.low + (lazy ? keys * kRegionChunk : 0);
    l.stages = stages;
    l.p = l.stage + stages * l.stage_bytes;
    l.misc = l.p + l.rows * 128;
    l.trig = l.misc + (int)sizeof(Misc);
    l.bytes = l.trig + (lazy ? kLoadWarps * 32 * keys * (int)sizeof(float2) : 0) + 1024;  // and room to align the start
    return l;
}

constexpr int kMaxSmem = 232448;
static_assert(make_layout(true, false, true, 1, 8, 2).bytes <= kMaxSmem, "shared memory of a CTA");
static_assert(make_layout(true, true, false, 1, 8, 2).bytes <= kMaxSmem, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // up to 4 blocks of 64 columns
constexpr uint32_t kTmemS = 256;  // 2 buffers of 64 columns

constexpr float kRaise = 8.f;

__device__ __forceinline__ int padded_rows(int rows) { return (rows + 15) & ~15; }

// -------------------------------------------------------------------- loads --
// One lane of each load warp: the boxes of the 16 rows of PV's step `step`, the next tile's table entries in flight
// meanwhile.
template <bool kMla, int kKeys>
__device__ __forceinline__ void load_tiles(const AttnArgs& a, const TileMaps& maps, const Layout& l, Misc* m, uint32_t smem,
                                           int step)
{
    const bool wide = maps.box == 16;
    const int boxes = wide ? 1 : 2;  // of two groups of 8 rows, or one each
    const bool bands = !maps.whole;
    const uint32_t bytes = (l.row_chunks + (bands ? kKeys : 0)) * (kRegionChunk / kSteps);
    const int layer_groups = (int)((long long)a.layer * a.g.num_pages * a.g.block_size / 8);
    Ring ring;
    for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
        const Work w = load_work(a, i);
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        const int value_plane = kMla ? 0 : w.it.band * l.values, key_plane = kMla ? 0 : w.it.band * kKeys;
        PageOf at[2];
        auto look_up = [&](long long key) {
            if (!by_box(maps, w, key)) return;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k < boxes) at[k] = page_of(a, maps, w, table_row, key + 16 * step + 8 * k);
        };
        look_up(w.it.key0);
        for (int t = 0; t < w.tiles; ++t) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            const bool box = by_box(maps, w, key);
            int y[2] = {-2, -2};  // the boxes as indices of groups of 8 rows; one that is not loaded lies before the first
            if (box) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (k < boxes) {
                        const long long slot = slot_of(a, at[k]);
                        if (slot >= 0) y[k] = layer_groups + (int)(slot >> 3);
                    }
            }
            if (t + 1 < w.tiles) look_up(key + kAttnKeys);
            const uint32_t full = smem_addr(&m->full[ring.stage]);
            if (!mbar_wait(smem_addr(&m->empty[ring.stage][step]), ring.phase ^ 1, &m->quit, a.status)) return;
            if (!box) {  // the copy warps' tile: only this lane's arrival
                mbar_arrive(full);
                ring.advance(l.stages);
                continue;
            }
            mbar_expect_tx(full, bytes);
            const uint32_t dst = smem + l.stage + ring.stage * l.stage_bytes;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k < boxes) {
                    const int group = 2 * step + k;
                    tma_box4(dst + group * l.row_chunks * kAtomBytes, &maps.rows, value_plane, y[k], full);
                    if (bands) tma_box4(dst + l.band + group * kKeys * kAtomBytes, &maps.bands, key_plane, y[k], full);
                }
            ring.advance(l.stages);
        }
    }
}

// Place of 16 bytes `v` of row `row` of a tile in a region whose groups hold `chunks` chunks.
__device__ __forceinline__ uint32_t place(uint32_t region, int chunks, int chunk, int row, int v)
{
    return region + ((row / 8) * chunks + chunk) * kAtomBytes + (row & 7) * 128 + ((v ^ (row & 7)) << 4);
}

__device__ __forceinline__ void store(uint32_t at, const uint4& y)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
}

// Lazy pools: the bands of a load warp's 16 rows of a tile, turned by their pending counts, to the stage as high and low
// parts.  The 8 lanes of a row have 16 bytes of each of its chunks; a lane's rows are 16 step + lane / 8 + 4 r.
template <int kKeys>
struct Turner {
    const AttnArgs& a;
    const Layout& l;
    float2* cs;  // cos, sin of `count`, this warp's
    int lane, v, r0;
    int count;
    bool valid;

    __device__ __forceinline__ void ensure(int c)
    {
        if (valid && c == count) return;
        const bool bf16 = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        __syncwarp();
        for (int j = lane; j < 32 * kKeys; j += 32) {
            float co, si;
            pending_trig(c, a.turn, 32 * kKeys, j, bf16, co, si);
            cs[j] = make_float2(co, si);
        }
        __syncwarp();
        count = c;
        valid = true;
    }

    // Chunk c of the rows whose count is `count`; other: the partner lane's 16 bytes, where a band is one chunk.
    template <bool kNaive, bool kHalfSplit>
    __device__ __forceinline__ void turn_chunk(int c, const uint4 (&x)[4][kKeys], const uint4 (&other)[4],
                                               const int (&pend)[4], uint32_t stage) const
    {
        float co[8], si[8];  // half-split: of 8 pairs, one value of each here, sin negative in first halves; else of 4
        const bool first = kKeys == 1 ? v < 4 : c < kKeys / 2;
        const int pair = kKeys == 1 ? 8 * (v & 3) : 64 * (c % (kKeys > 1 ? kKeys / 2 : 1)) + 8 * v;
#pragma unroll
        for (int k = 0; k < (kHalfSplit ? 8 : 4); ++k) {
            const float2 t = cs[kHalfSplit ? pair + k : 32 * c + 4 * v + k];
            co[k] = t.x;
            si[k] = kHalfSplit && first ? -t.y : t.y;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x[r][c]);
            // half-split: the other halves of this chunk's pairs
            const uint32_t* ow = reinterpret_cast<const uint32_t*>(kKeys == 1 ? &other[r] : &x[r][(c + kKeys / 2) % kKeys]);
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x0 = bf16_lo(xw[k]), x1 = bf16_hi(xw[k]);
                float q0, q1;
                if (kHalfSplit) {  // x' = x c - y s of the first half, y' = y c + x s of the second
                    const float y0 = bf16_lo(ow[k]) * si[2 * k], y1 = bf16_hi(ow[k]) * si[2 * k + 1];
                    q0 = kNaive ? round_bf16(x0 * co[2 * k]) + round_bf16(y0) : fmaf(x0, co[2 * k], y0);
                    q1 = kNaive ? round_bf16(x1 * co[2 * k + 1]) + round_bf16(y1) : fmaf(x1, co[2 * k + 1], y1);
                } else if (kNaive) {
                    turn_bf16(x0, x1, co[k], si[k], q0, q1);
                } else {
                    turn_fp32(x0, x1, co[k], si[k], q0, q1);
                }
                hw[k] = pack_bf16x2(q0, q1);
                // the naive arm's result is the rounded one
                lw[k] = kNaive ? 0u : pack_bf16x2(q0 - bf16_lo(hw[k]), q1 - bf16_hi(hw[k]));
            }
            if (pend[r] == count) {
                store(place(stage + l.band, kKeys, c, r0 + 4 * r, v), make_uint4(hw[0], hw[1], hw[2], hw[3]));
                store(place(stage + l.low, kKeys, c, r0 + 4 * r, v), make_uint4(lw[0], lw[1], lw[2], lw[3]));
            }
        }
    }

    // x, pend: this lane's rows.  Mostly all rows of a warp share a count: then one pass, in which the four rows' chains
    // run side by side (a row at a time took 1000 cycles each, by the warps that also copy the rows, and bound the
    // kernel: 64 requests of 16 heads over 4000 rows, 16 a page, 136 -> 88 us); else a pass for each count.
    __device__ __forceinline__ void rows(const uint4 (&x)[4][kKeys], const int (&pend)[4], uint32_t stage)
    {
        const bool naive = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        const bool half_split = a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
        uint4 other[4];
        if (kKeys == 1 && half_split) {
#pragma unroll
            for (int r = 0; r < 4; ++r) other[r] = shfl_xor_vec(x[r][0], 4);
        }
        unsigned left = 15;
        for (;;) {
            const unsigned lanes = __ballot_sync(0xffffffffu, left != 0);
            if (lanes == 0) return;
            int mine = pend[3];
#pragma unroll
            for (int r = 2; r >= 0; --r)
                if (left >> r & 1) mine = pend[r];
            const int c0 = __shfl_sync(0xffffffffu, mine, __ffs(lanes) - 1);
            if (c0 == 0) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (pend[r] == 0) {
                            store(place(stage + l.band, kKeys, c, r0 + 4 * r, v), x[r][c]);
                            store(place(stage + l.low, kKeys, c, r0 + 4 * r, v), make_uint4(0, 0, 0, 0));
                        }
            } else {
                ensure(c0);
#pragma unroll
                for (int c = 0; c < kKeys; ++c) {
                    if (half_split) {
                        if (naive) turn_chunk<true, true>(c, x, other, pend, stage);
                        else turn_chunk<false, true>(c, x, other, pend, stage);
                    } else {
                        if (naive) turn_chunk<true, false>(c, x, other, pend, stage);
                        else turn_chunk<false, false>(c, x, other, pend, stage);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (pend[r] == c0) left &= ~(1u << r);
        }
    }
};

// The load warps in a lazy pool: one lane issues the boxes of its 16 rows' values, then the whole warp turns their bands,
// which were read while it waited for the stage.
template <bool kMla, int kKeys>
__device__ __forceinline__ void load_lazy(const AttnArgs& a, const TileMaps& maps, const Layout& l, Misc* m, uint32_t smem,
                                          int step, float2* trig)
{
    const Geometry& g = a.g;
    const int lane = threadIdx.x & 31, v = lane & 7, r0 = 16 * step + lane / 8;
    const bool wide = maps.box == 16;
    const int layer_groups = (int)((long long)a.layer * g.num_pages * g.block_size / 8);
    Turner<kKeys> turner{a, l, trig, lane, v, r0, 0, false};
    Ring ring;
    for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
        const Work w = load_work(a, i);
        const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
        const int value_plane = kMla ? 0 : w.it.band * l.values, band_vec = kMla ? 0 : w.it.band * kKeys * 8;
        // pages two tiles ahead, bands and counts one
        PageOf next[4], box_next[2];
        long long box_slot[2];
        uint4 x[4][kKeys];
        int pend[4];
        auto look_up = [&](long long key) {
#pragma unroll
            for (int k = 0; k < 4; ++k) next[k] = page_of(a, maps, w, table_row, key + r0 + 4 * k);
            if (!by_box(maps, w, key)) return;
#pragma unroll
            for (int k = 0; k < 2; ++k) box_next[k] = page_of(a, maps, w, table_row, key + 16 * step + 8 * k);
        };
        auto read = [&](long long key) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const long long slot = slot_of(a, next[k]);
                const uint4* band = a.kv + band_off(g, a.layer, max(slot, 0ll)) + band_vec + v;
                pend[k] = slot >= 0 ? a.pending[slot] : 0;
#pragma unroll
                for (int c = 0; c < kKeys; ++c) x[k][c] = slot >= 0 ? ld_stream(band + 8 * c) : make_uint4(0, 0, 0, 0);
            }
            if (!by_box(maps, w, key)) return;
#pragma unroll
            for (int k = 0; k < 2; ++k) box_slot[k] = slot_of(a, box_next[k]);
        };
        if (w.tiles > 0) {
            look_up(w.it.key0);
            read(w.it.key0);
            if (w.tiles > 1) look_up(w.it.key0 + kAttnKeys);
        }
        for (int t = 0; t < w.tiles; ++t) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            const uint32_t full = smem_addr(&m->full[ring.stage]);
            const uint32_t stage = smem + l.stage + ring.stage * l.stage_bytes;
            if (!warp_wait(smem_addr(&m->empty[ring.stage][step]), ring.phase ^ 1, &m->quit, a.status)) return;
            if (elect_lane()) {
                if (by_box(maps, w, key)) {
                    mbar_expect_tx(full, l.row_chunks * (kRegionChunk / kSteps));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (wide && k == 1) break;
                        const int y = box_slot[k] >= 0 ? layer_groups + (int)(box_slot[k] >> 3) : -2;
                        tma_box4(stage + (2 * step + k) * l.row_chunks * kAtomBytes, &maps.rows, value_plane, y, full);
                    }
                } else {
                    mbar_arrive(full);
                }
            }
            __syncwarp();
            turner.rows(x, pend, stage);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            if (t + 1 < w.tiles) {
                read(key + kAttnKeys);
                if (t + 2 < w.tiles) look_up(key + 2 * kAttnKeys);
            }
            ring.advance(l.stages);
        }
    }
}

// ------------------------------------------------------------------- copies --
template <bool kMla, bool kLazy, int kKeys>
struct Copier {
    const AttnArgs& a;
    const TileMaps& maps;
    const Layout& l;
    Misc* m;
    uint32_t smem;
    int tid, v, r0;  // 16-byte chunk of a 128-byte row segment, first row

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, &m->quit, a.status); }

    // This thread's 16 bytes of row `row` in a chunk.
    __device__ __forceinline__ uint32_t q_place(int chunk, int row) const
    {
        return smem + chunk * l.q_chunk_bytes + row * 128 + ((v ^ (row & 7)) << 4);
    }
    __device__ __forceinline__ void queries(const Work& w)
    {
        const int group = a.q_heads / (kMla ? 1 : a.g.rope_heads);
#pragma unroll 1
        for (int r = r0; r < padded_rows(w.it.rows); r += 16) {
            const bool on = r < w.it.rows;
            const int row = w.it.row0 + (on ? r : 0);
            const long long tok = w.ch.tok0 + row / group, head = w.it.band * group + row % group;
            const uint4* band =
                static_cast<const uint4*>(a.q_rope.ptr) + (tok * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8;
            int chunk = 0;
            if (kMla) {
                const uint4* lat = static_cast<const uint4*>(a.q_latent.ptr) +
                                   (tok * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8;
#pragma unroll
                for (int c = 0; c < 8; ++c) cp_async16(q_place(c, r), lat + 8 * c + v, on);
                chunk = 8;
            }
#pragma unroll
            for (int c = 0; c < kKeys; ++c) cp_async16(q_place(chunk + c, r), band + 8 * c + v, on);
        }
        cp_async_arrive(smem_addr(&m->q_full));
    }

    __device__ __forceinline__ void run()
    {
        const Geometry& g = a.g;
        const int values = kMla ? 8 : l.values;
        Ring ring;
        uint32_t q_phase = 0;
        for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
            const Work w = load_work(a, i);
            if (w.tiles == 0) continue;
            if (!wait(smem_addr(&m->q_empty), q_phase ^ 1)) return;
            q_phase ^= 1;
            queries(w);
            const int32_t* table_row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
            const int value_vec = kMla ? 0 : w.it.band * values * 8, band_vec = kMla ? 0 : w.it.band * kKeys * 8;
            PageOf next[4];  // of rows r0 + 16 k of the tile to come
            auto look_up = [&](long long key) {
                if (by_box(maps, w, key)) return;
#pragma unroll
                for (int k = 0; k < 4; ++k) next[k] = page_of(a, maps, w, table_row, key + r0 + 16 * k);
            };
            look_up(w.it.key0);
            for (int t = 0; t < w.tiles; ++t) {
                const long long key = w.it.key0 + (long long)t * kAttnKeys;
                const uint32_t full = smem_addr(&m->full[ring.stage]);
                const uint32_t stage = smem + l.stage + ring.stage * l.stage_bytes;
                if (by_box(maps, w, key)) {  // the load warps' tile: only these warps' arrivals
                    look_up(key + kAttnKeys);
                    if (!wait(smem_addr(&m->empty[ring.stage][kSteps - 1]), ring.phase ^ 1)) return;
                    if (tid % 32 == 0) mbar_arrive_n(full, 32);
                    ring.advance(l.stages);
                    continue;
                }
                int slot[4];  // < 0: not loaded (a pool's rows that TMA can name are numbered in 32 bits)
#pragma unroll
                for (int k = 0; k < 4; ++k) slot[k] = (int)slot_of(a, next[k]);
                if (t + 1 < w.tiles) look_up(key + kAttnKeys);
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // rows r0 + 16 k are freed by PV's step k
                    const int r = r0 + 16 * k;
                    if (!wait(smem_addr(&m->empty[ring.stage][k]), ring.phase ^ 1)) return;
                    const uint4* val = a.kv + lat_off(g, a.layer, max(slot[k], 0)) + value_vec + v;
#pragma unroll kMla ? 8 : 1
                    for (int c = 0; c < values; ++c) cp_async16(place(stage, l.row_chunks, c, r, v), val + 8 * c, slot[k] >= 0);
                    if (!kLazy) {  // (in a lazy pool the load warps bring the bands)
                        const uint4* band = a.kv + band_off(g, a.layer, max(slot[k], 0)) + band_vec + v;
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            cp_async16(maps.whole ? place(stage, l.row_chunks, values + c, r, v)
                                                  : place(stage + l.band, kKeys, c, r, v),
                                       band + 8 * c, slot[k] >= 0);
                    }
                }
                cp_async_arrive(full);  // when the copies have landed
                ring.advance(l.stages);
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
    Ring ring;

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
    __device__ __forceinline__ void next(const AttnArgs& a, int stages)
    {
        ++index;
        ring.advance(stages);
        if (++tile == tiles) {
            ++item;
            settle(a);
        }
    }
};

template <bool kMla, bool kLazy, int kKeys>
__device__ __forceinline__ void issue_mmas(const AttnArgs& a, const TileMaps& maps, const Layout& l, Misc* m, uint32_t smem,
                                           uint32_t tmem)
{
    constexpr uint32_t kDescS = mma_desc(kAttnRows, kAttnKeys, false, false);
    constexpr int kAtom = kAtomBytes / 16;
    const int values = kMla ? 8 : l.values;
    const int blocks = (values + 1) / 2;  // of 128 value dimensions; the last may have 64 of no use
    const uint64_t q_mat = smem_matrix(smem, 16, 1024);
    const uint64_t row_mat = smem_matrix(smem + l.stage, 16, l.row_chunks * kAtomBytes);
    const uint64_t band_mat =
        smem_matrix(smem + l.stage + l.band, 16, (maps.whole ? l.row_chunks : kKeys) * kAtomBytes);
    const uint64_t low_mat = smem_matrix(smem + l.stage + l.low, 16, kKeys * kAtomBytes);
    const uint64_t v_mat = smem_matrix(smem + l.stage, kAtomBytes, l.row_chunks * kAtomBytes);
    const uint64_t p_mat = smem_matrix(smem + l.p, 16, 1024);
    const uint32_t q_chunk = l.q_chunk_bytes / 16, stage16 = l.stage_bytes / 16, step16 = 2 * l.row_chunks * kAtom;
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
        // S of a tile may run one tile ahead of its product with V: there are two S buffers
        if (!s.done() && s.index <= pv.index + 1 && test(smem_addr(&m->full[s.ring.stage]), s.ring.phase) &&
            (s.tile > 0 || test(smem_addr(&m->q_full), q_phase))) {
            fence_async_smem();
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t d = tmem + kTmemS + (s.index & 1) * 64;
                const uint32_t at = s.ring.stage * stage16;
                if (kMla) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(d, q_mat + (uint64_t)(c * q_chunk + 2 * k), row_mat + (uint64_t)(at + c * kAtom + 2 * k),
                                     kDescS, c > 0 || k > 0);
                }
#pragma unroll
                for (int c = 0; c < kKeys; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t q = q_mat + (uint64_t)(((kMla ? 8 : 0) + c) * q_chunk + 2 * k);
                        mma_bf16(d, q, band_mat + (uint64_t)(at + c * kAtom + 2 * k), kDescS, kMla || c > 0 || k > 0);
                        if (kLazy)  // the low part meets the same queries
                            mma_bf16(d, q, low_mat + (uint64_t)(at + c * kAtom + 2 * k), kDescS, true);
                    }
                mma_commit(smem_addr(&m->s_full[s.index & 1]));
                if (s.tile + 1 == s.tiles) mma_commit(smem_addr(&m->q_empty));
            }
            __syncwarp();
            if (s.tile == 0) q_phase ^= 1;
            s.next(a, l.stages);
            moved = true;
        }
        if (pv.index < s.index && test(smem_addr(&m->p_ready), pv.index & 1)) {
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t desc = mma_desc(128, pv.n, true, false);
                const uint32_t at = pv.ring.stage * stage16;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                    for (int b = 0; b < (kMla ? 4 : 2); ++b)
                        if (b < blocks)
                            mma_bf16(tmem + kTmemO + b * 64, v_mat + (uint64_t)(at + k * step16 + 2 * b * kAtom), p_mat + 2 * k,
                                     desc, pv.tile > 0 || k > 0);
                    mma_commit(smem_addr(&m->empty[pv.ring.stage][k]));
                }
                mma_commit(smem_addr(&m->pv_done));
            }
            __syncwarp();
            pv.next(a, l.stages);
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

// Multiply the `n` columns of the blocks of O^T by m->factor.
__device__ __forceinline__ void scale_output(Misc* m, uint32_t tmem_o, int blocks, int n)
{
    for (int b = 0; b < blocks; ++b)
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

// The softmax warps meet at named barriers, so when the CTA gives up they go through their tiles
// without waiting instead of leaving; the status word says that the output is not valid.
template <bool kMla>
__device__ __forceinline__ void run_softmax(const AttnArgs& a, const Layout& l, Misc* m, uint32_t smem, uint32_t tmem)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t tmem_o = tmem + kTmemO + lanes;
    const float scale2 = a.scale * kLog2e, unit = scale2 > 0.f ? scale2 : 1.f;
    const int group = a.q_heads / (kMla ? 1 : a.g.rope_heads);
    const int vdim = kMla ? 512 : 64 * l.values;
    const int blocks = kMla ? 4 : (l.values + 1) / 2;
    int index = 0;  // tiles before this one
    for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
        const Work w = load_work(a, i);
        // this thread's two rows, their limits, running maxima (log2) and its part of their sums: of the weights, for lse,
        // and of the weights as the product with V has them
        int row[2];
        long long limit[2];
        float top[2];
        float2 sum[2], used[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            row[h] = 16 * warp + lane / 4 + 8 * h;
            const int tok = (w.it.row0 + min(row[h], w.it.rows - 1)) / group;
            limit[h] = row[h] < w.it.rows ? (a.prefix ? w.ch.start : w.ch.start + tok + 1) : 0;
            top[h] = -INFINITY;
            sum[h] = used[h] = make_float2(0.f, 0.f);
        }
        const long long open = a.prefix ? w.ch.start : w.ch.start + w.it.row0 / group + 1;  // every row attends below this
        const int n = padded_rows(w.it.rows);
        for (int t = 0; t < w.tiles; ++t, ++index) {
            const long long key = w.it.key0 + (long long)t * kAttnKeys;
            mbar_wait(smem_addr(&m->s_full[index & 1]), (index >> 1) & 1, &m->quit, a.status);
            tcgen05_after_sync();
            float x[32];
            float tile_top[2] = {-INFINITY, -INFINITY};
            if (16 * warp < n) {
                uint32_t v[32];
                tmem_ld_16x64(tmem + kTmemS + lanes + (index & 1) * 64, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k]);
                if (scale2 <= 0.f) {  // (else the weights' exponents are formed in one step from the products)
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] *= scale2;
                }
                if (key + kAttnKeys > open || w.it.rows < n) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int col = 8 * (k / 4) + 2 * (lane % 4) + (k & 1);
                        if (key + col >= limit[(k >> 1) & 1]) x[k] = -INFINITY;
                    }
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) tile_top[(k >> 1) & 1] = fmaxf(tile_top[(k >> 1) & 1], x[k]);
                tile_top[0] = quad_max(tile_top[0]) * unit;
                tile_top[1] = quad_max(tile_top[1]) * unit;
            }
            const bool raise = any_of_softmax(tile_top[0] > top[0] + kRaise || tile_top[1] > top[1] + kRaise);
            float factor[2] = {1.f, 1.f};
            if (raise) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float old = top[h];
                    top[h] = fmaxf(old, tile_top[h]);
                    factor[h] = top[h] == -INFINITY ? 1.f : exp2f(old - top[h]);
                    sum[h].x *= factor[h];
                    sum[h].y *= factor[h];
                    used[h].x *= factor[h];
                    used[h].y *= factor[h];
                }
            }
            // Weights, and the weights rounded to bf16 for the product with V: a matrix instruction's operands have one type,
            // and a second product for the low parts would double the work of O^T.  The output is divided by the sum of
            // the rounded weights, so it is a mean of values whichever way they round: a row that attends to one row
            // alone gets that row's value, where a sum of other weights than the product's left up to 2^-8 of it.
            uint32_t p[16];
            if (16 * warp < n) {
                const float base[2] = {top[0] == -INFINITY ? 0.f : top[0], top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int h = k & 1;
                    float2 e = fma2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(unit, unit), make_float2(-base[h], -base[h]));
                    e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                    sum[h] = add2(sum[h], e);
                    p[k] = pack_bf16x2(e.x, e.y);
                    used[h] = add2(used[h], make_float2(bf16_lo(p[k]), bf16_hi(p[k])));
                }
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
                scale_output(m, tmem_o, blocks, n);
                softmax_sync();  // before the next rescale's factors
            }
            if (16 * warp < n) {
                // the 16 x 64 weights of the warp as 8 x 8 matrices: p[2 k + h] is columns 8 k .. of rows 8 h ..; lane l gives
                // the place of row l % 8 of matrix l / 8 of each four
                const int r = 16 * warp + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                    store_matrices(smem + l.p + r * 128 + (((k + (lane >> 4)) ^ (r & 7)) << 4), p[2 * k], p[2 * k + 1],
                                   p[2 * k + 2], p[2 * k + 3]);
            }
            fence_async_smem();
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&m->p_ready));
        }
        // the tile's result
        float sums[2] = {quad_sum(sum[0].x + sum[0].y), quad_sum(sum[1].x + sum[1].y)};
        float weights[2] = {quad_sum(used[0].x + used[0].y), quad_sum(used[1].x + used[1].y)};
        if (lane % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m->factor[row[h]] = weights[h] == 0.f ? 0.f : 1.f / weights[h];
                if (row[h] >= w.it.rows) continue;
                const float lse = sums[h] == 0.f ? -INFINITY : (top[h] + log2f(sums[h])) * kLn2;
                if (w.it.part >= 0) {
                    a.part_lse[(long long)w.it.part * kAttnRows + row[h]] = lse;
                } else if (a.lse) {
                    const int r = w.it.row0 + row[h];
                    a.lse[(long long)(w.ch.tok0 + r / group) * a.q_heads + w.it.band * group + r % group] = lse;
                }
            }
        }
        softmax_sync();
        if (w.tiles > 0) {
            mbar_wait(smem_addr(&m->pv_done), (index - 1) & 1, &m->quit, a.status);
            tcgen05_after_sync();
        }
        bool redo = false;
        for (int c = 0; c < n; c += 16)  // (P is free)
            redo |= put_rows<kAttnRows>(a, w, group, vdim, c, 32 * warp, 128, blocks, tmem_o + c, 64, m->factor + c,
                                        smem + l.p + warp * 1024);
        tcgen05_before_sync();
        redo = any_of_softmax(redo);  // and before the next item's factors
        if (threadIdx.x == 0) {
            a.redo[2 * i] = redo;
            if (redo) m->redo = 1;
        }
    }
}

template <bool kMla, bool kLazy, int kKeys>
__global__ void __launch_bounds__(kThreads, 1) attend_tile_kernel(const __grid_constant__ AttnArgs a,
                                                               const __grid_constant__ TileMaps maps)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const Layout l = kMla ? make_layout(true, kLazy, kLazy ? false : maps.whole != 0, 1, 8, 2)
                          : make_layout(false, kLazy, false, kKeys, maps.values, maps.stages);
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    Misc* m = reinterpret_cast<Misc*>(raw + (smem - smem_addr(raw)) + l.misc);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            // the load warps (lazy pools: and again for the turned bands) and every copy thread
            mbar_init(smem_addr(&m->full[s]), (kLazy ? 2 : 1) * kLoadWarps + kCopyThreads);
            for (int k = 0; k < kSteps; ++k) mbar_init(smem_addr(&m->empty[s][k]), 1);
        }
        mbar_init(smem_addr(&m->q_full), kCopyThreads);
        mbar_init(smem_addr(&m->q_empty), 1);
        mbar_init(smem_addr(&m->s_full[0]), 1);
        mbar_init(smem_addr(&m->s_full[1]), 1);
        mbar_init(smem_addr(&m->p_ready), kSoftmaxWarps);
        mbar_init(smem_addr(&m->pv_done), 1);
        mbar_init(smem_addr(&m->drained), 1);
        m->quit = m->redo = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&m->tmem), kTmemCols);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = m->tmem;
    wait_for_previous_grid();
    // (the next kernel is let in by this one's end: let in before, the join's waiting CTAs cost 15 us of a call of 26)
    if (a.header->pairs) {  // the plan is for the other kernel
    } else if (warp < kSoftmaxWarps) {
        run_softmax<kMla>(a, l, m, smem, tmem);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        issue_mmas<kMla, kLazy, kKeys>(a, maps, l, m, smem, tmem);
        // nothing is in flight when TMEM is freed
        if (elect_lane()) mma_commit(smem_addr(&m->drained));
        __syncwarp();
        const unsigned long long t0 = global_ns();
        while (!mbar_try(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
        }
    } else if (warp < kLoadWarp + kLoadWarps) {
        const int step = warp - kLoadWarp;
        if (kLazy) {
            float2* trig = reinterpret_cast<float2*>(raw + (smem - smem_addr(raw)) + l.trig) + step * 32 * kKeys;
            load_lazy<kMla, kKeys>(a, maps, l, m, smem, step, trig);
        } else {
            if (elect_lane()) load_tiles<kMla, kKeys>(a, maps, l, m, smem, step);
            __syncwarp();
        }
    } else {
        const int tid = threadIdx.x - 32 * (kLoadWarp + kLoadWarps);
        Copier<kMla, kLazy, kKeys> c{a, maps, l, m, smem, tid, tid % 8, tid / 8};
        c.run();
        cp_async_wait_all();
    }
    __syncthreads();
    let_loads_land(&m->quit);
    if (warp == kMmaWarp) {
        tcgen05_after_sync();
        tmem_free(tmem, kTmemCols);
    }
    const bool redo = m->redo && !m->quit;
    __syncthreads();  // before shared memory is written again
    if (redo) {
        for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i)
            if (a.redo[2 * i]) attend_rows<kThreads>(a, a.items[i], 0, a.items[i].rows, kAttnRows, raw);
    }
}

// Map of `rows` rows of row_vecs 16-byte vectors at `base`: 64 columns, 8 rows of a group, planes of 64 columns, groups;
// boxes of box_planes planes of box_groups groups.
bool make_map(EncodeTiled encode, CUtensorMap* map, const uint4* base, int64_t rows, int row_vecs, int planes, int box_planes,
              int box_groups)
{
    const cuuint64_t row = (cuuint64_t)row_vecs * 16;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)planes, (cuuint64_t)(rows / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)box_planes, (cuuint32_t)box_groups}, steps[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint4*>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using Kernel = void (*)(AttnArgs, TileMaps);

Kernel kernel_of(const Geometry& g)
{
    const bool lazy = (g.flags & LEYLINE_POOL_LAZY) != 0;
    if (g.rope_heads <= 1) return lazy ? attend_tile_kernel<true, true, 1> : attend_tile_kernel<true, false, 1>;
    switch (g.rope_dim) {
    case 64: return lazy ? attend_tile_kernel<false, true, 1> : attend_tile_kernel<false, false, 1>;
    case 128: return lazy ? attend_tile_kernel<false, true, 2> : attend_tile_kernel<false, false, 2>;
    default: return lazy ? attend_tile_kernel<false, true, 4> : attend_tile_kernel<false, false, 4>;
    }
}

Layout layout_of(const Geometry& g, const TileMaps& maps)
{
    return make_layout(g.rope_heads <= 1, (g.flags & LEYLINE_POOL_LAZY) != 0, maps.whole != 0, g.rope_dim / 64, maps.values,
                       maps.stages);
}

// The tiles' shared memory, or what attend_rows needs.
int smem_of(const Geometry& g, const TileMaps& maps)
{
    return std::max(layout_of(g, maps).bytes, (int)any_shape(g).bytes);
}

}  // namespace

bool attention_takes_tiles(const Geometry& g)
{
    if (g.num_pages * g.block_size * g.num_layers > INT32_MAX) return false;  // rows as 32-bit coordinates
    if (g.rope_heads <= 1) return g.latent_vecs == 64 && g.rope_vecs == 8;
    const int value = g.latent_dim / g.rope_heads;
    return value % 64 == 0 && value >= 64 && value <= 256 && (g.rope_dim == 64 || g.rope_dim == 128 || g.rope_dim == 256);
}

int attention_tile_prepare(const Geometry& g, const void* kv, TileMaps* maps)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return (int)cudaErrorNotSupported;
    const uint4* base = static_cast<const uint4*>(kv);
    const bool mla = g.rope_heads <= 1;
    // rows of every layer follow one another, in whole rows and in the arrays of a split-rope pool alike
    const int64_t rows = g.num_pages * g.block_size * g.num_layers;
    const int keys = g.rope_dim / 64;
    maps->values = g.latent_dim / 64 / (mla ? 1 : g.rope_heads);
    maps->whole = mla && !(g.flags & (LEYLINE_POOL_SPLIT_ROPE | LEYLINE_POOL_LAZY));
    maps->box = g.block_size % 16 == 0 ? 16 : g.block_size % 8 == 0 ? 8 : 0;
    maps->shift = -1;
    for (int k = 0; k < 31; ++k)
        if (g.block_size == 1 << k) maps->shift = k;
    maps->stages = mla ? 2 : kMaxStages;
    while (maps->stages > 1 && layout_of(g, *maps).bytes > kMaxSmem) --maps->stages;
    const int groups = maps->box / 8;
    const int planes = g.latent_dim / 64 + (maps->whole ? keys : 0);
    if (maps->box && (!make_map(encode, &maps->rows, base, rows, g.lat_row_vecs, planes,
                                maps->values + (maps->whole ? keys : 0), groups) ||
                      !make_map(encode, &maps->bands, base + g.rope_base_vecs, rows, g.rope_row_vecs,
                                keys * std::max(g.rope_heads, 1), keys, groups)))
        return (int)cudaErrorInvalidValue;
    return (int)cudaFuncSetAttribute(kernel_of(g), cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(g, *maps));
}

int launch_attention_tile(const AttnArgs& a, const TileMaps& maps, int ctas, void* stream)
{
    return (int)launch_dependent_smem(kernel_of(a.g), ctas, kThreads, smem_of(a.g, maps), (cudaStream_t)stream, a, maps);
}

}  // namespace leyline
