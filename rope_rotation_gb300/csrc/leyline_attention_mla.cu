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
//   warp 4     one thread issues every MMA
//   warps 5-8  copy queries and cache rows to shared memory (16-byte cp.async through the block
//              table), into a ring of 18 column chunks of 64 rows x 64 columns, two tiles' worth,
//              each with barriers of its own
// In a lazy pool the band of each row is turned by its pending count on the way, in fp32, and goes
// to shared memory as the sum of two bf16 values (a chunk for each): the scores then carry the turn
// to 2^-17, not to the 2^-9 of one bf16 rounding, which the other rows do not have either.
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
constexpr int kCopyWarps = 4;
constexpr int kCopyThreads = 32 * kCopyWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + 1 + kCopyWarps);

constexpr int kChunks = 9;                           // 64-wide column chunks of a row: latent 0..7, band 8
constexpr int kLatentChunks = 8;
constexpr int kChunkBytes = kAttnKeys * 128;         // 64 rows x 128 bytes
// The ring: a tile takes its band's chunk (lazy pools: high and low part), then the latent's.  18 is
// even and so are a lazy tile's 10, and 9 + 9 fill it: the two chunks of a block of O^T (2 x 64 value
// dimensions) always lie side by side.
constexpr int kSlots = 18;
constexpr int kQOff = 0;
constexpr int kRingOff = kQOff + kChunks * kChunkBytes;
constexpr int kPOff = kRingOff + kSlots * kChunkBytes;
constexpr int kMiscOff = kPOff + kChunkBytes;

struct Misc {
    unsigned long long full[kSlots];
    unsigned long long empty[kSlots];
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2];
    unsigned long long p_ready, pv_done, drained;
    uint32_t tmem;
    int quit;
    float factor[kAttnRows];              // rescale, then 1 / l
    float2 trig[kCopyWarps][32];          // lazy pools: cos, sin of the last pending count
};
constexpr int kSmemBytes = kMiscOff + (int)sizeof(Misc) + 1024;  // and room to align the start
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // 4 blocks of 64 columns
constexpr uint32_t kTmemS = 256;  // 2 buffers of 64 columns

constexpr float kRaise = 8.f;

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

// ------------------------------------------------------------------- copies --
struct Copier {
    const AttnArgs& a;
    Misc* m;
    uint32_t smem;
    int tid, v, r0;  // 16-byte chunk of a 128-byte row segment, first row
    int trig_count;  // pending count whose cos / sin this warp's slice holds
    bool trig_valid;

    // False (for the whole warp) when the CTA has given up.
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, &m->quit, a.status));
    }

    // Slots of this thread's rows (r0 + 16 i) of the tile at `key`; -1: not loaded.
    __device__ __forceinline__ void slots(const Work& w, long long key, int (&page)[4], int (&off)[4])
    {
        const int32_t* row = a.header->table + (long long)w.ch.req * a.header->max_blocks;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned pos = (unsigned)(key + r0 + 16 * i);
            const unsigned blk = pos / (unsigned)a.g.block_size;
            off[i] = (int)(pos - blk * (unsigned)a.g.block_size);
            page[i] = pos < (unsigned long long)w.end ? row[blk] : -1;
        }
    }

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

    __device__ __forceinline__ uint32_t place(uint32_t chunk_base, int row) const
    {
        return chunk_base + row * 128 + ((v ^ (row & 7)) << 4);
    }

    __device__ __forceinline__ void run()
    {
        const uint4* kv = a.kv;
        const Geometry& g = a.g;
        const int group = a.q_heads;
        int slot_at = 0;     // next slot of the ring
        uint32_t phase = 0;  // of its use
        uint32_t q_phase = 0;
        trig_valid = false;
        auto next_slot = [&] {
            if (++slot_at == kSlots) {
                slot_at = 0;
                phase ^= 1;
            }
        };
        auto store = [&](int slot, int r, const uint4& y) {
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(place(smem + kRingOff + slot * kChunkBytes, r)),
                         "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                         : "memory");
        };
        for (int i = a.cta_begin[blockIdx.x]; i < a.cta_begin[blockIdx.x + 1]; ++i) {
            const Work w = load_work(a, i);
            if (w.tiles == 0) continue;
            if (!wait(smem_addr(&m->q_empty), q_phase ^ 1)) return;
            q_phase ^= 1;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int r = r0 + 16 * k;
                const bool on = r < w.it.rows;
                const int row = w.it.row0 + (on ? r : 0);
                const long long tok = w.ch.tok0 + row / group, head = row % group;
                const uint4* lat =
                    static_cast<const uint4*>(a.q_latent.ptr) + (tok * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8;
                const uint4* band =
                    static_cast<const uint4*>(a.q_rope.ptr) + (tok * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8;
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    cp_async16(place(smem + kQOff + c * kChunkBytes, r), c < 8 ? lat + 8 * c + v : band + v, on);
            }
            cp_async_arrive(smem_addr(&m->q_full));
            int page[4], off[4];
            slots(w, w.it.key0, page, off);
            for (int t = 0; t < w.tiles; ++t) {
                const long long key = w.it.key0 + (long long)t * kAttnKeys;
                const uint4 *lat[4], *band[4];
                bool on[4];
                int pend[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    on[k] = page[k] >= 0 && page[k] < g.num_pages;
                    if (!on[k] && key + r0 + 16 * k < w.end) raise_status(a.status, ST_BAD_PAGE);
                    const long long slot = on[k] ? (long long)page[k] * g.block_size + off[k] : 0;
                    lat[k] = kv + lat_off(g, a.layer, slot) + v;
                    band[k] = kv + band_off(g, a.layer, slot) + v;
                    pend[k] = a.pending && on[k] ? a.pending[slot] : 0;
                }
                if (t + 1 < w.tiles) slots(w, key + kAttnKeys, page, off);  // in flight while this tile is copied
                // the band first: its slot is free again as soon as S is done
                if (!wait(smem_addr(&m->empty[slot_at]), phase ^ 1)) return;
                if (a.pending) {
                    uint4 hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) hi[k] = on[k] ? ld_stream(band[k]) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 x = hi[k];
                        turned(x, pend[k], hi[k], lo[k]);
                        store(slot_at, r0 + 16 * k, hi[k]);
                    }
                    fence_async_smem();
                    mbar_arrive(smem_addr(&m->full[slot_at]));
                    next_slot();
                    if (!wait(smem_addr(&m->empty[slot_at]), phase ^ 1)) return;
#pragma unroll
                    for (int k = 0; k < 4; ++k) store(slot_at, r0 + 16 * k, lo[k]);
                    fence_async_smem();
                    mbar_arrive(smem_addr(&m->full[slot_at]));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        cp_async16(place(smem + kRingOff + slot_at * kChunkBytes, r0 + 16 * k), band[k], on[k]);
                    cp_async_arrive(smem_addr(&m->full[slot_at]));
                }
                next_slot();
#pragma unroll 2
                for (int c = 0; c < kLatentChunks; ++c) {
                    if (!wait(smem_addr(&m->empty[slot_at]), phase ^ 1)) return;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        cp_async16(place(smem + kRingOff + slot_at * kChunkBytes, r0 + 16 * k), lat[k] + 8 * c, on[k]);
                    cp_async_arrive(smem_addr(&m->full[slot_at]));
                    next_slot();
                }
            }
        }
    }
};

// --------------------------------------------------------------------- MMAs --
// The tiles of the CTA's items in order, as the issuing thread walks them.
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

__device__ __forceinline__ void issue_mmas(const AttnArgs& a, Misc* m, uint32_t smem, uint32_t tmem)
{
    constexpr uint32_t kDescS = mma_desc(kAttnRows, kAttnKeys, false, false);
    const int band_chunks = a.pending ? 2 : 1;
    const int tile_chunks = band_chunks + kLatentChunks;
    TileCursor s, pv;
    s.start(a);
    pv.start(a);
    int chunk = 0;            // next chunk of S
    int s_slot = 0, pv_slot = 0;  // first slots of the two cursors' tiles
    uint32_t s_phase = 0;     // of slot s_slot + chunk
    uint32_t q_phase = 0;
    unsigned long long t0 = global_ns();
    while (!pv.done()) {
        bool moved = false;
        // S of a tile may run one tile ahead of its product with V: there are two S buffers
        if (!s.done() && s.index <= pv.index + 1) {
            const int at = s_slot + chunk < kSlots ? s_slot + chunk : s_slot + chunk - kSlots;
            bool ready = chunk > 0 || s.tile > 0 || mbar_test(smem_addr(&m->q_full), q_phase);
            ready = ready && mbar_test(smem_addr(&m->full[at]), s_phase);
            if (ready) {
                fence_async_smem();
                tcgen05_after_sync();
                const uint32_t k_at = smem + kRingOff + at * kChunkBytes;
                const uint32_t q_at = smem + kQOff + (chunk < band_chunks ? kLatentChunks : chunk - band_chunks) * kChunkBytes;
                const uint32_t d = tmem + kTmemS + (s.index & 1) * 64;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16(d, smem_matrix(q_at + k * 32, 16, 1024), smem_matrix(k_at + k * 32, 16, 1024), kDescS,
                             chunk > 0 || k > 0);
                if (at + 1 == kSlots) s_phase ^= 1;
                if (++chunk == tile_chunks) {
                    chunk = 0;
                    mma_commit(smem_addr(&m->s_full[s.index & 1]));
                    for (int c = 0; c < band_chunks; ++c) mma_commit(smem_addr(&m->empty[s_slot + c]));
                    s_slot += tile_chunks;
                    if (s_slot >= kSlots) s_slot -= kSlots;
                    if (s.tile == 0) q_phase ^= 1;
                    if (s.tile + 1 == s.tiles) mma_commit(smem_addr(&m->q_empty));
                    s.next(a);
                }
                moved = true;
            }
        }
        if (pv.index < s.index && mbar_test(smem_addr(&m->p_ready), pv.index & 1)) {
            tcgen05_after_sync();
            const uint32_t desc = mma_desc(128, pv.n, true, false);
            for (int b = 0; b < 4; ++b) {
                int at = pv_slot + band_chunks + 2 * b;
                if (at >= kSlots) at -= kSlots;
                const uint32_t v_at = smem + kRingOff + at * kChunkBytes;
#pragma unroll
                for (int k = 0; k < kAttnKeys / 16; ++k)
                    mma_bf16(tmem + kTmemO + b * 64, smem_matrix(v_at + k * 2048, kChunkBytes, 1024),
                             smem_matrix(smem + kPOff + k * 32, 16, 1024), desc, pv.tile > 0 || k > 0);
                mma_commit(smem_addr(&m->empty[at]));
                mma_commit(smem_addr(&m->empty[at + 1]));
            }
            mma_commit(smem_addr(&m->pv_done));
            pv_slot += tile_chunks;
            if (pv_slot >= kSlots) pv_slot -= kSlots;
            pv.next(a);
            moved = true;
        }
        if (moved) {
            t0 = global_ns();
        } else {
            if (*(volatile int*)&m->quit) break;
            if (global_ns() - t0 > kWaitLimit) {
                *(volatile int*)&m->quit = 1;
                raise_status(a.status, ST_TIMEOUT);
                break;
            }
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

__device__ __forceinline__ void run_softmax(const AttnArgs& a, Misc* m, uint32_t smem, uint32_t tmem)
{
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
                const float e0 = exp2f(x[2 * k] - base[h]), e1 = exp2f(x[2 * k + 1] - base[h]);
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
#pragma unroll
            for (int k = 0; k < 16; ++k) {  // value k: columns 8 (k / 2) + 2 (lane % 4), + 1 of row[k & 1]
                const int r = row[k & 1];
                const uint32_t at = smem + kPOff + r * 128 + (((k / 2) ^ (r & 7)) << 4) + 4 * (lane % 4);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(p[k]) : "memory");
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

__global__ void __launch_bounds__(kThreads, 1) attend_mla_kernel(const __grid_constant__ AttnArgs a)
{
    extern __shared__ unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    Misc* m = reinterpret_cast<Misc*>(raw + (smem - smem_addr(raw)) + kMiscOff);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_addr(&m->full[s]), kCopyThreads);
            mbar_init(smem_addr(&m->empty[s]), 1);
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
        run_softmax(a, m, smem, tmem);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        if ((threadIdx.x & 31) == 0) {
            issue_mmas(a, m, smem, tmem);
            // nothing is in flight when TMEM is freed
            mma_commit(smem_addr(&m->drained));
            const unsigned long long t0 = global_ns();
            while (!mbar_try(smem_addr(&m->drained), 0) && global_ns() - t0 < kWaitLimit) {
            }
        }
    } else {
        const int tid = threadIdx.x - 32 * (kMmaWarp + 1);
        Copier c{a, m, smem, tid, tid % 8, tid / 8, 0, false};
        c.run();
        cp_async_wait_all();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tcgen05_after_sync();
        tmem_free(tmem, kTmemCols);
    }
}

}  // namespace

int attention_mla_prepare()
{
    return (int)cudaFuncSetAttribute(attend_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

int launch_attention_mla(const AttnArgs& a, int ctas, void* stream)
{
    return (int)launch_dependent_smem(attend_mla_kernel, ctas, kThreads, kSmemBytes, (cudaStream_t)stream, a);
}

}  // namespace leyline
