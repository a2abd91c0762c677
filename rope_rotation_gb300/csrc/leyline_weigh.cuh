// leyline_weigh.cuh -- what the kernels that weigh rows on the tensor cores share (leyline_weigh_tile.cu,
// leyline_weigh_pair.cu): how a tile's keys come to shared memory, and how a product's columns are summed.
//
// Both operands of S^T = K Q^T lie in shared memory as chunks of 64 columns, 128 bytes a row, swizzled: 16 KB for the 128
// cache rows of a CTA.  A cache row is a TMEM lane, so a thread of the epilogue has a row of S^T and sums its columns in
// registers: no reduction across threads, and a masked or bad row spoils no other.
#pragma once

#include "leyline_attention.cuh"

namespace leyline {
namespace {

constexpr int kChunkBytes = kWeighKeys * 128;
constexpr int kMaxChunks = 10;  // of a key: 8 of the latent, the band and its low part
constexpr int kMaxStages = 13;

// The kind of rows.
struct Shape {
    int bands, group;
    int tokens, heads, blocks;  // query tile: tokens, heads of a token; tiles of a token's heads
    int latent, keys, low;      // chunks of a key: of the latent, of the band, of the band's low part
    int q_chunks, chunks;
    int stay_bytes, stages;     // shared memory of what stays; chunks that pass
};

__device__ __forceinline__ Shape make_shape(const WeighArgs& a, bool lazy)
{
    Shape s;
    const bool mla = a.g.rope_heads <= 1;
    s.bands = mla ? 1 : a.g.rope_heads;
    s.group = a.q_heads / s.bands;
    s.tokens = weigh_tokens(s.group);
    s.heads = min(s.group, kWeighCols);
    s.blocks = (s.group + kWeighCols - 1) / kWeighCols;
    s.latent = mla ? a.g.latent_vecs / 8 : 0;
    s.keys = a.g.head_vecs / 8;
    s.low = lazy ? s.keys : 0;
    s.q_chunks = s.latent + s.keys;
    s.chunks = s.q_chunks + s.low;
    s.stay_bytes = s.stages = 0;
    return s;
}

struct Tile {
    int key0, keys;  // cache rows of the request
};

__device__ __forceinline__ int padded(int cols) { return (cols + 15) & ~15; }

// The one of n requests whose work holds unit x.
__device__ __forceinline__ WeighReq find_request(const WeighReq* reqs, int n, long long x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (reqs[mid].begin <= x) lo = mid;
        else hi = mid - 1;
    }
    return reqs[lo];
}

// (A replayed plan's table may have more requests or rows than the weights.)
__device__ __forceinline__ bool weights_hold(const WeighArgs& a, const WeighReq& r)
{
    return r.req < a.num_reqs && r.end <= a.rows;
}

__device__ __forceinline__ void store_weight(const WeighArgs& a, const WeighReq& r, int key, float got)
{
    const int page = a.header->table[(long long)r.req * a.header->max_blocks + key / a.g.block_size];
    if (page < 0 || page >= a.g.num_pages) return;  // (the loads have raised the status)
    float* w = a.weights + r.req * a.req_stride + key;
    *w = a.decay == 0.f ? got : fmaf(a.decay, *w, got);
}

__device__ __forceinline__ uint4 load_smem(uint32_t at)
{
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void store_smem(uint32_t at, const uint4& x)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// A turned value as bf16, and what its rounding leaves (nothing in the naive arm, whose result is the rounded one).
__device__ __forceinline__ uint32_t split_value(bool naive, float q0, float q1, uint32_t& low)
{
    const uint32_t high = pack_bf16x2(q0, q1);
    low = naive ? 0u : pack_bf16x2(q0 - bf16_lo(high), q1 - bf16_hi(high));
    return high;
}
// Half-split pairs: 8 first halves (or second ones) `mine` turned with their others by t[0 .. 7].
__device__ __forceinline__ uint4 turned_half(bool naive, const uint4& mine, const uint4& other, const float2* t, bool first, uint4& low)
{
    const uint32_t* mw = reinterpret_cast<const uint32_t*>(&mine);
    const uint32_t* ow = reinterpret_cast<const uint32_t*>(&other);
    uint4 high;
    uint32_t* hw = reinterpret_cast<uint32_t*>(&high);
    uint32_t* lw = reinterpret_cast<uint32_t*>(&low);
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // x' = x c - y s of the first half, y' = y c + x s of the second
        const float4 u = *reinterpret_cast<const float4*>(t + 2 * e);
        const float a0 = bf16_lo(mw[e]), a1 = bf16_hi(mw[e]);
        const float b0 = bf16_lo(ow[e]) * (first ? -u.y : u.y), b1 = bf16_hi(ow[e]) * (first ? -u.w : u.w);
        const float q0 = naive ? round_bf16(a0 * u.x) + round_bf16(b0) : fmaf(a0, u.x, b0);
        const float q1 = naive ? round_bf16(a1 * u.z) + round_bf16(b1) : fmaf(a1, u.z, b1);
        hw[e] = split_value(naive, q0, q1, lw[e]);
    }
    return high;
}
// Interleaved pairs: 4 of them by t[0 .. 3].
__device__ __forceinline__ uint4 turned_pairs(bool naive, const uint4& mine, const float2* t, uint4& low)
{
    const uint32_t* mw = reinterpret_cast<const uint32_t*>(&mine);
    uint4 high;
    uint32_t* hw = reinterpret_cast<uint32_t*>(&high);
    uint32_t* lw = reinterpret_cast<uint32_t*>(&low);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float q0, q1;
        if (naive) turn_bf16(bf16_lo(mw[e]), bf16_hi(mw[e]), t[e].x, t[e].y, q0, q1);
        else turn_fp32(bf16_lo(mw[e]), bf16_hi(mw[e]), t[e].x, t[e].y, q0, q1);
        hw[e] = split_value(naive, q0, q1, lw[e]);
    }
    return high;
}

// cos and sin of count * theta_j of `pairs` pairs as a read of the pool forms them, rounded to bf16, by a warp.
__device__ __noinline__ void naive_trig(int count, const double* turn, int pairs, float2* cs)
{
    for (int j = threadIdx.x & 31; j < pairs; j += 32) {
        float c, s;
        pending_trig(count, turn, pairs, j, true, c, s);
        cs[j] = make_float2(c, s);
    }
}

// --------------------------------------------------------------------- keys --
// The warps that bring a CTA's 128 cache rows, kRows of them each: boxes of 16 or 8 rows by TMA where 8 divides the block
// size, else a row at a time.  In a lazy pool (kKeys > 0: the chunks of a band) they turn each row's band by its pending
// count, in fp32, into the sum of two bf16 values, as leyline_attention_tile.cu does: the scores carry it to 2^-17.
// The chunks of both CTAs of a pair are counted in the first, whose warps alone arrive for boxes (an arrival from the other
// CTA is slow), for all that are expected of both.
template <int kWarps, int kKeys>
struct KeyLoader {
    static constexpr bool kLazy = kKeys > 0;
    static constexpr int kTurned = kLazy ? kKeys : 1;
    static constexpr int kRows = kWeighKeys / kWarps;  // 16 or 32
    const WeighArgs& a;
    const WeighMaps& maps;
    const Shape& s;
    float2* cs;           // lazy pools: cos, sin of `count`, this warp's
    const double* turns;  // theta_j as a part of a whole turn
    int warp, lane;
    uint32_t rank;
    // of row kRows * warp + lane of the tile at `slot_key` of request `slot_req`: -1 where there is none
    long long slot = -1;
    int slot_key = -1, slot_req = -1;
    int next_page = -1, next_key = -1, next_req = -1;  // pages of the tile to come
    int count = 0;
    bool counted = false;

    // Whether this thread's row is one of a tile of `keys`.
    __device__ __forceinline__ bool has_row(int keys) const { return lane < kRows && kRows * warp + lane < keys; }
    __device__ __forceinline__ int page_of_row(const WeighReq& r, int key0, int keys) const
    {
        if (!has_row(keys)) return -1;
        const unsigned u = (unsigned)(key0 + kRows * warp + lane), B = (unsigned)a.g.block_size;
        return a.header->table[(long long)r.req * a.header->max_blocks + (maps.shift >= 0 ? u >> maps.shift : u / B)];
    }
    __device__ __forceinline__ long long slot_at(int page, int key0) const
    {
        if (page < 0 || page >= a.g.num_pages) return -1;
        const unsigned u = (unsigned)(key0 + kRows * warp + lane), B = (unsigned)a.g.block_size;
        return (long long)page * B + (u - (maps.shift >= 0 ? u >> maps.shift << maps.shift : u / B * B));
    }
    __device__ __forceinline__ void look_up(const WeighReq& r, const Tile& t)
    {
        if (slot_key == t.key0 && slot_req == r.req) return;
        const int page = next_key == t.key0 && next_req == r.req ? next_page : page_of_row(r, t.key0, t.keys);
        slot_key = t.key0;
        slot_req = r.req;
        slot = slot_at(page, t.key0);
        if (slot < 0 && has_row(t.keys)) raise_status(a.status, ST_BAD_PAGE);
    }
    // The pages of the next tile are read while this one is loaded.  (Asking for its rows in L2 as well, whole, cost more
    // than it gave: 16 decodes of 16 heads over some 30000 rows 107 -> 115 us.)
    __device__ __forceinline__ void look_ahead(const WeighReq& r, const Tile& t)
    {
        next_page = page_of_row(r, t.key0, t.keys);
        next_key = t.key0;
        next_req = r.req;
    }

    // cos and sin of c * theta_j: the angle in turns in fp64, less its whole ones, then in fp32.  They are off by 2^-22 of the
    // pair, where the scores carry a turned band to 2^-17.  (The product of the pool's two tables, in fp64, takes two loads
    // from L2 for each pair, and every warp was held up by it wherever the count changed: 64 decodes of 16 heads over some
    // 5000 rows, one a page, 157 us instead of 129.)
    __device__ __forceinline__ void ensure(int c)
    {
        if (counted && c == count) return;
        __syncwarp();
        if (a.g.precision == LEYLINE_ROTATE_BF16_NAIVE) {
            naive_trig(c, a.turn, 32 * kTurned, cs);
        } else {
#pragma unroll
            for (int i = 0; i < kTurned; ++i) {
                const double t = (double)c * turns[lane + 32 * i];
                float si, co;
                sincospif(2.f * (float)(t - rint(t)), &si, &co);
                cs[lane + 32 * i] = make_float2(co, si);
            }
        }
        __syncwarp();
        count = c;
        counted = true;
    }

    // Place of 16 bytes v of this warp's row r in a plane at `plane`, whose groups of 8 rows lie `pitch` bytes apart.
    __device__ __forceinline__ uint32_t place(uint32_t plane, int pitch, int r, int v) const
    {
        return plane + (kRows * warp + r) / 8 * pitch + (r & 7) * 128 + ((v ^ (r & 7)) << 4);
    }

    // Lazy pools: this warp's rows of chunks c0 and, if there are two, c1 of a band are copied as they are to planes 0 and 1
    // at `dst`, and their counts to `counts`, one for each row of the warp ...
    __device__ __forceinline__ void copy_bands(int band, int c0, int c1, bool two, uint32_t dst, int pitch, uint32_t counts) const
    {
        const int v = lane % 8;
#pragma unroll
        for (int k = 0; k < kRows / 4; ++k) {
            const int r = lane / 8 + 4 * k;
            const long long at = __shfl_sync(0xffffffffu, slot, r);
            const uint4* from = a.kv + band_off(a.g, a.layer, max(at, 0ll)) + band * a.g.head_vecs + v;
            cp_async16(place(dst, pitch, r, v), from + 8 * c0, at >= 0);
            if (two) cp_async16(place(dst + kAtomBytes, pitch, r, v), from + 8 * c1, at >= 0);
        }
        if (lane < kRows) cp_async4(counts + 4 * lane, a.pending + max(slot, 0ll), slot >= 0);
    }

    // ... and once they have landed turned there; what their rounding to bf16 leaves goes to the planes behind them.  Half-split
    // pairs: chunk c0 alone holds both halves of its pairs, or c0 and c1 the first and the second ones.  By pairs of rows,
    // whose chains run side by side.  (Held in registers from one tile to the next the bands spilled, and the spills waited
    // for their loads: 16 decodes of 16 heads over some 30000 rows 256 us.)
    template <bool kSplit, bool kTwo>
    __device__ __forceinline__ void turn_as(int c0, int c1, uint32_t dst, int pitch, const int* counts)
    {
        const bool naive = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        const int v = lane % 8;
        const uint32_t low = dst + (kTwo ? 2 : 1) * kAtomBytes;
        const bool first = kTwo || v < 4;  // x holds the first half of its pairs
#pragma unroll 1
        for (int k = 0; k < kRows / 4; k += 2) {
            const int r0 = lane / 8 + 4 * k;
            const int turns[2] = {counts[r0], counts[r0 + 4]};
            uint4 x[2], y[2];  // y: the other halves of the pairs, or chunk c1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[i] = load_smem(place(dst, pitch, r0 + 4 * i, v));
                if (kTwo) y[i] = load_smem(place(dst + kAtomBytes, pitch, r0 + 4 * i, v));
                else if (kSplit) y[i] = shfl_xor_vec(x[i], 4);
            }
            // mostly all rows of a warp share a count; else a pass for each
            bool left[2] = {true, true};
            for (;;) {
                const unsigned lanes = __ballot_sync(0xffffffffu, left[0] || left[1]);
                if (lanes == 0) break;
                const int n = __shfl_sync(0xffffffffu, left[0] ? turns[0] : turns[1], __ffs(lanes) - 1);
                if (n != 0) ensure(n);
                const float2* t = cs + (!kSplit ? 32 * c0 + 4 * v : kTwo ? 64 * c0 + 8 * v : 8 * (v & 3));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!left[i] || turns[i] != n) continue;
                    left[i] = false;
                    const uint32_t to = place(dst, pitch, r0 + 4 * i, v), to_low = place(low, pitch, r0 + 4 * i, v);
                    uint4 l = make_uint4(0, 0, 0, 0), m = l;
                    if (n != 0) {
                        store_smem(to, kSplit ? turned_half(naive, x[i], y[i], t, first, l) : turned_pairs(naive, x[i], t, l));
                        if (kTwo)
                            store_smem(to + kAtomBytes, kSplit ? turned_half(naive, y[i], x[i], t, false, m)
                                                               : turned_pairs(naive, y[i], t + 32 * (c1 - c0), m));
                    }
                    store_smem(to_low, l);
                    if (kTwo) store_smem(to_low + kAtomBytes, m);
                }
            }
        }
    }
    __device__ __forceinline__ void turn_bands(int c0, int c1, bool two, uint32_t dst, int pitch, const int* counts)
    {
        const bool split = a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
        if constexpr (kTurned == 1) {
            if (split) turn_as<true, false>(c0, c1, dst, pitch, counts);
            else turn_as<false, false>(c0, c1, dst, pitch, counts);
        } else {
            if (split) turn_as<true, true>(c0, c1, dst, pitch, counts);
            else turn_as<false, true>(c0, c1, dst, pitch, counts);
        }
        fence_async_smem();  // (slow: once for all)
        __syncwarp();
    }

    // An arrival of this warp (its lane 0) for what it has written to shared memory.
    __device__ __forceinline__ void arrive(uint32_t bar) const
    {
        cluster_arrive_smem(cluster_addr(bar, 0));
    }

    // This warp's rows of `n` planes from plane p on of the latents (whole MLA rows: and their band), or of the bands, to `dst`,
    // by boxes of as many planes; an arrival on `bar`.
    __device__ __forceinline__ void box_planes(bool in_rows, int box, int p, int n, uint32_t dst, uint32_t bar)
    {
        // the lane of a box's first row asks for it
        const CUtensorMap* map = in_rows ? &maps.rows[box] : &maps.bands[box];
        const int base = (int)((long long)a.layer * a.g.num_pages * a.g.block_size / 8);
        const uint32_t to = dst + (kRows * warp + lane) * 128 * n;
        if (lane == 0 && rank == 0) {
            mbar_expect_tx(bar, 2 * kRows * 128 * n);
            mbar_arrive(bar);
        }
        // (a box before the first row arrives as zeros)
        if (lane < kRows && lane % maps.box == 0)
            pair_box4(to, map, p, slot >= 0 ? base + (int)(slot >> 3) : -2, cluster_addr(bar, 0));
        __syncwarp();
    }
    // The same planes, those below `end` of them, a row at a time: to be arrived for when they have landed (an arrival of
    // every thread for its own, 256 a chunk, bound the kernel).
    __device__ __forceinline__ void copy_planes(bool in_rows, int p, int n, int end, uint32_t dst)
    {
        const int v = lane % 8;
#pragma unroll
        for (int k = 0; k < kRows / 4; ++k) {
            const int r = lane / 8 + 4 * k;
            const long long at = __shfl_sync(0xffffffffu, slot, r), from = max(at, 0ll);
            const uint4* row = (in_rows ? a.kv + lat_off(a.g, a.layer, from) : a.kv + band_off(a.g, a.layer, from)) + v;
            for (int c = p; c < min(p + n, end); ++c)
                cp_async16(place(dst + (c - p) * kAtomBytes, n * kAtomBytes, r, v), row + 8 * c, at >= 0);
        }
    }
    __device__ __forceinline__ bool copied() const { return maps.box == 0; }
};

// A query tile: tokens [tok, tok + toks) of a chunk, heads [head0, head0 + heads) of a band; column c is token c / heads.
struct Unit {
    ChunkDev ch;
    int band, tok, toks, head0, heads, cols;
};

// 16 bytes of query row `column` (of which this thread has the 16 bytes v of each chunk) of chunks [c0, c1) of a unit to row
// `row`, of the first of them at `dst` and of the next ones `pitch` bytes on; zeros behind its last one.
__device__ __forceinline__ void copy_query_row(const WeighArgs& a, const Shape& s, const Unit& u, int column, int row, int v, int c0,
                                               int c1, uint32_t dst, uint32_t pitch)
{
    const bool on = column < u.cols;
    const int col = on ? column : 0, tok = u.cols > 0 ? col / u.heads : 0;
    const long long t = u.cols > 0 ? u.ch.tok0 + u.tok + tok : 0, head = u.cols > 0 ? u.band * s.group + u.head0 + (col - tok * u.heads) : 0;
    const uint4* latent = static_cast<const uint4*>(a.q_latent.ptr) + (t * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8 + v;
    const uint4* band = static_cast<const uint4*>(a.q_rope.ptr) + (t * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8 + v;
    const uint32_t to = dst + row * 128 + ((v ^ (row & 7)) << 4);
    for (int c = c0; c < c1; ++c)
        cp_async16(to + (c - c0) * pitch, c < s.latent ? latent + 8 * c : band + 8 * (c - s.latent), on);
}

// ----------------------------------------------------------------- products --
// 64 columns of S^T, rows of 128 bytes in both operands; the keys' groups of 8 rows lie `pitch` bytes apart.
__device__ __forceinline__ void product(uint32_t d, uint32_t keys, int pitch, uint32_t queries, uint32_t desc, bool more)
{
    const uint64_t k = smem_matrix(keys, 16, pitch), q = smem_matrix(queries, 16, 1024);
#pragma unroll
    for (int e = 0; e < 4; ++e) pair_mma_bf16(d, k + (uint64_t)(2 * e), q + (uint64_t)(2 * e), desc, more || e > 0);
}

// ----------------------------------------------------------------- epilogue --
// Lazy pools: theta_j of a band's pairs as a part of a whole turn, to shared memory, by all threads.
__device__ __forceinline__ void load_turns(const WeighArgs& a, int pairs, double* turns)
{
    for (int j = threadIdx.x; j < pairs; j += blockDim.x) turns[j] = a.turn[j] * 0.15915494309189533577;  // 1 / (2 pi)
}

// Whether x holds in one of kWarps warps, which meet here (barrier 1).
template <int kWarps>
__device__ __forceinline__ bool any_of_warps(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %1, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "n"(32 * kWarps), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// What a column of a unit is given: its lse, and the rows that it attends to, those below `limit` (none without an lse).
struct Column {
    float lse = INFINITY;
    int limit = 0;

    __device__ __forceinline__ float neg() const { return -lse * kLog2e; }
    __device__ __forceinline__ int rows() const { return lse == -INFINITY ? 0 : limit; }
};

__device__ __forceinline__ Column column_of(const WeighArgs& a, const Shape& s, const Unit& u, int c)
{
    Column x;
    if (c >= u.cols) return x;
    const int tok = c / u.heads;
    x.lse = a.lse[(long long)(u.ch.tok0 + u.tok + tok) * a.q_heads + u.band * s.group + u.head0 + (c - tok * u.heads)];
    x.limit = (int)(a.prefix ? u.ch.start : u.ch.start + u.tok + tok + 1);
    return x;
}

// sum over `n` columns (a multiple of 16) of exp2(x * scale2 + neg), of this thread's TMEM lane from `tmem` on; where
// `masked`, of those alone whose limit lies above `key`, and of the columns below `cols` in any case (what lies behind
// them may be anything).  x is the sum of kParts accumulators, `pitch` TMEM columns apart.
template <int kParts = 1>
__device__ __forceinline__ float sum_columns(uint32_t tmem, int n, int cols, float scale2, const float* neg, const int* limit,
                                             int key, bool masked, int pitch = 0)
{
    constexpr int kBlocks = kParts > 1 ? 1 : 2;  // of 16 columns at a time
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int c1 = 0; c1 < n; c1 += 16 * kBlocks) {
        uint32_t v[2][16];
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (kParts > 1 || c1 + 16 * b < n) tmem_ld16(tmem + c1 + (kParts > 1 ? b * pitch : 16 * b), v[b]);
        tmem_wait_ld();
        auto add_to = [](uint32_t* x, const uint32_t* y) {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) + __uint_as_float(y[k]));
        };
        if (kParts > 1) add_to(v[0], v[1]);
        if (kParts > 2) {
            uint32_t w[2][16];
            tmem_ld16(tmem + c1 + 2 * pitch, w[0]);
            if (kParts > 3) tmem_ld16(tmem + c1 + 3 * pitch, w[1]);
            tmem_wait_ld();
            if (kParts > 3) add_to(w[0], w[1]);
            add_to(v[0], w[0]);
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int c0 = c1 + 16 * b;
            if (c0 >= n) break;
            const bool some = masked || c0 + 16 > cols;
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const float4 l = *reinterpret_cast<const float4*>(neg + c0 + k);
                float2 e0 = fma2(make_float2(__uint_as_float(v[b][k]), __uint_as_float(v[b][k + 1])),
                                 make_float2(scale2, scale2), make_float2(l.x, l.y));
                float2 e1 = fma2(make_float2(__uint_as_float(v[b][k + 2]), __uint_as_float(v[b][k + 3])),
                                 make_float2(scale2, scale2), make_float2(l.z, l.w));
                e0 = make_float2(exp2_approx(e0.x), exp2_approx(e0.y));
                e1 = make_float2(exp2_approx(e1.x), exp2_approx(e1.y));
                if (some) {
                    const int4 end = *reinterpret_cast<const int4*>(limit + c0 + k);
                    if (key >= end.x) e0.x = 0.f;
                    if (key >= end.y) e0.y = 0.f;
                    if (key >= end.z) e1.x = 0.f;
                    if (key >= end.w) e1.y = 0.f;
                }
                acc[0] = add2(acc[0], e0);
                acc[1] = add2(acc[1], e1);
            }
        }
    }
    return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
}

// Launch pairs of CTAs with programmatic stream serialization.
template <typename... KArgs, typename... Args>
cudaError_t launch_pairs(void (*kernel)(KArgs...), int pairs, int threads, size_t smem, cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace leyline
