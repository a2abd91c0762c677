// leyline_weigh_tile.cu -- the weight that a batch's queries give to each cache row, on the tensor cores of sm_103a: MLA
// rows and the grouped rows that attention takes in tiles.
//
//   S^T = K Q^T  [128 cache rows x up to 128 query rows],  w_s += sum over columns of exp2(S^T * scale * log2 e - lse * log2 e)
//
// A cache row is a TMEM lane, so a thread of the epilogue has a row of S^T and sums its columns in registers: no
// reduction across threads, and a masked or bad row spoils no other.  lse is given, so tiles need no common maximum.
//
// Both operands lie in shared memory as chunks of 64 columns, 128 bytes a row, swizzled.  One of them stays while the other
// passes through a ring of chunks, whichever the plan says (BatchHeader::weigh_mode):
//   queries stay  every request's query rows of a band fit one tile (decoding): the cache is read once, as it comes from
//                 HBM, in equal shares of 16 rows a CTA;
//   keys stay     more query rows: an item is a tile of 128 cache rows and a segment of the request's query tiles, whose
//                 queries pass; where a request's query tiles are cut into segments a second kernel adds their sums up.
//
// Roles: warps 0-3 epilogue, warp 4 issues the products, warps 5-12 load, 16 rows of a key chunk each (TMA boxes of 16 or
// 8 rows where 8 divides the block size, else a row at a time).  In a lazy pool they turn each row's band by its pending
// count, in fp32, into the sum of two bf16 values, as leyline_attention_tile.cu does: the scores carry it to 2^-17.
#include "leyline_attention.cuh"

namespace leyline {
namespace {

constexpr int kMmaWarp = 4, kLoadWarp = 5, kLoadWarps = 8;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kLoaders = 32 * kLoadWarps;

constexpr int kChunkBytes = kWeighKeys * 128;
constexpr int kMaxStages = 12;
constexpr int kMaxChunks = 10;  // of a key: 8 of the latent, the band and its low part
constexpr uint32_t kTmemCols = 256;  // two buffers of S^T

struct Misc {
    unsigned long long full[kMaxStages], empty[kMaxStages];
    unsigned long long stay_full[kMaxChunks], stay_empty;
    unsigned long long s_full[2], s_empty[2];
    unsigned long long drained;
    uint32_t tmem;
    int quit;
    alignas(16) float neg_lse[2][kWeighCols];  // of the columns, times log2 e
    int limit[2][kWeighCols];                  // rows below it are attended to
};
static_assert(kWeighSmem + sizeof(Misc) + kLoadWarps * 128 * sizeof(float2) + 1024 <= 232448, "shared memory of a CTA");

// What the roles agree on.
struct Shape {
    int mode, bands, group;
    int tokens, heads, blocks;     // query tile: tokens, heads of a token; tiles of a token's heads
    int latent, keys, low;         // chunks of a key: of the latent, of the band, of the band's low part
    int q_chunks, chunks;
    int q_rows;                    // rows of a query chunk that stays
    int stay_bytes, stages;
};

__device__ __forceinline__ Shape make_shape(const WeighArgs& a, bool lazy)
{
    Shape s;
    const bool mla = a.g.rope_heads <= 1;
    s.mode = a.header->weigh_mode;
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
    s.q_rows = a.header->weigh_cols;
    s.stay_bytes = s.mode == kQueriesStay ? s.bands * s.q_chunks * s.q_rows * 128 : s.chunks * kChunkBytes;
    s.stages = min(kMaxStages, (kWeighSmem - s.stay_bytes) / kChunkBytes);
    return s;
}

struct Tile {
    int key0, keys;  // cache rows
};

// A query tile: tokens [tok, tok + toks) of a chunk, heads [head0, head0 + heads) of a band; column c is token c / heads.
struct Unit {
    ChunkDev ch;
    int band, tok, toks, head0, heads, cols;
};

__device__ __forceinline__ int padded(int cols) { return (cols + 15) & ~15; }

// Every role walks the CTA's work in the same order:
//   queries(r, u)     the query tile u of every band is to stay; keys(r, t, band): the keys of a tile are
//   unit(r, t, u)     a product
//   flush(r, t, part) the tile's sums are complete (part < 0), or those of a segment are
//   release()         what stays is no longer used
template <class Role>
__device__ __forceinline__ void walk(const WeighArgs& a, const Shape& s, Role& role)
{
    const int n = a.header->weigh_reqs;
    const long long work = a.header->weigh_work;
    auto find = [&](long long x) {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.reqs[mid].begin <= x) lo = mid;
            else hi = mid - 1;
        }
        return a.reqs[lo];
    };
    // (a replayed plan's table may have more requests or rows than the weights)
    auto holds = [&](const WeighReq& r) { return r.req < a.num_reqs && r.end <= a.rows; };
    if (s.mode == kQueriesStay) {
        const long long g1 = work * (blockIdx.x + 1) / gridDim.x;
        for (long long g = work * blockIdx.x / gridDim.x; g < g1;) {
            const WeighReq r = find(g);
            const long long g_end = min(g1, (long long)(r.begin + (r.end + 15) / 16));
            if (!holds(r)) {
                role.refuse();
                g = g_end;
                continue;
            }
            const ChunkDev ch = a.chunks[r.chunk];
            Unit u{ch, 0, 0, ch.n, 0, s.group, ch.n * s.group};
            role.queries(r, u);
            const int end = (int)min((g_end - (long long)r.begin) * 16, (long long)r.end);
            for (int key0 = (int)(g - r.begin) * 16; key0 < end; key0 += kWeighKeys) {
                const Tile t{key0, min(kWeighKeys, end - key0)};
                for (u.band = 0; u.band < s.bands; ++u.band) role.unit(r, t, u);
                role.flush(r, t, -1);
            }
            role.release();
            g = g_end;
        }
        return;
    }
    for (long long i = blockIdx.x; i < work; i += gridDim.x) {
        const WeighReq r = find(i);
        if (!holds(r)) {
            role.refuse();
            continue;
        }
        const int local = (int)(i - r.begin), tile = local / r.segs;
        const Tile t{tile * kWeighKeys, (int)min((long long)kWeighKeys, (long long)r.end - (long long)tile * kWeighKeys)};
        const int u0 = (local - tile * r.segs) * a.header->weigh_seg, u1 = min(u0 + a.header->weigh_seg, r.units);
        const int per_band = r.units / s.bands;
        for (int band = u0 / per_band; band * per_band < u1; ++band) {
            const int lo = max(u0 - band * per_band, 0), hi = min(u1 - band * per_band, per_band);
            bool loaded = false;
            int at = 0;  // units of the chunks before
            for (int c = r.chunk; c >= 0 && at < hi;) {
                const ChunkDev ch = a.chunks[c];
                const int units = (ch.n + s.tokens - 1) / s.tokens * s.blocks;
                // query tiles whose last token lies before the cache rows attend to none of them
                const int skip = a.prefix ? (t.key0 < ch.start ? 0 : units)
                                          : (int)min((long long)units, max(0ll, (t.key0 - (long long)ch.start) / s.tokens * s.blocks));
                for (int x = max(lo - at, skip); x < min(hi - at, units); ++x) {
                    const int tok = x / s.blocks * s.tokens, toks = min(s.tokens, ch.n - tok);
                    const int head0 = x % s.blocks * kWeighCols, heads = min(s.heads, s.group - head0);
                    if (!loaded) role.keys(r, t, band);
                    loaded = true;
                    role.unit(r, t, Unit{ch, band, tok, toks, head0, heads, toks * heads});
                }
                at += units;
                c = ch.next;
            }
            if (loaded) role.release();
        }
        role.flush(r, t, r.segs > 1 ? r.part + local : -1);
    }
}

// --------------------------------------------------------------------- loads --
// kKeys: chunks of a band that are turned, 0 where none are.
template <int kKeys>
struct Loader {
    static constexpr bool kLazy = kKeys > 0;
    static constexpr int kTurned = kLazy ? kKeys : 1;
    const WeighArgs& a;
    const WeighMaps& maps;
    const QueryMaps& queries_map;
    const Shape& s;
    Misc* m;
    uint32_t smem;
    float2* cs;  // lazy pools: cos, sin of `count`, this warp's
    int warp, lane, tid;
    bool ok = true;
    Ring ring;
    uint32_t stay_phase = 0;
    // rows 16 warp + lane (lanes below 16) of the tile of keys at `slot_key` of request `slot_req`: -1 where there is none
    long long slot = -1;
    int slot_key = -1, slot_req = -1;
    int landing = 0;  // chunks of copied rows that have been asked for and not been arrived for
    int count = 0;
    bool counted = false;
    uint4 x[4][kTurned];  // bands of rows lane / 8 + 4 k
    int pend[4];

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity)
    {
        if (ok) ok = warp_wait(bar, parity, &m->quit, a.status);
        return ok;
    }

    __device__ __forceinline__ void look_up(const WeighReq& r, const Tile& t)
    {
        if (slot_key == t.key0 && slot_req == r.req) return;
        slot_key = t.key0;
        slot_req = r.req;
        slot = -1;
        const int row = 16 * warp + lane;
        if (lane >= 16 || row >= t.keys) return;
        const unsigned u = (unsigned)(t.key0 + row), B = (unsigned)a.g.block_size;
        const unsigned blk = maps.shift >= 0 ? u >> maps.shift : u / B;
        const int page = a.header->table[(long long)r.req * a.header->max_blocks + blk];
        if (page >= 0 && page < a.g.num_pages) slot = (long long)page * B + (u - blk * B);
        else raise_status(a.status, ST_BAD_PAGE);
    }

    // The bands to turn, in registers.
    __device__ __forceinline__ void read_bands(int band)
    {
        if constexpr (kLazy) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const long long at = __shfl_sync(0xffffffffu, slot, lane / 8 + 4 * k);
                const uint4* from = a.kv + band_off(a.g, a.layer, max(at, 0ll)) + band * a.g.head_vecs + lane % 8;
                pend[k] = at >= 0 ? a.pending[at] : 0;
#pragma unroll
                for (int c = 0; c < kTurned; ++c) x[k][c] = at >= 0 ? ld_stream(from + 8 * c) : make_uint4(0, 0, 0, 0);
            }
        }
    }

    __device__ __forceinline__ void ensure(int c)
    {
        if (counted && c == count) return;
        const bool bf16 = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        __syncwarp();
        for (int j = lane; j < 32 * kTurned; j += 32) {
            float co, si;
            pending_trig(c, a.turn, 32 * kTurned, j, bf16, co, si);
            cs[j] = make_float2(co, si);
        }
        __syncwarp();
        count = c;
        counted = true;
    }

    // Chunk c of the turned bands, or what its rounding to bf16 leaves of it, to the chunk at `dst`.
    __device__ __forceinline__ void store_turned(int c, bool low, uint32_t dst)
    {
        const bool naive = a.g.precision == LEYLINE_ROTATE_BF16_NAIVE;
        const bool split = a.g.pair_layout == LEYLINE_PAIRS_HALF_SPLIT;
        const int v = lane % 8, half = kTurned / 2;
        const bool first = kTurned == 1 ? v < 4 : c < half;
        uint4 mine[4], other[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mine[k] = x[k][0];
#pragma unroll
            for (int d = 1; d < kTurned; ++d)
                if (d == c) mine[k] = x[k][d];
            if (kTurned == 1) {
                other[k] = shfl_xor_vec(mine[k], 4);
            } else {
                other[k] = x[k][0];
#pragma unroll
                for (int d = 1; d < kTurned; ++d)
                    if (d == (first ? c + half : c - half)) other[k] = x[k][d];
            }
        }
        // mostly all rows of a warp share a count; else a pass for each
        unsigned left = 15;
        for (;;) {
            const unsigned lanes = __ballot_sync(0xffffffffu, left != 0);
            if (lanes == 0) return;
            int next = pend[3];
#pragma unroll
            for (int k = 2; k >= 0; --k)
                if (left >> k & 1) next = pend[k];
            const int c0 = __shfl_sync(0xffffffffu, next, __ffs(lanes) - 1);
            if (c0 != 0) ensure(c0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t* mw = reinterpret_cast<const uint32_t*>(&mine[k]);
                const uint32_t* ow = reinterpret_cast<const uint32_t*>(&other[k]);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float q0 = bf16_lo(mw[e]), q1 = bf16_hi(mw[e]);
                    if (c0 != 0) {
                        const float x0 = q0, x1 = q1;
                        if (split) {  // x' = x c - y s of the first half, y' = y c + x s of the second
                            const int pair = kTurned == 1 ? 8 * (v & 3) : 64 * (first ? c : c - half) + 8 * v;
                            const float2 t0 = cs[pair + 2 * e], t1 = cs[pair + 2 * e + 1];
                            const float y0 = bf16_lo(ow[e]) * (first ? -t0.y : t0.y), y1 = bf16_hi(ow[e]) * (first ? -t1.y : t1.y);
                            q0 = naive ? round_bf16(x0 * t0.x) + round_bf16(y0) : fmaf(x0, t0.x, y0);
                            q1 = naive ? round_bf16(x1 * t1.x) + round_bf16(y1) : fmaf(x1, t1.x, y1);
                        } else {
                            const float2 t = cs[32 * c + 4 * v + e];
                            if (naive) turn_bf16(x0, x1, t.x, t.y, q0, q1);
                            else turn_fp32(x0, x1, t.x, t.y, q0, q1);
                        }
                    }
                    w[e] = pack_bf16x2(q0, q1);
                    // the naive arm's result is the rounded one
                    if (low) w[e] = naive ? 0u : pack_bf16x2(q0 - bf16_lo(w[e]), q1 - bf16_hi(w[e]));
                }
                const int row = 16 * warp + lane / 8 + 4 * k;
                if (pend[k] == c0)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + row * 128 + ((v ^ (row & 7)) << 4)),
                                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                if (pend[k] == c0) left &= ~(1u << k);
            }
        }
    }

    // This warp's 16 rows of chunk c of the tile's keys to the chunk at `dst`; 32 arrivals on `bar`.
    __device__ __forceinline__ void key_chunk(int band, int c, uint32_t dst, uint32_t bar)
    {
        if (kLazy && c >= s.latent) {
            const int b = c - s.latent;
            store_turned(b < s.keys ? b : b - s.keys, b >= s.keys, dst);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_n(bar, 32);
            return;
        }
        const bool in_rows = c < s.latent || maps.whole;
        if (maps.box > 0) {
            const long long y0 = slot, y1 = __shfl_sync(0xffffffffu, slot, 8);
            if (lane == 0) {
                const CUtensorMap* map = in_rows ? &maps.rows : &maps.bands;
                const int plane = in_rows ? c : band * s.keys + (c - s.latent);
                const int base = (int)((long long)a.layer * a.g.num_pages * a.g.block_size / 8);
                const uint32_t to = dst + warp * 2048;
                const bool wide = maps.box == 16;
                const uint32_t bytes = (y0 >= 0 ? (wide ? 2048 : 1024) : 0) + (!wide && y1 >= 0 ? 1024 : 0);
                if (bytes > 0) mbar_expect_tx(bar, bytes);
                else mbar_arrive(bar);
                if (y0 >= 0) tma_box4(to, map, plane, base + (int)(y0 >> 3), bar);
                if (!wide && y1 >= 0) tma_box4(to + 1024, map, plane, base + (int)(y1 >> 3), bar);
                mbar_arrive_n(bar, 31);
            }
            __syncwarp();
            return;
        }
        const int v = lane % 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = lane / 8 + 4 * k, row = 16 * warp + r;
            const long long at = __shfl_sync(0xffffffffu, slot, r), from = max(at, 0ll);
            const uint4* p = c < s.latent ? a.kv + lat_off(a.g, a.layer, from) + 8 * c + v
                                          : a.kv + band_off(a.g, a.layer, from) + band * a.g.head_vecs + 8 * (c - s.latent) + v;
            cp_async16(dst + row * 128 + ((v ^ (row & 7)) << 4), p, at >= 0);
        }
        cp_async_commit();
    }
    // Whether key_chunk() leaves chunk c to be arrived for: an arrival of every lane when its copies land took
    // 256 arrivals a chunk, and bound the kernel.
    __device__ __forceinline__ bool copied(int c) const { return maps.box == 0 && !(kLazy && c >= s.latent); }

    // Arrive for chunks that have landed: all but the last `kLeft` asked for, of which the next one goes to stage ring.stage.
    template <int kLeft>
    __device__ __forceinline__ void arrive_landed()
    {
        if (landing <= kLeft) return;
        cp_async_wait<kLeft>();
        __syncwarp();
        for (; landing > kLeft; --landing) {
            const int stage = ring.stage >= landing ? ring.stage - landing : ring.stage - landing + s.stages;
            if (lane == 0) mbar_arrive_n(smem_addr(&m->full[stage]), 32);
        }
    }

    // Query rows tid / 8 + 32 k of a unit, below `rows`: 16 bytes of chunk c each.
    struct QueryRows {
        const uint4 *latent[4], *band[4];
        bool on[4];
    };
    __device__ __forceinline__ QueryRows query_rows(const Unit& u)
    {
        QueryRows q;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int col = tid / 8 + 32 * k;
            q.on[k] = col < u.cols;
            const int c = q.on[k] ? col : 0, tok = c / u.heads;
            const long long t = u.ch.tok0 + u.tok + tok, head = u.band * s.group + u.head0 + (c - tok * u.heads);
            q.latent[k] = static_cast<const uint4*>(a.q_latent.ptr) + (t * a.q_latent.token_stride + head * a.q_latent.head_stride) / 8 + tid % 8;
            q.band[k] = static_cast<const uint4*>(a.q_rope.ptr) + (t * a.q_rope.token_stride + head * a.q_rope.head_stride) / 8 + tid % 8;
        }
        return q;
    }
    __device__ __forceinline__ void query_chunk(const QueryRows& q, int rows, int c, uint32_t dst)
    {
        const int v = tid % 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = tid / 8 + 32 * k;
            if (row < rows)
                cp_async16(dst + row * 128 + ((v ^ (row & 7)) << 4),
                           c < s.latent ? q.latent[k] + 8 * c : q.band[k] + 8 * (c - s.latent), q.on[k]);
        }
    }

    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void release()
    {
        if (ok) arrive_landed<0>();
    }

    __device__ __forceinline__ void queries(const WeighReq&, Unit u)
    {
        if (!wait(smem_addr(&m->stay_empty), stay_phase ^ 1)) return;
        stay_phase ^= 1;
        for (u.band = 0; u.band < s.bands; ++u.band) {
            const QueryRows q = query_rows(u);
            for (int c = 0; c < s.q_chunks; ++c)
                query_chunk(q, s.q_rows, c, smem + (u.band * s.q_chunks + c) * s.q_rows * 128);
        }
        cp_async_arrive(smem_addr(&m->stay_full[0]));
    }

    __device__ __forceinline__ void keys(const WeighReq& r, const Tile& t, int band)
    {
        if (!wait(smem_addr(&m->stay_empty), stay_phase ^ 1)) return;
        stay_phase ^= 1;
        look_up(r, t);
        read_bands(band);
        for (int c = 0; c < s.chunks; ++c) key_chunk(band, c, smem + c * kChunkBytes, smem_addr(&m->stay_full[c]));
        if (maps.box > 0) return;
        cp_async_wait<0>();
        __syncwarp();
        for (int c = lane; c < s.chunks; c += 32)
            if (copied(c)) mbar_arrive_n(smem_addr(&m->stay_full[c]), 32);
    }

    __device__ __forceinline__ void unit(const WeighReq& r, const Tile& t, const Unit& u)
    {
        if (!ok) return;
        if (s.mode == kQueriesStay) {
            look_up(r, t);
            read_bands(u.band);
            for (int c = 0; c < s.chunks; ++c) {
                // (a stage is not waited for while more chunks are still to be arrived for than leave one free)
                if (copied(c)) arrive_landed<kWeighStages - 2>();
                else arrive_landed<0>();
                if (!wait(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1)) return;
                key_chunk(u.band, c, smem + s.stay_bytes + ring.stage * kChunkBytes, smem_addr(&m->full[ring.stage]));
                if (copied(c)) ++landing;
                ring.advance(s.stages);
            }
            return;
        }
        if (queries_map.usable) {  // a box of a chunk is as many instructions' work as its rows'
            const uint32_t bytes = s.heads * s.tokens * 128;
            for (int c = 0; c < s.q_chunks; ++c) {
                // Every warp waits for every stage and arrives for it, whichever asks for the box: one that left some out could
                // run a lap ahead or fall one behind, where the parity that it waits for means another lap.
                if (!wait(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1)) return;
                if (lane == 0) {
                    const uint32_t full = smem_addr(&m->full[ring.stage]);
                    if (c % kLoadWarps == warp) {
                        mbar_expect_tx(full, bytes);
                        const bool latent = c < s.latent;
                        tma_box3(smem + s.stay_bytes + ring.stage * kChunkBytes, latent ? &queries_map.latent : &queries_map.band,
                                 64 * (latent ? c : c - s.latent), u.band * s.group + u.head0, u.ch.tok0 + u.tok, full);
                        mbar_arrive_n(full, 31);
                    } else {
                        mbar_arrive_n(full, 32);
                    }
                }
                __syncwarp();
                ring.advance(s.stages);
            }
            return;
        }
        const QueryRows q = query_rows(u);
        const int rows = padded(u.cols);
        for (int c = 0; c < s.q_chunks; ++c) {
            if (!wait(smem_addr(&m->empty[ring.stage]), ring.phase ^ 1)) return;
            query_chunk(q, rows, c, smem + s.stay_bytes + ring.stage * kChunkBytes);
            cp_async_arrive(smem_addr(&m->full[ring.stage]));
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
        if (ok) ok = warp_wait(bar, parity, &m->quit, a.status);
        return ok;
    }
    __device__ __forceinline__ void refuse() {}
    __device__ __forceinline__ void flush(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void queries(const WeighReq&, const Unit&)
    {
        if (!wait(smem_addr(&m->stay_full[0]), stay_phase)) return;
        stay_ready = true;
    }
    __device__ __forceinline__ void keys(const WeighReq&, const Tile&, int) { stay_ready = false; }
    __device__ __forceinline__ void release()
    {
        if (ok && elect_lane()) mma_commit(smem_addr(&m->stay_empty));
        __syncwarp();
        stay_phase ^= 1;
    }
    // 64 columns of a product.
    __device__ __forceinline__ void product(uint32_t d, uint32_t keys, uint32_t queries, uint32_t desc, bool more)
    {
        const uint64_t k = smem_matrix(keys, 16, 1024), q = smem_matrix(queries, 16, 1024);
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_bf16(d, k + (uint64_t)(2 * e), q + (uint64_t)(2 * e), desc, more || e > 0);
    }
    __device__ __forceinline__ void unit(const WeighReq&, const Tile&, const Unit& u)
    {
        const int buf = index & 1;
        if (!wait(smem_addr(&m->s_empty[buf]), ((index >> 1) & 1) ^ 1)) return;
        ++index;
        const uint32_t d = tmem + buf * kWeighCols, desc = mma_desc(kWeighKeys, padded(u.cols), false, false);
        const bool queries_stay = s.mode == kQueriesStay;
        const int steps = queries_stay ? s.chunks : s.q_chunks;
        for (int c = 0; c < steps; ++c) {
            if (!queries_stay && !stay_ready) {
                if (!wait(smem_addr(&m->stay_full[c]), stay_phase)) return;
                if (s.low > 0 && c >= s.latent && !wait(smem_addr(&m->stay_full[c + s.low]), stay_phase)) return;
            }
            if (!wait(smem_addr(&m->full[ring.stage]), ring.phase)) return;
            fence_async_smem();
            tcgen05_after_sync();
            if (elect_lane()) {
                const uint32_t at = smem + s.stay_bytes + ring.stage * kChunkBytes;
                if (queries_stay) {
                    const int qc = c < s.q_chunks ? c : c - s.low;  // a band's low part meets the same queries
                    product(d, at, smem + (u.band * s.q_chunks + qc) * s.q_rows * 128, desc, c > 0);
                } else {
                    product(d, smem + c * kChunkBytes, at, desc, c > 0);
                    if (s.low > 0 && c >= s.latent) product(d, smem + (c + s.low) * kChunkBytes, at, desc, true);
                }
                mma_commit(smem_addr(&m->empty[ring.stage]));
                if (c + 1 == steps) mma_commit(smem_addr(&m->s_full[buf]));
            }
            __syncwarp();
            ring.advance(s.stages);
        }
        stay_ready = true;
    }
};

// ------------------------------------------------------------------ epilogue --
// The warps meet at a named barrier, so when the CTA gives up they go through their units without waiting, and write
// nothing; the status word says that the weights are not valid.
struct Summer {
    const WeighArgs& a;
    const Shape& s;
    Misc* m;
    uint32_t tmem;
    int warp, lane;
    int index = 0;
    float sum = 0.f;

    __device__ __forceinline__ void refuse()
    {
        if (threadIdx.x == 0) raise_status(a.status, ST_BAD_ROW);
    }
    __device__ __forceinline__ void queries(const WeighReq&, const Unit&) {}
    __device__ __forceinline__ void keys(const WeighReq&, const Tile&, int) {}
    __device__ __forceinline__ void release() {}

    __device__ __forceinline__ void unit(const WeighReq&, const Tile& t, const Unit& u)
    {
        const int buf = index & 1, c = threadIdx.x, n = padded(u.cols);
        float neg = -INFINITY;
        int limit = 0;
        if (c < u.cols) {
            const int tok = c / u.heads, head = u.band * s.group + u.head0 + (c - tok * u.heads);
            const float lse = a.lse[(long long)(u.ch.tok0 + u.tok + tok) * a.q_heads + head];
            neg = -lse * kLog2e;
            if (lse != -INFINITY) limit = (int)(a.prefix ? u.ch.start : u.ch.start + u.tok + tok + 1);
        }
        m->neg_lse[buf][c] = neg;
        m->limit[buf][c] = limit;
        // (and the columns are there for all warps)
        const bool masked = any_of_softmax(c < u.cols && limit < t.key0 + t.keys);
        mbar_wait(smem_addr(&m->s_full[buf]), (index >> 1) & 1, &m->quit, a.status);
        tcgen05_after_sync();
        if (32 * warp < t.keys) {
            const uint32_t from = tmem + buf * kWeighCols + ((uint32_t)(32 * warp) << 16);
            const float scale2 = a.scale * kLog2e;
            const int key = t.key0 + 32 * warp + lane;
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            for (int c0 = 0; c0 < n; c0 += 16) {
                uint32_t v[16];
                tmem_ld16(from + c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(&m->neg_lse[buf][c0 + k]);
                    float2 e0 = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), make_float2(scale2, scale2),
                                     make_float2(l.x, l.y));
                    float2 e1 = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])),
                                     make_float2(scale2, scale2), make_float2(l.z, l.w));
                    e0 = make_float2(exp2_approx(e0.x), exp2_approx(e0.y));
                    e1 = make_float2(exp2_approx(e1.x), exp2_approx(e1.y));
                    if (masked || c0 + 16 > u.cols) {  // (columns behind the last one hold anything)
                        const int4 to = *reinterpret_cast<const int4*>(&m->limit[buf][c0 + k]);
                        if (key >= to.x) e0.x = 0.f;
                        if (key >= to.y) e0.y = 0.f;
                        if (key >= to.z) e1.x = 0.f;
                        if (key >= to.w) e1.y = 0.f;
                    }
                    acc[0] = add2(acc[0], e0);
                    acc[1] = add2(acc[1], e1);
                }
            }
            sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        }
        tcgen05_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&m->s_empty[buf]));
        ++index;
    }

    __device__ __forceinline__ void flush(const WeighReq& r, const Tile& t, int part)
    {
        const int row = 32 * warp + lane;
        const float got = sum;
        sum = 0.f;
        if (row >= t.keys || *(volatile int*)&m->quit) return;
        if (part >= 0) {
            a.part[(long long)part * kWeighKeys + row] = got;
            return;
        }
        store_weight(a, r, t.key0 + row, got);
    }

    static __device__ __forceinline__ void store_weight(const WeighArgs& a, const WeighReq& r, int key, float got)
    {
        const int page = a.header->table[(long long)r.req * a.header->max_blocks + key / a.g.block_size];
        if (page < 0 || page >= a.g.num_pages) return;  // (the loads have raised the status)
        float* w = a.weights + r.req * a.req_stride + key;
        *w = a.decay == 0.f ? got : fmaf(a.decay, *w, got);
    }
};

template <int kKeys>
__global__ void __launch_bounds__(kThreads, 1) weigh_tile_kernel(const __grid_constant__ WeighArgs a,
                                                              const __grid_constant__ WeighMaps maps,
                                                              const __grid_constant__ QueryMaps queries_map)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t smem = (smem_addr(raw) + 1023) & ~1023u;
    unsigned char* base = raw + (smem - smem_addr(raw));
    Misc* m = reinterpret_cast<Misc*>(base + kWeighSmem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&m->full[i]), kLoaders);
            mbar_init(smem_addr(&m->empty[i]), 1);
        }
        for (int i = 0; i < kMaxChunks; ++i) mbar_init(smem_addr(&m->stay_full[i]), kLoaders);
        mbar_init(smem_addr(&m->stay_empty), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&m->s_full[i]), 1);
            mbar_init(smem_addr(&m->s_empty[i]), 4);
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
    wait_for_previous_grid();
    const Shape s = make_shape(a, kKeys > 0);
    if (warp < kMmaWarp) {
        Summer role{a, s, m, tmem, warp, lane};
        walk(a, s, role);
        tcgen05_before_sync();
    } else if (warp == kMmaWarp) {
        Issuer role{a, s, m, smem, tmem};
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
        Loader<kKeys> role{a, maps, queries_map, s, m, smem, trig, w, lane, (int)threadIdx.x - 32 * kLoadWarp};
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

// Sums of requests whose query tiles were cut into segments: a CTA for a tile of cache rows, the segments in order.
__global__ void __launch_bounds__(kWeighKeys) join_weights_kernel(const __grid_constant__ WeighArgs a)
{
    wait_for_previous_grid();
    const int n = a.header->weigh_reqs;
    for (int i = blockIdx.x; i < a.header->weigh_tiles; i += gridDim.x) {
        int lo = 0, hi = n - 1;  // the last request whose split tiles begin at or before this one: it has it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.reqs[mid].tile <= i) lo = mid;
            else hi = mid - 1;
        }
        const WeighReq r = a.reqs[lo];
        const int tile = i - r.tile;
        const long long key = (long long)tile * kWeighKeys + threadIdx.x;
        if (key >= r.end || r.req >= a.num_reqs || r.end > a.rows) continue;
        const float* p = a.part + ((long long)r.part + (long long)tile * r.segs) * kWeighKeys + threadIdx.x;
        float sum = 0.f;
        for (int k = 0; k < r.segs; ++k) sum += p[k * kWeighKeys];
        Summer::store_weight(a, r, (int)key, sum);
    }
}

using Kernel = void (*)(WeighArgs, WeighMaps, QueryMaps);

Kernel kernel_of(const Geometry& g)
{
    if (!(g.flags & LEYLINE_POOL_LAZY)) return weigh_tile_kernel<0>;
    return g.rope_dim == 64 ? weigh_tile_kernel<1> : g.rope_dim == 128 ? weigh_tile_kernel<2> : weigh_tile_kernel<4>;
}

constexpr int kSmemBytes = kWeighSmem + (int)sizeof(Misc) + kLoadWarps * 128 * (int)sizeof(float2) + 1024;

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

// Map of the queries `q` of `tokens` tokens, in boxes of 64 columns, `box_heads` heads and box_tokens tokens.  False: it
// cannot be had (axes that stand still), and the queries are copied a row at a time.
static bool query_map(CUtensorMap* map, const HeadsView& q, int dim, int heads, int64_t tokens, int box_heads, int box_tokens)
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

int launch_weigh_tile(const WeighArgs& a, const WeighMaps& maps, int64_t tokens, int ctas, int joins, void* stream)
{
    QueryMaps queries{};
    if (tokens > 0) {
        const Geometry& g = a.g;
        const int group = a.q_heads / std::max(g.rope_heads, 1), heads = std::min(group, kWeighCols), toks = weigh_tokens(group);
        queries.usable = query_map(&queries.band, a.q_rope, g.rope_dim, a.q_heads, tokens, heads, toks) &&
                         (g.rope_heads > 1 || query_map(&queries.latent, a.q_latent, g.latent_dim, a.q_heads, tokens, heads, toks));
    }
    cudaError_t e = launch_dependent_smem(kernel_of(a.g), ctas, kThreads, kSmemBytes, (cudaStream_t)stream, a, maps, queries);
    if (e == cudaSuccess && joins > 0) e = launch_dependent(join_weights_kernel, joins, kWeighKeys, (cudaStream_t)stream, a);
    return (int)e;
}

}  // namespace leyline
