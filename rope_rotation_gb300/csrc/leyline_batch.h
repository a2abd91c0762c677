// leyline_batch.h -- batches of new tokens: what the host plan hands to the kernels that
// append rows (leyline_append.cu) and attend over them (leyline_attention.cu).
//
// A plan lives in the batch's own device memory, at addresses that never change, so that
// captured graphs of a step's layers can be replayed after each new plan.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>
#include <vector>

#include "leyline_internal.h"

namespace leyline {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kAttnRows = 64;  // query rows (token, head) of a row tile
// Lazy pools of MLA rows: 48, since a turned band takes a chunk more of shared memory.
constexpr int kAttnRowsLazy = 48;
// Pairs of CTAs (leyline_attention_pair.cu): 64 of each.
constexpr int kPairRows = 128;
constexpr int kAttnKeys = 64;  // cache rows of a key tile

// The plan's header, first in the plan's device buffer.
struct BatchHeader {
    const int32_t* table;  // block table the plan was made for
    int32_t max_blocks;
    int32_t n_tokens;
    int32_t n_joins;
    int32_t pairs;  // attention by pairs of CTAs (leyline_attention_pair.cu)
    int32_t pad[2];
};

// One chunk, as attention sees it.
struct ChunkDev {
    int32_t req;
    int32_t n;       // tokens
    int32_t tok0;    // first token of the batch
    int32_t pad;
    int64_t start;   // row of the first token
};

// One piece of attention work: a tile of up to kAttnRows query rows of one chunk and key
// band (WorkShape::rows), over the cache rows [key0, key1).  Row r is token r / group, head band * group +
// r % group of the chunk (group = query heads per key band).  part < 0: the piece is all of
// the tile's work and writes the result; else it writes partial result `part`.
struct AttnItem {
    int32_t chunk;
    int32_t band;
    int32_t row0;
    int32_t rows;
    int32_t key0;
    int32_t key1;
    int32_t part;
    int32_t pad;
};

// A row tile whose work was split into pieces part0 .. part0 + parts - 1.
struct AttnJoin {
    int32_t chunk;
    int32_t band;
    int32_t row0;
    int32_t rows;
    int32_t part0;
    int32_t parts;
    int32_t pad[2];
};

// A run of up to kPlanRun tokens of one chunk, as the plan's install kernel sees it.
constexpr int kPlanRun = 32;
struct PlanRun {
    int32_t req;
    int32_t n;
    int32_t tok0;
    int32_t old_blocks;  // blocks the request had before the plan
    int64_t start;       // row of the run's first token
    int64_t rope_start;  // its rotary position
    int64_t pop;         // ring position of the page of block old_blocks
    int64_t new_len;     // >= 0: the length to store (the request's last run), else -1
};

// Where the parts of the plan lie in the batch's device buffer (bytes).
struct BatchLayout {
    size_t chunks, cta_begin, joins, items, bytes;
};

// Validated chunks of a plan and the pages they take.
struct ChunkPlan {
    std::vector<ChunkDev> chunks;
    std::vector<PlanRun> runs;
    std::vector<std::pair<int32_t, int64_t>> new_len;  // (request, length) of extended requests
    int64_t tokens = 0;
    int64_t pages = 0;
    bool rewrites = false;  // rows that existed before are written again
};
// Validate a batch's sizes for a pool's rows.
int check_sizes(const Geometry& g, int32_t max_chunks, int32_t max_tokens, int32_t q_heads);
// Validate a plan's chunks against the table's lengths and lay out their runs; pop_base is the
// ring position of the first page the plan takes.  Returns LEYLINE_OK or an error code (the
// message is set); changes nothing but *out.
int check_chunks(const Geometry& g, const leyline_block_table_t& bt, const leyline_chunk_t* chunks, int32_t n,
                 int64_t max_tokens, int64_t free_pages, int64_t pop_base, ChunkPlan* out);

// What an item costs beside its cache tiles: its queries, the output of 64 or 128 rows and, until the first scores are
// there, an idle tensor core.  2 or 8 cache tiles (measured with 2, 4, 6 and 8: 64 drafts over grouped rows 72.5, 73, 74,
// 74 us; by pairs a prompt chunk of 512 tokens of 128 heads 747, 741, 739, 737 us, ragged chunks 165, 164, 161, 159).
constexpr int32_t kItemCost = 2;
constexpr int32_t kItemCostPairs = 8;

// What the split of the attention's work goes by.
struct WorkShape {
    int32_t bands;  // key bands attention works on (1: MLA)
    int32_t group;  // query heads per band
    int32_t ctas;
    int32_t rows;   // query rows of a tile, at most kAttnRows, by pairs kPairRows (and ctas pairs)
    int32_t item_cost = kItemCost;  // of an item's queries and output, in cache tiles
};
// Where the split is written: items[row tiles + ctas], cta_begin[ctas + 1], joins[ctas].
struct Split {
    AttnItem* items;
    int32_t* cta_begin;
    AttnJoin* joins;
    int32_t n_items = 0;
    int32_t n_joins = 0;
    int32_t n_parts = 0;
};
void split_work(const WorkShape& w, const std::vector<ChunkDev>& chunks, Split* out);
bool pairs_are_faster(const WorkShape& w, const std::vector<ChunkDev>& chunks, bool copied = false);

struct HeadsView {
    void* ptr;
    int64_t token_stride;  // in elements
    int64_t head_stride;
};

// The memory of a view: `width` bytes at address + t * token_stride + h * head_stride (bytes, not negative).
struct Extent {
    uintptr_t address;
    int64_t tokens, heads;
    int64_t token_stride, head_stride;
    int64_t width;
};
// Whether two views share a byte.  Views whose address ranges meet are told apart if they share their token stride or
// their head stride (parts of one wider tensor do) and are not of very many pieces; else they count as overlapping.
bool overlap(Extent a, Extent b);

struct InstallArgs {
    const uint4* staged;   // pinned plan, copied to plan
    uint4* plan;
    const PlanRun* runs;   // pinned
    int64_t plan_vecs;
    int32_t n_runs;
    int32_t max_blocks;
    int32_t* table;
    int32_t* seq_lens_dev;
    const int32_t* free_q;
    int64_t q_cap;
    int32_t* pending;      // lazy pools, else nullptr
    const double* theta;   // theta_j, rope_dim / 2 values
    int64_t* slot;         // [tokens]
    float2* trig;          // [tokens][rope_dim / 2]
    int32_t* status;
    Geometry g;
};

struct AppendArgs {
    uint4* kv;
    const uint4* rows;
    int64_t row_stride;    // in 16-byte vectors
    const uint4* latent_norm;
    const uint4* key_norm;
    float eps;
    int32_t layer;
    const BatchHeader* header;
    const int64_t* slot;
    const float2* trig;
    Geometry g;
};

struct RotateArgs {
    HeadsView q, out;
    const uint4* norm;
    float eps;
    int32_t q_heads;
    const BatchHeader* header;
    const float2* trig;
    Geometry g;
};

struct AttnArgs {
    const uint4* kv;
    HeadsView q_latent, q_rope, out;  // q_latent.ptr nullptr for grouped rows
    float* lse;
    float scale;
    int32_t layer;
    int32_t prefix;        // attend to the rows before the chunk only
    int32_t q_heads;
    const BatchHeader* header;
    const ChunkDev* chunks;
    const AttnItem* items;
    const int32_t* cta_begin;  // [CTAs + 1]: each CTA's items
    const AttnJoin* joins;
    float* part_out;       // [parts][kAttnRows, by pairs kPairRows][value dim]
    float* part_lse;       // [parts][the same], natural log
    int32_t* redo;         // [items][2], set where a CTA's part of a tensor-core kernel's item has to be computed again
    const int32_t* pending;
    const double* turn;    // lazy pools' turn table
    int32_t* status;
    Geometry g;
};

static_assert(sizeof(AttnItem) % 16 == 0, "plans are copied in 16-byte vectors");

// Widest rows attention takes (leyline_batch_create checks them).
constexpr int kAttnMaxValue = 1024;
constexpr int kAttnMaxRope = 256;

// Tensor maps of a pool's rows, all layers', in groups of 8 rows and planes of 64 columns, for leyline_attention_tile.cu:
// the values (whole MLA rows: with their band), and the bands.
struct TileMaps {
    CUtensorMap rows, bands;
    CUtensorMap pair_keys, pair_values;  // leyline_attention_pair.cu
    int box;     // rows of a box, 8 or 16; 0: the block size is no multiple of 8
    int shift;   // log2 of the block size; -1: no power of two
    int values;  // planes of a band's values
    int whole;   // the band comes with the values
    int stages;  // cache tiles in shared memory
};

int launch_install(const InstallArgs& a, void* stream);
int launch_append(const AppendArgs& a, int64_t tokens, int sm_count, void* stream);
int launch_rotate(const RotateArgs& a, int64_t tokens, int sm_count, void* stream);
// Whether the rows go to the tensor-core kernel (leyline_attention_tile.cu).
bool attention_takes_tiles(const Geometry& g);
int attention_tile_prepare(const Geometry& g, const void* kv, TileMaps* maps);
int launch_attention_tile(const AttnArgs& a, const TileMaps& maps, int ctas, void* stream);
// Attention by pairs of CTAs (leyline_attention_pair.cu), for MLA rows of eager pools; after
// attention_tile_prepare.
int attention_pair_prepare(const Geometry& g, const void* kv, TileMaps* maps);
int launch_attention_pair(const AttnArgs& a, const TileMaps& maps, int pairs, void* stream);
// Fills *maps for the rows at kv and readies their kernel.
int attention_prepare(const Geometry& g, const void* kv, TileMaps* maps);
// `ctas` is the number of CTAs the plan's work was split over.
int launch_attention(const AttnArgs& a, const TileMaps& maps, int ctas, void* stream);
// joins: of tiles of `rows` query rows; many_parts: some of them of more than kFewParts.
constexpr int kFewParts = 16;
int launch_join(const AttnArgs& a, int joins, int rows, bool many_parts, void* stream);

}  // namespace leyline
