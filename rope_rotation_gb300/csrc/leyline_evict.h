// leyline_evict.h -- eviction of rows by their weights: what the C ABI (leyline_evict.cpp) hands to the kernels that
// choose the rows to keep (leyline_select.cu) and that drop the others (leyline_evict_rows.cu).
#pragma once

#include <cstdint>

#include "leyline_internal.h"

namespace leyline {

// Device status bit (leyline_sync_status), beside those of leyline_device.cuh: rows that a list must not name, or that the
// weights do not hold.
enum : int32_t { ST_BAD_ROW = 64 };

// Rows of a request that weighing, selecting and evicting take: their kernels count past its end in 32 bits (by 512 rows, 2^14
// and some 2000).
constexpr int64_t kMostRows = INT32_MAX - 65535;

// One request of a launch.
struct EvictReq {
    int32_t req;      // table row
    int32_t n_keep;
    int32_t first;    // select: rows always kept at either end
    int32_t last;
    int32_t len;      // rows before the call
    int32_t list;     // row of the caller's array of lists
    int32_t block_begin; // evict: kStageRows-row blocks of the launch's requests before this one
    int32_t pad;
    int64_t stage;       // evict: place of this request's kept rows in the staging arrays
    int64_t push;        // evict: ring position of the first page this request returns (mod q_cap)
};

// The requests of a launch travel as a kernel parameter.
constexpr int kEvictReqs = 32;
struct EvictSet {
    EvictReq req[kEvictReqs];
    int32_t n;
    int32_t pad;
};

struct SelectArgs {
    const float* weights;
    int64_t req_stride;
    int32_t* kept;
    int64_t kept_stride;
};

constexpr int kStageRows = 256;

// What the check of a list found, in device memory, one for each request of a launch.  Launches use two arrays of them in
// turn: a launch's commit readies the other one.
struct ListState {
    int32_t bad;   // not strictly ascending within [0, len): the first n_keep rows are kept instead
    int32_t hole;  // first i with kept[i] != i, or more than n_keep: rows before it stay where they are
};

struct EvictArgs {
    uint4* kv;
    int32_t* table;
    int32_t* seq_lens_dev;
    int32_t* free_q;
    int64_t q_cap;
    const int32_t* kept;
    int64_t kept_stride;
    float* weights;        // nullptr: none are kept
    int64_t req_stride;
    int32_t* pending;      // lazy pools, else nullptr
    ListState* state;
    ListState* next_state;
    // staged values of kept rows: weights, and pending turns or (one row a page) pages
    float* stage_w;
    int32_t* stage_i;
    int32_t* status;
    int32_t max_blocks;
    Geometry g;
};

// Each returns the cudaError_t of its launches as int.
int launch_select(const SelectArgs& a, const EvictSet& set, void* stream);
int evict_prepare();  // when a pool is created
int launch_evict(const EvictArgs& a, const EvictSet& set, void* stream);

}  // namespace leyline
