// Internal interface between the host API of the recurrent-state operators
// (gdn_recurrent_host.cpp) and their HIP kernels. Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "gdn_recurrent.h"

namespace gdn {

// Memory that a call walks through is read and written around the caches
// where it exceeds the last-level cache, which it would only flush.
constexpr int64_t LAST_LEVEL_BYTES = int64_t(256) << 20;

// Rows of q, k or v: token / head distances in elements, and how many of the
// H heads share one.
struct RowsOf {
    const void* p;
    int64_t ts, hs;
    int32_t share;
};

// ---- linear attention over prompts
constexpr int LA_MAX_JOBS = 3;

// Where the sequences lie, and the segments they are cut into.
struct LaUnits {
    int32_t H, n_units, dense;
    int32_t T;                // dense: tokens of a row
    int64_t total;
    const int32_t* offsets;   // packed: device [n_units + 1]
    int32_t seg_tokens;       // a multiple of 64
    int32_t n_segs;           // over all units
    int32_t join;             // the walk adds the slots up itself, no merge
    int32_t n_pages;
    const float* decay;       // [H]
};

// One pass of o_i = sum_{j <= i} d^{i-j} s_p (q_i . k_j) v_j + s_o d^{i+e} q_i S
// (positions from 0, in reversed time with rev) over every unit, with the
// state after it, S' = d^L S + sum_j s_w d^{L-e-j} k_j v_j^T. Here q and k are
// K wide and v is V wide whatever tensors they are: the gradients are passes
// of the same form with the tensors in other places.
struct LaJob {
    RowsOf q, k, v;
    const float* s_in;         // entry states (NULL: zero), by unit or by in_pages
    const int32_t* in_pages;
    float* s_out;              // states after the units, by unit or by out_pages; or NULL
    const int32_t* out_pages;
    float* slots;              // [n_segs][H]: the states entering the segments, or NULL
    int32_t K;                 // width of its q and k
    int32_t transposed;        // s_in and slots are read as V x K
    int32_t rev, e, o_f32;
    void* o;                   // [tokens][H][V]
    float s_p, s_w, s_o;
};
struct LaJobs {
    LaJob job[LA_MAX_JOBS];
    int32_t n;
};

// the segments' own contributions, into the slots after theirs (k, v, s_w, e, rev)
hipError_t launch_la_summary(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s);
// the slots' running states, from s_in
hipError_t launch_la_merge(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s);
// K, V: of every job, or of some where the others have them exchanged
hipError_t launch_la_main(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s);
// out [tokens][h][D] = sums of the H / h heads of x [tokens][H][D] that share one
hipError_t launch_la_group(const float* x, void* out, int64_t tokens, int H, int h, int D, int dtype, hipStream_t s);

// ---- single tokens
struct StepArgs {
    int32_t N, H, n_pages, dtype, o_dtype;
    float scale;
    RowsOf q, k, v;
    const float* decay;     // linear attention: [H]
    const float* g;         // gated delta rule: [N][H] or [N][H][K]
    const void* beta;       // [N][H]
    const int32_t* pages;   // NULL: page n
    float* state;
    void* o;
    int32_t kind;           // 0 linear attention, 1 scalar gate, 2 per-key gate
    int32_t use_exp2, qk_norm, beta_sig;
};
hipError_t launch_step(const StepArgs& a, int K, int V, hipStream_t s);

// ---- pages
constexpr int FORK_MAX = 8192;          // slots, and spare pages, of one fork
constexpr int COMPACT_MAX = 1 << 17;    // pages of one compaction

struct PoolArgs {
    char* dst;
    const char* src;
    int32_t n_layers, dst_pages, src_pages;
    int64_t page_bytes;
};
hipError_t launch_pages_copy(const PoolArgs& pool, const int32_t* dst_pages, const int32_t* src_pages, int n,
                             hipStream_t s);
// ws: where many slots or pages make a plan of its own, the count of copies,
// then sources and destinations of n each
hipError_t launch_fork(const PoolArgs& pool, const int32_t* table, const int32_t* parent, int n, const int32_t* spare,
                       int m, int32_t* new_table, int32_t* left, int32_t* ws, hipStream_t s);
hipError_t launch_compact(const PoolArgs& pool, const int32_t* table, int n, int32_t* new_table, int32_t* count,
                          int32_t* ws, hipStream_t s);

}  // namespace gdn
