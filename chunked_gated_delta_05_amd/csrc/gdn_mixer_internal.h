// Internal interface between the host API of the operators around the
// recurrent layers (gdn_mixer_host.cpp) and their HIP kernels. Not part of the
// public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "gdn_mixer.h"

namespace gdn {

// States of half the last-level cache or more are read and written around it:
// by the next token others have taken their place (states of three layers in
// turn, 128 sequences of D=8192: 67 MB 30 us through the caches, 34 around; 256
// sequences 71 and 66; 512, 135 and 124).
constexpr int64_t MX_AROUND_BYTES = int64_t(128) << 20;

// The sequences, and pieces of at most P tokens that they are cut into. The
// pieces of sequence u begin at number u * ceil(T / P) (rows), or, without a
// table, at floor(offset / P) + u (documents): the next sequence's begin no
// earlier than these end, and a few numbers stand for no piece.
struct MxUnits {
    int32_t dense, T, n_units, P;
    int32_t n_pieces;         // numbers of pieces
    int64_t total;            // tokens
    const int32_t* offsets;   // device [n_units + 1]
};

// Sums of the rows of x [rows][n] into up to three arrays that follow each
// other in a row (NULL: not wanted; lengths are multiples of 4). x has room for
// row_sums_rows(rows) more rows.
struct RowSums {
    float* p[3];
    int64_t n[3];
};
constexpr int SUM_ROWS = 64;   // of a workgroup, where there are many
constexpr int64_t row_sums_rows(int64_t rows) { return rows > 4 * SUM_ROWS ? (rows + SUM_ROWS - 1) / SUM_ROWS : 0; }
// of its largest launch
constexpr int64_t row_sums_workgroups(int64_t rows, int64_t n) {
    return (n + 63) / 64 * (row_sums_rows(rows) ? row_sums_rows(rows) : 1);
}
hipError_t launch_row_sums(float* x, int64_t rows, int64_t n, const RowSums& out, hipStream_t s);

struct ConvArgs {
    MxUnits un;
    int32_t D, W, dtype, w_f32, silu, n_pages;
    int64_t x_stride;
    const void *x, *weight, *bias;
    const void* s_in;
    const int32_t* in_pages;
    void* s_out;
    const int32_t* out_pages;
    void* y;
    // gradients
    const void *dout, *dfinal;
    void *dx, *dinitial;
    float *dweight, *dbias, *parts;   // parts [pieces][D (W + 1)]
};
constexpr int CONV_BWD_CHANNELS = 4;  // of a thread; the other kernels take 16 bytes of them
hipError_t launch_conv_fwd(const ConvArgs& a, bool states_after, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s);

constexpr int SCAN_KEEP = 16;         // tokens between the states kept for the gradients
constexpr int SCAN_TILE = 32;         // pieces are multiples of it
struct ScanArgs {
    MxUnits un;               // P: tokens of a segment
    MxUnits keep;             // the same with P = SCAN_KEEP: rows of h
    int32_t cut;              // some sequence has more than one segment
    int32_t join;             // a segment adds up those before it itself, no merge
    int32_t narrow;           // forward: a lane holds one state, nothing is cut
    int32_t D, G, S, dtype, softplus, n_pages;
    int32_t blocks, bwd_blocks;   // of channels in a group; the backward's workgroups hold half as many
    const void *u, *dt, *gate, *b, *c;
    int64_t u_stride, dt_stride, gate_stride, b_stride[2], c_stride[2];
    const float *A, *skip, *dt_bias;
    const float* s_in;
    const int32_t* in_pages;
    float* s_out;
    const int32_t* out_pages;
    float *slots, *sums;      // [pieces][D][S] states entering the segments, [pieces][D] their sums of dt'
    float* h;
    void* out;
    // gradients: here s_in is dht and s_out dh0
    const void* dout;
    void *du, *ddt, *dgate, *db, *dc;
    float *dA, *dskip, *ddt_bias;
    float *bc_parts;          // [G * bwd_blocks][tokens][2][S]
    float *a_parts;           // [pieces][D (S + 2)]
};
// Workgroups of the sums of dB and dC, and behind them those of dA, dskip and
// ddt_bias where these have few rows (else row_sums adds them up).
constexpr bool scan_sums_together(int64_t pieces) { return row_sums_rows(pieces) == 0; }
constexpr int64_t scan_bc_workgroups(int64_t tokens, int G, int S) { return (tokens * G * (S / 2) + 255) / 256; }
constexpr int64_t scan_sum_workgroups(int64_t tokens, int64_t pieces, int G, int D, int S) {
    return scan_bc_workgroups(tokens, G, S) + (scan_sums_together(pieces) ? row_sums_workgroups(pieces, int64_t(D) * (S + 2)) : 0);
}
// channels of a workgroup
constexpr int scan_channels(int S) { return S == 8 ? 128 : 2048 / S; }
constexpr int scan_narrow_channels(int S) { return S == 8 ? 32 : 16; }
hipError_t launch_scan_summary(const ScanArgs& a, bool reverse, hipStream_t s);
hipError_t launch_scan_merge(const ScanArgs& a, bool reverse, hipStream_t s);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t s);

struct RotaryArgs {
    int32_t T, Hq, Hk, D, R, dtype, w_f32, norm, interleaved, pos_i64;
    int64_t tokens;
    float eps, amplitude;
    int64_t q_stride[2], k_stride[2];
    const void *q, *k, *positions, *q_weight, *k_weight;
    const double* freqs;
    void *q_out, *k_out;
    const void *dq_out, *dk_out;
    void *dq, *dk;
    float *dq_weight, *dk_weight, *parts;   // parts [workgroups][2][D]
    int32_t workgroups;
};
// Tokens that a workgroup makes the angles of at a time: as many as leave every
// compute unit several workgroups
constexpr int ROTARY_TOKENS = 8;
constexpr int rotary_tokens(int64_t tokens) {
    int n = ROTARY_TOKENS;
    while (n > 1 && tokens < int64_t(n) * 2048) n /= 2;
    return n;
}
// workgroups of the backward, each with a row of partial sums
constexpr int32_t rotary_bwd_workgroups(int64_t tokens) {
    const int64_t all = (tokens + rotary_tokens(tokens) - 1) / rotary_tokens(tokens);
    return (int32_t)(all < 1024 ? all : 1024);
}
hipError_t launch_rotary_fwd(const RotaryArgs& a, hipStream_t s);
hipError_t launch_rotary_bwd(const RotaryArgs& a, hipStream_t s);

}  // namespace gdn
