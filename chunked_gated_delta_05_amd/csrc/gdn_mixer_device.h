// Device-side helpers of the operators around the recurrent layers: vectors of
// four values in either type, sequences and their pieces, sums over lanes.
#pragma once

#include "gdn_device.h"
#include "gdn_mixer_internal.h"

namespace gdn {

typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

// four values as they lie in memory, and as floats
template <typename T>
struct Four;
template <>
struct Four<float> {
    typedef f32x4 raw;
    static __device__ __forceinline__ f32x4 wide(raw x) { return x; }
    static __device__ __forceinline__ raw narrow(f32x4 x) { return x; }
};
template <>
struct Four<bf16> {
    typedef bf16x4 raw;
    static __device__ __forceinline__ f32x4 wide(raw x) { return __builtin_convertvector(x, f32x4); }
    static __device__ __forceinline__ raw narrow(f32x4 x) { return __builtin_convertvector(x, bf16x4); }
};
template <typename T>
__device__ __forceinline__ typename Four<T>::raw load4(const T* p) {
    return *reinterpret_cast<const typename Four<T>::raw*>(p);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 x) {
    *reinterpret_cast<typename Four<T>::raw*>(p) = Four<T>::narrow(x);
}

// the same through a buffer resource: what lies outside reads as zero and is not written
template <typename T>
__device__ __forceinline__ typename Four<T>::raw buffer_load4(rsrc_t r, uint32_t lane_bytes, uint32_t bytes) {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_bytes, bytes, 0));
    else return __builtin_bit_cast(bf16x4, __builtin_amdgcn_raw_buffer_load_b64(r, lane_bytes, bytes, 0));
}
template <typename T>
__device__ __forceinline__ void buffer_store4(rsrc_t r, uint32_t lane_bytes, uint32_t bytes, f32x4 x) {
    if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, lane_bytes, bytes, 0);
    else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, Four<T>::narrow(x)), r, lane_bytes, bytes, 0);
}

__device__ __forceinline__ float sigmoid1(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * LOG2E));
}
// d/dx of x sigmoid(x)
__device__ __forceinline__ float silu_slope(float x, float sg) { return sg * fmaf(x, 1.0f - sg, 1.0f); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x|. u = 1 + e loses what is
// small in e, which is what small steps consist of; log(1 + e) = log(u) + (e -
// (u - 1)) / u to first order in that loss. The division is left out: 2^-25 at
// most, where u is near 2. As a function of e off by 2.0e-7 of the value at most,
// over e from 1 to 1e-7 (the series of 2 atanh(e / (2 + e)), 2.4e-7, takes twice the
// instructions). e itself is off by the rounding of its exponent, so that the
// whole is off by 2.2e-7 from x = -1 up, 1.0e-6 at -16, 3.7e-6 at -80.
__device__ __forceinline__ float softplus1(float x) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(x) * LOG2E);
    const float u = 1.0f + e;
    return fmaxf(x, 0.0f) + fmaf(__builtin_amdgcn_logf(u), LN2, e - (u - 1.0f));
}

// ------------------------------------------------------------------ sequences
struct Seq {
    int64_t start;   // first token on the flat axis
    int32_t len;
};
__device__ __forceinline__ int64_t offset_of(const MxUnits& un, int u) {
    const int64_t o = un.offsets[u];
    return o < 0 ? 0 : (o > un.total ? un.total : o);
}
__device__ __forceinline__ Seq seq_of(const MxUnits& un, int u) {
    if (un.dense) return {(int64_t)u * un.T, un.T};
    const int64_t a = offset_of(un, u), b = offset_of(un, u + 1);
    return {a, b > a ? (int32_t)(b - a) : 0};
}
__device__ __forceinline__ int row_pieces(const MxUnits& un) { return un.T > un.P ? (un.T - 1) / un.P + 1 : 1; }
// number of a sequence's first piece
__device__ __forceinline__ int64_t piece_base(const MxUnits& un, int u, int64_t start) {
    return un.dense ? (int64_t)u * row_pieces(un) : start / un.P + u;
}
struct Piece {
    Seq seq;
    int32_t unit, first, end;   // tokens of the sequence
    bool none;                  // the number stands for no piece
};
__device__ __forceinline__ Piece piece_of(const MxUnits& un, int p) {
    Piece r;
    int64_t j;
    if (un.dense) {
        const int per = row_pieces(un);
        r.unit = p / per;
        j = p - r.unit * per;
        r.seq = seq_of(un, r.unit);
    } else {
        int lo = 0, hi = un.n_units;   // the last sequence that begins no later
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (offset_of(un, mid) / un.P + mid <= p) lo = mid;
            else hi = mid;
        }
        r.unit = lo;
        r.seq = seq_of(un, lo);
        j = p - (r.seq.start / un.P + lo);
    }
    const int64_t first = j * un.P;
    r.none = first < 0 || (first >= r.seq.len && j > 0);
    r.first = r.none ? 0 : (int32_t)first;
    r.end = r.seq.len - r.first > un.P ? r.first + un.P : r.seq.len;
    return r;
}
// the page of a sequence, or -1
__device__ __forceinline__ int64_t page_of(const int32_t* pages, int n_pages, int u) {
    if (!pages) return u;
    const int p = pages[u];
    return p < 0 || p >= n_pages ? -1 : p;
}

// ------------------------------------------------------------------ lanes
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(x), CTRL, 0xf, 0xf, true));
}
constexpr int QUAD_XOR1 = 0xB1, QUAD_XOR2 = 0x4E, ROW_ROR4 = 0x124, ROW_ROR8 = 0x128, HALF_MIRROR = 0x141;
constexpr int ROW_BCAST = 0x150;   // + i: lane i of 16 to all of them

// sum over N neighbouring lanes, in all of them
template <int N>
__device__ __forceinline__ float lane_sum(float x) {
    static_assert(N >= 1 && N <= 64, "");
    if constexpr (N >= 2) x += dpp<QUAD_XOR1>(x);
    if constexpr (N >= 4) x += dpp<QUAD_XOR2>(x);
    if constexpr (N >= 8) x += dpp<HALF_MIRROR>(x);   // every quad holds one value by now
    if constexpr (N >= 16) x += dpp<ROW_ROR8>(x);
    if constexpr (N >= 32) x += __shfl_xor(x, 16);
    if constexpr (N >= 64) x += __shfl_xor(x, 32);
    return x;
}
// Four values summed over groups of N neighbouring lanes: lane l gets value l %
// 4, or, with N = 2, values l % 2 (in r[0]) and 2 + l % 2 (r[1]). Each exchange
// halves the values: 3 instructions for two of them where sums in all lanes
// would take two exchanges each.
template <int N>
__device__ __forceinline__ f32x2 four_sums(f32x4 v, int lane) {
    static_assert(N == 2 || N == 4 || N == 8 || N == 16, "");
    if constexpr (N == 8) {   // mirrored first: every quad then holds the four pairs' sums
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += dpp<HALF_MIRROR>(v[i]);
    }
    const bool odd = lane & 1, high = lane & 2;
    const float a = (odd ? v[1] : v[0]) + dpp<QUAD_XOR1>(odd ? v[0] : v[1]);
    const float b = (odd ? v[3] : v[2]) + dpp<QUAD_XOR1>(odd ? v[2] : v[3]);
    if constexpr (N == 2) return f32x2{a, b};
    float r = (high ? b : a) + dpp<QUAD_XOR2>(high ? a : b);
    if constexpr (N == 16) {
        r += dpp<ROW_ROR8>(r);
        r += dpp<ROW_ROR4>(r);
    }
    return f32x2{r, 0.0f};
}

// ------------------------------------------------------------------ sums of rows
// Workgroup (of 256) w: row b = w / cols of out = rows [b q, b q + q) of x added
// up, 64 of its n columns: 16 threads a column vector, joined through LDS in a
// fixed order.
__device__ __forceinline__ void sum_rows(const float* x, int64_t rows, int64_t n, const RowSums& out, int q, unsigned cols,
                                         unsigned w) {
    __shared__ f32x4 part[16][17];
    const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4;
    const unsigned b = w / cols;
    const int64_t col = ((int64_t)(w - b * cols) * 16 + cl) * 4, r0 = (int64_t)b * q;
    const int64_t r1 = r0 + q < rows ? r0 + q : rows;
    f32x4 s = {0, 0, 0, 0};
    if (col < n) {
#pragma unroll 4
        for (int64_t r = r0 + rl; r < r1; r += 16) s += *reinterpret_cast<const f32x4*>(x + r * n + col);
    }
    part[rl][cl] = s;
    lds_barrier();
    if (rl == 0 && col < n) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][cl];
        int64_t at = col + (int64_t)b * n;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (at >= 0 && at < out.n[i] && out.p[i]) *reinterpret_cast<f32x4*>(out.p[i] + at) = s;
            at -= out.n[i];
        }
    }
}

}  // namespace gdn
