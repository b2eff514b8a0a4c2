// Device-side helpers of the operators around the recurrent layers: vectors of
// four values in either type, sequences and their pieces, sums over lanes.
#pragma once

#include "gdn_device.h"
#include "gdn_mixer_internal.h"

namespace gdn {

typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
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

__device__ __forceinline__ float sigmoid1(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * LOG2E));
}
// d/dx of x sigmoid(x)
__device__ __forceinline__ float silu_slope(float x, float sg) { return sg * fmaf(x, 1.0f - sg, 1.0f); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x|, and log(1 + e) = 2 atanh(s)
// with s = e / (2 + e) <= 1/3: the odd series up to s^13 leaves 2^-26. A sum of
// 1 and a small e would lose the small steps that matter.
__device__ __forceinline__ float softplus1(float x) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(x) * LOG2E);
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
    float p = 1.0f / 13;
    p = fmaf(p, q, 1.0f / 11);
    p = fmaf(p, q, 1.0f / 9);
    p = fmaf(p, q, 1.0f / 7);
    p = fmaf(p, q, 1.0f / 5);
    p = fmaf(p, q, 1.0f / 3);
    p = fmaf(p, q, 1.0f);
    return fmaf(2.0f * s, p, fmaxf(x, 0.0f));
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
// lanes below 32 get x summed over both halves of the wave, the others y
__device__ __forceinline__ float halves_sum(float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(f2u(x), f2u(y), false, false);
    return u2f(r[0]) + u2f(r[1]);
}
// even rows of 16 lanes get x summed over both rows of a half, odd ones y
__device__ __forceinline__ float rows_sum(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(f2u(x), f2u(y), false, false);
    return u2f(r[0]) + u2f(r[1]);
}

}  // namespace gdn
