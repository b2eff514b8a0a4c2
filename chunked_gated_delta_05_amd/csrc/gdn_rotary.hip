// Norms of queries and keys for each head and their rotation by position, in
// one pass, and the gradients.
//
// Bound by memory: a row is read once and written once. A lane holds two
// groups of four values that are each other's partners (or, beyond the rotated
// part and with interleaved pairs, neighbours), so that a rotation stays in the
// lane and only the sum of squares crosses lanes. The angles of a token are
// made once for all of its heads: the product with the position and its
// reduction to a quarter turn in 64 bits, sine and cosine of the rest in 32.
// (bf16, heads of 128: T=32768 with 32 and 8 of them 137 us, 4.9 TB/s; B=4 T=4096
// with 16 and 16 57 us, its gradients 83, 4.8.)
#include "gdn_mixer_device.h"

namespace gdn {

namespace {

constexpr int NT = 256;
constexpr int MAX_PAIRS = 128;

// cos and sin of a turn's fraction f: f = n / 4 + r, |r| <= 1/8, and the Taylor
// series of both on |x| <= pi / 4 (the first terms left out: 2^-29 of the sine's, 2^-33 of the cosine's)
__device__ __forceinline__ f32x2 cos_sin(double turns) {
    const double n = __builtin_rint(turns * 4.0);
    const float x = (float)((turns - n * 0.25) * 6.283185307179586), q = x * x;
    float s = 1.0f / 362880, c = -1.0f / 3628800;
    s = fmaf(s, q, -1.0f / 5040);
    s = fmaf(s, q, 1.0f / 120);
    s = fmaf(s, q, -1.0f / 6);
    s = fmaf(s * q, x, x);
    c = fmaf(c, q, 1.0f / 40320);
    c = fmaf(c, q, -1.0f / 720);
    c = fmaf(c, q, 1.0f / 24);
    c = fmaf(c, q, -0.5f);
    c = fmaf(c, q, 1.0f);
    const int k = (int)(n - 4.0 * __builtin_floor(n * 0.25));   // quarter, 0 .. 3
    const float a = k & 1 ? s : c, b = k & 1 ? c : s;
    return f32x2{k == 1 || k == 2 ? -a : a, k >= 2 ? -b : b};
}

// The angles of tokens [t0, t0 + n)
__device__ __forceinline__ void angles(const RotaryArgs& a, int64_t t0, int n, f32x2 (*cs)[MAX_PAIRS]) {
    const int pairs = a.R / 2;
    for (int i = threadIdx.x; i < n * pairs; i += NT) {
        const int tt = i / pairs, p = i - tt * pairs;
        const int64_t t = t0 + tt;
        const double pos = !a.positions ? (double)(t % a.T)
                           : a.pos_i64  ? (double)static_cast<const int64_t*>(a.positions)[t]
                                        : (double)static_cast<const int32_t*>(a.positions)[t];
        const double turns = pos * a.freqs[p] * 0.15915494309189535;
        cs[tt][p] = cos_sin(turns - __builtin_rint(turns)) * a.amplitude;
    }
}

// Lane l of a row's L: values [lo, lo + 4) and [hi, hi + 4)
struct Place {
    int lo, hi;
    bool on, rotated;
};
__device__ __forceinline__ Place place_of(const RotaryArgs& a, int l) {
    Place p;
    p.on = 8 * l < a.D;
    p.rotated = 8 * l < a.R;
    p.lo = 8 * l;
    p.hi = 8 * l + 4;
    if (p.rotated && !a.interleaved) {
        p.lo = 4 * l;
        p.hi = a.R / 2 + 4 * l;
    }
    return p;
}

// Rotates the pairs of a lane, by the angle or (SIGN -1) back
template <int SIGN>
__device__ __forceinline__ void turn(f32x4& x, f32x4& y, const f32x2* cs, bool interleaved) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(cs), v = *reinterpret_cast<const f32x4*>(cs + 2);
    const float c[4] = {u[0], u[2], v[0], v[2]}, s[4] = {SIGN * u[1], SIGN * u[3], SIGN * v[1], SIGN * v[3]};
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float a0 = x[2 * i], b0 = x[2 * i + 1], a1 = y[2 * i], b1 = y[2 * i + 1];
            x[2 * i] = fmaf(-b0, s[i], a0 * c[i]);
            x[2 * i + 1] = fmaf(a0, s[i], b0 * c[i]);
            y[2 * i] = fmaf(-b1, s[i + 2], a1 * c[i + 2]);
            y[2 * i + 1] = fmaf(a1, s[i + 2], b1 * c[i + 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a0 = x[i], b0 = y[i];
            x[i] = fmaf(-b0, s[i], a0 * c[i]);
            y[i] = fmaf(a0, s[i], b0 * c[i]);
        }
    }
}

__device__ __forceinline__ f32x4 weight4(const void* w, int at, int f32) {
    if (!w) return f32x4{1, 1, 1, 1};
    return f32 ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(w) + at)
               : Four<bf16>::wide(load4(static_cast<const bf16*>(w) + at));
}

__device__ __forceinline__ float dot4(f32x4 x, f32x4 y) {
    return fmaf(x[0], y[0], x[1] * y[1]) + fmaf(x[2], y[2], x[3] * y[3]);
}

__device__ __forceinline__ float inverse_norm(const RotaryArgs& a, float squares) {
    if (a.norm == GDN_NORM_NONE) return 1.0f;
    return 1.0f / __builtin_sqrtf((a.norm == GDN_NORM_RMS ? squares * (1.0f / a.D) : squares) + a.eps);
}

// Rows of a workgroup's tokens, dealt to its groups of L lanes: `tt` and `head`
// of row r, then of row r + NT / L, ...
struct Rows {
    int tt, head, dt, dh, heads;
    __device__ __forceinline__ Rows(int first, int step, int heads_)
        : tt(first / heads_), head(first % heads_), dt(step / heads_), dh(step % heads_), heads(heads_) {}
    __device__ __forceinline__ void next() {
        tt += dt;
        head += dh;
        if (head >= heads) {
            head -= heads;
            ++tt;
        }
    }
};

template <typename T, int L>
__global__ __launch_bounds__(NT) void rotary_fwd_kernel(RotaryArgs a, int tokens) {
    __shared__ __align__(16) f32x2 cs[ROTARY_TOKENS][MAX_PAIRS];
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)(a.tokens - t0 < tokens ? a.tokens - t0 : tokens);
    const int l = threadIdx.x % L;
    const Place p = place_of(a, l);
    f32x4 w[2][2];
    if (p.on) {
        w[0][0] = weight4(a.q_weight, p.lo, a.w_f32);
        w[0][1] = weight4(a.q_weight, p.hi, a.w_f32);
        w[1][0] = weight4(a.k_weight, p.lo, a.w_f32);
        w[1][1] = weight4(a.k_weight, p.hi, a.w_f32);
    }
    angles(a, t0, n, cs);
    lds_barrier();
    for (Rows r(threadIdx.x / L, NT / L, a.Hq + a.Hk); r.tt < n; r.next()) {
        const bool is_k = r.head >= a.Hq;
        const int head = is_k ? r.head - a.Hq : r.head;
        const int64_t t = t0 + r.tt;
        const T* in = is_k ? static_cast<const T*>(a.k) + t * a.k_stride[0] + head * a.k_stride[1]
                           : static_cast<const T*>(a.q) + t * a.q_stride[0] + head * a.q_stride[1];
        f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (p.on) {
            x = Four<T>::wide(load4(in + p.lo));
            y = Four<T>::wide(load4(in + p.hi));
        }
        const float s = inverse_norm(a, lane_sum<L>(dot4(x, x) + dot4(y, y)));
        if (!p.on) continue;
        x = x * s * (is_k ? w[1][0] : w[0][0]);
        y = y * s * (is_k ? w[1][1] : w[0][1]);
        if (p.rotated) turn<1>(x, y, &cs[r.tt][4 * l], a.interleaved);
        T* out = is_k ? static_cast<T*>(a.k_out) + (t * a.Hk + head) * a.D : static_cast<T*>(a.q_out) + (t * a.Hq + head) * a.D;
        store4(out + p.lo, x);
        store4(out + p.hi, y);
    }
}

// With n = r x: d n = weight (turned-back gradient), dx = r (dn - n <dn, n>)
// (the mean of the product for RMS, the sum for L2), dweight = sum of the
// turned-back gradient times n over rows.
template <typename T, int L>
__global__ __launch_bounds__(NT) void rotary_bwd_kernel(RotaryArgs a, int tokens) {
    __shared__ __align__(16) f32x2 cs[ROTARY_TOKENS][MAX_PAIRS];
    __shared__ f32x4 red[NT][4];
    const int l = threadIdx.x % L;
    const Place p = place_of(a, l);
    f32x4 w[2][2], dw[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) dw[i][0] = dw[i][1] = f32x4{0, 0, 0, 0};
    if (p.on) {
        w[0][0] = weight4(a.q_weight, p.lo, a.w_f32);
        w[0][1] = weight4(a.q_weight, p.hi, a.w_f32);
        w[1][0] = weight4(a.k_weight, p.lo, a.w_f32);
        w[1][1] = weight4(a.k_weight, p.hi, a.w_f32);
    }
    const float share = a.norm == GDN_NORM_RMS ? 1.0f / a.D : 1.0f;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.tokens; t0 += (int64_t)gridDim.x * tokens) {
        const int n = (int)(a.tokens - t0 < tokens ? a.tokens - t0 : tokens);
        lds_barrier();
        angles(a, t0, n, cs);
        lds_barrier();
        for (Rows r(threadIdx.x / L, NT / L, a.Hq + a.Hk); r.tt < n; r.next()) {
            const bool is_k = r.head >= a.Hq;
            const int head = is_k ? r.head - a.Hq : r.head;
            const int64_t t = t0 + r.tt;
            const T* in = is_k ? static_cast<const T*>(a.k) + t * a.k_stride[0] + head * a.k_stride[1]
                               : static_cast<const T*>(a.q) + t * a.q_stride[0] + head * a.q_stride[1];
            const int64_t row = is_k ? (t * a.Hk + head) * a.D : (t * a.Hq + head) * a.D;
            const T* grad = (is_k ? static_cast<const T*>(a.dk_out) : static_cast<const T*>(a.dq_out)) + row;
            f32x4 x = {0, 0, 0, 0}, y = x, dx = x, dy = x;
            if (p.on) {
                x = Four<T>::wide(load4(in + p.lo));
                y = Four<T>::wide(load4(in + p.hi));
                dx = Four<T>::wide(load4(grad + p.lo));
                dy = Four<T>::wide(load4(grad + p.hi));
                if (p.rotated) turn<-1>(dx, dy, &cs[r.tt][4 * l], a.interleaved);
            }
            const float s = inverse_norm(a, lane_sum<L>(dot4(x, x) + dot4(y, y)));
            x *= s;
            y *= s;
            if (is_k) {
                dw[1][0] += dx * x;
                dw[1][1] += dy * y;
            } else {
                dw[0][0] += dx * x;
                dw[0][1] += dy * y;
            }
            if (p.on) {
                dx *= is_k ? w[1][0] : w[0][0];
                dy *= is_k ? w[1][1] : w[0][1];
            }
            if (a.norm != GDN_NORM_NONE) {   // else the row has no part in it, finite or not
                const float dot = lane_sum<L>(dot4(dx, x) + dot4(dy, y)) * share;
                dx = s * (dx - x * dot);
                dy = s * (dy - y * dot);
            }
            if (!p.on) continue;
            T* out = (is_k ? static_cast<T*>(a.dk) : static_cast<T*>(a.dq)) + row;
            store4(out + p.lo, dx);
            store4(out + p.hi, dy);
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) red[threadIdx.x][i] = dw[i / 2][i % 2];
    lds_barrier();
    for (int i = threadIdx.x; i < 4 * L; i += NT) {
        const int lane = i / 4, which = i % 4;
        const Place o = place_of(a, lane);
        if (!o.on) continue;
        f32x4 s = red[lane][which];
        for (int j = lane + L; j < NT; j += L) s += red[j][which];
        *reinterpret_cast<f32x4*>(a.parts + ((int64_t)blockIdx.x * 2 + which / 2) * a.D + (which % 2 ? o.hi : o.lo)) = s;
    }
}

template <typename F>
hipError_t by_type(const RotaryArgs& a, F f) {
    auto with = [&](auto t) {
        if (a.D <= 64) f(t, std::integral_constant<int, 8>());
        else if (a.D <= 128) f(t, std::integral_constant<int, 16>());
        else f(t, std::integral_constant<int, 32>());
    };
    if (a.dtype == GDN_DTYPE_BF16) with(bf16());
    else with(float());
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary_fwd(const RotaryArgs& a, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const int n = rotary_tokens(a.tokens);
    const unsigned grid = (unsigned)((a.tokens + n - 1) / n);
    return by_type(a, [&](auto t, auto l) { rotary_fwd_kernel<decltype(t), l()><<<grid, NT, 0, s>>>(a, n); });
}

hipError_t launch_rotary_bwd(const RotaryArgs& a, hipStream_t s) {
    const int64_t d = a.D;
    if (a.tokens > 0) {
        const hipError_t e = by_type(a, [&](auto t, auto l) {
            rotary_bwd_kernel<decltype(t), l()><<<(unsigned)a.workgroups, NT, 0, s>>>(a, rotary_tokens(a.tokens));
        });
        if (e != hipSuccess || !a.parts) return e;
    }
    if (!a.dq_weight && !a.dk_weight) return hipSuccess;
    return launch_row_sums(a.parts, a.workgroups, 2 * d, RowSums{{a.dq_weight, a.dk_weight, nullptr}, {d, d, 0}}, s);
}

}  // namespace gdn
