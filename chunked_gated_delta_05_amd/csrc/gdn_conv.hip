// The short causal convolution of each channel: over prompts, its gradients,
// and single tokens; and the sums of partial rows that the gradients of
// parameters end in.
//
// A token's value costs W products for the two bytes it is read and written
// with: bound by memory. A thread walks a piece of a sequence for 16 bytes of
// neighbouring channels with the last W - 1 inputs in registers, so x is read
// once but for W - 1 tokens in front of each piece (bf16 T=8191 D=6144: 44 us,
// 4.6 TB/s, with four inputs in turn, 47 with more; B=4 T=4096 with its gradients
// 224, the gradients' walk 140 of them).
#include "gdn_mixer_device.h"

namespace gdn {

namespace {

constexpr int NT = 256;

// N neighbouring channels of a token
template <typename T, int N>
struct Chans {
    typedef T raw __attribute__((ext_vector_type(N)));
    static __device__ __forceinline__ raw load(const T* p) { return *reinterpret_cast<const raw*>(p); }
    static __device__ __forceinline__ void wide(raw x, float (&o)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = (float)x[i];
    }
    static __device__ __forceinline__ void store(T* p, const float (&x)[N]) {
        raw r;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = (T)x[i];
        *reinterpret_cast<raw*>(p) = r;
    }
};

// four neighbouring parameters
__device__ __forceinline__ f32x4 param4(const void* p, int64_t i, int f32) {
    return f32 ? *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i)
               : Four<bf16>::wide(load4(static_cast<const bf16*>(p) + i));
}

// Tap j of these channels, oldest first, and the bias
template <int W, int N>
struct Taps {
    float w[W][N], b[N];
    __device__ __forceinline__ void load(const ConvArgs& a, int ch) {
        f32x4 v[N * W / 4], c[N / 4];
#pragma unroll
        for (int i = 0; i < N * W / 4; ++i) v[i] = param4(a.weight, (int64_t)ch * W + 4 * i, a.w_f32);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) c[i] = a.bias ? param4(a.bias, ch + 4 * i, a.w_f32) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = v[(i * W + j) / 4][(i * W + j) % 4];
            b[i] = c[i / 4][i % 4];
        }
    }
    // z from the W - 1 inputs before x and x itself
    __device__ __forceinline__ void apply(const float (&past)[W - 1][N], const float (&x)[N], float (&z)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z[i] = fmaf(w[j][i], past[j][i], z[i]);
            z[i] = fmaf(w[W - 1][i], x[i], z[i]);
        }
    }
};
template <int R, int N>
__device__ __forceinline__ void shift(float (&past)[R][N], const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int j = 0; j + 1 < R; ++j) past[j][i] = past[j + 1][i];
        past[R - 1][i] = x[i];
    }
}

// The W - 1 inputs in front of token `first` of a sequence
template <typename T, int W, int N>
__device__ __forceinline__ void entry(const ConvArgs& a, const Piece& pc, int first, int ch, float (&past)[W - 1][N]) {
    const int64_t page = a.s_in ? page_of(a.in_pages, a.n_pages, pc.unit) : -1;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int p = first - (W - 1) + j;
        if (p >= 0) {
            Chans<T, N>::wide(Chans<T, N>::load(static_cast<const T*>(a.x) + (pc.seq.start + p) * a.x_stride + ch), past[j]);
        } else if (page >= 0) {
            Chans<T, N>::wide(Chans<T, N>::load(static_cast<const T*>(a.s_in) + (page * (W - 1) + p + W - 1) * a.D + ch), past[j]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) past[j][i] = 0.0f;
        }
    }
}

template <typename T, int W, int N>
__device__ __forceinline__ void leave(const ConvArgs& a, const Piece& pc, int ch, const float (&past)[W - 1][N]) {
    const int64_t page = page_of(a.out_pages, a.n_pages, pc.unit);
    if (page < 0) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        Chans<T, N>::store(static_cast<T*>(a.s_out) + (page * (W - 1) + j) * a.D + ch, past[j]);
}

// Thread of all -> piece and channels: channels run fastest, and a wave of few
// channels takes several pieces.
template <int N>
__device__ __forceinline__ bool work_of(const ConvArgs& a, int* piece, int* ch) {
    const uint32_t i = blockIdx.x * NT + threadIdx.x, nv = a.D / N;
    *piece = i / nv;
    *ch = (i - *piece * nv) * N;
    return *piece < a.un.n_pieces;
}

template <typename T, int W>
__global__ __launch_bounds__(NT) void conv_fwd_kernel(ConvArgs a) {
    constexpr int N = 16 / sizeof(T), AT = 8;      // tokens in flight
    typedef Chans<T, N> Ch;
    int piece, ch;
    if (!work_of<N>(a, &piece, &ch)) return;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none) return;
    Taps<W, N> taps;
    taps.load(a, ch);
    float past[W - 1][N];
    const T* x = static_cast<const T*>(a.x) + pc.seq.start * a.x_stride + ch;
    T* y = static_cast<T*>(a.y) + pc.seq.start * a.D + ch;
    typename Ch::raw next[AT];
    auto load = [&](int t0) {
#pragma unroll
        for (int i = 0; i < AT; ++i) next[i] = Ch::load(x + min(t0 + i, pc.end - 1) * a.x_stride);
    };
    if (pc.first < pc.end) load(pc.first);
    entry<T, W, N>(a, pc, pc.first, ch, past);
    // Whole tiles, and the last one apart: where the number of a tile's stores is
    // fixed the next tile's loads are waited for without them (45.7 to 44 us; in
    // fp32, T=8191 D=4096, 55.5 and 56).
    auto tile = [&](int t0, auto whole) {
        typename Ch::raw now[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) now[i] = next[i];
        if (whole()) load(t0 + AT);
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            if (!whole() && t0 + i >= pc.end) break;
            float v[N], z[N];
            Ch::wide(now[i], v);
            taps.apply(past, v, z);
            if (a.silu) {
#pragma unroll
                for (int j = 0; j < N; ++j) z[j] *= sigmoid1(z[j]);
            }
            Ch::store(y + (int64_t)(t0 + i) * a.D, z);
            shift(past, v);
        }
    };
    int t0 = pc.first;
    for (; t0 + AT <= pc.end; t0 += AT) tile(t0, std::true_type());
    if (t0 < pc.end) tile(t0, std::false_type());
    if (a.s_out && pc.end == pc.seq.len) leave<T, W, N>(a, pc, ch, past);
}

// The states after the sequences alone (one piece each), where they replace
// the states before, which a sequence's first piece reads.
template <typename T, int W>
__global__ __launch_bounds__(NT) void conv_state_kernel(ConvArgs a) {
    constexpr int N = 16 / sizeof(T);
    const uint32_t i = blockIdx.x * NT + threadIdx.x, nv = a.D / N, u = i / nv;
    if (u >= (uint32_t)a.un.n_units) return;
    const int ch = (i - u * nv) * N;
    const Seq seq = seq_of(a.un, u);
    const Piece pc = {seq, (int32_t)u, 0, seq.len, false};
    float past[W - 1][N];
    entry<T, W, N>(a, pc, seq.len, ch, past);
    leave<T, W, N>(a, pc, ch, past);
}

// ------------------------------------------------------------------ gradients
// Token t's dz meets the inputs t - W + 1 .. t; the walk emits the gradient of
// input t - W + 1, whose last term it is, so a piece walks W - 1 tokens past
// its end and, in the first piece, the entry state's gradients fall out of the
// same sum. Four channels a thread: eight, 16 bytes of bf16, need 256 registers
// and leave one wave a SIMD (B=4 T=4096 D=6144 with the forward: 260 us, 240).
template <typename T, int W>
__global__ __launch_bounds__(NT) void conv_bwd_kernel(ConvArgs a) {
    constexpr int N = CONV_BWD_CHANNELS, AT = 4;
    typedef Chans<T, N> Ch;
    int piece, ch;
    if (!work_of<N>(a, &piece, &ch)) return;
    const Piece pc = piece_of(a.un, piece);
    float dw[W][N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.0f;
    }
    if (!pc.none) {
        Taps<W, N> taps;
        taps.load(a, ch);
        float past[W - 1][N], dz[W][N];            // dz of the last W tokens
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) dz[j][i] = 0.0f;
        const T* x = static_cast<const T*>(a.x) + pc.seq.start * a.x_stride + ch;
        const T* dout = static_cast<const T*>(a.dout) + pc.seq.start * a.D + ch;
        const int len = pc.seq.len, stop = pc.end + W - 1;
        typename Ch::raw nx[AT], nd[AT];
        auto load = [&](int t0) {
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const int64_t t = min(t0 + i, len - 1);
                nx[i] = Ch::load(x + t * a.x_stride);
                nd[i] = Ch::load(dout + t * a.D);
            }
        };
        if (len > 0) load(pc.first);
        entry<T, W, N>(a, pc, pc.first, ch, past);
        // inner: of tiles that neither begin nor end the piece, which store as many
        // tokens each (230 to 225 us; B=2 T=2048 D=2048 35.6 to 33.2)
        auto tile = [&](int t0, auto inner) {
            typename Ch::raw cx[AT], cd[AT];
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                cx[i] = nx[i];
                cd[i] = nd[i];
            }
            if (inner() || (t0 + AT < stop && len > 0)) load(t0 + AT);
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const int t = t0 + i;
                if (!inner() && t >= stop) break;
                float v[N], g[N], z[N];
                if (inner() || t < len) {
                    Ch::wide(cx[i], v);
                    Ch::wide(cd[i], g);
                    if (a.silu) {
                        taps.apply(past, v, z);
#pragma unroll
                        for (int n = 0; n < N; ++n) g[n] *= silu_slope(z[n], sigmoid1(z[n]));
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < N; ++n) v[n] = g[n] = 0.0f;
                }
                if (inner() || t < pc.end) {
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        db[n] += g[n];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][n] = fmaf(g[n], past[j][n], dw[j][n]);
                        dw[W - 1][n] = fmaf(g[n], v[n], dw[W - 1][n]);
                    }
                }
                shift(past, v);
                shift(dz, g);
                const int p = t - (W - 1);         // whose gradient is complete
                if (!inner() && p < pc.first && pc.first > 0) continue;
                float dx[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    dx[n] = 0.0f;
#pragma unroll
                    for (int j = 0; j < W; ++j) dx[n] = fmaf(taps.w[j][n], dz[W - 1 - j][n], dx[n]);
                }
                if (!inner() && a.dfinal && p >= len - (W - 1)) {
                    float f[N];
                    Ch::wide(Ch::load(static_cast<const T*>(a.dfinal) +
                                      ((int64_t)pc.unit * (W - 1) + p - len + W - 1) * a.D + ch), f);
#pragma unroll
                    for (int n = 0; n < N; ++n) dx[n] += f[n];
                }
                if (inner() || p >= 0) Ch::store(static_cast<T*>(a.dx) + (pc.seq.start + p) * a.D + ch, dx);
                else if (a.dinitial)
                    Ch::store(static_cast<T*>(a.dinitial) + ((int64_t)pc.unit * (W - 1) + p + W - 1) * a.D + ch, dx);
            }
        };
        static_assert(W - 1 <= AT, "");
        int t0 = pc.first;
        tile(t0, std::false_type());
        for (t0 += AT; t0 + AT <= pc.end; t0 += AT) tile(t0, std::true_type());
        for (; t0 < stop; t0 += AT) tile(t0, std::false_type());
    }
    // this piece's row of sums: [D][W], then [D]
    float* row = a.parts + (int64_t)piece * a.D * (W + 1);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < W; ++j) row[(int64_t)(ch + n) * W + j] = dw[j][n];
#pragma unroll
    for (int n = 0; n < N; n += 4)
        *reinterpret_cast<f32x4*>(row + (int64_t)a.D * W + ch + n) = f32x4{db[n], db[n + 1], db[n + 2], db[n + 3]};
}

// ------------------------------------------------------------------ single tokens
template <typename T, int W>
__global__ __launch_bounds__(NT) void conv_step_kernel(ConvArgs a) {
    constexpr int N = 16 / sizeof(T);
    typedef Chans<T, N> Ch;
    const uint32_t i = blockIdx.x * NT + threadIdx.x, nv = a.D / N, n = i / nv;
    if (n >= (uint32_t)a.un.n_units) return;
    const int ch = (i - n * nv) * N;
    T* y = static_cast<T*>(a.y) + (int64_t)n * a.D + ch;
    const int64_t page = page_of(a.in_pages, a.n_pages, n);
    float z[N];
    if (page < 0 || page >= a.n_pages) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = 0.0f;
        Ch::store(y, z);
        return;
    }
    T* s = static_cast<T*>(a.s_out) + page * (W - 1) * a.D + ch;
    typename Ch::raw old[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) old[j] = Ch::load(s + (int64_t)j * a.D);
    const typename Ch::raw x = Ch::load(static_cast<const T*>(a.x) + n * a.x_stride + ch);
    Taps<W, N> taps;
    taps.load(a, ch);
    float past[W - 1][N], v[N];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Ch::wide(old[j], past[j]);
    Ch::wide(x, v);
    taps.apply(past, v, z);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<typename Ch::raw*>(s + (int64_t)j * a.D) = j + 1 < W - 1 ? old[j + 1] : x;
    if (a.silu) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] *= sigmoid1(z[j]);
    }
    Ch::store(y, z);
}

// ------------------------------------------------------------------ sums of rows
__global__ __launch_bounds__(NT) void row_sums_kernel(const float* x, int64_t rows, int64_t n, RowSums out, int q,
                                                      unsigned cols) {
    sum_rows(x, rows, n, out, q, cols, blockIdx.x);
}

template <typename F>
hipError_t by_type(const ConvArgs& a, F f) {
    auto with = [&](auto t) {
        if (a.W == 4) f(t, std::integral_constant<int, 4>());
        else if (a.W == 3) f(t, std::integral_constant<int, 3>());
        else f(t, std::integral_constant<int, 2>());
    };
    if (a.dtype == GDN_DTYPE_BF16) with(bf16());
    else with(float());
    return hipGetLastError();
}

unsigned grid_of(const ConvArgs& a, int64_t items) {
    const int n = a.dtype == GDN_DTYPE_BF16 ? 8 : 4;
    return (unsigned)((items * (a.D / n) + NT - 1) / NT);
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, bool states_after, hipStream_t s) {
    ConvArgs b = a;
    if (states_after) b.s_out = nullptr;
    const hipError_t e = by_type(a, [&](auto t, auto w) {
        conv_fwd_kernel<decltype(t), w()><<<grid_of(a, a.un.n_pieces), NT, 0, s>>>(b);
    });
    if (e != hipSuccess || !states_after) return e;
    return by_type(a, [&](auto t, auto w) {
        conv_state_kernel<decltype(t), w()><<<grid_of(a, a.un.n_units), NT, 0, s>>>(a);
    });
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) {
    const hipError_t e = by_type(a, [&](auto t, auto w) {
        const int64_t threads = a.un.n_pieces * (int64_t)(a.D / CONV_BWD_CHANNELS);
        conv_bwd_kernel<decltype(t), w()><<<(unsigned)((threads + NT - 1) / NT), NT, 0, s>>>(a);
    });
    if (e != hipSuccess) return e;
    const int64_t d = a.D;
    return launch_row_sums(a.parts, a.un.n_pieces, d * (a.W + 1),
                           RowSums{{a.dweight, a.dbias, nullptr}, {d * a.W, d, 0}}, s);
}

hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s) {
    if (a.un.n_units == 0) return hipSuccess;
    return by_type(a, [&](auto t, auto w) {
        conv_step_kernel<decltype(t), w()><<<grid_of(a, a.un.n_units), NT, 0, s>>>(a);
    });
}

// Many rows in two steps, so that a narrow row's sum is not one workgroup's;
// the first one's rows follow x's.
hipError_t launch_row_sums(float* x, int64_t rows, int64_t n, const RowSums& out, hipStream_t s) {
    const unsigned cols = (unsigned)((n + 63) / 64);
    const int64_t more = row_sums_rows(rows);
    if (more) {
        float* mid = x + rows * n;
        row_sums_kernel<<<(unsigned)(cols * more), NT, 0, s>>>(x, rows, n, RowSums{{mid, nullptr, nullptr}, {more * n, 0, 0}},
                                                               SUM_ROWS, cols);
        x = mid;
        rows = more;
    }
    row_sums_kernel<<<cols, NT, 0, s>>>(x, rows, n, out, (int)rows, cols);
    return hipGetLastError();
}

}  // namespace gdn
