// The selective state space scan: h = e^{dt A} h + dt u B for each channel and
// state, y = C h, over prompts, its gradients, and single tokens.
//
// A state differs from every other in its decays, so nothing of the recurrence
// is a matrix product: a token costs each state a product for the exponent, an
// exponential, the update (two operations) and one for y. The prompts' kernels
// are bound by vector issue, not by memory. The layout keeps everything else
// off the vector units: a lane holds four states of one channel, S / 4 lanes a
// channel, so that sums over states cross few lanes; what belongs to a token
// and channel (the softplus, the products with u, the gate) is computed once,
// by the thread that loads it, and read from LDS by the lanes that need it.
// Long sequences of few channels are cut into segments, whose own states are
// summed up first (summary), carried over (merge) and then entered with.
#include "gdn_mixer_device.h"

namespace gdn {

namespace {

constexpr int NT = 256;

template <int S>
struct Shape {
    static constexpr int LPC = S / 4;              // lanes of a channel
    static constexpr int CH = 1024 / S;            // channels of a workgroup
    static constexpr int CPW = 64 / LPC;           // of a wave
    static constexpr int V = CH / 4;               // vectors of a token's channels
    static constexpr int SV = S / 4;
};

// Channels of this workgroup: [ch, ch_end) in group g
struct Block {
    int g, ch, ch_end;
};
template <int S>
__device__ __forceinline__ Block block_of(const ScanArgs& a, int b) {
    const int g = b / a.blocks, per = a.D / a.G, ch = (b - g * a.blocks) * Shape<S>::CH;
    return {g, g * per + ch, (g + 1) * per};
}

// One tile's inputs in registers, on their way to LDS. A thread's channels are
// the same in every tile; tokens and channels past the end are read from the
// last ones and made to do nothing: dt = 0 is a decay of 1 and adds no input.
template <typename T, int S, int TT, bool GRAD>
struct Tile {
    typedef Shape<S> Sh;
    static constexpr int N = TT * Sh::V, NV = (N + NT - 1) / NT;         // vectors of u, dt, ..
    static constexpr int NB = 2 * TT * Sh::SV, NBV = (NB + NT - 1) / NT; // of B and C together
    typename Four<T>::raw u[NV], dt[NV], gate[NV], dout[GRAD ? NV : 1], bc[NBV];

    static __device__ __forceinline__ int row(int i) { return (threadIdx.x + i * NT) / Sh::V; }
    static __device__ __forceinline__ bool has(int i) { return N % NT == 0 || threadIdx.x + i * NT < N; }

    // tokens [t0, t0 + TT) of the sequence at start, of which those below end count
    __device__ __forceinline__ void load(const ScanArgs& a, const Block& k, int64_t start, int t0, int end) {
        const int cv = threadIdx.x % Sh::V;
        const int ch = min(k.ch + 4 * cv, k.ch_end - 4);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t t = start + min(t0 + row(i), end - 1);
            u[i] = load4(static_cast<const T*>(a.u) + t * a.u_stride + ch);
            dt[i] = load4(static_cast<const T*>(a.dt) + t * a.dt_stride + ch);
            if (a.gate) gate[i] = load4(static_cast<const T*>(a.gate) + t * a.gate_stride + ch);
            if constexpr (GRAD) dout[i] = load4(static_cast<const T*>(a.dout) + t * a.D + ch);
        }
#pragma unroll
        for (int i = 0; i < NBV; ++i) {
            const int j = min((int)threadIdx.x + i * NT, NB - 1), r = j % (NB / 2);
            const int64_t t = start + min(t0 + r / Sh::SV, end - 1);
            const bool is_c = j >= NB / 2;
            const T* p = is_c ? static_cast<const T*>(a.c) + t * a.c_stride[0] + k.g * a.c_stride[1]
                              : static_cast<const T*>(a.b) + t * a.b_stride[0] + k.g * a.b_stride[1];
            bc[i] = load4(p + 4 * (r % Sh::SV));
        }
    }
    // B and C as floats, [2][TT][S / 4]; zero past the end
    __device__ __forceinline__ void put_bc(f32x4* at, int t0, int end) const {
#pragma unroll
        for (int i = 0; i < NBV; ++i) {
            const int j = threadIdx.x + i * NT;
            if (NB % NT != 0 && j >= NB) break;
            const f32x4 x = Four<T>::wide(bc[i]);
            at[j] = t0 + (j % (NB / 2)) / Sh::SV < end ? x : f32x4{0, 0, 0, 0};
        }
    }
};

__device__ __forceinline__ f32x4 load_f4(const float* p, int ch) {
    return p ? *reinterpret_cast<const f32x4*>(p + ch) : f32x4{0, 0, 0, 0};
}

__device__ __forceinline__ f32x4 step_sizes(f32x4 raw, int softplus) {
    if (!softplus) return raw;
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = softplus1(raw[j]);
    return r;
}

// ------------------------------------------------------------------ prompts
template <typename T, int S>
__global__ __launch_bounds__(NT) void scan_fwd_kernel(ScanArgs a) {
    typedef Shape<S> Sh;
    constexpr int TT = SCAN_TILE, G4 = Sh::LPC < 4 ? Sh::LPC : 4;
    typedef Tile<T, S, TT, false> Tl;
    __shared__ f32x2 xs[TT][Sh::CH];                 // dt, dt u
    __shared__ f32x4 bc[2 * TT * Sh::SV];
    __shared__ float ys[TT][Sh::CH + 4];

    const int nb = a.G * a.blocks;
    const Block k = block_of<S>(a, blockIdx.x % nb);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = wave * Sh::CPW + lane / Sh::LPC, sl = lane % Sh::LPC;
    const bool mine = k.ch + c < k.ch_end;
    const int d = mine ? k.ch + c : k.ch_end - 1;
    const int64_t at = (int64_t)d * S + 4 * sl, page_size = (int64_t)a.D * S;

    const f32x4 A2 = *reinterpret_cast<const f32x4*>(a.A + at) * LOG2E;
    f32x4 h = {0, 0, 0, 0};
    if (a.cut) {
        h = *reinterpret_cast<const f32x4*>(a.slots + piece * page_size + at);
    } else if (a.s_in) {
        const int64_t page = page_of(a.in_pages, a.n_pages, pc.unit);
        if (page >= 0) h = *reinterpret_cast<const f32x4*>(a.s_in + page * page_size + at);
    }
    float* keep = a.h ? a.h + piece_base(a.keep, pc.unit, pc.seq.start) * page_size + at : nullptr;

    const int cv = threadIdx.x % Sh::V;
    const bool cv_ok = k.ch + 4 * cv < k.ch_end;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    const f32x4 bias = load_f4(a.dt_bias, cch), skip = load_f4(a.skip, cch);
    T* out = static_cast<T*>(a.out) + cch;

    Tl tile;
    if (pc.first < pc.end) tile.load(a, k, pc.seq.start, pc.first, pc.end);
    for (int t0 = pc.first; t0 < pc.end; t0 += TT) {
        f32x4 u[Tl::NV], gate[Tl::NV];
#pragma unroll
        for (int i = 0; i < Tl::NV; ++i) {
            u[i] = Four<T>::wide(tile.u[i]);
            gate[i] = Four<T>::wide(tile.gate[i]);
            f32x4 dt = step_sizes(Four<T>::wide(tile.dt[i]) + bias, a.softplus);
            if (t0 + Tl::row(i) >= pc.end) dt = f32x4{0, 0, 0, 0};
            if (Tl::has(i)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) xs[Tl::row(i)][4 * cv + j] = f32x2{dt[j], dt[j] * u[i][j]};
            }
        }
        tile.put_bc(bc, t0, pc.end);
        lds_barrier();
        if (t0 + TT < pc.end) tile.load(a, k, pc.seq.start, t0 + TT, pc.end);

        const int n = min(TT, pc.end - t0);
#pragma unroll 1
        for (int q = 0; q < n; q += 8) {
            if (keep && q % SCAN_KEEP == 0 && mine)
                *reinterpret_cast<f32x4*>(keep + (t0 + q) / SCAN_KEEP * page_size) = h;
#pragma unroll
            for (int r = 0; r < 8; r += G4) {
                float got = 0.0f;
#pragma unroll
                for (int e = 0; e < G4; ++e) {
                    const int t = q + r + e;
                    const f32x2 x = xs[t][c];
                    const f32x4 B = bc[t * Sh::SV + sl], C = bc[(TT + t) * Sh::SV + sl];
                    float y = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[j] = fmaf(__builtin_amdgcn_exp2f(x[0] * A2[j]), h[j], x[1] * B[j]);
                        y = j ? fmaf(C[j], h[j], y) : C[j] * h[j];
                    }
                    y = lane_sum<Sh::LPC>(y);
                    got = e == 0 || sl == e ? y : got;
                }
                if (sl < G4) ys[q + r + sl][c] = got;
            }
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < Tl::NV; ++i) {
            const int row = Tl::row(i);
            if (!Tl::has(i) || !cv_ok || t0 + row >= pc.end) continue;
            f32x4 y = *reinterpret_cast<const f32x4*>(&ys[row][4 * cv]) + skip * u[i];
            if (a.gate) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] *= gate[i][j] * sigmoid1(gate[i][j]);
            }
            store4(out + (pc.seq.start + t0 + row) * a.D, y);
        }
    }
    if (a.s_out && pc.end == pc.seq.len && mine) {
        const int64_t page = page_of(a.out_pages, a.n_pages, pc.unit);
        if (page >= 0) *reinterpret_cast<f32x4*>(a.s_out + page * page_size + at) = h;
    }
}

// A segment's own state, entered with zero, and the sum of its dt; in reverse
// the gradient that it passes on to the token in front of it. The segment that
// nothing follows needs neither.
template <typename T, int S, bool REVERSE>
__global__ __launch_bounds__(NT) void scan_summary_kernel(ScanArgs a) {
    typedef Shape<S> Sh;
    constexpr int TT = SCAN_TILE;
    typedef Tile<T, S, TT, REVERSE> Tl;
    __shared__ f32x2 xs[TT][Sh::CH];                 // dt and dt u, or dy
    __shared__ f32x4 bc[2 * TT * Sh::SV];

    const int nb = a.G * a.blocks;
    const Block k = block_of<S>(a, blockIdx.x % nb);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none || (REVERSE ? pc.first == 0 : pc.end == pc.seq.len)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = wave * Sh::CPW + lane / Sh::LPC, sl = lane % Sh::LPC;
    const bool mine = k.ch + c < k.ch_end;
    const int d = mine ? k.ch + c : k.ch_end - 1;
    const int64_t at = (int64_t)d * S + 4 * sl, page_size = (int64_t)a.D * S;
    const f32x4 A2 = *reinterpret_cast<const f32x4*>(a.A + at) * LOG2E;
    f32x4 h = {0, 0, 0, 0};
    float sum = 0.0f;
    const int cv = threadIdx.x % Sh::V;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    const f32x4 bias = load_f4(a.dt_bias, cch);

    Tl tile;
    const int tiles = (pc.end - pc.first + TT - 1) / TT;
    auto first_of = [&](int i) { return pc.first + (REVERSE ? tiles - 1 - i : i) * TT; };
    tile.load(a, k, pc.seq.start, first_of(0), pc.end);
    for (int it = 0; it < tiles; ++it) {
        const int t0 = first_of(it);
#pragma unroll
        for (int i = 0; i < Tl::NV; ++i) {
            f32x4 dt = step_sizes(Four<T>::wide(tile.dt[i]) + bias, a.softplus);
            f32x4 x;
            if constexpr (REVERSE) {
                x = Four<T>::wide(tile.dout[i]);
                if (a.gate) {
                    const f32x4 g = Four<T>::wide(tile.gate[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] *= g[j] * sigmoid1(g[j]);
                }
            } else {
                x = Four<T>::wide(tile.u[i]) * dt;
            }
            if (t0 + Tl::row(i) >= pc.end) dt = x = f32x4{0, 0, 0, 0};
            if (Tl::has(i)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) xs[Tl::row(i)][4 * cv + j] = f32x2{dt[j], x[j]};
            }
        }
        tile.put_bc(bc, t0, pc.end);
        lds_barrier();
        if (it + 1 < tiles) tile.load(a, k, pc.seq.start, first_of(it + 1), pc.end);
        const int n = min(TT, pc.end - t0);
#pragma unroll 1
        for (int q = 0; q < n; q += 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = REVERSE ? (n + 7) / 8 * 8 - 1 - q - e : q + e;
                const f32x2 x = xs[t][c];
                const f32x4 B = bc[((REVERSE ? TT : 0) + t) * Sh::SV + sl];
                sum += x[0];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e2 = __builtin_amdgcn_exp2f(x[0] * A2[j]);
                    if constexpr (REVERSE) h[j] = e2 * fmaf(x[1], B[j], h[j]);
                    else h[j] = fmaf(e2, h[j], x[1] * B[j]);
                }
            }
        }
        lds_barrier();
    }
    if (mine) {
        *reinterpret_cast<f32x4*>(a.slots + piece * page_size + at) = h;
        if (sl == 0) a.sums[(int64_t)piece * a.D + d] = sum;
    }
}

// The segments' own states become the states that they are entered with. A
// thread walks one value through a sequence's segments.
template <bool REVERSE>
__global__ __launch_bounds__(NT) void scan_merge_kernel(ScanArgs a, int blocks) {
    const int u = blockIdx.x / blocks;
    const int64_t page_size = (int64_t)a.D * a.S;
    const int64_t e = (int64_t)(blockIdx.x % blocks) * NT + threadIdx.x;
    if (e >= page_size) return;
    const Seq q = seq_of(a.un, u);
    const int64_t base = piece_base(a.un, u, q.start);
    const int n = q.len > a.un.P ? (q.len - 1) / a.un.P + 1 : 1;
    const int d = (int)(e / a.S);
    const float A2 = a.A[e] * LOG2E;
    float x = 0.0f;
    if (a.s_in) {
        const int64_t page = page_of(a.in_pages, a.n_pages, u);
        if (page >= 0) x = a.s_in[page * page_size + e];
    }
    constexpr int AHEAD = 8;
    float own[AHEAD], sum[AHEAD];
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i0 + i + 1 >= n) break;   // the last one's is not there
            const int64_t p = base + (REVERSE ? n - 1 - i0 - i : i0 + i);
            own[i] = a.slots[p * page_size + e];
            sum[i] = a.sums[p * a.D + d];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i0 + i >= n) break;
            const int64_t p = base + (REVERSE ? n - 1 - i0 - i : i0 + i);
            a.slots[p * page_size + e] = x;
            if (i0 + i + 1 < n) x = fmaf(__builtin_amdgcn_exp2f(sum[i] * A2), x, own[i]);
        }
    }
}

// ------------------------------------------------------------------ gradients
// A wave's sums over its channels of dB's and dC's terms (four states each in a
// lane): every exchange halves the values, so 8 values over 16 channels take 16
// operations. Where lane l's result belongs: value (l >> 5: dB, dC), state 4 sl
// + 2 bit 3 + bit 4 of l; with S = 64 bit 3 is of sl, and there are two results.
template <int S>
__device__ __forceinline__ f32x2 channel_sums(f32x4 b, f32x4 c, int lane) {
    const float r0 = halves_sum(b[0], c[0]), r1 = halves_sum(b[1], c[1]);
    const float r2 = halves_sum(b[2], c[2]), r3 = halves_sum(b[3], c[3]);
    float q0 = rows_sum(r0, r1), q1 = rows_sum(r2, r3);
    if constexpr (S <= 32) {
        q0 += dpp<ROW_ROR8>(q0);
        q1 += dpp<ROW_ROR8>(q1);
        if constexpr (S <= 16) {
            q0 += dpp<ROW_ROR4>(q0);
            q1 += dpp<ROW_ROR4>(q1);
        }
        q0 = lane & 8 ? q1 : q0;
        if constexpr (S == 8) q0 += dpp<QUAD_XOR2>(q0);
    }
    return f32x2{q0, q1};
}

template <typename T, int S>
__global__ __launch_bounds__(NT) void scan_bwd_kernel(ScanArgs a) {
    typedef Shape<S> Sh;
    constexpr int TT = SCAN_KEEP, G4 = Sh::LPC < 4 ? Sh::LPC : 4;
    typedef Tile<T, S, TT, true> Tl;
    __shared__ f32x4 xs[TT][Sh::CH];                 // dt, dt u, dy
    __shared__ f32x4 bc[2 * TT * Sh::SV];
    __shared__ float sums[3][TT][Sh::CH + 4];        // over states: B g, E h A, C h
    __shared__ float parts[4][TT][2 * S];            // over a wave's channels: dB, dC

    const int nb = a.G * a.blocks, blk = blockIdx.x % nb;
    const Block k = block_of<S>(a, blk);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = wave * Sh::CPW + lane / Sh::LPC, sl = lane % Sh::LPC;
    const bool mine = k.ch + c < k.ch_end;
    const int d = mine ? k.ch + c : k.ch_end - 1;
    const int64_t at = (int64_t)d * S + 4 * sl, page_size = (int64_t)a.D * S;
    // this piece's part of dA, and of dskip and ddt_bias
    float* part = a.a_parts + piece * ((int64_t)a.D * (S + 2));
    const int cv = threadIdx.x % Sh::V;
    const bool cv_ok = k.ch + 4 * cv < k.ch_end;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    f32x4 dA = {0, 0, 0, 0}, dskip = {0, 0, 0, 0}, dbias = {0, 0, 0, 0};

    if (!pc.none) {
        const f32x4 A2 = *reinterpret_cast<const f32x4*>(a.A + at) * LOG2E;
        f32x4 E = {0, 0, 0, 0};
        if (a.cut) E = *reinterpret_cast<const f32x4*>(a.slots + piece * page_size + at);
        else if (a.s_in) E = *reinterpret_cast<const f32x4*>(a.s_in + pc.unit * page_size + at);
        const float* keep = a.h + piece_base(a.keep, pc.unit, pc.seq.start) * page_size + at;
        const f32x4 bias = load_f4(a.dt_bias, cch), skip = load_f4(a.skip, cch);

        Tl tile;
        f32x4 entry = {0, 0, 0, 0};
        auto load = [&](int t0) {
            tile.load(a, k, pc.seq.start, t0, pc.end);
            entry = *reinterpret_cast<const f32x4*>(keep + t0 / TT * page_size);
        };
        const int last = pc.first + (pc.end - pc.first - 1) / TT * TT;
        if (pc.first < pc.end) load(last);
        for (int t0 = last; t0 >= pc.first && pc.first < pc.end; t0 -= TT) {
            f32x4 u[Tl::NV], dt[Tl::NV], raw[Tl::NV], gate[Tl::NV], dout[Tl::NV], dy[Tl::NV];
#pragma unroll
            for (int i = 0; i < Tl::NV; ++i) {
                u[i] = Four<T>::wide(tile.u[i]);
                raw[i] = Four<T>::wide(tile.dt[i]) + bias;
                dt[i] = step_sizes(raw[i], a.softplus);
                dy[i] = dout[i] = Four<T>::wide(tile.dout[i]);
                if (a.gate) {
                    gate[i] = Four<T>::wide(tile.gate[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dy[i][j] *= gate[i][j] * sigmoid1(gate[i][j]);
                }
                if (t0 + Tl::row(i) >= pc.end || !cv_ok) dt[i] = dy[i] = f32x4{0, 0, 0, 0};
                if (Tl::has(i)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        xs[Tl::row(i)][4 * cv + j] = f32x4{dt[i][j], dt[i][j] * u[i][j], dy[i][j], 0.0f};
                }
            }
            tile.put_bc(bc, t0, pc.end);
            const f32x4 h0 = entry;
            lds_barrier();
            if (t0 > pc.first) load(t0 - TT);

            // the states of the tile once more
            f32x4 h[TT], ea[TT];
#pragma unroll
            for (int t = 0; t < TT; t += G4) {
                float got = 0.0f;
#pragma unroll
                for (int e = 0; e < G4; ++e) {
                    const f32x4 x = xs[t + e][c];
                    const f32x4 B = bc[(t + e) * Sh::SV + sl], C = bc[(TT + t + e) * Sh::SV + sl];
                    float y = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ea[t + e][j] = __builtin_amdgcn_exp2f(x[0] * A2[j]);
                        h[t + e][j] = fmaf(ea[t + e][j], t + e ? h[t + e - 1][j] : h0[j], x[1] * B[j]);
                        y = j ? fmaf(C[j], h[t + e][j], y) : C[j] * h[t + e][j];
                    }
                    if (a.gate) {
                        y = lane_sum<Sh::LPC>(y);
                        got = e == 0 || sl == e ? y : got;
                    }
                }
                if (a.gate && sl < G4) sums[2][t + sl][c] = got;
            }
            // and their gradients, backwards
#pragma unroll
            for (int t = TT - G4; t >= 0; t -= G4) {
                float gu = 0.0f, gt = 0.0f;
#pragma unroll
                for (int e = G4 - 1; e >= 0; --e) {
                    const f32x4 x = xs[t + e][c];
                    const f32x4 B = bc[(t + e) * Sh::SV + sl], C = bc[(TT + t + e) * Sh::SV + sl];
                    f32x4 pb, pcv;
                    float su = 0.0f, st = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float g = fmaf(C[j], x[2], E[j]);
                        pb[j] = x[1] * g;
                        pcv[j] = x[2] * h[t + e][j];
                        su = j ? fmaf(B[j], g, su) : B[j] * g;
                        E[j] = ea[t + e][j] * g;
                        const float w = E[j] * (t + e ? h[t + e - 1][j] : h0[j]);
                        st = j ? fmaf(w, A2[j], st) : w * A2[j];
                        dA[j] = fmaf(w, x[0], dA[j]);
                    }
                    su = lane_sum<Sh::LPC>(su);
                    st = lane_sum<Sh::LPC>(st);
                    gu = e == G4 - 1 || sl == e ? su : gu;
                    gt = e == G4 - 1 || sl == e ? st : gt;
                    const f32x2 r = channel_sums<S>(pb, pcv, lane);
                    float* p = &parts[wave][t + e][(lane >> 5) * S + 4 * sl + ((lane >> 4) & 1)];
                    if constexpr (S == 64) {
                        p[0] = r[0];
                        p[2] = r[1];
                    } else {
                        p[(lane >> 3 & 1) * 2] = r[0];
                    }
                }
                if (sl < G4) {
                    sums[0][t + sl][c] = gu;
                    sums[1][t + sl][c] = gt;
                }
            }
            lds_barrier();
            // dB and dC of this workgroup's channels
            const int n = min(TT, pc.end - t0);
            for (int i = threadIdx.x; i < n * (2 * S / 4); i += NT) {
                const f32x4* p = reinterpret_cast<const f32x4*>(&parts[0][0][0]) + i;
                constexpr int W = TT * 2 * S / 4;
                const f32x4 r = (p[0] + p[W]) + (p[2 * W] + p[3 * W]);
                reinterpret_cast<f32x4*>(a.bc_parts + ((int64_t)blk * a.un.total + pc.seq.start + t0) * (2 * S))[i] = r;
            }
#pragma unroll
            for (int i = 0; i < Tl::NV; ++i) {
                const int row = Tl::row(i);
                if (!Tl::has(i) || !cv_ok || t0 + row >= pc.end) continue;
                const f32x4 gu = *reinterpret_cast<const f32x4*>(&sums[0][row][4 * cv]);
                const f32x4 gt = *reinterpret_cast<const f32x4*>(&sums[1][row][4 * cv]) * LN2;
                const int64_t o = (pc.seq.start + t0 + row) * a.D + cch;
                f32x4 ddt = gu * u[i] + gt;
                if (a.softplus) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) ddt[j] *= sigmoid1(raw[i][j]);
                }
                store4(static_cast<T*>(a.du) + o, dt[i] * gu + skip * dy[i]);
                store4(static_cast<T*>(a.ddt) + o, ddt);
                dskip += dy[i] * u[i];
                dbias += ddt;
                if (a.gate) {
                    f32x4 y = *reinterpret_cast<const f32x4*>(&sums[2][row][4 * cv]) + skip * u[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] *= dout[i][j] * silu_slope(gate[i][j], sigmoid1(gate[i][j]));
                    store4(static_cast<T*>(a.dgate) + o, y);
                }
            }
        }
        if (a.s_out && pc.first == 0 && mine) *reinterpret_cast<f32x4*>(a.s_out + pc.unit * page_size + at) = E;
    }
    // this piece's sums over its tokens
    if (mine) *reinterpret_cast<f32x4*>(part + at) = dA;
    lds_barrier();
    f32x4(*red)[NT] = reinterpret_cast<f32x4(*)[NT]>(S == 8 ? &sums[0][0][0] : &parts[0][0][0]);
    static_assert((S == 8 ? sizeof(sums) : sizeof(parts)) >= 2 * NT * sizeof(f32x4), "");
    red[0][threadIdx.x] = dskip;
    red[1][threadIdx.x] = dbias;
    lds_barrier();
    if (threadIdx.x < 2 * Sh::V && cv_ok) {
        const f32x4* p = red[threadIdx.x / Sh::V] + cv;
        f32x4 s = p[0];
        for (int i = Sh::V; i < NT; i += Sh::V) s += p[i];
        *reinterpret_cast<f32x4*>(part + page_size + (threadIdx.x / Sh::V) * a.D + cch) = s;
    }
}

// dB and dC: sums over the workgroups of a group's channels, four values a thread
template <typename T>
__global__ __launch_bounds__(NT) void scan_bc_kernel(ScanArgs a) {
    const int per = 2 * a.S / 4;
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x, rows = i / per;
    if (rows >= a.un.total * a.G) return;
    const int64_t t = rows / a.G;
    const int g = (int)(rows % a.G), v = (int)(i % per);
    const f32x4* p = reinterpret_cast<const f32x4*>(a.bc_parts) + ((int64_t)g * a.blocks * a.un.total + t) * per + v;
    const int64_t step = a.un.total * per;
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 8
    for (int b = 0; b < a.blocks; ++b) s += p[b * step];
    T* o = static_cast<T*>(v < per / 2 ? a.db : a.dc);
    store4(o + rows * a.S + 4 * (v % (per / 2)), s);
}

// ------------------------------------------------------------------ single tokens
// e^x h where x is near zero as h + h (e^x - 1): the decay itself, rounded next
// to 1 the same way at every token, would let a state that hardly decays drift.
__device__ __forceinline__ float decayed(float h, float x) {
    float p = 1.0f + x * (1.0f / 7);
    p = fmaf(x * (1.0f / 6), p, 1.0f);
    p = fmaf(x * (1.0f / 5), p, 1.0f);
    p = fmaf(x * (1.0f / 4), p, 1.0f);
    p = fmaf(x * (1.0f / 3), p, 1.0f);
    p = fmaf(x * (1.0f / 2), p, 1.0f);
    return fabsf(x) < 0.25f ? fmaf(h * x, p, h) : h * __builtin_amdgcn_exp2f(x * LOG2E);
}

// Bound by the bytes of the states, read once and written once; a thread holds
// four values of a state. AROUND: past the caches
template <typename T, int S, bool AROUND>
__global__ __launch_bounds__(NT) void scan_step_kernel(ScanArgs a) {
    constexpr int LPC = S / 4;
    const int per = (a.D * LPC + NT - 1) / NT;
    const int n = blockIdx.x / per, e = (blockIdx.x % per) * NT + threadIdx.x;
    const bool ok = e < a.D * LPC;
    const int d = ok ? e / LPC : a.D - 1, sl = e % LPC, g = d / (a.D / a.G);
    T* out = static_cast<T*>(a.out) + (int64_t)n * a.D + d;
    const int64_t page = page_of(a.in_pages, a.n_pages, n);
    if (page < 0 || page >= a.n_pages) {
        if (ok && sl == 0) *out = (T)0.0f;
        return;
    }
    f32x4* p = reinterpret_cast<f32x4*>(a.s_out + (page * a.D + d) * S + 4 * sl);
    f32x4 h = AROUND ? __builtin_nontemporal_load(p) : *p;
    const f32x4 A = *reinterpret_cast<const f32x4*>(a.A + (int64_t)d * S + 4 * sl);
    const f32x4 B = Four<T>::wide(load4(static_cast<const T*>(a.b) + n * a.b_stride[0] + g * a.b_stride[1] + 4 * sl));
    const f32x4 C = Four<T>::wide(load4(static_cast<const T*>(a.c) + n * a.c_stride[0] + g * a.c_stride[1] + 4 * sl));
    const float u = (float)static_cast<const T*>(a.u)[n * a.u_stride + d];
    float dt = (float)static_cast<const T*>(a.dt)[n * a.dt_stride + d] + (a.dt_bias ? a.dt_bias[d] : 0.0f);
    const float gate = a.gate ? (float)static_cast<const T*>(a.gate)[n * a.gate_stride + d] : 0.0f;
    const float skip = a.skip ? a.skip[d] : 0.0f;
    if (a.softplus) dt = softplus1(dt);
    const float du = dt * u;
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(du, B[j], decayed(h[j], dt * A[j]));
        y = fmaf(C[j], h[j], y);
    }
    if (ok) {
        if constexpr (AROUND) __builtin_nontemporal_store(h, p);
        else *p = h;
    }
    y = lane_sum<LPC>(y) + skip * u;
    if (a.gate) y *= gate * sigmoid1(gate);
    if (ok && sl == 0) *out = (T)y;
}

template <typename F>
hipError_t by_type(int dtype, int S, F f) {
    auto with = [&](auto t) {
        switch (S) {
            case 8: f(t, std::integral_constant<int, 8>()); break;
            case 16: f(t, std::integral_constant<int, 16>()); break;
            case 32: f(t, std::integral_constant<int, 32>()); break;
            default: f(t, std::integral_constant<int, 64>()); break;
        }
    };
    if (dtype == GDN_DTYPE_BF16) with(bf16());
    else with(float());
    return hipGetLastError();
}

unsigned grid_of(const ScanArgs& a) { return (unsigned)((int64_t)a.un.n_pieces * a.G * a.blocks); }

}  // namespace

hipError_t launch_scan_summary(const ScanArgs& a, bool reverse, hipStream_t s) {
    return by_type(a.dtype, a.S, [&](auto t, auto n) {
        if (reverse) scan_summary_kernel<decltype(t), n(), true><<<grid_of(a), NT, 0, s>>>(a);
        else scan_summary_kernel<decltype(t), n(), false><<<grid_of(a), NT, 0, s>>>(a);
    });
}

hipError_t launch_scan_merge(const ScanArgs& a, bool reverse, hipStream_t s) {
    const int blocks = (int)(((int64_t)a.D * a.S + NT - 1) / NT);
    const unsigned grid = (unsigned)((int64_t)a.un.n_units * blocks);
    if (reverse) scan_merge_kernel<true><<<grid, NT, 0, s>>>(a, blocks);
    else scan_merge_kernel<false><<<grid, NT, 0, s>>>(a, blocks);
    return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t s) {
    return by_type(a.dtype, a.S,
                   [&](auto t, auto n) { scan_fwd_kernel<decltype(t), n()><<<grid_of(a), NT, 0, s>>>(a); });
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s) {
    const hipError_t e = by_type(
        a.dtype, a.S, [&](auto t, auto n) { scan_bwd_kernel<decltype(t), n()><<<grid_of(a), NT, 0, s>>>(a); });
    if (e != hipSuccess) return e;
    const unsigned bc = (unsigned)((a.un.total * a.G * (2 * a.S / 4) + NT - 1) / NT);
    if (bc > 0) {
        if (a.dtype == GDN_DTYPE_BF16) scan_bc_kernel<bf16><<<bc, NT, 0, s>>>(a);
        else scan_bc_kernel<float><<<bc, NT, 0, s>>>(a);
    }
    const int64_t d = a.D;
    return launch_row_sums(a.a_parts, a.un.n_pieces, d * (a.S + 2),
                           RowSums{{a.dA, a.dskip, a.ddt_bias}, {d * a.S, d, d}}, s);
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t s) {
    const int n_seq = a.un.n_units;
    if (n_seq == 0) return hipSuccess;
    const int64_t grid = (int64_t)n_seq * (((int64_t)a.D * (a.S / 4) + NT - 1) / NT);
    const bool around = (int64_t)n_seq * a.D * a.S * 4 > MX_LAST_LEVEL_BYTES;
    return by_type(a.dtype, a.S, [&](auto t, auto n) {
        if (around) scan_step_kernel<decltype(t), n(), true><<<(unsigned)grid, NT, 0, s>>>(a);
        else scan_step_kernel<decltype(t), n(), false><<<(unsigned)grid, NT, 0, s>>>(a);
    });
}

}  // namespace gdn
