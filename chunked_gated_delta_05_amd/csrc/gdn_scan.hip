// The selective state space scan: h = e^{dt A} h + dt u B for each channel and
// state, y = C h, over prompts, its gradients, and single tokens.
//
// A state differs from every other in its decays, so nothing of the recurrence
// is a matrix product: a token costs each state a product for the exponent, an
// exponential, the update (two operations) and one for y. The prompts' kernels
// are bound by vector issue, not by memory: an exponential takes a SIMD 8.5
// cycles a wave, a product or sum 2.6 (with two waves or more; 4.7 with one), an
// exchange of lanes 4.2. The layout keeps everything else off the vector units:
// a lane holds four states of two channels, S / 4 lanes a pair, so that sums
// over states cross few lanes and B and C are read from LDS once for both; what
// belongs to a token and channel (the softplus, the products with u, the gate)
// is computed once, by the thread that loads it.
// Whole sequences of few channels are walked by one state a lane. Where even that
// would not fill the card sequences are cut into segments, whose own states are
// summed up first (summary), carried over (merge) and then entered with.
// bf16, S = 16, 537 million states times tokens (T=8192 D=4096; 268 MB would take
// 55 us): 185 us in six prompts, 207 in two rows, 224 in one, cut; 262 of 16 rows
// of T=1000 by two channels a lane; two rows with their gradients 730, 430 of them
// the gradients' walk.
#include "gdn_mixer_device.h"

namespace gdn {

namespace {

constexpr int NT = 256;                            // threads where the states do not matter
constexpr int FT = 16;                             // tokens of a tile
constexpr int KC = 2;                              // channels of a lane, neighbours; one in the backward
template <int S, int K = KC>
struct Shape {
    static constexpr int LPC = S / 4;              // lanes of a channel pair
    static constexpr int CH = scan_channels(S) * K / KC;   // channels of a workgroup
    static constexpr int CPW = K * 64 / LPC;       // of a wave
    static constexpr int V = CH / 4;               // vectors of a token's channels
    static constexpr int SV = S / 4;
    static constexpr int NW = CH / CPW;            // waves: 4, or 2 where they have many channels
    static constexpr int NT = 64 * NW;
    static __device__ __host__ __forceinline__ int blocks(const ScanArgs& a) { return (a.D / a.G + CH - 1) / CH; }
};

// A lane's channels and states
template <int S, int K = KC>
struct Lane {
    int lane, wave, c, sl;      // c: first channel in the workgroup
    bool mine;                  // the channels exist (they are of one vector of 8)
    int d;                      // of the first
    int64_t at;                 // of its states in a page; the second channel's follow S later
    __device__ __forceinline__ Lane(int ch, int ch_end) {
        lane = threadIdx.x & 63;
        wave = threadIdx.x >> 6;
        c = wave * Shape<S, K>::CPW + K * (lane / Shape<S, K>::LPC);
        sl = lane % Shape<S, K>::LPC;
        mine = ch + c < ch_end;
        d = mine ? ch + c : ch_end - K;
        at = (int64_t)d * S + 4 * sl;
    }
};
// K vectors, `step` values apart
template <typename V, int K>
__device__ __forceinline__ void load_states(V (&h)[K], const float* p, int step) {
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = *reinterpret_cast<const V*>(p + k * step);
}
template <typename V, int K>
__device__ __forceinline__ void store_states(float* p, const V (&h)[K], int step) {
#pragma unroll
    for (int k = 0; k < K; ++k) *reinterpret_cast<V*>(p + k * step) = h[k];
}

// Channels of this workgroup: [ch, ch_end) in group g
struct Block {
    int g, ch, ch_end;
};
template <typename Sh>
__device__ __forceinline__ Block block_of(const ScanArgs& a, int b) {
    const int per = a.D / a.G, blocks = Sh::blocks(a), g = b / blocks, ch = (b - g * blocks) * Sh::CH;
    return {g, g * per + ch, (g + 1) * per};
}

// Where a thread's vectors of a tile lie in a tensor [tokens][..]: a resource
// over the tile's tokens below the piece's end, so that tokens past it read as
// zero and are not written; 32-bit offsets made once, as a thread's channels
// and rows are the same in every tile.
template <typename T, typename Sh, int TT>
struct Rows {
    static constexpr int N = TT * Sh::V, NV = (N + Sh::NT - 1) / Sh::NT, STEP = Sh::NT / Sh::V;
    const T* base;
    int64_t stride;
    uint32_t lane;
    static __device__ __forceinline__ int row(int i) { return threadIdx.x / Sh::V + i * STEP; }
    static __device__ __forceinline__ bool has(int i) { return N % Sh::NT == 0 || row(i) < TT; }
    __device__ __forceinline__ Rows(const void* p, int64_t start, int64_t stride_, int ch)
        : base(static_cast<const T*>(p) + start * stride_), stride(stride_),
          lane((uint32_t)(row(0) * stride_ + ch) * (uint32_t)sizeof(T)) {}
    __device__ __forceinline__ rsrc_t tile(int t0, int end, int D) const {
        return make_rsrc(base + t0 * stride, (uint32_t)((min(TT, end - t0) - 1) * stride + D) * (uint32_t)sizeof(T));
    }
    __device__ __forceinline__ uint32_t bytes(int i) const { return (uint32_t)(i * STEP * stride) * (uint32_t)sizeof(T); }
    __device__ __forceinline__ void load(typename Four<T>::raw (&x)[NV], int t0, int end, int D) const {
        const rsrc_t r = tile(t0, end, D);
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = buffer_load4<T>(r, lane, bytes(i));
    }
};

// A tile's B and C in registers, on their way to LDS as floats [2][TT][S / 4]
template <typename T, typename Sh, int TT>
struct States {
    static constexpr int NB = 2 * TT * Sh::SV, NV = (NB + Sh::NT - 1) / Sh::NT;
    typename Four<T>::raw x[NV];
    __device__ __forceinline__ void load(const ScanArgs& a, int g, int64_t start, int t0, int end) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = min((int)threadIdx.x + i * Sh::NT, NB - 1), r = j % (NB / 2);
            const int64_t t = start + min(t0 + r / Sh::SV, end - 1);
            const T* p = j >= NB / 2 ? static_cast<const T*>(a.c) + t * a.c_stride[0] + g * a.c_stride[1]
                                     : static_cast<const T*>(a.b) + t * a.b_stride[0] + g * a.b_stride[1];
            x[i] = load4(p + 4 * (r % Sh::SV));
        }
    }
    // the same as [2][S][pitch], tokens along a row
    __device__ __forceinline__ void put_turned(float* at, int pitch, int t0, int end) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * Sh::NT;
            if (NB % Sh::NT != 0 && j >= NB) break;
            const int t = j % (NB / 2) / Sh::SV;
            const f32x4 v = t0 + t < end ? Four<T>::wide(x[i]) : f32x4{0, 0, 0, 0};
            float* o = at + (j / (NB / 2) * 4 * Sh::SV + j % Sh::SV * 4) * pitch + t;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k * pitch] = v[k];
        }
    }
    // zero past the end
    __device__ __forceinline__ void put(f32x4* at, int t0, int end) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * Sh::NT;
            if (NB % Sh::NT != 0 && j >= NB) break;
            const f32x4 v = Four<T>::wide(x[i]);
            at[j] = t0 + (j % (NB / 2)) / Sh::SV < end ? v : f32x4{0, 0, 0, 0};
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

// All that was loaded has arrived. Before a tile's stores and the first tile: the
// loads of the next one, issued a tile ago, would else be waited for behind the
// stores (B=2 T=4096 D=4096 215 to 207 us, with gradients 1% less).
__device__ __forceinline__ void wait_for_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// ------------------------------------------------------------------ segments
// The states that a segment is entered with, or in reverse the gradients: those
// in front of the sequence and the segments' own between, added up by the segment
// itself where there are few (join), by a merge beforehand where
// there are many.
template <bool REVERSE, int S, int K>
__device__ __forceinline__ void entry_states(const ScanArgs& a, const Piece& pc, int piece, const Lane<S, K>& l,
                                             const f32x4 (&A2)[K], f32x4 (&h)[K]) {
    const int64_t page_size = (int64_t)a.D * S;
    if (a.cut && !a.join) {
        load_states(h, a.slots + piece * page_size + l.at, S);
        return;
    }
    if (a.s_in) {
        const int64_t page = page_of(a.in_pages, a.n_pages, pc.unit);
        if (page >= 0) load_states(h, a.s_in + page * page_size + l.at, S);
    }
    if (!a.cut) return;
    const int n = REVERSE ? (pc.seq.len - 1) / a.un.P - pc.first / a.un.P : pc.first / a.un.P;   // segments before
    constexpr int AHEAD = 4;
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        f32x4 own[AHEAD][K];
        float sum[AHEAD][K];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t p = piece + (REVERSE ? 1 : -1) * (n - min(i0 + i, n - 1));
            load_states(own[i], a.slots + p * page_size + l.at, S);
#pragma unroll
            for (int k = 0; k < K; ++k) sum[i][k] = a.sums[p * a.D + l.d + k];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i0 + i >= n) break;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[k][j] = fmaf(__builtin_amdgcn_exp2f(sum[i][k] * A2[k][j]), h[k][j], own[i][k][j]);
        }
    }
}

// ------------------------------------------------------------------ prompts
// Four waves a SIMD where 128 registers hold what two channels of bf16 need (a
// training step's forward in 16 segments 9 us faster; one channel a lane, which
// would spill, 274 to 346 in 9 documents).
template <typename T, int S, int K>
__global__ __launch_bounds__((Shape<S, K>::NT), (sizeof(T) == 2 && S > 8 && K == 2 ? 4 : 2)) void scan_fwd_kernel(ScanArgs a) {
    typedef Shape<S, K> Sh;
    constexpr int TT = FT, E = 4 / K;                // E tokens give a lane four sums over states
    typedef Rows<T, Sh, TT> Rw;
    __shared__ __align__(16) f32x2 xs[TT][Sh::CH];   // dt, dt u
    __shared__ f32x4 bc[2 * TT * Sh::SV];
    __shared__ __align__(16) float ys[TT][Sh::CH + 4];

    const int nb = a.G * Sh::blocks(a);
    const Block k = block_of<Sh>(a, blockIdx.x % nb);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none) return;
    const Lane<S, K> l(k.ch, k.ch_end);
    const int64_t page_size = (int64_t)a.D * S;
    f32x4 A2[K], h[K] = {};
    load_states(A2, a.A + l.at, S);
#pragma unroll
    for (int i = 0; i < K; ++i) A2[i] *= LOG2E;
    entry_states<false, S, K>(a, pc, piece, l, A2, h);
    float* keep = a.h ? a.h + piece_base(a.keep, pc.unit, pc.seq.start) * page_size + l.at : nullptr;

    const int cv = threadIdx.x % Sh::V;
    const bool cv_ok = k.ch + 4 * cv < k.ch_end;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    const f32x4 bias = load_f4(a.dt_bias, cch), skip = load_f4(a.skip, cch);
    const Rw ru(a.u, pc.seq.start, a.u_stride, cch), rt(a.dt, pc.seq.start, a.dt_stride, cch),
        rg(a.gate, pc.seq.start, a.gate_stride, cch), ro(a.out, pc.seq.start, a.D, cch);

    typename Four<T>::raw u[Rw::NV], dt[Rw::NV], gate[Rw::NV] = {};
    States<T, Sh, TT> st;
    auto load = [&](int t0) {
        ru.load(u, t0, pc.end, a.D);
        rt.load(dt, t0, pc.end, a.D);
        if (a.gate) rg.load(gate, t0, pc.end, a.D);
        st.load(a, k.g, pc.seq.start, t0, pc.end);
    };
    if (pc.first < pc.end) load(pc.first);
    wait_for_loads();
    for (int t0 = pc.first; t0 < pc.end; t0 += TT) {
        typename Four<T>::raw own_u[Rw::NV], own_gate[Rw::NV];
#pragma unroll
        for (int i = 0; i < Rw::NV; ++i) {
            own_u[i] = u[i];
            own_gate[i] = gate[i];
            f32x4 t = step_sizes(Four<T>::wide(dt[i]) + bias, a.softplus);
            if (t0 + Rw::row(i) >= pc.end) t = f32x4{0, 0, 0, 0};   // a decay of 1, no input
            const f32x4 du = t * Four<T>::wide(u[i]);
            if (Rw::has(i)) {
                f32x4* x = reinterpret_cast<f32x4*>(&xs[Rw::row(i)][4 * cv]);
                x[0] = f32x4{t[0], du[0], t[1], du[1]};
                x[1] = f32x4{t[2], du[2], t[3], du[3]};
            }
        }
        st.put(bc, t0, pc.end);
        lds_barrier();
        if (t0 + TT < pc.end) load(t0 + TT);

        const int n = min(TT, pc.end - t0);
        struct Step {
            f32x2 x[K];
            f32x4 b, c;
        };
        auto read = [&](Step (&s)[E], int t) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (K == 2) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(&xs[t + e][l.c]);
                    s[e].x[0] = f32x2{x[0], x[1]};
                    s[e].x[1] = f32x2{x[2], x[3]};
                } else {
                    s[e].x[0] = xs[t + e][l.c];
                }
                s[e].b = bc[(t + e) * Sh::SV + l.sl];
                s[e].c = bc[(TT + t + e) * Sh::SV + l.sl];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto step = [&](const Step (&s)[E], int t) {
            f32x4 y;
#pragma unroll
            for (int e = 0; e < E; ++e) {
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h[i][j] = fmaf(__builtin_amdgcn_exp2f(s[e].x[i][0] * A2[i][j]), h[i][j], s[e].x[i][1] * s[e].b[j]);
                        sum = j ? fmaf(s[e].c[j], h[i][j], sum) : s[e].c[j] * h[i][j];
                    }
                    y[e * K + i] = sum;
                }
            }
            const f32x2 r = four_sums<Sh::LPC>(y, l.lane);
            const int v = l.lane & (Sh::LPC == 2 ? 1 : 3);
            ys[t + v / K][l.c + v % K] = r[0];
            if constexpr (Sh::LPC == 2) ys[t + (2 + v) / K][l.c + v % K] = r[1];
        };
        static_assert(TT == SCAN_KEEP, "");
        if (keep && l.mine) store_states(keep + t0 / TT * page_size, h, S);
        // some tokens' operands are on their way from LDS while others' run
        Step even[E], odd[E];
        read(even, 0);
#pragma unroll 1
        for (int q = 0; q < n; q += 2 * E) {
            read(odd, q + E);
            step(even, q);
            read(even, min(q + 2 * E, TT - E));
            step(odd, q + E);
        }
        lds_barrier();
        wait_for_loads();
        const rsrc_t out = ro.tile(t0, pc.end, a.D);
#pragma unroll
        for (int i = 0; i < Rw::NV; ++i) {
            if (!Rw::has(i) || !cv_ok) continue;
            f32x4 y = *reinterpret_cast<const f32x4*>(&ys[Rw::row(i)][4 * cv]) + skip * Four<T>::wide(own_u[i]);
            if (a.gate) {
                const f32x4 g = Four<T>::wide(own_gate[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] *= g[j] * sigmoid1(g[j]);
            }
            buffer_store4<T>(out, ro.lane, ro.bytes(i), y);
        }
    }
    if (a.s_out && pc.end == pc.seq.len && l.mine) {
        const int64_t page = page_of(a.out_pages, a.n_pages, pc.unit);
        if (page >= 0) store_states(a.s_out + page * page_size + l.at, h, S);
    }
}

// The same for whole sequences of few channels: a lane holds one state (of 32 and
// 64 states two and four), so that few sequences need not be cut, and walked
// twice, to fill the card (six prompts, T=8192 D=4096: 233 us cut, 180 so; T=160
// D=1024 15.6 and 9.6). A token costs a lane 10 instructions where the lane of
// eight states takes 7.5 a state: sums over 16 lanes, and dt and dt u from another
// lane. Two waves a SIMD issue one every 4 cycles, one wave every 7.
constexpr int NARROW_TILE = 64;
template <int S>
struct Narrow {
    static constexpr int Q = S <= 16 ? 1 : S / 16;  // states of a lane, LPC apart
    static constexpr int LPC = S / Q, CPW = 64 / LPC, NW = 4, NT = 64 * NW, CH = CPW * NW, V = CH / 4, SV = S / 4;
    static_assert(CH == scan_narrow_channels(S), "");
    static __device__ __host__ __forceinline__ int blocks(const ScanArgs& a) { return (a.D / a.G + CH - 1) / CH; }
};
typedef float f32x1 __attribute__((ext_vector_type(1)));
template <int S>
struct NarrowLane {
    static constexpr int STEP = Narrow<S>::LPC;    // from a state to the next
    int lane, c, sl, d;
    bool mine;
    int64_t at;
    __device__ __forceinline__ NarrowLane(int ch, int ch_end) {
        lane = threadIdx.x & 63;
        c = (threadIdx.x >> 6) * Narrow<S>::CPW + lane / Narrow<S>::LPC;
        sl = lane % Narrow<S>::LPC;
        mine = ch + c < ch_end;
        d = mine ? ch + c : ch_end - 1;
        at = (int64_t)d * S + sl;
    }
};
// In assembly: a and b added up with those 8 lanes away in a row of 16, a's sum in
// the lower lanes of a, b's in the upper ones. Adds that write only some quads
// take the place of selects; a value is exchanged two waits or more after it was
// written. Results are written before other inputs are read ("+&v").
#define GDN_HALVES(a, b) \
    "v_add_f32_dpp " a ", " a ", " a " row_ror:8 row_mask:0xf bank_mask:0x3\n" \
    "v_add_f32_dpp " a ", " b ", " b " row_ror:8 row_mask:0xf bank_mask:0xc\n"

// a and b added up with the partner lane's: lanes below it get a's sum, those above b's
template <int CTRL>
__device__ __forceinline__ float fold(float a, float b, bool above) {
    return (above ? b : a) + dpp<CTRL>(above ? a : b);
}
// Sixteen values over 16 lanes twice so, from 16 to 4 a lane: lanes 4 g .. 4 g + 3
// get values 4 g .. 4 g + 3 in y[0 .. 3], added up over the other quads (with
// selects 5 prompts of T=1000 D=4096 take 115 us, so 111). The wait at the end is
// for what follows.
__device__ __forceinline__ void fold16(float (&y)[16]) {
#define GDN_QUADS(a, b) \
    "v_add_f32_dpp " a ", " a ", " a " row_half_mirror row_mask:0xf bank_mask:0x5\n" \
    "v_add_f32_dpp " a ", " b ", " b " row_half_mirror row_mask:0xf bank_mask:0xa\n"
    asm("s_nop 1\n"
        GDN_HALVES("%0", "%8") GDN_HALVES("%1", "%9") GDN_HALVES("%2", "%10") GDN_HALVES("%3", "%11")
        GDN_HALVES("%4", "%12") GDN_HALVES("%5", "%13") GDN_HALVES("%6", "%14") GDN_HALVES("%7", "%15")
        "s_nop 1\n"
        GDN_QUADS("%0", "%4") GDN_QUADS("%1", "%5") GDN_QUADS("%2", "%6") GDN_QUADS("%3", "%7")
        "s_nop 1"
        : "+&v"(y[0]), "+&v"(y[1]), "+&v"(y[2]), "+&v"(y[3]), "+&v"(y[4]), "+&v"(y[5]), "+&v"(y[6]), "+&v"(y[7])
        : "v"(y[8]), "v"(y[9]), "v"(y[10]), "v"(y[11]), "v"(y[12]), "v"(y[13]), "v"(y[14]), "v"(y[15]));
#undef GDN_QUADS
}

template <typename F, int... I>
__device__ __forceinline__ void unrolled_(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}
// f of the constants 0 .. N - 1
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
    unrolled_(f, std::make_integer_sequence<int, N>());
}

template <typename T, int S>
__global__ __launch_bounds__(Narrow<S>::NT, 2) void scan_narrow_kernel(ScanArgs a) {
    typedef Narrow<S> Sh;
    constexpr int TT = NARROW_TILE, Q = Sh::Q, E = Q == 1 ? 8 : 4;   // E tokens' operands are read at a time
    typedef Rows<T, Sh, TT> Rw;
    // tokens along the rows, which are padded for the banks: 16 rows' next four tokens are read at once
    __shared__ __align__(16) f32x2 xs[Sh::CH][TT + 4];      // dt, dt u
    __shared__ __align__(16) float bc[2][S][TT + 4];
    __shared__ __align__(16) float ys[Sh::CH][TT + 4];

    const int nb = a.G * Sh::blocks(a);
    int blk = blockIdx.x % nb;
    if (nb % 8 == 0) blk = blk % 8 * (nb / 8) + blk / 8;    // neighbours share cache lines: on one die
    const Block k = block_of<Sh>(a, blk);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none) return;
    const NarrowLane<S> l(k.ch, k.ch_end);
    const int64_t page_size = (int64_t)a.D * S;
    f32x1 A2[Q], h[Q] = {};
    load_states(A2, a.A + l.at, l.STEP);
#pragma unroll
    for (int i = 0; i < Q; ++i) A2[i] *= LOG2E;
    if (a.s_in) {
        const int64_t page = page_of(a.in_pages, a.n_pages, pc.unit);
        if (page >= 0) load_states(h, a.s_in + page * page_size + l.at, l.STEP);
    }
    float* keep = a.h ? a.h + piece_base(a.keep, pc.unit, pc.seq.start) * page_size + l.at : nullptr;

    const int cv = threadIdx.x % Sh::V;
    const bool cv_ok = k.ch + 4 * cv < k.ch_end;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    const f32x4 bias = load_f4(a.dt_bias, cch), skip = load_f4(a.skip, cch);
    const Rw ru(a.u, pc.seq.start, a.u_stride, cch), rt(a.dt, pc.seq.start, a.dt_stride, cch),
        rg(a.gate, pc.seq.start, a.gate_stride, cch), ro(a.out, pc.seq.start, a.D, cch);
    typename Four<T>::raw u[Rw::NV], dt[Rw::NV], gate[Rw::NV] = {};
    States<T, Sh, TT> st;
    auto load = [&](int t0) {
        ru.load(u, t0, pc.end, a.D);
        rt.load(dt, t0, pc.end, a.D);
        if (a.gate) rg.load(gate, t0, pc.end, a.D);
        st.load(a, k.g, pc.seq.start, t0, pc.end);
    };
    if (pc.first < pc.end) load(pc.first);
    wait_for_loads();
    for (int t0 = pc.first; t0 < pc.end; t0 += TT) {
        typename Four<T>::raw own_u[Rw::NV], own_gate[Rw::NV];
#pragma unroll
        for (int i = 0; i < Rw::NV; ++i) {
            own_u[i] = u[i];
            own_gate[i] = gate[i];
            f32x4 t = step_sizes(Four<T>::wide(dt[i]) + bias, a.softplus);
            if (t0 + Rw::row(i) >= pc.end) t = f32x4{0, 0, 0, 0};   // a decay of 1, no input
            const f32x4 du = t * Four<T>::wide(u[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) xs[4 * cv + j][Rw::row(i)] = f32x2{t[j], du[j]};
        }
        st.put_turned(&bc[0][0][0], TT + 4, t0, pc.end);
        lds_barrier();
        if (t0 + TT < pc.end) load(t0 + TT);

        const int n = min(TT, pc.end - t0);
        // Of a channel with 16 lanes each lane holds one token's dt and dt u, which an
        // exchange hands to the others on its way into the product.
        constexpr bool HELD = Sh::LPC == 16;
        struct Step {
            f32x4 x[HELD ? 1 : E / 2], b[Q][E / 4], c[Q][E / 4];
        };
        auto read = [&](Step& s, int t) {
            if constexpr (!HELD) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) s.x[e] = *reinterpret_cast<const f32x4*>(&xs[l.c][t + 2 * e]);
            }
#pragma unroll
            for (int i = 0; i < Q; ++i)
#pragma unroll
                for (int e = 0; e < E / 4; ++e) {
                    s.b[i][e] = *reinterpret_cast<const f32x4*>(&bc[0][l.sl + i * l.STEP][t + 4 * e]);
                    s.c[i][e] = *reinterpret_cast<const f32x4*>(&bc[1][l.sl + i * l.STEP][t + 4 * e]);
                }
            __builtin_amdgcn_sched_barrier(0);
        };
        float y[16];
        f32x2 held = {0, 0};
        auto step = [&](const Step& s, auto first) {
            unrolled<E>([&](auto e) {
                float d, du;
                if constexpr (HELD) {
                    d = dpp<ROW_BCAST + first + e>(held[0]);
                    du = dpp<ROW_BCAST + first + e>(held[1]);
                } else {
                    d = s.x[e / 2][e % 2 * 2];
                    du = s.x[e / 2][e % 2 * 2 + 1];
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    h[i][0] = fmaf(__builtin_amdgcn_exp2f(d * A2[i][0]), h[i][0], du * s.b[i][e / 4][e % 4]);
                    sum = i ? fmaf(s.c[i][e / 4][e % 4], h[i][0], sum) : s.c[i][e / 4][e % 4] * h[i][0];
                }
                y[first + e] = sum;
            });
        };
        Step even, odd;
        f32x2 next = xs[l.c][HELD ? l.sl : 0];
        read(even, 0);
#pragma unroll 1
        for (int q = 0; q < n; q += 16) {
            static_assert(SCAN_KEEP == 16, "");
            if (keep && l.mine) store_states(keep + (t0 + q) / SCAN_KEEP * page_size, h, l.STEP);
            held = next;
            if (HELD) next = xs[l.c][min(q + 16, TT - 16) + l.sl];
            unrolled<16 / (2 * E)>([&](auto i) {
                constexpr int e = i * 2 * E;
                read(odd, q + e + E);
                step(even, std::integral_constant<int, e>());
                read(even, min(q + e + 2 * E, TT - E));
                step(odd, std::integral_constant<int, e + E>());
            });
            // the sums over states of 16 tokens: each exchange halves the tokens of a lane
            constexpr int NR = Sh::LPC == 16 ? 1 : 2;
            f32x4 r[NR];
            if constexpr (Sh::LPC == 16) fold16(y);
#pragma unroll
            for (int i = 0; i < 4 * NR; ++i) {
                float v = Sh::LPC == 16 ? y[i] : fold<HALF_MIRROR>(y[i], y[(i + 8) % 16], l.lane & 4);
                v += dpp<QUAD_XOR1>(v);
                v += dpp<QUAD_XOR2>(v);
                r[i / 4][i % 4] = v;
            }
            if ((l.lane & 3) == 0) {
                float* to = &ys[l.c][q];
                if constexpr (Sh::LPC == 16) {
                    *reinterpret_cast<f32x4*>(to + (l.lane & 12)) = r[0];
                } else {
                    *reinterpret_cast<f32x4*>(to + 2 * (l.lane & 4)) = r[0];
                    *reinterpret_cast<f32x4*>(to + 2 * (l.lane & 4) + 4) = r[1];
                }
            }
        }
        lds_barrier();
        wait_for_loads();
        const rsrc_t out = ro.tile(t0, pc.end, a.D);
#pragma unroll
        for (int i = 0; i < Rw::NV; ++i) {
            if (!cv_ok) continue;
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ys[4 * cv + j][Rw::row(i)];
            v += skip * Four<T>::wide(own_u[i]);
            if (a.gate) {
                const f32x4 g = Four<T>::wide(own_gate[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] *= g[j] * sigmoid1(g[j]);
            }
            buffer_store4<T>(out, ro.lane, ro.bytes(i), v);
        }
    }
    if (a.s_out && pc.end == pc.seq.len && l.mine) {
        const int64_t page = page_of(a.out_pages, a.n_pages, pc.unit);
        if (page >= 0) store_states(a.s_out + page * page_size + l.at, h, l.STEP);
    }
}

// A segment's own state, entered with zero, and the sum of its dt; in reverse
// the gradient that it passes on to the token in front of it. The segment that
// nothing follows needs neither.
template <typename T, int S, bool REVERSE>
__global__ __launch_bounds__(Shape<S>::NT, 2) void scan_summary_kernel(ScanArgs a) {
    typedef Shape<S> Sh;
    constexpr int TT = FT;
    typedef Rows<T, Sh, TT> Rw;
    __shared__ f32x4 xs[TT][Sh::CH / 2];             // dt and dt u, or dy, of two channels
    __shared__ f32x4 bc[2 * TT * Sh::SV];

    const int nb = a.G * Sh::blocks(a);
    const Block k = block_of<Sh>(a, blockIdx.x % nb);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    if (pc.none || (REVERSE ? pc.first == 0 : pc.end == pc.seq.len)) return;
    const Lane<S> l(k.ch, k.ch_end);
    const int64_t page_size = (int64_t)a.D * S;
    f32x4 A2[KC], h[KC] = {};
    load_states(A2, a.A + l.at, S);
#pragma unroll
    for (int i = 0; i < KC; ++i) A2[i] *= LOG2E;
    f32x4 sum = {0, 0, 0, 0};                        // of dt, of this thread's channels and rows
    const int cv = threadIdx.x % Sh::V;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    const f32x4 bias = load_f4(a.dt_bias, cch);

    const Rw rx(REVERSE ? a.dout : a.u, pc.seq.start, REVERSE ? a.D : a.u_stride, cch),
        rt(a.dt, pc.seq.start, a.dt_stride, cch), rg(a.gate, pc.seq.start, a.gate_stride, cch);
    typename Four<T>::raw u[Rw::NV], dt[Rw::NV], gate[Rw::NV] = {};
    States<T, Sh, TT> st;
    const int tiles = (pc.end - pc.first + TT - 1) / TT;
    auto first_of = [&](int i) { return pc.first + (REVERSE ? tiles - 1 - i : i) * TT; };
    auto load = [&](int t0) {
        rx.load(u, t0, pc.end, a.D);
        rt.load(dt, t0, pc.end, a.D);
        if (REVERSE && a.gate) rg.load(gate, t0, pc.end, a.D);
        st.load(a, k.g, pc.seq.start, t0, pc.end);
    };
    load(first_of(0));
    for (int it = 0; it < tiles; ++it) {
        const int t0 = first_of(it);
#pragma unroll
        for (int i = 0; i < Rw::NV; ++i) {
            f32x4 t = step_sizes(Four<T>::wide(dt[i]) + bias, a.softplus);
            if (t0 + Rw::row(i) >= pc.end || !Rw::has(i)) t = f32x4{0, 0, 0, 0};
            sum += t;
            f32x4 x = Four<T>::wide(u[i]);           // zero past the end
            if constexpr (REVERSE) {
                if (a.gate) {
                    const f32x4 g = Four<T>::wide(gate[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] *= g[j] * sigmoid1(g[j]);
                }
            } else {
                x *= t;
            }
            if (Rw::has(i)) {
                xs[Rw::row(i)][2 * cv] = f32x4{t[0], x[0], t[1], x[1]};
                xs[Rw::row(i)][2 * cv + 1] = f32x4{t[2], x[2], t[3], x[3]};
            }
        }
        st.put(bc, t0, pc.end);
        lds_barrier();
        if (it + 1 < tiles) load(first_of(it + 1));
        const int n = (min(TT, pc.end - t0) + 7) & ~7;
        struct Step {
            f32x4 x, b;
        };
        auto read = [&](Step (&s)[4], int q) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = REVERSE ? n - 1 - q - e : q + e;
                s[e] = Step{xs[t][l.c / 2], bc[((REVERSE ? TT : 0) + t) * Sh::SV + l.sl]};
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto step = [&](const Step (&s)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int i = 0; i < KC; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e2 = __builtin_amdgcn_exp2f(s[e].x[2 * i] * A2[i][j]);
                        if constexpr (REVERSE) h[i][j] = e2 * fmaf(s[e].x[2 * i + 1], s[e].b[j], h[i][j]);
                        else h[i][j] = fmaf(e2, h[i][j], s[e].x[2 * i + 1] * s[e].b[j]);
                    }
                }
            }
        };
        Step even[4], odd[4];
        read(even, 0);
#pragma unroll 1
        for (int q = 0; q < n; q += 8) {
            read(odd, q + 4);
            step(even);
            read(even, min(q + 8, n - 4));
            step(odd);
        }
        lds_barrier();
    }
    if (l.mine) {
        store_states(a.slots + piece * page_size + l.at, h, S);
    }
    f32x4* red = &xs[0][0];                          // nobody reads it any more
    static_assert(sizeof(xs) >= Sh::NT * sizeof(f32x4), "");
    red[threadIdx.x] = sum;
    lds_barrier();
    if (threadIdx.x < Sh::V && k.ch + 4 * cv < k.ch_end) {
        for (int i = cv + Sh::V; i < Sh::NT; i += Sh::V) sum += red[i];
        *reinterpret_cast<f32x4*>(a.sums + (int64_t)piece * a.D + cch) = sum;
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
// dB and dC are sums over channels, which lie across lanes. Their terms of four
// tokens (two vectors of four states a lane and token) are added up over lanes 8
// apart, which leaves one vector a lane, and go through LDS, where a lane finds
// one vector's terms of eight channels: 3 operations for each element where
// exchanges of lanes alone take 5 and the matrix unit, which holds up the vector
// units in fp32, 64 cycles (B=2 T=4096 D=4096: 430 us; both vectors through LDS
// 455, exchanges 750, products with ones 670; factors from LDS, in the sums, 470).
template <int S>
struct ChannelSums {
    static constexpr int LPC = S / 4, OUT = 8 * LPC;           // vectors that come out
    static constexpr bool FOLD = LPC < 16;                     // a row of 16 lanes has two channels or more
    static constexpr int SHARE = LPC < 8 ? 8 / LPC : 1;        // lanes of one of them
    static constexpr int ROUNDS = FOLD ? 1 : 2, VECTORS = FOLD ? 1 : 2;   // of a lane and token
    int first, turn;
    // the terms are read in an order that keeps 16 neighbouring lanes on different banks
    __device__ __forceinline__ ChannelSums(int lane) {
        const int o = lane / SHARE, row = o / LPC;
        turn = lane % SHARE;
        first = (FOLD ? row / 2 * 64 + row % 2 * 8 : row * 64) + o % LPC;
    }
    // A token's terms: dB's, added up over pairs of lanes, in the lower halves of
    // the rows, dC's in the upper ones
    static __device__ __forceinline__ void put(f32x4 (&to)[VECTORS][64], f32x4 b, f32x4 c, int lane) {
        if constexpr (FOLD) {
            float v[4] = {b[0], b[1], b[2], b[3]};
            asm("s_nop 1\n" GDN_HALVES("%0", "%4") GDN_HALVES("%1", "%5") GDN_HALVES("%2", "%6") GDN_HALVES("%3", "%7")
                : "+&v"(v[0]), "+&v"(v[1]), "+&v"(v[2]), "+&v"(v[3])
                : "v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]));
            to[0][lane] = f32x4{v[0], v[1], v[2], v[3]};
        } else {
            to[0][lane] = b;
            to[1][lane] = c;
        }
    }
    // p: this wave's vectors [token][VECTORS][lane]; out: [token][dB, dC][S / 4]
    __device__ __forceinline__ void sum(const f32x4* p, f32x4* out, int lane) const {
        constexpr int PER = FOLD ? 8 / LPC : 1;    // terms of a row of lanes
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            f32x4 s = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = turn * 4 + ((i + turn) & 3);
                s += p[first + r * 4 * 64 + k / PER * 16 + k % PER * LPC];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = lane_sum<SHARE>(s[j]);
            out[lane / SHARE + r * 64] = s;
        }
    }
};

template <typename T, int S>
__global__ __launch_bounds__((Shape<S, 1>::NT), 2) void scan_bwd_kernel(ScanArgs a) {
    typedef Shape<S, 1> Sh;
    constexpr int TT = SCAN_KEEP;
    typedef Rows<T, Sh, TT> Rw;
    __shared__ __align__(16) f32x2 xs[TT][Sh::CH];   // dt, dt u
    __shared__ __align__(16) float dys[TT][Sh::CH];
    __shared__ f32x4 bc[2 * TT * Sh::SV];
    __shared__ __align__(16) float sums[3][TT][Sh::CH + 4];   // over states: B g, E h A, C h
    __shared__ f32x4 parts[Sh::NW][TT][2 * Sh::SV];  // over a wave's channels: dB, dC
    __shared__ f32x4 terms[Sh::NW][4][ChannelSums<S>::VECTORS][64];   // of four tokens, by lanes

    const int nb = a.G * Sh::blocks(a), blk = blockIdx.x % nb;
    const Block k = block_of<Sh>(a, blk);
    const int piece = blockIdx.x / nb;
    const Piece pc = piece_of(a.un, piece);
    const Lane<S, 1> l(k.ch, k.ch_end);
    const int64_t page_size = (int64_t)a.D * S;
    // this piece's part of dA, and of dskip and ddt_bias
    float* part = a.a_parts + piece * ((int64_t)a.D * (S + 2));
    const int cv = threadIdx.x % Sh::V;
    const bool cv_ok = k.ch + 4 * cv < k.ch_end;
    const int cch = min(k.ch + 4 * cv, k.ch_end - 4);
    f32x4 dA = {0, 0, 0, 0}, dskip = {0, 0, 0, 0}, dbias = {0, 0, 0, 0};

    if (!pc.none) {
        const f32x4 A2 = *reinterpret_cast<const f32x4*>(a.A + l.at) * LOG2E;
        f32x4 E;
        {
            const f32x4 rate[1] = {A2};
            f32x4 e[1] = {};
            entry_states<true, S, 1>(a, pc, piece, l, rate, e);
            E = e[0];
        }
        const float* keep = a.h + piece_base(a.keep, pc.unit, pc.seq.start) * page_size + l.at;
        const f32x4 bias = load_f4(a.dt_bias, cch), skip = load_f4(a.skip, cch);
        const ChannelSums<S> channels(l.lane);

        const Rw ru(a.u, pc.seq.start, a.u_stride, cch), rt(a.dt, pc.seq.start, a.dt_stride, cch),
            rg(a.gate, pc.seq.start, a.gate_stride, cch), rd(a.dout, pc.seq.start, a.D, cch);
        typename Four<T>::raw u[Rw::NV], dt[Rw::NV], gate[Rw::NV] = {}, dout[Rw::NV];
        States<T, Sh, TT> st;
        f32x4 entry = {0, 0, 0, 0};
        auto load = [&](int t0) {
            ru.load(u, t0, pc.end, a.D);
            rt.load(dt, t0, pc.end, a.D);
            rd.load(dout, t0, pc.end, a.D);
            if (a.gate) rg.load(gate, t0, pc.end, a.D);
            st.load(a, k.g, pc.seq.start, t0, pc.end);
            entry = *reinterpret_cast<const f32x4*>(keep + t0 / TT * page_size);
        };
        const int last = pc.first + (pc.end - pc.first - 1) / TT * TT;
        if (pc.first < pc.end) load(last);
        wait_for_loads();
        for (int t0 = last; t0 >= pc.first && pc.first < pc.end; t0 -= TT) {
            typename Four<T>::raw own_u[Rw::NV], own_dt[Rw::NV], own_gate[Rw::NV], own_dout[Rw::NV];
#pragma unroll
            for (int i = 0; i < Rw::NV; ++i) {
                own_u[i] = u[i];
                own_dt[i] = dt[i];
                own_gate[i] = gate[i];
                own_dout[i] = dout[i];
                f32x4 t = step_sizes(Four<T>::wide(dt[i]) + bias, a.softplus);
                f32x4 dy = Four<T>::wide(dout[i]);   // zero past the end
                if (a.gate) {
                    const f32x4 g = Four<T>::wide(gate[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dy[j] *= g[j] * sigmoid1(g[j]);
                }
                if (t0 + Rw::row(i) >= pc.end || !cv_ok) t = dy = f32x4{0, 0, 0, 0};
                const f32x4 du = t * Four<T>::wide(u[i]);
                if (Rw::has(i)) {
                    const int row = Rw::row(i);
                    *reinterpret_cast<f32x4*>(&xs[row][4 * cv]) = f32x4{t[0], du[0], t[1], du[1]};
                    *reinterpret_cast<f32x4*>(&xs[row][4 * cv + 2]) = f32x4{t[2], du[2], t[3], du[3]};
                    *reinterpret_cast<f32x4*>(&dys[row][4 * cv]) = dy;
                }
            }
            st.put(bc, t0, pc.end);
            const f32x4 h0 = entry;
            lds_barrier();
            if (t0 > pc.first) load(t0 - TT);

            // the states of the tile once more, and the decays
            f32x4 h[TT], ea[TT];
#pragma unroll
            for (int t = 0; t < TT; t += 4) {
                f32x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 x = xs[t + e][l.c];
                    const f32x4 B = bc[(t + e) * Sh::SV + l.sl], C = bc[(TT + t + e) * Sh::SV + l.sl];
                    float s = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ea[t + e][j] = __builtin_amdgcn_exp2f(x[0] * A2[j]);
                        const float now = fmaf(ea[t + e][j], t + e ? h[t + e - 1][j] : h0[j], x[1] * B[j]);
                        h[t + e][j] = now;
                        s = j ? fmaf(C[j], now, s) : C[j] * now;
                    }
                    y[e] = s;
                }
                const f32x2 r = four_sums<Sh::LPC>(y, l.lane);
                sums[2][t + (l.lane & (Sh::LPC == 2 ? 1 : 3))][l.c] = r[0];
                if constexpr (Sh::LPC == 2) sums[2][t + 2 + l.sl][l.c] = r[1];
                __builtin_amdgcn_sched_barrier(0);
            }
            // and their gradients, backwards
#pragma unroll
            for (int t = TT - 4; t >= 0; t -= 4) {
                f32x4 su, sa;
#pragma unroll
                for (int e = 3; e >= 0; --e) {
                    const int n = t + e;
                    const f32x2 x = xs[n][l.c];
                    const float dy = dys[n][l.c];
                    const f32x4 B = bc[n * Sh::SV + l.sl], C = bc[(TT + n) * Sh::SV + l.sl];
                    f32x4 pb, pcv;
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float g = fmaf(C[j], dy, E[j]);
                        pb[j] = x[1] * g;
                        pcv[j] = dy * h[n][j];
                        s0 = j ? fmaf(B[j], g, s0) : B[j] * g;
                        E[j] = ea[n][j] * g;
                        const float w = E[j] * (n ? h[n - 1][j] : h0[j]);
                        s1 = j ? fmaf(w, A2[j], s1) : w * A2[j];
                        dA[j] = fmaf(w, x[0], dA[j]);
                    }
                    channels.put(terms[l.wave][e], pb, pcv, l.lane);
                    su[e] = s0;
                    sa[e] = s1;
                }
                asm volatile("" : "+v"(dA));         // else added up at the tile's end, its terms in registers until then
                __builtin_amdgcn_wave_barrier();     // a wave's LDS accesses keep their order
                channels.sum(&terms[l.wave][0][0][0], &parts[l.wave][t][0], l.lane);
                __builtin_amdgcn_wave_barrier();
                const f32x2 r0 = four_sums<Sh::LPC>(su, l.lane), r1 = four_sums<Sh::LPC>(sa, l.lane);
                sums[0][t + (l.lane & (Sh::LPC == 2 ? 1 : 3))][l.c] = r0[0];
                sums[1][t + (l.lane & (Sh::LPC == 2 ? 1 : 3))][l.c] = r1[0];
                if constexpr (Sh::LPC == 2) {
                    sums[0][t + 2 + l.sl][l.c] = r0[1];
                    sums[1][t + 2 + l.sl][l.c] = r1[1];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            lds_barrier();
            wait_for_loads();
            // dB and dC of this workgroup's channels
            const int n = min(TT, pc.end - t0);
            for (int i = threadIdx.x; i < n * 2 * Sh::SV; i += Sh::NT) {
                const f32x4* p = &parts[0][0][0] + i;
                constexpr int W = TT * 2 * Sh::SV;
                f32x4 r = p[0] + p[W];
                if constexpr (Sh::NW == 4) r += p[2 * W] + p[3 * W];
                reinterpret_cast<f32x4*>(a.bc_parts + ((int64_t)blk * a.un.total + pc.seq.start + t0) * (2 * S))[i] = r;
            }
            const Rw ro(a.du, pc.seq.start, a.D, cch);
            const rsrc_t du_out = ro.tile(t0, pc.end, a.D), ddt_out = Rw(a.ddt, pc.seq.start, a.D, cch).tile(t0, pc.end, a.D),
                         dgate_out = Rw(a.dgate, pc.seq.start, a.D, cch).tile(t0, pc.end, a.D);
#pragma unroll
            for (int i = 0; i < Rw::NV; ++i) {
                const int row = Rw::row(i);
                if (!Rw::has(i) || !cv_ok) continue;
                const f32x4 uu = Four<T>::wide(own_u[i]);    // zero past the end, as are dt, dy and dout
                const f32x4 x0 = *reinterpret_cast<const f32x4*>(&xs[row][4 * cv]),
                            x1 = *reinterpret_cast<const f32x4*>(&xs[row][4 * cv + 2]), t = {x0[0], x0[2], x1[0], x1[2]};
                const f32x4 dy = *reinterpret_cast<const f32x4*>(&dys[row][4 * cv]);
                const f32x4 gu = *reinterpret_cast<const f32x4*>(&sums[0][row][4 * cv]);
                const f32x4 gt = *reinterpret_cast<const f32x4*>(&sums[1][row][4 * cv]) * LN2;
                f32x4 ddt = gu * uu + gt;
                if (a.softplus) {
                    const f32x4 raw = Four<T>::wide(own_dt[i]) + bias;
#pragma unroll
                    for (int j = 0; j < 4; ++j) ddt[j] *= sigmoid1(raw[j]);
                }
                buffer_store4<T>(du_out, ro.lane, ro.bytes(i), t * gu + skip * dy);
                buffer_store4<T>(ddt_out, ro.lane, ro.bytes(i), ddt);
                dskip += dy * uu;
                if (t0 + row < pc.end) dbias += ddt;
                if (a.gate) {
                    const f32x4 g = Four<T>::wide(own_gate[i]), d = Four<T>::wide(own_dout[i]);
                    f32x4 y = *reinterpret_cast<const f32x4*>(&sums[2][row][4 * cv]) + skip * uu;
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] *= d[j] * silu_slope(g[j], sigmoid1(g[j]));
                    buffer_store4<T>(dgate_out, ro.lane, ro.bytes(i), y);
                }
            }
            lds_barrier();
        }
        if (a.s_out && pc.first == 0 && l.mine) *reinterpret_cast<f32x4*>(a.s_out + pc.unit * page_size + l.at) = E;
    }
    // this piece's sums over its tokens
    if (l.mine) *reinterpret_cast<f32x4*>(part + l.at) = dA;
    lds_barrier();
    typedef f32x4 Red[Sh::NT];
    float* room = S == 64 ? reinterpret_cast<float*>(&parts[0][0][0]) : &sums[0][0][0];
    Red* red = reinterpret_cast<Red*>(room);
    static_assert((S == 64 ? sizeof(parts) : sizeof(sums)) >= sizeof(Red), "");
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        red[0][threadIdx.x] = which ? dbias : dskip;
        lds_barrier();
        if (threadIdx.x < Sh::V && cv_ok) {
            f32x4 s = red[0][cv];
            for (int i = cv + Sh::V; i < Sh::NT; i += Sh::V) s += red[0][i];
            *reinterpret_cast<f32x4*>(part + page_size + which * a.D + cch) = s;
        }
        lds_barrier();
    }
}

// dB and dC: sums over the workgroups of a group's channels, four values a
// thread. The workgroups behind those add up the rows of dA, dskip and ddt_bias
// where these are few.
template <typename T>
__global__ __launch_bounds__(NT) void scan_bc_kernel(ScanArgs a, int blocks, unsigned bc_groups, RowSums out, unsigned cols) {
    if (blockIdx.x >= bc_groups) {
        sum_rows(a.a_parts, a.un.n_pieces, (int64_t)a.D * (a.S + 2), out, a.un.n_pieces, cols, blockIdx.x - bc_groups);
        return;
    }
    const int per = 2 * a.S / 4;
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x, rows = i / per;
    if (rows >= a.un.total * a.G) return;
    const int64_t t = rows / a.G;
    const int g = (int)(rows % a.G), v = (int)(i % per);
    const f32x4* p = reinterpret_cast<const f32x4*>(a.bc_parts) + ((int64_t)g * blocks * a.un.total + t) * per + v;
    const int64_t step = a.un.total * per;
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) s += p[b * step];
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

// Bound by the bytes of the states, read once and written once (256 sequences of
// D=8192 55 us, 5.2 TB/s); a thread holds four values of the state of N sequences.
// AROUND: past the caches
template <typename T, int S, int N, bool AROUND>
__global__ __launch_bounds__(NT) void scan_step_kernel(ScanArgs a) {
    constexpr int LPC = S / 4;
    const int per = (a.D * LPC + NT - 1) / NT;
    const int n0 = blockIdx.x / per * N, e = (blockIdx.x % per) * NT + threadIdx.x;
    const bool ok = e < a.D * LPC;
    const int d = ok ? e / LPC : a.D - 1, sl = e % LPC, g = d / (a.D / a.G);
    T* out = static_cast<T*>(a.out) + (int64_t)n0 * a.D + d;
    f32x4* at[N];
    f32x4 h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t page = n0 + i < a.un.n_units ? page_of(a.in_pages, a.n_pages, n0 + i) : -1;
        at[i] = page < 0 || page >= a.n_pages ? nullptr
                                              : reinterpret_cast<f32x4*>(a.s_out + (page * a.D + d) * S + 4 * sl);
        if (at[i]) h[i] = AROUND ? __builtin_nontemporal_load(at[i]) : *at[i];
    }
    const f32x4 A = *reinterpret_cast<const f32x4*>(a.A + (int64_t)d * S + 4 * sl);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int n = n0 + i;
        if (n >= a.un.n_units) break;
        if (!at[i]) {
            if (ok && sl == 0) out[(int64_t)i * a.D] = (T)0.0f;
            continue;
        }
        const f32x4 B = Four<T>::wide(load4(static_cast<const T*>(a.b) + n * a.b_stride[0] + g * a.b_stride[1] + 4 * sl));
        const f32x4 C = Four<T>::wide(load4(static_cast<const T*>(a.c) + n * a.c_stride[0] + g * a.c_stride[1] + 4 * sl));
        const float u = (float)static_cast<const T*>(a.u)[n * a.u_stride + d];
        float dt = (float)static_cast<const T*>(a.dt)[n * a.dt_stride + d] + bias;
        const float gate = a.gate ? (float)static_cast<const T*>(a.gate)[n * a.gate_stride + d] : 0.0f;
        if (a.softplus) dt = softplus1(dt);
        const float du = dt * u;
        float y = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[i][j] = fmaf(du, B[j], decayed(h[i][j], dt * A[j]));
            y = fmaf(C[j], h[i][j], y);
        }
        if (ok) {
            if constexpr (AROUND) __builtin_nontemporal_store(h[i], at[i]);
            else *at[i] = h[i];
        }
        y = lane_sum<LPC>(y) + skip * u;
        if (a.gate) y *= gate * sigmoid1(gate);
        if (ok && sl == 0) out[(int64_t)i * a.D] = (T)y;
    }
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

template <typename Sh>
unsigned grid_of(const ScanArgs& a) {
    return (unsigned)((int64_t)a.un.n_pieces * a.G * Sh::blocks(a));
}

}  // namespace

hipError_t launch_scan_summary(const ScanArgs& a, bool reverse, hipStream_t s) {
    return by_type(a.dtype, a.S, [&](auto t, auto n) {
        typedef Shape<n()> Sh;
        if (reverse) scan_summary_kernel<decltype(t), n(), true><<<grid_of<Sh>(a), Sh::NT, 0, s>>>(a);
        else scan_summary_kernel<decltype(t), n(), false><<<grid_of<Sh>(a), Sh::NT, 0, s>>>(a);
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
    return by_type(a.dtype, a.S, [&](auto t, auto n) {
        typedef Shape<n(), 2> Two;
        typedef Shape<n(), 1> One;
        typedef Narrow<n()> Few;
        // Fewer workgroups than two a compute unit hold half the channels each, which
        // are then twice as many (B=8 T=1000 D=4096, 256 of them, 183 to 156 us; 512 of
        // them 266 and 289).
        if (a.narrow) scan_narrow_kernel<decltype(t), n()><<<grid_of<Few>(a), Few::NT, 0, s>>>(a);
        else if (grid_of<Two>(a) >= 512) scan_fwd_kernel<decltype(t), n(), 2><<<grid_of<Two>(a), Two::NT, 0, s>>>(a);
        else scan_fwd_kernel<decltype(t), n(), 1><<<grid_of<One>(a), One::NT, 0, s>>>(a);
    });
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t s) {
    const hipError_t e = by_type(a.dtype, a.S, [&](auto t, auto n) {
        typedef Shape<n(), 1> Sh;
        scan_bwd_kernel<decltype(t), n()><<<grid_of<Sh>(a), Sh::NT, 0, s>>>(a);
    });
    if (e != hipSuccess) return e;
    const int64_t d = a.D, n = d * (a.S + 2);
    const RowSums out{{a.dA, a.dskip, a.ddt_bias}, {d * a.S, d, d}};
    const bool few = scan_sums_together(a.un.n_pieces);
    const unsigned bc = (unsigned)scan_bc_workgroups(a.un.total, a.G, a.S), cols = (unsigned)((n + 63) / 64);
    const unsigned grid = (unsigned)scan_sum_workgroups(a.un.total, a.un.n_pieces, a.G, a.D, a.S);
    if (grid > 0) {
        if (a.dtype == GDN_DTYPE_BF16) scan_bc_kernel<bf16><<<grid, NT, 0, s>>>(a, a.bwd_blocks, bc, out, cols);
        else scan_bc_kernel<float><<<grid, NT, 0, s>>>(a, a.bwd_blocks, bc, out, cols);
    }
    return few ? hipGetLastError() : launch_row_sums(a.a_parts, a.un.n_pieces, n, out, s);
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t s) {
    const int64_t n_seq = a.un.n_units;
    if (n_seq == 0) return hipSuccess;
    const int64_t blocks = ((int64_t)a.D * (a.S / 4) + NT - 1) / NT;
    const int64_t bytes = n_seq * a.D * a.S * 4;
    // Many sequences, four to a workgroup, which then read A once (512 of D=8192
    // one by one 117 us, four 107, eight 123).
    constexpr int ROWS = 4;
    return by_type(a.dtype, a.S, [&](auto t, auto n) {
        if (bytes >= MX_AROUND_BYTES)
            scan_step_kernel<decltype(t), n(), ROWS, true><<<(unsigned)((n_seq + ROWS - 1) / ROWS * blocks), NT, 0, s>>>(a);
        else if (n_seq * blocks >= 8192)
            scan_step_kernel<decltype(t), n(), ROWS, false><<<(unsigned)((n_seq + ROWS - 1) / ROWS * blocks), NT, 0, s>>>(a);
        else
            scan_step_kernel<decltype(t), n(), 1, false><<<(unsigned)(n_seq * blocks), NT, 0, s>>>(a);
    });
}

}  // namespace gdn
