// Linear attention with a decay for each head, over whole prompts.
//
// A sequence is cut into chunks of C tokens. With S the state entering a
// chunk, d the head's decay and positions i, j inside the chunk,
//     o_i = sum_{j <= i} d^{i-j} (q_i . k_j) v_j + d^{i+1} q_i S
//     S  <- d^C S + sum_j d^{C-1-j} k_j v_j^T
// so a chunk is four matrix products. A workgroup walks the chunks of one
// segment of one head: each of its four waves keeps a quarter of S's value
// columns in MFMA accumulators for the whole walk, and those registers are at
// once the operand of q S (an accumulator tile and an operand hold the same
// elements if the contraction's order is chosen to match). Long sequences
// with too few heads to fill the GPU are cut into segments: a first pass sums
// each segment's own k v^T, a merge makes them the states that enter, and the
// walk then runs on all segments at once.
//
// Products of bf16 inputs: bf16 MFMA, fp32 accumulation. Where a value
// computed in fp32 meets a bf16 operand it is split into bf16 terms, not
// rounded: two terms (16 bits) for the scores and for S in q S, whose result
// is rounded to the output's type, three (24 bits) for the decayed v that
// enters S, which is carried over the whole sequence and returned in fp32.
// fp32 inputs: fp32 MFMA.
//
// A partial chunk fills the last rows of its tile, with zero rows before
// them: the factors that enter S then stay those of a full chunk, and only
// d^{i+1} and d^C change.
#include "gdn_device.h"
#include "gdn_recurrent_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;
constexpr int NXCD = 8;

typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// d^n of a log decay g, in fp64: n runs over whole sequences, and the error
// of an fp32 exponent (n g) 2^-24 would show in the states. n = 0 gives 1 for
// g = -inf too.
__device__ __forceinline__ double dpow(double g, int64_t n) { return n == 0 ? 1.0 : exp((double)n * g); }

// x d^n with d^n held in two terms, so that a factor applied once a chunk
// over a long sequence does not add its own rounding up
struct Factor {
    float hi, lo;
    __device__ explicit Factor(double x) : hi((float)x), lo((float)(x - (double)(float)x)) {}
    __device__ __forceinline__ f32x4 operator*(f32x4 x) const {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(x[i], hi, x[i] * lo);
        return y;
    }
};

// Workgroups are handed to the XCDs in turn: gives each XCD a contiguous
// range of the work, so that workgroups reading the same rows share an L2.
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int x = b % NXCD, i = b / NXCD, per = n / NXCD, rem = n % NXCD;
    return x * per + (x < rem ? x : rem) + i;
}

struct Seg {
    int unit, index, count;   // the segment's place in its unit
    int64_t start;            // the unit's first token
    int len;                  // the unit's tokens
};

__device__ __forceinline__ int segs_of(int len, int seg_tokens) {
    return len > 0 ? (len + seg_tokens - 1) / seg_tokens : 1;
}

__device__ __forceinline__ void unit_range(const LaUnits& um, int u, int64_t& start, int& len) {
    int64_t a = um.offsets[u], b = um.offsets[u + 1];
    a = a < 0 ? 0 : (a > um.total ? um.total : a);
    b = b < a ? a : (b > um.total ? um.total : b);
    start = a;
    len = (int)(b - a);
}

// The segment of a flat index: units in order, each with its segments. unit
// is -1 beyond the last.
__device__ Seg find_seg(const LaUnits& um, int id) {
    Seg s;
    if (um.dense) {
        s.count = segs_of(um.T, um.seg_tokens);
        s.unit = id / s.count;
        s.index = id - s.unit * s.count;
        s.start = (int64_t)s.unit * um.T;
        s.len = um.T;
        if (s.unit >= um.n_units) s.unit = -1;
        return s;
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    s.unit = -1;
    for (int u0 = 0; u0 < um.n_units; u0 += 64) {
        int64_t start = 0;
        int len = 0, ns = 0;
        if (u0 + lane < um.n_units) {
            unit_range(um, u0 + lane, start, len);
            ns = segs_of(len, um.seg_tokens);
        }
        int inc = ns;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int y = __shfl_up(inc, m);
            if (lane >= m) inc += y;
        }
        const uint64_t after = __ballot(id < base + inc);
        if (after) {
            const int at = __ffsll((unsigned long long)after) - 1;
            s.unit = u0 + at;
            s.count = __builtin_amdgcn_readfirstlane(__shfl(ns, at));
            s.index = __builtin_amdgcn_readfirstlane(id - base - __shfl(inc - ns, at));
            s.len = __builtin_amdgcn_readfirstlane(__shfl(len, at));
            const uint32_t lo = __builtin_amdgcn_readfirstlane(__shfl((uint32_t)start, at));
            const uint32_t hi = __builtin_amdgcn_readfirstlane(__shfl((uint32_t)(start >> 32), at));
            s.start = (int64_t)(((uint64_t)hi << 32) | lo);
            return s;
        }
        base += __shfl(inc, 63);
    }
    return s;
}

__device__ __forceinline__ int page_of(const int32_t* pages, int unit, int n_pages) {
    if (!pages) return unit;
    const int p = pages[unit];
    return p >= 0 && p < n_pages ? p : -1;
}

// ------------------------------------------------------------------ tiles
// C rows of W elements in LDS in 16-byte units, a row's units exchanged by
// an XOR with the row number: 16 rows read at one column, and 4 rows read
// across, both spread over the banks.
template <typename T, int W>
struct Tile {
    static constexpr int EPU = 16 / sizeof(T);
    static constexpr int UNITS = W / EPU;
    static constexpr int MASK = (UNITS < 16 ? UNITS : 16) - 1;
    __device__ static __forceinline__ int at(int row, int unit) { return row * W + (unit ^ (row & MASK)) * EPU; }
    // element offset of (row, col); col's unit is swizzled, its place in the unit kept
    __device__ static __forceinline__ int el(int row, int col) { return at(row, col / EPU) + col % EPU; }
};

// One chunk of one tensor on its way from memory to its tile: each thread
// carries rows r0, r0 + STEP, ...
template <typename T, int W, int C>
struct Carrier {
    using TL = Tile<T, W>;
    static constexpr int STEP = NT / TL::UNITS;
    static constexpr int N = C / STEP;
    static_assert(N >= 1, "");
    u32x4 x[N];

    // tt0: time of tile row 0 (negative rows of a partial chunk stay zero)
    __device__ __forceinline__ void load(const RowsOf& r, int h, int64_t start, int len, int rev, int tt0, int shift) {
        const int row0 = threadIdx.x / TL::UNITS, unit = threadIdx.x % TL::UNITS;
        const int64_t t = (int64_t)tt0 + row0;
        const int64_t tok = rev ? start + len - 1 - t : start + t;
        const T* p = static_cast<const T*>(r.p) + tok * r.ts + (int64_t)(h / r.share) * r.hs + unit * TL::EPU;
        const int64_t step = (rev ? -STEP : STEP) * r.ts;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = u32x4{0, 0, 0, 0};
            if (row0 + i * STEP >= shift) x[i] = *reinterpret_cast<const u32x4*>(p + i * step);
        }
    }
    __device__ __forceinline__ void store(T* tile) const {
        const int row0 = threadIdx.x / TL::UNITS, unit = threadIdx.x % TL::UNITS;
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + TL::at(row0 + i * STEP, unit)) = x[i];
    }
};

// ------------------------------------------------------------------ operands
// Lane p + 16 g of a 16 x 16 x 32 bf16 product holds row (column) p and the
// contraction indices 8 g .. 8 g + 7; of a 16 x 16 x 4 fp32 product row p and
// index g, where four products take the indices 4 g .. 4 g + 3 in turn. The
// result's lane holds column p, rows 4 g .. 4 g + 3.
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

// 4 x 16 bf16 read across: lane p gets column p of the four rows
__device__ __forceinline__ s16x4 read_across(const bf16* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, p));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ bf16x8 top(f32x8 x) { return __builtin_convertvector(x, bf16x8); }
__device__ __forceinline__ f32x8 rest(f32x8 x, bf16x8 t) { return x - __builtin_convertvector(t, f32x8); }

template <typename T>
struct Shape;
template <>
struct Shape<bf16> {
    static constexpr int C = 64;    // tokens per chunk
    static constexpr int KS = 32;   // contraction of one operand
};
template <>
struct Shape<float> {
    static constexpr int C = 32;
    static constexpr int KS = 16;
};

// ------------------------------------------------------------------ the state
// A wave's part of S: CG groups of 16 value columns, KD / 16 tiles of 16 keys.
// bf16: row m of tile 2 t + u is key 32 t + 8 (m / 4) + 4 u + m % 4, so that
// tiles 2 t and 2 t + 1 hold, in each lane, the eight consecutive keys of an
// operand; fp32: row m of tile t is key 16 t + m.
template <typename T, int KD, int VD>
struct State {
    static constexpr int KT = KD / 16, CG = VD / 64;
    f32x4 s[KT][CG];

    __device__ static __forceinline__ int key0(int kt, int g) {   // of the lane's four rows
        if constexpr (sizeof(T) == 2) return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1);
        return 16 * kt + 4 * g;
    }
    __device__ static __forceinline__ int col(int cg) {
        return (threadIdx.x >> 6) * (VD / 4) + 16 * cg + (threadIdx.x & 15);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) s[kt][cg] = f32x4{0, 0, 0, 0};
    }
    __device__ void load(const float* p, int transposed) {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) {
                if (transposed) {
                    s[kt][cg] = *reinterpret_cast<const f32x4*>(p + col(cg) * KD + key0(kt, g));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[kt][cg][r] = p[(key0(kt, g) + r) * VD + col(cg)];
                }
            }
    }
    __device__ void store(float* p) const {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg)
#pragma unroll
                for (int r = 0; r < 4; ++r) p[(key0(kt, g) + r) * VD + col(cg)] = s[kt][cg][r];
    }
    __device__ __forceinline__ void scale(const Factor& f) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) s[kt][cg] = f * s[kt][cg];
    }
};

// A wave's columns of v as operands, rows of 32 (16) tokens each.
template <typename T, int VD>
struct ValueFrags;
template <int VD>
struct ValueFrags<bf16, VD> {
    static constexpr int CG = VD / 64, NS = 2;
    bf16x8 f[NS][CG];
    __device__ __forceinline__ void load(const bf16* tile) {
        const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4, w = threadIdx.x >> 6;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) {
                const int row = 32 * s + 8 * g + (p >> 2), c = w * (VD / 4) + 16 * cg + 4 * (p & 3);
                f[s][cg] = join(read_across(tile + Tile<bf16, VD>::el(row, c)),
                                read_across(tile + Tile<bf16, VD>::el(row + 4, c)));
            }
    }
};
template <int VD>
struct ValueFrags<float, VD> {
    static constexpr int CG = VD / 64, NS = 2;
    f32x4 f[NS][CG];
    __device__ __forceinline__ void load(const float* tile) {
        const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4, w = threadIdx.x >> 6;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    f[s][cg][r] = tile[Tile<float, VD>::el(16 * s + 4 * g + r, w * (VD / 4) + 16 * cg + p)];
    }
};

// S += sum_j wt[j] k_j v_j^T over a chunk
template <int KD, int VD>
__device__ __forceinline__ void add_outer(State<bf16, KD, VD>& st, const bf16* kt_, const ValueFrags<bf16, VD>& v,
                                          const float* wt) {
    const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    constexpr int CG = VD / 64;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const f32x8 w = *reinterpret_cast<const f32x8*>(wt + 32 * s + 8 * g);
        bf16x8 b[CG][3];
#pragma unroll
        for (int cg = 0; cg < CG; ++cg) {
            f32x8 x = w * __builtin_convertvector(v.f[s][cg], f32x8);
            b[cg][0] = top(x);
            x = rest(x, b[cg][0]);
            b[cg][1] = top(x);
            b[cg][2] = top(rest(x, b[cg][1]));
        }
        const int row = 32 * s + 8 * g + (p >> 2);
#pragma unroll
        for (int kt = 0; kt < KD / 16; ++kt) {
            const int c = 32 * (kt >> 1) + 8 * (p & 3) + 4 * (kt & 1);
            const bf16x8 a = join(read_across(kt_ + Tile<bf16, KD>::el(row, c)),
                                  read_across(kt_ + Tile<bf16, KD>::el(row + 4, c)));
#pragma unroll
            for (int cg = 0; cg < CG; ++cg)
#pragma unroll
                for (int x = 0; x < 3; ++x) st.s[kt][cg] = mfma(a, b[cg][x], st.s[kt][cg]);
        }
    }
}
template <int KD, int VD>
__device__ __forceinline__ void add_outer(State<float, KD, VD>& st, const float* kt_, const ValueFrags<float, VD>& v,
                                          const float* wt) {
    const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    constexpr int CG = VD / 64;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(wt + 16 * s + 4 * g);
        f32x4 b[CG];
#pragma unroll
        for (int cg = 0; cg < CG; ++cg) b[cg] = w * v.f[s][cg];
#pragma unroll
        for (int kt = 0; kt < KD / 16; ++kt) {
            f32x4 a;
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = kt_[Tile<float, KD>::el(16 * s + 4 * g + r, 16 * kt + p)];
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) st.s[kt][cg] = mfma(a, b[cg], st.s[kt][cg]);
        }
    }
}

// row `16 it + p` of a tile as an operand, contraction block t
template <int W>
__device__ __forceinline__ bf16x8 row_frag(const bf16* tile, int it, int t) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const bf16x8*>(tile + Tile<bf16, W>::at(16 * it + (lane & 15), 4 * t + (lane >> 4)));
}
template <int W>
__device__ __forceinline__ f32x4 row_frag(const float* tile, int it, int t) {
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const f32x4*>(tile + Tile<float, W>::at(16 * it + (lane & 15), 4 * t + (lane >> 4)));
}

// ------------------------------------------------------------------ kernels
template <typename T, int KD, int VD>
__global__ __launch_bounds__(NT, 2) void la_main(LaUnits um, LaJobs jobs) {
    constexpr int C = Shape<T>::C, KS = Shape<T>::KS, IT = C / 16, CG = VD / 64;
    constexpr bool BF = sizeof(T) == 2;
    __shared__ __attribute__((aligned(16))) T qt[C * KD];
    __shared__ __attribute__((aligned(16))) T kt[C * KD];
    __shared__ __attribute__((aligned(16))) T vt[C * VD];
    __shared__ __attribute__((aligned(16))) T pt[BF ? 2 : 1][C * C];   // scores; bf16: in two terms
    __shared__ __attribute__((aligned(32))) float wt[C];
    __shared__ float pw[2 * C], rf[C];
    using PT = Tile<T, C>;

    const int tid = threadIdx.x, lane = tid & 63, p = lane & 15, g = lane >> 4, wave = tid >> 6;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    const LaJob& jb = jobs.job[id % jobs.n];
    const int h = (id / jobs.n) % um.H, seg_id = id / jobs.n / um.H;
    const Seg sg = find_seg(um, seg_id);
    if (sg.unit < 0) return;
    const int seg0 = sg.index * um.seg_tokens;
    const int seg1 = min(sg.len, seg0 + um.seg_tokens);
    const int nch = seg1 > seg0 ? (seg1 - seg0 + C - 1) / C : 0;

    Carrier<T, KD, C> cq, ck;
    Carrier<T, VD, C> cv;
    auto fetch = [&](int c) {
        const int t0 = seg0 + c * C, shift = max(0, C - (seg1 - t0));
        cq.load(jb.q, h, sg.start, sg.len, jb.rev, t0 - shift, shift);
        ck.load(jb.k, h, sg.start, sg.len, jb.rev, t0 - shift, shift);
        cv.load(jb.v, h, sg.start, sg.len, jb.rev, t0 - shift, shift);
    };
    auto stage = [&]() {
        cq.store(qt);
        ck.store(kt);
        cv.store(vt);
    };
    if (nch > 0) fetch(0);

    State<T, KD, VD> st;
    const double gd = um.decay[h];
    {
        const float* from = nullptr;
        if (jb.slots) {
            from = jb.slots + ((int64_t)seg_id * um.H + h) * (KD * VD);
        } else if (jb.s_in) {
            const int page = page_of(jb.in_pages, sg.unit, um.n_pages);
            if (page >= 0) from = jb.s_in + ((int64_t)page * um.H + h) * (KD * VD);
        }
        if (from) st.load(from, jb.transposed);
        else st.zero();
    }
    for (int i = tid; i < 2 * C; i += NT) pw[i] = i < C ? 0.0f : (float)(jb.s_p * dpow(gd, i - C));
    if (tid < C) {
        wt[tid] = (float)(jb.s_w * dpow(gd, C - jb.e - tid));
        rf[tid] = (float)(jb.s_o * dpow(gd, tid + jb.e));
    }
    // score tiles above the diagonal that an operand reaches stay zero
    for (int i = tid; i < (BF ? 2 : 1) * C * C / PT::EPU; i += NT)
        reinterpret_cast<u32x4*>(&pt[0][0])[i] = u32x4{0, 0, 0, 0};
    const Factor full(dpow(gd, C));
    if (nch > 0) stage();
    lds_barrier();

    for (int c = 0; c < nch; ++c) {
        const int t0 = seg0 + c * C, L = min(C, seg1 - t0), shift = C - L;
        if (c + 1 < nch) fetch(c + 1);
        if (L < C) {   // the last chunk of a unit
            if (tid < C) rf[tid] = tid < shift ? 0.0f : (float)(jb.s_o * dpow(gd, tid - shift + jb.e));
            lds_barrier();
        }

        // scores of the lower triangle, transposed: tile n of the list for wave n % 4
        constexpr int TILES = IT * (IT + 1) / 2;
#pragma unroll
        for (int n0 = 0; n0 < TILES; n0 += 4) {
            const int n = n0 + wave;
            if (n < TILES) {
                const int it = BF ? (n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0) : (n >= 1 ? 1 : 0);
                const int jt = n - it * (it + 1) / 2;
                f32x4 acc = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < KD / KS; ++t) acc = mfma(row_frag<KD>(kt, jt, t), row_frag<KD>(qt, it, t), acc);
                const int gap = 16 * (it - jt) + p - 4 * g;
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] *= pw[C + gap - r];
                const int at = PT::el(16 * it + p, 16 * jt + 4 * g);
                if constexpr (BF) {
                    const bf16x4 hi = __builtin_convertvector(acc, bf16x4);
                    *reinterpret_cast<bf16x4*>(&pt[0][at]) = hi;
                    *reinterpret_cast<bf16x4*>(&pt[1][at]) =
                        __builtin_convertvector(acc - __builtin_convertvector(hi, f32x4), bf16x4);
                } else {
                    *reinterpret_cast<f32x4*>(&pt[0][at]) = acc;
                }
            }
        }

        ValueFrags<T, VD> vf;
        vf.load(vt);

        // o^T = (q S)^T, rows scaled by their distance from the chunk's start
        f32x4 o[IT][CG];
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) o[it][cg] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < KD / KS; ++t) {
            if constexpr (BF) {
                bf16x8 hi[CG], lo[CG];
#pragma unroll
                for (int cg = 0; cg < CG; ++cg) {
                    const f32x8 x = __builtin_shufflevector(st.s[2 * t][cg], st.s[2 * t + 1][cg], 0, 1, 2, 3, 4, 5, 6, 7);
                    hi[cg] = top(x);
                    lo[cg] = top(rest(x, hi[cg]));
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const bf16x8 b = row_frag<KD>(qt, it, t);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) {
                        o[it][cg] = mfma(hi[cg], b, o[it][cg]);
                        o[it][cg] = mfma(lo[cg], b, o[it][cg]);
                    }
                }
            } else {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const f32x4 b = row_frag<KD>(qt, it, t);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(st.s[t][cg], b, o[it][cg]);
                }
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const float f = rf[16 * it + p];
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) o[it][cg] *= f;
        }

        if (L < C) st.scale(Factor(dpow(gd, L)));
        else st.scale(full);
        add_outer<KD, VD>(st, kt, vf, wt);

        lds_barrier();   // scores written, tiles read
        if (c + 1 < nch) stage();
#pragma unroll
        for (int it = 0; it < IT; ++it) {
#pragma unroll
            for (int s = 0; s <= (it * 16) / KS; ++s) {
                if constexpr (BF) {
                    const bf16x8 hi = row_frag<C>(pt[0], it, s), lo = row_frag<C>(pt[1], it, s);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) {
                        o[it][cg] = mfma(vf.f[s][cg], hi, o[it][cg]);
                        o[it][cg] = mfma(vf.f[s][cg], lo, o[it][cg]);
                    }
                } else {
                    const f32x4 b = row_frag<C>(pt[0], it, s);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(vf.f[s][cg], b, o[it][cg]);
                }
            }
            const int row = 16 * it + p;
            if (row >= shift) {
                const int64_t t = (int64_t)t0 + row - shift;
                const int64_t tok = jb.rev ? sg.start + sg.len - 1 - t : sg.start + t;
                const int64_t at = (tok * um.H + h) * VD + wave * (VD / 4) + 4 * g;
#pragma unroll
                for (int cg = 0; cg < CG; ++cg) {
                    if (jb.o_f32)
                        *reinterpret_cast<f32x4*>(static_cast<float*>(jb.o) + at + 16 * cg) = o[it][cg];
                    else
                        *reinterpret_cast<bf16x4*>(static_cast<bf16*>(jb.o) + at + 16 * cg) =
                            __builtin_convertvector(o[it][cg], bf16x4);
                }
            }
        }
        lds_barrier();   // scores read, the next tiles written
    }

    if (jb.s_out && sg.index == sg.count - 1) {
        const int page = page_of(jb.out_pages, sg.unit, um.n_pages);
        if (page >= 0) st.store(jb.s_out + ((int64_t)page * um.H + h) * (KD * VD));
    }
}

// A segment's own contribution to the state after it, into the next slot of
// its unit. The last segment of a unit has no next one.
template <typename T, int KD, int VD>
__global__ __launch_bounds__(NT, 2) void la_summary(LaUnits um, LaJobs jobs) {
    constexpr int C = Shape<T>::C;
    __shared__ __attribute__((aligned(16))) T kt[2][C * KD];
    __shared__ __attribute__((aligned(16))) T vt[2][C * VD];
    __shared__ __attribute__((aligned(32))) float wt[C];
    const int tid = threadIdx.x;
    const int id = xcd_order(blockIdx.x, gridDim.x);
    const LaJob& jb = jobs.job[id % jobs.n];
    const int h = (id / jobs.n) % um.H, seg_id = id / jobs.n / um.H;
    const Seg sg = find_seg(um, seg_id);
    if (sg.unit < 0 || sg.index == sg.count - 1 || seg_id + 1 >= um.n_segs) return;
    const int seg0 = sg.index * um.seg_tokens, nch = um.seg_tokens / C;
    Carrier<T, KD, C> ck;
    Carrier<T, VD, C> cv;
    ck.load(jb.k, h, sg.start, sg.len, jb.rev, seg0, 0);
    cv.load(jb.v, h, sg.start, sg.len, jb.rev, seg0, 0);
    const double gd = um.decay[h];
    if (tid < C) wt[tid] = (float)(jb.s_w * dpow(gd, C - jb.e - tid));
    const Factor full(dpow(gd, C));
    State<T, KD, VD> st;
    st.zero();
    for (int c = 0; c < nch; ++c) {
        ck.store(kt[c & 1]);
        cv.store(vt[c & 1]);
        if (c + 1 < nch) {
            ck.load(jb.k, h, sg.start, sg.len, jb.rev, seg0 + (c + 1) * C, 0);
            cv.load(jb.v, h, sg.start, sg.len, jb.rev, seg0 + (c + 1) * C, 0);
        }
        lds_barrier();
        ValueFrags<T, VD> vf;
        vf.load(vt[c & 1]);
        st.scale(full);
        add_outer<KD, VD>(st, kt[c & 1], vf, wt);
    }
    st.store(jb.slots + ((int64_t)(seg_id + 1) * um.H + h) * (KD * VD));
}

// Slot s of a unit: from the contribution of segment s - 1 alone to the state
// entering segment s.
__global__ __launch_bounds__(NT) void la_merge(LaUnits um, LaJobs jobs, int kv) {
    const LaJob& jb = jobs.job[blockIdx.y];
    const int blocks = kv / (4 * NT);
    const int at = (blockIdx.x % blocks) * (4 * NT) + threadIdx.x * 4;
    const int h = (blockIdx.x / blocks) % um.H, unit = blockIdx.x / blocks / um.H;
    int first = 0, count;
    if (um.dense) {
        count = segs_of(um.T, um.seg_tokens);
        first = unit * count;
    } else {
        int64_t start;
        int len;
        for (int u0 = 0; u0 < unit; u0 += 64) {   // the segments of the units before
            int ns = 0;
            const int u = u0 + (threadIdx.x & 63);
            if (u < unit) {
                unit_range(um, u, start, len);
                ns = segs_of(len, um.seg_tokens);
            }
            for (int m = 32; m; m >>= 1) ns += __shfl_xor(ns, m);
            first += ns;
        }
        unit_range(um, unit, start, len);
        count = segs_of(len, um.seg_tokens);
    }
    count = min(count, um.n_segs - first);
    const Factor f(dpow(um.decay[h], um.seg_tokens));
    f32x4 e = {0, 0, 0, 0};
    if (jb.s_in) {
        const int page = page_of(jb.in_pages, unit, um.n_pages);
        if (page >= 0) e = *reinterpret_cast<const f32x4*>(jb.s_in + ((int64_t)page * um.H + h) * kv + at);
    }
    float* slot = jb.slots + ((int64_t)first * um.H + h) * kv + at;
    const int64_t pitch = (int64_t)um.H * kv;
    if (count > 0) *reinterpret_cast<f32x4*>(slot) = e;
    for (int s = 1; s < count; ++s) {
        f32x4* x = reinterpret_cast<f32x4*>(slot + s * pitch);
        e = f * e + *x;
        *x = e;
    }
}

__device__ __forceinline__ void put4(float* o, f32x4 x) { *reinterpret_cast<f32x4*>(o) = x; }
__device__ __forceinline__ void put4(bf16* o, f32x4 x) {
    *reinterpret_cast<bf16x4*>(o) = __builtin_convertvector(x, bf16x4);
}

// Sums of the heads that share one, in head order; four values a thread.
template <typename T>
__global__ __launch_bounds__(NT) void la_group(const float* x, T* out, int64_t n4, int group, int D4) {
    const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (i >= n4) return;
    const int64_t th = i / D4;   // token and shared head
    const int d = (int)(i - th * D4);
    const f32x4* p = reinterpret_cast<const f32x4*>(x) + th * group * D4 + d;
    f32x4 s = p[0];
    for (int j = 1; j < group; ++j) s += p[(int64_t)j * D4];
    put4(out + 4 * i, s);
}

template <typename T>
hipError_t main_t(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s) {
    const unsigned n = (unsigned)((int64_t)u.n_segs * u.H * j.n);
    if (K == 128 && V == 128) la_main<T, 128, 128><<<n, NT, 0, s>>>(u, j);
    else if (K == 128) la_main<T, 128, 64><<<n, NT, 0, s>>>(u, j);
    else if (V == 128) la_main<T, 64, 128><<<n, NT, 0, s>>>(u, j);
    else la_main<T, 64, 64><<<n, NT, 0, s>>>(u, j);
    return hipGetLastError();
}

template <typename T>
hipError_t summary_t(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s) {
    const unsigned n = (unsigned)((int64_t)u.n_segs * u.H * j.n);
    if (K == 128 && V == 128) la_summary<T, 128, 128><<<n, NT, 0, s>>>(u, j);
    else if (K == 128) la_summary<T, 128, 64><<<n, NT, 0, s>>>(u, j);
    else if (V == 128) la_summary<T, 64, 128><<<n, NT, 0, s>>>(u, j);
    else la_summary<T, 64, 64><<<n, NT, 0, s>>>(u, j);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_la_main(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s) {
    return dtype == GDN_DTYPE_BF16 ? main_t<bf16>(u, j, K, V, s) : main_t<float>(u, j, K, V, s);
}

hipError_t launch_la_summary(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s) {
    return dtype == GDN_DTYPE_BF16 ? summary_t<bf16>(u, j, K, V, s) : summary_t<float>(u, j, K, V, s);
}

hipError_t launch_la_merge(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s) {
    const int kv = K * V;
    la_merge<<<dim3((unsigned)((int64_t)u.n_units * u.H * (kv / (4 * NT))), j.n), NT, 0, s>>>(u, j, kv);
    return hipGetLastError();
}

hipError_t launch_la_group(const float* x, void* out, int64_t tokens, int H, int h, int D, int dtype, hipStream_t s) {
    const int64_t n4 = tokens * h * D / 4;
    if (n4 == 0) return hipSuccess;
    const unsigned blocks = (unsigned)((n4 + NT - 1) / NT);
    if (dtype == GDN_DTYPE_BF16) la_group<bf16><<<blocks, NT, 0, s>>>(x, static_cast<bf16*>(out), n4, H / h, D / 4);
    else la_group<float><<<blocks, NT, 0, s>>>(x, static_cast<float*>(out), n4, H / h, D / 4);
    return hipGetLastError();
}

}  // namespace gdn
