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
// rounded: two terms (16 bits) for what ends in o - the scores, S in q S, the
// decayed v that enters S - and three (24 bits) for the decayed v where S
// itself is returned in fp32. That is 8 bits more than a bf16 o keeps (its
// error is that of one rounding: 0.00166 relative, as of an fp32 evaluation,
// with 2 of 1000 values rounded to the other neighbour) and 8 fewer than an
// fp32 o could. fp32 inputs: fp32 MFMA.
//
// A partial chunk fills the last rows of its tile: the factors that enter S
// then stay those of a full chunk, and only d^{i+1} and d^C change.
#include "gdn_device.h"
#include "gdn_recurrent_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;
constexpr int NXCD = 8, NCU = 256;

typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// d^n of a log decay g, in fp64: n runs over whole sequences, and the error
// of an fp32 exponent (n g) 2^-24 would show in the states. n = 0 gives 1 for
// g = -inf too.
__device__ __forceinline__ double dpow(double g, int64_t n) { return n == 0 ? 1.0 : exp((double)n * g); }

// x d^n without adding up the rounding of d^n over the chunks of a long
// sequence: near 1 it is x + x (d^n - 1), whose error is that of d^n - 1;
// below 1/2 a value does not live long enough to add anything up.
struct Factor {
    float f;
    bool near_one;
    __device__ explicit Factor(double x) {   // x wave-uniform
        near_one = __builtin_amdgcn_readfirstlane(x > 0.5);
        f = u2f(__builtin_amdgcn_readfirstlane(f2u((float)(near_one ? x - 1.0 : x))));
    }
    __device__ __forceinline__ f32x4 operator*(f32x4 x) const {
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(x[i], f, near_one ? x[i] : 0.0f);
        return y;
    }
};

// Workgroups are handed to the XCDs in turn: gives each XCD a contiguous
// range of the work, so that workgroups reading the same rows share an L2.
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int x = b % NXCD, i = b / NXCD, per = n / NXCD, rem = n % NXCD;
    return x * per + (x < rem ? x : rem) + i;
}

// The same for work that comes longest first: each XCD gets `each` neighbours
// of every 8 `each` in turn, so that all of them take the long ones first.
__device__ __forceinline__ int xcd_deal(int b, int n, int each) {
    const int round = NXCD * each, whole = n / round * round;
    if (b >= whole) return whole + xcd_order(b - whole, n - whole);
    const int r = b % round;
    return b - r + r % NXCD * each + r / NXCD;
}

// The work of this workgroup. Where packed segments give some compute units a
// second workgroup, which is dealt to them in the order of the first, the
// longest ones come last of the first, so that they stay alone and the second
// ones meet the shorter ones: a chunk of K = V = 128 takes a workgroup alone on
// its unit 4.2 us with all units at work (3.1 with a quarter of them, 2.9 with
// a few), one of two 6.9 (T=32768 H=16 in 20 prompts: longest first throughout
// 218 us, like this 204).
__device__ __forceinline__ int work_of_block(const LaUnits& um, int each) {
    int b = blockIdx.x;
    const int n = gridDim.x;
    if (um.dense) return xcd_order(b, n);
    if (n > NCU && n <= 2 * NCU && b < NCU) b = NCU - 1 - b;
    return xcd_deal(b, n, max(1, each / NXCD));
}

struct Seg {
    int unit, index, count;   // the segment's place in its unit
    int id;                   // its place among all, units in order
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

// The segment that is id-th to be worked on; unit is -1 beyond the last.
// Packed units are of any lengths, and the last workgroups to start decide
// when a launch ends: of each 64 units first the segments of the full length,
// then the rest of each unit by falling length, in sixteenths of a full one
// (in order: 20 prompts of 32768 tokens and 32 heads 329 us, like this 285;
// gradients of 12 documents, T=16384 H=16, 336 and 283; only where many short
// ones fill the chip often over is it behind, T=32768 H=16 in 200 prompts 215
// and 227: equal lengths at once store their states at once).
__device__ Seg find_seg(const LaUnits& um, int id) {
    Seg s;
    if (um.dense) {
        s.count = segs_of(um.T, um.seg_tokens);
        s.unit = id / s.count;
        s.index = id - s.unit * s.count;
        s.id = id;
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
        const int full = len / um.seg_tokens;
        int inc = ns, finc = full;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int y = __shfl_up(inc, m), z = __shfl_up(finc, m);
            if (lane >= m) inc += y, finc += z;
        }
        const int total = __builtin_amdgcn_readlane(inc, 63), fulls = __builtin_amdgcn_readlane(finc, 63);
        if (id < base + total) {
            const int x = id - base;
            uint64_t here;
            if (x < fulls) {
                here = __ballot(x < finc);
            } else {
                const int key = ns > full ? (int)((int64_t)(len - full * um.seg_tokens) * 16 / um.seg_tokens) : -1;
                int before = fulls, k = 16;
                uint64_t mask = 0;
                do {
                    before += __popcll(mask);
                    mask = __ballot(key == --k);
                } while (k > 0 && x >= before + __popcll(mask));
                here = __ballot(key == k && x - before == (int)__popcll(mask & ((1ull << lane) - 1)));
            }
            const int at = __ffsll((unsigned long long)here) - 1;
            s.count = __builtin_amdgcn_readlane(ns, at);
            s.index = x < fulls ? x - __builtin_amdgcn_readlane(finc - full, at) : __builtin_amdgcn_readlane(full, at);
            s.id = base + __builtin_amdgcn_readlane(inc - ns, at) + s.index;
            // offsets that are not the host's end here rather than beyond the slots
            if (s.id < um.n_segs) s.unit = u0 + at;
            s.len = __builtin_amdgcn_readlane(len, at);
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)start, at);
            const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(start >> 32), at);
            s.start = (int64_t)(((uint64_t)hi << 32) | lo);
            return s;
        }
        base += total;
    }
    return s;
}

__device__ __forceinline__ int page_of(const int32_t* pages, int unit, int n_pages) {
    if (!pages) return unit;
    const int p = pages[unit];
    return p >= 0 && p < n_pages ? p : -1;
}

// ------------------------------------------------------------------ tiles
// Rows of W elements in LDS in 16-byte units, a row's units exchanged by an
// XOR with some of the row number's bits. Everything a lane reads of a tile
// is at one byte offset of the lane, XOR a multiple of 16 below the row
// length, plus a constant; the offsets are made anew from the thread's number
// in each chunk (fresh), since held in registers they would crowd out the
// state.
template <typename T, int W>
struct Tile {
    static constexpr int EPU = 16 / sizeof(T);
    static constexpr int UNITS = W / EPU;
    static constexpr int RB = W * sizeof(T);   // bytes of a row
    // A permutation of four row bits over the unit bits, made to spread the
    // rows that are read together - 16 at one column, four at four neighbouring
    // units - over the banks. Not all of the walk's accesses are free of
    // conflicts (20 packed prompts: 2.1e7 of la_main's 4.5e7 active LDS cycles
    // are counted as such; of which accesses, tiles or scores, is not known).
    // For bf16 the four are rows r .. r + 3, for fp32 rows r, r + 4, r + 8,
    // r + 12; a 128-byte row is half the banks, so its lowest row bit needs no
    // place.
    __device__ static constexpr int swizzle(int row) {
        const int lo = row & 3, hi = (row >> 2) & 3;
        if (UNITS < 16) return 4 * (lo >> 1) | hi;
        return sizeof(T) == 2 ? 4 * lo | hi : 4 * hi | lo;
    }
    __device__ static __forceinline__ int at(int row, int unit) { return row * RB + (unit ^ swizzle(row)) * 16; }
};

__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}
template <typename V>
__device__ __forceinline__ V lds_get(const char* base, int at) {
    return *reinterpret_cast<const V*>(base + at);
}

// 64 x 16 bytes from base + at (per lane, unsigned) to the 1 KiB of LDS at
// `lds`, straight from memory: no register is written, so nothing the
// compiler knows of is outstanding and it waits for nothing; data_arrived and
// a barrier come before the first read. Written in assembly because the
// builtin makes the compiler wait for every copy before any LDS read. m0 is a
// register that the compiler reserves, so it warns of the clobber; it has to
// know of it all the same, since it merges its own writes of m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(at), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// waits until at most the LATER youngest of this wave's memory accesses are
// in flight
template <int LATER>
__device__ __forceinline__ void data_arrived() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LATER) : "memory");
}
// lds_barrier for tiles that copy_to_lds writes behind the compiler's back
__device__ __forceinline__ void tile_barrier() {
    asm volatile("" ::: "memory");
    lds_barrier();
    asm volatile("" ::: "memory");
}

// One tensor's chunks on their way from memory to a tile. A wave's i-th copy
// brings the rows ROWS (WAVES i + wave) .. of the tile, 64 / UNITS of them.
template <typename T, int W, int C, int WAVES>
struct Feeder {
    using TL = Tile<T, W>;
    static constexpr int ROWS = 64 / TL::UNITS;     // rows of a copy
    static constexpr int N = C / (WAVES * ROWS);    // copies of a wave
    static_assert(N >= 1, "");
    const char* p;   // the next chunk's lowest token (wave-uniform)
    int64_t row;     // bytes from a tile row to the next (negative in reversed time)

    // t0: time of the first tile row
    __device__ __forceinline__ void init(const RowsOf& r, int h, int64_t start, int len, int rev, int t0) {
        const int64_t low = rev ? start + len - t0 - C : start + t0;
        p = static_cast<const char*>(r.p) + (low * r.ts + (int64_t)(h / r.share) * r.hs) * (int)sizeof(T);
        row = (rev ? -r.ts : r.ts) * (int)sizeof(T);
    }
    // shift: the chunk's first row is tile row `shift`; the rows before it get
    // a copy of it
    __device__ __forceinline__ void load(char* tile, int shift, int tid) {
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int row0 = ROWS * wave + lane / TL::UNITS, unit = lane % TL::UNITS;
        const uint32_t len = (uint32_t)(row < 0 ? -row : row);
        const uint32_t to = (uint32_t)(uintptr_t)LDS_PTR(char, tile) + 1024 * wave;
        const char* q = p - shift * row;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = max(row0 + WAVES * ROWS * i, shift);
            const int u = unit ^ TL::swizzle(row0 + WAVES * ROWS * i);
            copy_to_lds(q, (uint32_t)(row < 0 ? C - 1 - r : r) * len + 16 * u, to + 1024 * WAVES * i);
        }
        p += C * row;
    }
    // clears the rows before `shift`
    __device__ static __forceinline__ void clear(char* tile, int shift, int tid) {
        for (int i = tid; i < shift * TL::UNITS; i += 64 * WAVES) reinterpret_cast<u32x4*>(tile)[i] = u32x4{0, 0, 0, 0};
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
__device__ __forceinline__ s16x4 read_across(const char* base, int at) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, base + at));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The leading bf16 term of x, with x left holding what it leaves. The pairs'
// bits are taken apart by hand: from the vector conversion the compiler
// converts every element a second time.
template <int N>
struct Term {
    typedef bf16 vec __attribute__((ext_vector_type(N)));
    typedef float wide __attribute__((ext_vector_type(N)));
    typedef uint32_t words __attribute__((ext_vector_type(N / 2)));
};
template <int N>
__device__ __forceinline__ typename Term<N>::vec split(typename Term<N>::wide& x) {
    typename Term<N>::words w;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const f32x2 y = {x[2 * i], x[2 * i + 1]};
        const uint32_t u = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
        w[i] = u;
        x[2 * i] -= u2f(u << 16);
        x[2 * i + 1] -= u2f(u & 0xffff0000u);
    }
    return __builtin_bit_cast(typename Term<N>::vec, w);
}

template <typename T>
struct Shape;
template <>
struct Shape<bf16> {
    static constexpr int C = 64;    // tokens per chunk
    static constexpr int KS = 32;   // contraction of one operand
    typedef bf16x8 frag;
};
template <>
struct Shape<float> {
    static constexpr int C = 32;
    static constexpr int KS = 16;
    typedef f32x4 frag;
};

// Row 16 it + p of a tile as an operand, contraction block t; at:
// row_lane<T, W>(tid)
template <typename T, int W>
__device__ __forceinline__ int row_lane(int tid) {
    return Tile<T, W>::at(tid & 15, (tid & 63) >> 4);
}
template <typename T, int W>
__device__ __forceinline__ typename Shape<T>::frag row_frag(const char* tile, int at, int it, int t) {
    return lds_get<typename Shape<T>::frag>(tile, (at ^ (64 * t)) + it * 16 * Tile<T, W>::RB);
}

// Columns of a tile as an operand, tokens of block s (32 or 16 of them).
// bf16: four groups of four columns that the lanes p % 4 name; across_lane
// gives the address of the lane's group. fp32: the lane's column.
template <int W>
__device__ __forceinline__ int across_lane(int tid, int col) {   // col: of this lane's group
    const int p = tid & 15, g = (tid & 63) >> 4;
    return Tile<bf16, W>::at(8 * g + (p >> 2), col / 8) + col % 8 * 2;
}
template <int W>
__device__ __forceinline__ bf16x8 across_frag(const char* tile, int at, int s, int flip, int add) {
    constexpr int RB = Tile<bf16, W>::RB;
    // four rows on is another value of one row bit
    return join(read_across(tile, (at ^ flip) + 32 * s * RB + add),
                read_across(tile, (at ^ flip ^ 16 * Tile<bf16, W>::swizzle(4)) + (32 * s + 4) * RB + add));
}
template <int W>
__device__ __forceinline__ int column_lane(int tid, int col) {   // col: of this lane
    const int g = (tid & 63) >> 4;
    return Tile<float, W>::at(4 * g, col / 4) + col % 4 * 4;
}
template <int W>
__device__ __forceinline__ f32x4 column_frag(const char* tile, int at, int s, int flip) {
    constexpr int RB = Tile<float, W>::RB;
    f32x4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        x[r] = lds_get<float>(tile, (at ^ flip ^ (16 * Tile<float, W>::swizzle(r))) + (16 * s + r) * RB);
    return x;
}

// Scores in LDS: blocks of 16 rows x one contraction block (64 bytes a row),
// those on and below the diagonal only.
template <typename T>
struct Scores {
    static constexpr int C = Shape<T>::C, KS = Shape<T>::KS;
    static constexpr int block(int it, int s) {   // it: 16 rows, s: KS columns
        return KS == 32 ? (it < 2 ? it : 2 * it - 2) + s : it * (it + 1) / 2 + s;
    }
    static constexpr int BYTES = 1024 * (block(C / 16 - 1, C / KS - 1) + 1);   // of one term
    // unit u (16 bytes) of row p
    __device__ static __forceinline__ int at(int p, int u) { return p * 64 + (u ^ (p >> 2)) * 16; }
};

// ------------------------------------------------------------------ the state
// A wave's part of S: CG groups of 16 value columns, KD / 16 tiles of 16 keys.
// The columns of two groups alternate by fours, so that a lane's rows of o^T in
// both are eight consecutive values of o.
// bf16: row m of tile 2 t + u is key 32 t + 8 (m / 4) + 4 u + m % 4, so that
// tiles 2 t and 2 t + 1 hold, in each lane, the eight consecutive keys of an
// operand; fp32: row m of tile t is key 16 t + m.
template <typename T, int KD, int CG>
struct State {
    static constexpr int KT = KD / 16;
    using frag = typename Shape<T>::frag;
    f32x4 s[KT][CG];

    // the first of the lane's four rows: a part of the tile, a part of the lane
    __device__ static constexpr int key0(int kt) { return sizeof(T) == 2 ? 32 * (kt >> 1) + 4 * (kt & 1) : 16 * kt; }
    __device__ static __forceinline__ int lane_key(int g) { return sizeof(T) == 2 ? 8 * g : 4 * g; }
    static constexpr int COL_STEP = CG == 2 ? 4 : 0;   // from a group's column to the next group's
    __device__ static __forceinline__ int col(int tid, int cg) {
        const int p = tid & 15, w = tid >> 6;
        return CG == 2 ? 32 * w + 8 * (p >> 2) + 4 * cg + (p & 3) : 16 * w + p;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) s[kt][cg] = f32x4{0, 0, 0, 0};
    }
    // p: from the slice's first column (transposed: row) on, rows of W values.
    // A lane's part of the address is 32 bits, the rest the same in all lanes.
    __device__ __forceinline__ void load(const float* p, int W, int transposed) {
        const int tid = threadIdx.x, key = lane_key((tid & 63) >> 4), c = col(tid, 0);
        const char* q = reinterpret_cast<const char*>(p);
        const uint32_t lane = 4 * (transposed ? c * KD + key : key * W + c);
        if (transposed) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int cg = 0; cg < CG; ++cg)
                    s[kt][cg] = *reinterpret_cast<const f32x4*>(q + 4 * (cg * COL_STEP * KD + key0(kt)) + lane);
        } else {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg)
                        s[kt][cg][r] =
                            *reinterpret_cast<const float*>(q + 4 * ((key0(kt) + r) * W + cg * COL_STEP) + lane);
        }
    }
    // S <- f S + x
    __device__ __forceinline__ void join(const Factor& f, const State& x) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) s[kt][cg] = f * s[kt][cg] + x.s[kt][cg];
    }
    __device__ __forceinline__ void store(float* p, int W) const {
        const int tid = threadIdx.x, key = lane_key((tid & 63) >> 4), c = col(tid, 0);
        char* q = reinterpret_cast<char*>(p);
        const uint32_t lane = 4 * (key * W + c);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int cg = 0; cg < CG; ++cg)
                    *reinterpret_cast<float*>(q + 4 * ((key0(kt) + r) * W + cg * COL_STEP) + lane) = s[kt][cg][r];
    }
    __device__ __forceinline__ void scale(const Factor& f) {
        if (f.near_one) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int cg = 0; cg < CG; ++cg)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[kt][cg][r] = fmaf(s[kt][cg][r], f.f, s[kt][cg][r]);
        } else {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int cg = 0; cg < CG; ++cg) s[kt][cg] *= f.f;
        }
    }
    // S += sum_j wt[j] k_j v_j^T over a chunk; v as operands. bf16: wt v in
    // TERMS terms
    template <int TERMS>
    __device__ __forceinline__ void add(const char* kt_, int tid, const frag (*v)[CG], const float* wt) {
        const int g = (tid & 63) >> 4;
#pragma unroll
        for (int s_ = 0; s_ < 2; ++s_) {
            if constexpr (sizeof(T) == 2) {
                const int at = across_lane<KD>(tid, 8 * (tid & 3));
                const f32x8 w = *reinterpret_cast<const f32x8*>(wt + 32 * s_ + 8 * g);
                bf16x8 b[CG][TERMS];
#pragma unroll
                for (int cg = 0; cg < CG; ++cg) {
                    f32x8 x = w * __builtin_convertvector(v[s_][cg], f32x8);
#pragma unroll
                    for (int i = 0; i + 1 < TERMS; ++i) b[cg][i] = split<8>(x);
                    b[cg][TERMS - 1] = __builtin_convertvector(x, bf16x8);
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const bf16x8 a = across_frag<KD>(kt_, at, s_, 64 * (kt >> 1), 8 * (kt & 1));
#pragma unroll
                    for (int i = 0; i < TERMS; ++i)
#pragma unroll
                        for (int cg = 0; cg < CG; ++cg) s[kt][cg] = mfma(a, b[cg][i], s[kt][cg]);
                }
            } else {
                const int at = column_lane<KD>(tid, tid & 15);
                const f32x4 w = *reinterpret_cast<const f32x4*>(wt + 16 * s_ + 4 * g);
                f32x4 b[CG];
#pragma unroll
                for (int cg = 0; cg < CG; ++cg) b[cg] = w * v[s_][cg];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const f32x4 a = column_frag<KD>(kt_, at, s_, 64 * kt);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) s[kt][cg] = mfma(a, b[cg], s[kt][cg]);
                }
            }
        }
    }
};

// The wave's columns of v (State::col) as operands, two blocks of tokens.
template <typename T, int VD, int CG>
__device__ __forceinline__ void value_frags(const char* tile, int tid, typename Shape<T>::frag (*v)[CG]) {
    using ST = State<T, 128, CG>;   // its columns, whatever the keys
#pragma unroll
    for (int cg = 0; cg < CG; ++cg) {
        if constexpr (sizeof(T) == 2) {
            // the group of four that lane p % 4 names: the columns of rows 4 (p % 4) ..
            const int at = across_lane<VD>(tid, ST::col((tid & ~15) | 4 * (tid & 3), cg));
#pragma unroll
            for (int s = 0; s < 2; ++s) v[s][cg] = across_frag<VD>(tile, at, s, 0, 0);
        } else {
            const int at = column_lane<VD>(tid, ST::col(tid, cg));
#pragma unroll
            for (int s = 0; s < 2; ++s) v[s][cg] = column_frag<VD>(tile, at, s, 0);
        }
    }
}

// ------------------------------------------------------------------ kernels
// The walk: 4 KV + 2 C (K + V) flops a token and head, of which q S and the
// update of S run on two or three bf16 terms, so a chunk of K = V = 128 is 164
// to 196 MFMA of 16 cycles a wave next to about 800 vector instructions that
// split, scale and store. With full-length work on all units memory bounds it
// (B=16 T=4096 H=32: 485 us, 4.4 TB/s), with less the latency of one chunk's
// chain - scores, S's two terms, q S, P v, k v^T - which two workgroups a unit
// overlap: B=4 T=4096 H=16 81 us of 110 (the rest is the segments' states),
// 20 prompts of 32768 tokens and 32 heads 280 us, 2.7 TB/s. The same chain
// bounds fp32, whose MFMA alone would take half the time at a large product's
// rate (T=4096 H=16: 46 of 92 us). Eight waves a workgroup, deeper double buffers,
// fewer address instructions and other orders of the products gain nothing.
// Two workgroups a compute unit (77 KiB of LDS each for K = V = 128): the q
// and v tiles are free for the next chunk once the scores are written and
// q S and v are in registers, so only k has two tiles.
// Four waves of two column groups rather than eight of one (V = 128): an
// operand read from LDS then meets both groups (20 ragged prompts of 32768
// tokens, 32 heads: 321 us against 387).
template <typename T, int KD, int VD>
struct Tiles {
    static constexpr int C = Shape<T>::C, KB = C * KD * sizeof(T), VB = C * VD * sizeof(T);
    static constexpr int PB = (sizeof(T) == 2 ? 2 : 1) * Scores<T>::BYTES;
    alignas(1024) char qt[KB];
    char kt2[2 * KB];
    char vt[VB];
    char pt[PB];
    alignas(32) float wt[C];
    float pw[2 * C], rf[2][C];   // rf[1]: of a partial last chunk
};

// V: o's row, v0: this workgroup's first column of it
// TERMS: bf16 terms of the decayed v that enters S
template <typename T, int KD, int VD, int TERMS>
__device__ __forceinline__ void walk(const LaUnits& um, const LaJob& jb, const Seg& sg, int h, int V, int v0,
                                     Tiles<T, KD, VD>& tiles) {
    constexpr int WAVES = 4, NT = 64 * WAVES;
    constexpr int C = Shape<T>::C, KS = Shape<T>::KS, IT = C / 16, CG = VD / (16 * WAVES);
    constexpr bool BF = sizeof(T) == 2;
    constexpr int KB = C * KD * sizeof(T), PB = Scores<T>::BYTES;
    using SC = Scores<T>;
    using frag = typename Shape<T>::frag;
    char *const qt = tiles.qt, *const kt2 = tiles.kt2, *const vt = tiles.vt, *const pt = tiles.pt;
    float *const wt = tiles.wt, *const pw = tiles.pw;
    float (*const rf)[C] = tiles.rf;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seg0 = sg.index * um.seg_tokens;
    const int seg1 = min(sg.len, seg0 + um.seg_tokens);
    const int nch = seg1 > seg0 ? (seg1 - seg0 + C - 1) / C : 0;
    const int last_shift = nch * C - max(0, seg1 - seg0);   // tile rows before the last chunk's first

    Feeder<T, KD, C, WAVES> fq, fk;
    Feeder<T, VD, C, WAVES> fv;
    fq.init(jb.q, h, sg.start, sg.len, jb.rev, seg0);
    fk.init(jb.k, h, sg.start, sg.len, jb.rev, seg0);
    fv.init(jb.v, h, sg.start, sg.len, jb.rev, seg0);
    fv.p += v0 * (int)sizeof(T);
    auto shift_of = [&](int c) { return c + 1 < nch ? 0 : last_shift; };
    if (nch > 0) {
        fk.load(kt2, shift_of(0), tid);
        fq.load(qt, shift_of(0), tid);
        fv.load(vt, shift_of(0), tid);
    }

    const double gd = um.decay[h];
    State<T, KD, CG> st;
    {
        const int at = v0 * (jb.transposed ? KD : 1);
        const float* slot = jb.slots ? jb.slots + ((int64_t)sg.id * um.H + h) * (KD * V) + at : nullptr;
        const float* from = slot;
        if (jb.s_in && (!slot || um.join)) {
            const int page = page_of(jb.in_pages, sg.unit, um.n_pages);
            from = page >= 0 ? jb.s_in + ((int64_t)page * um.H + h) * (KD * V) + at : nullptr;
        } else if (um.join) {
            from = nullptr;
        }
        if (from) st.load(from, V, jb.transposed);
        else st.zero();
        if (slot && um.join) {   // the segments before: each its own contribution
            const Factor f(dpow(gd, um.seg_tokens));
            const int64_t pitch = (int64_t)um.H * (KD * V);
            for (int i = sg.index - 1; i >= 0; --i) {
                State<T, KD, CG> x;
                x.load(slot - i * pitch, V, jb.transposed);
                st.join(f, x);
            }
        }
    }
    if (tid < 4 * C) {   // four tables of C powers
        const int i = tid % C, table = tid / C;
        const int n = table == 0 ? i : table == 1 ? C - jb.e - i : table == 2 ? i + jb.e : i - last_shift + jb.e;
        const float x = (table == 0 ? jb.s_p : table == 1 ? jb.s_w : jb.s_o) * (float)dpow(gd, max(n, 0));
        if (table == 0) pw[C + i] = x;
        if (table == 1) wt[i] = x;
        if (table == 2) rf[0][i] = x;
        if (table == 3) rf[1][i] = i < last_shift ? 0.0f : x;
        if (table == 0) pw[i] = 0.0f;
    }
    const Factor full(dpow(gd, C)), last(dpow(gd, C - last_shift));
    // the parts of the diagonal's blocks that no score is written to
    for (int i = tid; i < (BF ? 2 : 1) * PB / 16; i += NT) reinterpret_cast<u32x4*>(pt)[i] = u32x4{0, 0, 0, 0};
    data_arrived<0>();
    tile_barrier();
    if (shift_of(0) && nch > 0) {
        fv.clear(vt, shift_of(0), tid);
        tile_barrier();
    }

    // o: bytes from a row to the next, the lowest of the next 16 rows, the lane's part from there
    const int es = jb.o_f32 ? 4 : 2;
    const int64_t orow = (jb.rev ? -1 : 1) * (int64_t)um.H * V * es;
    char* op = static_cast<char*>(jb.o) +
               ((jb.rev ? sg.start + sg.len - seg0 - 16 : sg.start + seg0) * um.H + h) * (V * es) + v0 * es;

    for (int c = 0; c < nch; ++c) {
        const int shift = shift_of(c);
        const bool more = c + 1 < nch;
        const float* rfc = rf[shift ? 1 : 0];
        const char* kt = kt2 + (c & 1) * KB;
        const int t_ = fresh(tid), p = t_ & 15, g = (t_ & 63) >> 4;
        const int row_at = row_lane<T, KD>(t_);
        if (more) fk.load(kt2 + (~c & 1) * KB, shift_of(c + 1), t_);

        // scores of the lower triangle, transposed: the wave's tiles of the list
        // (row tiles of 1, 2, .. tiles); the last waves do the last tile again
        // instead of waiting for the others
        constexpr int TILES = IT * (IT + 1) / 2, MINE = (TILES + WAVES - 1) / WAVES;
        int it_[MINE], jt_[MINE];
        f32x4 sc[MINE];
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int n = min(wave + i * WAVES, TILES - 1);
            it_[i] = BF ? (n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0) : (n >= 1 ? 1 : 0);
            jt_[i] = n - it_[i] * (it_[i] + 1) / 2;
            sc[i] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int t = 0; t < KD / KS; ++t)
#pragma unroll
            for (int i = 0; i < MINE; ++i)
                sc[i] = mfma(row_frag<T, KD>(kt, row_at, jt_[i], t), row_frag<T, KD>(qt, row_at, it_[i], t), sc[i]);
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const float* pwl = pw + C + 16 * (it_[i] - jt_[i]) + p - 4 * g;
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[i][r] *= pwl[-r];
            // row p of row tile it, columns 16 jt + 4 g ..: bf16 half a unit, fp32 a unit
            const int u = BF ? 2 * (jt_[i] & 1) + (g >> 1) : g;
            const int at = 1024 * SC::block(it_[i], BF ? jt_[i] >> 1 : jt_[i]) + SC::at(p, u) + (BF ? 8 * (g & 1) : 0);
            if constexpr (BF) {
                *reinterpret_cast<bf16x4*>(pt + at) = split<4>(sc[i]);
                *reinterpret_cast<bf16x4*>(pt + PB + at) = __builtin_convertvector(sc[i], bf16x4);
            } else {
                *reinterpret_cast<f32x4*>(pt + at) = sc[i];
            }
        }
        frag vf[2][CG];
        value_frags<T, VD, CG>(vt, t_, vf);

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
                    f32x8 x = __builtin_shufflevector(st.s[2 * t][cg], st.s[2 * t + 1][cg], 0, 1, 2, 3, 4, 5, 6, 7);
                    hi[cg] = split<8>(x);
                    lo[cg] = __builtin_convertvector(x, bf16x8);
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const bf16x8 b = row_frag<T, KD>(qt, row_at, it, t);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(hi[cg], b, o[it][cg]);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(lo[cg], b, o[it][cg]);
                }
            } else {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const f32x4 b = row_frag<T, KD>(qt, row_at, it, t);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(st.s[t][cg], b, o[it][cg]);
                }
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const float f = rfc[16 * it + p];
#pragma unroll
            for (int cg = 0; cg < CG; ++cg) o[it][cg] *= f;
        }
        tile_barrier();   // scores written, q and v read
        if (more) {
            fq.load(qt, shift_of(c + 1), t_);
            fv.load(vt, shift_of(c + 1), t_);
        }
        st.scale(shift ? last : full);

        const int p_at = SC::at(p, g);
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int s = 0; s <= (it * 16) / KS; ++s)
#pragma unroll
                for (int x = 0; x < (BF ? 2 : 1); ++x) {
                    const frag b = lds_get<frag>(pt + x * PB + 1024 * SC::block(it, s), p_at);
#pragma unroll
                    for (int cg = 0; cg < CG; ++cg) o[it][cg] = mfma(vf[s][cg], b, o[it][cg]);
                }
        // a lane's rows of o^T: 4 CG consecutive values of row p of o
        const uint32_t o_at =
            (uint32_t)(jb.rev ? 15 - p : p) * (uint32_t)(um.H * V * es) + CG * (16 * wave + 4 * g) * es;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            char* to = op + (16 * it - shift) * orow + o_at;
            if (16 * it + p < shift) continue;
            if (jb.o_f32) {
#pragma unroll
                for (int cg = 0; cg < CG; ++cg)
                    __builtin_nontemporal_store(o[it][cg], reinterpret_cast<f32x4*>(to) + cg);
            } else if constexpr (CG == 2) {
                const f32x8 x = __builtin_shufflevector(o[it][0], o[it][1], 0, 1, 2, 3, 4, 5, 6, 7);
                __builtin_nontemporal_store(__builtin_convertvector(x, bf16x8), reinterpret_cast<bf16x8*>(to));
            } else {
                __builtin_nontemporal_store(__builtin_convertvector(o[it][0], bf16x4), reinterpret_cast<bf16x4*>(to));
            }
        }
        op += C * orow;
        st.template add<TERMS>(kt, t_, vf, wt);

        // a chunk that is not the last has stored all its rows after the
        // copies, with at least one store for each it
        if (more) {
            data_arrived<IT>();
            tile_barrier();
            if (shift_of(c + 1)) {
                fv.clear(vt, shift_of(c + 1), t_);
                tile_barrier();
            }
        }
    }

    if (jb.s_out && sg.index == sg.count - 1) {
        const int page = page_of(jb.out_pages, sg.unit, um.n_pages);
        if (page >= 0) st.store(jb.s_out + ((int64_t)page * um.H + h) * (KD * V) + v0, V);
    }
}

// Three terms (24 bits) for a segment whose state is returned, two elsewhere.
template <typename T, int KD, int VD, bool STATES>
__device__ __forceinline__ void walk_job(const LaUnits& um, const LaJob& jb, const Seg& sg, int h, int V, int v0,
                                         Tiles<T, KD, VD>& tiles) {
    if constexpr (sizeof(T) == 4) walk<T, KD, VD, 1>(um, jb, sg, h, V, v0, tiles);
    else if (STATES && jb.s_out && sg.index == sg.count - 1) walk<T, KD, VD, 3>(um, jb, sg, h, V, v0, tiles);
    else walk<T, KD, VD, 2>(um, jb, sg, h, V, v0, tiles);
}

template <typename T, int KD, int VD, bool STATES>
__global__ __launch_bounds__(256, 2) void la_main(LaUnits um, LaJobs jobs, int slices) {
    __shared__ Tiles<T, KD, VD> tiles;
    int id = work_of_block(um, um.H * jobs.n * slices);
    const int slice = id % slices;
    id /= slices;
    const LaJob& jb = jobs.job[id % jobs.n];
    const Seg sg = find_seg(um, id / jobs.n / um.H);
    if (sg.unit < 0) return;
    walk_job<T, KD, VD, STATES>(um, jb, sg, (id / jobs.n) % um.H, VD * slices, VD * slice, tiles);
}

// Jobs of both K = 64, V = 128 and K = 128, V = 64: the gradients where q and
// v differ in width. One launch, since either alone leaves room (fp32, T=3001
// in 7 documents, H=8, K=128 V=64: 35.7 + 23.6 us apart, 54.7 together).
template <typename T, bool STATES>
__global__ __launch_bounds__(256, 2) void la_main_mixed(LaUnits um, LaJobs jobs) {
    __shared__ union {
        Tiles<T, 64, 128> a;
        Tiles<T, 128, 64> b;
    } tiles;
    const int id = work_of_block(um, um.H * jobs.n);
    const LaJob& jb = jobs.job[id % jobs.n];
    const int h = (id / jobs.n) % um.H;
    const Seg sg = find_seg(um, id / jobs.n / um.H);
    if (sg.unit < 0) return;
    if (jb.K == 64) walk_job<T, 64, 128, STATES>(um, jb, sg, h, 128, 0, tiles.a);
    else walk_job<T, 128, 64, STATES>(um, jb, sg, h, 64, 0, tiles.b);
}

// A segment's own contribution to the state after it, into the next slot of
// its unit. The last segment of a unit has no next one. Here eight waves of
// one group are ahead (B=1 T=2048 H=8 30 us against 32 in all): there is no
// q S and no score to read operands for, and two waves a SIMD overlap. Of B=4
// T=4096 H=16 29 us: three quarters of k and v read once more (100 MB, 3.4
// TB/s), the rest the first chunk's latency and the states' stores.
template <typename T, int KD, int VD, int TERMS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void la_summary(LaUnits um, LaJobs jobs) {
    constexpr int C = Shape<T>::C, KB = C * KD * sizeof(T), VB = C * VD * sizeof(T), CG = VD / (16 * WAVES);
    __shared__ __attribute__((aligned(1024))) char kt[2 * KB];
    __shared__ __attribute__((aligned(1024))) char vt[2 * VB];
    __shared__ __attribute__((aligned(32))) float wt[C];
    const int tid = threadIdx.x;
    const int id = work_of_block(um, um.H * jobs.n);
    const LaJob& jb = jobs.job[id % jobs.n];
    const int h = (id / jobs.n) % um.H;
    const Seg sg = find_seg(um, id / jobs.n / um.H);
    if (sg.unit < 0 || sg.index == sg.count - 1 || sg.id + 1 >= um.n_segs) return;
    const int seg0 = sg.index * um.seg_tokens, nch = um.seg_tokens / C;
    Feeder<T, KD, C, WAVES> fk;
    Feeder<T, VD, C, WAVES> fv;
    fk.init(jb.k, h, sg.start, sg.len, jb.rev, seg0);
    fv.init(jb.v, h, sg.start, sg.len, jb.rev, seg0);
    fk.load(kt, 0, tid);
    fv.load(vt, 0, tid);
    const double gd = um.decay[h];
    if (tid < C) wt[tid] = (float)(jb.s_w * dpow(gd, C - jb.e - tid));
    const Factor full(dpow(gd, C));
    State<T, KD, CG> st;
    st.zero();
    for (int c = 0; c < nch; ++c) {
        data_arrived<0>();
        tile_barrier();
        const int t_ = fresh(tid), b = c & 1;
        if (c + 1 < nch) {
            fk.load(kt + (b ^ 1) * KB, 0, t_);
            fv.load(vt + (b ^ 1) * VB, 0, t_);
        }
        typename Shape<T>::frag vf[2][CG];
        value_frags<T, VD, CG>(vt + b * VB, t_, vf);
        st.scale(full);
        st.template add<TERMS>(kt + b * KB, t_, vf, wt);
    }
    st.store(jb.slots + ((int64_t)(sg.id + 1) * um.H + h) * (KD * VD), VD);
}

// Slot s of a unit: from the contribution of segment s - 1 alone to the state
// entering segment s. Memory bounds it (256 segments and heads, 17 MB read and
// written, from the caches: 6.5 us).
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

// Sums of the heads that share one, in head order; four values a thread: no
// atomics, so the result is the same on every run. Memory bounds it (T=3001,
// 8 heads to 2, 128 wide, from the caches: 5 us).
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

template <typename T, bool STATES>
hipError_t main_t(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s) {
    const unsigned n = (unsigned)((int64_t)u.n_segs * u.H * j.n);
    for (int i = 0; i < j.n; ++i)
        if (j.job[i].K != K) {
            la_main_mixed<T, STATES><<<n, 256, 0, s>>>(u, j);
            return hipGetLastError();
        }
    // With at most half a compute unit's share of workgroups, two of them take
    // 64 value columns each (B=1 T=97 H=8 bf16: 15.1 to 11.9 us a call, T=512
    // H=8: 25 to 23); beyond it that only repeats the scores (T=8192 H=32: 106
    // to 120).
    const int slices = V == 128 && n <= 128 ? 2 : 1, VS = V / slices;
    if (K == 128 && VS == 128) la_main<T, 128, 128, STATES><<<n, 256, 0, s>>>(u, j, 1);
    else if (K == 128) la_main<T, 128, 64, STATES><<<n * slices, 256, 0, s>>>(u, j, slices);
    else if (VS == 128) la_main<T, 64, 128, STATES><<<n, 256, 0, s>>>(u, j, 1);
    else la_main<T, 64, 64, STATES><<<n * slices, 256, 0, s>>>(u, j, slices);
    return hipGetLastError();
}

template <typename T, int TERMS>
hipError_t summary_t(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t s) {
    const unsigned n = (unsigned)((int64_t)u.n_segs * u.H * j.n);
    if (K == 128 && V == 128) la_summary<T, 128, 128, TERMS, 8><<<n, 512, 0, s>>>(u, j);
    else if (K == 128) la_summary<T, 128, 64, TERMS, 4><<<n, 256, 0, s>>>(u, j);
    else if (V == 128) la_summary<T, 64, 128, TERMS, 8><<<n, 512, 0, s>>>(u, j);
    else la_summary<T, 64, 64, TERMS, 4><<<n, 256, 0, s>>>(u, j);
    return hipGetLastError();
}

// a third term (24 bits) only where a state is returned; fp32 has no terms
bool returns_state(const LaJobs& j) {
    for (int i = 0; i < j.n; ++i)
        if (j.job[i].s_out) return true;
    return false;
}

}  // namespace

hipError_t launch_la_main(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s) {
    if (dtype == GDN_DTYPE_F32) return main_t<float, false>(u, j, K, V, s);
    return returns_state(j) ? main_t<bf16, true>(u, j, K, V, s) : main_t<bf16, false>(u, j, K, V, s);
}

hipError_t launch_la_summary(const LaUnits& u, const LaJobs& j, int dtype, int K, int V, hipStream_t s) {
    if (dtype == GDN_DTYPE_F32) return summary_t<float, 1>(u, j, K, V, s);
    return returns_state(j) ? summary_t<bf16, 3>(u, j, K, V, s) : summary_t<bf16, 2>(u, j, K, V, s);
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
