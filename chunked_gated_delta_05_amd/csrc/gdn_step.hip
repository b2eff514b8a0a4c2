// Single-token steps: linear attention with a decay for each head, and the
// gated delta rule, on states kept in the pages of a cache.
//
// One step reads and writes a K x V fp32 state and does 5 (7 for the delta
// rule) operations on each of its elements: it is bound by the state's bytes.
// A workgroup takes VS value columns of one state, holds them in registers
// (so the state is read once and written once, whatever the operator needs
// from it), and every load of the state is issued before anything else.
// Columns are independent but for o, a sum over the K rows: each thread sums
// its rows, lanes and waves are joined by shuffles and one pass through LDS.
#include "gdn_device.h"
#include "gdn_recurrent_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return (float)*p; }

__device__ __forceinline__ void store4(void* o, int64_t at, f32x4 x, int o_dtype) {
    if (o_dtype == GDN_DTYPE_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(o) + at) = x;
    } else {
        typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4*>(static_cast<bf16*>(o) + at) = __builtin_convertvector(x, bf16x4);
    }
}

__device__ __forceinline__ float wave_sum(float x) {
    for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
    return x;
}

// A decay d = b^g as base + rest, base 1 or 0: next to 1 d itself is rounded by
// up to 2^-25, the same way for every token of a head that keeps its g, and
// that adds up over its memory (4096 tokens, g near -1e-3: 1.6e-4 of the
// state, like this below 2e-5). d - 1 is exact to its own last bit, and what
// x + x (d - 1) rounds differs from token to token. 0.1 us of 3.4 to 4.5 where
// a few states' latency counts; without a branch, which takes 0.15 more of the
// delta rule's.
struct Decay {
    float base, rest;
};
__device__ __forceinline__ Decay decay_of(float g, int use_exp2) {
    const float d = fpow(g, use_exp2);
    const bool near_one = d > 0.5f && d < 2.0f;
    const float rest = expm1f(use_exp2 ? g * 0.69314718055994531f : g);
    return {near_one ? 1.0f : 0.0f, near_one ? rest : d};
}
__device__ __forceinline__ f32x4 decayed(f32x4 x, Decay d) {
    f32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(x[j], d.rest, d.base * x[j]);
    return y;
}

// KIND: 0 linear attention, 1 delta rule with a scalar gate, 2 with a
// per-key gate. AROUND: the states are read and written around the caches
template <typename T, int KD, int VD, int VS, int KIND, bool AROUND>
__global__ __launch_bounds__(NT) void step_kernel(StepArgs a) {
    constexpr int CL = VS / 4;          // lanes across the columns, 16 bytes each
    constexpr int RG = NT / CL;         // rows in flight per pass
    constexpr int RPT = KD / RG;        // rows per thread: rg + RG i
    constexpr int SL = VD / VS;
    static_assert(RPT >= 1 && CL <= 64, "");
    __shared__ float qs[KD], ks[KD];
    __shared__ Decay ds[KIND == 2 ? KD : 1];
    __shared__ f32x4 part[2][4][CL];
    __shared__ float wsum[4][3];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cl = tid % CL, rg = tid / CL;
    const int sl = blockIdx.x % SL;
    const int h = (blockIdx.x / SL) % a.H, n = blockIdx.x / SL / a.H;
    const int64_t oat = ((int64_t)n * a.H + h) * VD + sl * VS + 4 * cl;
    const int page = a.pages ? a.pages[n] : n;
    if (page < 0 || page >= a.n_pages) {
        if (rg == 0) store4(a.o, oat, f32x4{0, 0, 0, 0}, a.o_dtype);
        return;
    }
    float* S = a.state + ((int64_t)page * a.H + h) * (KD * VD) + sl * VS + 4 * cl;
    f32x4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const f32x4* p = reinterpret_cast<const f32x4*>(S + (rg + RG * i) * VD);
        s[i] = AROUND ? __builtin_nontemporal_load(p) : *p;
    }
    auto put = [&](int i) {
        f32x4* p = reinterpret_cast<f32x4*>(S + (rg + RG * i) * VD);
        if constexpr (AROUND) __builtin_nontemporal_store(s[i], p);
        else *p = s[i];
    };

    const T* q = static_cast<const T*>(a.q.p) + n * a.q.ts + (h / a.q.share) * a.q.hs;
    const T* k = static_cast<const T*>(a.k.p) + n * a.k.ts + (h / a.k.share) * a.k.hs;
    const T* v = static_cast<const T*>(a.v.p) + n * a.v.ts + (h / a.v.share) * a.v.hs + sl * VS + 4 * cl;
    f32x4 vv;
#pragma unroll
    for (int j = 0; j < 4; ++j) vv[j] = load1(v + j);
    Decay dec = {1.0f, 0.0f};
    float beta = 0.0f;
    if constexpr (KIND == 0) dec = decay_of(a.decay[h], 0);
    if constexpr (KIND == 1) dec = decay_of(a.g[(int64_t)n * a.H + h], a.use_exp2);
    if constexpr (KIND > 0) {
        beta = load1(static_cast<const T*>(a.beta) + (int64_t)n * a.H + h);
        if (a.beta_sig) beta = sigmoid_f(beta);
    }
    float x = 0.0f, y = 0.0f;
    if (tid < KD) {
        x = load1(q + tid);
        y = load1(k + tid);
        qs[tid] = x;
        ks[tid] = y;
        if constexpr (KIND == 2) ds[tid] = decay_of(a.g[((int64_t)n * a.H + h) * KD + tid], a.use_exp2);
    }
    if constexpr (KIND > 0) {   // k.q and, for the norms, k.k and q.q
        const float kq = wave_sum(x * y), qq = wave_sum(x * x), kk = wave_sum(y * y);
        if (lane == 0) {
            wsum[wave][0] = kq;
            wsum[wave][1] = qq;
            wsum[wave][2] = kk;
        }
    }
    lds_barrier();
    float rq = 1.0f, rk = 1.0f, kq = 0.0f;
    if constexpr (KIND > 0) {
        constexpr int KW = KD / 64;
        float qq = 0.0f, kk = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            kq += wsum[w][0];
            qq += wsum[w][1];
            kk += wsum[w][2];
        }
        if (a.qk_norm) {
            rq = rnorm_f(qq);
            rk = rnorm_f(kk);
            kq *= rq * rk;
        }
    }

    f32x4 sq = {0, 0, 0, 0}, sk = {0, 0, 0, 0};   // column sums of q S and k S over this thread's rows
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        const float qr = qs[r], kr = ks[r];
        if constexpr (KIND == 0) {
            s[i] = decayed(s[i], dec) + kr * vv;
        } else {
            s[i] = decayed(s[i], KIND == 2 ? ds[r] : dec);
            sk += kr * s[i];
        }
        sq += qr * s[i];
    }
#pragma unroll
    for (int m = CL; m < 64; m <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sq[j] += __shfl_xor(sq[j], m);
            if constexpr (KIND > 0) sk[j] += __shfl_xor(sk[j], m);
        }
    }
    if (lane < CL) {
        part[0][wave][cl] = sq;
        if constexpr (KIND > 0) part[1][wave][cl] = sk;
    }
    if constexpr (KIND == 0) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) put(i);
    }
    lds_barrier();
    sq = part[0][0][cl] + part[0][1][cl] + part[0][2][cl] + part[0][3][cl];
    if constexpr (KIND > 0) {
        sk = (part[1][0][cl] + part[1][1][cl] + part[1][2][cl] + part[1][3][cl]) * rk;
        const f32x4 br = beta * (vv - sk);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            s[i] += (ks[rg + RG * i] * rk) * br;
            put(i);
        }
        sq = sq * rq + kq * br;
    }
    if (rg == 0) store4(a.o, oat, sq * a.scale, a.o_dtype);
}

template <typename T, int KD, int VD, int KIND>
hipError_t launch(const StepArgs& a, hipStream_t s) {
    const int64_t states = (int64_t)a.N * a.H;
    // Few states: 32 columns a workgroup, for four times the workgroups (16
    // states: 3.6 us a kernel). Many: all columns, so that a workgroup's 64 KiB
    // lie together (8192 states: 211 us against 216). Beyond the last-level
    // cache around the caches (8192 states, 512 MB: 211 to 188 us), within it
    // through them (4096 states, 256 MB: 80 us against 94).
    if (states < 512) {
        constexpr int VS = 32;
        step_kernel<T, KD, VD, VS, KIND, false><<<(unsigned)(states * (VD / VS)), NT, 0, s>>>(a);
    } else if (states * (KD * VD * 4) <= LAST_LEVEL_BYTES) {
        step_kernel<T, KD, VD, VD, KIND, false><<<(unsigned)states, NT, 0, s>>>(a);
    } else {
        step_kernel<T, KD, VD, VD, KIND, true><<<(unsigned)states, NT, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const StepArgs& a, int K, int V, hipStream_t s) {
    if (a.kind == 1) return launch<T, 128, 128, 1>(a, s);
    if (a.kind == 2) return launch<T, 128, 128, 2>(a, s);
    if (K == 128) return V == 128 ? launch<T, 128, 128, 0>(a, s) : launch<T, 128, 64, 0>(a, s);
    return V == 128 ? launch<T, 64, 128, 0>(a, s) : launch<T, 64, 64, 0>(a, s);
}

}  // namespace

hipError_t launch_step(const StepArgs& a, int K, int V, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    return a.dtype == GDN_DTYPE_BF16 ? launch_t<bf16>(a, K, V, s) : launch_t<float>(a, K, V, s);
}

}  // namespace gdn
