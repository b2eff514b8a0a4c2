// Host side of the operators around the recurrent layers (include/gdn_mixer.h):
// argument validation, workspace layout and launch order. Every check runs
// before the first HIP call, so a rejected call enqueues nothing and the checks
// can be exercised without a GPU.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "gdn_mixer.h"
#include "gdn_mixer_internal.h"

namespace {

using gdn::ConvArgs;
using gdn::MxUnits;
using gdn::RotaryArgs;
using gdn::ScanArgs;

constexpr int64_t kMaxElems = int64_t(1) << 40;                   // sanity bound on any tensor
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 256;         // of a launch along x, in workgroups of 256
// Segments of a sequence up to which each adds up those before its own, which
// saves the launch of a merge (T=160 D=1024 20.1 to 15.8 us, T=800 26.7 to 23.8,
// gradients alone of T=160 29.6 to 27.1, T=400 32 to 30, B=2 T=4096 D=4096 503
// either way; where 32 of them do, T=1000 D=4096 147 to 156).
constexpr int64_t kJoin = 16;
constexpr int32_t kMaxTokens = INT32_MAX - 4096;                  // of a sequence: its tiles' ends are ints

int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool aligned16(const void* p) { return aligned(p, 16); }

template <typename... P>
bool all_aligned16(P... p) {
    return (aligned16(p) && ...);
}

bool overlap(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && a_bytes && b_bytes && (x < y ? y - x < a_bytes : x - y < b_bytes);
}

bool dtype_ok(int32_t d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

bool flag_ok(int32_t f) { return f == 0 || f == 1; }

int64_t elem_bytes(int32_t d) { return d == GDN_DTYPE_BF16 ? 2 : 4; }

// token distances of less than this keep a tile's rows within 32-bit offsets
constexpr int64_t kMaxStrideBytes = int64_t(1) << 24;

bool stride_small(int64_t s, int32_t dtype) { return s * elem_bytes(dtype) < kMaxStrideBytes; }

// a distance that keeps rows 16-byte aligned and n of them below 2^60 elements
bool stride_ok(int64_t s, int64_t n, int32_t dtype) {
    const int64_t lim = int64_t(1) << 60;
    return s >= 0 && s <= lim && s * elem_bytes(dtype) % 16 == 0 && (n <= 0 || s <= lim / n);
}

gdn_status run(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_DEVICE; }

// The size query and the checks of a given workspace.
gdn_status check_workspace(int64_t need, void* workspace, size_t* workspace_bytes, bool* query) {
    if (workspace_bytes == nullptr) return GDN_ERR_INVALID;
    if (need < 256) need = 256;
    *query = workspace == nullptr;
    if (*query || *workspace_bytes < (size_t)need) {
        const gdn_status st = *query ? GDN_OK : GDN_ERR_CAPACITY;
        *workspace_bytes = (size_t)need;
        return st;
    }
    return reinterpret_cast<uintptr_t>(workspace) % 256 == 0 ? GDN_OK : GDN_ERR_INVALID;
}

// ------------------------------------------------------------------ sequences
struct Seqs {
    MxUnits un;        // P and n_pieces still open
    int64_t longest;
};

gdn_status check_seqs(int32_t B, int32_t T, int32_t n_units, const int32_t* host, const int32_t* dev, Seqs* s) {
    memset(s, 0, sizeof(*s));
    if (B < 1 || T < 0 || n_units < 0) return GDN_ERR_INVALID;
    MxUnits& u = s->un;
    u.T = T;
    u.total = int64_t(B) * T;
    s->longest = T;
    if (n_units == 0) {
        u.dense = 1;
        u.n_units = B;
    } else {
        if (B != 1 || !host || !dev) return GDN_ERR_INVALID;
        if (host[0] != 0 || host[n_units] != T) return GDN_ERR_INVALID;
        s->longest = 0;
        for (int32_t i = 0; i < n_units; ++i) {
            if (host[i] >= host[i + 1]) return GDN_ERR_INVALID;
            const int64_t len = int64_t(host[i + 1]) - host[i];
            s->longest = len > s->longest ? len : s->longest;
        }
        u.n_units = n_units;
        u.offsets = dev;
    }
    return s->longest > kMaxTokens ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

// Whether states before and after share memory. False: without page lists they
// overlap by part, so that one sequence would read what another has written.
bool check_states(const void* s_in, const int32_t* in_pages, const void* s_out, const int32_t* out_pages, uint64_t page,
                  int32_t units, int32_t n_pages, bool* in_place) {
    *in_place = overlap(s_in, page * (in_pages ? n_pages : units), s_out, page * (out_pages ? n_pages : units));
    return !*in_place || in_pages || out_pages || s_in == s_out;
}

// numbers of pieces of P tokens: gdn_mixer_internal.h
int64_t pieces(const MxUnits& u, int64_t P) {
    if (u.dense) return int64_t(u.n_units) * (u.T > P ? (u.T + P - 1) / P : 1);
    return u.total / P + u.n_units;
}

// pieces of P tokens that there are
int64_t segments(const MxUnits& u, const int32_t* host, int64_t P) {
    if (u.dense) return pieces(u, P);
    int64_t n = 0;
    for (int32_t i = 0; i < u.n_units; ++i) n += (int64_t(host[i + 1]) - host[i] + P - 1) / P;
    return n;
}

// false: more than a launch's numbers
bool cut(MxUnits* u, int64_t P) {
    const int64_t n = pieces(*u, P);
    if (n > INT32_MAX || P > INT32_MAX) return false;
    u->P = (int32_t)P;
    u->n_pieces = (int32_t)n;
    return true;
}

// ------------------------------------------------------------------ convolution
int64_t vector_channels(int32_t dtype) { return 16 / elem_bytes(dtype); }

// longest: the largest piece; channels: of a thread. A piece reads W - 1 tokens
// before its own (its gradients as many after, and write a row of sums), but a
// thread waits for memory every few tokens: pieces are as long as leave enough
// threads to keep the memory busy (forward and gradients in pieces of 16, 64
// and 128: B=4 T=4096 D=6144 304, 245 and 240 us, B=2 T=2048 D=2048 35, 64 and
// 109; 256: 268 and 202).
gdn_status check_conv(const gdn_conv_desc* d, int64_t longest, int64_t channels, ConvArgs* a) {
    if (d == nullptr) return GDN_ERR_INVALID;
    if (d->W < 2 || d->W > 4) return GDN_ERR_UNSUPPORTED;
    if (d->D < 1 || d->D % 8 != 0 || !dtype_ok(d->dtype) || !dtype_ok(d->w_dtype) || !flag_ok(d->silu)) return GDN_ERR_INVALID;
    Seqs s;
    const gdn_status st = check_seqs(d->B, d->T, d->n_units, d->offsets_host, d->offsets_dev, &s);
    if (st != GDN_OK) return st;
    if (s.un.total > kMaxElems / d->D || !stride_ok(d->x_stride, s.un.total, d->dtype)) return GDN_ERR_INVALID;
    memset(a, 0, sizeof(*a));
    a->un = s.un;
    const int64_t vectors = d->D / channels;
    int64_t P = longest;
    while (P > 8 && pieces(s.un, P) * vectors < 100000) P /= 2;
    if (!cut(&a->un, P) || int64_t(a->un.n_pieces) * vectors > kMaxThreads || int64_t(s.un.n_units) * vectors > kMaxThreads)
        return GDN_ERR_UNSUPPORTED;
    a->D = d->D;
    a->W = d->W;
    a->dtype = d->dtype;
    a->w_f32 = d->w_dtype == GDN_DTYPE_F32;
    a->silu = d->silu;
    a->x_stride = d->x_stride;
    return GDN_OK;
}

}  // namespace

extern "C" gdn_status gdn_conv_fwd(const gdn_conv_desc* d, const void* x, const void* weight, const void* bias,
                                   const void* s_in, const int32_t* in_pages, void* s_out, const int32_t* out_pages,
                                   int32_t n_pages, void* y, hipStream_t stream) {
    ConvArgs a;
    const gdn_status st = check_conv(d, 64, vector_channels(d ? d->dtype : 0), &a);
    if (st != GDN_OK) return st;
    if (!weight || (a.un.total > 0 && (!x || !y))) return GDN_ERR_INVALID;
    if (n_pages < 0 || (in_pages && !s_in) || (out_pages && !s_out)) return GDN_ERR_INVALID;
    if (!all_aligned16(x, weight, bias, s_in, s_out, y)) return GDN_ERR_INVALID;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.s_in = s_in;
    a.in_pages = in_pages;
    a.s_out = s_out;
    a.out_pages = out_pages;
    a.n_pages = n_pages;
    a.y = y;
    bool in_place;
    if (!check_states(s_in, in_pages, s_out, out_pages, uint64_t(d->W - 1) * d->D * elem_bytes(d->dtype), a.un.n_units, n_pages,
                      &in_place))
        return GDN_ERR_INVALID;
    return run(gdn::launch_conv_fwd(a, in_place, stream));
}

extern "C" gdn_status gdn_conv_bwd(const gdn_conv_desc* d, const void* x, const void* weight, const void* bias,
                                   const void* s_in, const void* dout, const void* dfinal, void* dx, float* dweight,
                                   float* dbias, void* dinitial, void* workspace, size_t* workspace_bytes,
                                   hipStream_t stream) {
    ConvArgs a;
    gdn_status st = check_conv(d, 128, gdn::CONV_BWD_CHANNELS, &a);
    if (st != GDN_OK) return st;
    const int64_t rows = int64_t(a.un.n_pieces) + gdn::row_sums_rows(a.un.n_pieces);
    if (rows > kMaxElems / (int64_t(d->D) * (d->W + 1))) return GDN_ERR_UNSUPPORTED;
    if (gdn::row_sums_workgroups(a.un.n_pieces, int64_t(d->D) * (d->W + 1)) > kMaxThreads / 256) return GDN_ERR_UNSUPPORTED;
    bool query = false;
    st = check_workspace(rows * d->D * (d->W + 1) * 4, workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    if (!weight || !dweight || (a.un.total > 0 && (!x || !dout || !dx))) return GDN_ERR_INVALID;
    if (!all_aligned16(x, weight, bias, s_in, dout, dfinal, dx, dweight, dbias, dinitial)) return GDN_ERR_INVALID;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.s_in = s_in;
    a.dout = dout;
    a.dfinal = dfinal;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dinitial = dinitial;
    a.parts = static_cast<float*>(workspace);
    return run(gdn::launch_conv_bwd(a, stream));
}

extern "C" gdn_status gdn_conv_step(const gdn_conv_desc* d, const void* x, const void* weight, const void* bias,
                                    const int32_t* pages, int32_t n_pages, void* state, void* y, hipStream_t stream) {
    if (d != nullptr && d->B == 0 && d->T == 1) return GDN_OK;
    ConvArgs a;
    const gdn_status st = check_conv(d, 8, vector_channels(d ? d->dtype : 0), &a);
    if (st != GDN_OK) return st;
    if (d->T != 1 || d->n_units != 0 || n_pages < 0) return GDN_ERR_INVALID;
    if (!x || !weight || !y || (n_pages > 0 && !state) || !all_aligned16(x, weight, bias, state, y)) return GDN_ERR_INVALID;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.in_pages = pages;
    a.n_pages = n_pages;
    a.s_out = state;
    a.y = y;
    return run(gdn::launch_conv_step(a, stream));
}

// ------------------------------------------------------------------ scan
namespace {

struct Scan {
    ScanArgs a;
    int64_t slots, sums;   // bytes in front of the workspace
};

// Tokens that the workgroups of whole sequences, nb each, bring to the compute
// unit that gets the most, dealt out in turn.
int64_t fullest(const MxUnits& u, const int32_t* host, int64_t nb, int64_t P) {
    if (u.dense) return (u.n_units * nb + 255) / 256 * u.T;
    int64_t step[257] = {}, all = 0, most = 0, on = 0;
    for (int32_t i = 0; i < u.n_units; ++i) {
        const int64_t len = int64_t(host[i + 1]) - host[i], at = (host[i] / P + i) * nb % 256, end = at + nb % 256;
        all += nb / 256 * len;
        step[at] += len;
        step[end < 256 ? end : 256] -= len;
        if (end > 256) {
            step[0] += len;
            step[end - 256] -= len;
        }
    }
    for (int i = 0; i < 256; ++i) {
        on += step[i];
        most = on > most ? on : most;
    }
    return all + most;
}

// The forward of sequences that would leave compute units with less than two
// workgroups of one channel a lane: walked whole by one state a lane, or cut. Both
// are estimated in ns. One state a lane: 16 for each token of the longest sequence
// and `state` for each token of the waves that a SIMD gets; a cut 10.5 us for its
// launches and short walks and 1.45 times the waves' part, level (cut and whole:
// D=4096, one sequence of T=400 25 and 19 us, 1000 42.5 and 40.7, 2000 68 and 78;
// four of 1000 113 and 92; D=1024, T=300 16 and 14.3, 400 17.3 and 18.4; 12
// documents, T=16384, 134 and 172; S=64 D=1024, one and four of T=1000 44 and 87,
// 112 and 90. Beyond: eight of T=1000 D=4096 156 with one channel a lane and 168
// with one state). Other S, cut and whole again: S=8 D=1024, one of T=200 15.6 and
// 12.4, 400 16.9 and 20.9, four of 400 22 and 21.7, of 1000 33.5 and 47, D=4096 one of
// 1000 33 and 47; S=32 D=1024, one of T=200 14.8 and 14, 400 17.6 and 23.7, four of 400
// 33.7 and 25.4, of 1000 61 and 56, of 2000 109 and 105; S=64 D=1024, one of T=200 17.3
// and 21.5, 400 25 and 37, four of 400 57 and 40, of 2000 202 and 174. fp32 takes as
// long whole and up to a quarter longer cut (S=8 D=4096 T=1000 41), for which there is
// no term; storing h adds 2 to 6% whole, 0 to 4% cut. The rule takes the faster side of
// all these. It takes the slower one for a few ragged documents (five of 210 to 402
// tokens, D=1536 G=2, cut: 28 and 25, 32 and 27, 47 and 41, 82 and 63 at S=8 to 64; in
// fp32 29 and 25, 32 and 27.5, 48 and 41, 70 and 64), for two of T=2000 D=4096 S=8
// (whole: 83 and 92) and, in fp32, four of T=2000 D=1024 S=16 (cut: 79 and 74).
bool whole_pays(const ScanArgs& a, const int32_t* host, int64_t longest, int64_t P) {
    const double state = a.S == 8 ? 26 : a.S == 16 ? 18.5 : a.S == 32 ? 32 : 67;
    const int ch = gdn::scan_narrow_channels(a.S);
    const int64_t nb = int64_t(a.G) * ((a.D / a.G + ch - 1) / ch), most = fullest(a.un, host, nb, P);
    return 16.0 * longest + state * most < 10500 + 1.45 * state * a.un.total * nb / 256;
}

gdn_status check_scan(const gdn_scan_desc* d, bool forward, Scan* s) {
    if (d == nullptr) return GDN_ERR_INVALID;
    if (d->S != 8 && d->S != 16 && d->S != 32 && d->S != 64) return GDN_ERR_UNSUPPORTED;
    if (d->D < 1 || d->G < 1 || d->D % d->G != 0 || d->D / d->G % 8 != 0) return GDN_ERR_INVALID;
    if (!dtype_ok(d->dtype) || !flag_ok(d->softplus)) return GDN_ERR_INVALID;
    Seqs q;
    const gdn_status st = check_seqs(d->B, d->T, d->n_units, d->offsets_host, d->offsets_dev, &q);
    if (st != GDN_OK) return st;
    const int64_t total = q.un.total;
    if (total > kMaxElems / d->D || int64_t(q.un.n_units) > kMaxElems / d->S / d->D) return GDN_ERR_INVALID;
    if (!stride_ok(d->u_stride, total, d->dtype) || !stride_ok(d->dt_stride, total, d->dtype) ||
        !stride_ok(d->gate_stride, total, d->dtype) || !stride_ok(d->b_stride[0], total, d->dtype) ||
        !stride_ok(d->c_stride[0], total, d->dtype) || !stride_ok(d->b_stride[1], d->G, d->dtype) ||
        !stride_ok(d->c_stride[1], d->G, d->dtype))
        return GDN_ERR_INVALID;
    if (!stride_small(d->u_stride, d->dtype) || !stride_small(d->dt_stride, d->dtype) ||
        !stride_small(d->gate_stride, d->dtype) || !stride_small(d->D, d->dtype))
        return GDN_ERR_UNSUPPORTED;
    memset(s, 0, sizeof(*s));
    ScanArgs& a = s->a;
    a.D = d->D;
    a.G = d->G;
    a.S = d->S;
    a.dtype = d->dtype;
    a.softplus = d->softplus;
    a.u_stride = d->u_stride;
    a.dt_stride = d->dt_stride;
    a.gate_stride = d->gate_stride;
    memcpy(a.b_stride, d->b_stride, sizeof(a.b_stride));
    memcpy(a.c_stride, d->c_stride, sizeof(a.c_stride));
    const int ch = gdn::scan_channels(d->S), per = d->D / d->G;
    a.blocks = (per + ch - 1) / ch;
    a.bwd_blocks = (per + ch / 2 - 1) / (ch / 2);
    a.un = a.keep = q.un;
    if (!cut(&a.keep, gdn::SCAN_KEEP)) return GDN_ERR_UNSUPPORTED;
    if (a.keep.n_pieces > kMaxElems / d->S / d->D) return GDN_ERR_UNSUPPORTED;
    // Segments. A cut costs a second walk (summary and main take 0.7 and 1 of a
    // whole walk's time) and two launches with a merge between. So nothing is cut
    // unless one sequence takes longer, on a compute unit of its own, than both
    // walks of everything on all 256 (with gradients D=1024, one sequence of T=96
    // whole and cut 54 and 57 us, 128 67 and 56).
    // Four workgroups run on a unit at a time and share its issue, so all take about
    // as long as the most of them on one unit, at segments of P tokens (and 10 for a
    // start); where fewer are left, instructions wait (kRest). Of 2 to 8 on a unit the best (3 documents,
    // T=6000 D=4096, in 28 segments 202 us, in 48 176; 12, T=16384 D=1024, 155 and
    // 134; B=2 T=4096 D=4096 with gradients, 16, 32 and 64: 785, 756 and 762). None
    // is shorter than what the merge, which walks through them one by one, saves.
    const int64_t tile = gdn::SCAN_TILE, whole = (q.longest + tile - 1) / tile * tile;
    const int64_t walks = int64_t(a.G) * a.blocks;
    int64_t P = whole > 0 ? whole : tile;
    const bool few = forward && int64_t(q.un.n_units) * a.G * a.bwd_blocks < 512;
    a.narrow = few && whole_pays(a, d->offsets_host, q.longest, P);
    if (few ? !a.narrow : q.longest > 1.4 * double(total) * walks / 256 + (forward ? 130 : 85)) {
        const int64_t least = ((int64_t)sqrt(0.44 * double(q.longest)) + tile) / tile * tile, most = P;
        const bool many = q.un.n_units > 64;   // sequences to count through: four a unit it is
        constexpr double kRest[4] = {0, 1.7, 2.4, 3.15};
        double best = 0;
        for (int per = many ? 4 : 2; per <= (many ? 4 : 8); ++per) {
            int64_t lo = least < most ? least : most, hi = most;
            while (lo < hi) {
                const int64_t mid = (lo + hi) / 2 / tile * tile;
                if (segments(q.un, d->offsets_host, mid) * walks <= per * 256) hi = mid;
                else lo = mid + tile;
            }
            const int64_t on = (segments(q.un, d->offsets_host, hi) * walks + 255) / 256;
            const double cost = double(hi + 10) * (on / 4 * 4 + kRest[on % 4]);
            if (best == 0 || cost < best) {
                best = cost;
                P = hi;
            }
        }
    }
    if (!cut(&a.un, P)) return GDN_ERR_UNSUPPORTED;
    a.cut = q.longest > P;
    a.join = a.cut && (q.longest + P - 1) / P <= kJoin;
    const int64_t merge = int64_t(q.un.n_units) * ((int64_t(d->D) * d->S + 255) / 256) * 256;
    if (a.un.n_pieces > kMaxThreads / 256 / walks || merge > kMaxThreads) return GDN_ERR_UNSUPPORTED;
    if (a.cut) {
        s->slots = align256(int64_t(a.un.n_pieces) * d->D * d->S * 4);
        s->sums = align256(int64_t(a.un.n_pieces) * d->D * 4);
    }
    return GDN_OK;
}

void scan_inputs(ScanArgs* a, const void* u, const void* dt, const float* A, const void* B, const void* C,
                 const float* skip, const void* gate, const float* dt_bias) {
    a->u = u;
    a->dt = dt;
    a->A = A;
    a->b = B;
    a->c = C;
    a->skip = skip;
    a->gate = gate;
    a->dt_bias = dt_bias;
}

}  // namespace

extern "C" int64_t gdn_scan_h_rows(const gdn_scan_desc* d) {
    Scan s;
    return check_scan(d, true, &s) == GDN_OK ? s.a.keep.n_pieces : -1;
}

extern "C" gdn_status gdn_scan_fwd(const gdn_scan_desc* d, const void* u, const void* dt, const float* A,
                                   const void* B, const void* C, const float* skip, const void* gate,
                                   const float* dt_bias, const float* s_in, const int32_t* in_pages, float* s_out,
                                   const int32_t* out_pages, int32_t n_pages, float* h, void* out, void* workspace,
                                   size_t* workspace_bytes, hipStream_t stream) {
    Scan s;
    gdn_status st = check_scan(d, true, &s);
    if (st != GDN_OK) return st;
    bool query = false;
    st = check_workspace(s.slots + s.sums, workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    ScanArgs& a = s.a;
    if (!A || (a.un.total > 0 && (!u || !dt || !B || !C || !out))) return GDN_ERR_INVALID;
    if (n_pages < 0 || (in_pages && !s_in) || (out_pages && !s_out)) return GDN_ERR_INVALID;
    if (!all_aligned16(u, dt, A, B, C, skip, gate, dt_bias, s_in, s_out, h, out)) return GDN_ERR_INVALID;
    scan_inputs(&a, u, dt, A, B, C, skip, gate, dt_bias);
    a.s_in = s_in;
    a.in_pages = in_pages;
    a.s_out = s_out;
    a.out_pages = out_pages;
    a.n_pages = n_pages;
    a.h = h;
    a.out = out;
    // a sequence's last segment may replace the state before its others have read
    // it: where the two share memory the merge reads it in front of all
    bool in_place;
    if (!check_states(s_in, in_pages, s_out, out_pages, uint64_t(d->D) * d->S * 4, a.un.n_units, n_pages, &in_place))
        return GDN_ERR_INVALID;
    if (in_place) a.join = 0;
    if (a.cut) {
        a.slots = static_cast<float*>(workspace);
        a.sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + s.slots);
        if (gdn::launch_scan_summary(a, false, stream) != hipSuccess) return GDN_ERR_DEVICE;
        if (!a.join && gdn::launch_scan_merge(a, false, stream) != hipSuccess) return GDN_ERR_DEVICE;
    }
    return run(gdn::launch_scan_fwd(a, stream));
}

extern "C" gdn_status gdn_scan_bwd(const gdn_scan_desc* d, const void* u, const void* dt, const float* A,
                                   const void* B, const void* C, const float* skip, const void* gate,
                                   const float* dt_bias, const float* h, const void* dout, const float* dht, void* du,
                                   void* ddt, float* dA, void* dB, void* dC, float* dskip, void* dgate,
                                   float* ddt_bias, float* dh0, void* workspace, size_t* workspace_bytes,
                                   hipStream_t stream) {
    Scan s;
    gdn_status st = check_scan(d, false, &s);
    if (st != GDN_OK) return st;
    ScanArgs& a = s.a;
    const int64_t walks = int64_t(a.G) * a.bwd_blocks;
    if (a.un.n_pieces > kMaxThreads / 256 / walks) return GDN_ERR_UNSUPPORTED;
    if (a.un.total > kMaxElems / (walks * 2 * d->S) || a.un.total * d->G * (d->S / 2) > kMaxThreads) return GDN_ERR_UNSUPPORTED;
    const int64_t rows = int64_t(a.un.n_pieces) + gdn::row_sums_rows(a.un.n_pieces);
    if (rows > kMaxElems / (int64_t(d->D) * (d->S + 2)) ||
        gdn::row_sums_workgroups(a.un.n_pieces, int64_t(d->D) * (d->S + 2)) > kMaxThreads / 256)
        return GDN_ERR_UNSUPPORTED;
    if (gdn::scan_sum_workgroups(a.un.total, a.un.n_pieces, d->G, d->D, d->S) > kMaxThreads / 256) return GDN_ERR_UNSUPPORTED;
    const int64_t bc = align256(walks * a.un.total * 2 * d->S * 4), ap = align256(rows * d->D * (d->S + 2) * 4);
    bool query = false;
    st = check_workspace(s.slots + s.sums + bc + ap, workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    if (!A || !dA || (a.un.total > 0 && (!u || !dt || !B || !C || !h || !dout || !du || !ddt || !dB || !dC))) return GDN_ERR_INVALID;
    if (a.un.total > 0 && (gate == nullptr) != (dgate == nullptr)) return GDN_ERR_INVALID;
    if (!all_aligned16(u, dt, A, B, C, skip, gate, dt_bias, h, dout, dht, du, ddt, dA, dB, dC, dskip, dgate, ddt_bias, dh0))
        return GDN_ERR_INVALID;
    const uint64_t states = uint64_t(a.un.n_units) * d->D * d->S * 4;
    if (dh0 != dht && overlap(dh0, states, dht, states)) return GDN_ERR_INVALID;
    if (dh0 && dh0 == dht) a.join = 0;   // as in gdn_scan_fwd
    scan_inputs(&a, u, dt, A, B, C, skip, gate, dt_bias);
    a.s_in = dht;
    a.s_out = dh0;
    a.h = const_cast<float*>(h);
    a.dout = dout;
    a.du = du;
    a.ddt = ddt;
    a.dgate = dgate;
    a.db = dB;
    a.dc = dC;
    a.dA = dA;
    a.dskip = dskip;
    a.ddt_bias = ddt_bias;
    char* base = static_cast<char*>(workspace);
    a.slots = reinterpret_cast<float*>(base);
    a.sums = reinterpret_cast<float*>(base + s.slots);
    a.bc_parts = reinterpret_cast<float*>(base + s.slots + s.sums);
    a.a_parts = reinterpret_cast<float*>(base + s.slots + s.sums + bc);
    if (a.cut) {
        if (gdn::launch_scan_summary(a, true, stream) != hipSuccess) return GDN_ERR_DEVICE;
        if (!a.join && gdn::launch_scan_merge(a, true, stream) != hipSuccess) return GDN_ERR_DEVICE;
    }
    return run(gdn::launch_scan_bwd(a, stream));
}

extern "C" gdn_status gdn_scan_step(const gdn_scan_desc* d, const void* u, const void* dt, const float* A,
                                    const void* B, const void* C, const float* skip, const void* gate,
                                    const float* dt_bias, const int32_t* pages, int32_t n_pages, float* state,
                                    void* out, hipStream_t stream) {
    if (d != nullptr && d->B == 0 && d->T == 1) return GDN_OK;
    Scan s;
    const gdn_status st = check_scan(d, true, &s);
    if (st != GDN_OK) return st;
    if (d->T != 1 || d->n_units != 0 || n_pages < 0) return GDN_ERR_INVALID;
    ScanArgs& a = s.a;
    if (!u || !dt || !A || !B || !C || !out || (n_pages > 0 && !state)) return GDN_ERR_INVALID;
    if (!all_aligned16(u, dt, A, B, C, skip, gate, dt_bias, state, out)) return GDN_ERR_INVALID;
    if (n_pages > kMaxElems / d->S / d->D) return GDN_ERR_INVALID;
    scan_inputs(&a, u, dt, A, B, C, skip, gate, dt_bias);
    a.in_pages = pages;
    a.n_pages = n_pages;
    a.s_out = state;
    a.out = out;
    return run(gdn::launch_scan_step(a, stream));
}

// ------------------------------------------------------------------ norms and rotation
namespace {

gdn_status check_rotary(const gdn_rotary_desc* d, RotaryArgs* a) {
    if (d == nullptr) return GDN_ERR_INVALID;
    if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->Hk < 1 || d->D < 1 || d->R < 0 || d->R > d->D) return GDN_ERR_INVALID;
    if (d->D % 8 != 0 || d->R % 8 != 0 || d->D > 256) return GDN_ERR_UNSUPPORTED;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->w_dtype) || !flag_ok(d->interleaved) || !flag_ok(d->pos_i64)) return GDN_ERR_INVALID;
    if (d->norm != GDN_NORM_NONE && d->norm != GDN_NORM_RMS && d->norm != GDN_NORM_L2) return GDN_ERR_INVALID;
    if (!isfinite(d->amplitude) || !isfinite(d->eps) || d->eps < 0) return GDN_ERR_INVALID;
    const int64_t tokens = int64_t(d->B) * d->T, heads = int64_t(d->Hq) + d->Hk;
    if (heads > 65536 || tokens > kMaxElems / (heads * d->D)) return GDN_ERR_INVALID;
    if (!stride_ok(d->q_stride[0], tokens, d->dtype) || !stride_ok(d->k_stride[0], tokens, d->dtype) ||
        !stride_ok(d->q_stride[1], d->Hq, d->dtype) || !stride_ok(d->k_stride[1], d->Hk, d->dtype))
        return GDN_ERR_INVALID;
    if (tokens > kMaxThreads / 256) return GDN_ERR_UNSUPPORTED;
    memset(a, 0, sizeof(*a));
    a->T = d->T;
    a->Hq = d->Hq;
    a->Hk = d->Hk;
    a->D = d->D;
    a->R = d->R;
    a->dtype = d->dtype;
    a->w_f32 = d->w_dtype == GDN_DTYPE_F32;
    a->norm = d->norm;
    a->interleaved = d->interleaved;
    a->pos_i64 = d->pos_i64;
    a->tokens = tokens;
    a->eps = d->eps;
    a->amplitude = d->amplitude;
    memcpy(a->q_stride, d->q_stride, sizeof(a->q_stride));
    memcpy(a->k_stride, d->k_stride, sizeof(a->k_stride));
    a->workgroups = gdn::rotary_bwd_workgroups(tokens);
    return GDN_OK;
}

// what is read one by one may be a slice of a longer array
bool angles_aligned(const gdn_rotary_desc* d, const double* freqs, const void* positions) {
    return aligned(freqs, 8) && aligned(positions, d->pos_i64 ? 8 : 4);
}

bool contiguous(const int64_t* stride, int32_t heads, int32_t D) {
    return stride[0] == int64_t(heads) * D && (heads == 1 || stride[1] == D);
}

}  // namespace

extern "C" gdn_status gdn_qk_rotary_fwd(const gdn_rotary_desc* d, const void* q, const void* k, const double* freqs,
                                        const void* positions, const void* q_weight, const void* k_weight,
                                        void* q_out, void* k_out, hipStream_t stream) {
    RotaryArgs a;
    const gdn_status st = check_rotary(d, &a);
    if (st != GDN_OK) return st;
    if (a.tokens > 0 && (!q || !k || !q_out || !k_out || (d->R > 0 && !freqs))) return GDN_ERR_INVALID;
    if (!angles_aligned(d, freqs, positions) || !all_aligned16(q, k, q_weight, k_weight, q_out, k_out)) return GDN_ERR_INVALID;
    if ((q && q_out == q && !contiguous(d->q_stride, d->Hq, d->D)) || (k && k_out == k && !contiguous(d->k_stride, d->Hk, d->D)))
        return GDN_ERR_INVALID;
    a.q = q;
    a.k = k;
    a.freqs = freqs;
    a.positions = positions;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_out = q_out;
    a.k_out = k_out;
    return run(gdn::launch_rotary_fwd(a, stream));
}

extern "C" gdn_status gdn_qk_rotary_bwd(const gdn_rotary_desc* d, const void* q, const void* k, const double* freqs,
                                        const void* positions, const void* q_weight, const void* k_weight,
                                        const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                                        float* dk_weight, void* workspace, size_t* workspace_bytes,
                                        hipStream_t stream) {
    RotaryArgs a;
    gdn_status st = check_rotary(d, &a);
    if (st != GDN_OK) return st;
    const int64_t rows = int64_t(a.workgroups) + gdn::row_sums_rows(a.workgroups);
    bool query = false;
    st = check_workspace(rows * 2 * d->D * 4, workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    if (a.tokens > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk || (d->R > 0 && !freqs))) return GDN_ERR_INVALID;
    if ((q_weight == nullptr) != (dq_weight == nullptr) || (k_weight == nullptr) != (dk_weight == nullptr)) return GDN_ERR_INVALID;
    if (!angles_aligned(d, freqs, positions) ||
        !all_aligned16(q, k, q_weight, k_weight, dq_out, dk_out, dq, dk, dq_weight, dk_weight))
        return GDN_ERR_INVALID;
    a.q = q;
    a.k = k;
    a.freqs = freqs;
    a.positions = positions;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.dq_out = dq_out;
    a.dk_out = dk_out;
    a.dq = dq;
    a.dk = dk;
    a.dq_weight = dq_weight;
    a.dk_weight = dk_weight;
    a.parts = q_weight || k_weight ? static_cast<float*>(workspace) : nullptr;
    return run(gdn::launch_rotary_bwd(a, stream));
}
