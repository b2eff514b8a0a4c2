// Host side of the recurrent-state operators (include/gdn_recurrent.h):
// argument validation, workspace layout and launch order. Every check runs
// before the first HIP call, so a rejected call enqueues nothing and the
// checks can be exercised without a GPU.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>

#include "gdn_recurrent.h"
#include "gdn_recurrent_internal.h"

namespace {

using gdn::LaJob;
using gdn::LaJobs;
using gdn::LaUnits;
using gdn::RowsOf;

constexpr int64_t kMaxElems = int64_t(1) << 40;   // sanity bound on any tensor
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 256;   // of a launch along x, in workgroups of 256
constexpr int kChunk = 64;
// With at most this many segments in a sequence each walk adds up those before
// its own instead of a merge in front of all (B=4 T=4096 H=16 in 4: 117 to 108
// us, its gradients 246 to 233; in 8 the longest sum takes as long as the
// merge: B=2, 65 and 63; fp32 T=1000 H=32 60 and 66).
constexpr int kJoin = 4;

int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

struct Range {
    const void* p;
    uint64_t bytes;
};

bool overlap(const Range& a, const Range& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

// whether what a call writes is apart from what it reads and else writes
bool apart(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    for (const Range* w = written.begin(); w != written.end(); ++w) {
        for (const Range& r : read)
            if (overlap(*w, r)) return false;
        for (const Range* x = w + 1; x != written.end(); ++x)
            if (overlap(*w, *x)) return false;
    }
    return true;
}

bool width_ok(int32_t w) { return w == 64 || w == 128; }

bool dtype_ok(int32_t d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

int64_t elem_bytes(int32_t d) { return d == GDN_DTYPE_BF16 ? 2 : 4; }

// distances that keep every row 16-byte aligned and any offset below 2^62
bool strides_ok(const int64_t* s, int64_t rows, int64_t heads, int32_t dtype) {
    const int64_t lim = int64_t(1) << 60;
    for (int i = 0; i < 2; ++i) {
        if (s[i] < 0 || s[i] > lim || s[i] * elem_bytes(dtype) % 16 != 0) return false;
        const int64_t n = i == 0 ? rows : heads;
        if (n > 0 && s[i] > lim / n) return false;
    }
    return true;
}

// ------------------------------------------------------------------ prompts
struct Prompt {
    LaUnits u;
    int64_t tokens, longest, chunks;
    bool cut;      // some sequence has more than one segment
};

// segments of at most seg chunks
int64_t segments(const gdn_linattn_desc* d, const LaUnits& u, int64_t seg) {
    const int64_t tokens = seg * kChunk;
    auto of = [&](int64_t len) { return len > 0 ? (len + tokens - 1) / tokens : 1; };
    if (u.dense) return of(d->T) * u.n_units;
    int64_t n = 0;
    for (int32_t i = 0; i < u.n_units; ++i) n += of(int64_t(d->offsets_host[i + 1]) - d->offsets_host[i]);
    return n;
}

// About how long n segments of at most seg chunks take. One workgroup's chunk
// is 2.9 us (fp32 7) and its sum of k v^T 1.5 (2.5) with few at work; all units
// together do a chunk in a 200th of that (each is slower then: 4.2 us, fp32
// 12.2, one workgroup a unit). The last segments to start leave units idle for
// about 0.6 of a segment. A cut costs a launch of 5 us, 4 more for a merge,
// and its states, 64 KiB each for K = V = 128, about 6 TB/s. Whether to cut at
// all is decided by it, which matters where a few chunks are walked before a
// second launch has begun (measured whole and cut: bf16 H=8 T=192 13.2 and
// 16.8 us, fp32 T=128 19.4 and 22.2, 12 prompts T=4096 37 and 44; gradients,
// bf16 H=32 T=320 19 and 34, B=4 T=512 H=16 39 and 54; forward T=512 H=8 about
// 28 and 21).
double micros(const gdn_linattn_desc* d, const LaUnits& u, int walks, int64_t work, int64_t seg, int64_t n) {
    const bool f32 = d->dtype == GDN_DTYPE_F32;
    const double walk = f32 ? 7.0 : 2.9, sum = f32 ? 2.5 : 1.5;
    const int sums = walks > 1 ? 2 : 1;   // states of the forward, and of its gradients
    double t = fmax(seg * walk, work * walk / 200 + 0.6 * seg * walk);
    if (n > u.n_units) {
        const double parts = double(n) / u.n_units;
        const bool join = parts <= kJoin;
        t += (join ? 5 : 9) + fmax(seg * sum, double(n - u.n_units) * seg * d->H * sums * sum / 200);
        t += double(n) * d->H * d->K * d->V * 4 * (sums + (join ? walks * (parts - 1) / 2 : 2 * sums + walks)) / 6e6;
    }
    return t;
}

// walks: of every sequence, in one launch
gdn_status check_prompt(const gdn_linattn_desc* d, int walks, Prompt* p) {
    if (d == nullptr) return GDN_ERR_INVALID;
    if (!width_ok(d->K) || !width_ok(d->V)) return GDN_ERR_UNSUPPORTED;
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->Hq < 1 || d->Hk < 1 || d->Hv < 1) return GDN_ERR_INVALID;
    if (d->H % d->Hq || d->H % d->Hk || d->H % d->Hv) return GDN_ERR_INVALID;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->o_dtype) || !isfinite(d->scale)) return GDN_ERR_INVALID;
    memset(p, 0, sizeof(*p));
    p->tokens = int64_t(d->B) * d->T;
    if (p->tokens * d->H > kMaxElems / 128) return GDN_ERR_INVALID;
    if (!strides_ok(d->q_stride, p->tokens, d->Hq, d->dtype) || !strides_ok(d->k_stride, p->tokens, d->Hk, d->dtype) ||
        !strides_ok(d->v_stride, p->tokens, d->Hv, d->dtype))
        return GDN_ERR_INVALID;
    // a chunk's rows are reached by 32-bit offsets
    const int64_t span = (int64_t(1) << 31) / kChunk;
    const int64_t es = elem_bytes(d->dtype);
    if (int64_t(d->H) * 128 * 4 > span || d->q_stride[0] * es > span || d->k_stride[0] * es > span ||
        d->v_stride[0] * es > span)
        return GDN_ERR_UNSUPPORTED;
    LaUnits& u = p->u;
    u.H = d->H;
    u.T = d->T;
    u.total = p->tokens;
    if (d->n_units < 0) return GDN_ERR_INVALID;
    if (d->n_units == 0) {
        u.dense = 1;
        u.n_units = d->B;
        p->longest = d->T;
        p->chunks = int64_t(d->B) * ((d->T + int64_t(kChunk) - 1) / kChunk);
    } else {
        if (d->B != 1 || !d->offsets_host || !d->offsets_dev) return GDN_ERR_INVALID;
        const int32_t* o = d->offsets_host;
        if (o[0] != 0 || o[d->n_units] != p->tokens) return GDN_ERR_INVALID;
        for (int32_t i = 0; i < d->n_units; ++i) {
            if (o[i] >= o[i + 1]) return GDN_ERR_INVALID;
            const int64_t len = int64_t(o[i + 1]) - o[i];
            p->longest = len > p->longest ? len : p->longest;
            p->chunks += (len + kChunk - 1) / kChunk;
        }
        u.n_units = d->n_units;
        u.offsets = d->offsets_dev;
    }
    // Segments, in chunks. A workgroup alone on its compute unit walks nearly
    // as fast as two together, and every cut costs states between the parts.
    // Rows of one length: as many equal parts as 256 workgroups have room for
    // (B=4 T=4096 H=16 bf16: 114 us at 256 and 111 at 512; T=4096 H=16 45 and
    // 52, its gradients 81 and 100; fp32 T=1000 H=32 60 and 66; T=3000, B=3
    // H=16, 288 workgroups 94 and 240 of them 78).
    // Packed sequences run longest first, and the work of all walks of a launch
    // levels itself unless one sequence is longer than about a compute unit's
    // share: then none is cut (20 prompts, T=32768 H=16, longest 1.35 shares:
    // 204 us whole, 229 and 219 with 256 and 512 parts; gradients of 12
    // documents, T=16384 H=16, 0.84: 222, 266 and 272). Beyond that parts of
    // half a share, which fill both places of a unit (5 prompts, T=32768 H=16:
    // 213, in parts of a share 225; 3 prompts, T=9000 H=32: 116 and 126; fp32 gradients
    // of 7 documents, T=3001 H=8: 105, at a third of a share 116).
    // At least two chunks, or one where a chunk's products take fp32 MFMA's
    // time (B=1 T=2048 H=8 at 1, 2 and 4 chunks: bf16 40, 34 and 38 us, fp32
    // 47, 55 and 85 us).
    const int64_t longest = (p->longest + kChunk - 1) / kChunk, work = p->chunks * d->H * walks;
    const int64_t least = d->dtype == GDN_DTYPE_F32 ? 1 : 2;
    int64_t seg = longest;
    if (u.dense) {
        const int64_t parts = 256 / (int64_t(u.n_units) * d->H);
        if (parts > 1) seg = (longest + parts - 1) / parts;
    } else if (longest * 256 * 5 > work * 7) {
        seg = (work + 511) / 512;
    }
    if (seg < least) seg = least;
    int64_t n = segments(d, u, seg);
    if (n > u.n_units && micros(d, u, walks, work, longest, u.n_units) <= micros(d, u, walks, work, seg, n)) {
        seg = longest;
        n = u.n_units;
    }
    u.seg_tokens = (int32_t)(seg * kChunk);
    if (seg * kChunk + p->longest > INT32_MAX) return GDN_ERR_UNSUPPORTED;   // a segment's end is an int
    p->cut = n > u.n_units;
    u.join = p->cut && (longest + seg - 1) / seg <= kJoin;
    // threads for a segment's head: la_main 256 for each walk, la_summary up to 512 for each kind of
    // state; la_merge one for four values of a sequence's state
    const int64_t each = walks > 1 ? (p->cut ? 1024 : 768) : (p->cut ? 512 : 256);
    if (n * d->H * each > kMaxThreads) return GDN_ERR_UNSUPPORTED;
    if (p->cut && int64_t(u.n_units) * d->H * (d->K * d->V / 4) > kMaxThreads) return GDN_ERR_UNSUPPORTED;
    u.n_segs = (int32_t)n;
    return GDN_OK;
}

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

int64_t slot_bytes(const Prompt& p, const gdn_linattn_desc* d) {
    return p.cut ? align256(int64_t(p.u.n_segs) * d->H * d->K * d->V * 4) : 0;
}

RowsOf rows(const void* ptr, const int64_t* stride, int32_t share) { return RowsOf{ptr, stride[0], stride[1], share}; }

// contiguous [tokens][h][W]
RowsOf rows(const void* ptr, int32_t h, int32_t W) { return RowsOf{ptr, int64_t(h) * W, W, 1}; }

gdn_status run(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_DEVICE; }

}  // namespace

extern "C" gdn_status gdn_linattn_fwd(const gdn_linattn_desc* d, const void* q, const void* k, const void* v,
                                      const float* decay, const float* s_in, const int32_t* in_pages, float* s_out,
                                      const int32_t* out_pages, int32_t n_pages, void* o, void* workspace,
                                      size_t* workspace_bytes, hipStream_t stream) {
    Prompt p;
    gdn_status st = check_prompt(d, 1, &p);
    if (st != GDN_OK) return st;
    bool query = false;
    st = check_workspace(slot_bytes(p, d), workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    if (!decay || (p.tokens > 0 && (!q || !k || !v || !o))) return GDN_ERR_INVALID;
    if (n_pages < 0 || (in_pages && !s_in) || (out_pages && !s_out)) return GDN_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(s_in) || !aligned16(s_out))
        return GDN_ERR_INVALID;
    p.u.n_pages = n_pages;
    p.u.decay = decay;
    LaJobs jobs;
    memset(&jobs, 0, sizeof(jobs));
    jobs.n = 1;
    LaJob& j = jobs.job[0];
    j.q = rows(q, d->q_stride, d->H / d->Hq);
    j.k = rows(k, d->k_stride, d->H / d->Hk);
    j.v = rows(v, d->v_stride, d->H / d->Hv);
    j.s_in = s_in;
    j.in_pages = in_pages;
    j.s_out = s_out;
    j.out_pages = out_pages;
    j.K = d->K;
    j.e = 1;
    j.o_f32 = d->o_dtype == GDN_DTYPE_F32;
    j.o = o;
    j.s_p = j.s_o = d->scale;
    j.s_w = 1.0f;
    // a sequence's last segment may replace the state before its others have
    // read it: where the two share memory the merge reads it in front of all
    if (s_in && s_out) {
        const int64_t page = int64_t(d->H) * d->K * d->V;
        const float *in_end = s_in + page * (in_pages ? n_pages : p.u.n_units),
                    *out_end = s_out + page * (out_pages ? n_pages : p.u.n_units);
        if (s_in < out_end && s_out < in_end) p.u.join = 0;
    }
    if (p.cut) {
        j.slots = static_cast<float*>(workspace);
        if (gdn::launch_la_summary(p.u, jobs, d->dtype, d->K, d->V, stream) != hipSuccess) return GDN_ERR_DEVICE;
        if (!p.u.join && gdn::launch_la_merge(p.u, jobs, d->K, d->V, stream) != hipSuccess) return GDN_ERR_DEVICE;
    }
    return run(gdn::launch_la_main(p.u, jobs, d->dtype, d->K, d->V, stream));
}

extern "C" gdn_status gdn_linattn_bwd(const gdn_linattn_desc* d, const void* q, const void* k, const void* v,
                                      const float* decay, const float* s_in, const void* dout, const float* dht,
                                      void* dq, void* dk, void* dv, float* dh0, void* workspace,
                                      size_t* workspace_bytes, hipStream_t stream) {
    Prompt p;
    gdn_status st = check_prompt(d, 3, &p);
    if (st != GDN_OK) return st;
    // la_group has a thread for four values of a shared head
    if ((d->Hq < d->H && p.tokens * d->Hq * (d->K / 4) > kMaxThreads) ||
        (d->Hk < d->H && p.tokens * d->Hk * (d->K / 4) > kMaxThreads) ||
        (d->Hv < d->H && p.tokens * d->Hv * (d->V / 4) > kMaxThreads))
        return GDN_ERR_UNSUPPORTED;
    // slots of S and of its gradient, then the per-head gradients of shared heads
    const int64_t slots = slot_bytes(p, d);
    auto part_bytes = [&](int32_t h, int32_t W) {
        return h == d->H ? int64_t(0) : align256(p.tokens * d->H * W * 4);
    };
    const int64_t bq = part_bytes(d->Hq, d->K), bk = part_bytes(d->Hk, d->K), bv = part_bytes(d->Hv, d->V);
    bool query = false;
    st = check_workspace(2 * slots + bq + bk + bv, workspace, workspace_bytes, &query);
    if (st != GDN_OK || query) return st;
    if (!decay || (p.tokens > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv))) return GDN_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(s_in) || !aligned16(dht) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dh0))
        return GDN_ERR_INVALID;
    // dh0 may be dht or s_in, which the other walks of its launch read: then a
    // merge reads them in front of all, or dh0's walk comes after the others
    const uint64_t states = uint64_t(p.u.n_units) * d->H * d->K * d->V * 4;
    const bool over_dht = overlap({dh0, states}, {dht, states}), over_s_in = overlap({dh0, states}, {s_in, states});
    if ((over_dht && dh0 != dht) || (over_s_in && dh0 != s_in)) return GDN_ERR_INVALID;
    const bool last = (over_dht || over_s_in) && !p.cut;
    if (over_dht || over_s_in) p.u.join = 0;
    p.u.decay = decay;
    char* base = static_cast<char*>(workspace);
    float* s_slots = p.cut ? reinterpret_cast<float*>(base) : nullptr;
    float* d_slots = p.cut ? reinterpret_cast<float*>(base + slots) : nullptr;
    float* pq = bq ? reinterpret_cast<float*>(base + 2 * slots) : nullptr;
    float* pk = bk ? reinterpret_cast<float*>(base + 2 * slots + bq) : nullptr;
    float* pv = bv ? reinterpret_cast<float*>(base + 2 * slots + bq + bk) : nullptr;
    const RowsOf rq = rows(q, d->q_stride, d->H / d->Hq), rk = rows(k, d->k_stride, d->H / d->Hk),
                 rv = rows(v, d->v_stride, d->H / d->Hv), rd = rows(dout, d->H, d->V);
    const int32_t f32 = d->dtype == GDN_DTYPE_F32;

    // dq_i = scale [sum_{j <= i} d^{i-j} (do_i . v_j) k_j + d^{i+1} S do_i]
    LaJob jq;
    memset(&jq, 0, sizeof(jq));
    jq.q = rd;
    jq.k = rv;
    jq.v = rk;
    jq.s_in = s_in;
    jq.slots = s_slots;
    jq.transposed = 1;
    jq.e = 1;
    jq.o = pq ? pq : dq;
    jq.o_f32 = pq || f32;
    jq.s_p = jq.s_o = d->scale;
    jq.s_w = 1.0f;
    // dk_j = sum_{i >= j} d^{i-j} scale (v_j . do_i) q_i + d^{T-1-j} D v_j, D the gradient arriving
    // at the end; in reversed time D's power starts at 0
    LaJob jk;
    memset(&jk, 0, sizeof(jk));
    jk.q = rv;
    jk.k = rd;
    jk.v = rq;
    jk.s_in = dht;
    jk.slots = d_slots;
    jk.transposed = 1;
    jk.rev = 1;
    jk.o = pk ? pk : dk;
    jk.o_f32 = pk || f32;
    jk.s_p = jk.s_w = d->scale;
    jk.s_o = 1.0f;
    // dv_j = sum_{i >= j} d^{i-j} scale (k_j . q_i) do_i + d^{T-1-j} D^T k_j; its state ends as dh0
    LaJob jv;
    memset(&jv, 0, sizeof(jv));
    jv.q = rk;
    jv.k = rq;
    jv.v = rd;
    jv.s_in = dht;
    jv.s_out = dh0;
    jv.slots = d_slots;
    jv.rev = 1;
    jv.o = pv ? pv : dv;
    jv.o_f32 = pv || f32;
    jv.s_p = jv.s_w = d->scale;
    jv.s_o = 1.0f;

    LaJobs jobs;
    memset(&jobs, 0, sizeof(jobs));
    if (p.cut) {
        jobs.n = 2;
        LaJob& a = jobs.job[0];   // the forward states
        a.k = rk;
        a.v = rv;
        a.s_in = s_in;
        a.slots = s_slots;
        a.e = 1;
        a.s_w = 1.0f;
        jobs.job[1] = jv;         // their gradients
        if (gdn::launch_la_summary(p.u, jobs, d->dtype, d->K, d->V, stream) != hipSuccess) return GDN_ERR_DEVICE;
        if (!p.u.join && gdn::launch_la_merge(p.u, jobs, d->K, d->V, stream) != hipSuccess) return GDN_ERR_DEVICE;
    }
    jq.K = jk.K = d->V;
    jv.K = d->K;
    jobs.job[0] = jq;
    jobs.job[1] = jk;
    jobs.job[2] = jv;
    jobs.n = last ? 2 : 3;
    if (gdn::launch_la_main(p.u, jobs, d->dtype, d->V, d->K, stream) != hipSuccess) return GDN_ERR_DEVICE;
    if (last) {
        jobs.job[0] = jv;
        jobs.n = 1;
        if (gdn::launch_la_main(p.u, jobs, d->dtype, d->K, d->V, stream) != hipSuccess) return GDN_ERR_DEVICE;
    }
    if (pq && gdn::launch_la_group(pq, dq, p.tokens, d->H, d->Hq, d->K, d->dtype, stream) != hipSuccess)
        return GDN_ERR_DEVICE;
    if (pk && gdn::launch_la_group(pk, dk, p.tokens, d->H, d->Hk, d->K, d->dtype, stream) != hipSuccess)
        return GDN_ERR_DEVICE;
    if (pv && gdn::launch_la_group(pv, dv, p.tokens, d->H, d->Hv, d->V, d->dtype, stream) != hipSuccess)
        return GDN_ERR_DEVICE;
    return GDN_OK;
}

// ------------------------------------------------------------------ single tokens
namespace {

gdn_status check_step(const gdn_step_desc* d, const void* q, const void* k, const void* v, const int32_t* pages,
                      float* state, void* o, gdn::StepArgs* a) {
    if (d == nullptr) return GDN_ERR_INVALID;
    if (!width_ok(d->K) || !width_ok(d->V)) return GDN_ERR_UNSUPPORTED;
    if (d->N < 0 || d->H < 1 || d->Hq < 1 || d->Hk < 1 || d->Hv < 1 || d->n_pages < 0) return GDN_ERR_INVALID;
    if (d->H % d->Hq || d->H % d->Hk || d->H % d->Hv) return GDN_ERR_INVALID;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->o_dtype) || !isfinite(d->scale)) return GDN_ERR_INVALID;
    if (int64_t(d->N) * d->H * 256 > kMaxThreads) return GDN_ERR_UNSUPPORTED;   // a workgroup a state
    if (int64_t(d->n_pages) * d->H > kMaxElems / (128 * 128)) return GDN_ERR_INVALID;
    if (!strides_ok(d->q_stride, d->N, d->Hq, d->dtype) || !strides_ok(d->k_stride, d->N, d->Hk, d->dtype) ||
        !strides_ok(d->v_stride, d->N, d->Hv, d->dtype))
        return GDN_ERR_INVALID;
    if (d->N > 0 && (!q || !k || !v || !o || (d->n_pages > 0 && !state))) return GDN_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(state)) return GDN_ERR_INVALID;
    memset(a, 0, sizeof(*a));
    a->N = d->N;
    a->H = d->H;
    a->n_pages = d->n_pages;
    a->dtype = d->dtype;
    a->o_dtype = d->o_dtype;
    a->scale = d->scale;
    a->q = rows(q, d->q_stride, d->H / d->Hq);
    a->k = rows(k, d->k_stride, d->H / d->Hk);
    a->v = rows(v, d->v_stride, d->H / d->Hv);
    a->pages = pages;
    a->state = state;
    a->o = o;
    return GDN_OK;
}

}  // namespace

extern "C" gdn_status gdn_linattn_step(const gdn_step_desc* d, const void* q, const void* k, const void* v,
                                       const float* decay, const int32_t* pages, float* state, void* o,
                                       hipStream_t stream) {
    gdn::StepArgs a;
    const gdn_status st = check_step(d, q, k, v, pages, state, o, &a);
    if (st != GDN_OK) return st;
    if (!decay) return GDN_ERR_INVALID;
    a.decay = decay;
    return run(gdn::launch_step(a, d->K, d->V, stream));
}

extern "C" gdn_status gdn_recurrent_step(const gdn_step_desc* d, int32_t gate_kind, int32_t use_exp2, const void* q,
                                         const void* k, const void* v, const float* g, const void* beta,
                                         const int32_t* pages, float* state, void* o, int32_t flags,
                                         hipStream_t stream) {
    gdn::StepArgs a;
    const gdn_status st = check_step(d, q, k, v, pages, state, o, &a);
    if (st != GDN_OK) return st;
    if (d->K != 128 || d->V != 128) return GDN_ERR_UNSUPPORTED;
    if (gate_kind != GDN_GATE_SCALAR && gate_kind != GDN_GATE_PER_KEY) return GDN_ERR_INVALID;
    if (use_exp2 != 0 && use_exp2 != 1) return GDN_ERR_INVALID;
    if (flags & ~(GDN_FLAG_QK_L2NORM | GDN_FLAG_BETA_SIGMOID)) return GDN_ERR_INVALID;
    if (d->N > 0 && (!g || !beta)) return GDN_ERR_INVALID;
    a.g = g;
    a.beta = beta;
    a.kind = gate_kind == GDN_GATE_PER_KEY ? 2 : 1;
    a.use_exp2 = use_exp2;
    a.qk_norm = (flags & GDN_FLAG_QK_L2NORM) != 0;
    a.beta_sig = (flags & GDN_FLAG_BETA_SIGMOID) != 0;
    return run(gdn::launch_step(a, d->K, d->V, stream));
}

// ------------------------------------------------------------------ pages
namespace {

gdn_status check_pool(const void* pool, int32_t n_layers, int32_t n_pages, int64_t page_bytes) {
    if (n_layers < 0 || n_pages < 0 || page_bytes < 16 || page_bytes % 16 != 0) return GDN_ERR_INVALID;
    if (page_bytes > (kMaxElems * 16) / (int64_t(n_layers) * n_pages + 1)) return GDN_ERR_INVALID;
    if (int64_t(n_layers) * n_pages > 0 && !pool) return GDN_ERR_INVALID;
    return aligned16(pool) ? GDN_OK : GDN_ERR_INVALID;
}

}  // namespace

extern "C" size_t gdn_pages_workspace_ints(int32_t n) { return 1 + 2 * (size_t)(n > 0 ? n : 0); }

// Every workgroup of a small fork or compaction makes its own plan from the
// inputs while the first one writes the outputs, so none of these may be an
// input.
static Range ints(const int32_t* p, int64_t n) { return Range{p, 4 * (uint64_t)n}; }

extern "C" gdn_status gdn_pages_copy(void* dst_pool, int32_t dst_n_pages, const void* src_pool, int32_t src_n_pages,
                                     int32_t n_layers, int64_t page_bytes, const int32_t* dst_pages,
                                     const int32_t* src_pages, int32_t n, hipStream_t stream) {
    gdn_status st = check_pool(dst_pool, n_layers, dst_n_pages, page_bytes);
    if (st == GDN_OK) st = check_pool(src_pool, n_layers, src_n_pages, page_bytes);
    if (st != GDN_OK) return st;
    if (n < 0 || (n > 0 && (!dst_pages || !src_pages))) return GDN_ERR_INVALID;
    const gdn::PoolArgs a{static_cast<char*>(dst_pool), static_cast<const char*>(src_pool), n_layers, dst_n_pages,
                          src_n_pages, page_bytes};
    return run(gdn::launch_pages_copy(a, dst_pages, src_pages, n, stream));
}

extern "C" gdn_status gdn_pages_fork(void* pool, int32_t n_layers, int32_t n_pages, int64_t page_bytes,
                                     const int32_t* table, const int32_t* parent, int32_t n_slots,
                                     const int32_t* spare, int32_t n_spare, int32_t* new_table, int32_t* left,
                                     int32_t* workspace, hipStream_t stream) {
    const gdn_status st = check_pool(pool, n_layers, n_pages, page_bytes);
    if (st != GDN_OK) return st;
    if (n_slots < 0 || n_spare < 0) return GDN_ERR_INVALID;
    if (n_slots > gdn::FORK_MAX || n_spare > gdn::FORK_MAX) return GDN_ERR_UNSUPPORTED;
    if (n_slots > 0 && (!table || !parent || !new_table)) return GDN_ERR_INVALID;
    if ((n_spare > 0 && !spare) || (n_slots + n_spare > 0 && !left) || !workspace) return GDN_ERR_INVALID;
    if (!apart({ints(new_table, n_slots), ints(left, n_slots + n_spare),
                ints(workspace, (int64_t)gdn_pages_workspace_ints(n_slots))},
               {ints(table, n_slots), ints(parent, n_slots), ints(spare, n_spare)}))
        return GDN_ERR_INVALID;
    const gdn::PoolArgs a{static_cast<char*>(pool), static_cast<const char*>(pool), n_layers, n_pages, n_pages,
                          page_bytes};
    return run(gdn::launch_fork(a, table, parent, n_slots, spare, n_spare, new_table, left, workspace, stream));
}

extern "C" gdn_status gdn_pages_compact(void* pool, int32_t n_layers, int32_t n_pages, int64_t page_bytes,
                                        const int32_t* table, int32_t n_slots, int32_t* new_table, int32_t* count,
                                        int32_t* workspace, hipStream_t stream) {
    const gdn_status st = check_pool(pool, n_layers, n_pages, page_bytes);
    if (st != GDN_OK) return st;
    if (n_slots < 0) return GDN_ERR_INVALID;
    if (n_pages > gdn::COMPACT_MAX) return GDN_ERR_UNSUPPORTED;
    if (n_slots > 0 && (!table || !new_table)) return GDN_ERR_INVALID;
    if (!count || !workspace) return GDN_ERR_INVALID;
    if (!apart({ints(new_table, n_slots), ints(count, 1),
                ints(workspace, (int64_t)gdn_pages_workspace_ints(n_pages))},
               {ints(table, n_slots)}))
        return GDN_ERR_INVALID;
    const gdn::PoolArgs a{static_cast<char*>(pool), static_cast<const char*>(pool), n_layers, n_pages, n_pages,
                          page_bytes};
    return run(gdn::launch_compact(a, table, n_slots, new_table, count, workspace, stream));
}
