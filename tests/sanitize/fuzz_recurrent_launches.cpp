// What the recurrent-state operators' host code hands to the kernels, under
// AddressSanitizer and UndefinedBehaviorSanitizer: random valid calls, with
// launch stubs that keep the launches of a call and check them against it.
// Every tensor has addresses of its own unless a call is made in place;
// nothing may dereference them.
//   - segments cover the sequences: as many as their lengths ask for;
//   - a launch has fewer than 2^32 threads;
//   - no state is replaced while a walk may still read it;
//   - plans never write what they read.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "gdn_recurrent.h"
#include "gdn_recurrent_internal.h"

namespace {
std::mt19937_64 rng(20260417);
int64_t uni(int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(rng); }
int64_t pick(std::initializer_list<int64_t> xs) { return xs.begin()[uni(0, xs.size() - 1)]; }
int64_t log_uni(int64_t lo, int64_t hi) {
    int bits = 0;
    for (int64_t x = hi; x; x >>= 1) ++bits;
    return std::min(hi, std::max(lo, uni(0, (int64_t(1) << uni(0, bits)))));
}

void fail(const char* what) {
    fprintf(stderr, "launch check: %s\n", what);
    abort();
}
template <typename P = void>
P* place(int i) {   // 64 TiB apart
    return reinterpret_cast<P*>(uintptr_t(i + 1) << 46);
}

struct Call {
    const gdn_linattn_desc* d = nullptr;
    int64_t states = 0;   // bytes of all sequences' states
} now;
long launches[7], in_place_calls;

void threads(int64_t blocks, int64_t each) {
    if (blocks < 1 || blocks * each >= int64_t(1) << 32) fail("threads");
}
bool meet(const void* a, const void* b, int64_t bytes) {
    const intptr_t x = (intptr_t)a, y = (intptr_t)b;
    return a && b && x < y + bytes && y < x + bytes;
}
void check_units(const gdn::LaUnits& u, const gdn::LaJobs& j) {
    const gdn_linattn_desc& d = *now.d;
    if (u.seg_tokens < 64 || u.seg_tokens % 64 || j.n < 1 || j.n > gdn::LA_MAX_JOBS) fail("units");
    int64_t n = 0, longest = 0, most = 0;
    const int64_t units = d.n_units ? d.n_units : d.B;
    for (int64_t i = 0; i < units; ++i) {
        const int64_t len = d.n_units ? d.offsets_host[i + 1] - d.offsets_host[i] : d.T;
        const int64_t segs = std::max<int64_t>(1, (len + u.seg_tokens - 1) / u.seg_tokens);
        n += segs;
        most = std::max(most, segs);
        longest = std::max(longest, len);
    }
    if (u.n_units != units || u.dense != (d.n_units == 0) || u.T != d.T || u.total != int64_t(d.B) * d.T) fail("sequences");
    if (u.n_segs != n) fail("segments do not cover the sequences");
    if (longest + u.seg_tokens > INT32_MAX) fail("a segment's end");
    if (u.join && most > 4) fail("long joins");
}
}  // namespace

namespace gdn {
hipError_t launch_la_summary(const LaUnits& u, const LaJobs& j, int, int, int V, hipStream_t) {
    ++launches[0];
    check_units(u, j);
    threads(int64_t(u.n_segs) * u.H * j.n, V == 128 ? 512 : 256);
    return hipSuccess;
}
hipError_t launch_la_merge(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t) {
    ++launches[1];
    check_units(u, j);
    threads(int64_t(u.n_units) * u.H, K * V / 4);
    return hipSuccess;
}
hipError_t launch_la_main(const LaUnits& u, const LaJobs& j, int, int K, int V, hipStream_t) {
    ++launches[2];
    check_units(u, j);
    threads(int64_t(u.n_segs) * u.H * j.n, 256);
    for (int a = 0; a < j.n; ++a) {
        if (j.job[a].K != K && j.job[a].K != V) fail("widths");
        for (int b = 0; b < j.n; ++b) {
            const LaJob &w = j.job[a], &r = j.job[b];
            if (!w.s_out || w.out_pages || r.in_pages || !meet(w.s_out, r.s_in, now.states)) continue;
            const bool reads = !r.slots || u.join;   // else the entry states are in the slots
            if (reads && (a != b || u.join)) fail("a state is replaced while a walk may read it");
        }
    }
    return hipSuccess;
}
hipError_t launch_la_group(const float*, void*, int64_t tokens, int, int h, int D, int, hipStream_t) {
    ++launches[3];
    if (tokens) threads((tokens * h * D / 4 + 255) / 256, 256);
    return hipSuccess;
}
hipError_t launch_step(const StepArgs& a, int, int, hipStream_t) {
    ++launches[4];
    if (a.N) threads(int64_t(a.N) * a.H, 256);
    return hipSuccess;
}
hipError_t launch_pages_copy(const PoolArgs&, const int32_t*, const int32_t*, int, hipStream_t) { return hipSuccess; }
static void plan(std::initializer_list<std::pair<const int32_t*, int64_t>> out,
                 std::initializer_list<std::pair<const int32_t*, int64_t>> in) {
    for (const auto& o : out)
        for (const auto& i : in)
            if (o.second > 0 && i.second > 0 && o.first < i.first + i.second && i.first < o.first + o.second)
                fail("a plan writes what it reads");
}
hipError_t launch_fork(const PoolArgs&, const int32_t* table, const int32_t* parent, int n, const int32_t* spare, int m,
                       int32_t* new_table, int32_t* left, int32_t* ws, hipStream_t) {
    ++launches[5];
    plan({{new_table, n}, {left, n + m}, {ws, 1 + 2 * n}}, {{table, n}, {parent, n}, {spare, m}});
    return hipSuccess;
}
hipError_t launch_compact(const PoolArgs& p, const int32_t* table, int n, int32_t* new_table, int32_t* count,
                          int32_t* ws, hipStream_t) {
    ++launches[6];
    plan({{new_table, n}, {count, 1}, {ws, 1 + 2 * p.src_pages}}, {{table, n}});
    return hipSuccess;
}
}  // namespace gdn

namespace {
void declared(gdn_status s) {
    if (s != GDN_OK && s != GDN_ERR_INVALID && s != GDN_ERR_UNSUPPORTED) fail("status");
}

void prompt(bool bwd) {
    gdn_linattn_desc d;
    memset(&d, 0, sizeof(d));
    d.H = (int32_t)pick({1, 2, 6, 8, 16, 32, 64});
    d.Hq = (int32_t)pick({1, d.H, d.H});
    d.Hk = (int32_t)pick({1, d.H, d.H});
    d.Hv = (int32_t)pick({1, d.H, d.H});
    d.K = (int32_t)pick({64, 128});
    d.V = (int32_t)pick({64, 128});
    d.dtype = (int32_t)uni(0, 1);
    d.o_dtype = (int32_t)uni(0, 1);
    d.scale = 0.1f;
    int64_t* strides[] = {d.q_stride, d.k_stride, d.v_stride};
    const int32_t heads[] = {d.Hq, d.Hk, d.Hv}, widths[] = {d.K, d.K, d.V};
    for (int i = 0; i < 3; ++i) {
        strides[i][0] = int64_t(heads[i]) * widths[i];
        strides[i][1] = widths[i];
    }
    std::vector<int32_t> offs;
    if (uni(0, 1)) {
        d.B = 1;
        d.n_units = (int32_t)log_uni(1, 300);
        offs.push_back(0);
        const int64_t most = pick({3, 100, 5000, 300000});
        for (int i = 0; i < d.n_units; ++i) offs.push_back(offs.back() + (int32_t)log_uni(1, most));
        d.T = offs.back();
        d.offsets_host = offs.data();
        d.offsets_dev = place<int32_t>(0);
    } else {
        d.B = (int32_t)log_uni(1, int64_t(1) << uni(0, 21));
        d.T = (int32_t)log_uni(0, std::max<int64_t>(1, (int64_t(1) << 31) / d.B / d.H));
    }
    now.d = &d;
    now.states = int64_t(d.n_units ? d.n_units : d.B) * d.H * d.K * d.V * 4;
    const int over = (int)uni(0, 3);   // the state that is replaced: none, dht (s_in), s_in
    float* s_in = uni(0, 3) ? place<float>(1) : nullptr;
    float* dht = uni(0, 3) ? place<float>(2) : nullptr;
    float* out = over == 1 && bwd && dht ? dht : over && s_in ? s_in : place<float>(3);
    in_place_calls += out != place<float>(3);
    auto call = [&](void* ws, size_t* n) {
        return bwd ? gdn_linattn_bwd(&d, place(4), place(5), place(6), place<float>(7), s_in, place(8), dht, place(9),
                                     place(10), place(11), out, ws, n, nullptr)
                   : gdn_linattn_fwd(&d, place(4), place(5), place(6), place<float>(7), s_in, nullptr, out, nullptr, 0,
                                     place(8), ws, n, nullptr);
    };
    size_t need = 0;
    const gdn_status st = call(nullptr, &need);
    declared(st);
    if (st == GDN_OK && call(place(12), &need) != GDN_OK) fail("a valid call is refused");
}

void step() {
    gdn_step_desc d;
    memset(&d, 0, sizeof(d));
    d.N = (int32_t)log_uni(0, int64_t(1) << uni(0, 28));
    d.H = d.Hq = d.Hk = d.Hv = (int32_t)pick({1, 8, 32, 64});
    d.K = d.V = 128;
    d.dtype = d.o_dtype = 1;
    d.scale = 1;
    d.n_pages = 1;
    for (int64_t* s : {d.q_stride, d.k_stride, d.v_stride}) {
        s[0] = int64_t(d.H) * 128;
        s[1] = 128;
    }
    declared(gdn_linattn_step(&d, place(0), place(1), place(2), place<float>(3), place<int32_t>(4), place<float>(5),
                              place(6), nullptr));
}

void plans() {
    const int n = (int)log_uni(0, 2000), m = (int)log_uni(0, 600), pages = (int)log_uni(1, 5000);
    int32_t* b[7];   // near each other: most calls overlap somewhere
    for (int32_t*& p : b) p = place<int32_t>(0) + uni(0, 40000);
    declared(gdn_pages_fork(place(1), 1, pages, 16, b[0], b[1], n, b[2], m, b[3], b[4], b[5], nullptr));
    declared(gdn_pages_compact(place(1), 1, pages, 16, b[0], n, b[3], b[4], b[5], nullptr));
}
}  // namespace

int main() {
    for (int i = 0; i < 40000; ++i) {
        prompt(i & 1);
        step();
        plans();
    }
    printf("launches: summary %ld merge %ld main %ld group %ld step %ld fork %ld compact %ld; in place %ld\n", launches[0],
           launches[1], launches[2], launches[3], launches[4], launches[5], launches[6], in_place_calls);
    for (long n : launches)
        if (n < 1000) return 2;
    return in_place_calls < 1000 ? 2 : 0;
}
