// Host-side fuzz of the recurrent-state operators' C ABI under
// AddressSanitizer and UndefinedBehaviorSanitizer: random descriptors,
// offsets, strides, sizes and pointers. The launch functions are stubs that
// check what the host code hands them: regions inside the workspace, a segment
// at least for each sequence. Input pointers are fake addresses that nothing may
// dereference. Exit status 0 when every call returned a declared status.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "gdn_recurrent.h"
#include "gdn_recurrent_internal.h"

namespace {
std::mt19937_64 rng(20261206);
int pick(std::initializer_list<int> xs) {
    return *(xs.begin() + std::uniform_int_distribution<size_t>(0, xs.size() - 1)(rng));
}
int uni(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
bool rarely() { return uni(0, 19) == 0; }

char* const FAKE = reinterpret_cast<char*>(uintptr_t(1) << 40);
template <typename P = void>
P* fake() {   // sometimes NULL, sometimes misaligned
    return rarely() ? nullptr : reinterpret_cast<P*>(FAKE + (rarely() ? 4 : 0));
}
long counts[6], launches;
std::vector<char> workspace(1 << 20);
const char* region_lo = nullptr;
size_t region_bytes = 0;

void fail(const char* what) {
    fprintf(stderr, "recurrent stub: %s\n", what);
    abort();
}
void tally(gdn_status s) {
    if (s < GDN_OK || s > GDN_ERR_CAPACITY) fail("undeclared status");
    counts[s]++;
}
void in_workspace(const void* p, int64_t bytes, const char* what) {
    const char* c = static_cast<const char*>(p);
    if (c < region_lo || bytes < 0 || c + bytes > region_lo + region_bytes || (uintptr_t)c % 256) fail(what);
}
}  // namespace

namespace gdn {
static void check_units(const LaUnits& u, const LaJobs& j, int K, int V) {
    ++launches;
    if (u.H < 1 || u.n_units < 1 || u.n_segs < u.n_units || u.seg_tokens < 64 || u.seg_tokens % 64) fail("units");
    if (j.n < 1 || j.n > LA_MAX_JOBS) fail("jobs");
    for (int i = 0; i < j.n; ++i)
        if (j.job[i].slots) in_workspace(j.job[i].slots, int64_t(u.n_segs) * u.H * K * V * 4, "slots");
}
hipError_t launch_la_summary(const LaUnits& u, const LaJobs& j, int, int K, int V, hipStream_t) {
    check_units(u, j, K, V);
    for (int i = 0; i < j.n; ++i)
        if (!j.job[i].slots) fail("summary without slots");
    return hipSuccess;
}
hipError_t launch_la_merge(const LaUnits& u, const LaJobs& j, int K, int V, hipStream_t) {
    check_units(u, j, K, V);
    return hipSuccess;
}
hipError_t launch_la_main(const LaUnits& u, const LaJobs& j, int, int K, int V, hipStream_t) {
    check_units(u, j, K, V);
    return hipSuccess;
}
hipError_t launch_la_group(const float* x, void*, int64_t tokens, int H, int h, int D, int, hipStream_t) {
    if (H % h || h == H) fail("group");
    in_workspace(x, tokens * H * D * 4, "per-head gradients");
    return hipSuccess;
}
hipError_t launch_step(const StepArgs& a, int K, int V, hipStream_t) {
    if (a.N < 0 || a.H < 1 || (K != 64 && K != 128) || (V != 64 && V != 128)) fail("step");
    if (a.kind && (K != 128 || V != 128)) fail("delta step widths");
    return hipSuccess;
}
static void check_pool(const PoolArgs& p) {
    if (p.page_bytes < 16 || p.page_bytes % 16 || p.n_layers < 0 || p.dst_pages < 0 || p.src_pages < 0) fail("pool");
}
hipError_t launch_pages_copy(const PoolArgs& p, const int32_t*, const int32_t*, int n, hipStream_t) {
    check_pool(p);
    if (n < 0) fail("pairs");
    return hipSuccess;
}
hipError_t launch_fork(const PoolArgs& p, const int32_t*, const int32_t*, int n, const int32_t*, int m, int32_t*,
                       int32_t*, int32_t*, hipStream_t) {
    check_pool(p);
    if (n < 0 || n > FORK_MAX || m < 0 || m > FORK_MAX) fail("fork sizes");
    return hipSuccess;
}
hipError_t launch_compact(const PoolArgs& p, const int32_t*, int n, int32_t*, int32_t*, int32_t*, hipStream_t) {
    check_pool(p);
    if (n < 0 || p.src_pages > COMPACT_MAX) fail("compact sizes");
    return hipSuccess;
}
}  // namespace gdn

namespace {
void stride(int64_t* s, int heads, int W) {
    s[1] = rarely() ? uni(-3, 1000) : W;
    s[0] = rarely() ? pick({0, -8, 7, 1 << 24, 1 << 28}) : int64_t(heads) * W;
    if (rarely()) s[0] = (int64_t(1) << uni(30, 62));
}

void fuzz_prompt(bool bwd) {
    gdn_linattn_desc d;
    memset(&d, 0, sizeof(d));
    d.B = pick({1, 1, 2, 3, 0});
    d.T = pick({0, 1, 63, 64, 65, 200, 5000, 70000, 1 << 30, -1});
    d.H = pick({1, 2, 6, 8, 32, 0, 70000});
    d.Hq = pick({1, 2, d.H, 5});
    d.Hk = pick({1, d.H, d.H, 0});
    d.Hv = pick({1, d.H, d.H});
    d.K = pick({64, 128, 128, 96});
    d.V = pick({64, 128, 128, 256});
    d.dtype = pick({0, 1, 1, 2});
    d.o_dtype = pick({0, 1, 1, -1});
    d.scale = rarely() ? 1.0f / 0.0f : 0.1f;
    stride(d.q_stride, d.Hq, d.K);
    stride(d.k_stride, d.Hk, d.K);
    stride(d.v_stride, d.Hv, d.V);
    std::vector<int32_t> offs;
    if (uni(0, 1)) {
        d.n_units = uni(-1, 12);
        const int64_t total = int64_t(d.B) * d.T;
        offs.resize(std::max(d.n_units, 0) + 1);
        for (auto& o : offs) o = total > 0 ? uni(0, (int)std::min<int64_t>(total, 1 << 30)) : 0;
        std::sort(offs.begin(), offs.end());
        offs.front() = 0;
        offs.back() = (int32_t)std::min<int64_t>(std::max<int64_t>(total, 0), INT32_MAX);
        d.offsets_host = rarely() ? nullptr : offs.data();
        d.offsets_dev = fake<int32_t>();
    }
    size_t need = 0;
    auto call = [&](void* ws, size_t* n) {
        return bwd ? gdn_linattn_bwd(&d, fake(), fake(), fake(), fake<float>(), fake<float>(), fake(), fake<float>(), fake(),
                                     fake(), fake(), fake<float>(), ws, n, nullptr)
                   : gdn_linattn_fwd(&d, fake(), fake(), fake(), fake<float>(), fake<float>(),
                                     uni(0, 1) ? fake<int32_t>() : nullptr, fake<float>(),
                                     uni(0, 1) ? fake<int32_t>() : nullptr, uni(-1, 9), fake(), ws, n, nullptr);
    };
    const gdn_status q = call(nullptr, &need);
    tally(q);
    if (q != GDN_OK) return;
    // a fake workspace as large as asked: nothing may be read or written in it
    region_lo = FAKE;
    region_bytes = need;
    size_t given = rarely() ? need / 2 : need;
    tally(call(rarely() ? FAKE + 64 : FAKE, &given));
    tally(call(FAKE, nullptr));
}

void fuzz_step() {
    gdn_step_desc d;
    memset(&d, 0, sizeof(d));
    d.N = pick({0, 1, 7, 300, -1, 1 << 30});
    d.H = pick({1, 4, 32, 0});
    d.Hq = pick({1, d.H, 3});
    d.Hk = pick({1, d.H});
    d.Hv = pick({1, d.H, d.H, 0});
    d.K = pick({64, 128, 128, 32});
    d.V = pick({64, 128, 128});
    d.dtype = pick({0, 1, 3});
    d.o_dtype = pick({0, 1});
    d.scale = 1;
    d.n_pages = pick({0, 1, 400, -2, INT32_MAX});
    stride(d.q_stride, d.Hq, d.K);
    stride(d.k_stride, d.Hk, d.K);
    stride(d.v_stride, d.Hv, d.V);
    tally(gdn_linattn_step(&d, fake(), fake(), fake(), fake<float>(), fake<int32_t>(), fake<float>(), fake(), nullptr));
    tally(gdn_recurrent_step(&d, pick({0, 1, 2}), pick({0, 1, 5}), fake(), fake(), fake(), fake<float>(), fake(),
                             fake<int32_t>(), fake<float>(), fake(), pick({0, 4, 8, 12, 1}), nullptr));
}

void fuzz_pages() {
    const int layers = pick({0, 1, 16, -1}), pages = pick({0, 1, 1000, 1 << 17, 1 << 18, -1, INT32_MAX});
    const int64_t bytes = pick({16, 64, 1 << 20, 0, 24, -16});
    const int n = pick({0, 1, 100, 8192, 8193, -1});
    int32_t* table = fake<int32_t>();
    tally(gdn_pages_copy(fake(), pages, fake(), pick({0, 5, -1}), layers, bytes, fake<int32_t>(), fake<int32_t>(), n,
                         nullptr));
    tally(gdn_pages_fork(fake(), layers, pages, bytes, table, fake<int32_t>(), n, fake<int32_t>(), pick({0, 9, 8193, -1}),
                         rarely() ? table : reinterpret_cast<int32_t*>(FAKE + 4096), fake<int32_t>(), fake<int32_t>(),
                         nullptr));
    tally(gdn_pages_compact(fake(), layers, pages, bytes, table, n,
                            rarely() ? table : reinterpret_cast<int32_t*>(FAKE + 4096), fake<int32_t>(), fake<int32_t>(),
                            nullptr));
    if (gdn_pages_workspace_ints(n) < 1) fail("workspace ints");
}
}  // namespace

int main() {
    for (int i = 0; i < 60000; ++i) {
        fuzz_prompt(i & 1);
        fuzz_step();
        fuzz_pages();
    }
    printf("statuses: ok %ld invalid %ld unsupported %ld device %ld capacity %ld, launches %ld\n", counts[0], counts[1],
           counts[2], counts[3], counts[4], launches);
    return launches > 1000 ? 0 : 2;
}
