// Host-side fuzz of the C ABI of the operators around the recurrent layers
// under AddressSanitizer and UndefinedBehaviorSanitizer: random descriptors,
// offsets, strides, sizes and pointers. The launch functions are stubs that check
// what the host code hands them: regions inside the workspace, pieces that cover
// every token once, launches within HIP's limit. Input pointers are fake
// addresses that nothing may dereference. Exit status 0 when every call returned
// a declared status.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "gdn_mixer.h"
#include "gdn_mixer_internal.h"

namespace {
std::mt19937_64 rng(20261209);
int uni(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
int pick(std::initializer_list<int> xs) { return *(xs.begin() + uni(0, (int)xs.size() - 1)); }
bool rarely() { return uni(0, 19) == 0; }

char* const FAKE = reinterpret_cast<char*>(uintptr_t(1) << 40);
template <typename P = void>
P* fake() {   // sometimes NULL, sometimes misaligned
    return rarely() && rarely() ? nullptr : reinterpret_cast<P*>(FAKE + (rarely() && rarely() ? 4 : 0));
}
template <typename P = void>
P* maybe() {
    return uni(0, 1) ? fake<P>() : nullptr;
}
long counts[6], launches;
std::vector<char> memory(1 << 12);
const char* region_lo = nullptr;
size_t region_bytes = 0;
const int32_t* host_offsets = nullptr;

void fail(const char* what) {
    fprintf(stderr, "mixer stub: %s\n", what);
    abort();
}
void tally(gdn_status s) {
    if (s < GDN_OK || s > GDN_ERR_CAPACITY) fail("undeclared status");
    counts[s]++;
}
void in_workspace(const void* p, int64_t bytes, const char* what) {
    const char* c = static_cast<const char*>(p);
    if (bytes < 0 || c < region_lo || c + bytes > region_lo + region_bytes || (uintptr_t)c % 256) fail(what);
}
void in_grid(int64_t workgroups) {
    if (workgroups < 0 || workgroups * 256 >= (int64_t(1) << 32)) fail("grid");
}
// the device's numbering of pieces: no two share a number, all are below n_pieces
void check_units(const gdn::MxUnits& u) {
    ++launches;
    if (u.n_units < 1 || u.P < 1 || u.n_pieces < u.n_units) fail("units");
    int64_t next = 0;
    for (int32_t i = 0; i < u.n_units && i < 2000; ++i) {
        const int64_t start = u.dense ? int64_t(i) * u.T : host_offsets[i];
        const int64_t len = u.dense ? u.T : host_offsets[i + 1] - host_offsets[i];
        const int64_t per = len > u.P ? (len - 1) / u.P + 1 : 1;
        const int64_t base = u.dense ? i * (u.T > u.P ? (u.T - 1) / u.P + 1 : 1) : start / u.P + i;
        if (base < next) fail("pieces overlap");
        next = base + per;
        if (next > u.n_pieces) fail("pieces beyond their number");
    }
}
int vector_of(int dtype) { return dtype == GDN_DTYPE_BF16 ? 8 : 4; }
}  // namespace

namespace gdn {
hipError_t launch_conv_fwd(const ConvArgs& a, bool, hipStream_t) {
    check_units(a.un);
    in_grid((int64_t(a.un.n_pieces) * (a.D / vector_of(a.dtype)) + 255) / 256);
    return hipSuccess;
}
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t) {
    check_units(a.un);
    in_grid((int64_t(a.un.n_pieces) * (a.D / CONV_BWD_CHANNELS) + 255) / 256);
    const int64_t rows = a.un.n_pieces + row_sums_rows(a.un.n_pieces);
    in_workspace(a.parts, rows * a.D * (a.W + 1) * 4, "parts");
    in_grid(row_sums_workgroups(a.un.n_pieces, int64_t(a.D) * (a.W + 1)));
    return hipSuccess;
}
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t) {
    check_units(a.un);
    return hipSuccess;
}
static void check_scan(const ScanArgs& a) {
    check_units(a.un);
    check_units(a.keep);
    if (a.un.P % SCAN_TILE) fail("segment");
    in_grid(int64_t(a.un.n_pieces) * a.G * a.bwd_blocks);
    if (a.cut) {
        in_workspace(a.slots, int64_t(a.un.n_pieces) * a.D * a.S * 4, "slots");
        in_workspace(a.sums, int64_t(a.un.n_pieces) * a.D * 4, "sums");
    }
}
hipError_t launch_scan_summary(const ScanArgs& a, bool, hipStream_t) {
    check_scan(a);
    return hipSuccess;
}
hipError_t launch_scan_merge(const ScanArgs& a, bool, hipStream_t) {
    in_grid(int64_t(a.un.n_units) * ((int64_t(a.D) * a.S + 255) / 256));
    return hipSuccess;
}
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t) {
    check_scan(a);
    if (a.narrow) {
        if (a.cut) fail("one state a lane and cut");
        const int ch = scan_narrow_channels(a.S);
        in_grid(int64_t(a.un.n_pieces) * a.G * ((a.D / a.G + ch - 1) / ch));
    }
    return hipSuccess;
}
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t) {
    check_scan(a);
    const int64_t rows = a.un.n_pieces + row_sums_rows(a.un.n_pieces);
    in_workspace(a.a_parts, rows * a.D * (a.S + 2) * 4, "a_parts");
    in_workspace(a.bc_parts, int64_t(a.G) * a.bwd_blocks * a.un.total * 2 * a.S * 4, "bc_parts");
    in_grid((a.un.total * a.G * (a.S / 2) + 255) / 256);
    in_grid(row_sums_workgroups(a.un.n_pieces, int64_t(a.D) * (a.S + 2)));
    return hipSuccess;
}
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t) {
    check_units(a.un);
    in_grid(int64_t(a.un.n_units) * ((int64_t(a.D) * (a.S / 4) + 255) / 256));
    return hipSuccess;
}
hipError_t launch_rotary_fwd(const RotaryArgs& a, hipStream_t) {
    ++launches;
    in_grid(a.tokens);
    return hipSuccess;
}
hipError_t launch_rotary_bwd(const RotaryArgs& a, hipStream_t) {
    ++launches;
    if (a.parts) in_workspace(a.parts, (a.workgroups + row_sums_rows(a.workgroups)) * int64_t(2) * a.D * 4, "parts");
    return hipSuccess;
}
}  // namespace gdn

namespace {
std::vector<int32_t> offsets;
template <typename D>
void sequences(D& d) {
    d.B = pick({1, 1, 2, 7, 300, 0, -1});
    d.T = pick({0, 1, 2, 15, 16, 17, 33, 1000, 20000, 1 << 28, INT32_MAX, -3});
    d.n_units = 0;
    if (uni(0, 2) == 0) {
        d.B = rarely() ? 2 : 1;
        const int n = pick({1, 2, 5, 300});
        offsets.assign(1, 0);
        for (int i = 0; i < n; ++i) offsets.push_back(offsets.back() + pick({1, 2, 7, 16, 100, 3000}) + (rarely() && rarely() ? -20 : 0));
        if (rarely()) offsets.back() = INT32_MAX;
        d.T = offsets.back() - (rarely() ? 1 : 0);
        d.n_units = n;
        d.offsets_host = rarely() ? nullptr : offsets.data();
        d.offsets_dev = fake<const int32_t>();
        host_offsets = offsets.data();
    }
}
int64_t stride(int64_t least) {
    if (rarely()) return pick({-8, 4, 0, 1 << 20});
    if (rarely() && rarely()) return int64_t(1) << uni(20, 62);
    return least + 8 * uni(0, 3);
}
// runs a call with no workspace, then with one of the size that it asked for (none of
// it is touched), with a shorter one and with a misaligned one
template <typename F>
void with_workspace(F call) {
    size_t bytes = 0;
    const gdn_status q = call((void*)nullptr, &bytes);
    tally(q);
    if (q != GDN_OK) return;
    char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(memory.data()) + 255) / 256 * 256);
    region_lo = base;
    region_bytes = bytes;
    size_t given = bytes;
    tally(call((void*)base, &given));
    given = bytes - 1;
    if (call((void*)base, &given) != GDN_ERR_CAPACITY || given != bytes) fail("a short workspace");
    given = bytes;
    if (call((void*)(base + 64), &given) == GDN_OK) fail("a misaligned workspace");
}
}  // namespace

int main() {
    for (int i = 0; i < 60000; ++i) {
        gdn_conv_desc c;
        memset(&c, 0, sizeof c);
        sequences(c);
        c.D = pick({8, 16, 64, 4096, 1 << 20, 12, 0, -8});
        c.W = pick({2, 3, 4, 4, 1, 5});
        c.dtype = rarely() ? 7 : uni(0, 1);
        c.w_dtype = rarely() ? -1 : uni(0, 1);
        c.silu = rarely() ? 2 : uni(0, 1);
        c.x_stride = stride(c.D);
        tally(gdn_conv_fwd(rarely() ? nullptr : &c, fake(), fake(), maybe(), maybe(), maybe<const int32_t>(), maybe(),
                           maybe<const int32_t>(), pick({0, 5, -1}), fake(), nullptr));
        with_workspace([&](void* ws, size_t* n) {
            return gdn_conv_bwd(&c, fake(), fake(), maybe(), maybe(), fake(), maybe(), fake(), fake<float>(),
                                maybe<float>(), maybe(), ws, n, nullptr);
        });
        if (uni(0, 1)) c.T = 1, c.n_units = 0;
        tally(gdn_conv_step(&c, fake(), fake(), maybe(), maybe<const int32_t>(), pick({0, 5, 1 << 20, -1}), fake(), fake(), nullptr));

        gdn_scan_desc s;
        memset(&s, 0, sizeof s);
        sequences(s);
        s.G = pick({1, 1, 2, 3, 0});
        s.D = pick({8, 24, 64, 96, 4096, 1 << 20, 20}) * (uni(0, 1) ? std::max(1, s.G) : 1);
        s.S = pick({8, 16, 16, 32, 64, 12});
        s.dtype = rarely() ? 5 : uni(0, 1);
        s.softplus = rarely() ? 3 : uni(0, 1);
        s.u_stride = stride(s.D);
        s.dt_stride = stride(s.D);
        s.gate_stride = stride(s.D);
        for (int j = 0; j < 2; ++j) s.b_stride[j] = stride(j ? s.S : s.S * s.G), s.c_stride[j] = stride(j ? s.S : s.S * s.G);
        if (gdn_scan_h_rows(&s) < -1) fail("h rows");
        const float* gate = maybe<const float>();
        with_workspace([&](void* ws, size_t* n) {
            return gdn_scan_fwd(&s, fake(), fake(), fake<float>(), fake(), fake(), maybe<float>(), gate, maybe<float>(),
                                maybe<float>(), maybe<const int32_t>(), maybe<float>(), maybe<const int32_t>(),
                                pick({0, 5, -1}), maybe<float>(), fake(), ws, n, nullptr);
        });
        with_workspace([&](void* ws, size_t* n) {
            return gdn_scan_bwd(&s, fake(), fake(), fake<float>(), fake(), fake(), maybe<float>(), gate, maybe<float>(),
                                fake<float>(), fake(), maybe<float>(), fake(), fake(), fake<float>(), fake(), fake(),
                                maybe<float>(), rarely() ? nullptr : (void*)gate, maybe<float>(), maybe<float>(), ws, n,
                                nullptr);
        });
        if (uni(0, 1)) s.T = 1, s.n_units = 0;
        tally(gdn_scan_step(&s, fake(), fake(), fake<float>(), fake(), fake(), maybe<float>(), gate, maybe<float>(),
                            maybe<const int32_t>(), pick({0, 5, 1 << 20, -1}), fake<float>(), fake(), nullptr));

        gdn_rotary_desc r;
        memset(&r, 0, sizeof r);
        r.B = pick({1, 2, 300, 0});
        r.T = pick({0, 1, 9, 5000, 1 << 24, INT32_MAX, -1});
        r.Hq = pick({1, 2, 32, 0});
        r.Hk = pick({1, 4, 1 << 20});
        r.D = pick({8, 64, 80, 128, 256, 264, 12});
        r.R = pick({0, 8, 64, 128, 20, -8});
        r.dtype = rarely() ? 9 : uni(0, 1);
        r.w_dtype = rarely() ? 9 : uni(0, 1);
        r.norm = rarely() ? 4 : uni(0, 2);
        r.interleaved = rarely() ? 2 : uni(0, 1);
        r.pos_i64 = uni(0, 1);
        r.eps = rarely() ? -1.0f : 1e-6f;
        r.amplitude = rarely() ? 1.0f / 0.0f : 1.0f;
        r.q_stride[0] = stride(int64_t(r.Hq) * r.D);
        r.q_stride[1] = stride(r.D);
        r.k_stride[0] = stride(int64_t(r.Hk) * r.D);
        r.k_stride[1] = stride(r.D);
        char* other = FAKE + (1 << 20);
        tally(gdn_qk_rotary_fwd(&r, fake(), fake(), maybe<double>(), maybe(), maybe(), maybe(), uni(0, 1) ? fake() : (void*)other,
                                (void*)other, nullptr));
        void* qw = maybe();
        with_workspace([&](void* ws, size_t* n) {
            return gdn_qk_rotary_bwd(&r, fake(), fake(), fake<double>(), maybe(), qw, nullptr, fake(), fake(), fake(), fake(),
                                     rarely() ? nullptr : (float*)qw, nullptr, ws, n, nullptr);
        });
    }
    printf("statuses: ok %ld invalid %ld unsupported %ld device %ld capacity %ld; launches: %ld\n", counts[0], counts[1],
           counts[2], counts[3], counts[4], launches);
    for (int s : {GDN_OK, GDN_ERR_INVALID, GDN_ERR_UNSUPPORTED})
        if (!counts[s]) fail("a status never occurred");
    if (launches < 1000) fail("hardly any launch");
    return 0;
}
