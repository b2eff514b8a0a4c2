// What gdn_mixer_host.cpp hands to the kernels for chosen calls, with launch
// stubs that take it down. One check a run, named by the argument; exit status 0
// when it holds. Pointers are fake addresses that nothing may dereference.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <string>
#include <vector>

#include "gdn_mixer.h"
#include "gdn_mixer_internal.h"

namespace {
struct Launch {
    std::string name;
    gdn::ScanArgs scan;
};
std::vector<Launch> launches;
gdn::ScanArgs none() {
    gdn::ScanArgs a;
    memset(&a, 0, sizeof a);
    return a;
}
hipError_t note(const char* name, const gdn::ScanArgs& a = none()) {
    launches.push_back({name, a});
    return hipSuccess;
}
void expect(bool ok, const char* what, long long x = 0) {
    if (ok) return;
    fprintf(stderr, "mixer plans: %s (%lld)\n", what, x);
    exit(1);
}
}  // namespace

namespace gdn {
hipError_t launch_conv_fwd(const ConvArgs&, bool, hipStream_t) { return note("conv_fwd"); }
hipError_t launch_conv_bwd(const ConvArgs&, hipStream_t) { return note("conv_bwd"); }
hipError_t launch_conv_step(const ConvArgs&, hipStream_t) { return note("conv_step"); }
hipError_t launch_scan_summary(const ScanArgs& a, bool, hipStream_t) { return note("summary", a); }
hipError_t launch_scan_merge(const ScanArgs& a, bool, hipStream_t) { return note("merge", a); }
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t) { return note("scan_fwd", a); }
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t) { return note("scan_bwd", a); }
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t) { return note("scan_step", a); }
hipError_t launch_rotary_fwd(const RotaryArgs&, hipStream_t) { return note("rotary_fwd"); }
hipError_t launch_rotary_bwd(const RotaryArgs&, hipStream_t) { return note("rotary_bwd"); }
}  // namespace gdn

namespace {
char* const FAKE = reinterpret_cast<char*>(uintptr_t(1) << 40);
template <typename P = void>
P* at(int i) {   // apart from each other by more than any tensor here
    return reinterpret_cast<P*>(FAKE + (int64_t(i) << 41));
}

gdn_scan_desc scan_desc(int B, int T, int D, int S) {
    gdn_scan_desc d;
    memset(&d, 0, sizeof d);
    d.B = B, d.T = T, d.D = D, d.G = 1, d.S = S;
    d.dtype = GDN_DTYPE_BF16;
    d.softplus = 1;
    d.u_stride = d.dt_stride = d.gate_stride = D;
    d.b_stride[0] = d.b_stride[1] = d.c_stride[0] = d.c_stride[1] = S;
    return d;
}
gdn_status scan_bwd(const gdn_scan_desc& d, const float* dht, float* dh0) {
    launches.clear();
    size_t bytes = 0;
    auto call = [&](void* ws) {
        return gdn_scan_bwd(&d, at(0), at(1), at<float>(2), at(3), at(4), nullptr, nullptr, nullptr, at<float>(5), at(6), dht, at(7),
                            at(8), at<float>(9), at(10), at(11), nullptr, nullptr, nullptr, dh0, ws, &bytes, nullptr);
    };
    const gdn_status st = call(nullptr);
    return st == GDN_OK ? call(at(12)) : st;
}

// A cut walk back of at most 16 segments a sequence adds up those behind each
// segment itself, whether there are states or not; a merge goes in front where
// there are more, or where dh0 replaces dht.
void joins() {
    int joined = 0, merged = 0;
    constexpr int kSizes[][3] = {{2, 4096, 4096}, {1, 400, 1024}, {1, 160, 1024}, {1, 4096, 64}, {1, 900, 128}};
    for (const auto& [B, T, D] : kSizes) {
        const gdn_scan_desc d = scan_desc(B, T, D, 16);
        const struct {
            const float* dht;
            float* dh0;
        } states[] = {{nullptr, nullptr}, {at<float>(13), nullptr}, {nullptr, at<float>(14)}, {at<float>(13), at<float>(14)}};
        for (const auto& s : states) {
            expect(scan_bwd(d, s.dht, s.dh0) == GDN_OK, "refused", T);
            const gdn::ScanArgs& a = launches.back().scan;
            expect(a.cut, "not cut", T);
            const bool few = (T + a.un.P - 1) / a.un.P <= 16;
            expect(a.join == few, "join", T);
            expect(launches.size() == (few ? 2u : 3u) && launches[0].name == "summary", "launches", T);
            expect(few || launches[1].name == "merge", "merge", T);
            ++(few ? joined : merged);
        }
        expect(scan_bwd(d, at<float>(13), at<float>(13)) == GDN_OK, "refused in place", T);
        expect(!launches.back().scan.join && launches.size() == 3 && launches[1].name == "merge", "in place without a merge", T);
    }
    expect(joined > 0 && merged > 0, "one kind only", joined);
}
// Without page lists the states may be replaced in place or lie apart; where they
// overlap by part a sequence would read what another has written.
template <typename F>
void overlaps(int units, int64_t page, F call) {
    char* s = at<char>(20);
    const int32_t *none = nullptr, *pages = at<const int32_t>(21);
    const struct {
        int64_t from;
        bool in_paged, out_paged, ok;
    } cases[] = {{0, false, false, true},          {page, false, false, false},  {-page, false, false, false},
                 {64, false, false, false},        {units * page - 16, false, false, false},
                 {units * page, false, false, true}, {-units * page, false, false, true},
                 {page, true, true, true},         {page, true, false, true},    {page, false, true, true}};
    for (const auto& c : cases) {
        launches.clear();
        const gdn_status st = call(s, c.in_paged ? pages : none, s + c.from, c.out_paged ? pages : none);
        expect(st == (c.ok ? GDN_OK : GDN_ERR_INVALID), "states that overlap", c.from);
        expect(launches.empty() != c.ok, "launches", c.from);
    }
    for (int null = 0; null < 3; ++null)
        expect(call(null != 1 ? nullptr : s, none, null != 2 ? nullptr : s, none) == GDN_OK, "states left out", null);
}
void states() {
    for (int n : {2, 3}) {
        gdn_conv_desc c;
        memset(&c, 0, sizeof c);
        c.B = n, c.T = 2, c.D = 64, c.W = 4, c.dtype = c.w_dtype = GDN_DTYPE_BF16, c.x_stride = 64;
        overlaps(n, 3 * 64 * 2, [&](char* in, const int32_t* ip, char* out, const int32_t* op) {
            return gdn_conv_fwd(&c, at(0), at(1), nullptr, in, ip, out, op, 8, at(2), nullptr);
        });
        for (int T : {5, 900}) {          // whole and cut
            const gdn_scan_desc d = scan_desc(n, T, 64, 16);
            overlaps(n, 64 * 16 * 4, [&](char* in, const int32_t* ip, char* out, const int32_t* op) {
                size_t bytes = 0;
                auto run = [&](void* ws) {
                    return gdn_scan_fwd(&d, at(0), at(1), at<float>(2), at(3), at(4), nullptr, nullptr, nullptr, (float*)in, ip,
                                        (float*)out, op, 8, nullptr, at(5), ws, &bytes, nullptr);
                };
                const gdn_status st = run(nullptr);
                return st == GDN_OK ? run(at(6)) : st;
            });
        }
    }
}
// The sums of dB and dC share a launch with those of dA where these are few: both
// have to fit into one.
void limits() {
    for (const auto& [T, ok] : {std::pair{4294965, true}, std::pair{4294966, true}, std::pair{4294967, false}}) {
        const gdn_scan_desc d = scan_desc(250, T, 8, 8);
        expect(scan_bwd(d, nullptr, nullptr) == (ok ? GDN_OK : GDN_ERR_UNSUPPORTED), "sums beyond a launch", T);
        expect(launches.size() == (ok ? 1u : 0u), "launches", T);
        const int64_t bc = (int64_t(250) * T * 4 + 255) / 256, cols = (8 * (8 + 2) + 63) / 64;
        expect(((bc + cols) * 256 < int64_t(1) << 32) == ok, "the test's sizes", T);
    }
}
}  // namespace

int main(int argc, char** argv) {
    const std::string what = argc > 1 ? argv[1] : "";
    if (what == "joins") joins();
    else if (what == "states") states();
    else if (what == "limits") limits();
    else return 2;
    printf("%s: ok\n", what.c_str());
    return 0;
}
