// Torch marshalling of the operators around the recurrent layers
// (include/gdn_mixer.h), as gdn_torch.cpp does for the recurrent states'.
#include "gdn_torch.h"

#include "gdn_mixer.h"

namespace {

using namespace gdn_torch;

std::vector<int64_t> with(at::IntArrayRef lead, std::initializer_list<int64_t> rest) {
    std::vector<int64_t> s(lead.begin(), lead.end());
    s.insert(s.end(), rest);
    return s;
}

at::IntArrayRef lead_of(const Tensor& t, int64_t n) { return t.sizes().slice(0, t.dim() - n); }

// Distance of tokens in elements of [B,T,D] or [tokens,D], as row_strides has it for rows with heads
int64_t token_stride(const char* name, const Tensor& t) {
    const auto n = t.sizes(), s = t.strides();
    const int64_t d = t.dim(), D = n[d - 1];
    if (D > 1 && s[d - 1] != 1) invalid(std::string(name) + ": the values of a row must be contiguous");
    int64_t ts = s[d - 2];
    if (d == 3) {
        if (n[0] * n[1] <= 1) ts = D;
        else if (n[1] == 1) ts = s[0];
        else if (n[0] > 1 && s[0] != n[1] * ts) invalid(std::string(name) + ": batch rows must follow each other at the token stride");
    } else if (n[0] <= 1) {
        ts = D;
    }
    if (ts * t.element_size() % 16 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 || ts < 0)
        invalid(std::string(name) + ": rows must be 16-byte aligned");
    return ts;
}

void check_like(const char* name, const Tensor& t, ScalarType dtype, const std::vector<int64_t>& shape) {
    if (!t.defined()) invalid(std::string(name) + " is required");
    if (t.scalar_type() != dtype) invalid(std::string(name) + " must be " + dtype_text(dtype) + ", got " + dtype_text(t.scalar_type()));
    if (t.sizes() != at::IntArrayRef(shape)) invalid(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

typedef std::initializer_list<std::pair<const char*, const Tensor*>> Named;

void check_devices(const Tensor& first, Named others) {
    need_gpu("inputs", first);
    for (const auto& [name, t] : others) check_device(name, *t, first.device());
}

void need_dense(const Tensor& t, Named all) {
    for (const auto& [name, x] : all)
        if (x->defined() && reinterpret_cast<uintptr_t>(x->data_ptr()) % 16) invalid(std::string(name) + " must be 16-byte aligned");
}

// Sequences of [B,T,..] or, with meta's device offsets, [T,..]
template <typename Desc>
int64_t sequences(Desc& d, at::IntArrayRef lead, const Tensor& offsets, int64_t n_units, int64_t host) {
    if (lead.size() == 1 && !offsets.defined()) invalid("packed inputs need meta");
    if (lead.size() == 2 && offsets.defined()) invalid("meta goes with packed inputs");
    d.B = lead.size() == 2 ? narrow(lead[0], "B") : 1;
    d.T = narrow(lead[lead.size() - 1], "T");
    if (!offsets.defined()) return d.B;
    if (n_units < 1) invalid("meta has no documents");
    check_tensor("meta's device offsets", offsets, ScalarType::Int, {n_units + 1});
    d.n_units = narrow(n_units, "units");
    d.offsets_host = reinterpret_cast<const int32_t*>(host);
    d.offsets_dev = ptr<int32_t>(offsets);
    return n_units;
}

// States by sequence or in a pool with pages; the pools' pages in n_pages
void check_states(const char* name, const Tensor& t, const char* pages_name, const Tensor& pages, ScalarType dtype,
                  int64_t units, int64_t rows, int64_t cols, int64_t* n_pages) {
    if (pages.defined()) {
        check_tensor(pages_name, pages, ScalarType::Int, {units});
        if (!t.defined() || t.dim() != 3) invalid(std::string(name) + " must be a pool of pages when its pages are given");
    }
    if (!t.defined()) return;
    const int64_t n = pages.defined() ? t.size(0) : units;
    check_tensor(name, t, dtype, {n, rows, cols});
    if (!pages.defined()) return;
    if (*n_pages >= 0 && *n_pages != n)
        invalid("the pools have " + std::to_string(*n_pages) + " and " + std::to_string(n) + " pages");
    *n_pages = n;
}

// Without pages the states may be replaced in place, or lie apart
void check_states_apart(const Tensor& s_in, const Tensor& in_pages, const Tensor& final_out, const Tensor& out_pages) {
    if (in_pages.defined() || out_pages.defined() || !s_in.defined() || !final_out.defined()) return;
    if (s_in.data_ptr() != final_out.data_ptr()) check_apart(final_out, {{"initial_state", &s_in}});
}

int32_t parameters(std::initializer_list<std::pair<const char*, const Tensor*>> all) {
    ScalarType t = ScalarType::Undefined;
    for (const auto& [name, p] : all) {
        if (!p->defined()) continue;
        if (t == ScalarType::Undefined) t = p->scalar_type();
        if (p->scalar_type() != t) invalid(std::string(name) + " must be " + dtype_text(t) + ", got " + dtype_text(p->scalar_type()));
    }
    return t == ScalarType::Undefined ? GDN_DTYPE_F32 : dtype_code(t);
}

PyObject* tuple(std::initializer_list<const Tensor*> all) {
    PyObject* r = PyTuple_New((Py_ssize_t)all.size());
    Py_ssize_t i = 0;
    for (const Tensor* t : all) PyTuple_SET_ITEM(r, i++, t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None));
    return r;
}

PyObject* dict(Named all) {
    PyObject* r = PyDict_New();
    for (const auto& [name, t] : all) {
        if (!t->defined()) continue;
        PyObject* x = THPVariable_Wrap(*t);
        PyDict_SetItemString(r, name, x);
        Py_DECREF(x);
    }
    return r;
}

Tensor floats(const Tensor& like, at::IntArrayRef shape) { return at::empty(shape, like.options().dtype(ScalarType::Float)); }

// ---- convolution
struct Conv {
    gdn_conv_desc d;
    int64_t units, n_pages = -1;
};

Conv conv(const Tensor& x, const Tensor& weight, const Tensor& bias, bool silu, int64_t lead) {
    if (!x.defined() || (lead ? x.dim() != lead + 1 : x.dim() != 2 && x.dim() != 3))
        invalid(lead ? "x must have shape [N,D]" : "x must have shape [B,T,D] or [T,D]");
    if (!weight.defined() || weight.dim() != 2) invalid("weight must be [D,W]");
    Conv c;
    memset(&c.d, 0, sizeof(c.d));
    const int64_t D = x.size(-1);
    c.d.D = narrow(D, "D");
    c.d.W = narrow(weight.size(1), "W");
    c.d.dtype = dtype_code(x.scalar_type());
    c.d.silu = silu;
    c.d.w_dtype = parameters({{"weight", &weight}, {"bias", &bias}});
    check_tensor("weight", weight, weight.scalar_type(), {D, weight.size(1)});
    if (bias.defined()) check_tensor("bias", bias, bias.scalar_type(), {D});
    if (D % 8) invalid("x has " + std::to_string(D) + " channels, not a multiple of 8");
    if (c.d.W < 2 || c.d.W > 4) throw std::logic_error("convolutions of " + std::to_string(c.d.W) + " taps");
    need_dense(x, {{"weight", &weight}, {"bias", &bias}});
    return c;
}

PyObject* conv_fwd(const Arguments& a) {
    a.count(13);
    const Tensor x = a.tensor(0, "x"), weight = a.tensor(1, "weight"), bias = a.tensor(2, "bias"),
                 offsets = a.tensor(4, "meta"), s_in = a.tensor(7, "initial_state"),
                 in_pages = a.tensor(8, "initial_pages"), final_out = a.tensor(10, "final_out"),
                 out_pages = a.tensor(11, "final_pages"), out = a.tensor(12, "out");
    Conv c = conv(x, weight, bias, a.flag(3), 0);
    const int64_t units = sequences(c.d, lead_of(x, 1), offsets, a.integer(5), a.integer(6));
    c.d.x_stride = token_stride("x", x);
    check_states("initial_state", s_in, "initial_pages", in_pages, x.scalar_type(), units, c.d.W - 1, c.d.D, &c.n_pages);
    check_states("final_out", final_out, "final_pages", out_pages, x.scalar_type(), units, c.d.W - 1, c.d.D, &c.n_pages);
    if (out.defined()) check_tensor("out", out, x.scalar_type(), x.sizes());
    check_apart(out, {{"x", &x}, {"weight", &weight}, {"bias", &bias}, {"initial_state", &s_in}, {"final_out", &final_out}});
    check_apart(final_out, {{"x", &x}, {"weight", &weight}, {"bias", &bias}});
    check_states_apart(s_in, in_pages, final_out, out_pages);
    need_dense(x, {{"initial_state", &s_in}, {"final_out", &final_out}, {"out", &out}});
    check_devices(x, {{"weight", &weight}, {"bias", &bias}, {"unit metadata", &offsets}, {"initial_state", &s_in},
                      {"initial_pages", &in_pages}, {"final_out", &final_out}, {"final_pages", &out_pages}, {"out", &out}});
    const Guard guard(x.device());
    const Tensor y = out.defined() ? out : at::empty(x.sizes(), x.options());
    Tensor fin = final_out;
    if (!fin.defined() && a.flag(9)) fin = at::empty({units, c.d.W - 1, c.d.D}, x.options());
    check(gdn_conv_fwd(&c.d, ptr(x), ptr(weight), ptr(bias), ptr(s_in), ptr<int32_t>(in_pages), ptr(fin),
                       ptr<int32_t>(out_pages), narrow(c.n_pages < 0 ? 0 : c.n_pages, "n_pages"), ptr(y),
                       stream_of(x.device())),
          "gdn_conv_fwd");
    written({&out, &final_out});
    return tuple({&y, &fin});
}

PyObject* conv_bwd(const Arguments& a) {
    a.count(12);
    const Tensor x = a.tensor(0, "x"), weight = a.tensor(1, "weight"), bias = a.tensor(2, "bias"),
                 dout = a.tensor(3, "dout"), offsets = a.tensor(5, "meta"), s_in = a.tensor(8, "initial_state"),
                 dfinal = a.tensor(9, "dfinal"), given = a.tensor(11, "workspace");
    Conv c = conv(x, weight, bias, a.flag(4), 0);
    const int64_t units = sequences(c.d, lead_of(x, 1), offsets, a.integer(6), a.integer(7));
    c.d.x_stride = token_stride("x", x);
    if (!dout.defined()) invalid("dout is required");
    check_tensor("dout", dout, x.scalar_type(), x.sizes());
    const std::vector<int64_t> sshape = {units, c.d.W - 1, c.d.D};
    if (s_in.defined()) check_tensor("initial_state", s_in, x.scalar_type(), sshape);
    if (dfinal.defined()) check_tensor("dfinal", dfinal, x.scalar_type(), sshape);
    need_dense(x, {{"dout", &dout}, {"initial_state", &s_in}, {"dfinal", &dfinal}});
    check_devices(x, {{"weight", &weight}, {"bias", &bias}, {"unit metadata", &offsets}, {"dout", &dout},
                      {"initial_state", &s_in}, {"dfinal", &dfinal}});
    const Guard guard(x.device());
    size_t bytes = 0;
    check(gdn_conv_bwd(&c.d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, x.device());
    bytes = (size_t)ws.numel();
    const Tensor dx = at::empty(x.sizes(), x.options()), dw = floats(x, weight.sizes()),
                 db = bias.defined() ? floats(x, bias.sizes()) : Tensor(),
                 di = a.flag(10) ? at::empty(sshape, x.options()) : Tensor();
    check(gdn_conv_bwd(&c.d, ptr(x), ptr(weight), ptr(bias), ptr(s_in), ptr(dout), ptr(dfinal), ptr(dx),
                       ptr<float>(dw), ptr<float>(db), ptr(di), ptr(ws), &bytes, stream_of(x.device())),
          "gdn_conv_bwd");
    return dict({{"dx", &dx}, {"dweight", &dw}, {"dbias", &db}, {"dinitial", &di}});
}

PyObject* conv_step(const Arguments& a) {
    a.count(7);
    const Tensor x = a.tensor(0, "x"), weight = a.tensor(1, "weight"), state = a.tensor(2, "state"),
                 bias = a.tensor(3, "bias"), pages = a.tensor(5, "pages"), out = a.tensor(6, "out");
    Conv c = conv(x, weight, bias, a.flag(4), 1);
    const int64_t N = x.size(0);
    if (!state.defined() || state.dim() != 3) invalid("state must be [n_pages, W - 1, D]");
    check_tensor("state", state, x.scalar_type(), {state.size(0), c.d.W - 1, c.d.D});
    if (!pages.defined() && state.size(0) < N)
        invalid("state has " + std::to_string(state.size(0)) + " pages for " + std::to_string(N) + " rows");
    if (pages.defined()) check_tensor("pages", pages, ScalarType::Int, {N});
    if (out.defined()) check_tensor("out", out, x.scalar_type(), x.sizes());
    check_apart(out, {{"x", &x}, {"weight", &weight}, {"bias", &bias}, {"state", &state}});
    check_apart(state, {{"x", &x}, {"weight", &weight}, {"bias", &bias}});
    need_dense(x, {{"state", &state}, {"out", &out}});
    c.d.B = narrow(N, "N");
    c.d.T = 1;
    c.d.x_stride = token_stride("x", x);
    check_devices(x, {{"weight", &weight}, {"bias", &bias}, {"state", &state}, {"pages", &pages}, {"out", &out}});
    const Guard guard(x.device());
    const Tensor y = out.defined() ? out : at::empty(x.sizes(), x.options());
    check(gdn_conv_step(&c.d, ptr(x), ptr(weight), ptr(bias), ptr<int32_t>(pages), narrow(state.size(0), "n_pages"),
                        ptr(state), ptr(y), stream_of(x.device())),
          "gdn_conv_step");
    written({&state, &out});
    return THPVariable_Wrap(y);
}

// ---- scan
struct ScanIn {
    Tensor u, dt, A, B, C, skip, gate, dt_bias;
};

// arguments 0 .. 7
ScanIn scan_in(const Arguments& a) {
    return {a.tensor(0, "u"), a.tensor(1, "dt"), a.tensor(2, "A"), a.tensor(3, "B"), a.tensor(4, "C"),
            a.tensor(5, "skip"), a.tensor(6, "gate"), a.tensor(7, "dt_bias")};
}

gdn_scan_desc scan(const ScanIn& x, bool softplus, int64_t lead_dims) {
    if (!x.u.defined() || (lead_dims ? x.u.dim() != lead_dims + 1 : x.u.dim() != 2 && x.u.dim() != 3))
        invalid(lead_dims ? "u must have shape [N,D]" : "u must have shape [B,T,D] or [T,D]");
    if (!x.A.defined() || x.A.dim() != 2) invalid("A must be fp32 [D,S]");
    if (!x.B.defined() || x.B.dim() != x.u.dim() + 1) invalid("B must have shape [..,G,S]");
    const ScalarType t = x.u.scalar_type();
    const int64_t D = x.u.size(-1), S = x.A.size(1), G = x.B.size(-2);
    gdn_scan_desc d;
    memset(&d, 0, sizeof(d));
    d.D = narrow(D, "D");
    d.S = narrow(S, "S");
    d.G = narrow(G, "G");
    d.dtype = dtype_code(t);
    d.softplus = softplus;
    const at::IntArrayRef lead = lead_of(x.u, 1);
    check_like("dt", x.dt, t, with(lead, {D}));
    check_like("B", x.B, t, with(lead, {G, S}));
    check_like("C", x.C, t, with(lead, {G, S}));
    if (x.gate.defined()) check_like("gate", x.gate, t, with(lead, {D}));
    check_tensor("A", x.A, ScalarType::Float, {D, S});
    if (x.skip.defined()) check_tensor("skip", x.skip, ScalarType::Float, {D});
    if (x.dt_bias.defined()) check_tensor("dt_bias", x.dt_bias, ScalarType::Float, {D});
    if (S != 8 && S != 16 && S != 32 && S != 64) throw std::logic_error("scans of " + std::to_string(S) + " states");
    if (G < 1 || D % G || D / G % 8)
        invalid("u has " + std::to_string(D) + " channels, which do not divide into " + std::to_string(G) + " groups of a multiple of 8");
    d.u_stride = token_stride("u", x.u);
    d.dt_stride = token_stride("dt", x.dt);
    if (x.gate.defined()) d.gate_stride = token_stride("gate", x.gate);
    row_strides("B", x.B, d.b_stride);
    row_strides("C", x.C, d.c_stride);
    need_dense(x.u, {{"A", &x.A}, {"skip", &x.skip}, {"dt_bias", &x.dt_bias}});
    return d;
}

void scan_devices(const ScanIn& x, Named more) {
    check_devices(x.u, {{"dt", &x.dt}, {"A", &x.A}, {"B", &x.B}, {"C", &x.C}, {"skip", &x.skip}, {"gate", &x.gate},
                        {"dt_bias", &x.dt_bias}});
    check_devices(x.u, more);
}

void scan_apart(const Tensor& out, const ScanIn& x) {
    check_apart(out, {{"u", &x.u}, {"dt", &x.dt}, {"A", &x.A}, {"B", &x.B}, {"C", &x.C}, {"skip", &x.skip},
                      {"gate", &x.gate}, {"dt_bias", &x.dt_bias}});
}

PyObject* scan_fwd(const Arguments& a) {
    a.count(20);
    const ScanIn x = scan_in(a);
    const Tensor offsets = a.tensor(9, "meta"), s_in = a.tensor(12, "initial_state"),
                 in_pages = a.tensor(13, "initial_pages"), final_out = a.tensor(15, "final_out"),
                 out_pages = a.tensor(16, "final_pages"), out = a.tensor(18, "out"), given = a.tensor(19, "workspace");
    gdn_scan_desc d = scan(x, a.flag(8), 0);
    const int64_t units = sequences(d, lead_of(x.u, 1), offsets, a.integer(10), a.integer(11));
    int64_t n_pages = -1;
    check_states("initial_state", s_in, "initial_pages", in_pages, ScalarType::Float, units, d.D, d.S, &n_pages);
    check_states("final_out", final_out, "final_pages", out_pages, ScalarType::Float, units, d.D, d.S, &n_pages);
    if (out.defined()) check_tensor("out", out, x.u.scalar_type(), x.u.sizes());
    scan_apart(out, x);
    check_apart(out, {{"initial_state", &s_in}, {"final_out", &final_out}});
    scan_apart(final_out, x);
    check_states_apart(s_in, in_pages, final_out, out_pages);
    need_dense(x.u, {{"initial_state", &s_in}, {"final_out", &final_out}, {"out", &out}});
    scan_devices(x, {{"unit metadata", &offsets}, {"initial_state", &s_in}, {"initial_pages", &in_pages},
                     {"final_out", &final_out}, {"final_pages", &out_pages}, {"out", &out}});
    const Guard guard(x.u.device());
    size_t bytes = 0;
    check(gdn_scan_fwd(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr, nullptr, 0, nullptr, nullptr, nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, x.u.device());
    bytes = (size_t)ws.numel();
    const Tensor o = out.defined() ? out : at::empty(x.u.sizes(), x.u.options());
    const Tensor h = a.flag(17) ? floats(x.u, {gdn_scan_h_rows(&d), d.D, d.S}) : Tensor();
    Tensor fin = final_out;
    if (!fin.defined() && a.flag(14)) fin = floats(x.u, {units, d.D, d.S});
    check(gdn_scan_fwd(&d, ptr(x.u), ptr(x.dt), ptr<float>(x.A), ptr(x.B), ptr(x.C), ptr<float>(x.skip), ptr(x.gate),
                       ptr<float>(x.dt_bias), ptr<float>(s_in), ptr<int32_t>(in_pages), ptr<float>(fin),
                       ptr<int32_t>(out_pages), narrow(n_pages < 0 ? 0 : n_pages, "n_pages"), ptr<float>(h), ptr(o),
                       ptr(ws), &bytes, stream_of(x.u.device())),
          "gdn_scan_fwd");
    written({&out, &final_out});
    return tuple({&o, &fin, &h});
}

PyObject* scan_bwd(const Arguments& a) {
    a.count(17);
    const ScanIn x = scan_in(a);
    const Tensor dout = a.tensor(9, "dout"), h = a.tensor(10, "h"), offsets = a.tensor(11, "meta"),
                 dht = a.tensor(14, "dht"), given = a.tensor(16, "workspace");
    gdn_scan_desc d = scan(x, a.flag(8), 0);
    const int64_t units = sequences(d, lead_of(x.u, 1), offsets, a.integer(12), a.integer(13));
    if (!dout.defined()) invalid("dout is required");
    check_tensor("dout", dout, x.u.scalar_type(), x.u.sizes());
    if (!h.defined()) invalid("h is required: gdn_scan_fwd returns it with want_h");
    const std::vector<int64_t> sshape = {units, d.D, d.S};
    if (dht.defined()) check_tensor("dht", dht, ScalarType::Float, sshape);
    const int64_t rows = gdn_scan_h_rows(&d);
    if (rows >= 0) check_tensor("h", h, ScalarType::Float, {rows, d.D, d.S});
    need_dense(x.u, {{"dout", &dout}, {"h", &h}, {"dht", &dht}});
    scan_devices(x, {{"unit metadata", &offsets}, {"dout", &dout}, {"h", &h}, {"dht", &dht}});
    const Guard guard(x.u.device());
    size_t bytes = 0;
    check(gdn_scan_bwd(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, x.u.device());
    bytes = (size_t)ws.numel();
    const Tensor du = at::empty(x.u.sizes(), x.u.options()), ddt = at::empty(x.u.sizes(), x.u.options()),
                 dB = at::empty(x.B.sizes(), x.u.options()), dC = at::empty(x.B.sizes(), x.u.options()),
                 dA = floats(x.u, x.A.sizes()), dgate = x.gate.defined() ? at::empty(x.u.sizes(), x.u.options()) : Tensor(),
                 dskip = x.skip.defined() ? floats(x.u, {d.D}) : Tensor(),
                 dbias = x.dt_bias.defined() ? floats(x.u, {d.D}) : Tensor(),
                 dh0 = a.flag(15) ? floats(x.u, sshape) : Tensor();
    check(gdn_scan_bwd(&d, ptr(x.u), ptr(x.dt), ptr<float>(x.A), ptr(x.B), ptr(x.C), ptr<float>(x.skip), ptr(x.gate),
                       ptr<float>(x.dt_bias), ptr<float>(h), ptr(dout), ptr<float>(dht), ptr(du), ptr(ddt),
                       ptr<float>(dA), ptr(dB), ptr(dC), ptr<float>(dskip), ptr(dgate), ptr<float>(dbias),
                       ptr<float>(dh0), ptr(ws), &bytes, stream_of(x.u.device())),
          "gdn_scan_bwd");
    return dict({{"du", &du}, {"ddt", &ddt}, {"dA", &dA}, {"dB", &dB}, {"dC", &dC}, {"dskip", &dskip},
                 {"dgate", &dgate}, {"ddt_bias", &dbias}, {"dh0", &dh0}});
}

PyObject* scan_step(const Arguments& a) {
    a.count(12);
    const ScanIn x = scan_in(a);
    const Tensor state = a.tensor(9, "state"), pages = a.tensor(10, "pages"), out = a.tensor(11, "out");
    gdn_scan_desc d = scan(x, a.flag(8), 1);
    const int64_t N = x.u.size(0);
    if (!state.defined() || state.dim() != 3) invalid("state must be [n_pages, D, S]");
    check_tensor("state", state, ScalarType::Float, {state.size(0), d.D, d.S});
    if (!pages.defined() && state.size(0) < N)
        invalid("state has " + std::to_string(state.size(0)) + " pages for " + std::to_string(N) + " rows");
    if (pages.defined()) check_tensor("pages", pages, ScalarType::Int, {N});
    if (out.defined()) check_tensor("out", out, x.u.scalar_type(), x.u.sizes());
    scan_apart(out, x);
    check_apart(out, {{"state", &state}});
    scan_apart(state, x);
    need_dense(x.u, {{"state", &state}, {"out", &out}});
    d.B = narrow(N, "N");
    d.T = 1;
    scan_devices(x, {{"state", &state}, {"pages", &pages}, {"out", &out}});
    const Guard guard(x.u.device());
    const Tensor o = out.defined() ? out : at::empty(x.u.sizes(), x.u.options());
    check(gdn_scan_step(&d, ptr(x.u), ptr(x.dt), ptr<float>(x.A), ptr(x.B), ptr(x.C), ptr<float>(x.skip), ptr(x.gate),
                        ptr<float>(x.dt_bias), ptr<int32_t>(pages), narrow(state.size(0), "n_pages"),
                        ptr<float>(state), ptr(o), stream_of(x.u.device())),
          "gdn_scan_step");
    written({&state, &out});
    return THPVariable_Wrap(o);
}

// ---- norms and rotation
struct RotaryIn {
    Tensor q, k, freqs, positions, q_weight, k_weight;
};

// arguments 0 .. 9: q, k, freqs, positions, norm, q_weight, k_weight, eps, interleaved, amplitude
RotaryIn rotary_in(const Arguments& a) {
    return {a.tensor(0, "q"), a.tensor(1, "k"), a.tensor(2, "freqs"), a.tensor(3, "positions"),
            a.tensor(5, "q_weight"), a.tensor(6, "k_weight")};
}

float number(const Arguments& a, int i, const char* what) {
    const double x = PyFloat_AsDouble(a.a[i]);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        invalid(std::string(what) + " must be a number");
    }
    return (float)x;
}

gdn_rotary_desc rotary(const Arguments& a, const RotaryIn& x) {
    if (!x.q.defined() || (x.q.dim() != 3 && x.q.dim() != 4)) invalid("q must have shape [B,T,Hq,D] or [T,Hq,D]");
    if (!x.k.defined() || x.k.dim() != x.q.dim()) invalid("k must have q's tokens and width");
    gdn_rotary_desc d;
    memset(&d, 0, sizeof(d));
    const int64_t D = x.q.size(-1);
    const at::IntArrayRef lead = lead_of(x.q, 2);
    check_like("k", x.k, x.q.scalar_type(), with(lead, {x.k.size(-2), D}));
    d.B = lead.size() == 2 ? narrow(lead[0], "B") : 1;
    d.T = narrow(lead[lead.size() - 1], "T");
    d.Hq = narrow(x.q.size(-2), "heads");
    d.Hk = narrow(x.k.size(-2), "heads");
    if (d.Hq < 1 || d.Hk < 1) invalid("q and k need heads");
    d.D = narrow(D, "D");
    d.dtype = dtype_code(x.q.scalar_type());
    if (D < 8 || D % 8 || D > 256) throw std::logic_error("rows of " + std::to_string(D) + " values");
    if (x.freqs.defined()) {
        check_tensor("freqs", x.freqs, ScalarType::Double, {x.freqs.numel()});
        const int64_t R = 2 * x.freqs.numel();
        if (R > D) invalid("freqs turn " + std::to_string(R) + " of " + std::to_string(D) + " values");
        if (R % 8) throw std::logic_error("rotations of " + std::to_string(R) + " values");
        d.R = (int32_t)R;
    }
    if (x.positions.defined()) {
        const ScalarType t = x.positions.scalar_type();
        if (t != ScalarType::Int && t != ScalarType::Long) invalid("positions must be torch.int32 or torch.int64, got " + dtype_text(t));
        check_tensor("positions", x.positions, t, lead);
        d.pos_i64 = t == ScalarType::Long;
    } else if (lead.size() == 1 && d.R > 0) {
        invalid("packed q and k need positions");
    }
    d.norm = narrow(a.integer(4), "norm");
    d.w_dtype = parameters({{"q_weight", &x.q_weight}, {"k_weight", &x.k_weight}});
    if (x.q_weight.defined()) check_tensor("q_weight", x.q_weight, x.q_weight.scalar_type(), {D});
    if (x.k_weight.defined()) check_tensor("k_weight", x.k_weight, x.k_weight.scalar_type(), {D});
    d.eps = number(a, 7, "eps");
    d.interleaved = a.flag(8);
    d.amplitude = number(a, 9, "amplitude");
    row_strides("q", x.q, d.q_stride);
    row_strides("k", x.k, d.k_stride);
    need_dense(x.q, {{"q_weight", &x.q_weight}, {"k_weight", &x.k_weight}});
    return d;
}

// One of the inputs itself, or apart from all of them
void check_in_place(const char* name, const Tensor& out, const Tensor& in, Named others) {
    if (!out.defined()) return;
    check_apart(out, others);
    if (!(in.is_contiguous() && out.data_ptr() == in.data_ptr())) check_apart(out, {{name, &in}});
}

void rotary_devices(const RotaryIn& x, Named more) {
    check_devices(x.q, {{"k", &x.k}, {"freqs", &x.freqs}, {"positions", &x.positions}, {"q_weight", &x.q_weight},
                        {"k_weight", &x.k_weight}});
    check_devices(x.q, more);
}

PyObject* rotary_fwd(const Arguments& a) {
    a.count(12);
    const RotaryIn x = rotary_in(a);
    const Tensor q_out = a.tensor(10, "q_out"), k_out = a.tensor(11, "k_out");
    const gdn_rotary_desc d = rotary(a, x);
    if (q_out.defined()) check_tensor("q_out", q_out, x.q.scalar_type(), x.q.sizes());
    if (k_out.defined()) check_tensor("k_out", k_out, x.k.scalar_type(), x.k.sizes());
    const Named rest = {{"freqs", &x.freqs}, {"positions", &x.positions}, {"q_weight", &x.q_weight}, {"k_weight", &x.k_weight}};
    check_in_place("q", q_out, x.q, rest);
    check_in_place("k", k_out, x.k, rest);
    check_apart(q_out, {{"k", &x.k}, {"k_out", &k_out}});
    check_apart(k_out, {{"q", &x.q}});
    need_dense(x.q, {{"q_out", &q_out}, {"k_out", &k_out}});
    rotary_devices(x, {{"q_out", &q_out}, {"k_out", &k_out}});
    const Guard guard(x.q.device());
    const Tensor q = q_out.defined() ? q_out : at::empty(x.q.sizes(), x.q.options()),
                 k = k_out.defined() ? k_out : at::empty(x.k.sizes(), x.k.options());
    check(gdn_qk_rotary_fwd(&d, ptr(x.q), ptr(x.k), ptr<double>(x.freqs), ptr(x.positions), ptr(x.q_weight),
                            ptr(x.k_weight), ptr(q), ptr(k), stream_of(x.q.device())),
          "gdn_qk_rotary_fwd");
    written({&q_out, &k_out});
    return tuple({&q, &k});
}

PyObject* rotary_bwd(const Arguments& a) {
    a.count(13);
    const RotaryIn x = rotary_in(a);
    const Tensor dq_out = a.tensor(10, "dq_out"), dk_out = a.tensor(11, "dk_out"), given = a.tensor(12, "workspace");
    const gdn_rotary_desc d = rotary(a, x);
    if (!dq_out.defined()) invalid("dq_out is required");
    if (!dk_out.defined()) invalid("dk_out is required");
    check_tensor("dq_out", dq_out, x.q.scalar_type(), x.q.sizes());
    check_tensor("dk_out", dk_out, x.k.scalar_type(), x.k.sizes());
    need_dense(x.q, {{"dq_out", &dq_out}, {"dk_out", &dk_out}});
    rotary_devices(x, {{"dq_out", &dq_out}, {"dk_out", &dk_out}});
    const Guard guard(x.q.device());
    size_t bytes = 0;
    check(gdn_qk_rotary_bwd(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                            nullptr, nullptr, nullptr, nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, x.q.device());
    bytes = (size_t)ws.numel();
    const Tensor dq = at::empty(x.q.sizes(), x.q.options()), dk = at::empty(x.k.sizes(), x.k.options()),
                 dqw = x.q_weight.defined() ? floats(x.q, {d.D}) : Tensor(),
                 dkw = x.k_weight.defined() ? floats(x.q, {d.D}) : Tensor();
    check(gdn_qk_rotary_bwd(&d, ptr(x.q), ptr(x.k), ptr<double>(x.freqs), ptr(x.positions), ptr(x.q_weight),
                            ptr(x.k_weight), ptr(dq_out), ptr(dk_out), ptr(dq), ptr(dk), ptr<float>(dqw),
                            ptr<float>(dkw), ptr(ws), &bytes, stream_of(x.q.device())),
          "gdn_qk_rotary_bwd");
    return dict({{"dq", &dq}, {"dk", &dk}, {"dq_weight", &dqw}, {"dk_weight", &dkw}});
}

PyMethodDef methods[] = {method<conv_fwd>("conv_fwd"),     method<conv_bwd>("conv_bwd"),
                         method<conv_step>("conv_step"),   method<scan_fwd>("scan_fwd"),
                         method<scan_bwd>("scan_bwd"),     method<scan_step>("scan_step"),
                         method<rotary_fwd>("rotary_fwd"), method<rotary_bwd>("rotary_bwd"),
                         {nullptr, nullptr, 0, nullptr}};

}  // namespace

PyMethodDef* mixer_methods() { return methods; }
