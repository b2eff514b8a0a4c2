// Torch marshalling of the recurrent-state operators (include/gdn_recurrent.h):
// the argument checks, output and workspace allocation and the current stream
// behind binding.py's functions of the same names. It is native because a
// decode step's kernel takes 4 us: done in Python, the checks of one call take
// four times as long. Functions take their arguments by position and are
// called through binding.py only. ValueError: a contract violation;
// NotImplementedError, RuntimeError: as check() in binding.py.
#include "gdn_torch.h"

#include "gdn_recurrent.h"

namespace {

using namespace gdn_torch;

// q, k, v of one dtype and leading shape, with heads that divide H
void check_qkv(const Tensor& q, const Tensor& k, const Tensor& v, int64_t H, const char* lead_text) {
    const int64_t d = k.dim();
    const std::pair<const char*, const Tensor*> all[] = {{"q", &q}, {"k", &k}, {"v", &v}};
    for (const auto& [name, t] : all) {
        if (!t->defined() || t->dim() != d || t->sizes().slice(0, d - 2) != k.sizes().slice(0, d - 2))
            invalid(std::string(name) + " must have shape " + lead_text + " like k");
        if (t->scalar_type() != k.scalar_type())
            invalid(std::string(name) + " must be " + dtype_text(k.scalar_type()) + ", got " + dtype_text(t->scalar_type()));
        if (t->size(d - 2) < 1 || H < 1 || H % t->size(d - 2))
            invalid(std::string(name) + " has " + std::to_string(t->size(d - 2)) + " heads, which do not divide " + std::to_string(H));
    }
    if (q.size(d - 1) != k.size(d - 1))
        invalid("q must have k's width " + std::to_string(k.size(d - 1)) + ", got " + std::to_string(q.size(d - 1)));
}

// ---- prompts
struct Prompt {
    gdn_linattn_desc d;
    int64_t units;
    c10::Device dev{c10::DeviceType::CPU};
    std::vector<int64_t> lead;   // token axes

    std::vector<int64_t> tokens(std::initializer_list<int64_t> rest) const {
        std::vector<int64_t> s(lead);
        s.insert(s.end(), rest);
        return s;
    }
};

// offsets: the device offsets of packed documents or undefined; n_units and
// host: their number and host copy
Prompt prompt(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& decay, const Tensor& offsets,
              int64_t n_units, int64_t host, ScalarType o_dtype) {
    if (!k.defined() || (k.dim() != 3 && k.dim() != 4))
        invalid("linear attention inputs must have shape [B,T,h,K] or [T,h,K]");
    if (k.dim() == 3 && !offsets.defined()) invalid("packed inputs [T,h,K] need meta");
    if (k.dim() == 4 && offsets.defined()) invalid("meta goes with packed inputs [T,h,K]");
    if (!decay.defined() || decay.dim() != 1) invalid("decay must be fp32 [H]");
    check_qkv(q, k, v, decay.size(0), "[..,heads,width]");
    Prompt p;
    const int64_t n = k.dim();
    p.lead.assign(k.sizes().begin(), k.sizes().end() - 2);
    memset(&p.d, 0, sizeof(p.d));
    p.d.B = n == 4 ? narrow(k.size(0), "B") : 1;
    p.d.T = narrow(k.size(n - 3), "T");
    p.d.H = narrow(decay.size(0), "H");
    p.d.Hq = narrow(q.size(n - 2), "heads");
    p.d.Hk = narrow(k.size(n - 2), "heads");
    p.d.Hv = narrow(v.size(n - 2), "heads");
    p.d.K = narrow(k.size(n - 1), "K");
    p.d.V = narrow(v.size(n - 1), "V");
    p.d.dtype = dtype_code(k.scalar_type());
    p.d.o_dtype = dtype_code(o_dtype);
    row_strides("q", q, p.d.q_stride);
    row_strides("k", k, p.d.k_stride);
    row_strides("v", v, p.d.v_stride);
    p.units = n == 4 ? p.d.B : n_units;
    if (offsets.defined()) {
        if (n_units < 1) invalid("meta has no documents");
        check_tensor("meta's device offsets", offsets, ScalarType::Int, {n_units + 1});
        p.d.n_units = narrow(n_units, "units");
        p.d.offsets_host = reinterpret_cast<const int32_t*>(host);
        p.d.offsets_dev = ptr<int32_t>(offsets);
    }
    p.dev = k.device();
    check_tensor("decay", decay, ScalarType::Float, {decay.size(0)});
    return p;
}

void prompt_devices(const Prompt& p, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& decay,
                    const Tensor& offsets) {
    need_gpu("inputs", k);
    check_device("q", q, p.dev);
    check_device("v", v, p.dev);
    check_device("decay", decay, p.dev);
    check_device("unit metadata", offsets, p.dev);
}

PyObject* linattn_fwd(const Arguments& a) {
    a.count(16);
    const Tensor q = a.tensor(0, "q"), k = a.tensor(1, "k"), v = a.tensor(2, "v"), decay = a.tensor(3, "decay");
    const Tensor offsets = a.tensor(5, "meta"), s_in = a.tensor(8, "initial_state"),
                 in_pages = a.tensor(9, "initial_pages"), final_out = a.tensor(11, "final_out"),
                 out_pages = a.tensor(12, "final_pages"), out = a.tensor(14, "out"), given = a.tensor(15, "workspace");
    if (!k.defined()) invalid("linear attention inputs must have shape [B,T,h,K] or [T,h,K]");
    const ScalarType ot = a.o_dtype(13, out, k.scalar_type());
    Prompt p = prompt(q, k, v, decay, offsets, a.integer(6), a.integer(7), ot);
    p.d.scale = a.scale(4, p.d.K);
    const std::vector<int64_t> oshape = p.tokens({p.d.H, p.d.V});
    if (out.defined()) check_tensor("out", out, ot, oshape);
    if (in_pages.defined()) check_tensor("initial_pages", in_pages, ScalarType::Int, {p.units});
    if (out_pages.defined()) check_tensor("final_pages", out_pages, ScalarType::Int, {p.units});
    int64_t n_pages = -1;
    auto state = [&](const char* name, const Tensor& t, const Tensor& pages) {
        if (pages.defined() && (!t.defined() || t.dim() != 4))
            invalid(std::string(name) + " must be a pool [n_pages,H,K,V] when its pages are given");
        if (!t.defined()) return;
        const int64_t n = pages.defined() ? t.size(0) : p.units;
        check_tensor(name, t, ScalarType::Float, {n, p.d.H, p.d.K, p.d.V});
        if (pages.defined()) {
            if (n_pages >= 0 && n_pages != n)
                invalid("the pools have " + std::to_string(n_pages) + " and " + std::to_string(n) + " pages");
            n_pages = n;
        }
    };
    state("initial_state", s_in, in_pages);
    state("final_out", final_out, out_pages);
    check_apart(out, {{"q", &q}, {"k", &k}, {"v", &v}, {"initial_state", &s_in}, {"final_out", &final_out}});
    prompt_devices(p, q, k, v, decay, offsets);
    check_device("out", out, p.dev);
    check_device("initial_state", s_in, p.dev);
    check_device("initial_pages", in_pages, p.dev);
    check_device("final_out", final_out, p.dev);
    check_device("final_pages", out_pages, p.dev);
    const Guard guard(p.dev);
    size_t bytes = 0;
    check(gdn_linattn_fwd(&p.d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr,
                          nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, p.dev);
    bytes = (size_t)ws.numel();
    const Tensor o = out.defined() ? out : at::empty(oshape, k.options().dtype(ot));
    Tensor fin = final_out;
    if (!fin.defined() && a.flag(10))
        fin = at::empty({p.units, p.d.H, p.d.K, p.d.V}, k.options().dtype(ScalarType::Float));
    check(gdn_linattn_fwd(&p.d, ptr(q), ptr(k), ptr(v), ptr<float>(decay), ptr<float>(s_in), ptr<int32_t>(in_pages),
                          ptr<float>(fin), ptr<int32_t>(out_pages), narrow(n_pages < 0 ? 0 : n_pages, "n_pages"),
                          ptr(o), ptr(ws), &bytes, stream_of(p.dev)),
          "gdn_linattn_fwd");
    written({&out, &final_out});
    PyObject* po = THPVariable_Wrap(o);
    PyObject* pf = fin.defined() ? THPVariable_Wrap(fin) : Py_NewRef(Py_None);
    PyObject* r = PyTuple_Pack(2, po, pf);
    Py_DECREF(po);
    Py_DECREF(pf);
    return r;
}

PyObject* linattn_bwd(const Arguments& a) {
    a.count(13);
    const Tensor q = a.tensor(0, "q"), k = a.tensor(1, "k"), v = a.tensor(2, "v"), decay = a.tensor(3, "decay"),
                 dout = a.tensor(4, "dout"), offsets = a.tensor(6, "meta"), s_in = a.tensor(9, "initial_state"),
                 dht = a.tensor(10, "dht"), given = a.tensor(12, "workspace");
    if (!k.defined()) invalid("linear attention inputs must have shape [B,T,h,K] or [T,h,K]");
    dtype_code(k.scalar_type());
    Prompt p = prompt(q, k, v, decay, offsets, a.integer(7), a.integer(8), k.scalar_type());
    p.d.scale = a.scale(5, p.d.K);
    if (!dout.defined()) invalid("dout is required");
    check_tensor("dout", dout, k.scalar_type(), p.tokens({p.d.H, p.d.V}));
    const std::vector<int64_t> sshape = {p.units, p.d.H, p.d.K, p.d.V};
    if (s_in.defined()) check_tensor("initial_state", s_in, ScalarType::Float, sshape);
    if (dht.defined()) check_tensor("dht", dht, ScalarType::Float, sshape);
    prompt_devices(p, q, k, v, decay, offsets);
    check_device("dout", dout, p.dev);
    check_device("initial_state", s_in, p.dev);
    check_device("dht", dht, p.dev);
    const Guard guard(p.dev);
    size_t bytes = 0;
    check(gdn_linattn_bwd(&p.d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                          nullptr, nullptr, nullptr, &bytes, nullptr),
          "workspace query");
    const Tensor ws = workspace_of(given, bytes, p.dev);
    bytes = (size_t)ws.numel();
    const Tensor dq = at::empty(q.sizes(), k.options()), dk = at::empty(k.sizes(), k.options()),
                 dv = at::empty(v.sizes(), k.options());
    const Tensor dh0 = a.flag(11) ? at::empty(sshape, k.options().dtype(ScalarType::Float)) : Tensor();
    check(gdn_linattn_bwd(&p.d, ptr(q), ptr(k), ptr(v), ptr<float>(decay), ptr<float>(s_in), ptr(dout), ptr<float>(dht),
                          ptr(dq), ptr(dk), ptr(dv), ptr<float>(dh0), ptr(ws), &bytes, stream_of(p.dev)),
          "gdn_linattn_bwd");
    PyObject* r = PyDict_New();
    const std::pair<const char*, const Tensor*> all[] = {{"dq", &dq}, {"dk", &dk}, {"dv", &dv}, {"dh0", &dh0}};
    for (const auto& [name, t] : all) {
        if (!t->defined()) continue;
        PyObject* x = THPVariable_Wrap(*t);
        PyDict_SetItemString(r, name, x);
        Py_DECREF(x);
    }
    return r;
}

// ---- single tokens
gdn_step_desc step(const Tensor& q, const Tensor& k, const Tensor& v, int64_t H, const Tensor& state,
                   const Tensor& pages, const Tensor& out, ScalarType ot) {
    check_qkv(q, k, v, H, "[N,heads,width]");
    if (!state.defined() || state.dim() != 4) invalid("state must be [n_pages, H, K, V]");
    const int64_t N = k.size(0), K = k.size(2), V = v.size(2);
    check_tensor("state", state, ScalarType::Float, {state.size(0), H, K, V});
    if (!pages.defined() && state.size(0) < N)
        invalid("state has " + std::to_string(state.size(0)) + " pages for " + std::to_string(N) + " rows");
    if (pages.defined()) check_tensor("pages", pages, ScalarType::Int, {N});
    if (out.defined()) check_tensor("out", out, ot, {N, H, V});
    gdn_step_desc d;
    memset(&d, 0, sizeof(d));
    d.N = narrow(N, "N");
    d.H = narrow(H, "H");
    d.Hq = narrow(q.size(1), "heads");
    d.Hk = narrow(k.size(1), "heads");
    d.Hv = narrow(v.size(1), "heads");
    d.K = narrow(K, "K");
    d.V = narrow(V, "V");
    d.dtype = dtype_code(k.scalar_type());
    d.o_dtype = dtype_code(ot);
    d.n_pages = narrow(state.size(0), "n_pages");
    row_strides("q", q, d.q_stride);
    row_strides("k", k, d.k_stride);
    row_strides("v", v, d.v_stride);
    check_apart(out, {{"q", &q}, {"k", &k}, {"v", &v}, {"state", &state}});
    return d;
}

void step_devices(const Tensor& k, std::initializer_list<std::pair<const char*, const Tensor*>> others) {
    need_gpu("inputs", k);
    for (const auto& [name, t] : others) check_device(name, *t, k.device());
}

PyObject* linattn_step(const Arguments& a) {
    a.count(9);
    const Tensor q = a.tensor(0, "q"), k = a.tensor(1, "k"), v = a.tensor(2, "v"), decay = a.tensor(3, "decay"),
                 state = a.tensor(4, "state"), pages = a.tensor(6, "pages"), out = a.tensor(8, "out");
    if (!k.defined() || k.dim() != 3) invalid("step inputs must have shape [N, heads, width]");
    if (!decay.defined() || decay.dim() != 1) invalid("decay must be fp32 [H]");
    const ScalarType ot = a.o_dtype(7, out, k.scalar_type());
    gdn_step_desc d = step(q, k, v, decay.size(0), state, pages, out, ot);
    d.scale = a.scale(5, d.K);
    check_tensor("decay", decay, ScalarType::Float, {d.H});
    step_devices(k, {{"q", &q}, {"v", &v}, {"state", &state}, {"pages", &pages}, {"decay", &decay}, {"out", &out}});
    const Guard guard(k.device());
    const Tensor o = out.defined() ? out : at::empty({d.N, d.H, d.V}, k.options().dtype(ot));
    check(gdn_linattn_step(&d, ptr(q), ptr(k), ptr(v), ptr<float>(decay), ptr<int32_t>(pages), ptr<float>(state),
                           ptr(o), stream_of(k.device())),
          "gdn_linattn_step");
    written({&state, &out});
    return THPVariable_Wrap(o);
}

PyObject* recurrent_step(const Arguments& a) {
    a.count(12);
    const Tensor q = a.tensor(0, "q"), k = a.tensor(1, "k"), v = a.tensor(2, "v"), g = a.tensor(3, "g"),
                 beta = a.tensor(4, "beta"), state = a.tensor(5, "state"), pages = a.tensor(7, "pages"),
                 out = a.tensor(11, "out");
    if (!k.defined() || k.dim() != 3) invalid("step inputs must have shape [N, heads, width]");
    if (!beta.defined() || beta.dim() != 2) invalid("beta must be [N, H]");
    if (!g.defined() || (g.dim() != 2 && g.dim() != 3))
        invalid("g must be [N, H] (scalar gate) or [N, H, K] (per-key gate)");
    const ScalarType ot = a.o_dtype(10, out, k.scalar_type());
    gdn_step_desc d = step(q, k, v, beta.size(1), state, pages, out, ot);
    d.scale = a.scale(6, d.K);
    if (g.dim() == 2) check_tensor("g", g, ScalarType::Float, {d.N, d.H});
    else check_tensor("g", g, ScalarType::Float, {d.N, d.H, d.K});
    check_tensor("beta", beta, k.scalar_type(), {d.N, d.H});
    step_devices(k, {{"q", &q}, {"v", &v}, {"state", &state}, {"pages", &pages}, {"g", &g}, {"beta", &beta}, {"out", &out}});
    const Guard guard(k.device());
    const Tensor o = out.defined() ? out : at::empty({d.N, d.H, d.V}, k.options().dtype(ot));
    check(gdn_recurrent_step(&d, g.dim() == 3 ? GDN_GATE_PER_KEY : GDN_GATE_SCALAR, a.flag(8), ptr(q), ptr(k), ptr(v),
                             ptr<float>(g), ptr(beta), ptr<int32_t>(pages), ptr<float>(state), ptr(o),
                             narrow(a.integer(9), "flags"), stream_of(k.device())),
          "gdn_recurrent_step");
    written({&state, &out});
    return THPVariable_Wrap(o);
}

// ---- pages
struct Pool {
    int32_t layers, pages;
    int64_t bytes;   // of a page
};

Pool pool_of(const char* name, const Tensor& t) {
    if (!t.defined() || t.dim() < 3) invalid(std::string(name) + " must be [n_layers, n_pages, ...]");
    if (!t.is_contiguous()) invalid(std::string(name) + " must be contiguous");
    int64_t nb = t.element_size();
    for (int64_t i = 2; i < t.dim(); ++i) nb *= t.size(i);
    if (nb == 0 || nb % 16 || reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
        invalid(std::string(name) + ": pages must be a multiple of 16 bytes and 16-byte aligned, got " + std::to_string(nb) + " bytes");
    return Pool{narrow(t.size(0), "n_layers"), narrow(t.size(1), "n_pages"), nb};
}

int32_t list_of(const char* name, const Tensor& t) {
    if (!t.defined()) invalid(std::string(name) + " is required");
    check_tensor(name, t, ScalarType::Int, {t.numel()});
    return narrow(t.numel(), name);
}

Tensor ints(const Tensor& like, int64_t n) { return at::empty({n}, like.options().dtype(ScalarType::Int)); }

PyObject* pair(const Tensor& x, const Tensor& y) {
    PyObject* a = THPVariable_Wrap(x);
    PyObject* b = THPVariable_Wrap(y);
    PyObject* r = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return r;
}

PyObject* pages_copy(const Arguments& a) {
    a.count(4);
    const Tensor dst = a.tensor(0, "dst_pool"), src = a.tensor(1, "src_pool"), dp = a.tensor(2, "dst_pages"),
                 sp = a.tensor(3, "src_pages");
    const Pool d = pool_of("dst_pool", dst), s = pool_of("src_pool", src);
    if (src.scalar_type() != dst.scalar_type() || s.layers != d.layers || src.sizes().slice(2) != dst.sizes().slice(2))
        invalid("the pools differ in dtype, layers or page shape");
    const int32_t n = list_of("dst_pages", dp);
    if (!sp.defined()) invalid("src_pages is required");
    check_tensor("src_pages", sp, ScalarType::Int, {n});
    need_gpu("pools", dst);
    check_device("src_pool", src, dst.device());
    check_device("dst_pages", dp, dst.device());
    check_device("src_pages", sp, dst.device());
    const Guard guard(dst.device());
    check(gdn_pages_copy(ptr(dst), d.pages, ptr(src), s.pages, d.layers, d.bytes, ptr<int32_t>(dp), ptr<int32_t>(sp), n,
                         stream_of(dst.device())),
          "gdn_pages_copy");
    written({&dst});
    Py_RETURN_NONE;
}

PyObject* pages_fork(const Arguments& a) {
    a.count(4);
    const Tensor pool = a.tensor(0, "pool"), table = a.tensor(1, "table"), parent = a.tensor(2, "parent"),
                 spare = a.tensor(3, "spare");
    const Pool p = pool_of("pool", pool);
    const int32_t n = list_of("table", table);
    if (!parent.defined()) invalid("parent is required");
    check_tensor("parent", parent, ScalarType::Int, {n});
    const int32_t m = spare.defined() ? list_of("spare", spare) : 0;
    need_gpu("pools", pool);
    check_device("table", table, pool.device());
    check_device("parent", parent, pool.device());
    check_device("spare", spare, pool.device());
    const Guard guard(pool.device());
    const Tensor made = ints(pool, n), left = ints(pool, (int64_t)n + m),
                 ws = ints(pool, (int64_t)gdn_pages_workspace_ints(n));
    check(gdn_pages_fork(ptr(pool), p.layers, p.pages, p.bytes, ptr<int32_t>(table), ptr<int32_t>(parent), n,
                         ptr<int32_t>(spare), m, ptr<int32_t>(made), ptr<int32_t>(left), ptr<int32_t>(ws),
                         stream_of(pool.device())),
          "gdn_pages_fork");
    written({&pool});
    return pair(made, left);
}

PyObject* pages_compact(const Arguments& a) {
    a.count(2);
    const Tensor pool = a.tensor(0, "pool"), table = a.tensor(1, "table");
    const Pool p = pool_of("pool", pool);
    const int32_t n = list_of("table", table);
    need_gpu("pools", pool);
    check_device("table", table, pool.device());
    const Guard guard(pool.device());
    const Tensor made = ints(pool, n), count = ints(pool, 1), ws = ints(pool, (int64_t)gdn_pages_workspace_ints(p.pages));
    check(gdn_pages_compact(ptr(pool), p.layers, p.pages, p.bytes, ptr<int32_t>(table), n, ptr<int32_t>(made),
                            ptr<int32_t>(count), ptr<int32_t>(ws), stream_of(pool.device())),
          "gdn_pages_compact");
    written({&pool});
    return pair(made, count);
}

// ---- module
PyMethodDef methods[] = {method<linattn_fwd>("linattn_fwd"),       method<linattn_bwd>("linattn_bwd"),
                         method<linattn_step>("linattn_step"),     method<recurrent_step>("recurrent_step"),
                         method<pages_copy>("pages_copy"),         method<pages_fork>("pages_fork"),
                         method<pages_compact>("pages_compact"),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMethodDef* mixer_methods();   // gdn_mixer_torch.cpp

PyMODINIT_FUNC PyInit__native() {
    PyObject* m = PyModule_Create(&module_def);
    if (m && PyModule_AddFunctions(m, mixer_methods()) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
