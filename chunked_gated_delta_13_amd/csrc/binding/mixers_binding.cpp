// Binding of the token mixers: tensors in, one call of the C ABI each.
//
// A token of these operators keeps the device busy for a few microseconds, so checks and marshalling
// count: here they take about 1 us of a call (2.5 with two tensors to allocate), written in Python 5.5 to
// 9.  One token of the convolution, of the scan and of the attention takes 4.6, 4.9 and 10.2 us a call, 3.4,
// 3.8 and 6.4 of them the host's part of the library's own launches.  The entry points of libkda are handed over by
// bind(), so that a process holds one copy of the library; nothing here is linked to it.
#include <Python.h>

#include <string.h>

#include <cmath>
#include <string>
#include <type_traits>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

using at::Tensor;
typedef c10::SmallVector<int64_t, 6> Shape;

struct Library {
    decltype(&kda_conv_prefill) conv_prefill;
    decltype(&kda_conv_step) conv_step;
    decltype(&kda_ssm_prefill_workspace_bytes) ssm_prefill_workspace_bytes;
    decltype(&kda_ssm_prefill) ssm_prefill;
    decltype(&kda_ssm_step) ssm_step;
    decltype(&kda_window_prefill_workspace_bytes) window_prefill_workspace_bytes;
    decltype(&kda_window_prefill) window_prefill;
    decltype(&kda_window_step_workspace_bytes) window_step_workspace_bytes;
    decltype(&kda_window_step) window_step;
} lib;
PyObject* on_status = nullptr;   // called with a status and the name of the call that returned it

struct WrongValue : torch::PyTorchError {
    using PyTorchError::PyTorchError;
    PyObject* python_type() override { return PyExc_ValueError; }
};
struct WrongType : torch::PyTorchError {
    using PyTorchError::PyTorchError;
    PyObject* python_type() override { return PyExc_TypeError; }
};

std::string text(const std::string& s) { return s; }
std::string text(int64_t n) { return std::to_string(n); }
std::string text(c10::Device d) { return d.str(); }
std::string text(at::ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }
std::string text(c10::IntArrayRef s) {
    std::string o = "(";
    for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
    return o + (s.size() == 1 ? ",)" : ")");
}

// An error whose message joins its parts.
template <typename E, typename... P> E refusal(const P&... parts) { return E((text(parts) + ...)); }

// The calls' arguments, in the order the wrappers pass them.
struct Args {
    PyObject* const* a;
    const Tensor& tensor(int i, const char* name) const {
        if (!THPVariable_Check(a[i])) throw refusal<WrongType>(name, " must be a tensor, got ", Py_TYPE(a[i])->tp_name);
        return THPVariable_Unpack(a[i]);
    }
    const Tensor* optional(int i, const char* name) const { return a[i] == Py_None ? nullptr : &tensor(i, name); }
    int size(int i) const {   // sizes are 32-bit numbers at the library's entry points
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(a[i], &over);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        if (over || v > INT32_MAX || v < -INT32_MAX) throw refusal<WrongValue>("sizes must fit 32 bits, got ", over ? std::string("more") : std::to_string(v));
        return (int)v;
    }
    bool truth(int i) const {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) throw python_error();
        return v != 0;
    }
    float scale(int i, int64_t d) const {
        if (a[i] == Py_None) return 1.0f / std::sqrt((float)(d > 0 ? d : 1));
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return (float)v;
    }
};

int size(int64_t n) {
    if (n > INT32_MAX) throw refusal<WrongValue>("sizes must fit 32 bits, got ", n);
    return (int)n;
}

// What the tensors of one call have in common.
struct Common {
    const char* where;
    at::ScalarType type;
    c10::Device dev;
    kda_dtype_t code;

    Common(const char* where_, const Tensor& t) : where(where_), type(t.scalar_type()), dev(t.device()) {
        if (!t.is_cuda()) throw refusal<WrongValue>(where, " runs on a HIP device; got a tensor on ", dev);
        if (type == at::kBFloat16) code = KDA_BF16;
        else if (type == at::kFloat) code = KDA_F32;
        else throw refusal<WrongType>("inputs must be bfloat16 or float32, got ", type);
    }
    // exactly this type, shape and device
    void like(const char* name, const Tensor& t, at::ScalarType ty, c10::IntArrayRef shape) const {
        if (t.scalar_type() != ty) throw refusal<WrongType>(name, " must be ", ty, ", got ", t.scalar_type());
        if (t.sizes() != shape) throw refusal<WrongValue>(name, " must have shape ", shape, ", got ", t.sizes());
        if (t.device() != dev) throw refusal<WrongValue>(name, " must be on ", dev, ", got ", t.device());
        memory(name, t);
    }
    // Batches of torch.vmap, wrappers of torch.func and fake tensors have none that a kernel could use.
    static void memory(const char* name, const Tensor& t) {
        if (!t.has_storage() || (t.numel() > 0 && t.const_data_ptr() == nullptr))
            throw refusal<WrongValue>(name, " has no memory of its own (calls inside torch.vmap, torch.func or a fake tensor mode are not supported)");
    }
    void whole(const char* name, const Tensor& t, at::ScalarType ty, c10::IntArrayRef shape) const {
        like(name, t, ty, shape);
        if (!t.is_contiguous()) throw refusal<WrongValue>(name, " must be contiguous");
    }
    // A tensor whose first `lead` axes are rows and whose other axes (none, one or two) are contiguous inside
    // a row: the stride between rows in elements.
    long long rows(const char* name, const Tensor& t, c10::IntArrayRef shape, int lead) const {
        like(name, t, type, shape);
        const c10::IntArrayRef st = t.strides();
        int64_t width = 1;
        for (int i = (int)shape.size() - 1; i >= lead; --i) {
            if (shape[i] > 1 && st[i] != width && t.numel() > 0) throw refusal<WrongValue>(name, ": the elements of a token must be contiguous");
            width *= shape[i];
        }
        if (lead == 1) return shape[0] > 1 ? st[0] : width;
        const int64_t step = shape[1] > 1 ? st[1] : (shape[0] > 1 ? st[0] : width);
        if (shape[0] > 1 && shape[1] > 0 && st[0] != step * shape[1])
            throw refusal<WrongValue>(name, ": sequence b must start at row b * T of evenly spaced rows");
        return step;
    }
    Tensor fresh(c10::IntArrayRef shape, at::ScalarType ty) const { return at::empty(shape, at::TensorOptions().dtype(ty).device(dev)); }

    // The library call on the current stream of the tensors' device; that device has to be current.  The
    // arguments are plain values, formed before the interpreter lock is released: taking a tensor's pointer
    // can throw, and an exception must not leave the part that runs without the lock.
    template <typename F, typename... A> bool call(F* f, A... a) const {
        static_assert((std::is_scalar_v<A> && ...), "pointers, numbers and enumerators only");
        void* stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = f(a..., stream);
        Py_END_ALLOW_THREADS
        if (st == KDA_OK) return true;
        PyObject* r = PyObject_CallFunction(on_status, "is", st, where);
        Py_XDECREF(r);
        if (r) PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, st);
        return false;
    }
};

// Makes a device current for as long as it lives, where another one is.
struct OnDevice {
    c10::OptionalDeviceGuard guard;
    explicit OnDevice(c10::Device dev) {
        if (c10::hip::current_device() != dev.index()) guard.reset_device(dev);
    }
};

void* ptr(const Tensor& t) { return t.data_ptr(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T> T* at_type(const Tensor* t) { return reinterpret_cast<T*>(ptr(t)); }

// An output: the caller's tensor, a new one, or none.
struct Output {
    Tensor own;
    PyObject* given = nullptr;
    bool none = false;
    void* ptr() const { return none ? nullptr : (given ? THPVariable_Unpack(given).data_ptr() : own.data_ptr()); }
    PyObject* object() const {
        if (none) Py_RETURN_NONE;
        if (!given) return THPVariable_Wrap(own);
        Py_INCREF(given);
        return given;
    }
};
// Argument i, checked, or a new tensor where it is None; `wanted` false leaves it out then.
struct Pending {
    Output out;
    Shape shape;
    at::ScalarType type;
    Pending(const Common& c, const Args& a, int i, const char* name, at::ScalarType ty, c10::IntArrayRef s, bool wanted = true)
        : shape(s.begin(), s.end()), type(ty) {
        if (const Tensor* t = a.optional(i, name)) {
            c.whole(name, *t, ty, s);
            out.given = a.a[i];
        } else {
            out.none = !wanted;
        }
    }
    const Output& make(const Common& c) {
        if (!out.given && !out.none) out.own = c.fresh(shape, type);
        return out;
    }
};

// The caller's workspace if it is large enough, else a new one.
struct Workspace {
    Tensor own;
    void* p = nullptr;
    size_t bytes = 0;
    Workspace(const Common& c, const Tensor* t, size_t need) {
        if (t) {
            if (t->device() != c.dev) throw refusal<WrongValue>("workspace must be on ", c.dev, ", got ", t->device());
            if (!t->is_contiguous()) throw refusal<WrongValue>("workspace must be contiguous");
            Common::memory("workspace", *t);
            bytes = (size_t)t->numel() * t->element_size();
            if (bytes >= need) {
                p = t->data_ptr();
                return;
            }
        }
        bytes = need;
        if (need == 0) return;
        own = c.fresh({(int64_t)need}, at::kByte);
        p = own.data_ptr();
    }
};

PyObject* pair(const Output& a, const Output& b) {
    PyObject* x = a.object();
    PyObject* y = x ? b.object() : nullptr;
    PyObject* t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// x, w, bias, state, lens, silu, y, state_out, return_state
PyObject* conv_prefill(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 9)) return nullptr;
    const Args a{args};
    const Tensor &x = a.tensor(0, "x"), &w = a.tensor(1, "w");
    const Common c("conv_prefill", x);
    if (x.dim() != 3 || w.dim() != 2) throw refusal<WrongValue>("x must be [B, T, D] and w [D, W]");
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2), W = w.size(1);
    const long long xs = c.rows("x", x, x.sizes(), 2);
    c.whole("w", w, c.type, {D, W});
    const Tensor *bias = a.optional(2, "bias"), *state = a.optional(3, "state"), *lens = a.optional(4, "lens");
    if (bias) c.whole("bias", *bias, c.type, {D});
    if (W < 1) throw refusal<WrongValue>("w must have at least one tap");
    if (state) c.whole("state", *state, c.type, {B, W - 1, D});
    if (lens) c.whole("lens", *lens, at::kInt, {B});
    const int b = size(B), t = size(T), d = size(D), taps = size(W), silu = a.truth(5);
    Pending py(c, a, 6, "y", c.type, {B, T, D}), pso(c, a, 7, "state_out", c.type, {B, W - 1, D}, a.truth(8));
    const OnDevice on(c.dev);
    const Output &y = py.make(c), &so = pso.make(c);
    if (!c.call(lib.conv_prefill, ptr(x), ptr(w), ptr(bias), ptr(state), at_type<int>(lens), y.ptr(), so.ptr(), b, t, d,
                taps, xs, silu, c.code))
        return nullptr;
    return pair(y, so);
    END_HANDLE_TH_ERRORS
}

// x, w, state, bias, silu, y
PyObject* conv_step(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 6)) return nullptr;
    const Args a{args};
    const Tensor &x = a.tensor(0, "x"), &w = a.tensor(1, "w"), &state = a.tensor(2, "state");
    const Common c("conv_step", x);
    if (x.dim() != 2 || w.dim() != 2) throw refusal<WrongValue>("x must be [N, D] and w [D, W]");
    const int64_t N = x.size(0), D = x.size(1), W = w.size(1);
    const long long xs = c.rows("x", x, x.sizes(), 1);
    c.whole("w", w, c.type, {D, W});
    const Tensor* bias = a.optional(3, "bias");
    if (bias) c.whole("bias", *bias, c.type, {D});
    if (W < 1) throw refusal<WrongValue>("w must have at least one tap");
    c.whole("state", state, c.type, {N, W - 1, D});
    const int n = size(N), d = size(D), taps = size(W), silu = a.truth(4);
    Pending py(c, a, 5, "y", c.type, {N, D});
    const OnDevice on(c.dev);
    const Output& y = py.make(c);
    if (!c.call(lib.conv_step, ptr(x), ptr(w), ptr(bias), ptr(state), y.ptr(), n, d, taps, xs, silu, c.code))
        return nullptr;
    return y.object();
    END_HANDLE_TH_ERRORS
}

// Arguments 0 .. 4 (x, dt, A, Bm, Cm) and from `o` on D, z, dt_bias of both forms of the scan.
struct Scan {
    const Tensor &x, &dt, &A, &Bm, &Cm;
    const Tensor *D, *z, *dt_bias;
    int H, G, n, p;
    long long xs, ds, bs, cs, zs = 0;

    Scan(const Common& c, const Args& a, int o, int lead)
        : x(a.tensor(0, "x")), dt(a.tensor(1, "dt")), A(a.tensor(2, "A")), Bm(a.tensor(3, "Bm")), Cm(a.tensor(4, "Cm")),
          D(a.optional(o, "D")), z(a.optional(o + 1, "z")), dt_bias(a.optional(o + 2, "dt_bias")) {
        if (x.dim() != lead + 2) throw refusal<WrongValue>(lead == 2 ? "x must be [B, T, H, p]" : "x must be [N, H, p]");
        if (Bm.dim() != lead + 2)
            throw refusal<WrongValue>("Bm must have one axis of groups and one of state channels after the tokens");
        Shape hd(x.sizes().begin(), x.sizes().begin() + lead + 1);
        Shape gn(x.sizes().begin(), x.sizes().begin() + lead);
        gn.push_back(Bm.size(lead));
        gn.push_back(Bm.size(lead + 1));
        H = size(x.size(lead));
        p = size(x.size(lead + 1));
        G = size(Bm.size(lead));
        n = size(Bm.size(lead + 1));
        xs = c.rows("x", x, x.sizes(), lead);
        ds = c.rows("dt", dt, hd, lead);
        bs = c.rows("Bm", Bm, gn, lead);
        cs = c.rows("Cm", Cm, gn, lead);
        if (z) zs = c.rows("z", *z, x.sizes(), lead);
        c.whole("A", A, at::kFloat, {H});
        if (D) c.whole("D", *D, at::kFloat, {H});
        if (dt_bias) c.whole("dt_bias", *dt_bias, at::kFloat, {H});
    }
};

// x, dt, A, Bm, Cm, S0, D, z, dt_bias, lens, seg_len, y, S_T, return_state, workspace
PyObject* ssm_prefill(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 15)) return nullptr;
    const Args a{args};
    const Common c("ssm_prefill", a.tensor(0, "x"));
    const Scan q(c, a, 6, 2);
    const int64_t B = q.x.size(0), T = q.x.size(1);
    const Tensor *S0 = a.optional(5, "S0"), *lens = a.optional(9, "lens");
    if (S0) c.whole("S0", *S0, at::kFloat, {B, q.H, q.n, q.p});
    if (lens) c.whole("lens", *lens, at::kInt, {B});
    const int b = size(B), t = size(T), seg = a.size(10);
    Pending py(c, a, 11, "y", c.type, q.x.sizes()), ps(c, a, 12, "S_T", at::kFloat, {B, q.H, q.n, q.p}, a.truth(13));
    const Tensor* room = a.optional(14, "workspace");
    const OnDevice on(c.dev);
    const Workspace ws(c, room, lib.ssm_prefill_workspace_bytes(b, t, q.H, q.G, q.n, q.p, c.code, seg));
    const Output &y = py.make(c), &S = ps.make(c);
    if (!c.call(lib.ssm_prefill, ptr(q.x), ptr(q.dt), at_type<float>(&q.A), ptr(q.Bm), ptr(q.Cm), at_type<float>(q.D),
                ptr(q.z), at_type<float>(q.dt_bias), at_type<float>(S0), at_type<int>(lens), y.ptr(),
                reinterpret_cast<float*>(S.ptr()), b, t, q.H, q.G, q.n, q.p, q.xs, q.ds, q.bs, q.cs, q.zs, c.code, seg,
                ws.p, ws.bytes))
        return nullptr;
    return pair(y, S);
    END_HANDLE_TH_ERRORS
}

// x, dt, A, Bm, Cm, S, D, z, dt_bias, y
PyObject* ssm_step(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 10)) return nullptr;
    const Args a{args};
    const Common c("ssm_step", a.tensor(0, "x"));
    const Scan q(c, a, 6, 1);
    const Tensor& S = a.tensor(5, "S");
    const int64_t N = q.x.size(0);
    c.whole("S", S, at::kFloat, {N, q.H, q.n, q.p});
    const int n = size(N);
    Pending py(c, a, 9, "y", c.type, q.x.sizes());
    const OnDevice on(c.dev);
    const Output& y = py.make(c);
    if (!c.call(lib.ssm_step, ptr(q.x), ptr(q.dt), at_type<float>(&q.A), ptr(q.Bm), ptr(q.Cm), at_type<float>(q.D),
                ptr(q.z), at_type<float>(q.dt_bias), at_type<float>(&S), y.ptr(), n, q.H, q.G, q.n, q.p, q.xs, q.ds, q.bs,
                q.cs, q.zs, c.code))
        return nullptr;
    return y.object();
    END_HANDLE_TH_ERRORS
}

// Arguments 0 .. 2 (q, k, v) of both forms of the attention, its caches (from `o` on) and its window.
struct Attention {
    const Tensor &q, &k, &v;
    const Tensor *kc, *vc;
    int H, Hkv, d, window, sinks;
    long long qs, ks, vs;

    Attention(const Common& c, const Args& a, int window_at, int o, int lead)
        : q(a.tensor(0, "q")), k(a.tensor(1, "k")), v(a.tensor(2, "v")), kc(a.optional(o, "k_cache")), vc(a.optional(o + 1, "v_cache")) {
        if (q.dim() != lead + 2) throw refusal<WrongValue>(lead == 2 ? "q must be [B, T, H, d]" : "q must be [N, H, d]");
        if (k.dim() != lead + 2) throw refusal<WrongValue>("k must have one axis of heads and one of channels after the tokens");
        H = size(q.size(lead));
        d = size(q.size(lead + 1));
        Hkv = size(k.size(lead));
        window = a.size(window_at);
        sinks = a.size(window_at + 1);
        Shape kv(q.sizes().begin(), q.sizes().begin() + lead);
        kv.push_back(Hkv);
        kv.push_back(d);
        qs = c.rows("q", q, q.sizes(), lead);
        ks = c.rows("k", k, kv, lead);
        vs = c.rows("v", v, kv, lead);
        if ((kc == nullptr) != (vc == nullptr)) throw refusal<WrongValue>("k_cache and v_cache come together");
        if (kc) {
            const Shape cache{q.size(0), (int64_t)sinks + window, Hkv, d};
            c.whole("k_cache", *kc, c.type, cache);
            c.whole("v_cache", *vc, c.type, cache);
        }
    }
};

// q, k, v, window, sinks, scale, k_cache, v_cache, start, lens, o, workspace
PyObject* window_prefill(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 12)) return nullptr;
    const Args a{args};
    const Common c("window_prefill", a.tensor(0, "q"));
    const Attention q(c, a, 3, 6, 2);
    const int64_t B = q.q.size(0), T = q.q.size(1);
    const Tensor *start = a.optional(8, "start"), *lens = a.optional(9, "lens");
    if (start) c.whole("start", *start, at::kInt, {B});
    if (lens) c.whole("lens", *lens, at::kInt, {B});
    const int b = size(B), t = size(T);
    const float scale = a.scale(5, q.d);
    Pending po(c, a, 10, "o", c.type, q.q.sizes());
    const Tensor* room = a.optional(11, "workspace");
    const OnDevice on(c.dev);
    const Workspace ws(c, room, lib.window_prefill_workspace_bytes(b, t, q.H, q.Hkv, q.d, q.window, q.sinks, c.code, start != nullptr));
    const Output& o = po.make(c);
    if (!c.call(lib.window_prefill, ptr(q.q), ptr(q.k), ptr(q.v), ptr(q.kc), ptr(q.vc), at_type<int>(start),
                at_type<int>(lens), o.ptr(), b, t, q.H, q.Hkv, q.d, q.window, q.sinks, scale, q.qs, q.ks, q.vs, c.code,
                ws.p, ws.bytes))
        return nullptr;
    return o.object();
    END_HANDLE_TH_ERRORS
}

// q, k, v, k_cache, v_cache, pos, window, sinks, scale, o, workspace
PyObject* window_step(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    HANDLE_TH_ERRORS
    if (!arity(nargs, 11)) return nullptr;
    const Args a{args};
    const Common c("window_step", a.tensor(0, "q"));
    a.tensor(3, "k_cache");
    a.tensor(4, "v_cache");
    const Attention q(c, a, 6, 3, 1);
    const Tensor& pos = a.tensor(5, "pos");
    const int64_t N = q.q.size(0);
    c.whole("pos", pos, at::kInt, {N});
    const int n = size(N);
    const float scale = a.scale(8, q.d);
    Pending po(c, a, 9, "o", c.type, q.q.sizes());
    const Tensor* room = a.optional(10, "workspace");
    const OnDevice on(c.dev);
    const Workspace ws(c, room, lib.window_step_workspace_bytes(n, q.H, q.Hkv, q.d, q.window, q.sinks, c.code));
    const Output& o = po.make(c);
    if (!c.call(lib.window_step, ptr(q.q), ptr(q.k), ptr(q.v), ptr(q.kc), ptr(q.vc), at_type<int>(&pos), o.ptr(), n, q.H,
                q.Hkv, q.d, q.window, q.sinks, scale, q.qs, q.ks, q.vs, c.code, ws.p, ws.bytes))
        return nullptr;
    return o.object();
    END_HANDLE_TH_ERRORS
}

// addresses of libkda's entry points, in the order of `Library`, and the function that raises for a status
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    constexpr int kEntries = sizeof(Library) / sizeof(void*);
    if (!arity(nargs, kEntries + 1)) return nullptr;
    void* entry[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        entry[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    memcpy(&lib, entry, sizeof(lib));
    Py_INCREF(args[kEntries]);
    Py_XDECREF(on_status);
    on_status = args[kEntries];
    Py_RETURN_NONE;
}

#define KDA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_METHOD(bind),     KDA_METHOD(conv_prefill),   KDA_METHOD(conv_step),   KDA_METHOD(ssm_prefill),
                         KDA_METHOD(ssm_step), KDA_METHOD(window_prefill), KDA_METHOD(window_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mixers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mixers(void) { return PyModule_Create(&module); }
