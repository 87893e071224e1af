// Python calls of the token-sequence operators.  The functions here read and check the tensors,
// make the device and the stream current, allocate what the call returns and enter the C
// library.  A decoding step is a row of such calls, each of a few microseconds on the device: read
// attribute by attribute in Python, a call's tensors alone took 14 to 20 us of the host, here 2 to 4.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <limits.h>
#include <stdarg.h>

#include <optional>

#include "vdm.h"

namespace {

PyObject* g_check = nullptr;   // raises the package's error of a status

[[noreturn]] void refuse(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(PyExc_ValueError, fmt, ap);
    va_end(ap);
    throw python_error();
}

struct Ref {   // an owned reference
    PyObject* p;
    explicit Ref(PyObject* o) : p(o) {
        if (!p) throw python_error();
    }
    Ref(const Ref&) = delete;
    ~Ref() { Py_DECREF(p); }
};

std::string text(c10::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor (got %s)", name, Py_TYPE(o)->tp_name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) refuse("%s must be a dense tensor", name);
    return t;
}

// nothing here has a backward pass: a call that would have to be differentiated is refused
void no_grad(const char* name, const at::Tensor& t) {
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse("%s requires a gradient, which this call does not compute: detach it, or call under torch.no_grad()", name);
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
        refuse("%s carries a forward-mode tangent, which this call does not propagate: unpack it first", name);
}

// written in place: a graph that has kept the tensor notices (inference tensors have no version)
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

const at::Tensor& cuda_tensor(const char* name, PyObject* o) {
    const at::Tensor& t = tensor(name, o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor (got one on %s)", name, t.device().str().c_str());
    return t;
}

vdm_dtype seq_dtype(const char* name, const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return VDM_BF16;
    if (t.scalar_type() == at::kFloat) return VDM_F32;
    refuse("%s must be bfloat16 or float32 (got %s)", name, c10::toString(t.scalar_type()));
}

// a [tokens, heads, D] tensor against the call's sizes (-1: any)
vdm_heads heads(const char* name, const at::Tensor& t, const at::Tensor& like, int64_t T, int64_t H, int64_t D) {
    if (t.dim() != 3 || (T >= 0 && t.size(0) != T) || (H >= 0 && t.size(1) != H) || (D >= 0 && t.size(2) != D)) {
        auto w = [](int64_t x) { return x < 0 ? std::string("*") : std::to_string(x); };
        refuse("%s must have shape [%s, %s, %s] (got %s)", name, w(T).c_str(), w(H).c_str(), w(D).c_str(), text(t.sizes()).c_str());
    }
    if (t.scalar_type() != like.scalar_type())
        refuse("%s must be %s (got %s)", name, c10::toString(like.scalar_type()), c10::toString(t.scalar_type()));
    if (t.device() != like.device())
        refuse("%s is on %s, the call's other tensors on %s", name, t.device().str().c_str(), like.device().str().c_str());
    no_grad(name, t);
    if (t.size(1) > INT_MAX || t.size(2) > INT_MAX) refuse("%s: sizes %s do not fit", name, text(t.sizes()).c_str());
    if (t.numel() && t.size(2) > 1 && t.stride(2) != 1)
        refuse("%s: the elements of a head must be contiguous (stride %lld)", name, (long long)t.stride(2));
    return vdm_heads{t.data_ptr(), t.stride(0), t.stride(1)};
}

// a contiguous int32 tensor of the given shape on the call's device
const int32_t* index(const char* name, const at::Tensor& t, c10::Device dev, c10::IntArrayRef shape) {
    if (t.scalar_type() != at::kInt || t.device() != dev || t.sizes() != shape || !t.is_contiguous())
        refuse("%s must be a contiguous int32 tensor of shape %s on %s (got %s, %s, %s)", name, text(shape).c_str(), dev.str().c_str(),
               c10::toString(t.scalar_type()), text(t.sizes()).c_str(), t.device().str().c_str());
    return static_cast<const int32_t*>(t.data_ptr());
}

int32_t sequences(const char* name, const at::Tensor& cu) {
    if (cu.dim() != 1 || cu.size(0) < 1 || cu.size(0) > INT_MAX)
        refuse("%s must hold B + 1 offsets (got shape %s)", name, text(cu.sizes()).c_str());
    return (int32_t)(cu.size(0) - 1);
}

const float* gain(const char* name, PyObject* o, int64_t D, c10::Device dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& g = tensor(name, o);
    if (g.scalar_type() != at::kFloat || g.dim() != 1 || g.size(0) != D || g.device() != dev || !g.is_contiguous())
        refuse("%s must be a contiguous float32 tensor of shape [%lld] on %s", name, (long long)D, dev.str().c_str());
    no_grad(name, g);
    return static_cast<const float*>(g.data_ptr());
}

int64_t attr_int(PyObject* o, const char* name) {
    Ref r(PyObject_GetAttrString(o, name));
    const int64_t v = PyLong_AsLongLong(r.p);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}

// The device of a call's tensors made current, and its stream: the given one or that device's
// current one.  What the call allocates belongs to that stream.
struct On {
    std::optional<c10::cuda::CUDAGuard> device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    vdm_stream stream;
    On(c10::Device dev, PyObject* s) {
        if (s == Py_None) {
            device.emplace(dev);
            stream = (vdm_stream)c10::cuda::getCurrentCUDAStream(dev.index()).stream();
            return;
        }
        const int64_t index = attr_int(s, "device_index");
        if (index != dev.index()) refuse("the stream is of cuda:%lld, the tensors of %s", (long long)index, dev.str().c_str());
        const auto st = c10::cuda::CUDAStream::unpack3(attr_int(s, "stream_id"), (c10::DeviceIndex)index,
                                                       static_cast<c10::DeviceType>(attr_int(s, "device_type")));
        guard.emplace(st);
        stream = (vdm_stream)st.stream();
    }
};

// Without the interpreter's lock, as the ctypes calls: a launch waits while the device's queue is full, an allocation for the
// device.  f touches no Python object.
template <typename F> auto unlocked(F f) {
    struct Gate {
        PyThreadState* s = PyEval_SaveThread();
        ~Gate() { PyEval_RestoreThread(s); }
    } gate;
    return f();
}
at::Tensor empty(c10::IntArrayRef sizes, const at::TensorOptions& o) {
    return unlocked([&] { return at::empty(sizes, o); });
}

void check(vdm_status s) {
    if (s == VDM_OK) return;
    Ref r(PyObject_CallFunction(g_check, "i", (int)s));
    refuse("status %d", (int)s);   // the call above raises
}

struct Cache {
    vdm_kv_cache c;
    const at::Tensor* k;
    at::Tensor hold[4];
};

void read_cache(PyObject* o, Cache& out) {
    auto get = [&](const char* n, at::Tensor& hold) {
        Ref r(PyObject_GetAttrString(o, n));
        if (r.p == Py_None) return false;
        hold = tensor(n, r.p);
        no_grad(n, hold);
        return true;
    };
    at::Tensor &k = out.hold[0], &v = out.hold[1];
    if (!get("k", k) || !get("v", v) || k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() ||
        k.device() != v.device() || !k.is_contiguous() || !v.is_contiguous())
        refuse("cache: k and v must be contiguous tensors [num_pages, H, page_size, D] of one dtype and device");
    vdm_kv_cache& c = out.c;
    switch (k.scalar_type()) {
        case at::kFloat: c.dtype = VDM_CACHE_F32; break;
        case at::kBFloat16: c.dtype = VDM_CACHE_BF16; break;
        case at::kByte:
        case at::kFloat8_e4m3fn: c.dtype = VDM_CACHE_E4M3; break;
        default: refuse("cache: dtype %s not float32, bfloat16, uint8 or float8_e4m3fn", c10::toString(k.scalar_type()));
    }
    for (int i = 0; i < 4; ++i)
        if (k.size(i) > INT_MAX) refuse("cache: sizes %s do not fit", text(k.sizes()).c_str());
    c.num_pages = (int32_t)k.size(0), c.H = (int32_t)k.size(1), c.page_size = (int32_t)k.size(2), c.D = (int32_t)k.size(3);
    c.k = k.data_ptr(), c.v = v.data_ptr();
    c.k_scale = c.v_scale = nullptr;
    if (c.dtype == VDM_CACHE_E4M3) {
        const char* names[2] = {"k_scale", "v_scale"};
        for (int i = 0; i < 2; ++i) {
            at::Tensor& s = out.hold[2 + i];
            if (!get(names[i], s) || s.scalar_type() != at::kByte || s.sizes() != k.sizes().slice(0, 3) || s.device() != k.device() ||
                !s.is_contiguous())
                refuse("cache: an 8-bit cache needs contiguous uint8 scales [num_pages, H, page_size]");
            (i ? c.v_scale : c.k_scale) = static_cast<uint8_t*>(s.data_ptr());
        }
    }
    out.k = &k;
}

struct Tables {
    int32_t B, max_pages;
    const int32_t *cu, *len, *table;
};

Tables read_tables(const Cache& c, PyObject* cu_o, PyObject* len_o, PyObject* table_o, c10::Device dev) {
    const at::Tensor &cu = tensor("cu", cu_o), &len = tensor("kv_len", len_o), &table = tensor("table", table_o);
    Tables t;
    t.B = sequences("cu", cu);
    if (c.k->device() != dev)
        refuse("the cache is on %s, the call's other tensors on %s", c.k->device().str().c_str(), dev.str().c_str());
    if (table.dim() != 2 || table.size(1) > INT_MAX) refuse("table must be [B, max_pages] (got %s)", text(table.sizes()).c_str());
    t.max_pages = (int32_t)table.size(1);
    t.cu = index("cu", cu, dev, {t.B + 1});
    t.len = index("kv_len", len, dev, {t.B});
    t.table = index("table", table, dev, {t.B, t.max_pages});
    return t;
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
        throw python_error();
    }
}

// (q, k, positions, rope, q_gain, k_gain, eps, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 10);
    const at::Tensor& q = cuda_tensor("q", a[0]);
    const vdm_dtype dt = seq_dtype("q", q);
    const vdm_heads hq = heads("q", q, q, -1, -1, -1);
    const c10::Device dev = q.device();
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    int64_t Hk = 0;
    vdm_heads hk{}, hko{};
    const bool with_k = a[1] != Py_None;
    if (with_k) {
        const at::Tensor& k = tensor("k", a[1]);
        hk = heads("k", k, q, T, -1, D);
        Hk = k.size(1);
    }
    const float *gq = gain("q_gain", a[4], D, dev), *gk = gain("k_gain", a[5], D, dev);
    vdm_rope rope{};
    const int32_t* pos = nullptr;
    at::Tensor f;
    if (a[3] != Py_None) {
        Ref fr(PyObject_GetAttrString(a[3], "inv_freq")), in(PyObject_GetAttrString(a[3], "interleaved")),
            ms(PyObject_GetAttrString(a[3], "mscale"));
        f = tensor("rope.inv_freq", fr.p);
        if (f.scalar_type() != at::kDouble || f.dim() != 1 || f.device() != dev || !f.is_contiguous() || f.size(0) > INT_MAX / 2)
            refuse("rope.inv_freq must be a contiguous float64 tensor [rot_dim/2] on %s", dev.str().c_str());
        no_grad("rope.inv_freq", f);
        if (a[2] == Py_None) refuse("a rotation needs positions");
        rope.rot_dim = (int32_t)(2 * f.size(0));
        rope.interleaved = truth(in.p);
        rope.inv_freq = static_cast<const double*>(f.data_ptr());
        rope.mscale = (float)number(ms.p);
        pos = index("positions", tensor("positions", a[2]), dev, {T});
    }
    const float eps = (float)number(a[6]);
    On on(dev, a[9]);
    at::Tensor qo = a[7] == Py_None ? empty({T, Hq, D}, q.options()) : tensor("q_out", a[7]), ko;
    const vdm_heads hqo = heads("q_out", qo, q, T, Hq, D);
    if (with_k) {
        ko = a[8] == Py_None ? empty({T, Hk, D}, q.options()) : tensor("k_out", a[8]);
        hko = heads("k_out", ko, q, T, Hk, D);
    }
    check(unlocked([&] { return vdm_qk_norm_rope(dt, T, (int32_t)Hq, (int32_t)Hk, (int32_t)D, &hq, with_k ? &hk : nullptr, gq, gk, eps,
                           a[3] == Py_None ? nullptr : &rope, pos, &hqo, with_k ? &hko : nullptr, on.stream); }));
    if (a[7] != Py_None) written(qo);
    if (with_k && a[8] != Py_None) written(ko);
    Ref r0(a[7] == Py_None ? THPVariable_Wrap(qo) : Py_NewRef(a[7]));
    Ref r1(!with_k ? Py_NewRef(Py_None) : a[8] == Py_None ? THPVariable_Wrap(ko) : Py_NewRef(a[8]));
    return PyTuple_Pack(2, r0.p, r1.p);
    END_HANDLE_TH_ERRORS
}

// (cache, k, v, cu, kv_len, table, stream)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 7);
    const at::Tensor &k = cuda_tensor("k", a[1]), &v = tensor("v", a[2]);
    const vdm_dtype dt = seq_dtype("k", k);
    Cache c;
    read_cache(a[0], c);
    const int64_t T = k.dim() ? k.size(0) : 0;
    const Tables t = read_tables(c, a[3], a[4], a[5], k.device());
    const vdm_heads hk = heads("k", k, k, T, c.c.H, c.c.D), hv = heads("v", v, k, T, c.c.H, c.c.D);
    On on(k.device(), a[6]);
    check(unlocked([&] { return vdm_cache_write(&c.c, dt, &hk, &hv, T, t.cu, t.len, t.table, t.max_pages, t.B, on.stream); }));
    for (const at::Tensor& x : c.hold)
        if (x.defined()) written(x);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (cache, kv_len, table, cu, k, v, stream): the cache's tokens into k and v
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 7);
    Cache c;
    read_cache(a[0], c);
    if (!c.k->is_cuda()) refuse("cache.k must be a CUDA tensor (got one on %s)", c.k->device().str().c_str());
    const Tables t = read_tables(c, a[3], a[1], a[2], c.k->device());
    const at::Tensor &k = cuda_tensor("k", a[4]), &v = tensor("v", a[5]);
    const vdm_dtype dt = seq_dtype("out", k);
    const int64_t T = k.dim() ? k.size(0) : 0;
    const vdm_heads hk = heads("k", k, k, T, c.c.H, c.c.D), hv = heads("v", v, k, T, c.c.H, c.c.D);
    if (k.device() != c.k->device()) refuse("out is on %s, the cache on %s", k.device().str().c_str(), c.k->device().str().c_str());
    On on(k.device(), a[6]);
    check(unlocked([&] { return vdm_cache_read(&c.c, dt, t.len, t.table, t.max_pages, t.cu, t.B, T, &hk, &hv, on.stream); }));
    written(k), written(v);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// what both attention calls share: parameters, output, workspace, result
struct Attention {
    vdm_attention p;
    at::Tensor out, lse, ws;
    vdm_heads ho;
    size_t ws_bytes = 0;
    PyObject* given;

    // a: causal, scale, out, want_lse, workspace
    Attention(const at::Tensor& q, int64_t Hk, PyObject* const* a) : given(a[2]) {
        p.Hq = (int32_t)q.size(1), p.Hk = (int32_t)Hk, p.D = (int32_t)q.size(2);
        p.dtype = seq_dtype("q", q);
        p.causal = truth(a[0]);
        p.scale = (float)(a[1] == Py_None ? 1.0 / std::sqrt((double)q.size(2)) : number(a[1]));
    }
    void allocate(const at::Tensor& q, int32_t B, int64_t max_kv, PyObject* const* a) {
        const int64_t T = q.size(0);
        out = given == Py_None ? empty({T, q.size(1), q.size(2)}, q.options()) : tensor("out", given);
        ho = heads("out", out, q, T, q.size(1), q.size(2));
        if (truth(a[3])) lse = empty({T, q.size(1)}, q.options().dtype(at::kFloat));
        if (a[4] == Py_None) {
            check(vdm_attention_workspace_size(&p, B, T, max_kv, &ws_bytes));
            if (ws_bytes) ws = empty({(int64_t)ws_bytes}, q.options().dtype(at::kByte));
        } else {
            ws = tensor("workspace", a[4]);
            if (ws.device() != q.device() || !ws.is_contiguous())
                refuse("workspace must be a contiguous tensor on %s", q.device().str().c_str());
            ws_bytes = ws.nbytes();
        }
    }
    float* lse_ptr() const { return lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr; }
    void* ws_ptr() const { return ws.defined() ? ws.data_ptr() : nullptr; }
    PyObject* result() const {
        if (given != Py_None) written(out);
        Ref o(given == Py_None ? THPVariable_Wrap(out) : Py_NewRef(given));
        if (!lse.defined()) return Py_NewRef(o.p);
        Ref l(THPVariable_Wrap(lse));
        return PyTuple_Pack(2, o.p, l.p);
    }
};

// (q, k, v, cu_q, cu_k, causal, scale, out, want_lse, workspace, stream)
PyObject* attention_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 11);
    const at::Tensor &q = cuda_tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    seq_dtype("q", q);
    const vdm_heads hq = heads("q", q, q, -1, -1, -1);
    const int64_t D = q.size(2);
    const vdm_heads hk = heads("k", k, q, -1, -1, D);
    const int64_t Tk = k.size(0), Hk = k.size(1);
    const vdm_heads hv = heads("v", v, q, Tk, Hk, D);
    Attention at(q, Hk, a + 5);
    const at::Tensor& cq = tensor("cu_q", a[3]);
    const int32_t B = sequences("cu_q", cq);
    const int32_t* pq = index("cu_q", cq, q.device(), {B + 1});
    if (a[4] == Py_None && Tk != q.size(0)) refuse("queries and keys of different lengths need cu_k");
    const int32_t* pk = a[4] == Py_None ? pq : index("cu_k", tensor("cu_k", a[4]), q.device(), {B + 1});
    On on(q.device(), a[10]);
    at.allocate(q, B, Tk, a + 5);
    check(unlocked([&] { return vdm_attention_packed(&at.p, &hq, &hk, &hv, pq, pk, B, q.size(0), Tk, &at.ho, at.lse_ptr(), at.ws_ptr(), at.ws_bytes, on.stream); }));
    return at.result();
    END_HANDLE_TH_ERRORS
}

// (q, cache, cu_q, kv_len, table, causal, scale, out, want_lse, workspace, stream)
PyObject* attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 11);
    const at::Tensor& q = cuda_tensor("q", a[0]);
    seq_dtype("q", q);
    const vdm_heads hq = heads("q", q, q, -1, -1, -1);
    Cache c;
    read_cache(a[1], c);
    Attention at(q, c.c.H, a + 5);
    const Tables t = read_tables(c, a[2], a[3], a[4], q.device());
    On on(q.device(), a[10]);
    at.allocate(q, t.B, (int64_t)t.max_pages * c.c.page_size, a + 5);
    check(unlocked([&] { return vdm_attention_paged(&at.p, &hq, &c.c, t.cu, t.len, t.table, t.max_pages, t.B, q.size(0), &at.ho, at.lse_ptr(), at.ws_ptr(),
                              at.ws_bytes, on.stream); }));
    return at.result();
    END_HANDLE_TH_ERRORS
}

// the package's function that raises its error of a status
PyObject* set_check(PyObject*, PyObject* f) {
    Py_XDECREF(g_check);
    g_check = Py_NewRef(f);
    Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"set_check", set_check, METH_O, nullptr},
                         {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"cache_write", fast(cache_write), METH_FASTCALL, nullptr},
                         {"cache_read", fast(cache_read), METH_FASTCALL, nullptr},
                         {"attention_packed", fast(attention_packed), METH_FASTCALL, nullptr},
                         {"attention_paged", fast(attention_paged), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seq", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seq() { return PyModule_Create(&module); }
