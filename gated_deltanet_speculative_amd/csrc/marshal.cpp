// Tensor arguments of the round calls, checked and taken apart natively: the binding spends about a tenth of a
// microsecond on a tensor here, half of one in Python, and a small call has up to fifteen of them.  Nothing of the
// C ABI library is used, and the library uses nothing of this.
//
//   ptr(tensor, name, dtype, shape, device)   its address
//   opt(tensor or None, ...)                  the same, or None
//   view(tensor, name, dtype, shape, device)  a gdn_heads_view of a [C, N, heads, D] tensor as bytes
//   init(refuse)                              before these: refuse(tensor, name, dtype, shape, device) is called with a
//                                             tensor of another type, shape, device or layout, and raises
//
// The calls of gdn_kv4.h and gdn_logits.h are made from here: f is the function's address, shape that of its shape struct,
// the tensors come in the order of the C arguments (None for NULL), the stream is the last one; the result is the
// call's code.  (Through ctypes the arguments of a rotary write cost 5 us, those of a commit of 16 layers 8 us;
// the launch itself costs 4.)
//
//   rope_kv4_write(f, shape, device, q, k, v, inv_freq, cache, slot_ids, page_table, seq_len, positions, pair_axis, parents,
//                  lane_nodes, q_norm, k_norm, eps, interleaved, q_out, status, stream)
//   paged_attention_kv4(f, shape, device, q, cache, slot_ids, page_table, seq_len, parents, lane_nodes, scale, gate, gate_mode,
//                       out, workspace, status, stream)
//   kv4_commit_layers(f, shape, device, caches, slot_ids, page_table, seq_len, parents, lane_nodes, accept_node, new_len, status,
//                     stream)
//   kv4_read_layers(f, shape, device, caches, slot_ids, page_table, first_row, lane_nodes, k_out, v_out, status, stream)
//   adjust_logits(f, shape, device, logits, the nine rules in their order, mask, tokens, parents, lane_nodes, slot_ids, out,
//                 workspace, status, stream)
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "gdn_kv4.h"
#include "gdn_logits.h"

namespace {

PyObject *g_refuse = nullptr;

// The tensor where it has this dtype, shape and device; else nullptr with the error of refuse() set.
const at::Tensor *checked(PyObject *const *a, Py_ssize_t n, bool contiguous) {
    if (!g_refuse || n != 5 || !THPDtype_Check(a[2]) || !PyTuple_Check(a[3])) {
        PyErr_SetString(PyExc_TypeError, "expected (tensor, name, dtype, shape, device), after init(refuse)");
        return nullptr;
    }
    const long device = PyLong_AsLong(a[4]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    if (THPVariable_Check(a[0])) {
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const Py_ssize_t dims = PyTuple_GET_SIZE(a[3]);
        bool same = t.scalar_type() == reinterpret_cast<THPDtype *>(a[2])->scalar_type && t.dim() == dims &&
                    t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided;
        for (Py_ssize_t k = 0; same && k < dims; ++k) {
            const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(a[3], k));
            if (want == -1 && PyErr_Occurred()) return nullptr;
            same = t.size(k) == want;
        }
        if (same && (!contiguous || t.is_contiguous())) return &t;
    }
    PyObject *r = PyObject_CallFunctionObjArgs(g_refuse, a[0], a[1], a[2], a[3], a[4], nullptr);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_ValueError, "unsuitable tensor");
    }
    return nullptr;
}

PyObject *ptr(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS  // (a tensor without storage or with symbolic sizes throws)
    const at::Tensor *t = checked(a, n, true);
    return t ? PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t->data_ptr())) : nullptr;
    END_HANDLE_TH_ERRORS
}

PyObject *opt(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n == 5 && a[0] == Py_None) Py_RETURN_NONE;
    return ptr(self, a, n);
}

// The gdn_heads_view of a tensor [C, N, heads, D]; false with an error set where there is none.
bool view_of(const at::Tensor &t, PyObject *name, gdn_heads_view *v) {
    const int64_t C = t.size(0), N = t.size(1), heads = t.size(2);
    if (t.size(3) > 1 && t.stride(3) != 1) {
        PyErr_Format(PyExc_ValueError, "%U: values of one head must be contiguous", name);
        return false;
    }
    if (N > 1 && C > 1 && t.stride(0) != N * t.stride(1)) {
        PyErr_Format(PyExc_ValueError, "%U: token rows must be evenly strided across lanes", name);
        return false;
    }
    *v = gdn_heads_view{t.data_ptr(), N > 1 ? t.stride(1) : C > 1 ? t.stride(0) : 0, heads > 1 ? t.stride(2) : 0};
    return true;
}

PyObject *view(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor *t = checked(a, n, false);
    if (!t) return nullptr;
    if (t->dim() != 4) {
        PyErr_SetString(PyExc_TypeError, "a view has four dimensions");
        return nullptr;
    }
    gdn_heads_view v;
    if (!view_of(*t, a[1], &v)) return nullptr;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&v), sizeof v);
    END_HANDLE_TH_ERRORS
}

// A dimension of a tensor argument, -1 where it is none
int64_t size_of(PyObject *o, int64_t dims, int64_t k) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.dim() == dims ? t.size(k) : -1;
}

// The arguments of one call, taken in their order.  After the first unsuitable one `bad` is set, with the Python error, and
// every further one is NULL.
class Arguments {
public:
    Arguments(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : a_(a), bad(n != want || !g_refuse) {
        if (bad) PyErr_Format(PyExc_TypeError, "expected %zd arguments, after init(refuse)", want);
        f_ = bad ? nullptr : PyLong_AsVoidPtr(next());
        shape_ = bad ? nullptr : PyLong_AsVoidPtr(next());
        device_ = bad ? -1 : PyLong_AsLong(next());
        fail(PyErr_Occurred() != nullptr);
    }
    template <typename F>
    F *function() const { return reinterpret_cast<F *>(f_); }
    template <typename S>
    const S *shape() const { return static_cast<const S *>(shape_); }

    // A tensor's address.  Required where `optional` is false; a layer axis of `layers` in front of the shape where that is not 0
    void *ptr(const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional = true, int64_t layers = 0) {
        const at::Tensor *t = tensor(name, type, shape, optional, true, layers);
        return t ? t->data_ptr() : nullptr;
    }
    int32_t *i32(const char *name, std::initializer_list<int64_t> shape, bool optional = true) {
        return static_cast<int32_t *>(ptr(name, at::kInt, shape, optional));
    }
    float *f32(const char *name, std::initializer_list<int64_t> shape, bool optional = true) {
        return static_cast<float *>(ptr(name, at::kFloat, shape, optional));
    }
    // A view of a tensor; a null address for None
    gdn_heads_view heads(const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
        gdn_heads_view v{};
        if (const at::Tensor *t = tensor(name, type, shape, optional, false, 0)) {
            PyObject *text = PyUnicode_FromString(name);
            fail(!text || !view_of(*t, text, &v));
            Py_XDECREF(text);
        }
        return v;
    }
    // Rows of a tensor [C, N, V], evenly strided: the address, and the stride
    void *rows(const char *name, at::ScalarType type, int64_t C, int64_t N, int64_t V, int64_t *stride) {
        const at::Tensor *t = tensor(name, type, {C, N, V}, false, false, 0);
        if (!t) return nullptr;
        *stride = N > 1 ? t->stride(1) : C > 1 ? t->stride(0) : V;
        if ((V > 1 && t->stride(2) != 1) || (N > 1 && C > 1 && t->stride(0) != N * *stride)) {
            PyErr_Format(PyExc_ValueError, "%s: the values of a row must be contiguous and the rows evenly strided", name);
            bad = true;
        }
        return bad ? nullptr : t->data_ptr();
    }
    // A contiguous float32 tensor of any shape: address and bytes
    void *workspace(size_t *bytes) {
        PyObject *o = bad ? Py_None : next();
        *bytes = 0;
        if (o == Py_None) return nullptr;
        if (THPVariable_Check(o)) {
            const at::Tensor &t = THPVariable_Unpack(o);
            if (t.scalar_type() == at::kFloat && t.is_cuda() && t.get_device() == device_ && t.layout() == at::kStrided && t.is_contiguous()) {
                *bytes = t.nbytes();
                return t.data_ptr();
            }
        }
        PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous float32 tensor on the call's device");
        bad = true;
        return nullptr;
    }
    double number() {
        const double v = bad ? 0.0 : PyFloat_AsDouble(next());
        fail(!bad && PyErr_Occurred());
        return v;
    }
    long integer() {
        const long v = bad ? 0 : PyLong_AsLong(next());
        fail(!bad && PyErr_Occurred());
        return v;
    }
    hipStream_t stream() {
        hipStream_t s = bad ? nullptr : static_cast<hipStream_t>(PyLong_AsVoidPtr(next()));
        fail(!bad && PyErr_Occurred());
        return s;
    }
    // One layer's 4-bit cache: a tuple of four tensors
    gdn_kv4_cache cache(const gdn_attn_shape &s) { return four(bad ? nullptr : next(), s, 0); }
    // The layers' caches: such a tuple with a leading layer axis, or a sequence of them; their number, 0 where bad
    int caches(const gdn_attn_shape &s, gdn_kv4_cache (&to)[GDN_MAX_LAYERS]) {
        PyObject *o = bad ? nullptr : next();
        if (!o) return 0;
        if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4 && !PyTuple_Check(PyTuple_GET_ITEM(o, 0))) {
            const int64_t size = size_of(PyTuple_GET_ITEM(o, 0), 5, 0), n = size < 0 ? 1 : size;  // (no such tensor: refused below)
            if (!count(n)) return 0;
            const gdn_kv4_cache first = four(o, s, n);
            const size_t rows = (size_t)s.n_pages * s.n_kv_heads * s.page_size, codes = rows * (s.head_dim / 2), scales = rows * (s.head_dim / 32);
            for (int64_t l = 0; l < n && !bad; ++l)
                to[l] = gdn_kv4_cache{static_cast<char *>(first.k_codes) + l * codes, static_cast<char *>(first.k_scales) + l * scales,
                                      static_cast<char *>(first.v_codes) + l * codes, static_cast<char *>(first.v_scales) + l * scales};
            return bad ? 0 : (int)n;
        }
        PyObject *items = PySequence_Fast(o, "the caches must be a Kv4Cache, or a sequence of them");
        if (!items) bad = true;
        if (!items) return 0;
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(items);
        if (count(n))
            for (Py_ssize_t l = 0; l < n && !bad; ++l) to[l] = four(PySequence_Fast_GET_ITEM(items, l), s, 0);
        Py_DECREF(items);
        return bad ? 0 : (int)n;
    }
    // The code of a call that was made, or the error
    PyObject *result(int code) const { return bad ? nullptr : PyLong_FromLong(code); }

private:
    PyObject *const *a_;
    void *f_, *shape_;
    long device_;
    int at_ = 0;

    PyObject *next() { return a_[at_++]; }
    void fail(bool now) { bad = bad || now; }
    bool count(int64_t n) {
        if (n >= 1 && n <= GDN_MAX_LAYERS) return true;
        PyErr_Format(PyExc_ValueError, "%lld layers, expected 1..%d", (long long)n, GDN_MAX_LAYERS);
        bad = true;
        return false;
    }
    const at::Tensor *tensor(const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional, bool contiguous,
                             int64_t layers) {
        if (bad) return nullptr;
        PyObject *o = next();
        if (o == Py_None && optional) return nullptr;
        return suitable(o, name, type, shape, contiguous, layers);
    }
    const at::Tensor *suitable(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, bool contiguous,
                               int64_t layers) {
        if (THPVariable_Check(o)) {
            const at::Tensor &t = THPVariable_Unpack(o);
            const int64_t lead = layers > 0;
            bool same = t.scalar_type() == type && t.dim() == (int64_t)shape.size() + lead && t.is_cuda() && t.get_device() == device_ &&
                        t.layout() == at::kStrided && (!lead || t.size(0) == layers);
            int64_t k = lead;
            for (auto n = shape.begin(); same && n != shape.end(); ++n, ++k) same = t.size(k) == *n;
            if (same && (!contiguous || t.is_contiguous())) return &t;
        }
        bad = true;
        PyObject *want = PyTuple_New((Py_ssize_t)shape.size() + (layers > 0));
        if (!want) return nullptr;
        Py_ssize_t k = 0;
        if (layers > 0) PyTuple_SET_ITEM(want, k++, PyLong_FromLongLong(layers));
        for (int64_t n : shape) PyTuple_SET_ITEM(want, k++, PyLong_FromLongLong(n));
        PyObject *r = PyObject_CallFunction(g_refuse, "OsOOl", o, name, reinterpret_cast<PyObject *>(torch::getTHPDtype(type)), want, device_);
        Py_DECREF(want);
        if (r) {
            Py_DECREF(r);
            PyErr_SetString(PyExc_ValueError, "unsuitable tensor");
        }
        return nullptr;
    }
    gdn_kv4_cache four(PyObject *o, const gdn_attn_shape &s, int64_t layers) {
        gdn_kv4_cache c{};
        if (bad) return c;
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) {
            PyErr_SetString(PyExc_TypeError, "the cache must be a Kv4Cache");
            bad = true;
            return c;
        }
        static const char *const names[4] = {"cache.k", "cache.k_scale", "cache.v", "cache.v_scale"};
        void *p[4] = {};
        for (int j = 0; j < 4 && !bad; ++j) {
            const at::Tensor *t = suitable(PyTuple_GET_ITEM(o, j), names[j], at::kByte,
                                           {s.n_pages, s.n_kv_heads, s.page_size, s.head_dim / (j % 2 ? 32 : 2)}, true, layers);
            p[j] = t ? t->data_ptr() : nullptr;
        }
        return gdn_kv4_cache{p[0], p[1], p[2], p[3]};
    }

public:
    bool bad;
};

at::ScalarType type_of(int32_t dtype) { return dtype == GDN_DTYPE_F32 ? at::kFloat : dtype == GDN_DTYPE_BF16 ? at::kBFloat16 : at::kHalf; }

PyObject *rope_kv4_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Arguments g(a, n, 22);
    if (g.bad) return nullptr;
    const gdn_attn_shape &s = *g.shape<gdn_attn_shape>();
    const int64_t C = s.n_seqs, N = s.n_nodes, Hq = s.n_q_heads, Hkv = s.n_kv_heads, D = s.head_dim;
    const bool wide = THPVariable_Check(a[3]) && THPVariable_Unpack(a[3]).scalar_type() == at::kFloat;
    const int32_t x = wide ? GDN_DTYPE_F32 : s.dtype;
    const int64_t half = size_of(a[6], 1, 0), axes = a[11] == Py_None ? 1 : size_of(a[11], 3, 2);
    if (half < 0 || axes < 0) {
        PyErr_SetString(PyExc_ValueError, half < 0 ? "inv_freq must be a one-dimensional float64 tensor of rot_dim / 2 entries"
                                                   : "positions must be a [C, N, n_axes] int32 tensor");
        return nullptr;
    }
    const gdn_heads_view q = g.heads("q", type_of(x), {C, N, Hq, D}), k = g.heads("k", type_of(x), {C, N, Hkv, D}), v = g.heads("v", type_of(x), {C, N, Hkv, D});
    gdn_rope rope{};
    rope.inv_freq = static_cast<double *>(g.ptr("inv_freq", at::kDouble, {half}, false));
    const gdn_kv4_cache cache = g.cache(s);
    const int32_t *slots = g.i32("slot_ids", {C}, false), *table = g.i32("page_table", {s.n_slots, s.max_pages}, false),
                  *len = g.i32("seq_len", {s.n_slots}, false);
    rope.positions = g.i32("positions", {C, N, axes});
    rope.pair_axis = g.i32("pair_axis", {half});
    const int32_t *parents = g.i32("parents", {C, N}), *nodes = g.i32("lane_nodes", {C});
    rope.q_norm = g.f32("q_norm", {D});
    rope.k_norm = g.f32("k_norm", {D});
    rope.eps = (float)g.number();
    rope.interleaved = (int32_t)g.integer();
    rope.n_axes = (int32_t)axes;
    rope.rot_dim = (int32_t)(2 * half);
    void *out = g.ptr("q_out", type_of(s.dtype), {C, N, Hq, D}, false);
    int32_t *status = g.i32("status", {1}, false);
    hipStream_t stream = g.stream();
    if (g.bad) return nullptr;
    return g.result(g.function<decltype(gdn_rope_kv4_write)>()(&s, x, &q, &k, &v, &rope, &cache, slots, table, len, parents, nodes, out, status, stream));
    END_HANDLE_TH_ERRORS
}

PyObject *paged_attention_kv4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Arguments g(a, n, 17);
    if (g.bad) return nullptr;
    const gdn_attn_shape &s = *g.shape<gdn_attn_shape>();
    const int64_t C = s.n_seqs, N = s.n_nodes, Hq = s.n_q_heads, D = s.head_dim;
    const at::ScalarType type = type_of(s.dtype);
    const void *q = g.ptr("q", type, {C, N, Hq, D}, false);
    const gdn_kv4_cache cache = g.cache(s);
    const int32_t *slots = g.i32("slot_ids", {C}, false), *table = g.i32("page_table", {s.n_slots, s.max_pages}, false),
                  *len = g.i32("seq_len", {s.n_slots}, false), *parents = g.i32("parents", {C, N}), *nodes = g.i32("lane_nodes", {C});
    const float scale = (float)g.number();
    const gdn_heads_view gate = g.heads("gate", type, {C, N, Hq, D}, true);
    const int32_t mode = (int32_t)g.integer();
    void *out = g.ptr("out", type, {C, N, Hq, D}, false);
    size_t bytes;
    void *work = g.workspace(&bytes);
    int32_t *status = g.i32("status", {1}, false);
    hipStream_t stream = g.stream();
    if (g.bad) return nullptr;
    return g.result(g.function<decltype(gdn_paged_attention_kv4)>()(&s, q, &cache, slots, table, len, parents, nodes, scale, gate.p ? &gate : nullptr,
                                                                    mode, out, work, bytes, status, stream));
    END_HANDLE_TH_ERRORS
}

PyObject *kv4_commit_layers(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Arguments g(a, n, 13);
    if (g.bad) return nullptr;
    const gdn_attn_shape &s = *g.shape<gdn_attn_shape>();
    const int64_t C = s.n_seqs, N = s.n_nodes;
    gdn_kv4_cache caches[GDN_MAX_LAYERS];
    const int layers = g.caches(s, caches);
    const int32_t *slots = g.i32("slot_ids", {C}, false), *table = g.i32("page_table", {s.n_slots, s.max_pages}, false),
                  *len = g.i32("seq_len", {s.n_slots}, false), *parents = g.i32("parents", {C, N}), *nodes = g.i32("lane_nodes", {C}),
                  *accept = g.i32("accept_node", {C}, false);
    int32_t *new_len = g.i32("new_len", {s.n_slots}, false), *status = g.i32("status", {1}, false);
    hipStream_t stream = g.stream();
    if (g.bad) return nullptr;
    return g.result(g.function<decltype(gdn_kv4_commit_layers)>()(&s, layers, caches, slots, table, len, parents, nodes, accept, new_len, status, stream));
    END_HANDLE_TH_ERRORS
}

PyObject *kv4_read_layers(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Arguments g(a, n, 12);
    if (g.bad) return nullptr;
    const gdn_attn_shape &s = *g.shape<gdn_attn_shape>();
    const int64_t C = s.n_seqs, N = s.n_nodes;
    gdn_kv4_cache caches[GDN_MAX_LAYERS];
    const int layers = g.caches(s, caches);
    const int32_t *slots = g.i32("slot_ids", {C}, false), *table = g.i32("page_table", {s.n_slots, s.max_pages}, false),
                  *first = g.i32("first_row", {C}, false), *nodes = g.i32("lane_nodes", {C});
    void *k = g.ptr("k_out", type_of(s.dtype), {layers, C, N, s.n_kv_heads, s.head_dim}, false),
         *v = g.ptr("v_out", type_of(s.dtype), {layers, C, N, s.n_kv_heads, s.head_dim}, false);
    int32_t *status = g.i32("status", {1}, false);
    hipStream_t stream = g.stream();
    if (g.bad) return nullptr;
    return g.result(g.function<decltype(gdn_kv4_read_layers)>()(&s, layers, caches, slots, table, first, nodes, k, v, status, stream));
    END_HANDLE_TH_ERRORS
}

PyObject *adjust_logits(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Arguments g(a, n, 22);
    if (g.bad) return nullptr;
    const gdn_logits_shape &s = *g.shape<gdn_logits_shape>();
    const int64_t C = s.n_seqs, N = s.n_nodes, P = s.n_slots, V = s.vocab;
    int64_t stride = 0;
    const void *logits = g.rows("logits", type_of(s.dtype), C, N, V, &stride);
    gdn_logit_rules r{};
    r.history = g.i32("history", {P, s.max_history});
    r.history_len = g.i32("history_len", {P});
    r.prompt_len = g.i32("prompt_len", {P});
    r.repetition = g.f32("repetition", {P});
    r.presence = g.f32("presence", {P});
    r.frequency = g.f32("frequency", {P});
    r.bias_tokens = g.i32("bias_tokens", {P, s.max_bias});
    r.bias = g.f32("bias", {P, s.max_bias});
    r.temperature = g.f32("temperature", {P});
    const int32_t *mask = g.i32("mask", {C, N, (V + 31) / 32}), *tokens = g.i32("tokens", {C, N}), *parents = g.i32("parents", {C, N}),
                  *nodes = g.i32("lane_nodes", {C}), *slots = g.i32("slot_ids", {C}, false);
    void *out = g.ptr("out", type_of(s.out_dtype), {C, N, V}, false);
    size_t bytes;
    void *work = g.workspace(&bytes);
    int32_t *status = g.i32("status", {1}, false);
    hipStream_t stream = g.stream();
    if (g.bad) return nullptr;
    return g.result(g.function<decltype(gdn_adjust_logits)>()(&s, logits, stride, &r, mask, tokens, parents, nodes, slots, out, work, bytes, status, stream));
    END_HANDLE_TH_ERRORS
}

PyObject *init(PyObject *, PyObject *refuse) {
    Py_INCREF(refuse);
    Py_XSETREF(g_refuse, refuse);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_O, "the function that raises for an unsuitable tensor"},
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(ptr)), METH_FASTCALL, "address of a checked tensor"},
    {"opt", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(opt)), METH_FASTCALL, "the same, None for None"},
    {"rope_kv4_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rope_kv4_write)), METH_FASTCALL, "gdn_rope_kv4_write"},
    {"paged_attention_kv4", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(paged_attention_kv4)), METH_FASTCALL,
     "gdn_paged_attention_kv4"},
    {"kv4_commit_layers", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv4_commit_layers)), METH_FASTCALL, "gdn_kv4_commit_layers"},
    {"kv4_read_layers", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(kv4_read_layers)), METH_FASTCALL, "gdn_kv4_read_layers"},
    {"adjust_logits", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(adjust_logits)), METH_FASTCALL, "gdn_adjust_logits"},
    {"view", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(view)), METH_FASTCALL, "a gdn_heads_view as bytes"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "checked tensor arguments of the round calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
