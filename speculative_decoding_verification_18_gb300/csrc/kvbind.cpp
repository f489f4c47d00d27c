// Argument marshalling of the paged cache calls (kvcache.py): checks of the
// tensors' types, shapes, layouts and device, then the C call of
// include/specverify_kv.h.  In C++ because a call is made per layer and step: the
// same checks in Python and ctypes cost more than the smallest calls take on the
// GPU (one token's append, launch included: 16.5 us there, 4.1 us here).

#include "bind.h"
#include "specverify_kv.h"

namespace {

decltype(&spec_kv_append) g_append;
decltype(&spec_kv_attention) g_attention;
decltype(&spec_kv_attention_window) g_window;
decltype(&spec_kv_commit) g_commit;

// A [B, N, heads, dim] tensor whose dim is contiguous.
void* tokens(const at::Tensor& x, const char* name, int64_t B, int64_t N, int64_t heads,
             int64_t dim, at::ScalarType t, sv_strides* s) {
    if (x.scalar_type() != t)
        type(std::string(name) + " must be " + c10::toString(t) + ", not " +
             c10::toString(x.scalar_type()));
    if (x.sizes() != at::IntArrayRef({B, N, heads, dim}))
        value(std::string(name) + " has shape " + shape_of(x.sizes()) + ", not " +
              shape_of(at::IntArrayRef({B, N, heads, dim})));
    if (dim > 1 && x.stride(3) != 1)
        value(std::string("the last dimension of ") + name + " must be contiguous");
    // the stride of a dimension of one entry means nothing: the contiguous one
    s->head = heads > 1 ? x.stride(2) : dim;
    s->token = N > 1 ? x.stride(1) : heads * s->head;
    s->batch = B > 1 ? x.stride(0) : N * s->token;
    return x.data_ptr();
}

sv_dtype value_type(const at::Tensor& x, const char* name) {
    if (x.scalar_type() == at::kBFloat16) return SV_BF16;
    if (x.scalar_type() == at::kHalf) return SV_F16;
    type(std::string(name) + " must be bfloat16 or float16, not " + c10::toString(x.scalar_type()));
}

const sv_kv_cache* cache_of(PyObject* o) {
    return static_cast<const sv_kv_cache*>(PyLong_AsVoidPtr(o));
}
void sequences(int64_t B, PyObject* rows) {
    const long n = PyLong_AsLong(rows);
    if (n != B)
        value("the table has " + std::to_string(n) + " sequences, not " + std::to_string(B));
}

// (cache, rows of the table, device, k, v, kv_len, q, q_out, rope, parents, num_new, status,
//  stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const sv_kv_cache* c = cache_of(a[0]);
        const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
        if (k.dim() != 4) value("k must be [B, N, heads, dim]");
        const int64_t B = k.size(0), N = k.size(1), H = k.size(2), D = k.size(3);
        if (H != c->heads || D != c->dim)
            value("k has " + std::to_string(H) + " heads of " + std::to_string(D) + ", the cache " +
                  std::to_string(c->heads) + " of " + std::to_string(c->dim));
        sequences(B, a[1]);
        const sv_dtype t = value_type(k, "k");
        sv_strides ks, vs, qs = {};
        void* kp = tokens(k, "k", B, N, H, D, k.scalar_type(), &ks);
        void* vp = tokens(v, "v", B, N, H, D, k.scalar_type(), &vs);
        if (ks.batch != vs.batch || ks.token != vs.token || ks.head != vs.head)
            value("k and v must have the same strides");
        void *qp = nullptr, *op = nullptr;
        int64_t hq = H;
        if (a[6] != Py_None) {
            const at::Tensor& q = tensor(a[6], "q");
            hq = q.dim() == 4 ? q.size(2) : 0;
            qp = tokens(q, "q", B, N, hq, D, k.scalar_type(), &qs);
            if (a[7] == Py_None) value("q needs q_out");
            op = vector(a[7], "q_out", {B, N, hq, D}, k.scalar_type(), k.scalar_type());
        }
        const void* lens = ints(tensor(a[5], "kv_len").defined() ? a[5] : Py_None, "kv_len", {B});
        const void* par = ints(a[9], "parents", {B, N});
        const void* num = ints(a[10], "num_new", {B});
        void* st = vector(a[11], "status", {B}, at::kInt, at::kUInt32);
        Devices d;
        d.add(k, "k");
        d.add(v, "v");
        add(d, a[5], "kv_len");
        if (qp) add(d, a[6], "q"), add(d, a[7], "q_out");
        add(d, a[9], "parents");
        add(d, a[10], "num_new");
        add(d, a[11], "status");
        d.check((int)PyLong_AsLong(a[2]));
        const sv_rope* rope = a[8] == Py_None ? nullptr
                                              : static_cast<const sv_rope*>(PyLong_AsVoidPtr(a[8]));
        return g_append(c, rope, qp, qp ? &qs : nullptr, kp, vp, &ks, t, (const int32_t*)lens,
                        (const int32_t*)num, (const int32_t*)par, (int)B, (int)N, (int)hq, op,
                        (uint32_t*)st, stream_of(a[12]));
    });
}

// (cache, rows of the table, device, q, kv_len, out, ws, scale, parents, num_new, status, stream),
// and with a window: its length and the number of first slots
PyObject* attend(PyObject* const* a, Py_ssize_t n, bool windowed) {
    return guarded(n, windowed ? 14 : 12, [&] {
        const sv_kv_cache* c = cache_of(a[0]);
        const at::Tensor& q = tensor(a[3], "q");
        if (q.dim() != 4) value("q must be [B, N, q_heads, dim]");
        const int64_t B = q.size(0), N = q.size(1), hq = q.size(2), D = q.size(3);
        if (D != c->dim)
            value("q has heads of " + std::to_string(D) + ", the cache of " +
                  std::to_string(c->dim));
        sequences(B, a[1]);
        const sv_dtype t = value_type(q, "q");
        sv_strides qs;
        void* qp = tokens(q, "q", B, N, hq, D, q.scalar_type(), &qs);
        const void* lens = ints(tensor(a[4], "kv_len").defined() ? a[4] : Py_None, "kv_len", {B});
        tensor(a[5], "out");
        void* out = vector(a[5], "out", {B, N, hq, D}, q.scalar_type(), q.scalar_type());
        const at::Tensor& w = tensor(a[6], "ws");
        void* ws = vector(a[6], "ws", {w.numel()}, at::kByte, at::kByte);
        const double scale = PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred()) return SV_OK;
        const int window = windowed ? number(a[12], "window") : 0;
        const int sinks = windowed ? number(a[13], "sinks") : 0;
        const void* par = ints(a[8], "parents", {B, N});
        const void* num = ints(a[9], "num_new", {B});
        void* st = vector(a[10], "status", {B}, at::kInt, at::kUInt32);
        Devices d;
        d.add(q, "q");
        add(d, a[4], "kv_len");
        add(d, a[5], "out");
        add(d, a[6], "ws");
        add(d, a[8], "parents");
        add(d, a[9], "num_new");
        add(d, a[10], "status");
        d.check((int)PyLong_AsLong(a[2]));
        if (windowed)
            return g_window(c, qp, &qs, t, (const int32_t*)lens, (const int32_t*)num,
                            (const int32_t*)par, (float)scale, window, sinks, (int)B, (int)N,
                            (int)hq, out, ws, (size_t)w.numel(), (uint32_t*)st,
                            stream_of(a[11]));
        return g_attention(c, qp, &qs, t, (const int32_t*)lens, (const int32_t*)num,
                           (const int32_t*)par, (float)scale, (int)B, (int)N, (int)hq, out, ws,
                           (size_t)w.numel(), (uint32_t*)st, stream_of(a[11]));
    });
}
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) { return attend(a, n, false); }
PyObject* attention_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return attend(a, n, true);
}

// (cache, rows of the table, device, layers, layer stride, kv_len, num_accepted, kv_len_out,
//  out_nodes, status, stream)
PyObject* commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const sv_kv_cache* c = cache_of(a[0]);
        const at::Tensor& len = tensor(a[5], "kv_len");
        if (len.dim() != 1) value("kv_len must be [B]");
        const int64_t B = len.size(0);
        sequences(B, a[1]);
        int64_t N = 65;
        if (a[8] != Py_None) {
            const at::Tensor& nodes = tensor(a[8], "out_nodes");
            N = nodes.dim() == 2 ? nodes.size(1) : 0;
        }
        const void* lens = ints(a[5], "kv_len", {B});
        const void* nodes = ints(a[8], "out_nodes", {B, N});
        tensor(a[6], "num_accepted");
        const void* acc = ints(a[6], "num_accepted", {B});
        tensor(a[7], "kv_len_out");
        void* out = ints(a[7], "kv_len_out", {B});
        void* st = vector(a[9], "status", {B}, at::kInt, at::kUInt32);
        Devices d;
        add(d, a[5], "kv_len");
        add(d, a[6], "num_accepted");
        add(d, a[7], "kv_len_out");
        add(d, a[8], "out_nodes");
        add(d, a[9], "status");
        d.check((int)PyLong_AsLong(a[2]));
        return g_commit(c, (int)PyLong_AsLong(a[3]), PyLong_AsLongLong(a[4]), (const int32_t*)lens,
                        (const int32_t*)nodes, (const int32_t*)acc, (int)B, (int)N, (int32_t*)out,
                        (uint32_t*)st, stream_of(a[10]));
    });
}

// The library's entry points, as kvcache.py has loaded them.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "four entry points");
        return nullptr;
    }
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_attention = reinterpret_cast<decltype(g_attention)>(PyLong_AsVoidPtr(a[1]));
    g_commit = reinterpret_cast<decltype(g_commit)>(PyLong_AsVoidPtr(a[2]));
    g_window = reinterpret_cast<decltype(g_window)>(PyLong_AsVoidPtr(a[3]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(append), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(attention), METH_FASTCALL, nullptr},
    {"attention_window", reinterpret_cast<PyCFunction>(attention_window), METH_FASTCALL, nullptr},
    {"commit", reinterpret_cast<PyCFunction>(commit), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kvbind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvbind() { return PyModule_Create(&g_module); }
