// Argument marshalling of the log-probability calls (logprobs.py): checks of the
// tensors' types, shapes, layouts and device, then the C call of
// include/specverify_logprobs.h.  In C++ for the reason that kvbind.cpp gives.

#include <vector>

#include "bind.h"
#include "specverify_logprobs.h"

namespace {

decltype(&spec_logprobs) g_logprobs;
decltype(&spec_logprobs_grad) g_grad;

// A [..., V] tensor as rows that lie equally far apart.
struct Rows {
    void* p;
    std::vector<int64_t> lead;  // the dimensions before the last
    int64_t rows = 1, V, stride;
    sv_dtype dtype;
    Rows(const at::Tensor& x, const char* name) {
        if (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kFloat)
            type(std::string(name) + " must be bfloat16 or float32, not " +
                 c10::toString(x.scalar_type()));
        dtype = x.scalar_type() == at::kFloat ? SV_F32 : SV_BF16;
        if (x.dim() < 2) value(std::string(name) + " must be [..., V]");
        V = x.size(-1);
        if (V > 1 && x.stride(-1) != 1)
            value(std::string("the last dimension of ") + name + " must be contiguous");
        if (V > INT_MAX) value(std::string(name) + " has too long rows");
        lead.assign(x.sizes().begin(), x.sizes().end() - 1);
        int64_t next = -1;  // what the dimension before must be apart
        stride = V;
        for (int64_t i = x.dim() - 2; i >= 0; --i) {
            const int64_t n = x.size(i);
            rows *= n;
            if (n <= 1) continue;  // (the stride of one entry means nothing)
            if (next < 0) stride = x.stride(i);
            else if (x.stride(i) != next)
                value(std::string("the rows of ") + name + " must lie equally far apart");
            next = x.stride(i) * n;
        }
        if (rows > INT_MAX) value(std::string(name) + " has too many rows");
        p = x.data_ptr();
    }
    std::vector<int64_t> with(int64_t last) const {
        std::vector<int64_t> s(lead);
        s.push_back(last);
        return s;
    }
};

// The tokens asked about: one per row, or a last dimension more.
int64_t given_of(const at::Tensor& t, const Rows& rows) {
    if (t.sizes() == at::IntArrayRef(rows.lead)) return 1;
    if (t.dim() != (int64_t)rows.lead.size() + 1)
        value("tokens have shape " + shape_of(t.sizes()) + ", the rows " + shape_of(rows.lead));
    return t.size(-1);
}
void* floats(PyObject* o, const char* name, at::IntArrayRef shape) {
    return vector(o, name, shape, at::kFloat, at::kFloat);
}
double real(PyObject* o, const char* name) {
    const double x = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        type(std::string(name) + " must be a number");
    }
    return x;
}

// (logits, tokens, logprobs, ws, T, entropy, normalizer, top_tokens, top_logprobs, status, stream)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor& l = tensor(a[0], "logits");
        const Rows r(l, "logits");
        const at::Tensor& t = tensor(a[1], "tokens");
        const int64_t given = given_of(t, r);
        const auto shape = t.dim() == (int64_t)r.lead.size() ? r.lead : r.with(given);
        const void* tok = ints(a[1], "tokens", shape);
        tensor(a[2], "logprobs");
        void* lp = floats(a[2], "logprobs", shape);
        const at::Tensor& w = tensor(a[3], "ws");
        void* ws = vector(a[3], "ws", {w.numel()}, at::kByte, at::kByte);
        const double T = real(a[4], "T");
        void* ent = floats(a[5], "entropy", r.lead);
        void* norm = floats(a[6], "normalizer", r.with(2));
        if ((a[7] == Py_None) != (a[8] == Py_None))
            value("top_tokens and top_logprobs come together");
        int64_t top = 0;
        if (a[7] != Py_None) {
            const at::Tensor& x = tensor(a[7], "top_tokens");
            top = x.dim() ? x.size(-1) : 0;
            if (top > INT_MAX) value("top_tokens has too many places");
        }
        void* tt = ints(a[7], "top_tokens", r.with(top));
        void* tl = floats(a[8], "top_logprobs", r.with(top));
        void* st = vector(a[9], "status", r.lead, at::kInt, at::kUInt32);
        if (given > INT_MAX) value("too many tokens per row");
        Devices d;
        d.add(l, "logits");
        static const char* const names[] = {"tokens", "logprobs", "ws"};
        for (int i = 0; i < 3; ++i) add(d, a[i + 1], names[i]);
        static const char* const more[] = {"entropy", "normalizer", "top_tokens", "top_logprobs",
                                           "status"};
        for (int i = 0; i < 5; ++i) add(d, a[i + 5], more[i]);
        d.check();
        return g_logprobs(r.p, r.dtype, r.stride, (const int32_t*)tok, (float)T, (int)r.rows,
                          (int)r.V, (int)given, (int)top, (float*)lp, (float*)norm, (float*)ent,
                          (int32_t*)tt, (float*)tl, ws, (size_t)w.numel(), (uint32_t*)st,
                          stream_of(a[10]));
    });
}

// (logits, tokens, normalizer, grad_logprobs, grad_logits, T, entropy, grad_entropy, status,
//  stream)
PyObject* grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor& l = tensor(a[0], "logits");
        const Rows r(l, "logits");
        const at::Tensor& t = tensor(a[1], "tokens");
        const int64_t given = given_of(t, r);
        const auto shape = t.dim() == (int64_t)r.lead.size() ? r.lead : r.with(given);
        const void* tok = ints(a[1], "tokens", shape);
        tensor(a[2], "normalizer");
        const void* norm = floats(a[2], "normalizer", r.with(2));
        tensor(a[3], "grad_logprobs");
        const void* g = floats(a[3], "grad_logprobs", shape);
        const at::Tensor& out = tensor(a[4], "grad_logits");
        if (out.scalar_type() != l.scalar_type())
            type(std::string("grad_logits must be ") + c10::toString(l.scalar_type()) + ", not " +
                 c10::toString(out.scalar_type()));
        if (out.sizes() != l.sizes())
            value("grad_logits has shape " + shape_of(out.sizes()) + ", not " +
                  shape_of(l.sizes()));
        const Rows o(out, "grad_logits");
        const double T = real(a[5], "T");
        const void* ent = floats(a[6], "entropy", r.lead);
        const void* ge = floats(a[7], "grad_entropy", r.lead);
        if (ge && !ent) value("grad_entropy needs entropy");
        void* st = vector(a[8], "status", r.lead, at::kInt, at::kUInt32);
        if (given > INT_MAX) value("too many tokens per row");
        Devices d;
        d.add(l, "logits");
        static const char* const names[] = {"tokens", "normalizer", "grad_logprobs", "grad_logits"};
        for (int i = 0; i < 4; ++i) add(d, a[i + 1], names[i]);
        static const char* const more[] = {"entropy", "grad_entropy", "status"};
        for (int i = 0; i < 3; ++i) add(d, a[i + 6], more[i]);
        d.check();
        return g_grad(r.p, r.dtype, r.stride, (const int32_t*)tok, (const float*)norm,
                      (const float*)ent, (const float*)g, (const float*)ge, (float)T, (int)r.rows,
                      (int)r.V, (int)given, o.p, o.stride, (uint32_t*)st, stream_of(a[9]));
    });
}

// The library's entry points, as logprobs.py has loaded them.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "two entry points");
        return nullptr;
    }
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(PyLong_AsVoidPtr(a[0]));
    g_grad = reinterpret_cast<decltype(g_grad)>(PyLong_AsVoidPtr(a[1]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"logprobs", reinterpret_cast<PyCFunction>(logprobs), METH_FASTCALL, nullptr},
    {"grad", reinterpret_cast<PyCFunction>(grad), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_lpbind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lpbind() { return PyModule_Create(&g_module); }
