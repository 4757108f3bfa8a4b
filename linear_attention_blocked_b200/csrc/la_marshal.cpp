// la_marshal.cpp -- the short way from torch tensors to the C ABI's softmax
// entry points.  A decode step of one request takes 7 us on the GPU; checking
// and marshalling its tensors in Python takes 11 us next to 5 for the call
// itself.  Each function here does the same for the plain case (tensors of the
// right types and shapes on the current device, its current stream, no
// workspace passed) and returns what the Python function returns; an int is a
// status other than LA_OK; None means that the call is not of the plain kind,
// and the Python code takes it, with its full checks and messages.
#include <Python.h>

#include <algorithm>
#include <array>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "lightning_attn.h"

namespace {

constexpr auto BF16 = at::kBFloat16, FP32 = at::kFloat, INT32 = at::kInt;

// A tensor argument: exactly torch.Tensor, contiguous, on `dev`, of this type.
struct Arg {
    const at::Tensor *t = nullptr;
    bool ok(PyObject *o, at::ScalarType type, int dim, int dev) {
        if (!THPVariable_CheckExact(o)) return false;
        t = &THPVariable_Unpack(o);
        return t->is_cuda() && t->scalar_type() == type && t->dim() == dim && t->is_contiguous() &&
               (dev < 0 || t->get_device() == dev);
    }
    int64_t size(int i) const { return t->size(i); }
    bool sized(std::initializer_list<int64_t> s) const { return t->sizes().equals(at::IntArrayRef(s)); }
    void *ptr() const { return t->data_ptr(); }
};

bool small(int64_t x) { return x <= 0x7fffffff; }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, int dev) {
    return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), c10::nullopt);
}

// An output: one that was passed (and fits), or one to be made, or (not `want`ed) none.
struct Output {
    at::Tensor t;
    std::array<int64_t, 3> sizes;
    int dim;
    at::ScalarType type;
    bool make_it;
    bool ok(PyObject *o, std::initializer_list<int64_t> s, at::ScalarType ty, int dev, bool want = true) {
        dim = (int)s.size();
        std::copy(s.begin(), s.end(), sizes.begin());
        type = ty;
        make_it = want && o == Py_None;
        if (o == Py_None) return true;
        Arg a;
        if (!a.ok(o, type, dim, dev) || !a.sized(s)) return false;
        t = *a.t;
        return true;
    }
    void *ptr(int dev) {
        if (make_it) t = make(at::IntArrayRef(sizes.data(), dim), type, dev);
        return t.defined() ? t.data_ptr() : nullptr;
    }
};

// Other Python threads run meanwhile: an allocation or a launch may block (a full launch
// queue), and what it waits for may need one of them.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// q [T, H, d], k and v [T, Hkv, d] on the current device
struct Qkv {
    Arg q, k, v;
    int T, H, Hkv, d, dev;
    bool ok(PyObject *const *a) {
        if (!q.ok(a[0], BF16, 3, -1)) return false;
        dev = q.t->get_device();
        if (dev != c10::cuda::current_device() || !k.ok(a[1], BF16, 3, dev) || !v.ok(a[2], BF16, 3, dev)) return false;
        if (!small(q.size(0)) || !small(q.size(1)) || !small(q.size(2)) || !small(k.size(1))) return false;
        T = (int)q.size(0);
        H = (int)q.size(1);
        d = (int)q.size(2);
        Hkv = (int)k.size(1);
        return k.sized({T, Hkv, d}) && v.sized({T, Hkv, d}) && H > 0 && Hkv > 0 && H % Hkv == 0;
    }
};

struct Cache {
    Arg k, v, table, lens;
    int n_pages, page, max_pages;
    bool ok(PyObject *const *a, const Qkv &x, int n) {
        if (!k.ok(a[0], BF16, 4, x.dev) || !v.ok(a[1], BF16, 4, x.dev) || !table.ok(a[2], INT32, 2, x.dev) ||
            !lens.ok(a[3], INT32, 1, x.dev))
            return false;
        if (!small(k.size(0)) || !small(k.size(2)) || !small(table.size(1))) return false;
        n_pages = (int)k.size(0);
        page = (int)k.size(2);
        max_pages = (int)table.size(1);
        return k.sized({n_pages, x.Hkv, page, x.d}) && v.sized({n_pages, x.Hkv, page, x.d}) &&
               table.sized({n, max_pages}) && lens.size(0) == n;
    }
};

struct CachePtrs {
    void *k, *v;
    const int *table, *lens;
    explicit CachePtrs(const Cache &c)
        : k(c.k.ptr()), v(c.v.ptr()), table((const int *)c.table.ptr()), lens((const int *)c.lens.ptr()) {}
};

struct Workspace {
    size_t bytes;
    at::Tensor t;
    void *at = nullptr;
    Workspace(size_t n, int dev) : bytes(n) {
        if (!n) return;
        t = make({(int64_t)n}, at::kByte, dev);
        at = t.data_ptr();
    }
};

cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

bool number(PyObject *o, float &x) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    x = (float)v;
    return true;
}
bool length(PyObject *o, int &x) {
    int overflow = 0;
    const long v = PyLong_Check(o) ? PyLong_AsLongAndOverflow(o, &overflow) : (overflow = 1, 0L);
    if (overflow || v < 0 || v > INT32_MAX) return false;
    x = (int)v;
    return true;
}

// 1 or 0; -1 for what has no truth value
int truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) PyErr_Clear();
    return x;
}

PyObject *result(la_status st, const at::Tensor &out, const at::Tensor &lse) {
    if (st != LA_OK) return PyLong_FromLong(st);
    PyObject *a = THPVariable_Wrap(out);
    PyObject *b = lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(Py_None);
    return Py_BuildValue("(NN)", a, b);
}

// A C++ exception (an allocation that failed, before anything was launched): the
// Python code tries again and raises torch's own error.
template <class F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const std::exception &) {
        Py_RETURN_NONE;
    }
}

// (q, k, v, cu_seqlens, max_seqlen, scale, out, lse, want_lse)
PyObject *prefill_varlen(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Qkv x;
        Arg cu;
        float scale;
        int longest;
        if (n != 9 || !x.ok(a) || !cu.ok(a[3], INT32, 1, x.dev) || cu.size(0) < 1 || !small(cu.size(0)) ||
            !length(a[4], longest) || !number(a[5], scale))
            Py_RETURN_NONE;
        Output out, lse;
        const int want = truth(a[8]);
        if (want < 0 || !out.ok(a[6], {x.T, x.H, x.d}, BF16, x.dev) || !lse.ok(a[7], {x.T, x.H}, FP32, x.dev, want))
            Py_RETURN_NONE;
        const int nseq = (int)cu.size(0) - 1;
        const void *q = x.q.ptr(), *k = x.k.ptr(), *v = x.v.ptr();
        const int *seqs = (const int *)cu.ptr();
        const la_status st = [&] {
            Unlocked free;
            void *o = out.ptr(x.dev), *l = lse.ptr(x.dev);
            Workspace ws(la_softmax_prefill_varlen_workspace_size(nseq, x.T, x.H, x.Hkv, x.d), x.dev);
            return la_softmax_prefill_varlen(q, k, v, seqs, nseq, x.T, longest, x.H, x.Hkv, x.d, scale, o, (float *)l,
                                             ws.at, ws.bytes, stream_of(x.dev));
        }();
        return result(st, out.t, lse.t);
    });
}

// (q, k, v, cu_seqlens, max_seqlen, k_cache, v_cache, page_table, cache_lens, scale, out, lse, want_lse)
PyObject *prefill_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Qkv x;
        Arg cu;
        Cache c;
        float scale;
        int longest;
        if (n != 13 || !x.ok(a) || !cu.ok(a[3], INT32, 1, x.dev) || cu.size(0) < 1 || !small(cu.size(0)) ||
            !length(a[4], longest) || !c.ok(a + 5, x, (int)cu.size(0) - 1) || !number(a[9], scale))
            Py_RETURN_NONE;
        Output out, lse;
        const int want = truth(a[12]);
        if (want < 0 || !out.ok(a[10], {x.T, x.H, x.d}, BF16, x.dev) || !lse.ok(a[11], {x.T, x.H}, FP32, x.dev, want))
            Py_RETURN_NONE;
        const int nseq = (int)cu.size(0) - 1;
        const void *q = x.q.ptr(), *k = x.k.ptr(), *v = x.v.ptr();
        const int *seqs = (const int *)cu.ptr();
        const CachePtrs p(c);
        const la_status st = [&] {
            Unlocked free;
            void *o = out.ptr(x.dev), *l = lse.ptr(x.dev);
            Workspace ws(la_softmax_prefill_paged_workspace_size(nseq, x.T, x.H, x.Hkv, x.d, c.page, c.max_pages), x.dev);
            return la_softmax_prefill_paged(q, k, v, seqs, nseq, x.T, longest, x.H, x.Hkv, x.d, scale, p.k, p.v,
                                            c.n_pages, c.page, p.table, c.max_pages, p.lens, o, (float *)l, ws.at,
                                            ws.bytes, stream_of(x.dev));
        }();
        return result(st, out.t, lse.t);
    });
}

// (q, k, v, k_cache, v_cache, page_table, cache_lens, scale, out, fp32, lse, want_lse)
PyObject *decode_paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Qkv x;
        Cache c;
        float scale;
        if (n != 12 || !x.ok(a) || !c.ok(a + 3, x, x.T) || !number(a[7], scale)) Py_RETURN_NONE;
        Output out, lse;
        const auto type = a[9] == Py_True ? FP32 : BF16;
        const int want = truth(a[11]);
        if (want < 0 || !out.ok(a[8], {x.T, x.H, x.d}, type, x.dev) || !lse.ok(a[10], {x.T, x.H}, FP32, x.dev, want))
            Py_RETURN_NONE;
        const void *q = x.q.ptr(), *k = x.k.ptr(), *v = x.v.ptr();
        const CachePtrs p(c);
        const la_status st = [&] {
            Unlocked free;
            void *o = out.ptr(x.dev), *l = lse.ptr(x.dev);
            Workspace ws(la_softmax_decode_paged_workspace_size(x.T, x.H, x.Hkv, x.d, c.page, c.max_pages), x.dev);
            return la_softmax_decode_paged(q, k, v, x.T, x.H, x.Hkv, x.d, scale, p.k, p.v, c.n_pages, c.page, p.table,
                                           c.max_pages, p.lens, o, type == FP32 ? LA_FP32 : LA_BF16, (float *)l, ws.at,
                                           ws.bytes, stream_of(x.dev));
        }();
        return result(st, out.t, lse.t);
    });
}

// (q, k, v, out, lse, dout, cu_seqlens, max_seqlen, scale, dq, dk, dv)
PyObject *prefill_backward_varlen(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Qkv x;
        Arg out, lse, dout, cu;
        float scale;
        int longest;
        if (n != 12 || !x.ok(a) || !out.ok(a[3], BF16, 3, x.dev) || !out.sized({x.T, x.H, x.d}) ||
            !lse.ok(a[4], FP32, 2, x.dev) || !lse.sized({x.T, x.H}) || !dout.ok(a[5], BF16, 3, x.dev) ||
            !dout.sized({x.T, x.H, x.d}) || !cu.ok(a[6], INT32, 1, x.dev) || cu.size(0) < 1 || !small(cu.size(0)) ||
            !length(a[7], longest) || !number(a[8], scale))
            Py_RETURN_NONE;
        Output dq, dk, dv;
        if (!dq.ok(a[9], {x.T, x.H, x.d}, BF16, x.dev) || !dk.ok(a[10], {x.T, x.Hkv, x.d}, BF16, x.dev) ||
            !dv.ok(a[11], {x.T, x.Hkv, x.d}, BF16, x.dev))
            Py_RETURN_NONE;
        const int nseq = (int)cu.size(0) - 1;
        const void *q = x.q.ptr(), *k = x.k.ptr(), *v = x.v.ptr(), *o = out.ptr(), *g = dout.ptr();
        const float *l = (const float *)lse.ptr();
        const int *seqs = (const int *)cu.ptr();
        const la_status st = [&] {
            Unlocked free;
            void *to_q = dq.ptr(x.dev), *to_k = dk.ptr(x.dev), *to_v = dv.ptr(x.dev);
            Workspace ws(la_softmax_prefill_backward_varlen_workspace_size(nseq, x.T, x.H, x.Hkv, x.d), x.dev);
            return la_softmax_prefill_backward_varlen(q, k, v, o, l, g, seqs, nseq, x.T, longest, x.H, x.Hkv, x.d, scale,
                                                      to_q, to_k, to_v, ws.at, ws.bytes, stream_of(x.dev));
        }();
        if (st != LA_OK) return PyLong_FromLong(st);
        return Py_BuildValue("(NNN)", THPVariable_Wrap(dq.t), THPVariable_Wrap(dk.t), THPVariable_Wrap(dv.t));
    });
}

// (k_cache, v_cache, src, dst): () when done
PyObject *copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Arg k, v, src, dst;
        if (n != 4 || !k.ok(a[0], BF16, 4, -1)) Py_RETURN_NONE;
        const int dev = k.t->get_device();
        if (dev != c10::cuda::current_device() || !v.ok(a[1], BF16, 4, dev) || !v.t->sizes().equals(k.t->sizes()) ||
            !src.ok(a[2], INT32, 1, dev) || !dst.ok(a[3], INT32, 1, dev) || src.size(0) != dst.size(0))
            Py_RETURN_NONE;
        for (int i = 0; i < 4; ++i)
            if (!small(k.size(i))) Py_RETURN_NONE;
        if (!small(src.size(0))) Py_RETURN_NONE;
        const int pages = (int)k.size(0), heads = (int)k.size(1), page = (int)k.size(2), d = (int)k.size(3);
        const int count = (int)src.size(0);
        void *kp = k.ptr(), *vp = v.ptr();
        const int *from = (const int *)src.ptr(), *to = (const int *)dst.ptr();
        const la_status st = [&] {
            Unlocked free;
            return la_cache_copy_pages(kp, vp, pages, page, heads, d, from, to, count, stream_of(dev));
        }();
        return st == LA_OK ? PyTuple_New(0) : PyLong_FromLong(st);
    });
}

PyMethodDef methods[] = {
    {"prefill_varlen", (PyCFunction)(void (*)(void))prefill_varlen, METH_FASTCALL, nullptr},
    {"prefill_backward_varlen", (PyCFunction)(void (*)(void))prefill_backward_varlen, METH_FASTCALL, nullptr},
    {"prefill_paged", (PyCFunction)(void (*)(void))prefill_paged, METH_FASTCALL, nullptr},
    {"decode_paged", (PyCFunction)(void (*)(void))decode_paged, METH_FASTCALL, nullptr},
    {"copy_pages", (PyCFunction)(void (*)(void))copy_pages, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
