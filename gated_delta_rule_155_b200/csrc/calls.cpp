// calls.cpp — the binding's short calls: the entry points whose kernels take a few microseconds, with
// well-formed torch tensors, checked and marshalled in C++ (about 5 us a call; in Python 10 to 20).
//
// Every function takes the tensors of the Python function of its name and answers
//   None         not taken: something is not as the fast path needs it (a shape, a dtype, a device, an
//                allocation that failed); the Python function then checks argument by argument and raises
//   int          the status of the C entry point, not KDA_OK
//   otherwise    the call's result
// No exception leaves a function.  The C entry points are reached through their addresses (init).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kda.h"

namespace {

struct Entries {
    decltype(&kda_gdr_decode) decode;
    decltype(&kda_gdr_workspace_size) gdr_bytes;
    decltype(&kda_gdr_forward) forward;
    decltype(&kda_gdr_backward) backward;
    decltype(&kda_pages_fork) fork;
    decltype(&kda_pages_free) free_;
    decltype(&kda_pages_workspace_size) pages_bytes;
    decltype(&kda_pages_compact) compact;
} lib{};

// A tensor argument: false unless it is exactly a torch.Tensor on the current device, contiguous.
struct Arg {
    const at::Tensor *t = nullptr;
    bool none = false;
};
bool take(PyObject *o, int device, Arg &a)
{
    if (o == Py_None) {
        a.none = true;
        return true;
    }
    if (!THPVariable_CheckExact(o)) return false;
    a.t = &THPVariable_Unpack(o);
    return a.t->is_cuda() && a.t->get_device() == device && a.t->is_contiguous();
}
bool has(const Arg &a, at::ScalarType type, at::IntArrayRef sizes) { return a.t && a.t->scalar_type() == type && a.t->sizes() == sizes; }
template <typename T = void>
T *ptr(const Arg &a) { return a.t ? static_cast<T *>(a.t->data_ptr()) : nullptr; }
bool io_type(at::ScalarType t, kda_dtype_t &io)
{
    io = t == at::kFloat ? KDA_F32 : KDA_BF16;
    return t == at::kFloat || t == at::kBFloat16;
}
bool fits_int(std::initializer_list<int64_t> v)
{
    for (int64_t x : v)
        if (x < 0 || x > 0x7fffffff) return false;
    return true;
}
PyObject *result(kda_status_t st, PyObject *value)   // value: a new reference
{
    if (st == KDA_OK) return value;
    Py_DECREF(value);
    return PyLong_FromLong(st);
}
template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
kda_stream_t stream_of(int device) { return (kda_stream_t)c10::cuda::getCurrentCUDAStream(device).stream(); }

// q, k, v, g, beta, state, index, out
PyObject *gdr_decode(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 8) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[8];
        for (int i = 0; i < 8; ++i)
            if (!take(o[i], dev, a[i]) || (i < 6 && a[i].none)) Py_RETURN_NONE;
        const at::Tensor &q = *a[0].t, &v = *a[2].t;
        const int64_t d = q.dim();
        kda_dtype_t io;
        if ((d != 3 && d != 4) || v.dim() != d || !io_type(q.scalar_type(), io)) Py_RETURN_NONE;
        const int64_t N = q.size(0), T = d == 4 ? q.size(1) : 1, Hk = q.size(d - 2), dk = q.size(d - 1), Hv = v.size(d - 2), dv = v.size(d - 1);
        const auto type = q.scalar_type();
        const int64_t wide[4] = {N, T, Hv, dv}, flat[3] = {N, Hv, dv}, gw[3] = {N, T, Hv}, gf[2] = {N, Hv};
        const at::IntArrayRef sv = d == 4 ? at::IntArrayRef(wide) : at::IntArrayRef(flat), sg = d == 4 ? at::IntArrayRef(gw) : at::IntArrayRef(gf);
        if (!has(a[1], type, q.sizes()) || !has(a[2], type, sv) || !has(a[3], type, sg) || !has(a[4], type, sg)) Py_RETURN_NONE;
        if (a[5].t->dim() != 4) Py_RETURN_NONE;
        const int64_t P = a[6].none ? N : a[5].t->size(0);
        if (!has(a[5], at::kFloat, {P, Hv, dk, dv}) || (!a[6].none && !has(a[6], at::kInt, {N}))) Py_RETURN_NONE;
        if (!a[7].none && !has(a[7], type, sv)) Py_RETURN_NONE;
        if (!fits_int({N, T, Hk, Hv, dk, dv, P})) Py_RETURN_NONE;
        at::Tensor out = a[7].none ? at::empty_like(v) : *a[7].t;
        const kda_status_t st = lib.decode(ptr(a[0]), ptr(a[1]), ptr(a[2]), ptr(a[3]), ptr(a[4]), ptr<float>(a[5]), ptr<int>(a[6]), (int)P,
                                           out.data_ptr(), (int)N, (int)T, (int)Hk, (int)Hv, (int)dk, (int)dv, io, stream_of(dev));
        if (st != KDA_OK) return PyLong_FromLong(st);
        if (!a[7].none) {
            Py_INCREF(o[7]);
            return o[7];
        }
        return THPVariable_Wrap(out);
    });
}

// The sizes of q, k, v, g, beta (a[0..4]), packed where cu is given; false where they do not fit together.
struct Shape {
    int64_t N, T, Hk, Hv, dk, dv;
    kda_dtype_t io;
    bool of(const Arg *a, const Arg &cu)
    {
        const at::Tensor &q = *a[0].t, &v = *a[2].t;
        const bool packed = !cu.none;
        const int64_t d = packed ? 3 : 4;
        if (q.dim() != d || v.dim() != d || !io_type(q.scalar_type(), io)) return false;
        const auto type = q.scalar_type();
        N = T = q.size(0);
        if (packed) {
            if (cu.t->dim() != 1 || cu.t->size(0) < 2 || cu.t->scalar_type() != at::kInt) return false;
            N = cu.t->size(0) - 1;
        } else {
            if (q.size(1) > 0x7fffffff) return false;
            T = N * q.size(1);
        }
        Hk = q.size(d - 2), dk = q.size(d - 1), Hv = v.size(d - 2), dv = v.size(d - 1);
        const int64_t s4[4] = {q.size(0), packed ? 0 : q.size(1), Hv, dv}, s3[3] = {q.size(0), Hv, dv}, g3[3] = {s4[0], s4[1], Hv}, g2[2] = {s4[0], Hv};
        const at::IntArrayRef sv = packed ? at::IntArrayRef(s3) : at::IntArrayRef(s4), sg = packed ? at::IntArrayRef(g2) : at::IntArrayRef(g3);
        return has(a[1], type, q.sizes()) && has(a[2], type, sv) && has(a[3], type, sg) && has(a[4], type, sg) && fits_int({N, T, Hk, Hv, dk, dv});
    }
};

// q, k, v, g, beta, cu_seqlens, initial_state, out, final_state, initial_index, final_index -> out
PyObject *gdr_forward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 11) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[11];
        for (int i = 0; i < 11; ++i)
            if (!take(o[i], dev, a[i]) || (i < 5 && a[i].none)) Py_RETURN_NONE;
        Shape x;
        if (!x.of(a, a[5])) Py_RETURN_NONE;
        const int64_t N = x.N, T = x.T, Hk = x.Hk, Hv = x.Hv, dk = x.dk, dv = x.dv;
        const kda_dtype_t io = x.io;
        const at::Tensor &v = *a[2].t;
        if (!a[7].none && !has(a[7], v.scalar_type(), v.sizes())) Py_RETURN_NONE;
        int64_t pages = 0;
        for (int i = 0; i < 2; ++i) {          // initial, final: the state and its index
            const Arg &s = a[i ? 8 : 6], &x = a[i ? 10 : 9];
            if (s.none) {
                if (!x.none) Py_RETURN_NONE;
                continue;
            }
            if (s.t->dim() != 4 || (!x.none && !has(x, at::kInt, {N}))) Py_RETURN_NONE;
            const int64_t P = x.none ? N : s.t->size(0);
            if (!has(s, at::kFloat, {P, Hv, dk, dv})) Py_RETURN_NONE;
            if (!x.none) {
                if (pages && pages != P) Py_RETURN_NONE;
                pages = P;
            }
        }
        if (!fits_int({pages})) Py_RETURN_NONE;
        size_t bytes = 0;
        if (lib.gdr_bytes((int)N, (int)T, (int)Hk, (int)Hv, (int)dk, (int)dv, io, 0, &bytes) != KDA_OK) Py_RETURN_NONE;
        at::Tensor out = a[7].none ? at::empty_like(v) : *a[7].t, ws;
        if (bytes) ws = at::empty({(int64_t)bytes}, v.options().dtype(at::kByte));
        const kda_status_t st = lib.forward(ptr(a[0]), ptr(a[1]), ptr(a[2]), ptr(a[3]), ptr(a[4]), ptr<float>(a[6]), ptr<int>(a[9]), out.data_ptr(),
                                            ptr<float>(a[8]), ptr<int>(a[10]), (int)pages, ptr<int>(a[5]), bytes ? ws.data_ptr() : nullptr, bytes,
                                            (int)N, (int)T, (int)Hk, (int)Hv, (int)dk, (int)dv, io, stream_of(dev));
        if (st != KDA_OK) return PyLong_FromLong(st);
        if (!a[7].none) {
            Py_INCREF(o[7]);
            return o[7];
        }
        return THPVariable_Wrap(out);
    });
}

// q, k, v, g, beta, d_out, cu_seqlens, initial_state, d_final_state, d_initial_state -> (dq, dk, dv, dg, dbeta)
PyObject *gdr_backward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 10) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[10];
        for (int i = 0; i < 10; ++i)
            if (!take(o[i], dev, a[i]) || (i < 6 && a[i].none)) Py_RETURN_NONE;
        Shape x;
        if (!x.of(a, a[6])) Py_RETURN_NONE;
        const at::Tensor &v = *a[2].t;
        if (!has(a[5], v.scalar_type(), v.sizes())) Py_RETURN_NONE;
        for (int i = 7; i < 10; ++i)
            if (!a[i].none && !has(a[i], at::kFloat, {x.N, x.Hv, x.dk, x.dv})) Py_RETURN_NONE;
        const int N = (int)x.N, T = (int)x.T, Hk = (int)x.Hk, Hv = (int)x.Hv, dk = (int)x.dk, dv = (int)x.dv;
        size_t bytes = 0;
        if (lib.gdr_bytes(N, T, Hk, Hv, dk, dv, x.io, 1, &bytes) != KDA_OK) Py_RETURN_NONE;
        at::Tensor d[5], ws;
        for (int i = 0; i < 5; ++i) d[i] = at::empty_like(*a[i].t);
        if (bytes) ws = at::empty({(int64_t)bytes}, v.options().dtype(at::kByte));
        const kda_status_t st = lib.backward(ptr(a[0]), ptr(a[1]), ptr(a[2]), ptr(a[3]), ptr(a[4]), ptr<float>(a[7]), ptr<int>(a[6]), ptr(a[5]),
                                             ptr<float>(a[8]), d[0].data_ptr(), d[1].data_ptr(), d[2].data_ptr(), d[3].data_ptr(), d[4].data_ptr(),
                                             ptr<float>(a[9]), bytes ? ws.data_ptr() : nullptr, bytes, N, T, Hk, Hv, dk, dv, x.io, stream_of(dev));
        if (st != KDA_OK) return PyLong_FromLong(st);
        PyObject *r = PyTuple_New(5);
        for (int i = 0; r && i < 5; ++i) {
            PyObject *t = THPVariable_Wrap(d[i]);
            if (!t) {
                Py_DECREF(r);
                return nullptr;
            }
            PyTuple_SET_ITEM(r, i, t);
        }
        return r;
    });
}

// layers, pages and bytes of a page of a cache
bool cache_of(const Arg &a, int64_t &L, int64_t &P, size_t &bytes)
{
    if (!a.t || a.t->dim() < 3) return false;
    L = a.t->size(0);
    P = a.t->size(1);
    if (L < 1 || P < 1 || !fits_int({L, P})) return false;
    bytes = (size_t)(a.t->numel() / (L * P)) * a.t->element_size();
    return true;
}
bool ids_of(const Arg &a, int64_t &n)
{
    if (!a.t || a.t->dim() != 1 || a.t->scalar_type() != at::kInt) return false;
    n = a.t->size(0);
    return fits_int({n});
}

// cache, refs, parents -> children
PyObject *pages_fork(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[3];
        int64_t L, P, m;
        size_t bytes;
        for (int i = 0; i < 3; ++i)
            if (!take(o[i], dev, a[i])) Py_RETURN_NONE;
        if (!cache_of(a[0], L, P, bytes) || !has(a[1], at::kInt, {P}) || !ids_of(a[2], m)) Py_RETURN_NONE;
        at::Tensor children = at::empty_like(*a[2].t);
        const kda_status_t st = lib.fork(ptr(a[0]), bytes, (int)L, (int)P, ptr<int>(a[1]), ptr<int>(a[2]), children.data_ptr<int>(), (int)m, stream_of(dev));
        if (st != KDA_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(children);
    });
}

// refs, ids -> True
PyObject *pages_free(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 2) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[2];
        int64_t P, m;
        if (!take(o[0], dev, a[0]) || !take(o[1], dev, a[1]) || !ids_of(a[0], P) || !ids_of(a[1], m)) Py_RETURN_NONE;
        Py_INCREF(Py_True);
        return result(lib.free_(ptr<int>(a[0]), (int)P, ptr<int>(a[1]), (int)m, stream_of(dev)), Py_True);
    });
}

// cache, refs, table -> live
PyObject *pages_compact(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject * {
        const int dev = c10::cuda::current_device();
        Arg a[3];
        int64_t L, P;
        size_t page = 0, bytes = 0;
        for (int i = 0; i < 3; ++i)
            if (!take(o[i], dev, a[i])) Py_RETURN_NONE;
        if (!cache_of(a[0], L, P, page) || !has(a[1], at::kInt, {P})) Py_RETURN_NONE;
        const int64_t m = a[2].none ? 0 : a[2].t->numel();
        if ((!a[2].none && a[2].t->scalar_type() != at::kInt) || !fits_int({m})) Py_RETURN_NONE;
        if (lib.pages_bytes((int)P, &bytes) != KDA_OK) Py_RETURN_NONE;
        at::Tensor live = at::empty({1}, a[1].t->options()), ws = at::empty({(int64_t)bytes}, a[1].t->options().dtype(at::kByte));
        const kda_status_t st = lib.compact(ptr(a[0]), page, (int)L, (int)P, ptr<int>(a[1]), ptr<int>(a[2]), (int)m, live.data_ptr<int>(),
                                            ws.data_ptr(), bytes, stream_of(dev));
        if (st != KDA_OK) return PyLong_FromLong(st);
        return THPVariable_Wrap(live);
    });
}

// The addresses of the entry points, in the order of Entries
PyObject *init(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (n != (Py_ssize_t)(sizeof(lib) / sizeof(void *))) {
        PyErr_SetString(PyExc_TypeError, "init takes the address of each entry point");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        void *p = PyLong_AsVoidPtr(o[i]);
        if (!p) return nullptr;
        reinterpret_cast<void **>(&lib)[i] = p;
    }
    Py_RETURN_NONE;
}

#define KDA_CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_CALL(init),       KDA_CALL(gdr_decode), KDA_CALL(gdr_forward), KDA_CALL(gdr_backward), KDA_CALL(pages_fork),
                         KDA_CALL(pages_free), KDA_CALL(pages_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Short calls of the kda binding", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
