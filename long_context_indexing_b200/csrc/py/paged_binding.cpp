// paged_binding.cpp -- the paged cache's two per-token calls without ctypes.
//
// A decode loop calls lsa_paged_append and lsa_paged_attn once per layer and
// token; through Python's checks and ctypes a call costs 9 to 10 us of host time,
// more than the kernels of a small batch take.  Here the tensors' types, shapes,
// strides and devices are read from C++ and the same C entries are called.
//
// Each function takes the tensors as the Python functions of the same names do and
// returns what they return; NotImplemented when any check fails (the Python path
// then repeats the checks and says what is wrong) or when the cache's device is not
// current; an int, the lsa_status, when the C entry refused the call.  torch's own
// errors (out of memory) are raised as torch raises them.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "lsa.h"

namespace {

decltype(&lsa_paged_append) g_append = nullptr;
decltype(&lsa_paged_attn) g_attn = nullptr;

const at::Tensor* tensor(PyObject* o)
{
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Elements between token rows of a bfloat16 [B][Nq][H][d] tensor with contiguous
// rows at one distance; -1: it is not one.  H < 0: any.
int64_t rows(const at::Tensor* t, int64_t dev, int64_t B, int64_t Nq, int64_t H, int64_t d)
{
    if (!t || t->scalar_type() != at::kBFloat16 || t->dim() != 4 || !t->is_cuda() ||
        t->get_device() != dev)
        return -1;
    const auto s = t->sizes(), st = t->strides();
    if (s[0] != B || s[1] != Nq || s[3] != d || (H >= 0 && s[2] != H)) return -1;
    const int64_t row = Nq > 1 ? st[1] : (B > 1 ? st[0] : s[2] * d);
    if (st[3] != 1 || (st[2] != d && s[2] > 1) || (st[0] != Nq * row && B > 1)) return -1;
    return row;
}

bool flat(const at::Tensor* t, int64_t dev, at::ScalarType type, at::IntArrayRef shape)
{
    return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev &&
           t->sizes() == shape && t->is_contiguous();
}

// The cache (lsa_paged_kv address, device index) when its device is current.
const lsa_paged_kv* cache(PyObject* addr, PyObject* index, int64_t* dev)
{
    const auto* kv = static_cast<const lsa_paged_kv*>(PyLong_AsVoidPtr(addr));
    *dev = PyLong_AsLongLong(index);
    if (!kv || PyErr_Occurred() || *dev != (int64_t)c10::cuda::current_device()) {
        PyErr_Clear();
        return nullptr;
    }
    return kv;
}

#define NO Py_RETURN_NOTIMPLEMENTED

// append(cache address, device, k, v, start, n_new, q, q_out, inv_freq, interleaved)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 10) NO;
    HANDLE_TH_ERRORS
    {
        int64_t dev;
        const lsa_paged_kv* kv = cache(a[0], a[1], &dev);
        const at::Tensor *k = tensor(a[2]), *v = tensor(a[3]), *start = tensor(a[4]);
        if (!kv || !k || k->dim() != 4) NO;
        const int64_t B = kv->B, Nq = k->size(1);
        const int64_t ks = rows(k, dev, B, Nq, kv->Hkv, kv->d);
        const int64_t vs = rows(v, dev, B, Nq, kv->Hkv, kv->d);
        if (Nq < 1 || ks < 0 || vs < 0 || !flat(start, dev, at::kInt, {B})) NO;
        const at::Tensor* n_new = nullptr;
        if (a[5] != Py_None && !flat(n_new = tensor(a[5]), dev, at::kInt, {B})) NO;
        const at::Tensor* q = nullptr;
        int64_t qs = 0, Hq = 0;
        at::Tensor made;
        const at::Tensor* q_out = nullptr;
        if (a[6] != Py_None) {
            q = tensor(a[6]);
            qs = rows(q, dev, B, Nq, -1, kv->d);
            if (qs < 0) NO;
            Hq = q->size(2);
            if (a[7] == Py_None) {
                // (the call leaves the rows of padding as they are)
                made = n_new ? at::zeros(q->sizes(), q->options())
                             : at::empty(q->sizes(), q->options(), at::MemoryFormat::Contiguous);
                q_out = &made;
            } else if (!flat(q_out = tensor(a[7]), dev, at::kBFloat16, q->sizes())) {
                NO;
            }
        } else if (a[7] != Py_None) {
            NO;
        }
        const at::Tensor* inv = nullptr;
        if (a[8] != Py_None) {
            inv = tensor(a[8]);
            if (!inv || inv->dim() != 1 || !flat(inv, dev, at::kFloat, inv->sizes())) NO;
        }
        const int inter = PyObject_IsTrue(a[9]);
        if (inter < 0) return nullptr;
        void* st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        lsa_status rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_append(kv, k->data_ptr(), ks, v->data_ptr(), vs, q ? q->data_ptr() : nullptr, qs,
                      q ? q_out->data_ptr() : nullptr, Nq, (int)Hq, start->data_ptr<int>(),
                      n_new ? n_new->data_ptr<int>() : nullptr,
                      inv ? inv->data_ptr<float>() : nullptr, inv ? (int)(2 * inv->numel()) : 0,
                      inter, st);
        Py_END_ALLOW_THREADS
        if (rc != LSA_OK) return PyLong_FromLong(rc);
        if (!q) Py_RETURN_NONE;
        if (a[7] == Py_None) return THPVariable_Wrap(std::move(made));
        Py_INCREF(a[7]);
        return a[7];
    }
    END_HANDLE_TH_ERRORS
}

// attn(cache address, device, Q, indices, counts, scale, return_lse, out)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 8) NO;
    HANDLE_TH_ERRORS
    {
        int64_t dev;
        const lsa_paged_kv* kv = cache(a[0], a[1], &dev);
        const at::Tensor *Q = tensor(a[2]), *idx = tensor(a[3]), *cnt = tensor(a[4]);
        if (!kv || !Q || Q->dim() != 4 || !idx || idx->dim() != 3) NO;
        const int64_t B = Q->size(0), Nq = Q->size(1), Hq = Q->size(2), d = Q->size(3);
        const int64_t s_max = idx->size(2);
        if (B != kv->B || d != kv->d || Nq < 1 || s_max > INT32_MAX ||
            !flat(Q, dev, at::kBFloat16, Q->sizes()) || !flat(idx, dev, at::kInt, {B, Nq, s_max}) ||
            !flat(cnt, dev, at::kInt, {B, Nq}))
            NO;
        double scale = 1.0 / std::sqrt((double)d);
        if (a[5] != Py_None) {
            scale = PyFloat_AsDouble(a[5]);
            if (PyErr_Occurred()) return nullptr;
        }
        const int want = PyObject_IsTrue(a[6]);
        if (want < 0) return nullptr;
        at::Tensor made, lse;
        const at::Tensor* out = nullptr;
        if (a[7] == Py_None) {
            made = at::empty(Q->sizes(), Q->options());
            out = &made;
        } else if (!flat(out = tensor(a[7]), dev, at::kBFloat16, Q->sizes())) {
            NO;
        }
        if (want) lse = at::empty({B, Nq, Hq}, Q->options().dtype(at::kFloat));
        void* st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        lsa_status rc;
        Py_BEGIN_ALLOW_THREADS
        rc = g_attn(kv, Q->data_ptr(), Nq, (int)Hq, idx->data_ptr<int>(), cnt->data_ptr<int>(),
                    (int)s_max, (float)scale, out->data_ptr(),
                    want ? lse.data_ptr<float>() : nullptr, st);
        Py_END_ALLOW_THREADS
        if (rc != LSA_OK) return PyLong_FromLong(rc);
        PyObject* o = a[7] == Py_None ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[7]);
        if (!o || !want) return o;
        PyObject* l = THPVariable_Wrap(std::move(lse));
        PyObject* both = l ? PyTuple_Pack(2, o, l) : nullptr;
        Py_DECREF(o);
        Py_XDECREF(l);
        return both;
    }
    END_HANDLE_TH_ERRORS
}

// bind(address of lsa_paged_append, address of lsa_paged_attn)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "bind takes two addresses");
        return nullptr;
    }
    g_append = (decltype(g_append))PyLong_AsVoidPtr(a[0]);
    g_attn = (decltype(g_attn))PyLong_AsVoidPtr(a[1]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attn", (PyCFunction)(void (*)(void))attn, METH_FASTCALL, nullptr},
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding()
{
    PyObject* m = PyModule_Create(&module);
    // the torch it was compiled for: another one's tensors have another layout
    if (m && PyModule_AddStringConstant(m, "torch_version", LSA_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
