// Python entry of the calls that a decode makes for every token of every layer: the paged cache's
// append, attend and evict. Checks the tensors (CUDA, one device, contiguous, type, shape) and
// calls libkvp.so with that device current, on the given stream or the device's current one.
//
// A decode step's kernels run for a few microseconds, so its host time counts: the same checks by
// Python attribute reads and a ctypes call took 16 to 18 us a call (an append of one token, an
// attention of 2111 rows), the two launches among them. The functions' addresses are handed over
// by the package, which loads the library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kvp.h"

namespace {

decltype(&kvp_cache_append) append_fn;
decltype(&kvp_cache_attend) attend_fn;
decltype(&kvp_cache_evict) evict_fn;

// Reads the arguments of one call; the first refusal sets a Python error and later ones keep it.
struct Reader {
    bool ok = true;
    int device = -1;
    at::ScalarType cache_type = at::kBFloat16;
    kvp_cache_shape shape{};

    void refuse(const char* name, const char* what) {
        if (ok) PyErr_Format(PyExc_ValueError, "%s %s", name, what);
        ok = false;
    }

    // a ctypes structure of the size of T
    template <typename T>
    void structure(PyObject* o, const char* name, T* to) {
        Py_buffer b;
        if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
            PyErr_Clear();
            return refuse(name, "is not the structure that this call takes");
        }
        if (b.len == (Py_ssize_t)sizeof(T)) memcpy(to, b.buf, sizeof(T));
        else refuse(name, "is not the structure that this call takes");
        PyBuffer_Release(&b);
    }

    void read_shape(PyObject* o) {
        structure(o, "shape", &shape);
        cache_type = shape.dtype == KVP_FP16 ? at::kHalf : at::kBFloat16;
    }

    // NULL for None (where optional)
    const at::Tensor* tensor(PyObject* o, const char* name, at::ScalarType type, bool optional = false) {
        if (!ok) return nullptr;
        if (o == Py_None) {
            if (!optional) refuse(name, "is required");
            return nullptr;
        }
        if (!THPVariable_Check(o)) return refuse(name, "must be a CUDA tensor"), nullptr;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) return refuse(name, "must be a CUDA tensor"), nullptr;
        if (t.scalar_type() != type) {
            if (ok) PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
            ok = false;
            return nullptr;
        }
        if (!t.is_contiguous()) return refuse(name, "must be contiguous"), nullptr;
        if (device < 0) device = t.get_device();
        if (t.get_device() != device) return refuse(name, "is on another device than the tensors before it"), nullptr;
        return &t;
    }

    void* pointer(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef sizes, bool optional = false) {
        const at::Tensor* t = tensor(o, name, type, optional);
        if (t == nullptr) return nullptr;
        if (t->sizes() != sizes) {
            PyObject* is = PyObject_GetAttrString(o, "shape");
            std::string want = "(";
            for (int64_t x : sizes) want += std::to_string(x) + ", ";
            if (is) PyErr_Format(PyExc_ValueError, "%s has shape %S, expected %s)", name, is, want.c_str());
            Py_XDECREF(is);
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }

    uint16_t* pool(PyObject* o, const char* name) {
        return (uint16_t*)pointer(o, name, cache_type, {shape.num_pages, shape.page_size, shape.head_dim});
    }
    float* weights(PyObject* o, const char* name, bool optional = false) {
        return (float*)pointer(o, name, at::kFloat, {shape.num_pages, shape.page_size}, optional);
    }
    int32_t* heads(PyObject* o, const char* name, bool optional = false) {
        return (int32_t*)pointer(o, name, at::kInt, {shape.batch, shape.hkv}, optional);
    }
    int32_t* pages(PyObject* o) { return (int32_t*)pointer(o, "table", at::kInt, {shape.batch, shape.hkv, shape.max_pages}); }

    // None (the device's current stream), a torch.cuda.Stream, or a cudaStream_t as a number
    void* stream(PyObject* o) {
        if (!ok) return nullptr;
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        PyObject* number = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        void* s = number ? PyLong_AsVoidPtr(number) : nullptr;
        Py_XDECREF(number);
        if (PyErr_Occurred()) ok = false;
        return s;
    }

    template <typename F, typename... Args>
    PyObject* call(F fn, Args... args) {
        if (!ok) return nullptr;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        return PyLong_FromLong(fn(args...));
    }
};

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
    return false;
}

// shape, k_new, v_new, k_pages, v_pages, table, lens, lens_out, acc, weight, counts, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_is(n, 12)) return nullptr;
    Reader r;
    r.read_shape(a[0]);
    const kvp_cache_shape& s = r.shape;
    const at::Tensor* k = r.tensor(a[1], "k_new", r.cache_type);
    if (k == nullptr) return nullptr;
    const bool ragged = a[10] != Py_None;
    if (k->dim() != (ragged ? 3 : 4)) {
        r.refuse("k_new", ragged ? "must be [b, hkv * n, d] with counts" : "must be [b, hkv, n, d]");
        return nullptr;
    }
    const int64_t rows = ragged ? k->size(1) / (s.hkv > 0 ? s.hkv : 1) : k->size(2);
    if (rows > INT32_MAX) return r.refuse("k_new", "has too many rows"), nullptr;
    const int64_t flat[] = {s.batch, s.hkv * rows, s.head_dim}, whole[] = {s.batch, s.hkv, rows, s.head_dim};
    const at::IntArrayRef sizes = ragged ? at::IntArrayRef(flat, 3) : at::IntArrayRef(whole, 4);
    auto* kp = (uint16_t*)r.pointer(a[1], "k_new", r.cache_type, sizes);
    auto* vp = (uint16_t*)r.pointer(a[2], "v_new", r.cache_type, sizes);
    auto *kc = r.pool(a[3], "k_pages"), *vc = r.pool(a[4], "v_pages");
    auto* table = r.pages(a[5]);
    auto *lens = r.heads(a[6], "lens"), *lens_out = r.heads(a[7], "lens_out");
    auto* acc = r.weights(a[8], "acc", true);
    auto* weight = (float*)r.pointer(a[9], "weight", at::kFloat, sizes.slice(0, sizes.size() - 1), true);
    auto* counts = r.heads(a[10], "counts", true);
    void* stream = r.stream(a[11]);
    return r.call(append_fn, &s, kp, vp, (int32_t)rows, counts, weight, kc, vc, acc, table, lens, lens_out, stream);
}

// shape, q, k_pages, v_pages, table, lens, out, lse, acc, workspace, stream
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_is(n, 11)) return nullptr;
    Reader r;
    r.read_shape(a[0]);
    const kvp_cache_shape& s = r.shape;
    const int64_t heads[] = {s.batch, s.hq, s.head_dim};
    auto* q = (uint16_t*)r.pointer(a[1], "q", r.cache_type, heads);
    auto *kc = r.pool(a[2], "k_pages"), *vc = r.pool(a[3], "v_pages");
    auto* table = r.pages(a[4]);
    auto* lens = r.heads(a[5], "lens");
    auto* out = (uint16_t*)r.pointer(a[6], "out", r.cache_type, heads);
    auto* lse = (float*)r.pointer(a[7], "lse", at::kFloat, at::IntArrayRef(heads, 2), true);
    auto* acc = r.weights(a[8], "acc", true);
    const at::Tensor* ws = r.tensor(a[9], "workspace", at::kByte);
    void* stream = r.stream(a[10]);
    if (!r.ok) return nullptr;
    return r.call(attend_fn, &s, q, kc, vc, table, lens, out, lse, acc, ws->data_ptr(), (size_t)ws->numel(), stream);
}

// shape, evict, k_pages, v_pages, acc, acc_out, table, lens, lens_out, src, budgets, workspace, stream
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_is(n, 13)) return nullptr;
    Reader r;
    r.read_shape(a[0]);
    const kvp_cache_shape& s = r.shape;
    kvp_evict e{};
    r.structure(a[1], "evict", &e);
    auto *kc = r.pool(a[2], "k_pages"), *vc = r.pool(a[3], "v_pages");
    auto *acc = r.weights(a[4], "acc"), *acc_out = r.weights(a[5], "acc_out");
    auto* table = r.pages(a[6]);
    auto *lens = r.heads(a[7], "lens"), *lens_out = r.heads(a[8], "lens_out");
    auto* src = (int32_t*)r.pointer(a[9], "src", at::kInt, {s.batch, s.hkv, e.budget}, true);
    auto* budgets = r.heads(a[10], "budgets", true);
    const at::Tensor* ws = r.tensor(a[11], "workspace", at::kByte);
    void* stream = r.stream(a[12]);
    if (!r.ok) return nullptr;
    return r.call(evict_fn, &s, &e, budgets, kc, vc, acc, acc_out, table, lens, lens_out, src, ws->data_ptr(), (size_t)ws->numel(), stream);
}

// The library's functions, as addresses: append, attend, evict.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_is(n, 3)) return nullptr;
    append_fn = (decltype(append_fn))PyLong_AsVoidPtr(a[0]);
    attend_fn = (decltype(attend_fn))PyLong_AsVoidPtr(a[1]);
    evict_fn = (decltype(evict_fn))PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// An exception of torch's (a device that is not there) as a Python one.
template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return f(self, a, n);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {{"use", (PyCFunction)(void*)guarded<use>, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void*)guarded<append>, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void*)guarded<attend>, METH_FASTCALL, nullptr},
                         {"evict", (PyCFunction)(void*)guarded<evict>, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvp_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvp_binding() { return PyModule_Create(&module); }
