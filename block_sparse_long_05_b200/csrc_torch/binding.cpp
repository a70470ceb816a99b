// binding.cpp -- the paged-cache calls of libmsa on torch tensors, as a CPython
// module (_msa_torch).
//
// These calls take 5 to 15 us on the GPU and are made once per layer and token,
// so what they cost on the host shows: checking a dozen tensors and marshalling
// two dozen arguments in Python (ctypes) took 7 to 11 us per call beside the
// launch, here it is 1 to 2 us.  The functions check types, shapes, strides and
// devices, make the outputs that were not given, and pass pointers to the C ABI
// (include/msa.h); no computation happens here.  libmsa itself does not know
// torch: bind() takes the addresses of its functions.
//
// Each function returns the call's outputs (None where there are none), or the
// status code as an int where it is not MSA_OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include "msa.h"

namespace {

decltype(&msa_kv_append) f_append;
decltype(&msa_kv_append_i8) f_append_i8;
decltype(&msa_kv_gather) f_gather;
decltype(&msa_kv_gather_i8) f_gather_i8;
decltype(&msa_attn_paged) f_attn;
decltype(&msa_attn_paged_i8) f_attn_i8;
decltype(&msa_sparse_attn_paged_i8) f_sparse_i8;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};  // a Python exception is set

using at::ScalarType;

const char *type_name(ScalarType t) {
    switch (t) {
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Char: return "torch.int8";
        case ScalarType::Int: return "torch.int32";
        default: return "torch.float32";
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The tensors of a call lie on the workspace's device.
struct Call {
    int device;
    void *ws;
    size_t ws_bytes;

    void place(const at::Tensor &t, ScalarType type, const char *name) const {
        if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
        if (t.scalar_type() != type) throw Refused(std::string(name) + " must be " + type_name(type));
        if (t.get_device() != device)
            throw Refused(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the workspace on cuda:" +
                          std::to_string(device));
    }
    // A contiguous tensor of this type.
    const at::Tensor &take(PyObject *o, ScalarType type, const char *name) const {
        const at::Tensor &t = tensor(o, name);
        place(t, type, name);
        if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
        return t;
    }
    // A packed bf16 tensor whose rows are contiguous, and the elements between them.
    const at::Tensor &rows(PyObject *o, int64_t dims, const char *name, int64_t &stride) const {
        const at::Tensor &t = tensor(o, name);
        place(t, ScalarType::BFloat16, name);
        if (t.dim() != dims) throw Refused(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
        int64_t width = 1;
        for (int64_t i = dims - 1; i > 0; --i) {
            if (t.size(i) != 1 && t.stride(i) != width) throw Refused(std::string(name) + ": each row must be contiguous");
            width *= t.size(i);
        }
        stride = t.size(0) > 1 ? t.stride(0) : width;
        return t;
    }
    at::Tensor make(at::IntArrayRef shape, ScalarType type) const {
        return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt);
    }
    // `given`, or a new tensor.
    at::Tensor output(PyObject *given, at::IntArrayRef shape, ScalarType type, const char *name) const {
        if (given == Py_None) return make(shape, type);
        const at::Tensor &t = take(given, type, name);
        if (t.sizes() != shape) throw Refused(std::string(name) + " has the wrong shape");
        return t;
    }
};

struct Stores {
    at::Tensor k, v, ks, vs;
    int pages, block, Hkv, d;
};

Stores stores(const Call &c, PyObject *const *a, bool i8) {  // k_pages, v_pages, k_scales, v_scales
    Stores s;
    const ScalarType type = i8 ? ScalarType::Char : ScalarType::BFloat16;
    s.k = c.take(a[0], type, "k_pages");
    s.v = c.take(a[1], type, "v_pages");
    if (s.k.dim() != 4 || s.v.sizes() != s.k.sizes())
        throw Refused("k_pages and v_pages must be [num_pages, block, Hkv, d]");
    if (i8) {
        s.ks = c.take(a[2], ScalarType::Float, "k_scales");
        s.vs = c.take(a[3], ScalarType::Float, "v_scales");
        const int64_t want[3] = {s.k.size(0), s.k.size(2), s.k.size(1)};
        if (s.ks.sizes() != at::IntArrayRef(want, 3) || s.vs.sizes() != at::IntArrayRef(want, 3))
            throw Refused("k_scales and v_scales must be [num_pages, Hkv, block]");
    }
    for (int i = 0; i < 4; ++i)
        if (s.k.size(i) > INT32_MAX) throw Refused("k_pages: a dimension is too large");
    s.pages = static_cast<int>(s.k.size(0));
    s.block = static_cast<int>(s.k.size(1));
    s.Hkv = static_cast<int>(s.k.size(2));
    s.d = static_cast<int>(s.k.size(3));
    return s;
}

struct Step {
    at::Tensor table, cu, len;
    int stride, Bt;
    const int32_t *t() const { return table.const_data_ptr<int32_t>(); }
};

Step step(const Call &c, PyObject *const *a) {  // page_table, cu, kv_len
    Step s;
    s.table = c.take(a[0], ScalarType::Int, "page_table");
    s.cu = c.take(a[1], ScalarType::Int, "cu");
    s.len = c.take(a[2], ScalarType::Int, "kv_len");
    const int64_t Bt = s.len.dim() == 1 ? s.len.size(0) : -1;
    if (s.table.dim() != 2 || s.table.size(0) != Bt || s.cu.dim() != 1 || s.cu.size(0) != Bt + 1 || Bt > INT32_MAX ||
        s.table.size(1) > INT32_MAX)
        throw Refused("page_table must be [Bt, page_stride], cu [Bt + 1], kv_len [Bt]");
    s.stride = static_cast<int>(s.table.size(1));
    s.Bt = static_cast<int>(Bt);
    return s;
}

int integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
    return static_cast<int>(v);
}

int rows_of(const at::Tensor &t, const char *name) {
    if (t.size(0) > INT32_MAX) throw Refused(std::string(name) + " has too many rows");
    return static_cast<int>(t.size(0));
}

// The stream of a call: the device's current one, or the given one, which is then
// current until the guard ends, so that the outputs' memory is its own.
void *stream_of(PyObject *o, int device, c10::cuda::OptionalCUDAStreamGuard &guard) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    PyObject *raw = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!raw) throw PythonError();
    void *p = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (!p && PyErr_Occurred()) throw PythonError();
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), static_cast<c10::DeviceIndex>(device)));
    return p;
}

// Arguments 0..2 of every function: the workspace's address, bytes and device.
Call call_of(PyObject *const *a) {
    Call c;
    c.ws = PyLong_AsVoidPtr(a[0]);
    c.ws_bytes = PyLong_AsSize_t(a[1]);
    c.device = integer(a[2], "device");
    if (PyErr_Occurred()) throw PythonError();
    return c;
}

void want(Py_ssize_t n, Py_ssize_t expected) {
    if (n != expected) throw Refused("wrong number of arguments");
}

template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const PythonError &) {
    } catch (const std::exception &e) {  // (c10::Error among them)
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (!t) throw PythonError();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

// ws, bytes, device, stream, i8, k, v, k_pages, v_pages, k_scales, v_scales,
// page_table, cu, kv_len, k_idx, k_idx_pages
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 16);
        const Call c = call_of(a);
        const bool i8 = a[4] == Py_True;
        const Stores s = stores(c, a + 7, i8);
        const Step p = step(c, a + 11);
        int64_t sk, sv, sx = 0;
        const at::Tensor &k = c.rows(a[5], 3, "k", sk), &v = c.rows(a[6], 3, "v", sv);
        const int64_t shape[3] = {k.size(0), s.Hkv, s.d};
        if (k.sizes() != at::IntArrayRef(shape, 3) || v.sizes() != k.sizes()) throw Refused("k and v must be [total, Hkv, d]");
        const int total = rows_of(k, "k");
        const void *x = nullptr;
        void *xp = nullptr;
        int d_idx = 0;
        if (a[14] != Py_None || a[15] != Py_None) {
            if (a[14] == Py_None || a[15] == Py_None) throw Refused("k_idx and k_idx_pages go together");
            const at::Tensor &ki = c.rows(a[14], 2, "k_idx", sx);
            const at::Tensor &kp = c.take(a[15], ScalarType::BFloat16, "k_idx_pages");
            const int64_t want_pages[3] = {s.pages, s.block, ki.size(1)};
            if (ki.size(0) != total || kp.sizes() != at::IntArrayRef(want_pages, 3))
                throw Refused("k_idx must be [total, d_idx], k_idx_pages [num_pages, block, d_idx]");
            x = ki.data_ptr();
            xp = kp.data_ptr();
            d_idx = static_cast<int>(ki.size(1));
        }
        int code = MSA_OK;
        if (total) {  // (a step without rows has nothing to write, and no pointers to check)
            c10::cuda::OptionalCUDAStreamGuard on;
            void *st = stream_of(a[3], c.device, on);
            const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
            code = i8 ? f_append_i8(k.data_ptr(), sk, v.data_ptr(), sv, x, sx, s.k.data_ptr<int8_t>(), s.v.data_ptr<int8_t>(),
                                    s.ks.data_ptr<float>(), s.vs.data_ptr<float>(), xp, p.t(), p.stride, s.pages,
                                    p.cu.const_data_ptr<int32_t>(), p.len.const_data_ptr<int32_t>(), p.Bt, total, s.Hkv, s.d,
                                    d_idx, s.block, c.ws, c.ws_bytes, st)
                      : f_append(k.data_ptr(), sk, v.data_ptr(), sv, x, sx, s.k.data_ptr(), s.v.data_ptr(), xp, p.t(), p.stride,
                                 s.pages, p.cu.const_data_ptr<int32_t>(), p.len.const_data_ptr<int32_t>(), p.Bt, total, s.Hkv,
                                 s.d, d_idx, s.block, c.ws, c.ws_bytes, st);
        }
        if (code) return PyLong_FromLong(code);
        Py_RETURN_NONE;
    });
}

// ws, bytes, device, stream, i8, total, k_pages, v_pages, k_scales, v_scales,
// page_table, cu, kv_len, k, v
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 15);
        const Call c = call_of(a);
        const bool i8 = a[4] == Py_True;
        const int total = integer(a[5], "total");
        if (total < 0) throw Refused("total must not be negative");
        const Stores s = stores(c, a + 6, i8);
        const Step p = step(c, a + 10);
        const int64_t shape[3] = {total, s.Hkv, s.d};
        c10::cuda::OptionalCUDAStreamGuard on;
        void *st = stream_of(a[3], c.device, on);
        const at::Tensor k = c.output(a[13], at::IntArrayRef(shape, 3), ScalarType::BFloat16, "k");
        const at::Tensor v = c.output(a[14], at::IntArrayRef(shape, 3), ScalarType::BFloat16, "v");
        int code = MSA_OK;
        if (total) {
            const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
            code = i8 ? f_gather_i8(s.k.const_data_ptr<int8_t>(), s.v.const_data_ptr<int8_t>(), s.ks.const_data_ptr<float>(),
                                    s.vs.const_data_ptr<float>(), p.t(), p.stride, s.pages, p.cu.const_data_ptr<int32_t>(),
                                    p.len.const_data_ptr<int32_t>(), k.data_ptr(), v.data_ptr(), p.Bt, total, s.Hkv, s.d, s.block,
                                    c.ws, c.ws_bytes, st)
                      : f_gather(s.k.data_ptr(), s.v.data_ptr(), p.t(), p.stride, s.pages, p.cu.const_data_ptr<int32_t>(),
                                 p.len.const_data_ptr<int32_t>(), k.data_ptr(), v.data_ptr(), p.Bt, total, s.Hkv, s.d, s.block,
                                 c.ws, c.ws_bytes, st);
        }
        return code ? PyLong_FromLong(code) : pair(k, v);
    });
}

// ws, bytes, device, stream, i8, q, k_pages, v_pages, k_scales, v_scales,
// page_table, cu, kv_len, window, sinks, max_q, out, lse
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 18);
        const Call c = call_of(a);
        const bool i8 = a[4] == Py_True;
        const Stores s = stores(c, a + 6, i8);
        const Step p = step(c, a + 10);
        int64_t sq;
        const at::Tensor &q = c.rows(a[5], 3, "q", sq);
        if (q.size(2) != s.d || q.size(1) > INT32_MAX) throw Refused("q must be [total, Hq, d]");
        const int total = rows_of(q, "q"), Hq = static_cast<int>(q.size(1));
        const int window = integer(a[13], "window"), sinks = integer(a[14], "sinks");
        const int max_q = a[15] == Py_None ? 0 : integer(a[15], "max_q");
        c10::cuda::OptionalCUDAStreamGuard on;
        void *st = stream_of(a[3], c.device, on);
        const at::Tensor out = c.output(a[16], q.sizes(), ScalarType::BFloat16, "out");
        const at::Tensor lse = c.output(a[17], q.sizes().slice(0, 2), ScalarType::Float, "lse");
        int code = MSA_OK;
        if (total) {
            const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
            code = i8 ? f_attn_i8(q.data_ptr(), sq, s.k.const_data_ptr<int8_t>(), s.v.const_data_ptr<int8_t>(),
                                  s.ks.const_data_ptr<float>(), s.vs.const_data_ptr<float>(), p.t(), p.stride, s.pages,
                                  p.cu.const_data_ptr<int32_t>(), p.len.const_data_ptr<int32_t>(), out.data_ptr(),
                                  lse.data_ptr<float>(), p.Bt, total, max_q, Hq, s.Hkv, s.d, s.block, window, sinks, c.ws,
                                  c.ws_bytes, st)
                      : f_attn(q.data_ptr(), sq, s.k.data_ptr(), s.v.data_ptr(), p.t(), p.stride, s.pages,
                               p.cu.const_data_ptr<int32_t>(), p.len.const_data_ptr<int32_t>(), out.data_ptr(),
                               lse.data_ptr<float>(), p.Bt, total, max_q, Hq, s.Hkv, s.d, s.block, window, sinks, c.ws,
                               c.ws_bytes, st);
        }
        return code ? PyLong_FromLong(code) : pair(out, lse);
    });
}

// ws, bytes, device, stream, q, k_pages, v_pages, k_scales, v_scales,
// page_table, T, ids, out, lse
PyObject *sparse(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 14);
        const Call c = call_of(a);
        const Stores s = stores(c, a + 5, true);
        const at::Tensor &q = c.take(a[4], ScalarType::BFloat16, "q");
        const at::Tensor &table = c.take(a[9], ScalarType::Int, "page_table");
        const at::Tensor &ids = c.take(a[11], ScalarType::Int, "ids");
        const int T = integer(a[10], "T");
        if (q.dim() != 4 || q.size(1) != 1 || q.size(3) != s.d || q.size(2) > INT32_MAX || ids.dim() != 3 ||
            ids.size(0) != q.size(0) || ids.size(1) != 1 || ids.size(2) > INT32_MAX || table.dim() != 2 ||
            table.size(0) != q.size(0) || table.size(1) > INT32_MAX)
            throw Refused("q must be [Bt, 1, Hq, d], ids [Bt, 1, K], page_table [Bt, page_stride]");
        c10::cuda::OptionalCUDAStreamGuard on;
        void *st = stream_of(a[3], c.device, on);
        const at::Tensor out = c.output(a[12], q.sizes(), ScalarType::BFloat16, "out");
        const at::Tensor lse = c.output(a[13], q.sizes().slice(0, 3), ScalarType::Float, "lse");
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(c.device)));
        const int code = f_sparse_i8(q.data_ptr(), s.k.const_data_ptr<int8_t>(), s.v.const_data_ptr<int8_t>(),
                                     s.ks.const_data_ptr<float>(), s.vs.const_data_ptr<float>(), table.const_data_ptr<int32_t>(),
                                     static_cast<int>(table.size(1)), s.pages, ids.const_data_ptr<int32_t>(), out.data_ptr(),
                                     lse.data_ptr<float>(), rows_of(q, "q"), T, static_cast<int>(q.size(2)), s.Hkv, s.d, s.block,
                                     static_cast<int>(ids.size(2)), c.ws, c.ws_bytes, st);
        return code ? PyLong_FromLong(code) : pair(out, lse);
    });
}

// Addresses of msa_kv_append, msa_kv_append_i8, msa_kv_gather,
// msa_kv_gather_i8, msa_attn_paged, msa_attn_paged_i8, msa_sparse_attn_paged_i8.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 7);
        void *p[7];
        for (int i = 0; i < 7; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (PyErr_Occurred()) throw PythonError();
            if (!p[i]) throw Refused("a null address");
        }
        f_append = reinterpret_cast<decltype(f_append)>(p[0]);
        f_append_i8 = reinterpret_cast<decltype(f_append_i8)>(p[1]);
        f_gather = reinterpret_cast<decltype(f_gather)>(p[2]);
        f_gather_i8 = reinterpret_cast<decltype(f_gather_i8)>(p[3]);
        f_attn = reinterpret_cast<decltype(f_attn)>(p[4]);
        f_attn_i8 = reinterpret_cast<decltype(f_attn_i8)>(p[5]);
        f_sparse_i8 = reinterpret_cast<decltype(f_sparse_i8)>(p[6]);
        Py_RETURN_NONE;
    });
}

#define MSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MSA_METHOD(bind), MSA_METHOD(append), MSA_METHOD(gather), MSA_METHOD(attend), MSA_METHOD(sparse),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_msa_torch", "Paged-cache calls of libmsa on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__msa_torch(void) { return PyModule_Create(&module); }
