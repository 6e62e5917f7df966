// Python binding of the bounded-cache calls of include/qsa.h (argument checks,
// outputs, pointers and the current stream; no computation). These calls take
// 10 to 20 us on the GPU at serving sizes, so what the host does before each of
// them counts: measured on the GB300's Arm host, a call of decode attention
// took 24 us through ctypes with its checks in Python and takes 7.4 us here, 4.5 where outputs and
// scratch are given.
//
// Each function takes all its arguments by position and returns its tensors,
// or the status as an int when the library refused the call; a bad argument
// raises ValueError.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/qsa.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
// A Python error is set already.
struct PythonError {};

[[noreturn]] __attribute__((format(printf, 1, 2))) void refuse(const char *format, ...) {
    char text[512];
    va_list args;
    va_start(args, format);
    vsnprintf(text, sizeof(text), format, args);
    va_end(args);
    throw Refused(text);
}

const Tensor &cuda_tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a CUDA tensor", name);
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    return t;
}

// A CUDA tensor on device `index` of one of the types and `dims` dimensions, contiguous in its last.
const Tensor &checked(PyObject *o, const char *name, std::initializer_list<ScalarType> types, int64_t dims, int index) {
    const Tensor &t = cuda_tensor(o, name);
    if (t.get_device() != index)
        refuse("%s must be on cuda:%d, is on cuda:%d", name, index, static_cast<int>(t.get_device()));
    bool good = false;
    for (ScalarType s : types) good = good || t.scalar_type() == s;
    if (!good) {
        std::string wanted;
        for (ScalarType s : types) wanted += (wanted.empty() ? "" : " or ") + std::string(c10::toString(s));
        refuse("%s must be %s, got %s", name, wanted.c_str(), c10::toString(t.scalar_type()));
    }
    if (t.dim() != dims || (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1))
        refuse("%s must be a %d-d tensor, contiguous in its last dimension", name, static_cast<int>(dims));
    return t;
}

// A stride; 0 for a dimension of one element, whose stride is arbitrary.
int64_t stride(const Tensor &t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }
int64_t row_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

int number(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    if (v < INT_MIN || v > INT_MAX) refuse("%s is out of range", name);
    return static_cast<int>(v);
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return static_cast<float>(v);
}
int size32(int64_t n, const char *name) {
    if (n > INT_MAX) refuse("%s is too large", name);
    return static_cast<int>(n);
}

qsa_dtype kind(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return QSA_F32;
        case at::kHalf: return QSA_F16;
        case at::kBFloat16: return QSA_BF16;
        default: return QSA_I8;
    }
}

// `o` checked as a contiguous output of that shape and type, or a new one.
Tensor made(PyObject *o, const char *name, at::IntArrayRef shape, ScalarType type, int index) {
    if (o == Py_None)   // past the dispatcher: decode attention's outputs and scratch 2.9 us, by at::empty 4.3
        return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt));
    const Tensor &t = checked(o, name, {type}, static_cast<int64_t>(shape.size()), index);
    if (t.sizes() != shape || !t.is_contiguous()) refuse("%s must be contiguous, of the result's shape", name);
    return t;
}

// The scratch a user gave, or memory of torch's allocator, which goes back to it (for
// later work on this stream) when the call has queued its kernels.
struct Scratch {
    void *ptr = nullptr;
    size_t bytes = 0;
    c10::DataPtr own;
};
Scratch scratch_of(PyObject *o, size_t need, int index) {
    Scratch r;
    if (o == Py_None) {
        if (need == 0) return r;
        r.own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
        r.ptr = r.own.get();
        r.bytes = need;
        return r;
    }
    const Tensor &t = checked(o, "scratch", {at::kByte}, 1, index);
    if (static_cast<size_t>(t.numel()) < need) refuse("scratch must have at least %zu bytes", need);
    r.ptr = t.data_ptr();
    r.bytes = static_cast<size_t>(t.numel());
    return r;
}

qsa_kv_pages pages(PyObject *k_pages, PyObject *v_pages, PyObject *k_scale, PyObject *v_scale, int index) {
    const Tensor &k = checked(k_pages, "k_pages", {at::kBFloat16, at::kHalf, at::kChar}, 4, index);
    const Tensor &v = checked(v_pages, "v_pages", {k.scalar_type()}, 4, index);
    if (k.size(3) != QSA_D || v.sizes() != k.sizes() || stride(v, 0) != stride(k, 0) || stride(v, 1) != stride(k, 1) ||
        stride(v, 2) != stride(k, 2))
        refuse("k_pages and v_pages must both be [npages, page_size, nkv, 128], of the same strides");
    qsa_kv_pages kv = {};
    kv.k = k.data_ptr();
    kv.v = v.data_ptr();
    kv.dtype = kind(k);
    kv.npages = size32(k.size(0), "npages");
    kv.page_size = size32(k.size(1), "page_size");
    kv.nkv = size32(k.size(2), "nkv");
    kv.page_stride = stride(k, 0);
    kv.cell_stride = stride(k, 1);
    kv.head_stride = stride(k, 2);
    if (kv.dtype != QSA_I8) {
        if (k_scale != Py_None || v_scale != Py_None) refuse("scales are for int8 pages only");
        return kv;
    }
    const Tensor *scales[2];
    PyObject *given[2] = {k_scale, v_scale};
    for (int i = 0; i < 2; ++i) {
        const char *name = i == 0 ? "k_scale_f16" : "v_scale_f16";
        const Tensor &t = cuda_tensor(given[i], name);
        if (t.get_device() != index || t.element_size() != 2 || t.dim() != 3 || t.size(0) != k.size(0) ||
            t.size(1) != k.size(1) || t.size(2) != k.size(2))
            refuse("%s must be [npages, page_size, nkv] binary16 values beside int8 pages", name);
        scales[i] = &t;
    }
    for (int64_t d = 0; d < 3; ++d)
        if (stride(*scales[0], d) != stride(*scales[1], d)) refuse("k_scale_f16 and v_scale_f16 must have the same strides");
    kv.k_scale_f16 = static_cast<uint16_t *>(scales[0]->data_ptr());
    kv.v_scale_f16 = static_cast<uint16_t *>(scales[1]->data_ptr());
    kv.scale_page_stride = stride(*scales[0], 0);
    kv.scale_cell_stride = stride(*scales[0], 1);
    kv.scale_head_stride = stride(*scales[0], 2);
    return kv;
}

cudaStream_t current_stream(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

PyObject *tuple(std::initializer_list<Tensor> tensors) {
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    if (r == nullptr) throw PythonError();
    Py_ssize_t i = 0;
    for (const Tensor &t : tensors) {
        PyObject *o = THPVariable_Wrap(t);
        if (o == nullptr) {
            Py_DECREF(r);
            throw PythonError();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Runs `body`, turning what it throws into Python errors.
template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
        return nullptr;
    }
    try {
        return body();
    } catch (const PythonError &) {
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {   // torch's own errors, running out of memory among them
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// q, k_pages, v_pages, page_table, lens, k_scale, v_scale, window, sinks, scale, mass, mass_out, out, lse, scratch
PyObject *paged_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const int index = static_cast<int>(cuda_tensor(a[1], "k_pages").get_device());
        const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(index));
        const qsa_kv_pages kv = pages(a[1], a[2], a[5], a[6], index);
        const ScalarType cells = THPVariable_Unpack(a[1]).scalar_type();
        const Tensor &q = cells == at::kChar ? checked(a[0], "q", {at::kFloat, at::kHalf, at::kBFloat16}, 3, index)
                                             : checked(a[0], "q", {cells}, 3, index);
        const int nseq = size32(q.size(0), "nseq"), nheads = size32(q.size(1), "nheads");
        if (q.size(2) != QSA_D || nheads < 1 || kv.nkv < 1 || nheads % kv.nkv != 0)
            refuse("q must be [nseq, a multiple of %d, %d]", kv.nkv, QSA_D);
        const Tensor &table = checked(a[3], "page_table", {at::kInt}, 2, index), &lens = checked(a[4], "lens", {at::kInt}, 1, index);
        if (lens.size(0) != table.size(0)) refuse("page_table and lens must have one row per sequence");
        if (table.size(0) != nseq) refuse("page_table must have one row per query");
        const int cols = size32(table.size(1), "page_table's width");
        const int64_t capacity = static_cast<int64_t>(cols) * kv.page_size;
        const float *mass = nullptr;
        float *mass_out = nullptr;
        int64_t mass_stride = 0;
        if (a[10] != Py_None) {
            PyObject *into = a[11] == Py_None ? a[10] : a[11];
            const Tensor &m = checked(a[10], "mass", {at::kFloat}, 2, index), &o = checked(into, "mass_out", {at::kFloat}, 2, index);
            if (m.size(0) != nseq || m.size(1) < capacity || o.size(0) != nseq || o.size(1) < capacity)
                refuse("mass and mass_out must be [%d, >= %lld]", nseq, static_cast<long long>(capacity));
            if (stride(m, 0) != stride(o, 0)) refuse("mass and mass_out must have the same strides");
            mass = m.data_ptr<float>();
            mass_out = o.data_ptr<float>();
            mass_stride = nseq > 1 ? m.stride(0) : std::max(m.size(1), o.size(1));
        } else if (a[11] != Py_None) {
            refuse("mass_out needs mass");
        }
        const int window = number(a[7], "window"), sinks = number(a[8], "sinks");
        const float scale = real(a[9]);
        const Tensor out = made(a[12], "out", {nseq, nheads, QSA_D}, q.scalar_type(), index);
        const Tensor lse = made(a[13], "lse", {nseq, nheads}, at::kFloat, index);
        const size_t need = qsa_paged_attn_scratch_bytes(nseq, nheads, kv.nkv, cols, kv.page_size, mass != nullptr);
        const Scratch scratch = scratch_of(a[14], need, index);
        const qsa_status status = qsa_paged_attn(
            q.data_ptr(), kind(q), stride(q, 0), stride(q, 1), nseq, nheads, &kv, table.data_ptr<int32_t>(), cols,
            row_stride(table), lens.data_ptr<int32_t>(), window, sinks, scale, out.data_ptr(), lse.data_ptr<float>(), mass,
            mass_out, mass_stride, scratch.ptr, scratch.bytes, current_stream(index));
        return status == QSA_OK ? tuple({out, lse}) : PyLong_FromLong(status);
    });
}

// q, k, v, cu_q, cu_k, max_q, window, sinks, scale, out, lse, scratch
PyObject *window_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const int index = static_cast<int>(cuda_tensor(a[0], "q").get_device());
        const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(index));
        const Tensor &q = checked(a[0], "q", {at::kBFloat16, at::kHalf}, 3, index);
        const Tensor &k = checked(a[1], "k", {q.scalar_type()}, 3, index), &v = checked(a[2], "v", {q.scalar_type()}, 3, index);
        const int total_q = size32(q.size(0), "total_q"), nheads = size32(q.size(1), "nheads");
        const int total_k = size32(k.size(0), "total_k"), nkv = size32(k.size(1), "nkv");
        if (q.size(2) != QSA_D || k.size(2) != QSA_D || v.sizes() != k.sizes() || nkv < 1 || nheads < 1 || nheads % nkv != 0)
            refuse("q must be [total_q, nheads, 128] and k, v [total_k, nkv, 128] with nheads a multiple of nkv");
        const Tensor &cu_q = checked(a[3], "cu_q", {at::kInt}, 1, index), &cu_k = checked(a[4], "cu_k", {at::kInt}, 1, index);
        if (cu_q.size(0) < 1 || cu_q.size(0) != cu_k.size(0))
            refuse("cu_q and cu_k must both have one more element than there are sequences");
        const int nseq = size32(cu_q.size(0) - 1, "nseq");
        int max_q = number(a[5], "max_q");
        if (max_q < 0) refuse("max_q must not be negative");
        max_q = std::min(max_q, total_q);
        const int window = number(a[6], "window"), sinks = number(a[7], "sinks");
        const float scale = real(a[8]);
        const Tensor out = made(a[9], "out", {total_q, nheads, QSA_D}, q.scalar_type(), index);
        const Tensor lse = made(a[10], "lse", {total_q, nheads}, at::kFloat, index);
        const Scratch scratch = scratch_of(a[11], qsa_window_attn_scratch_bytes(nseq, total_q, max_q, nheads, nkv), index);
        const int64_t strides[6] = {stride(q, 0), stride(q, 1), stride(k, 0), stride(k, 1), stride(v, 0), stride(v, 1)};
        const qsa_status status = qsa_window_attn(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), kind(q), strides, cu_q.data_ptr<int32_t>(), cu_k.data_ptr<int32_t>(),
            nseq, total_q, total_k, max_q, nheads, nkv, window, sinks, scale, out.data_ptr(), lse.data_ptr<float>(),
            scratch.ptr, scratch.bytes, current_stream(index));
        return status == QSA_OK ? tuple({out, lse}) : PyLong_FromLong(status);
    });
}

// k_pages, v_pages, page_table, lens, mass, new_table, budget, sinks, recent, k_scale, v_scale, kept, new_lens, new_mass
PyObject *cache_evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        const int index = static_cast<int>(cuda_tensor(a[0], "k_pages").get_device());
        const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(index));
        const qsa_kv_pages kv = pages(a[0], a[1], a[9], a[10], index);
        const Tensor &table = checked(a[2], "page_table", {at::kInt}, 2, index), &lens = checked(a[3], "lens", {at::kInt}, 1, index);
        if (lens.size(0) != table.size(0)) refuse("page_table and lens must have one row per sequence");
        const int nseq = size32(table.size(0), "nseq"), cols = size32(table.size(1), "page_table's width");
        const Tensor &mass = checked(a[4], "mass", {at::kFloat}, 2, index);
        const Tensor &new_table = checked(a[5], "new_table", {at::kInt}, 2, index);
        if (new_table.size(0) != nseq) refuse("new_table must have one row per sequence");
        const int new_cols = size32(new_table.size(1), "new_table's width");
        const int64_t capacity = static_cast<int64_t>(cols) * kv.page_size, room = static_cast<int64_t>(new_cols) * kv.page_size;
        if (mass.size(0) != nseq || mass.size(1) < capacity)
            refuse("mass must be [%d, >= %lld]", nseq, static_cast<long long>(capacity));
        const int budget = number(a[6], "budget"), sinks = number(a[7], "sinks"), recent = number(a[8], "recent");
        if (budget < 1 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget || budget > room)
            refuse("budget must be at least 1 and sinks + recent, and fit the new table's pages");
        const Tensor kept = made(a[11], "kept", {nseq, budget}, at::kInt, index);
        const Tensor new_lens = made(a[12], "new_lens", {nseq}, at::kInt, index);
        const Tensor new_mass = a[13] == Py_None ? made(Py_None, "new_mass", {nseq, room}, at::kFloat, index)
                                                 : checked(a[13], "new_mass", {at::kFloat}, 2, index);
        if (new_mass.size(0) != nseq || new_mass.size(1) < budget) refuse("new_mass must be [%d, >= %d]", nseq, budget);
        const qsa_status status = qsa_cache_evict(
            &kv, nseq, table.data_ptr<int32_t>(), cols, row_stride(table), lens.data_ptr<int32_t>(), mass.data_ptr<float>(),
            row_stride(mass), new_table.data_ptr<int32_t>(), new_cols, row_stride(new_table), budget, sinks, recent,
            kept.data_ptr<int32_t>(), new_lens.data_ptr<int32_t>(), new_mass.data_ptr<float>(), row_stride(new_mass),
            size32(new_mass.size(1), "new_mass"), current_stream(index));
        return status == QSA_OK ? tuple({kept, new_lens, new_mass}) : PyLong_FromLong(status);
    });
}

PyMethodDef methods[] = {
    {"paged_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attn)), METH_FASTCALL, nullptr},
    {"window_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(window_attn)), METH_FASTCALL, nullptr},
    {"cache_evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qsa_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qsa_ops() { return PyModule_Create(&module); }
