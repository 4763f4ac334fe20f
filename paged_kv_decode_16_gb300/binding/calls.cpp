// calls.cpp -- the Python side of the calls that serve with selected pages
// (include/pagedkv.h): torch tensors checked and passed on to the C entry points.
//
// The functions of a decode step last a few microseconds, and eleven tensors' dtype,
// device, contiguity and address cost as much again when Python asks for each
// (0.25 us a tensor; here 0.03).  This module does nothing else: it has the checks of
// arguments, raises ValueError / TypeError for what the binding refuses, and returns
// the status of the library's call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits.h>

#include <exception>

#include "pagedkv.h"

namespace {

// Thrown once a Python error is set.
struct Raised {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* name) {
    PyErr_Format(type, format, name);
    throw Raised();
}

int to_int(int64_t x, const char* name) {
    if (x < INT_MIN || x > INT_MAX) refuse(PyExc_ValueError, "%s is too large", name);
    return (int)x;
}

int int_arg(PyObject* o, const char* name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    return to_int(x, name);
}

double float_arg(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return x;
}

void* address_arg(PyObject* o) {  // an int, or None
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
}

constexpr auto kI32 = at::kInt;

// The device and stream of a call, and its tensors' checks.
class Call {
public:
    // `stream`: None (the current one) or a cudaStream_t as an int.
    explicit Call(PyObject* stream)
        : device_(c10::cuda::current_device()),
          stream_(stream == Py_None
                      ? static_cast<pkv_stream>(c10::cuda::getCurrentCUDAStream(device_).stream())
                      : static_cast<pkv_stream>(address_arg(stream))) {}

    int device() const { return device_; }
    pkv_stream stream() const { return stream_; }

    // A tensor of `dtype` with `ndim` dims (-1: any) on the call's device.
    const at::Tensor& any(PyObject* o, const char* name, at::ScalarType dtype, int ndim) const {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a CUDA device", name);
        if (t.get_device() != device_) {
            PyErr_Format(PyExc_ValueError,
                         "%s is on cuda:%d but the current device is cuda:%d: call inside "
                         "torch.cuda.device(%d)",
                         name, (int)t.get_device(), device_, (int)t.get_device());
            throw Raised();
        }
        if (t.scalar_type() != dtype) {
            PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, c10::toString(dtype),
                         c10::toString(t.scalar_type()));
            throw Raised();
        }
        if (ndim >= 0 && t.dim() != ndim) {
            PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %d", name, ndim,
                         (int)t.dim());
            throw Raised();
        }
        return t;
    }
    const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType dtype, int ndim) const {
        const at::Tensor& t = any(o, name, dtype, ndim);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
        return t;
    }
    // The same with a number of elements.
    const at::Tensor& vec(PyObject* o, const char* name, at::ScalarType dtype, int64_t n) const {
        const at::Tensor& t = dense(o, name, dtype, 1);
        if (t.numel() != n) {
            PyErr_Format(PyExc_ValueError, "%s must hold %lld values, got %lld", name, (long long)n,
                         (long long)t.numel());
            throw Raised();
        }
        return t;
    }
    // The status word: an int32 tensor or None.
    uint32_t* status(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = dense(o, "dev_status", kI32, -1);
        if (t.numel() < 1) refuse(PyExc_ValueError, "%s must hold an int32", "dev_status");
        return static_cast<uint32_t*>(t.data_ptr());
    }
    // [tokens][heads][head_dim] whose heads are contiguous; *stride: between tokens.
    const at::Tensor& rows(PyObject* o, const char* name, at::ScalarType dtype, int64_t tokens,
                           int64_t heads, int64_t head_dim, int64_t* stride) const {
        const at::Tensor& t = any(o, name, dtype, 3);
        if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != head_dim) {
            PyErr_Format(PyExc_ValueError,
                         "%s must be [tokens, heads, head_dim] = [%lld, %lld, %lld], got "
                         "[%lld, %lld, %lld]",
                         name, (long long)tokens, (long long)heads, (long long)head_dim,
                         (long long)t.size(0), (long long)t.size(1), (long long)t.size(2));
            throw Raised();
        }
        if (t.numel() && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != head_dim)))
            refuse(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
        *stride = tokens > 1 ? t.stride(0) : heads * head_dim;
        return t;
    }

private:
    int device_;
    pkv_stream stream_;
};

template <typename T = int32_t>
T* ptr(const at::Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

pkv_dtype dtype_code(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kHalf) return PKV_F16;
    if (t.scalar_type() == at::kBFloat16) return PKV_BF16;
    PyErr_Format(PyExc_ValueError, "%s: dtype %s not supported (float16 or bfloat16)", name,
                 c10::toString(t.scalar_type()));
    throw Raised();
}

// A 16-bit pool and what its handle says.
struct PoolArg {
    const pkv_pool* handle;
    int num_pages, page_size, n_kv_heads, head_dim;
    at::ScalarType dtype;
    // (handle as an int, or None once destroyed; device as an int, or None: not known)
    PoolArg(PyObject* address, PyObject* device, const Call& call) {
        handle = static_cast<const pkv_pool*>(address_arg(address));
        if (!handle) refuse(PyExc_ValueError, "%s destroyed", "pool");
        pkv_dtype dt;
        kv_pool_info(handle, &num_pages, &page_size, &n_kv_heads, &head_dim, &dt);
        if (dt != PKV_F16 && dt != PKV_BF16)
            refuse(PyExc_ValueError, "%s must be a 16-bit pool (kv_pool_create)", "pool");
        dtype = dt == PKV_F16 ? at::kHalf : at::kBFloat16;
        if (device != Py_None && int_arg(device, "device") != call.device())
            refuse(PyExc_ValueError, "%s is on another device than the call", "pool");
    }
};

// The library's call without the interpreter's lock.
template <typename F>
PyObject* run(F f) {
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong((long)st);
}

PyObject* tables_build(PyObject* const* a) {
    const Call c(a[14]);
    const at::Tensor& table = c.dense(a[5], "page_table", kI32, 2);
    const int64_t B = table.size(0);
    const at::Tensor& cached = c.vec(a[0], "cached_lens", kI32, B);
    const at::Tensor& fresh = c.vec(a[1], "new_lens", kI32, B);
    const at::Tensor& free_pages = c.dense(a[2], "free_pages", kI32, 1);
    const int32_t* begin = a[3] == Py_None ? nullptr : ptr(c.vec(a[3], "free_begin", kI32, 1));
    const at::Tensor& end = c.vec(a[4], "free_end", kI32, 1);
    const int page_size = int_arg(a[6], "page_size"), num_pages = int_arg(a[7], "num_pages");
    const at::Tensor& lens = c.vec(a[8], "context_lens", kI32, B);
    const at::Tensor& starts = c.vec(a[9], "query_starts", kI32, B + 1);
    const at::Tensor& slots = c.dense(a[12], "slots", at::kLong, 1);
    const int64_t N = slots.numel();
    const at::Tensor& pos = c.vec(a[10], "positions", kI32, N);
    const at::Tensor& seq = c.vec(a[11], "seq_ids", kI32, N);
    uint32_t* status = c.status(a[13]);
    const int batch = to_int(B, "batch"), n_free = to_int(free_pages.numel(), "free_pages"),
              cols = to_int(table.size(1), "page_table"), tokens = to_int(N, "slots");
    return run([&] {
        return paged_tables_build(ptr(cached), ptr(fresh), batch, ptr(free_pages), n_free, begin,
                                  ptr(end), page_size, num_pages, ptr(table), cols, ptr(lens),
                                  ptr(starts), tokens, ptr(pos), ptr(seq), ptr<int64_t>(slots),
                                  status, c.stream());
    });
}

PyObject* append_tokens(PyObject* const* a) {
    const Call c(a[13]);
    const PoolArg p(a[0], a[1], c);
    const at::Tensor& slots = c.dense(a[4], "slots", at::kLong, 1);
    const int64_t N = slots.numel(), D = p.head_dim;
    int64_t ks = 0, vs = 0, qs = 0, os = 0, heads = 0;
    const at::Tensor& k = c.rows(a[2], "k_new", p.dtype, N, p.n_kv_heads, D, &ks);
    const at::Tensor& v = c.rows(a[3], "v_new", p.dtype, N, p.n_kv_heads, D, &vs);
    const pkv_rope* rope = static_cast<const pkv_rope*>(address_arg(a[7]));
    const int32_t* pos = nullptr;
    const void *q = nullptr, *qw = nullptr, *kw = nullptr;
    void* out = nullptr;
    const float eps = (float)float_arg(a[11]);
    if (!rope) {
        for (int i : {5, 6, 8})
            if (a[i] != Py_None)
                refuse(PyExc_ValueError, "%s need a rope", "q, q_out and positions");
        if (a[9] != Py_None || a[10] != Py_None)
            refuse(PyExc_ValueError, "%s need a rope", "the norm weights");
    } else {
        if (a[6] == Py_None) refuse(PyExc_ValueError, "%s needs positions", "a rope");
        pos = ptr(c.vec(a[6], "positions", kI32, N));
        if ((a[5] == Py_None) != (a[8] == Py_None))
            refuse(PyExc_ValueError, "give %s, or neither", "q and q_out");
        if (a[5] != Py_None) {
            heads = c.any(a[5], "q", p.dtype, 3).size(1);
            q = c.rows(a[5], "q", p.dtype, N, heads, D, &qs).data_ptr();
            out = c.rows(a[8], "q_out", p.dtype, N, heads, D, &os).data_ptr();
        } else if (a[9] != Py_None) {
            refuse(PyExc_ValueError, "%s needs q", "q_norm_weight");
        }
        if (a[9] != Py_None) qw = c.vec(a[9], "q_norm_weight", p.dtype, D).data_ptr();
        if (a[10] != Py_None) kw = c.vec(a[10], "k_norm_weight", p.dtype, D).data_ptr();
    }
    uint32_t* status = c.status(a[12]);
    const int tokens = to_int(N, "slots"), hq = to_int(heads, "q");
    return run([&] {
        return kv_append_tokens(p.handle, k.data_ptr(), ks, v.data_ptr(), vs, ptr<int64_t>(slots),
                                tokens, q, qs, hq, pos, rope, qw, kw, eps, out, os, status,
                                c.stream());
    });
}

PyObject* page_bounds(PyObject* const* a) {
    const Call c(a[5]);
    const PoolArg p(a[0], a[1], c);
    const at::Tensor& slots = c.dense(a[2], "slots", at::kLong, 1);
    const at::Tensor& bounds = c.dense(a[3], "bounds", p.dtype, 4);
    if (bounds.size(0) != p.num_pages || bounds.size(1) != p.n_kv_heads || bounds.size(2) != 2 ||
        bounds.size(3) != p.head_dim)
        refuse(PyExc_ValueError, "%s must be [num_pages, Hkv, 2, D] matching the pool", "bounds");
    uint32_t* status = c.status(a[4]);
    const int tokens = to_int(slots.numel(), "slots");
    return run([&] {
        return kv_page_bounds(p.handle, ptr<int64_t>(slots), tokens, bounds.data_ptr(), status,
                              c.stream());
    });
}

// q [B][Hq][D] of a selection or its attention, and the batch's table, lengths and lists.
struct Batch {
    const at::Tensor &q, &table, &lens, &selected;
    pkv_dtype dtype;
    int B, Hq, D, cols, heads, keep;
    static const at::Tensor& query(const Call& c, PyObject* o) {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", "q");
        const at::Tensor& t = THPVariable_Unpack(o);
        dtype_code(t, "q");
        return c.dense(o, "q", t.scalar_type(), 3);
    }
    Batch(const Call& c, PyObject* q_, PyObject* table_, PyObject* lens_, PyObject* selected_)
        : q(query(c, q_)),
          table(c.dense(table_, "page_table", kI32, 2)),
          lens(c.dense(lens_, "context_lens", kI32, 1)),
          selected(c.dense(selected_, "selected", kI32, 3)) {
        dtype = dtype_code(q, "q");
        if (table.size(0) != q.size(0) || lens.size(0) != q.size(0) ||
            selected.size(0) != q.size(0))
            refuse(PyExc_ValueError, "%s != batch", "page_table rows, context_lens or selected");
        B = to_int(q.size(0), "batch");
        Hq = to_int(q.size(1), "q");
        D = to_int(q.size(2), "q");
        cols = to_int(table.size(1), "page_table");
        heads = to_int(selected.size(1), "selected");
        keep = to_int(selected.size(2), "selected");
    }
};

PyObject* select_pages(PyObject* const* a) {
    const Call c(a[10]);
    const Batch b(c, a[0], a[2], a[3], a[5]);
    const at::Tensor& bounds = c.dense(a[1], "bounds", b.q.scalar_type(), 4);
    if (bounds.size(2) != 2 || bounds.size(3) != b.D || bounds.size(1) != b.heads)
        refuse(PyExc_ValueError,
               "%s must be [num_pages, Hkv, 2, D] and selected [B, Hkv, max_pages]", "bounds");
    const at::Tensor& ws = c.dense(a[6], "workspace", at::kByte, -1);
    const int page_size = int_arg(a[4], "page_size"), first = int_arg(a[7], "keep_first"),
              last = int_arg(a[8], "keep_last");
    uint32_t* status = c.status(a[9]);
    const int pages = to_int(bounds.size(0), "bounds");
    return run([&] {
        return paged_select_pages(b.q.data_ptr(), bounds.data_ptr(), ptr(b.table), b.cols,
                                  ptr(b.lens), b.B, b.Hq, b.heads, b.D, page_size, pages, b.dtype,
                                  first, last, b.keep, ptr(b.selected), ws.data_ptr(),
                                  (size_t)ws.numel(), status, c.stream());
    });
}

PyObject* attention_selected(PyObject* const* a) {
    const Call c(a[9]);
    const Batch b(c, a[0], a[3], a[4], a[5]);
    const at::ScalarType dt = b.q.scalar_type();
    const at::Tensor& k = c.dense(a[1], "k_pool", dt, 4);
    const at::Tensor& v = c.dense(a[2], "v_pool", dt, 4);
    const at::Tensor& out = c.dense(a[7], "out", dt, 3);
    if (k.size(3) != b.D || v.sizes() != k.sizes() || out.sizes() != b.q.sizes())
        refuse(PyExc_ValueError, "%s [B, Hq, D] and pools [NP, Hkv, P, D] disagree", "q/out");
    if (b.heads != k.size(1))
        refuse(PyExc_ValueError, "%s must be [B, Hkv, max_pages]", "selected");
    const float scale = (float)float_arg(a[6]);
    uint32_t* status = c.status(a[8]);
    const int pages = to_int(k.size(0), "k_pool"), page_size = to_int(k.size(2), "k_pool");
    return run([&] {
        return paged_decode_attention_selected(
            b.q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr(b.table), b.cols, ptr(b.lens),
            ptr(b.selected), b.keep, b.B, b.Hq, b.heads, b.D, page_size, pages, b.dtype, scale,
            out.data_ptr(), status, c.stream());
    });
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != ARGS) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
    try {
        return F(args);
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, ARGS>)),
            METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<tables_build, 15>("paged_tables_build"),
    method<append_tokens, 14>("kv_append_tokens"),
    method<page_bounds, 6>("kv_page_bounds"),
    method<select_pages, 11>("paged_select_pages"),
    method<attention_selected, 10>("paged_decode_attention_selected"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedkv_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__pagedkv_calls() { return PyModule_Create(&module); }
