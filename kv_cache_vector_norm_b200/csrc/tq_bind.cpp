// The paged-cache calls' marshalling for Python: checks of the tensors and one call of the C ABI.  A decode step's calls
// take 2 to 5 us on the GPU and pass up to ten tensors each; checked attribute by attribute in Python, a call took 8 to
// 12 us on the host, here 3 to 5.  Nothing is computed here.
//
// Every function returns the tq_status of its call, or raises TypeError (not a tensor, dtype, device) or ValueError
// (shape, layout) before it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/tq.h"

namespace {

constexpr int64_t kPage = 16;

struct Refused : std::exception {};                      // a Python error has been set

[[noreturn]] void refuse(PyObject* kind, const std::string& what) {
    PyErr_SetString(kind, what.c_str());
    throw Refused();
}

std::string list(at::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    return t;
}

// TQ_F16 or TQ_BF16 of a tensor of pages or queries.
int page_dtype(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kHalf) return TQ_F16;
    if (t.scalar_type() == at::kBFloat16) return TQ_BF16;
    refuse(PyExc_TypeError, std::string(name) + " must be float16 or bfloat16, got " + c10::toString(t.scalar_type()));
}

void same(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device device) {
    if (t.scalar_type() != type || t.device() != device)
        refuse(PyExc_TypeError, std::string(name) + " must be a " + c10::toString(type) + " tensor on " + device.str() + ", got " +
                                    c10::toString(t.scalar_type()) + " on " + t.device().str());
}

// Address of a contiguous tensor of this type, shape and device.
template <typename P>
P* need(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, c10::Device device) {
    const at::Tensor& t = tensor(o, name);
    same(t, name, type, device);
    if (t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be contiguous with shape " + list(at::IntArrayRef(shape)) + ", got " +
                                     list(t.sizes()) + (t.is_contiguous() ? "" : " (not contiguous)"));
    return static_cast<P*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}

// The stride of a dimension, or `dense` where it has one entry or none: its stride there says nothing, and may be anything.
int64_t stride(const at::Tensor& t, int64_t dim, int64_t dense) { return t.size(dim) > 1 ? t.stride(dim) : dense; }

// Sizes go through int fields: what does not fit is given as -1, which every entry point refuses.
int as_int(int64_t v) { return v >= 0 && v <= INT32_MAX ? static_cast<int>(v) : -1; }

// Runs f(stream) with the tensors' device current, on that device's current stream.
template <typename F>
PyObject* on_device(c10::Device device, F f) {
    const c10::cuda::CUDAGuard guard(device);
    return PyLong_FromLong(f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(device.index()).stream())));
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

// A workspace of the caller's, or one of the size that is needed.
struct Workspace {
    at::Tensor own;
    void* data = nullptr;
    size_t bytes = 0;
    Workspace(PyObject* given, size_t needed, c10::Device device) {
        if (given != Py_None) {
            const at::Tensor& t = tensor(given, "workspace");
            if (t.device() != device) refuse(PyExc_TypeError, "workspace must be on " + device.str());
            if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
            data = t.data_ptr();
            bytes = t.nbytes();
        } else if (needed) {
            own = at::empty({static_cast<int64_t>(needed)}, at::TensorOptions().dtype(at::kByte).device(device));
            data = own.data_ptr();
            bytes = needed;
        }
    }
};

// plan_pages(new_lens, seq_lens, block_table, free_pages, free_state, slots, row_start, start_pos, seq_lens_out,
//            free_state_out, num_kv_heads, max_tokens)
PyObject* plan_pages(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 12);
    const at::Tensor& first = cuda_tensor(v[0], "new_lens");
    const c10::Device dev = first.device();
    const int64_t b = first.numel(), heads = integer(v[10]), tokens = integer(v[11]);
    const at::Tensor &table = tensor(v[2], "block_table"), &ring = tensor(v[3], "free_pages");
    const int64_t width = table.dim() ? table.size(-1) : 0, pages = ring.numel();
    const auto i32 = at::kInt;
    tq_plan_args a = {};
    a.batch = as_int(b);
    a.num_kv_heads = as_int(heads);
    a.max_blocks = as_int(width);
    a.num_pages = as_int(pages);
    a.max_tokens = tokens;
    a.new_lens = need<int32_t>(v[0], "new_lens", i32, {b}, dev);
    a.seq_lens = need<int32_t>(v[1], "seq_lens", i32, {b}, dev);
    a.block_table = need<int32_t>(v[2], "block_table", i32, {b, width}, dev);
    a.free_pages = need<int32_t>(v[3], "free_pages", i32, {pages}, dev);
    a.free_state = need<int32_t>(v[4], "free_state", i32, {2}, dev);
    a.slots = need<int64_t>(v[5], "slots", at::kLong, {tokens * heads}, dev);
    a.row_start = need<int32_t>(v[6], "row_start", i32, {b + 1}, dev);
    a.start_pos = need<int32_t>(v[7], "start_pos", i32, {b}, dev);
    a.seq_lens_out = need<int32_t>(v[8], "seq_lens_out", i32, {b}, dev);
    a.free_state_out = need<int32_t>(v[9], "free_state_out", i32, {2}, dev);
    return on_device(dev, [&](void* st) { return tq_plan_pages(&a, st); });
}

// append_pages(k, v, slots, k_pool, v_pool, bounds): None where there is none
PyObject* append_pages(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 6);
    const at::Tensor& k = cuda_tensor(v[0], "k");
    tq_append_args a = {};
    a.dtype = page_dtype(k, "k");
    const c10::Device dev = k.device();
    if (k.dim() != 3 || k.stride(2) != 1) refuse(PyExc_ValueError, "k must be [N, H_kv, d] with unit stride along d");
    const int64_t rows = k.size(0), heads = k.size(1), d = k.size(2);
    PyObject* some = v[3] != Py_None ? v[3] : v[4] != Py_None ? v[4] : v[5];
    if (some == Py_None) refuse(PyExc_ValueError, "append_pages needs k_pool, v_pool or bounds");
    const at::Tensor& pool = tensor(some, "the pool");
    const int64_t pages = pool.dim() ? pool.size(0) : 0;
    a.head_dim = as_int(d);
    a.num_kv_heads = as_int(heads);
    a.num_pages = as_int(pages);
    a.num_tokens = rows;
    a.k = k.data_ptr();
    a.k_token_stride = stride(k, 0, heads * d);
    a.k_head_stride = stride(k, 1, d);
    if (v[1] != Py_None) {
        const at::Tensor& t = tensor(v[1], "v");
        same(t, "v", k.scalar_type(), dev);
        if (t.sizes() != k.sizes() || t.stride(2) != 1) refuse(PyExc_ValueError, "v must be [N, H_kv, d] like k, with unit stride along d");
        a.v = t.data_ptr();
        a.v_token_stride = stride(t, 0, heads * d);
        a.v_head_stride = stride(t, 1, d);
    } else if (v[4] != Py_None) {
        refuse(PyExc_ValueError, "v_pool needs v");
    }
    a.slots = need<int64_t>(v[2], "slots", at::kLong, {rows * heads}, dev);
    if (v[3] != Py_None) a.k_pool = need<void>(v[3], "k_pool", k.scalar_type(), {pages, heads, kPage, d}, dev);
    if (v[4] != Py_None) a.v_pool = need<void>(v[4], "v_pool", k.scalar_type(), {pages, heads, kPage, d}, dev);
    if (v[5] != Py_None) a.bounds = need<void>(v[5], "bounds", k.scalar_type(), {pages, heads, 2, d}, dev);
    return on_device(dev, [&](void* st) { return tq_append_pages(&a, st); });
}

// A query [B, H_q, d] whose sequences may lie apart.
const at::Tensor& query(PyObject* o) {
    const at::Tensor& q = cuda_tensor(o, "q");
    page_dtype(q, "q");
    if (q.dim() != 3 || q.stride(2) != 1 || stride(q, 1, q.size(2)) != q.size(2))
        refuse(PyExc_ValueError, "q must be [B, H_q, d] with contiguous heads");
    return q;
}

// select_pages(q, bounds, block_table, seq_lens, pages, lens, workspace or None, budget, keep_first, keep_last)
PyObject* select_pages(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 10);
    const at::Tensor& q = query(v[0]);
    const c10::Device dev = q.device();
    const at::Tensor &bounds = tensor(v[1], "bounds"), &table = tensor(v[2], "block_table");
    if (bounds.dim() != 4) refuse(PyExc_ValueError, "bounds must be [num_pages, H_kv, 2, d]");
    const int64_t b = q.size(0), d = q.size(2), pages = bounds.size(0), heads = bounds.size(1);
    const int64_t width = table.dim() ? table.size(-1) : 0, budget = integer(v[7]);
    tq_select_args a = {};
    a.dtype = page_dtype(q, "q");
    a.batch = as_int(b);
    a.num_q_heads = as_int(q.size(1));
    a.num_kv_heads = as_int(heads);
    a.head_dim = as_int(d);
    a.max_blocks = as_int(width);
    a.num_pages = as_int(pages);
    a.budget = as_int(budget);
    a.keep_first = as_int(integer(v[8]));
    a.keep_last = as_int(integer(v[9]));
    a.q = q.data_ptr();
    a.q_stride = stride(q, 0, q.size(1) * d);
    a.bounds = need<void>(v[1], "bounds", q.scalar_type(), {pages, heads, 2, d}, dev);
    a.block_table = need<int32_t>(v[2], "block_table", at::kInt, {b, width}, dev);
    a.seq_lens = need<int32_t>(v[3], "seq_lens", at::kInt, {b}, dev);
    a.pages = need<int32_t>(v[4], "pages", at::kInt, {b, heads, budget}, dev);
    a.lens = need<int32_t>(v[5], "lens", at::kInt, {b, heads}, dev);
    return on_device(dev, [&](void* st) {
        size_t bytes = 0;
        if (v[6] == Py_None) {
            const tq_status s = tq_select_pages_workspace_bytes(&a, &bytes);
            if (s != TQ_OK) return s;
        }
        const Workspace w(v[6], bytes, dev);
        a.workspace = w.data;
        a.workspace_bytes = w.bytes;
        return tq_select_pages(&a, st);
    });
}

// attend_pages(q, k_pool, v_pool, block_table, seq_lens, out, workspace or None, scale)
PyObject* attend_pages(PyObject* const* v, Py_ssize_t n) {
    arguments(n, 8);
    const at::Tensor& q = query(v[0]);
    const c10::Device dev = q.device();
    const at::Tensor &kp = tensor(v[1], "k_pool"), &vp = tensor(v[2], "v_pool"), &table = tensor(v[3], "block_table");
    const int64_t b = q.size(0), hq = q.size(1), d = q.size(2);
    if (kp.dim() != 4) refuse(PyExc_ValueError, "k_pool must be [num_pages, H_kv, 16, d]");
    const int64_t pages = kp.size(0), heads = kp.size(1), width = table.dim() ? table.size(-1) : 0;
    const std::initializer_list<int64_t> shape = {pages, heads, kPage, d};
    auto pool = [&](const at::Tensor& t, const char* name) {         // each page contiguous, pages may lie apart
        same(t, name, q.scalar_type(), dev);
        if (t.sizes() != at::IntArrayRef(shape) || t.stride(3) != 1 || t.stride(2) != d || stride(t, 1, kPage * d) != kPage * d)
            refuse(PyExc_ValueError, std::string(name) + " must be " + list(at::IntArrayRef(shape)) + ", each page contiguous; got " +
                                         list(t.sizes()) + ", strides " + list(t.strides()));
        return t.data_ptr();
    };
    tq_attend_pages_args a = {};
    a.dtype = page_dtype(q, "q");
    a.batch = as_int(b);
    a.num_q_heads = as_int(hq);
    a.num_kv_heads = as_int(heads);
    a.head_dim = as_int(d);
    a.max_blocks = as_int(width);
    a.num_pages = as_int(pages);
    a.selected = table.dim() == 3;
    a.scale = static_cast<float>(PyFloat_AsDouble(v[7]));
    if (PyErr_Occurred()) throw Refused();
    a.q = q.data_ptr();
    a.q_stride = stride(q, 0, q.size(1) * d);
    a.k_pool = pool(kp, "k_pool");
    a.v_pool = pool(vp, "v_pool");
    a.k_page_stride = stride(kp, 0, heads * kPage * d);
    a.v_page_stride = stride(vp, 0, heads * kPage * d);
    if (a.selected) {
        a.block_table = need<int32_t>(v[3], "block_table", at::kInt, {b, heads, width}, dev);
        a.seq_lens = need<int32_t>(v[4], "seq_lens", at::kInt, {b, heads}, dev);
    } else {
        a.block_table = need<int32_t>(v[3], "block_table", at::kInt, {b, width}, dev);
        a.seq_lens = need<int32_t>(v[4], "seq_lens", at::kInt, {b}, dev);
    }
    a.out = need<float>(v[5], "out", at::kFloat, {b, hq, d}, dev);
    return on_device(dev, [&](void* st) {
        size_t bytes = 0;
        if (v[6] == Py_None) {
            const tq_status s = tq_attend_pages_workspace_bytes(&a, &bytes);
            if (s != TQ_OK) return s;
        }
        const Workspace w(v[6], bytes, dev);
        a.workspace = w.data;
        a.workspace_bytes = w.bytes;
        return tq_attend_pages(&a, st);
    });
}

// No C++ exception leaves a Python entry.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(args, n);
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<plan_pages>("plan_pages"), method<append_pages>("append_pages"), method<select_pages>("select_pages"),
                         method<attend_pages>("attend_pages"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Marshalling of the paged-cache calls of libtq.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
