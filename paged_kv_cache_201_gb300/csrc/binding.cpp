// The short way of the Python binding into the 4-bit cache's and the page calls: checks of the tensors, their pointers,
// the current stream and the call, in one step.
//
// These calls take a few microseconds on the GPU and up to eleven tensors.  Checked and marshalled in Python, a call costs the
// host 7 to 10 us; from here 2 to 3, most of it the launch.  A function returns the call's status, or None where
// anything about an argument is not as it should be: the caller then goes the long way, which says what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "paged_attn.h"

namespace {

constexpr auto kInt = at::kInt;

struct Refused {};  // an argument is not as it should be

// The interpreter is others' while a call is made: a launch waits where the stream's queue is full.  Every argument is read
// before.  It costs a call 0.1 us (two calls over 261 rows 4.5 -> 4.7 us).
struct WithoutInterpreter {
    PyThreadState *const state = PyEval_SaveThread();
    ~WithoutInterpreter() { PyEval_RestoreThread(state); }
};

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o)) throw Refused{};
    return THPVariable_Unpack(o);
}

int int_of(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) throw Refused{};
    return (int)v;
}

// The device of t, which must be the current one.
int this_device(const at::Tensor &t) {
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device()) throw Refused{};
    return (int)t.get_device();
}

void *dense(const at::Tensor &t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
        throw Refused{};
    return t.data_ptr();
}
int32_t *ints(PyObject *o, int dev, at::IntArrayRef shape) { return static_cast<int32_t *>(dense(tensor(o), dev, kInt, shape)); }
int32_t *ints_or_null(PyObject *o, int dev, at::IntArrayRef shape) { return o == Py_None ? nullptr : ints(o, dev, shape); }

int type_code(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return PA_F32;
        case at::kHalf: return PA_F16;
        case at::kBFloat16: return PA_BF16;
        default: throw Refused{};
    }
}

// A stream's handle, or None: the current one.
void *stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void *s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw Refused{};
    return s;
}

// Elements between the tokens of [tokens, heads, head_dim] rows with dense heads; 0: dense, whatever a stride that nothing uses
// says.
int64_t token_stride(const at::Tensor &t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != shape) throw Refused{};
    if (t.is_contiguous()) return 0;
    if (t.stride(2) != 1 || t.stride(1) != shape[2] || t.stride(0) < shape[1] * shape[2]) throw Refused{};
    return t.stride(0);
}

// Page size of a 4-bit pool.
int page_size(const at::Tensor &kv, int64_t D) {
    if (kv.dim() != 3 || D <= 0 || kv.size(2) * 8 % (9 * D) != 0) throw Refused{};
    const int64_t ps = kv.size(2) * 8 / (9 * D);
    if (ps != 16 && ps != 32 && ps != 64) throw Refused{};
    return (int)ps;
}

void in_range(std::initializer_list<int64_t> sizes) {
    for (int64_t s : sizes)
        if (s > INT32_MAX) throw Refused{};
}

pa_dims dims_of(int64_t batch, int64_t q_len, int64_t Hq, int64_t Hkv, int64_t D, int ps, int64_t pages, int64_t width, int dtype,
                int64_t stride) {
    in_range({batch, q_len, Hq, Hkv, D, width});
    return {(int32_t)batch, (int32_t)q_len, (int32_t)Hq, (int32_t)Hkv, (int32_t)D, ps, pages, (int32_t)width, dtype, stride};
}

int multiprocessors(int dev) {
    static int count[128];  // the same value whoever writes it
    if (dev < 0 || dev >= 128) throw Refused{};
    if (!count[dev] && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) throw Refused{};
    return count[dev];
}

// append_kv4(k_new, v_new, slots, kv, stream)
int append_kv4(PyObject *const *a) {
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &kv = tensor(a[3]);
    if (k.dim() != 3) throw Refused{};
    const int dev = this_device(k);
    const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
    const int ps = page_size(kv, D);
    void *pool = dense(kv, dev, at::kByte, {kv.size(0), Hkv, kv.size(2)});
    const int32_t *slots = ints(a[2], dev, {T});
    const int64_t ks = token_stride(k, dev, k.scalar_type(), {T, Hkv, D}), vs = token_stride(v, dev, k.scalar_type(), {T, Hkv, D});
    const pa_dims d = dims_of(1, T, Hkv, Hkv, D, ps, kv.size(0), 0, type_code(k), 0);
    const void *kp = k.data_ptr(), *vp = v.data_ptr();
    void *stream = stream_of(a[4], dev);
    const WithoutInterpreter others;
    return paged_attn_append_kv4(kp, vp, slots, ks, vs, pool, &d, stream);
}

// gather_kv4(kv, slots, k_out, v_out, stream)
int gather_kv4(PyObject *const *a) {
    const at::Tensor &kv = tensor(a[0]), &k = tensor(a[2]);
    if (k.dim() != 3) throw Refused{};
    const int dev = this_device(k);
    const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
    const int ps = page_size(kv, D);
    const void *pool = dense(kv, dev, at::kByte, {kv.size(0), Hkv, kv.size(2)});
    const int32_t *slots = ints(a[1], dev, {T});
    void *ko = dense(k, dev, k.scalar_type(), {T, Hkv, D}), *vo = dense(tensor(a[3]), dev, k.scalar_type(), {T, Hkv, D});
    const pa_dims d = dims_of(1, T, Hkv, Hkv, D, ps, kv.size(0), 0, type_code(k), 0);
    void *stream = stream_of(a[4], dev);
    const WithoutInterpreter others;
    return paged_attn_gather_kv4(pool, slots, ko, vo, &d, stream);
}

// fwd_kv4(q, kv, block_table, seq_lens, causal, q_offset, scale, out, lse, q_start, stream, workspace)
int fwd_kv4(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0]), &kv = tensor(a[1]), &table = tensor(a[2]);
    const bool packed = a[9] != Py_None;
    if (table.dim() != 2 || q.dim() != (packed ? 3 : 4) || kv.dim() != 3) throw Refused{};
    const int dev = this_device(q), lead = (int)q.dim() - 2;
    const int64_t B = table.size(0), W = table.size(1), Hq = q.size(-2), D = q.size(-1), Sq = q.size(lead - 1), Hkv = kv.size(1);
    const int ps = page_size(kv, D);
    if (!packed && q.size(0) != B) throw Refused{};
    const void *pool = dense(kv, dev, at::kByte, kv.sizes());
    const int32_t *bt = ints(a[2], dev, {B, W}), *lens = ints(a[3], dev, {B}), *qo = ints_or_null(a[5], dev, {B}),
                  *qs = ints_or_null(a[9], dev, {B + 1});
    int64_t stride = 0;
    if (!q.is_contiguous()) {
        if (!packed) throw Refused{};
        stride = token_stride(q, dev, q.scalar_type(), q.sizes());
    }
    void *out = dense(tensor(a[7]), dev, q.scalar_type(), q.sizes());
    void *lse = a[8] == Py_None ? nullptr : dense(tensor(a[8]), dev, at::kFloat, q.sizes().slice(0, (size_t)lead + 1));
    const double scale = PyFloat_AsDouble(a[6]);
    const int causal = PyObject_IsTrue(a[4]);
    if (PyErr_Occurred() || causal < 0) throw Refused{};
    const pa_dims d = dims_of(B, Sq, Hq, Hkv, D, ps, kv.size(0), W, type_code(q), stride);
    at::Tensor own;
    void *ws = nullptr;
    int64_t size = 0;
    if (a[11] != Py_None) {
        const at::Tensor &given = tensor(a[11]);
        ws = dense(given, dev, at::kByte, given.sizes());
        size = given.numel();
    } else if ((size = paged_attn_kv4_workspace_bytes(&d, packed, multiprocessors(dev))) > 0) {
        if (a[10] != Py_None) throw Refused{};  // on another stream: the long way tells the allocator
        own = at::empty({size}, q.options().dtype(at::kByte));
        ws = own.data_ptr();
    } else {
        size = 0;  // none, or a shape that the call refuses
    }
    const void *qp = q.data_ptr();
    void *stream = stream_of(a[10], dev);
    const WithoutInterpreter others;
    return paged_attn_fwd_kv4(qp, pool, bt, lens, qs, causal, qo, (float)scale, out, static_cast<float *>(lse), &d, ws, size, stream);
}

// What the page calls take: block_table, seq_lens, page_shares, free_pages, free_count.
struct Pages {
    int dev;
    int64_t B, W, F, P;
    int32_t *table, *lens, *shares, *free, *count;
    Pages(PyObject *bt, PyObject *sl, PyObject *sh, PyObject *fp, PyObject *fc) {
        const at::Tensor &t = tensor(bt), &s = tensor(sh), &f = tensor(fp);
        if (t.dim() != 2 || s.dim() != 1 || f.dim() != 1) throw Refused{};
        dev = this_device(t);
        B = t.size(0), W = t.size(1), F = f.size(0), P = s.size(0);
        in_range({B, W, F});
        table = ints(bt, dev, {B, W});
        lens = ints(sl, dev, {B});
        shares = ints(sh, dev, {P});
        free = ints(fp, dev, {F});
        count = ints(fc, dev, {1});
    }
};

int64_t length(PyObject *o) {
    const at::Tensor &t = tensor(o);
    if (t.dim() != 1 || t.size(0) > INT32_MAX) throw Refused{};
    return t.size(0);
}

// fork(parents, children, block_table, seq_lens, lens_out, page_shares, free_pages, free_count, free_left, copies, page_size,
//      prefix_lens, stream)
int fork_rows(PyObject *const *a) {
    const Pages p(a[2], a[3], a[5], a[6], a[7]);
    const int64_t n = length(a[0]);
    const int32_t *parents = ints(a[0], p.dev, {n}), *children = ints(a[1], p.dev, {n}), *prefixes = ints_or_null(a[11], p.dev, {n});
    int32_t *lens_out = ints(a[4], p.dev, {p.B}), *left = ints(a[8], p.dev, {1}), *copies = ints(a[9], p.dev, {n, 2});
    const int ps = int_of(a[10]);
    void *stream = stream_of(a[12], p.dev);
    const WithoutInterpreter others;
    return paged_attn_fork(parents, children, prefixes, (int)n, p.table, p.lens, lens_out, p.shares, p.free, (int)p.F, p.count, left,
                           copies, (int)p.B, ps, p.P, (int)p.W, stream);
}

// free(rows, block_table, seq_lens, lens_out, page_shares, free_pages, free_count, free_left, page_size, stream)
int free_rows(PyObject *const *a) {
    const Pages p(a[1], a[2], a[4], a[5], a[6]);
    const int64_t n = length(a[0]);
    const int32_t *rows = ints(a[0], p.dev, {n});
    int32_t *lens_out = ints(a[3], p.dev, {p.B}), *left = ints(a[7], p.dev, {1});
    const int ps = int_of(a[8]);
    void *stream = stream_of(a[9], p.dev);
    const WithoutInterpreter others;
    return paged_attn_free(rows, (int)n, p.table, p.lens, lens_out, p.shares, p.free, (int)p.F, p.count, left, (int)p.B, ps, p.P,
                           (int)p.W, stream);
}

// compact(block_table, seq_lens, page_shares, free_pages, free_count, moves, n_moves, page_map, page_size, stream)
int compact_rows(PyObject *const *a) {
    const Pages p(a[0], a[1], a[2], a[3], a[4]);
    int32_t *moves = ints(a[5], p.dev, {p.P / 2, 2}), *n_moves = ints(a[6], p.dev, {1}), *map = ints(a[7], p.dev, {p.P});
    const int ps = int_of(a[8]);
    void *stream = stream_of(a[9], p.dev);
    const WithoutInterpreter others;
    return paged_attn_compact(p.table, p.lens, p.shares, p.free, (int)p.F, p.count, moves, n_moves, map, (int)p.B, ps, p.P, (int)p.W,
                              stream);
}

// Bytes of a page of pool `t`, dense and of P pages on this device.
int64_t page_bytes(const at::Tensor &t, int dev, int64_t P) {
    if (t.dim() < 2 || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || P < 1 || t.size(0) != P) throw Refused{};
    return t.numel() / P * (int64_t)t.element_size();
}

// check_pools(pools, block_table, page_shares): 0 if paged_attn_copy_pages takes them all, in lists of any length
int check_pools(PyObject *const *a) {
    const at::Tensor &shares = tensor(a[2]);
    if (!PyList_Check(a[0]) || shares.dim() != 1) throw Refused{};
    const int dev = this_device(tensor(a[1]));
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(a[0]); ++i) {
        const at::Tensor &t = tensor(PyList_GET_ITEM(a[0], i));
        const int64_t bytes = page_bytes(t, dev, shares.size(0));
        if (bytes < 4 || bytes % 4 != 0 || bytes > INT32_MAX || reinterpret_cast<uintptr_t>(t.data_ptr()) % 4 != 0) throw Refused{};
    }
    return 0;
}

// copy_pages(pools, pairs, n_pairs, stream)
int copy_pages(PyObject *const *a) {
    if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) throw Refused{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
    const at::Tensor &pairs = tensor(a[1]);
    if (n < 1 || n > PA_COPY_MAX_POOLS || pairs.dim() != 2) throw Refused{};
    const int dev = this_device(pairs);
    const int32_t *pp = ints(a[1], dev, {pairs.size(0), 2}), *count = ints_or_null(a[2], dev, {1});
    in_range({pairs.size(0)});
    void *pool[PA_COPY_MAX_POOLS];
    int64_t bytes[PA_COPY_MAX_POOLS], P = 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(a[0], i));
        if (i == 0) P = t.dim() ? t.size(0) : 0;
        bytes[i] = page_bytes(t, dev, P);
        pool[i] = t.data_ptr();
    }
    const int most = (int)pairs.size(0);
    void *stream = stream_of(a[3], dev);
    const WithoutInterpreter others;
    return paged_attn_copy_pages(pool, bytes, (int)n, pp, most, count, P, stream);
}

template <int (*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %zd arguments", N);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (...) {  // Refused, or an error of torch's (out of memory): the long way meets it again
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define PA_ENTRY(name, function, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<function, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PA_ENTRY("append_kv4", append_kv4, 5), PA_ENTRY("gather_kv4", gather_kv4, 5), PA_ENTRY("fwd_kv4", fwd_kv4, 12),
    PA_ENTRY("fork", fork_rows, 13),            PA_ENTRY("free", free_rows, 10),       PA_ENTRY("compact", compact_rows, 10),
    PA_ENTRY("copy_pages", copy_pages, 4), PA_ENTRY("check_pools", check_pools, 3), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_attn_binding() { return PyModule_Create(&module); }
