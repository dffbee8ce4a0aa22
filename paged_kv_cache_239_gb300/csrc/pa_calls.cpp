// pa_calls.cpp -- the calls of a speculation step from Python: a CPython module beside the
// library that looks at the tensors (type, shape, contiguity, device), takes torch's current
// stream and calls the C ABI.
//
// Why not through ctypes as the other calls: a step makes five of these per layer or step, each
// with up to a dozen small tensors, and their kernels run for 3 to 10 us.  From Python the
// checks and the marshalling take 8 - 9 us of the host per call; here the launch is most of it.
//
// Each function returns the library's code, kBadTensor where a tensor is not what the call
// takes (BlockPool then finds out which and why), kWrongDevice where the pool is not on the
// current device.  Nothing throws across the module.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "pagedattn.h"

namespace {

constexpr long kBadTensor = -1, kWrongDevice = -2;

struct Refused {
    long code;
};

// The arguments of one call, in order; anything unexpected is thrown as Refused.
struct Args {
    PyObject* const* at;
    Py_ssize_t left;
    PyObject* next() {
        if (left-- <= 0) throw Refused{kBadTensor};
        return *at++;
    }
    long long integer() {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Refused{kBadTensor};
        return v;
    }
    int int32() {
        const long long v = integer();
        if (v != (int)v) throw Refused{kBadTensor};
        return (int)v;
    }
    double real() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Refused{kBadTensor};
        return v;
    }
    template <class T>
    T* handle() {  // an address, None: NULL
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        void* v = PyLong_AsVoidPtr(o);
        if (!v && PyErr_Occurred()) throw Refused{kBadTensor};
        return static_cast<T*>(v);
    }
    const at::Tensor* tensor(bool may_be_none = false) {
        PyObject* o = next();
        if (may_be_none && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) throw Refused{kBadTensor};
        return &THPVariable_Unpack(o);
    }
};

// What every call begins with: the pool's handle and device; and the stream at its end.
struct Call {
    Args a;
    pa_pool* pool;
    int device;
    Call(PyObject* const* args, Py_ssize_t n) : a{args, n}, pool(a.handle<pa_pool>()), device(a.int32()) {}

    void dense(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) const {
        if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || t.get_device() != device)
            throw Refused{kBadTensor};
    }
    template <class T>
    T* ints(at::IntArrayRef shape, at::ScalarType type = at::kInt, bool may_be_none = false) {
        const at::Tensor* t = a.tensor(may_be_none);
        if (!t) return nullptr;
        dense(*t, type, shape);
        return static_cast<T*>(t->data_ptr());
    }
    // The raw stream: the one given, or torch's current one.
    pa_stream_t stream() {
        PyObject* o = a.next();
        if (a.left != 0) throw Refused{kBadTensor};
        if (device < 0 || c10::cuda::current_device() != device) throw Refused{kWrongDevice};
        if (o == Py_None) return reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
        void* v = PyLong_AsVoidPtr(o);
        if (!v && PyErr_Occurred()) throw Refused{kBadTensor};
        return static_cast<pa_stream_t>(v);
    }
};

template <class F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, F body) {
    long rc;
    try {
        Call c(args, n);
        rc = body(c);
    } catch (const Refused& r) {
        PyErr_Clear();
        rc = r.code;
    } catch (...) {  // (torch's own checks)
        PyErr_Clear();
        rc = kBadTensor;
    }
    return PyLong_FromLong(rc);
}

template <class F>
long unlocked(F call) noexcept {  // (a launch waits where the stream's queue is full)
    long rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return rc;
}

// A dimension that fits the ABI's int.
int64_t extent(const at::Tensor& t, int i) {
    const int64_t n = t.size(i);
    if (n > INT_MAX) throw Refused{kBadTensor};
    return n;
}

at::ScalarType pool_type(int code) { return code == PA_DTYPE_BF16 ? at::kBFloat16 : at::kFloat; }

// (pool, device, num_blocks, stack, tables, cached_lens, new_counts, num_tokens, parents, context_lens,
// query_starts, slots, positions, tree_masks, mask_words, stream)
PyObject* plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Call& c) {
        const int64_t nb = c.a.integer();
        int* stack = c.ints<int>({nb + 1});
        const at::Tensor& bt = *c.a.tensor();
        if (bt.dim() != 2) throw Refused{kBadTensor};
        const int64_t batch = extent(bt, 0), maxb = extent(bt, 1);
        c.dense(bt, at::kInt, {batch, maxb});
        const int* cached = c.ints<int>({batch});
        const int* counts = c.ints<int>({batch});
        const int tokens = c.a.int32();
        const int* parents = c.ints<int>({tokens}, at::kInt, true);
        int* lens = c.ints<int>({batch});
        int* starts = c.ints<int>({batch + 1});
        int64_t* slots = c.ints<int64_t>({tokens}, at::kLong);
        int* positions = c.ints<int>({tokens});
        const at::Tensor* masks = c.a.tensor(true);
        const int words = c.a.int32();
        if (masks) c.dense(*masks, at::kInt, {tokens, words});
        const pa_stream_t s = c.stream();
        int* tables = static_cast<int*>(bt.data_ptr());
        uint32_t* bits = masks ? static_cast<uint32_t*>(masks->data_ptr()) : nullptr;
        return unlocked([&] {
            return pa_device_plan_tokens(c.pool, stack, tables, (int)maxb, cached, counts, parents, (int)batch, tokens, lens,
                                         starts, slots, positions, bits, words, s);
        });
    });
}

// (pool, device, num_blocks, stack, tables, context_lens, new_lens, stream)
PyObject* trim(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Call& c) {
        const int64_t nb = c.a.integer();
        int* stack = c.ints<int>({nb + 1});
        const at::Tensor& bt = *c.a.tensor();
        if (bt.dim() != 2) throw Refused{kBadTensor};
        const int64_t batch = extent(bt, 0), maxb = extent(bt, 1);
        c.dense(bt, at::kInt, {batch, maxb});
        const int* lens = c.ints<int>({batch});
        const int* new_lens = c.ints<int>({batch});
        const pa_stream_t s = c.stream();
        int* tables = static_cast<int*>(bt.data_ptr());
        return unlocked([&] {
            return pa_device_trim_sequences(c.pool, stack, tables, (int)maxb, lens, new_lens, (int)batch, s);
        });
    });
}

// (pool, device, slots, parents, tokens, targets, context_lens, query_starts, max_path, counts, nodes,
// next_tokens, next_lens, stream)
PyObject* accept(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Call& c) {
        const at::Tensor& slots = *c.a.tensor();
        if (slots.dim() != 1) throw Refused{kBadTensor};
        const int64_t rows = extent(slots, 0);
        c.dense(slots, at::kLong, {rows});
        const int* parents = c.ints<int>({rows});
        const int* tokens = c.ints<int>({rows});
        const int* targets = c.ints<int>({rows});
        const at::Tensor& lens = *c.a.tensor();
        if (lens.dim() != 1) throw Refused{kBadTensor};
        const int64_t batch = extent(lens, 0);
        c.dense(lens, at::kInt, {batch});
        const int* starts = c.ints<int>({batch + 1});
        const int most = c.a.int32();
        int* counts = c.ints<int>({batch});
        int* nodes = c.ints<int>({batch, most});
        int* next_tokens = c.ints<int>({batch});
        int* next_lens = c.ints<int>({batch});
        const pa_stream_t s = c.stream();
        const int64_t* at = static_cast<const int64_t*>(slots.data_ptr());
        const int* context = static_cast<const int*>(lens.data_ptr());
        return unlocked([&] {
            return pa_device_accept_tree(c.pool, at, parents, tokens, targets, context, starts, (int)batch, (int)rows, most,
                                         counts, nodes, next_tokens, next_lens, s);
        });
    });
}

// (pool, device, type, head_dim, layer, out, q, tables, context_lens, query_starts, tree_masks, scale, workspace,
// stream)
PyObject* tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Call& c) {
        const at::ScalarType type = pool_type(c.a.int32());
        const int64_t d = c.a.integer();
        const int layer = c.a.int32();
        const at::Tensor &out = *c.a.tensor(), &q = *c.a.tensor(), &bt = *c.a.tensor();
        if (q.dim() != 3 || bt.dim() != 2) throw Refused{kBadTensor};
        const int64_t tokens = extent(q, 0), heads = extent(q, 1), batch = extent(bt, 0), maxb = extent(bt, 1);
        c.dense(q, type, {tokens, heads, d});
        c.dense(out, type, {tokens, heads, d});
        c.dense(bt, at::kInt, {batch, maxb});
        const int* lens = c.ints<int>({batch});
        const int* starts = c.ints<int>({batch + 1});
        const at::Tensor& masks = *c.a.tensor();
        if (masks.dim() != 2) throw Refused{kBadTensor};
        const int64_t words = extent(masks, 1);
        c.dense(masks, at::kInt, {tokens, words});
        const float scale = (float)c.a.real();
        const at::Tensor* ws = c.a.tensor(true);
        if (ws && (ws->get_device() != c.device || !ws->is_contiguous())) throw Refused{kBadTensor};
        const pa_stream_t s = c.stream();
        void *to = out.data_ptr(), *from = q.data_ptr(), *work = ws ? ws->data_ptr() : nullptr;
        const int* tables = static_cast<const int*>(bt.data_ptr());
        const uint32_t* bits = static_cast<const uint32_t*>(masks.data_ptr());
        const size_t bytes = ws ? ws->nbytes() : 0;
        return unlocked([&] {
            return pa_tree_attention(to, from, c.pool, layer, tables, (int)maxb, lens, starts, bits, (int)words, (int)batch,
                                     (int)tokens, (int)heads, scale, work, bytes, s);
        });
    });
}

// (pool, device, type, kv_heads, head_dim, layer, out, q, k, v, rope, q_weight, k_weight, eps, positions, slots,
// stream)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Call& c) {
        const at::ScalarType type = pool_type(c.a.int32());
        const int64_t hkv = c.a.integer(), d = c.a.integer();
        const int layer = c.a.int32();
        const at::Tensor &out = *c.a.tensor(), &q = *c.a.tensor();
        if (q.dim() != 3) throw Refused{kBadTensor};
        const int64_t tokens = extent(q, 0), heads = extent(q, 1);
        // rows of heads, any stride between the tokens
        auto rows = [&](const at::Tensor& t, int64_t h) {
            if (t.scalar_type() != type || t.sizes() != at::IntArrayRef({tokens, h, d}) || t.get_device() != c.device)
                throw Refused{kBadTensor};
            if (tokens && (t.stride(2) != 1 || (h > 1 && t.stride(1) != d))) throw Refused{kBadTensor};
            return tokens > 1 ? t.stride(0) : h * d;
        };
        const int64_t qs = rows(q, heads);
        const at::Tensor& k = *c.a.tensor();
        const int64_t ks = rows(k, hkv);
        const at::Tensor& v = *c.a.tensor();
        const int64_t vs = rows(v, hkv);
        c.dense(out, type, {tokens, heads, d});
        const pa_rope* rope = c.a.handle<pa_rope>();
        const void* qw = c.ints<void>({d}, type, true);
        const void* kw = c.ints<void>({d}, type, true);
        const float eps = (float)c.a.real();
        const int* positions = c.ints<int>({tokens});
        const int64_t* slots = c.ints<int64_t>({tokens}, at::kLong);
        const pa_stream_t s = c.stream();
        void *to = out.data_ptr(), *q0 = q.data_ptr(), *k0 = k.data_ptr(), *v0 = v.data_ptr();
        return unlocked([&] {
            return pa_norm_rope_write_kv_slots(c.pool, layer, to, q0, qs, k0, ks, v0, vs, rope, qw, kw, eps, positions, slots,
                                               (int)tokens, (int)heads, s);
        });
    });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CALL(plan), CALL(trim), CALL(accept), CALL(tree), CALL(append), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "pagedcalls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pagedcalls() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddIntConstant(m, "WRONG_DEVICE", kWrongDevice)) Py_CLEAR(m);
    return m;
}
