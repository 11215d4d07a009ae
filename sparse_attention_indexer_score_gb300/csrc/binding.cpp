// Python entry points of the append and attention calls: tensors to the C ABI's
// pointers, sizes and strides, and nothing else.
//
// These calls take a few microseconds on the GPU for a small decode step, less
// than a ctypes call with a dozen tensors takes to prepare (15 to 20 us on the
// host of a GB300, most of it attribute reads), so their marshalling is native.
// Argument errors raise ValueError here or RuntimeError with the C ABI's code.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "../../include/dsa.h"

namespace {

struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};

void need(bool ok, const char* what) {
    if (!ok) throw BadArgument(what);
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    need(THPVariable_Check(o), what);
    return THPVariable_Unpack(o);
}

// A call's device is its caches'; every other tensor's address goes to kernels there.
const at::Tensor& tensor(PyObject* o, const at::Device& device, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (t.device() != device)
        throw BadArgument("every tensor must be on the caches' device (" + device.str() + "), not on " +
                          t.device().str());
    return t;
}

bool given(PyObject* o) { return o != Py_None; }

// A dimension of one element (or none) may come with any stride, which the C calls would check: another in its place.
int64_t stride(const at::Tensor& t, int64_t d, int64_t instead = 0) { return t.size(d) > 1 ? t.stride(d) : instead; }

// Whether a dimension's elements lie one behind the other.
bool dense(const at::Tensor& t, int64_t d) { return t.numel() == 0 || t.size(d) == 1 || t.stride(d) == 1; }

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw BadArgument("sizes must be whole numbers");
    }
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {   // a tensor of several elements, say
        PyErr_Clear();
        throw BadArgument("flags must be true or false");
    }
    return v == 1;
}

void* pointer(const at::Tensor& t) { return t.data_ptr(); }

int32_t* status_word(PyObject* o, const at::Device& device) {
    if (!given(o)) return nullptr;
    const at::Tensor& t = tensor(o, device, "status must be a tensor");
    need(t.scalar_type() == at::kInt && t.numel() >= 1, "status must be int32");
    return static_cast<int32_t*>(pointer(t));
}

// The caches' GPU, current for the call: launches, SM counts and new tensors go by the current device.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;

    explicit OnDevice(const at::Device& device) {
        need(device.is_cuda(), "the caches must be CUDA tensors");
        if (c10::cuda::current_device() != device.index()) guard.set_device(device);
        stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    }
};

void check(int rc, const char* call) {
    if (rc == DSA_OK) return;
    const char* what = rc == DSA_ERR_INVALID       ? "invalid argument"
                       : rc == DSA_ERR_UNSUPPORTED ? "unsupported"
                                                   : "CUDA launch or driver error";
    throw std::runtime_error(std::string(call) + ": " + what);
}

// The caches, and what every other tensor of the call goes by.
struct Cache {
    dsa_kv_cache c;
    at::ScalarType type;
    at::Device device;
};

Cache cache_of(PyObject* k_cache, PyObject* v_cache) {
    const at::Tensor& k = tensor(k_cache, "k_cache must be a tensor");
    const at::Tensor& v = tensor(v_cache, k.device(), "v_cache must be a tensor");
    const at::ScalarType type = k.scalar_type();
    need((type == at::kBFloat16 || type == at::kHalf) && v.scalar_type() == type,
         "k_cache and v_cache must both be BF16 or both FP16");
    need(k.dim() == 4 && k.size(1) == DSA_PAGE_TOKENS && v.sizes() == k.sizes(),
         "k_cache and v_cache must be [pages, 64, heads, dim]");
    need(k.stride(3) == 1 && v.stride(3) == 1, "cache columns must be contiguous");
    dsa_kv_cache c;
    c.k = pointer(k), c.v = pointer(v);
    c.num_pages = k.size(0), c.heads = k.size(2), c.dim = k.size(3);
    c.k_page_stride = stride(k, 0), c.k_token_stride = stride(k, 1), c.k_head_stride = stride(k, 2);
    c.v_page_stride = stride(v, 0), c.v_token_stride = stride(v, 1), c.v_head_stride = stride(v, 2);
    c.dtype = type == at::kBFloat16 ? DSA_BF16 : DSA_FP16;
    return Cache{c, type, k.device()};
}

// [n, heads, dim] of the cache's type with contiguous columns.
const at::Tensor& rows_of(PyObject* o, const Cache& cache, const char* what) {
    const at::Tensor& t = tensor(o, cache.device, what);
    need(t.scalar_type() == cache.type && t.dim() == 3 && t.size(2) == cache.c.dim && t.stride(2) == 1, what);
    return t;
}

const at::Tensor& list_of(PyObject* o, const at::Device& device, at::ScalarType type, int64_t n, const char* what) {
    const at::Tensor& t = tensor(o, device, what);
    need(t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && t.is_contiguous(), what);
    return t;
}

// The caller's output tensor, or a new one like q.
at::Tensor output(PyObject* o, const at::Tensor& q, const char* what) {
    if (!given(o)) return at::empty(q.sizes(), q.options());
    const at::Tensor& t = tensor(o, q.device(), what);
    need(t.scalar_type() == q.scalar_type() && t.sizes() == q.sizes() && t.stride(2) == 1, what);
    return t;
}

// k, v, slots, k_cache, v_cache, positions, cos_sin, q, q_out, interleaved, status
PyObject* kv_append(PyObject* const* a) {
    const Cache cache = cache_of(a[3], a[4]);
    const dsa_kv_cache& c = cache.c;
    constexpr const char* kv = "k and v must be [n, heads, dim] of the cache's type with contiguous columns";
    const at::Tensor &k = rows_of(a[0], cache, kv), &v = rows_of(a[1], cache, kv);
    need(k.size(1) == c.heads && v.sizes() == k.sizes(), kv);
    const int64_t n = k.size(0);
    const at::Tensor& slots =
        list_of(a[2], cache.device, at::kLong, n, "slots must be contiguous int64 [n], one per key");
    const int64_t* positions = nullptr;
    const float* cos_sin = nullptr;
    int64_t rot = 0, max_pos = 0, cs_stride = 0;
    if (given(a[6])) {
        constexpr const char* angles = "cos_sin must be FP32 [positions, rot] with contiguous rows";
        const at::Tensor& t = tensor(a[6], cache.device, angles);
        need(t.scalar_type() == at::kFloat && t.dim() == 2 && dense(t, 1), angles);
        positions = static_cast<const int64_t*>(
            pointer(list_of(a[5], cache.device, at::kLong, n, "positions must be contiguous int64 [n]")));
        cos_sin = static_cast<const float*>(pointer(t));
        max_pos = t.size(0), rot = t.size(1), cs_stride = stride(t, 0, rot);
    }
    const void* q_ptr = nullptr;
    void* out_ptr = nullptr;
    int64_t q_heads = 0, qt = 0, qh = 0, ot = 0, oh = 0;
    at::Tensor out;
    if (given(a[7])) {
        constexpr const char* qs = "q must be [n, q_heads, dim] of the cache's type with contiguous columns";
        const at::Tensor& q = rows_of(a[7], cache, qs);
        need(q.size(0) == n, qs);
        out = output(a[8], q, "q_out must match q");
        q_heads = q.size(1), qt = stride(q, 0), qh = stride(q, 1), ot = stride(out, 0), oh = stride(out, 1);
        q_ptr = pointer(q), out_ptr = pointer(out);
    } else {
        need(!given(a[8]), "q_out needs q");
    }
    const bool interleaved = truth(a[9]);
    int32_t* const status = status_word(a[10], cache.device);
    const OnDevice on(cache.device);
    check(dsa_kv_append(&c, pointer(k), stride(k, 0), stride(k, 1), pointer(v), stride(v, 0), stride(v, 1),
                        q_ptr, qt, qh, q_heads, out_ptr, ot, oh, n, static_cast<const int64_t*>(pointer(slots)),
                        positions, cos_sin, cs_stride, max_pos, rot, interleaved, status, on.stream),
          "dsa_kv_append");
    if (!out.defined()) Py_RETURN_NONE;
    if (given(a[8])) {
        Py_INCREF(a[8]);
        return a[8];
    }
    return THPVariable_Wrap(out);
}

// What the two attention calls share: q, k_cache, v_cache, block_table, starts, row_ends.
struct Attention {
    Cache cache;
    const dsa_kv_cache& c = cache.c;
    at::Tensor q, out, lse;
    const int32_t *table, *starts, *ends;
    int64_t bt_stride, pages, requests, rows, heads;
    float* lse_ptr = nullptr;
    float scale;

    Attention(PyObject* const* a, PyObject* scale_o, PyObject* out_o, PyObject* want_lse)
        : cache(cache_of(a[1], a[2])) {
        q = rows_of(a[0], cache, "q must be [rows, heads, dim] of the cache's type with contiguous columns");
        constexpr const char* bt = "block_table must be int32 [requests, pages] with contiguous rows";
        const at::Tensor& t = tensor(a[3], cache.device, bt);
        need(t.scalar_type() == at::kInt && t.dim() == 2 && dense(t, 1), bt);
        requests = t.size(0), pages = t.size(1), bt_stride = stride(t, 0, pages);
        rows = q.size(0), heads = q.size(1);
        table = static_cast<const int32_t*>(pointer(t));
        starts = static_cast<const int32_t*>(
            pointer(list_of(a[4], cache.device, at::kInt, requests + 1,
                            "starts must be contiguous int32, one entry per request and one more")));
        ends = static_cast<const int32_t*>(pointer(list_of(
            a[5], cache.device, at::kInt, rows, "row_ends must be contiguous int32, one bound per query row")));
        scale = given(scale_o) ? static_cast<float>(PyFloat_AsDouble(scale_o))
                               : static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.dim)));
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw BadArgument("scale must be a number");
        }
        out = output(out_o, q, "out must match q");
        if (truth(want_lse)) {
            lse = at::empty({rows, heads}, q.options().dtype(at::kFloat));
            lse_ptr = static_cast<float*>(pointer(lse));
        }
    }

    at::Tensor workspace(PyObject* o, int64_t max_query_len, int64_t k) const {
        if (given(o)) {
            const at::Tensor& t = tensor(o, cache.device, "workspace must be a tensor");
            need(t.is_contiguous(), "workspace must be contiguous");
            return t;
        }
        const size_t n = dsa_attend_workspace_size(rows, requests, heads, c.heads, c.dim, max_query_len, k);
        return at::empty({static_cast<int64_t>(n < 256 ? 256 : n)}, q.options().dtype(at::kByte));
    }

    PyObject* result(PyObject* out_o) const {
        PyObject* pair = PyTuple_New(2);
        if (!pair) return nullptr;
        if (given(out_o)) Py_INCREF(out_o);
        PyTuple_SET_ITEM(pair, 0, given(out_o) ? out_o : THPVariable_Wrap(out));
        if (!lse.defined()) Py_INCREF(Py_None);
        PyTuple_SET_ITEM(pair, 1, lse.defined() ? THPVariable_Wrap(lse) : Py_None);
        return pair;
    }
};

// q, k_cache, v_cache, block_table, starts, row_ends, max_query_len, prefix_pages, prefix_len, scale, out, want_lse,
// workspace, status
PyObject* attend_paged(PyObject* const* a) {
    const Attention x(a, a[9], a[10], a[11]);
    const int64_t max_query_len = whole(a[6]), prefix_len = whole(a[8]);
    const int32_t* prefix = nullptr;
    if (prefix_len != 0) {
        constexpr const char* what = "prefix_pages must be contiguous int32 and hold prefix_len keys";
        const at::Tensor& t = tensor(a[7], x.cache.device, what);
        need(t.scalar_type() == at::kInt && t.is_contiguous() && t.numel() * DSA_PAGE_TOKENS >= prefix_len, what);
        prefix = static_cast<const int32_t*>(pointer(t));
    }
    int32_t* const status = status_word(a[13], x.cache.device);
    const at::Tensor ws = x.workspace(a[12], max_query_len, 0);
    const OnDevice on(x.cache.device);
    check(dsa_attend_paged(&x.c, pointer(x.q), stride(x.q, 0), stride(x.q, 1), x.heads, x.table, x.bt_stride, x.pages,
                           x.starts, x.ends, x.requests, x.rows, max_query_len, prefix, prefix_len, x.scale,
                           pointer(x.out), stride(x.out, 0), stride(x.out, 1), x.lse_ptr, pointer(ws), ws.nbytes(),
                           status, on.stream),
          "dsa_attend_paged");
    return x.result(a[10]);
}

// q, k_cache, v_cache, block_table, starts, row_ends, topk, scale, out, want_lse, workspace, status
PyObject* attend_selected(PyObject* const* a) {
    const Attention x(a, a[7], a[8], a[9]);
    constexpr const char* what = "topk must be int32 [rows, k] with contiguous rows";
    const at::Tensor& t = tensor(a[6], x.cache.device, what);
    need(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == x.rows && dense(t, 1), what);
    const int64_t k = t.size(1);
    int32_t* const status = status_word(a[11], x.cache.device);
    const at::Tensor ws = x.workspace(a[10], 1, k > 0 ? k : 1);
    const OnDevice on(x.cache.device);
    check(dsa_attend_selected(&x.c, pointer(x.q), stride(x.q, 0), stride(x.q, 1), x.heads, x.table, x.bt_stride,
                              x.pages, x.starts, x.ends, x.requests, x.rows, static_cast<const int32_t*>(pointer(t)),
                              stride(t, 0, k), k, x.scale, pointer(x.out), stride(x.out, 0), stride(x.out, 1),
                              x.lse_ptr, pointer(ws), ws.nbytes(), status, on.stream),
          "dsa_attend_selected");
    return x.result(a[8]);
}

// A fixed number of positional arguments; C++ exceptions become Python ones.
template <PyObject* (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return kCall(args);
    } catch (const BadArgument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <PyObject* (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name) {
    PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t) = entry<kCall, kArgs>;
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<kv_append, 11>("kv_append"), method<attend_paged, 14>("attend_paged"),
                         method<attend_selected, 12>("attend_selected"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dsa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dsa_binding() { return PyModule_Create(&module); }
