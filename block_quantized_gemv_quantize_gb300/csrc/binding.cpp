// The paged cache's and the sparse layer's calls from Python without Python's share of the work: reads
// the tensors, checks them, makes their device the current one, allocates the outputs
// and calls the library.  A call that it would refuse, or whose tensors it does not
// know how to take, returns None and goes through the ctypes binding (_lib.py), which
// does the same and says what is wrong.  Only host code: the kernels are the
// library's, by the addresses of its entry points that init() and init_sparse() get.  A call of
// attn_paged takes the host 7 us, of kv_read with new outputs 5 and of kv_write 2, by
// ctypes 20, 15 and 8, beside 2 to 10 us of kernels on small inputs.
// As many calls are the sparse layer's: a router, two products, MXFP4 rows in and out.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "qgemv.h"

namespace {

// the library's entry points, by the addresses that init() gets
decltype(&::kv_write) kv_write_entry;
decltype(&::kv_read) kv_read_entry;
decltype(&::attn_paged) attn_entry;
decltype(&::kv_page_bytes) page_bytes_entry;
decltype(&::attn_paged_workspace_bytes) workspace_bytes_entry;
decltype(&::quantize_mxfp4) quantize_entry;
decltype(&::dequantize_mxfp4) dequantize_entry;
decltype(&::moe_route) route_entry;
decltype(&::moe_route_workspace_bytes) route_bytes_entry;
decltype(&::mxfp4_pack_bytes) pack_bytes_entry;
decltype(&::qgemm_mxfp4) gemm_entry;
decltype(&::moe_gate_up_mxfp4) gate_up_entry;
decltype(&::moe_down_mxfp4) down_entry;
decltype(&::qgemm_mxfp4_workspace_bytes) product_bytes_entry[3];

int type_code(const at::Tensor& t)
{
    switch (t.scalar_type()) {
    case at::kFloat: return 0;
    case at::kHalf: return 1;
    case at::kBFloat16: return 2;
    default: return -1;
    }
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// [tokens, heads, head_dim] on `device`, rows contiguous
bool rows_ok(const at::Tensor& t, c10::Device device)
{
    return t.is_cuda() && t.device() == device && t.dim() == 3 && (t.size(2) <= 1 || t.stride(2) == 1);
}

bool cache_ok(const at::Tensor& t, c10::Device device, size_t page, int64_t& pages)
{
    if (page == 0 || t.scalar_type() != at::kByte || t.device() != device || !t.is_contiguous()) return false;
    pages = t.numel() / (int64_t)page;
    return pages > 0 && t.numel() % (int64_t)page == 0;
}

bool slots_ok(const at::Tensor& t, c10::Device device)
{
    return t.scalar_type() == at::kLong && t.dim() == 1 && t.is_contiguous() && t.device() == device;
}

// a Python int that fits an int; -1 in `bad` otherwise
int as_int(PyObject* o, bool& bad)
{
    const long v = PyLong_Check(o) ? PyLong_AsLong(o) : (bad = true, 0);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        bad = true;
    }
    if (v > INT32_MAX || v < INT32_MIN) bad = true;
    return (int)v;
}

at::Tensor empty(c10::IntArrayRef sizes, at::ScalarType type, c10::Device device)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

// Runs f without the interpreter's lock, which comes back if f throws, too.
template <typename F>
int unlocked(F f)
{
    struct Released {
        PyThreadState* state = PyEval_SaveThread();
        ~Released() { PyEval_RestoreThread(state); }
    } released;
    return f();
}

// kv_write(cache, k, v, slots, fmt, page_tokens) -> status
PyObject* call_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor *cache, *k, *v, *slots;
    if (n_args != 6 || !(cache = tensor(a[0])) || !(k = tensor(a[1])) || !(v = tensor(a[2])) || !(slots = tensor(a[3])))
        Py_RETURN_NONE;
    bool bad = false;
    const int fmt = as_int(a[4], bad), page = as_int(a[5], bad), type = type_code(*k);
    const auto device = k->device();
    if (bad || type < 0 || !rows_ok(*k, device) || !rows_ok(*v, device) || v->sizes() != k->sizes() ||
        v->scalar_type() != k->scalar_type() || !slots_ok(*slots, device) || slots->size(0) != k->size(0) ||
        k->numel() == 0 || k->size(0) > INT32_MAX || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX)
        Py_RETURN_NONE;
    const int n = (int)k->size(0), heads = (int)k->size(1), dim = (int)k->size(2);
    int64_t pages;
    if (!cache_ok(*cache, device, page_bytes_entry(fmt, page, heads, dim), pages)) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    return PyLong_FromLong(unlocked([&] {
        return kv_write_entry(fmt, type, k->data_ptr(), k->stride(0), k->stride(1), v->data_ptr(), v->stride(0),
                              v->stride(1), static_cast<const int64_t*>(slots->data_ptr()), cache->data_ptr(), pages,
                              page, n, heads, dim, stream);
    }));
}

// kv_read(cache, slots, fmt, page_tokens, n_kv_heads, head_dim, type, k or None, v or None) -> status or (k, v)
PyObject* call_kv_read(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor *cache, *slots;
    if (n_args != 9 || !(cache = tensor(a[0])) || !(slots = tensor(a[1])) || !cache->is_cuda()) Py_RETURN_NONE;
    bool bad = false;
    const int fmt = as_int(a[2], bad), page = as_int(a[3], bad), heads = as_int(a[4], bad), dim = as_int(a[5], bad);
    int type = as_int(a[6], bad);
    const auto device = cache->device();
    int64_t pages;
    if (bad || !slots_ok(*slots, device) || slots->size(0) == 0 || slots->size(0) > INT32_MAX ||
        !cache_ok(*cache, device, page_bytes_entry(fmt, page, heads, dim), pages))
        Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);
    const int64_t n = slots->size(0), sizes[3] = {n, heads, dim};
    at::Tensor k, v;
    if (a[7] == Py_None && a[8] == Py_None) {
        const at::ScalarType types[3] = {at::kFloat, at::kHalf, at::kBFloat16};
        if (type < 0 || type > 2) Py_RETURN_NONE;
        k = empty(sizes, types[type], device);
        v = empty(sizes, types[type], device);
    } else {
        const at::Tensor *gk = tensor(a[7]), *gv = tensor(a[8]);
        if (!gk || !gv || !rows_ok(*gk, device) || !rows_ok(*gv, device) || gk->sizes() != c10::IntArrayRef(sizes) ||
            gv->sizes() != gk->sizes() || gv->scalar_type() != gk->scalar_type() || (type = type_code(*gk)) < 0)
            Py_RETURN_NONE;
        k = *gk;
        v = *gv;
    }
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    const int status = unlocked([&] {
        return kv_read_entry(fmt, type, cache->data_ptr(), pages, page, static_cast<const int64_t*>(slots->data_ptr()),
                             k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), (int)n,
                             heads, dim, stream);
    });
    if (status) return PyLong_FromLong(status);
    if (a[7] != Py_None) return PyTuple_Pack(2, a[7], a[8]);
    PyObject *pk = THPVariable_Wrap(std::move(k)), *pv = THPVariable_Wrap(std::move(v));
    PyObject* both = pk && pv ? PyTuple_Pack(2, pk, pv) : nullptr;
    Py_XDECREF(pk);
    Py_XDECREF(pv);
    return both;
}

// One workspace for each (device, stream), never freed, as the program may end
// after CUDA has.  A call's two kernels share it: its lock keeps another thread's
// from coming between them.
struct Workspace {
    std::mutex lock;
    at::Tensor memory;
};

Workspace& workspace(c10::Device device, void* stream)
{
    static auto* all = new std::map<std::pair<int, void*>, Workspace>;
    static auto* lock = new std::mutex;
    const std::lock_guard<std::mutex> held(*lock);
    return (*all)[{device.index(), stream}];
}

// attn_paged(q, cache, page_table, kv_lens, fmt, page_tokens, n_kv_heads, rows, scale or None, window, out or None,
//            lse or None, ws or None) -> status or out
PyObject* call_attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor *q, *cache, *table, *lens, *lse = nullptr;
    if (n_args != 13 || !(q = tensor(a[0])) || !(cache = tensor(a[1])) || !(table = tensor(a[2])) ||
        !(lens = tensor(a[3])) || (a[11] != Py_None && !(lse = tensor(a[11]))))
        Py_RETURN_NONE;
    bool bad = false;
    const int fmt = as_int(a[4], bad), page = as_int(a[5], bad), kv_heads = as_int(a[6], bad), rows = as_int(a[7], bad);
    const int window = as_int(a[9], bad), type = type_code(*q);
    const auto device = q->device();
    if (bad || rows < 1 || type < 0 || !rows_ok(*q, device) || q->numel() == 0 || q->size(0) > INT32_MAX ||
        q->size(1) > INT32_MAX || q->size(2) > INT32_MAX || table->scalar_type() != at::kInt || table->dim() != 2 ||
        (table->size(1) > 1 && table->stride(1) != 1) || table->size(1) > INT32_MAX || table->device() != device ||
        lens->scalar_type() != at::kInt || lens->dim() != 1 || !lens->is_contiguous() || lens->device() != device)
        Py_RETURN_NONE;
    const int64_t n = q->size(0), batch = table->size(0), max_pages = table->size(1);
    const int heads = (int)q->size(1), dim = (int)q->size(2);
    int64_t pages;
    if (batch < 1 || n != batch * rows || lens->size(0) != batch || max_pages < 1 ||
        !cache_ok(*cache, device, page_bytes_entry(fmt, page, kv_heads, dim), pages))
        Py_RETURN_NONE;
    if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != n || lse->size(1) != heads ||
                !lse->is_contiguous() || lse->device() != device))
        Py_RETURN_NONE;
    double scale = 1.0 / std::sqrt((double)dim);
    if (a[8] != Py_None) {
        scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
    }
    const size_t need = workspace_bytes_entry(type, rows, heads, kv_heads, dim);
    if (need == 0) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);  // (the capture query below asks the current device's stream)
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    at::Tensor out, ws;
    Workspace* shared = nullptr;
    if (a[10] == Py_None) {
        out = empty(q->sizes(), q->scalar_type(), device);
    } else {
        const at::Tensor* given = tensor(a[10]);
        if (!given || !rows_ok(*given, device) || given->sizes() != q->sizes() || given->scalar_type() != q->scalar_type())
            Py_RETURN_NONE;
        out = *given;
    }
    if (a[12] != Py_None) {
        const at::Tensor* given = tensor(a[12]);
        if (!given || given->device() != device || given->scalar_type() != at::kByte || !given->is_contiguous()) Py_RETURN_NONE;
        ws = *given;
    } else if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
        ws = empty({(int64_t)need}, at::kByte, device);  // its graph's own
    } else {
        shared = &workspace(device, stream);
    }
    const int64_t ld = batch > 1 ? table->stride(0) : std::max(table->stride(0), max_pages);
    const int status = unlocked([&] {
        std::unique_lock<std::mutex> held;
        if (shared) {
            held = std::unique_lock<std::mutex>(shared->lock);
            if (!shared->memory.defined() || (size_t)shared->memory.numel() < need)
                shared->memory = empty({(int64_t)need}, at::kByte, device);
            ws = shared->memory;
        }
        return attn_entry(fmt, type, q->data_ptr(), q->stride(0), q->stride(1), cache->data_ptr(), pages, page,
                          static_cast<const int32_t*>(table->data_ptr()), ld, (int)max_pages,
                          static_cast<const int32_t*>(lens->data_ptr()), out.data_ptr(), out.stride(0), out.stride(1),
                          lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws.data_ptr(), (size_t)ws.numel(),
                          (int)batch, rows, heads, kv_heads, dim, (float)scale, window, stream);
    });
    if (status) return PyLong_FromLong(status);
    if (a[10] != Py_None) return Py_NewRef(a[10]);
    return THPVariable_Wrap(std::move(out));
}

// [rows, values] on `device`, rows contiguous and apart; the row stride goes to ld
bool matrix_ok(const at::Tensor& t, c10::Device device, int64_t& ld)
{
    if (!t.is_cuda() || t.device() != device || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) ||
        (t.size(0) > 1 && t.stride(0) < t.size(1)))
        return false;
    ld = t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
    return true;
}

bool array_ok(const at::Tensor& t, c10::Device device, at::ScalarType type, int64_t numel)
{
    return t.scalar_type() == type && t.device() == device && t.is_contiguous() && t.numel() == numel;
}

// A call's workspace: the given one, or memory of its own; false: not one to take.
bool scratch(PyObject* given, size_t need, c10::Device device, at::Tensor& ws)
{
    if (given != Py_None) {
        const at::Tensor* t = tensor(given);
        if (!t || t->device() != device || t->scalar_type() != at::kByte || !t->is_contiguous()) return false;
        ws = *t;
    } else if (need) {
        ws = empty({(int64_t)need}, at::kByte, device);
    }
    return true;
}

// quantize_mxfp4(x, out or None) -> status or out
PyObject* call_quantize(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor* x;
    int64_t ld;
    if (n_args != 2 || !(x = tensor(a[0])) || !matrix_ok(*x, x->device(), ld)) Py_RETURN_NONE;
    const int type = type_code(*x);
    const auto device = x->device();
    const int64_t n = x->size(0), k = x->size(1);
    if (type < 0 || n < 1 || k < 32 || k % 32 || k > INT32_MAX) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out;
    if (a[1] == Py_None) {
        out = empty({n, k / 32, 17}, at::kByte, device);
    } else {
        const at::Tensor* given = tensor(a[1]);
        if (!given || given->dim() != 3 || given->size(0) != n || given->size(1) != k / 32 ||
            !array_ok(*given, device, at::kByte, n * (k / 32) * 17))
            Py_RETURN_NONE;
        out = *given;
    }
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    const int status = unlocked([&] { return quantize_entry(type, x->data_ptr(), ld, out.data_ptr(), n, (int)k, stream); });
    if (status) return PyLong_FromLong(status);
    if (a[1] != Py_None) return Py_NewRef(a[1]);
    return THPVariable_Wrap(std::move(out));
}

// dequantize_mxfp4(blocks, type, out or None) -> status or out
PyObject* call_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor* blocks;
    if (n_args != 3 || !(blocks = tensor(a[0])) || !blocks->is_cuda() || blocks->dim() != 3 || blocks->size(2) != 17 ||
        blocks->scalar_type() != at::kByte || !blocks->is_contiguous())
        Py_RETURN_NONE;
    bool bad = false;
    int type = as_int(a[1], bad);
    const auto device = blocks->device();
    const int64_t n = blocks->size(0), k = blocks->size(1) * 32;
    if (bad || n < 1 || k < 32 || k > INT32_MAX) Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out;
    int64_t ld = k;
    if (a[2] == Py_None) {
        const at::ScalarType types[3] = {at::kFloat, at::kHalf, at::kBFloat16};
        if (type < 0 || type > 2) Py_RETURN_NONE;
        out = empty({n, k}, types[type], device);
    } else {
        const at::Tensor* given = tensor(a[2]);
        if (!given || !matrix_ok(*given, device, ld) || given->size(0) != n || given->size(1) != k || (type = type_code(*given)) < 0)
            Py_RETURN_NONE;
        out = *given;
    }
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    const int status =
        unlocked([&] { return dequantize_entry(type, blocks->data_ptr(), out.data_ptr(), ld, n, (int)k, stream); });
    if (status) return PyLong_FromLong(status);
    if (a[2] != Py_None) return Py_NewRef(a[2]);
    return THPVariable_Wrap(std::move(out));
}

// moe_route(logits, top_k, score, renormalize, scale, ws or None) -> status or (ids, weights, offsets, order)
PyObject* call_route(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor* logits;
    int64_t ld;
    if (n_args != 6 || !(logits = tensor(a[0])) || !matrix_ok(*logits, logits->device(), ld)) Py_RETURN_NONE;
    bool bad = false;
    const int top_k = as_int(a[1], bad), score = as_int(a[2], bad), type = type_code(*logits);
    const int renormalize = PyObject_IsTrue(a[3]);
    const double scale = PyFloat_AsDouble(a[4]);
    if ((scale == -1.0 && PyErr_Occurred()) || renormalize < 0) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const auto device = logits->device();
    const int64_t tokens = logits->size(0), experts = logits->size(1);
    if (bad || type < 0 || (score != QGEMV_SOFTMAX && score != QGEMV_SIGMOID) || tokens < 1 || tokens > INT32_MAX || experts < 1 ||
        experts > 1024 || top_k < 1 || top_k > 32 || top_k > experts || tokens * top_k > (1 << 30) || !std::isfinite((float)scale))
        Py_RETURN_NONE;
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor ws;
    if (!scratch(a[5], route_bytes_entry((int)tokens, (int)experts, top_k), device, ws)) Py_RETURN_NONE;
    at::Tensor ids = empty({tokens, top_k}, at::kInt, device), weights = empty({tokens, top_k}, at::kFloat, device);
    at::Tensor offsets = empty({experts + 1}, at::kInt, device), order = empty({tokens * top_k}, at::kInt, device);
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    const int status = unlocked([&] {
        return route_entry(type, logits->data_ptr(), ld, static_cast<int32_t*>(ids.data_ptr()),
                           static_cast<float*>(weights.data_ptr()), static_cast<int32_t*>(offsets.data_ptr()),
                           static_cast<int32_t*>(order.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                           ws.defined() ? (size_t)ws.numel() : 0, (int)tokens, (int)experts, top_k, score, renormalize,
                           (float)scale, stream);
    });
    if (status) return PyLong_FromLong(status);
    at::Tensor* made[4] = {&ids, &weights, &offsets, &order};
    PyObject* all = PyTuple_New(4);
    for (int i = 0; all && i < 4; ++i) {
        PyObject* one = THPVariable_Wrap(std::move(*made[i]));
        if (!one) Py_CLEAR(all);
        else PyTuple_SET_ITEM(all, i, one);
    }
    return all;
}

// product(which, w, w2 or None, x, offsets, order or None, weights or None, top_k, N, out or None, ws or None) -> status or
// out; which: 0 qgemm_mxfp4, 1 moe_gate_up_mxfp4, 2 moe_down_mxfp4
PyObject* call_product(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    const at::Tensor *w, *w2 = nullptr, *x, *offsets, *order = nullptr, *weights = nullptr;
    int64_t ldx, ldy;
    if (n_args != 11 || !(w = tensor(a[1])) || (a[2] != Py_None && !(w2 = tensor(a[2]))) || !(x = tensor(a[3])) ||
        !(offsets = tensor(a[4])) || (a[5] != Py_None && !(order = tensor(a[5]))) ||
        (a[6] != Py_None && !(weights = tensor(a[6]))) || !matrix_ok(*x, x->device(), ldx))
        Py_RETURN_NONE;
    bool bad = false;
    const int which = as_int(a[0], bad), top_k = as_int(a[7], bad), N = as_int(a[8], bad), type = type_code(*x);
    const auto device = x->device();
    const int64_t rows = x->size(0), K = x->size(1), experts = offsets->numel() - 1;
    if (bad || which < 0 || which > 2 || (which == 1) != (w2 != nullptr) || (which == 2) != (weights != nullptr) || type < 0 ||
        top_k < 1 || top_k > 32 || rows < 1 || K > INT32_MAX || offsets->dim() != 1 || experts < 1 || experts > 1024 ||
        !array_ok(*offsets, device, at::kInt, experts + 1) || (!order && top_k != 1))
        Py_RETURN_NONE;
    const int64_t tokens = which == 2 ? rows / top_k : rows, slots = tokens * top_k;
    const int64_t pack = (int64_t)pack_bytes_entry((int)experts, N, (int)K);
    if (slots > (1 << 30) || (which == 2 && (slots != rows || weights->dim() != 2 || weights->size(1) != top_k ||
                                             !array_ok(*weights, device, at::kFloat, slots))) ||
        pack == 0 || w->dim() != 1 || !array_ok(*w, device, at::kByte, pack) ||
        (w2 && (w2->dim() != 1 || !array_ok(*w2, device, at::kByte, pack))) ||
        (order && (order->dim() != 1 || !array_ok(*order, device, at::kInt, slots))))
        Py_RETURN_NONE;
    const int64_t out_rows = which == 2 ? tokens : slots;
    const c10::cuda::CUDAGuard guard(device);
    at::Tensor out, ws;
    if (a[9] == Py_None) {
        out = empty({out_rows, N}, x->scalar_type(), device);
        ldy = N;
    } else {
        const at::Tensor* given = tensor(a[9]);
        if (!given || !matrix_ok(*given, device, ldy) || given->size(0) != out_rows || given->size(1) != N ||
            given->scalar_type() != x->scalar_type())
            Py_RETURN_NONE;
        out = *given;
    }
    if (!scratch(a[10], product_bytes_entry[which](type, (int)tokens, top_k, (int)experts, (int)K, N), device, ws)) Py_RETURN_NONE;
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    const int status = unlocked([&] {
        const int32_t* at = static_cast<const int32_t*>(offsets->data_ptr());
        const int32_t* by = order ? static_cast<const int32_t*>(order->data_ptr()) : nullptr;
        void* memory = ws.defined() ? ws.data_ptr() : nullptr;
        const size_t bytes = ws.defined() ? (size_t)ws.numel() : 0;
        if (which == 0)
            return gemm_entry(type, w->data_ptr(), x->data_ptr(), ldx, at, by, out.data_ptr(), ldy, memory, bytes, (int)tokens,
                              top_k, (int)experts, (int)K, N, stream);
        if (which == 1)
            return gate_up_entry(type, w->data_ptr(), w2->data_ptr(), x->data_ptr(), ldx, at, by, out.data_ptr(), ldy, memory,
                                 bytes, (int)tokens, top_k, (int)experts, (int)K, N, stream);
        return down_entry(type, w->data_ptr(), x->data_ptr(), ldx, at, by, static_cast<const float*>(weights->data_ptr()),
                          out.data_ptr(), ldy, memory, bytes, (int)tokens, top_k, (int)experts, (int)K, N, stream);
    });
    if (status) return PyLong_FromLong(status);
    if (a[9] != Py_None) return Py_NewRef(a[9]);
    return THPVariable_Wrap(std::move(out));
}

// What throws (an allocation that fails) goes to the ctypes binding, which meets
// the same and raises it as torch does.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    try {
        return F(self, args, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// N addresses of entry points
template <int N>
bool addresses(PyObject* const* a, Py_ssize_t n_args, void* (&p)[N])
{
    if (n_args != N) {
        PyErr_Format(PyExc_TypeError, "%d addresses", N);
        return false;
    }
    for (int i = 0; i < N; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return false;
        }
    return true;
}

// init(addresses of kv_write, kv_read, attn_paged, kv_page_bytes, attn_paged_workspace_bytes)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    void* p[5];
    if (!addresses(a, n_args, p)) return nullptr;
    kv_write_entry = reinterpret_cast<decltype(kv_write_entry)>(p[0]);
    kv_read_entry = reinterpret_cast<decltype(kv_read_entry)>(p[1]);
    attn_entry = reinterpret_cast<decltype(attn_entry)>(p[2]);
    page_bytes_entry = reinterpret_cast<decltype(page_bytes_entry)>(p[3]);
    workspace_bytes_entry = reinterpret_cast<decltype(workspace_bytes_entry)>(p[4]);
    Py_RETURN_NONE;
}

// init_sparse(addresses of quantize_mxfp4, dequantize_mxfp4, moe_route, moe_route_workspace_bytes, mxfp4_pack_bytes,
//             qgemm_mxfp4, moe_gate_up_mxfp4, moe_down_mxfp4 and the three's workspace queries)
PyObject* init_sparse(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    void* p[11];
    if (!addresses(a, n_args, p)) return nullptr;
    quantize_entry = reinterpret_cast<decltype(quantize_entry)>(p[0]);
    dequantize_entry = reinterpret_cast<decltype(dequantize_entry)>(p[1]);
    route_entry = reinterpret_cast<decltype(route_entry)>(p[2]);
    route_bytes_entry = reinterpret_cast<decltype(route_bytes_entry)>(p[3]);
    pack_bytes_entry = reinterpret_cast<decltype(pack_bytes_entry)>(p[4]);
    gemm_entry = reinterpret_cast<decltype(gemm_entry)>(p[5]);
    gate_up_entry = reinterpret_cast<decltype(gate_up_entry)>(p[6]);
    down_entry = reinterpret_cast<decltype(down_entry)>(p[7]);
    for (int i = 0; i < 3; ++i) product_bytes_entry[i] = reinterpret_cast<decltype(&::qgemm_mxfp4_workspace_bytes)>(p[8 + i]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {{"init", FAST(init), METH_FASTCALL, nullptr},
                         {"init_sparse", FAST(init_sparse), METH_FASTCALL, nullptr},
                         {"kv_write", FAST(guarded<call_kv_write>), METH_FASTCALL, nullptr},
                         {"kv_read", FAST(guarded<call_kv_read>), METH_FASTCALL, nullptr},
                         {"attn_paged", FAST(guarded<call_attn_paged>), METH_FASTCALL, nullptr},
                         {"quantize_mxfp4", FAST(guarded<call_quantize>), METH_FASTCALL, nullptr},
                         {"dequantize_mxfp4", FAST(guarded<call_dequantize>), METH_FASTCALL, nullptr},
                         {"moe_route", FAST(guarded<call_route>), METH_FASTCALL, nullptr},
                         {"product", FAST(guarded<call_product>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qgemv_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qgemv_calls() { return PyModule_Create(&module); }
