// The paged cache's calls from Python without Python's share of the work: reads
// the tensors, checks them, makes their device the current one, allocates the outputs
// and calls the library.  A call that it would refuse, or whose tensors it does not
// know how to take, returns None and goes through the ctypes binding (_lib.py), which
// does the same and says what is wrong.  Only host code: the kernels are the
// library's, by the addresses of its entry points that init() gets.  A call of
// attn_paged takes the host 7 us, of kv_read with new outputs 5 and of kv_write 2, by
// ctypes 20, 15 and 8, beside 2 to 10 us of kernels on small inputs.
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

// init(addresses of kv_write, kv_read, attn_paged, kv_page_bytes, attn_paged_workspace_bytes)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n_args)
{
    void* p[5];
    if (n_args != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    for (int i = 0; i < 5; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    kv_write_entry = reinterpret_cast<decltype(kv_write_entry)>(p[0]);
    kv_read_entry = reinterpret_cast<decltype(kv_read_entry)>(p[1]);
    attn_entry = reinterpret_cast<decltype(attn_entry)>(p[2]);
    page_bytes_entry = reinterpret_cast<decltype(page_bytes_entry)>(p[3]);
    workspace_bytes_entry = reinterpret_cast<decltype(workspace_bytes_entry)>(p[4]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {{"init", FAST(init), METH_FASTCALL, nullptr},
                         {"kv_write", FAST(guarded<call_kv_write>), METH_FASTCALL, nullptr},
                         {"kv_read", FAST(guarded<call_kv_read>), METH_FASTCALL, nullptr},
                         {"attn_paged", FAST(guarded<call_attn_paged>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qgemv_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qgemv_calls() { return PyModule_Create(&module); }
