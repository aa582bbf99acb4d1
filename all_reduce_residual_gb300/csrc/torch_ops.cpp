// torch_ops.cpp: the attention operators on torch tensors (the module
// _torch_ops behind attention.py). It checks shapes, dtypes, devices and
// strides, allocates outputs and scratch through torch's caching allocator
// and calls the C ABI of include/arf.h; no arithmetic happens here.
//
// Why not ctypes, as the rest of the binding: a decode step makes several of
// these calls per layer, with six to eight tensors each. On the host of a
// GB300 the marshalling of one call in Python took 22 to 28 us, ten times
// the kernel's time; here a call takes 2.4 us with its outputs given (1.6 of
// them the launch), 3.8 with outputs made; a page copy 2.9, and 0.04 more per
// layer beyond the first.
#include <ATen/core/Tensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/GradMode.h>
#include <c10/core/StorageImpl.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "arf.h"

namespace {

using at::ScalarType;
using at::Tensor;

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": a tensor is required");
    return THPVariable_Unpack(o);
}

// What an argument that is a C integer, or a handle's address, holds.
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int32_t integer32(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, ": ", v, " does not fit in 32 bits");
    return (int32_t)v;
}

arf_dtype_t io_dtype(const Tensor& t, const char* name) {
    if (t.scalar_type() == ScalarType::BFloat16) return ARF_BF16;
    TORCH_CHECK_VALUE(t.scalar_type() == ScalarType::Half, name, ": unsupported dtype ", t.scalar_type(),
                      ": bf16 or fp16");
    return ARF_FP16;
}

void on_device(const Tensor& t, const char* name, int device) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == device, name, " is on ", t.device(), ", expected cuda:", device);
}

// These calls record no gradients: a tensor that wants one is refused rather
// than left out of it without a word.
void no_gradient(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, which this call does not record: detach it, or call under torch.no_grad()");
}
// A given tensor was written: what autograd has saved of it is stale.
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* o) {
    if (!none(o)) written(THPVariable_Unpack(o));
}

// t [rows, heads, D]; sizes below 0 are free.
arf_heads_t heads(const Tensor& t, const char* name, ScalarType dtype, int device, int64_t rows = -1, int64_t n = -1,
                  int64_t D = -1) {
    TORCH_CHECK_VALUE(t.dim() == 3 && (rows < 0 || t.size(0) == rows) && (n < 0 || t.size(1) == n) &&
                          (D < 0 || t.size(2) == D),
                      name, ": shape ", t.sizes(), ", expected [rows, heads, D] that fit the other arguments");
    TORCH_CHECK_VALUE(t.scalar_type() == dtype, name, ": dtype ", t.scalar_type(), " != ", dtype);
    on_device(t, name, device);
    no_gradient(t, name);
    TORCH_CHECK_VALUE(t.stride(2) == 1 || t.size(2) <= 1, name, ": the elements of a head must be contiguous");
    TORCH_CHECK_VALUE(t.size(1) <= INT32_MAX, name, ": too many heads");
    return {t.data_ptr(), t.stride(0), t.stride(1), (int)t.size(1)};
}

const void* index(PyObject* o, const char* name, ScalarType dtype, int device, int64_t n) {
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.scalar_type() == dtype && t.dim() == 1 && t.size(0) == n, name, ": ", t.scalar_type(), " ",
                      t.sizes(), ", expected ", dtype, " [", n, "]");
    on_device(t, name, device);
    TORCH_CHECK_VALUE(n <= 1 || t.stride(0) == 1, name, " must be contiguous");
    return t.data_ptr();
}

// The stream of a call: the current one, or the given torch stream.
class Stream {
  public:
    Stream(PyObject* given, int device) : device_(device) {
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device);
        raw_ = current_ = current.stream();
        if (none(given)) return;
        PyObject* raw = PyObject_GetAttrString(given, "cuda_stream");
        if (!raw) throw python_error();
        raw_ = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
        Py_DECREF(raw);
        if (PyErr_Occurred()) throw python_error();
    }
    // Memory of torch's caching allocator, from the pool of the stream that
    // will write it: what was freed on another stream may still be in use by
    // work queued there. On the current device, or a given stream's (the
    // library refuses another device than the current one).
    c10::Storage memory(size_t bytes) const {
        if (raw_ == current_) return allocate(bytes);
        const c10::cuda::CUDAStreamGuard guard(of(raw_));
        return allocate(bytes);
    }
    // An output: it may also be read on the current stream, until it is freed.
    void shared(const Tensor& t) const {
        if (raw_ != current_ && t.defined()) t.record_stream(of(current_).unwrap());
    }
    void* raw() const { return raw_; }

  private:
    static c10::Storage allocate(size_t bytes) {
        c10::Allocator* allocator = c10::GetAllocator(c10::DeviceType::CUDA);
        return c10::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                                  allocator->allocate(bytes), allocator, true));
    }
    c10::cuda::CUDAStream of(cudaStream_t s) const {
        return c10::cuda::getStreamFromExternal(s, (c10::DeviceIndex)device_);
    }
    int device_;
    cudaStream_t raw_ = nullptr, current_ = nullptr;
};

// A contiguous tensor in memory of a call's stream. What torch.empty does,
// without its dispatch.
Tensor part(c10::Storage storage, at::IntArrayRef size, ScalarType dtype, size_t offset) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                     c10::scalarTypeToTypeMeta(dtype));
    impl->set_storage_offset((int64_t)(offset / c10::elementSize(dtype)));
    impl->set_sizes_contiguous(size);
    return Tensor(std::move(impl));
}
size_t bytes_of(at::IntArrayRef size, ScalarType dtype) {
    return (size_t)c10::multiply_integers(size) * c10::elementSize(dtype);
}
Tensor empty(const Stream& stream, at::IntArrayRef size, ScalarType dtype) {
    return part(stream.memory(bytes_of(size, dtype)), size, dtype, 0);
}

// Two contiguous tensors in one allocation, the second 256-byte aligned: the
// allocator's time per call is most of a small call's. They are views of one
// storage, as the parts of a fused projection are.
struct Pair {
    Tensor first, second;
};
Pair empty_pair(const Stream& stream, at::IntArrayRef size0, ScalarType dtype0, at::IntArrayRef size1,
                ScalarType dtype1) {
    const size_t at = (bytes_of(size0, dtype0) + 255) & ~(size_t)255;
    const c10::Storage all = stream.memory(at + bytes_of(size1, dtype1));
    return {part(all, size0, dtype0, 0), part(all, size1, dtype1, at)};
}

// The C struct behind a handle object of attention.py: its attribute `key`
// is a tuple (address of the struct, device index; of a cache also whether it
// may be written, and the tensors whose versions count what is written to its
// keys and to its values).
PyObject* kCacheKey = nullptr;  // the attributes' names, interned at import
PyObject* kTableKey = nullptr;

// The tuple (a borrowed reference: `o` holds it) and the struct's address.
struct Handle {
    PyObject* key;
    int64_t at;
};
Handle handle_of(PyObject* o, PyObject* name, Py_ssize_t size, const char* what, int device) {
    PyObject* key = PyObject_GetAttr(o, name);
    if (!key) {
        PyErr_Clear();
        TORCH_CHECK_VALUE(false, "a ", what, " is required");
    }
    Py_DECREF(key);
    const bool fits = PyTuple_Check(key) && PyTuple_GET_SIZE(key) == size;
    const int64_t at = fits ? PyLong_AsLongLong(PyTuple_GET_ITEM(key, 0)) : 0;
    const int64_t dev = fits ? PyLong_AsLongLong(PyTuple_GET_ITEM(key, 1)) : -1;
    if (PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(at != 0, "a ", what, " is required");
    TORCH_CHECK_VALUE(dev == device, "the ", what, " is on device ", dev, ", expected cuda:", device);
    return {key, at};
}
struct Cache {
    const arf_kv_cache_t* c;
    PyObject* key;
    void check_writable() const {
        TORCH_CHECK_VALUE(PyTuple_GET_ITEM(key, 2) == Py_True,
                          "the KVCache's keys and values share elements: it can only be read");
    }
    PyObject* base(int i) const { return PyTuple_GET_ITEM(key, 3 + i); }
    const arf_kv_cache_t* operator->() const { return c; }
};
Cache cache_of(PyObject* o, int device) {
    const Handle h = handle_of(o, kCacheKey, 5, "KVCache", device);
    return {reinterpret_cast<const arf_kv_cache_t*>(h.at), h.key};
}
const arf_rotary_t* rotary_of(PyObject* o, int device) {
    return reinterpret_cast<const arf_rotary_t*>(handle_of(o, kTableKey, 2, "RotaryTable", device).at);
}

// A closed Workspace's handle is None: the library refuses a null workspace.
arf_workspace_t workspace(PyObject* o) { return none(o) ? nullptr : reinterpret_cast<arf_workspace_t>(integer(o)); }

void arguments(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_VALUE(got == want, got, " arguments, expected ", want); }

PyObject* status(arf_status_t st) { return PyLong_FromLong((long)st); }

// rotary(ws, device, q, k, positions, table, q_out, k_out, stream)
// -> (q_out, k_out), or the status of a call that was refused
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 9);
    const int device = (int)integer(a[1]);
    const Tensor& q = tensor(a[2], "q");
    const arf_dtype_t dt = io_dtype(q, "q");
    const ScalarType st = q.scalar_type();
    const arf_heads_t qh = heads(q, "q", st, device);
    const int64_t T = q.size(0), D = q.size(2);
    TORCH_CHECK_VALUE(D <= INT32_MAX, "q: D is too large");
    const void* pos = index(a[4], "positions", ScalarType::Int, device, T);
    const arf_rotary_t* table = rotary_of(a[5], device);
    const Stream stream(a[8], device);
    const bool has_k = !none(a[3]);
    arf_heads_t kh = {}, ko = {};
    if (has_k) kh = heads(tensor(a[3], "k"), "k", st, device, T, -1, D);
    Tensor q_out, k_out;
    arf_heads_t qo;
    if (none(a[6])) {
        if (has_k && none(a[7])) {
            Pair made = empty_pair(stream, q.sizes(), st, tensor(a[3], "k").sizes(), st);
            q_out = std::move(made.first), k_out = std::move(made.second);
        } else {
            q_out = empty(stream, q.sizes(), st);
        }
        qo = {q_out.data_ptr(), qh.heads * D, D, qh.heads};
    } else {
        qo = heads(tensor(a[6], "q_out"), "q_out", st, device, T, qh.heads, D);
    }
    if (has_k) {
        if (none(a[7])) {
            if (!k_out.defined()) k_out = empty(stream, tensor(a[3], "k").sizes(), st);
            ko = {k_out.data_ptr(), kh.heads * D, D, kh.heads};
        } else {
            ko = heads(tensor(a[7], "k_out"), "k_out", st, device, T, kh.heads, D);
        }
    } else {
        TORCH_CHECK_VALUE(none(a[7]), "k_out without k");
    }
    stream.shared(q_out);
    stream.shared(k_out);
    const arf_status_t r = arf_rotary(workspace(a[0]), table, static_cast<const int32_t*>(pos), T, (int)D, dt, &qh, &qo,
                                      has_k ? &kh : nullptr, has_k ? &ko : nullptr, stream.raw());
    if (r != ARF_OK) return status(r);
    written(a[6]);
    written(a[7]);
    PyObject* out = PyTuple_New(2);
    if (!out) throw python_error();
    PyObject* first = a[6];
    PyObject* second = has_k ? a[7] : Py_None;
    if (q_out.defined()) first = THPVariable_Wrap(std::move(q_out)); else Py_INCREF(first);
    if (k_out.defined()) second = THPVariable_Wrap(std::move(k_out)); else Py_INCREF(second);
    PyTuple_SET_ITEM(out, 0, first);
    PyTuple_SET_ITEM(out, 1, second);
    return out;
    END_HANDLE_TH_ERRORS
}

// rotary_append(ws, device, q, k, v, positions, slots, table, cache, q_out, stream)
// -> q_out (or None), or the status
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 11);
    const int device = (int)integer(a[1]);
    const Tensor& k = tensor(a[3], "k");
    const arf_dtype_t dt = io_dtype(k, "k");
    const ScalarType st = k.scalar_type();
    const Cache cache = cache_of(a[8], device);
    cache.check_writable();
    TORCH_CHECK_VALUE(k.dim() == 3, "k: shape ", k.sizes(), ", expected [rows, heads, D]");
    const int64_t T = k.size(0), D = cache->head_dim;
    const arf_heads_t kh = heads(k, "k", st, device, T, cache->kv_heads, D);
    const arf_heads_t vh = heads(tensor(a[4], "v"), "v", st, device, T, cache->kv_heads, D);
    const void* slots = index(a[6], "slots", ScalarType::Long, device, T);
    const arf_rotary_t* table = none(a[7]) ? nullptr : rotary_of(a[7], device);
    const bool has_q = !none(a[2]);
    TORCH_CHECK_VALUE(table || (!has_q && none(a[5])),
                      "without a rotary table only k and v are appended: q and positions must be None");
    TORCH_CHECK_VALUE(has_q || none(a[9]), "q_out without q");
    const void* pos = table ? index(a[5], "positions", ScalarType::Int, device, T) : nullptr;
    const Stream stream(a[10], device);
    arf_heads_t qh = {}, qo = {};
    Tensor q_out;
    if (has_q) {
        const Tensor& q = tensor(a[2], "q");
        qh = heads(q, "q", st, device, T, -1, D);
        if (none(a[9])) {
            q_out = empty(stream, q.sizes(), st);
            qo = {q_out.data_ptr(), qh.heads * D, D, qh.heads};
            stream.shared(q_out);
        } else {
            qo = heads(tensor(a[9], "q_out"), "q_out", st, device, T, qh.heads, D);
        }
    }
    const arf_status_t r = arf_rotary_append(workspace(a[0]), table, static_cast<const int32_t*>(pos),
                                             static_cast<const int64_t*>(slots), T, dt, has_q ? &qh : nullptr,
                                             has_q ? &qo : nullptr, &kh, &vh, cache.c, stream.raw());
    if (r != ARF_OK) return status(r);
    written(a[9]);
    for (int i = 0; i < 2; ++i) written(tensor(cache.base(i), "pages"));
    if (q_out.defined()) return THPVariable_Wrap(std::move(q_out));
    PyObject* out = has_q ? a[9] : Py_None;
    Py_INCREF(out);
    return out;
    END_HANDLE_TH_ERRORS
}

// paged_decode(ws, device, q, cache, block_table, lens, scale, softcap, window, out, lse, stream)
// -> (out, lse), or the status
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 12);
    const int device = (int)integer(a[1]);
    const Tensor& q = tensor(a[2], "q");
    const arf_dtype_t dt = io_dtype(q, "q");
    const ScalarType st = q.scalar_type();
    const Cache cache = cache_of(a[3], device);
    const arf_heads_t qh = heads(q, "q", st, device);
    const int64_t B = q.size(0), D = q.size(2);
    TORCH_CHECK_VALUE(D == cache->head_dim && cache->kv_heads > 0 && qh.heads % cache->kv_heads == 0, "q: ", qh.heads,
                      " heads of ", D, " do not fit a cache with ", cache->kv_heads, " of ", cache->head_dim);
    const Tensor& table = tensor(a[4], "block_table");
    TORCH_CHECK_VALUE(table.scalar_type() == ScalarType::Int && table.dim() == 2 && table.size(0) == B, "block_table: ",
                      table.scalar_type(), " ", table.sizes(), ", expected int32 [", B, ", pages]");
    on_device(table, "block_table", device);
    const int64_t width = table.size(1);
    TORCH_CHECK_VALUE(width <= 1 || table.stride(1) == 1, "block_table: rows must be contiguous");
    TORCH_CHECK_VALUE(width <= INT32_MAX, "block_table is too wide");
    const void* lens = index(a[5], "lens", ScalarType::Int, device, B);
    const float scale = none(a[6]) ? (float)(1.0 / std::sqrt((double)D)) : (float)real(a[6]);
    const float cap = (float)real(a[7]);
    const int32_t window = integer32(a[8], "window");
    const Stream stream(a[11], device);
    Tensor out, lse;
    arf_heads_t oh;
    if (none(a[9])) {
        if (none(a[10])) {
            Pair made = empty_pair(stream, q.sizes(), st, {B, (int64_t)qh.heads}, ScalarType::Float);
            out = std::move(made.first), lse = std::move(made.second);
        } else {
            out = empty(stream, q.sizes(), st);
        }
        oh = {out.data_ptr(), qh.heads * D, D, qh.heads};
        stream.shared(out);
    } else {
        oh = heads(tensor(a[9], "out"), "out", st, device, B, qh.heads, D);
    }
    float* lse_ptr;
    if (none(a[10])) {
        if (!lse.defined()) lse = empty(stream, {B, qh.heads}, ScalarType::Float);
        lse_ptr = static_cast<float*>(lse.data_ptr());
        stream.shared(lse);
    } else {
        const Tensor& l = tensor(a[10], "lse");
        TORCH_CHECK_VALUE(l.scalar_type() == ScalarType::Float && l.dim() == 2 && l.size(0) == B &&
                              l.size(1) == qh.heads && l.is_contiguous(),
                          "lse: contiguous float32 [", B, ", ", qh.heads, "] expected");
        on_device(l, "lse", device);
        no_gradient(l, "lse");
        lse_ptr = static_cast<float*>(l.data_ptr());
    }
    // scratch of the caching allocator (512-byte aligned), from the pool of
    // the call's stream: work before and after it there may use the same
    // memory, work on other streams may not
    size_t bytes = 0;
    const arf_status_t need =
        arf_paged_decode_scratch_bytes(workspace(a[0]), cache.c, B, qh.heads, (int32_t)width, window, &bytes);
    if (need != ARF_OK) return status(need);
    Tensor scratch;
    if (bytes > 0) scratch = empty(stream, {(int64_t)bytes}, ScalarType::Byte);
    const arf_status_t r =
        arf_paged_decode(workspace(a[0]), cache.c, B, dt, &qh, static_cast<const int32_t*>(table.data_ptr()),
                         B > 1 ? table.stride(0) : width, (int32_t)width, static_cast<const int32_t*>(lens), scale, cap,
                         window, &oh, lse_ptr, bytes > 0 ? scratch.data_ptr() : nullptr, bytes, stream.raw());
    if (r != ARF_OK) return status(r);
    written(a[9]);
    written(a[10]);
    PyObject* pair = PyTuple_New(2);
    if (!pair) throw python_error();
    PyObject* first = a[9];
    PyObject* second = a[10];
    if (out.defined()) first = THPVariable_Wrap(std::move(out)); else Py_INCREF(first);
    if (lse.defined()) second = THPVariable_Wrap(std::move(lse)); else Py_INCREF(second);
    PyTuple_SET_ITEM(pair, 0, first);
    PyTuple_SET_ITEM(pair, 1, second);
    return pair;
    END_HANDLE_TH_ERRORS
}

// Page numbers: a CPU int32 tensor or a sequence of integers.
std::vector<int32_t> page_numbers(PyObject* o, const char* name) {
    std::vector<int32_t> v;
    if (THPVariable_Check(o)) {
        const Tensor& t = THPVariable_Unpack(o);
        TORCH_CHECK_VALUE(t.scalar_type() == ScalarType::Int && t.dim() == 1 && t.device().is_cpu(), name,
                          ": page numbers as a sequence or a CPU int32 tensor");
        const int32_t* p = static_cast<const int32_t*>(t.data_ptr());
        const int64_t step = t.stride(0);
        v.resize((size_t)t.size(0));
        for (size_t i = 0; i < v.size(); ++i) v[i] = p[(int64_t)i * step];
        return v;
    }
    PyObject* seq = PySequence_Fast(o, "page numbers as a sequence or a CPU int32 tensor");
    if (!seq) throw python_error();
    try {
        v.resize((size_t)PySequence_Fast_GET_SIZE(seq));
        for (size_t i = 0; i < v.size(); ++i) v[i] = integer32(PySequence_Fast_GET_ITEM(seq, (Py_ssize_t)i), name);
    } catch (...) {
        Py_DECREF(seq);
        throw;
    }
    Py_DECREF(seq);
    return v;
}

// copy_pages(ws, device, caches (a list or tuple), src, dst, stream) -> status
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const int device = (int)integer(a[1]);
    TORCH_CHECK_VALUE(PyList_Check(a[2]) || PyTuple_Check(a[2]), "caches: a list or a tuple");
    std::vector<arf_kv_cache_t> caches;
    std::vector<Cache> handles;
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[2]);
    TORCH_CHECK_VALUE(count > 0, "at least one cache is required");
    TORCH_CHECK_VALUE(count <= INT32_MAX, "too many caches");
    caches.reserve((size_t)count);
    handles.reserve((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        handles.push_back(cache_of(PySequence_Fast_GET_ITEM(a[2], i), device));
        handles.back().check_writable();
        caches.push_back(*handles.back().c);
    }
    const std::vector<int32_t> src = page_numbers(a[3], "src"), dst = page_numbers(a[4], "dst");
    TORCH_CHECK_VALUE(src.size() == dst.size(), src.size(), " sources and ", dst.size(), " destinations");
    TORCH_CHECK_VALUE(src.size() <= INT32_MAX, "too many pages");
    const Stream stream(a[5], device);
    const arf_status_t r = arf_copy_pages(workspace(a[0]), caches.data(), (int)count, src.data(), dst.data(),
                                          (int)src.size(), stream.raw());
    if (r != ARF_OK) return status(r);
    PyObject* last[2] = {nullptr, nullptr};  // layers are often views of one tensor
    for (const Cache& cache : handles)
        for (int i = 0; i < 2; ++i)
            if (cache.base(i) != last[i]) written(tensor(last[i] = cache.base(i), "pages"));
    return status(r);
    END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef kMethods[] = {{"rotary", fast(rotary), METH_FASTCALL, nullptr},
                          {"rotary_append", fast(rotary_append), METH_FASTCALL, nullptr},
                          {"paged_decode", fast(paged_decode), METH_FASTCALL, nullptr},
                          {"copy_pages", fast(copy_pages), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_ops", "The attention operators on torch tensors.", -1, kMethods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__torch_ops() {
    kCacheKey = PyUnicode_InternFromString("_cache_key");
    kTableKey = PyUnicode_InternFromString("_table_key");
    return kCacheKey && kTableKey ? PyModule_Create(&kModule) : nullptr;
}
