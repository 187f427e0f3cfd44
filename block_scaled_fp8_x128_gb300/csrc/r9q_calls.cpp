// The Python side of the attention block's calls (QK norm with rotation, the 4-bit
// cache, the attention over it): checks of the tensors and the C call.
//
// These kernels run for a few microseconds, as long as a dozen attribute reads in
// Python take, so the checks are made here, on the tensors themselves.  Nothing else
// is: each function takes its arguments by position, makes the outputs that are None
// and calls the entry point of include/r9q.h of the same name.  It returns the outputs,
// or the entry point's code as an int where that is not 0, or one of the codes below where
// the call has to be made another way (nothing has been done then); a tensor of the wrong type,
// shape, layout or device raises as the rest of the binding does.  The caller has made the
// tensors' device and the call's stream the current ones.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>
#include <initializer_list>

#include "r9q.h"

namespace {

struct Raised {};            // a Python error is set

// The call is to be recorded by autograd.
constexpr int kRecorded = 1;
// The stream is being captured, and the workspace is not the caller's own: the capture needs one of its own.
constexpr int kCaptured = 2;

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

using Shape = std::initializer_list<int64_t>;

// Type and shape, and that the tensor is on `device`.
const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type, Shape shape, at::Device device) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s: tensor must be on a CUDA device", name);
    if (t.device() != device) raise(PyExc_ValueError, "%s: tensor is on another device than the others", name);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    const at::IntArrayRef have = t.sizes(), want(shape.begin(), shape.size());
    if (have != want) {
        std::string a, b;
        for (int64_t n : want) a += (a.empty() ? "" : ", ") + std::to_string(n);
        for (int64_t n : have) b += (b.empty() ? "" : ", ") + std::to_string(n);
        raise(PyExc_ValueError, "%s: expected shape (%s), got (%s)", name, a.c_str(), b.c_str());
    }
    return t;
}

// The address of a contiguous tensor; null for None.
void* address(PyObject* o, const char* name, at::ScalarType type, Shape shape, at::Device device) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = checked(o, name, type, shape, device);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: tensor must be contiguous", name);
    return t.data_ptr();
}

// A bf16 [T][H][D] tensor with contiguous vectors: its address, token and head strides.
struct Heads {
    void* p;
    int64_t ts, hs;
};
Heads heads(PyObject* o, const char* name, Shape shape, at::Device device) {
    const at::Tensor& t = checked(o, name, at::kBFloat16, shape, device);
    if (t.size(2) > 1 && t.stride(2) != 1)
        raise(PyExc_ValueError, "%s: the last dimension must be contiguous", name);
    return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// Sizes of a tensor of `dims` dimensions.
at::IntArrayRef sizes(const at::Tensor& t, const char* name, int dims) {
    if (t.dim() != dims) raise(PyExc_ValueError, "%s: expected %d dimensions, got %d", name, dims, (int)t.dim());
    return t.sizes();
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}
void* stream(PyObject* o) { return reinterpret_cast<void*>(integer(o)); }

// New contiguous tensors of the current stream from torch's allocator, without the dispatcher.  Those of one call that live together share an
// allocation: each costs about a microsecond, as much as all checks of a call.
using Storage = c10::intrusive_ptr<c10::StorageImpl>;
size_t elements(at::IntArrayRef shape) {
    size_t n = 1;
    for (int64_t s : shape) n *= (size_t)s;
    return n;
}
Storage allocate(size_t bytes, at::Device device) {
    const c10::DeviceGuard guard(device);
    return c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                 c10::GetAllocator(device.type()), /*resizable=*/true);
}
PyObject* part(Storage storage, size_t from, at::ScalarType type, at::IntArrayRef shape) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset((int64_t)from);
    return THPVariable_Wrap(std::move(t));
}
// An output: the caller's, or a new one.  A new reference.
PyObject* output(PyObject* o, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
    if (o != Py_None) return Py_NewRef(o);
    return part(allocate(elements(shape) * c10::elementSize(type), device), 0, type, shape);
}
// Outputs that are let go unless they are returned.
struct Outputs {
    PyObject* o[4] = {};
    int n = 0;
    ~Outputs() {
        for (int i = 0; i < n; ++i) Py_XDECREF(o[i]);
    }
    PyObject* add(PyObject* x) { return o[n++] = x; }
    // Two: the caller's, or both new, of one allocation.
    void add(PyObject* a, at::IntArrayRef a_shape, at::ScalarType a_type, PyObject* b, at::IntArrayRef b_shape,
             at::ScalarType b_type, at::Device device) {
        if (a != Py_None || b != Py_None) {
            add(output(a, a_type, a_shape, device));
            add(output(b, b_type, b_shape, device));
            return;
        }
        const size_t size = c10::elementSize(b_type);
        const size_t from = (elements(a_shape) * c10::elementSize(a_type) + 255) / 256 * (256 / size);
        const Storage storage = allocate((from + elements(b_shape)) * size, device);
        add(part(storage, 0, a_type, a_shape));
        add(part(storage, from, b_type, b_shape));
    }
    PyObject* done(int rc) {
        if (rc) return PyLong_FromLong(rc);
        if (n == 0) Py_RETURN_NONE;
        if (n == 1) return Py_NewRef(o[0]);
        PyObject* t = PyTuple_New(n);
        if (!t) throw Raised();
        for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(t, i, Py_NewRef(o[i]));
        return t;
    }
};

// Weights, tables and positions, from five consecutive arguments (wq, wk, cos, sin, positions).
struct Rope {
    const float *wq, *wk, *cos, *sin;
    const int64_t* pos;
    int64_t rot, npos;
};
Rope rope(PyObject* const* a, int64_t T, int64_t D, at::Device device) {
    Rope r = {};
    r.wq = static_cast<const float*>(address(a[0], "wq", at::kFloat, {D}, device));
    r.wk = static_cast<const float*>(address(a[1], "wk", at::kFloat, {D}, device));
    if (a[2] == Py_None) return r;
    const at::IntArrayRef table = sizes(tensor(a[2], "cos"), "cos", 2);
    r.npos = table[0];
    r.rot = 2 * table[1];
    r.cos = static_cast<const float*>(address(a[2], "cos", at::kFloat, {table[0], table[1]}, device));
    r.sin = static_cast<const float*>(address(a[3], "sin", at::kFloat, {table[0], table[1]}, device));
    r.pos = static_cast<const int64_t*>(address(a[4], "positions", at::kLong, {T}, device));
    return r;
}

// The cache, from four consecutive arguments (k, kp, v, vp).
struct Cache {
    uint8_t *k, *v;
    void *kp, *vp;
    int64_t pages, heads, page, dim;
};
Cache cache(PyObject* const* a, at::Device device) {
    const at::IntArrayRef s = sizes(tensor(a[0], "cache.k"), "cache.k", 4);
    Cache c = {};
    c.pages = s[0];
    c.heads = s[1];
    c.page = s[2];
    c.dim = 2 * s[3];
    const Shape codes = {s[0], s[1], s[2], s[3]}, pairs = {s[0], s[1], s[2], 2};
    c.k = static_cast<uint8_t*>(address(a[0], "cache.k", at::kByte, codes, device));
    c.kp = address(a[1], "cache.kp", at::kBFloat16, pairs, device);
    c.v = static_cast<uint8_t*>(address(a[2], "cache.v", at::kByte, codes, device));
    c.vp = address(a[3], "cache.vp", at::kBFloat16, pairs, device);
    return c;
}
void fits(const Cache& c, int64_t heads, int64_t dim) {
    if (c.heads != heads || c.dim != dim)
        raise(PyExc_ValueError, "cache: expected %lld heads of %lld, got %lld of %lld", (long long)heads,
              (long long)dim, (long long)c.heads, (long long)c.dim);
}

struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
};
Workspace workspace(PyObject* o, at::Device device) {
    Workspace w;
    if (o == Py_None) return w;
    const at::Tensor& t = tensor(o, "workspace");
    if (t.device() != device || !t.is_contiguous())
        raise(PyExc_ValueError, "workspace: must be contiguous and on the tensors' device");
    w.p = t.data_ptr();
    w.bytes = t.nbytes();
    return w;
}

bool captured(PyObject* theirs, PyObject* on) {          // not the caller's workspace, on a stream that is captured
    unsigned long long id = 0;
    return !truth(theirs) && r9q_stream_capture_id(stream(on), &id) == R9Q_OK && id != 0;
}

// ---- the calls ----
// workspace, theirs: the workspace, and whether it is the caller's own.

// q, k, wq, wk, cos, sin, positions, eps, interleaved, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const at::Device dev = q.device();
    const at::IntArrayRef s = sizes(q, "q", 3), ks = sizes(k, "k", 3);
    const int64_t T = s[0], Hq = s[1], D = s[2], Hk = ks[1];
    const Heads qh = heads(a[0], "q", {T, Hq, D}, dev), kh = heads(a[1], "k", {T, Hk, D}, dev);
    const Rope r = rope(a + 2, T, D, dev);
    if (a[9] == Py_None && a[10] == Py_None && c10::GradMode::is_enabled() &&
        (q.requires_grad() || k.requires_grad() || tensor(a[2], "wq").requires_grad() || tensor(a[3], "wk").requires_grad()))
        return PyLong_FromLong(kRecorded);
    Outputs out;
    out.add(a[9], s, at::kBFloat16, a[10], ks, at::kBFloat16, dev);
    const Heads qo = heads(out.o[0], "q_out", {T, Hq, D}, dev), ko = heads(out.o[1], "k_out", {T, Hk, D}, dev);
    return out.done(r9q_qk_norm_rope(qh.p, qh.ts, qh.hs, kh.p, kh.ts, kh.hs, r.wq, r.wk, r.cos, r.sin, r.pos, qo.p, qo.ts,
                                     qo.hs, ko.p, ko.ts, ko.hs, T, Hq, Hk, D, r.rot, r.npos, number(a[7]),
                                     truth(a[8]) ? R9Q_ROPE_INTERLEAVED : 0, stream(a[11])));
}

// dq_out, dk_out, q, k, wq, wk, cos, sin, positions, eps, interleaved, dq, dk, dwq, dwk, workspace, theirs, stream
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
    if (captured(a[16], a[17])) return PyLong_FromLong(kCaptured);
    const at::Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k");
    const at::Device dev = q.device();
    const at::IntArrayRef s = sizes(q, "q", 3), ks = sizes(k, "k", 3);
    const int64_t T = s[0], Hq = s[1], D = s[2], Hk = ks[1];
    const Heads gq = heads(a[0], "dq_out", {T, Hq, D}, dev), gk = heads(a[1], "dk_out", {T, Hk, D}, dev);
    const Heads qh = heads(a[2], "q", {T, Hq, D}, dev), kh = heads(a[3], "k", {T, Hk, D}, dev);
    const Rope r = rope(a + 4, T, D, dev);
    const Workspace w = workspace(a[15], dev);
    Outputs out;
    out.add(a[11], s, at::kBFloat16, a[12], ks, at::kBFloat16, dev);
    out.add(a[13], {D}, at::kFloat, a[14], {D}, at::kFloat, dev);
    const Heads dq = heads(out.o[0], "dq", {T, Hq, D}, dev), dk = heads(out.o[1], "dk", {T, Hk, D}, dev);
    float* dwq = static_cast<float*>(address(out.o[2], "dwq", at::kFloat, {D}, dev));
    float* dwk = static_cast<float*>(address(out.o[3], "dwk", at::kFloat, {D}, dev));
    return out.done(r9q_qk_norm_rope_bwd(gq.p, gq.ts, gq.hs, gk.p, gk.ts, gk.hs, qh.p, qh.ts, qh.hs, kh.p, kh.ts, kh.hs,
                                         r.wq, r.wk, r.cos, r.sin, r.pos, dq.p, dq.ts, dq.hs, dk.p, dk.ts, dk.hs, dwq,
                                         dwk, T, Hq, Hk, D, r.rot, r.npos, number(a[9]),
                                         truth(a[10]) ? R9Q_ROPE_INTERLEAVED : 0, w.p, w.bytes, stream(a[17])));
}

// q, k, v, wq, wk, cos, sin, positions, cache.k, .kp, .v, .vp, slots, eps, interleaved, q_out, stream
PyObject* qk_norm_rope_kv4(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const at::Device dev = q.device();
    const at::IntArrayRef s = sizes(q, "q", 3), ks = sizes(k, "k", 3);
    const int64_t T = s[0], Hq = s[1], D = s[2], Hk = ks[1];
    const Heads qh = heads(a[0], "q", {T, Hq, D}, dev), kh = heads(a[1], "k", {T, Hk, D}, dev);
    const Heads vh = heads(a[2], "v", {T, Hk, D}, dev);
    const Rope r = rope(a + 3, T, D, dev);
    const Cache c = cache(a + 8, dev);
    fits(c, Hk, D);
    const int64_t* slots = static_cast<const int64_t*>(address(a[12], "slots", at::kLong, {T}, dev));
    Outputs out;
    const Heads qo = heads(out.add(output(a[15], at::kBFloat16, s, dev)), "q_out", {T, Hq, D}, dev);
    return out.done(r9q_qk_norm_rope_kv4(qh.p, qh.ts, qh.hs, kh.p, kh.ts, kh.hs, vh.p, vh.ts, vh.hs, r.wq, r.wk, r.cos,
                                         r.sin, r.pos, qo.p, qo.ts, qo.hs, c.k, c.kp, c.v, c.vp, slots, T, Hq, Hk, D,
                                         r.rot, r.npos, c.pages, c.page, number(a[13]),
                                         truth(a[14]) ? R9Q_ROPE_INTERLEAVED : 0, stream(a[16])));
}

// k, v, cache.k, .kp, .v, .vp, slots, stream
PyObject* kv4_append(PyObject* const* a) {
    const at::Tensor& k = tensor(a[0], "k");
    const at::Device dev = k.device();
    const at::IntArrayRef s = sizes(k, "k", 3);
    const int64_t T = s[0], Hk = s[1], D = s[2];
    const Heads kh = heads(a[0], "k", {T, Hk, D}, dev), vh = heads(a[1], "v", {T, Hk, D}, dev);
    const Cache c = cache(a + 2, dev);
    fits(c, Hk, D);
    const int64_t* slots = static_cast<const int64_t*>(address(a[6], "slots", at::kLong, {T}, dev));
    return Outputs().done(r9q_kv4_append(kh.p, kh.ts, kh.hs, vh.p, vh.ts, vh.hs, c.k, c.kp, c.v, c.vp, slots, T, Hk, D,
                                         c.pages, c.page, stream(a[7])));
}

// cache.k, .kp, .v, .vp, slots, k, v, stream
PyObject* kv4_gather(PyObject* const* a) {
    const at::Tensor& at_slots = tensor(a[4], "slots");
    const at::Device dev = at_slots.device();
    const int64_t T = sizes(at_slots, "slots", 1)[0];
    const Cache c = cache(a, dev);
    const int64_t* slots = static_cast<const int64_t*>(address(a[4], "slots", at::kLong, {T}, dev));
    const Shape shape = {T, c.heads, c.dim};
    Outputs out;
    out.add(a[5], shape, at::kBFloat16, a[6], shape, at::kBFloat16, dev);
    void* k = address(out.o[0], "k", at::kBFloat16, shape, dev);
    void* v = address(out.o[1], "v", at::kBFloat16, shape, dev);
    return out.done(r9q_kv4_gather(c.k, c.kp, c.v, c.vp, slots, T, c.heads, c.dim, c.pages, c.page, k, v, stream(a[7])));
}

// q, cache.k, .kp, .v, .vp, block_table, seq_lens, scale, window, out, lse, return_lse, workspace, theirs, stream
PyObject* kv4_attention(PyObject* const* a) {
    if (captured(a[13], a[14])) return PyLong_FromLong(kCaptured);
    const at::Tensor& q = tensor(a[0], "q");
    const at::Device dev = q.device();
    const at::IntArrayRef s = sizes(q, "q", 4);
    const int64_t B = s[0], Lq = s[1], Hq = s[2], D = s[3];
    checked(a[0], "q", at::kBFloat16, {B, Lq, Hq, D}, dev);
    if (D > 1 && q.stride(3) != 1) raise(PyExc_ValueError, "q: the last dimension must be contiguous");
    const Cache c = cache(a + 1, dev);
    fits(c, c.heads, D);
    if (c.heads < 1 || Hq % c.heads) raise(PyExc_ValueError, "q's heads must be a multiple of the cache's");
    const int64_t width = sizes(tensor(a[5], "block_table"), "block_table", 2)[1];
    const int32_t* table = static_cast<const int32_t*>(address(a[5], "block_table", at::kInt, {B, width}, dev));
    const int32_t* lens = static_cast<const int32_t*>(address(a[6], "seq_lens", at::kInt, {B}, dev));
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : number(a[7]);
    const Workspace w = workspace(a[12], dev);
    const bool with_lse = truth(a[11]);
    Outputs out;
    if (with_lse)
        out.add(a[9], s, at::kBFloat16, a[10], {B, Lq, Hq}, at::kFloat, dev);
    else
        out.add(output(a[9], at::kBFloat16, s, dev));
    void* o = address(out.o[0], "out", at::kBFloat16, {B, Lq, Hq, D}, dev);
    float* lse = static_cast<float*>(address(with_lse ? out.o[1] : a[10], "lse", at::kFloat, {B, Lq, Hq}, dev));
    return out.done(r9q_kv4_attention(q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), c.k, c.kp, c.v, c.vp, table,
                                      lens, o, lse, B, Lq, Hq, c.heads, D, c.pages, c.page, width, integer(a[8]), scale,
                                      w.p, w.bytes, stream(a[14])));
}

template <PyObject* (*CALL)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return CALL(args);
    } catch (const Raised&) {
        return nullptr;
    } catch (const c10::OutOfMemoryError& e) {   // as torch raises it: torch.OutOfMemoryError
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
        return nullptr;
    } catch (const std::exception& e) {          // another of torch's own
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}
template <PyObject* (*CALL)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<CALL, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<qk_norm_rope, 12>("qk_norm_rope"),
                           method<qk_norm_rope_bwd, 18>("qk_norm_rope_bwd"),
                           method<qk_norm_rope_kv4, 17>("qk_norm_rope_kv4"),
                           method<kv4_append, 8>("kv4_append"),
                           method<kv4_gather, 8>("kv4_gather"),
                           method<kv4_attention, 15>("kv4_attention"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
    PyObject* m = PyModule_Create(&g_module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", R9Q_TORCH_VERSION) ||                  // what it was built for
              PyModule_AddIntConstant(m, "RECORDED", kRecorded) || PyModule_AddIntConstant(m, "CAPTURED", kCaptured)))
        Py_CLEAR(m);
    return m;
}
