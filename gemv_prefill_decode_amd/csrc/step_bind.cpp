// Python binding of the decode step's entry points (module _step).
//
// A decode step's kernels take a few microseconds, and reading five to nine
// tensors' types, devices, shapes and strides through the interpreter took as
// long again: the norm's call costs 3.5 us on the host, launch included
// (through ctypes 7.1), the page tables' 3.9 (8.0).  The module only checks
// tensors and passes their pointers and strides to the C-ABI functions whose
// addresses bind() was given; it raises TypeError and ValueError for tensors
// that do not fit together and returns the library's status.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "qmm.h"

namespace {

decltype(&qmm_paged_extend) p_extend;
decltype(&qmm_kv_append) p_append;
decltype(&qmm_paged_attention) p_attention;
decltype(&qmm_paged_attention_workspace_bytes) p_workspace;
decltype(&qmm_add_rmsnorm) p_norm;
decltype(&qmm_add_rmsnorm_q8) p_norm_q8;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Refused{};
}

std::string list_of(at::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

// A tensor on the device `dev` (any device: -1) of this type.
const at::Tensor& tensor(PyObject* o, const char* what, at::ScalarType type, int64_t dev) {
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, std::string(what) + " must be a device (cuda/hip) tensor, got " + Py_TYPE(o)->tp_name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(what) + " must be a " + at::toString(type) + " device (cuda/hip) tensor, got " +
                                    at::toString(t.scalar_type()) + " on " + t.device().str());
    if (dev >= 0 && t.get_device() != dev)
        refuse(PyExc_ValueError, std::string(what) + " is on " + t.device().str() + ", other tensors on device " +
                                     std::to_string(dev));
    return t;
}

[[noreturn]] void misshapen(const at::Tensor& t, const char* what, const std::string& shape) {
    refuse(PyExc_ValueError, std::string(what) + " must be " + shape + ", got " + list_of(t.sizes()) + " with strides " +
                                 list_of(t.strides()));
}

// Pointer of a contiguous tensor of this shape.
void* packed(PyObject* o, const char* what, at::ScalarType type, int64_t dev, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(o, what, type, dev);
    if (t.sizes() != shape || !t.is_contiguous()) misshapen(t, what, "contiguous " + list_of(shape));
    return t.data_ptr();
}

// Float rows [n, row], or [n, heads, row / heads] with the heads side by side; rows any stride apart.
struct Rows {
    float* p = nullptr;
    int64_t ld = 0;
};
Rows rows(PyObject* o, const char* what, int64_t dev, int64_t n, int64_t row, int64_t heads = 0) {
    const at::Tensor& t = tensor(o, what, at::kFloat, dev);
    const auto size = t.sizes(), stride = t.strides();
    bool ok = size.size() == 2 && size[0] == n && size[1] == row && (row == 1 || stride[1] == 1);
    if (!ok && heads > 0 && size.size() == 3)
        ok = size[0] == n && size[1] == heads && size[2] == row / heads && (size[2] == 1 || stride[2] == 1) &&
             (heads == 1 || stride[1] == size[2]);
    if (!ok)
        misshapen(t, what, list_of({n, row}) + (heads > 0 ? " or " + list_of({n, heads, row / heads}) : std::string()) +
                               " with contiguous rows");
    return Rows{(float*)t.data_ptr(), n > 1 ? stride[0] : row};
}
Rows rows_or_none(PyObject* o, const char* what, int64_t dev, int64_t n, int64_t row) {
    return o == Py_None ? Rows{} : rows(o, what, dev, n, row);
}

struct Table {
    int32_t* p;
    int64_t width, ld;
};
Table table_of(PyObject* o, int64_t dev, int64_t batch) {
    const at::Tensor& t = tensor(o, "block_table", at::kInt, dev);
    if (t.dim() != 2 || t.size(0) != batch || (t.size(1) > 1 && t.stride(1) != 1))
        misshapen(t, "block_table", "[" + std::to_string(batch) + ", max_pages] with contiguous rows");
    return Table{(int32_t*)t.data_ptr(), t.size(1), batch > 1 ? t.stride(0) : t.size(1)};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}
int64_t length(PyObject* o, const char* what, int64_t dev) {
    const at::Tensor& t = tensor(o, what, at::kInt, dev);
    if (t.dim() != 1) misshapen(t, what, "one-dimensional");
    return t.size(0);
}

// f(arguments) with C++ exceptions turned into Python's: none passes this boundary.
template <int64_t (*F)(PyObject* const*)>
PyObject* entry(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
        return nullptr;
    }
    try {
        return PyLong_FromLongLong(F(args));
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}
template <int64_t (*F)(PyObject* const*), Py_ssize_t N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return entry<F>(args, n, N);
}

// The library call without the interpreter's lock: a launch waits where the
// stream's queue is full.
template <typename F, typename... A>
int64_t unlocked(F f, A... a) {
    PyThreadState* state = PyEval_SaveThread();
    const int64_t r = f(a...);
    PyEval_RestoreThread(state);
    return r;
}

hipStream_t stream_of(PyObject* o) { return (hipStream_t)(uintptr_t)integer(o); }

int64_t bind(PyObject* const* a) {
    p_extend = (decltype(p_extend))(uintptr_t)integer(a[0]);
    p_append = (decltype(p_append))(uintptr_t)integer(a[1]);
    p_attention = (decltype(p_attention))(uintptr_t)integer(a[2]);
    p_workspace = (decltype(p_workspace))(uintptr_t)integer(a[3]);
    p_norm = (decltype(p_norm))(uintptr_t)integer(a[4]);
    p_norm_q8 = (decltype(p_norm_q8))(uintptr_t)integer(a[5]);
    return 0;
}

// device(t, name): the device index of a device tensor
int64_t device(PyObject* const* a) {
    const char* what = PyUnicode_AsUTF8(a[1]);
    if (!what) throw Refused{};
    if (!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).is_cuda())
        refuse(PyExc_TypeError, std::string(what) + " must be a device (cuda/hip) tensor");
    return THPVariable_Unpack(a[0]).get_device();
}

// stream, dev, block_table, cached_lens, new_lens, free_pages, page_size, n_rows, seq_lens, slots, positions, pages_used
int64_t paged_extend(PyObject* const* a) {
    const int64_t dev = integer(a[1]), page = integer(a[6]), n_rows = integer(a[7]);
    const int64_t batch = length(a[3], "cached_lens", dev), n_free = length(a[5], "free_pages", dev);
    const Table t = table_of(a[2], dev, batch);
    auto i32 = [&](int i, const char* what, int64_t n) { return (int32_t*)packed(a[i], what, at::kInt, dev, {n}); };
    return unlocked(p_extend, t.p, t.ld, i32(8, "seq_lens", batch), i32(9, "slots", n_rows), i32(10, "positions", n_rows),
                    i32(11, "pages_used", 1), i32(3, "cached_lens", batch), i32(4, "new_lens", batch),
                    i32(5, "free_pages", n_free), batch, t.width, page, n_free, n_rows, stream_of(a[0]));
}

// stream, dev, cache, k, v, slots
int64_t kv_append(PyObject* const* a) {
    const int64_t dev = integer(a[1]);
    const auto* c = (const qmm_kv_cache*)(uintptr_t)integer(a[2]);
    const int64_t n = length(a[5], "slots", dev), row = c->n_kv * c->head_dim;
    const Rows k = rows(a[3], "k", dev, n, row, c->n_kv), v = rows(a[4], "v", dev, n, row, c->n_kv);
    const auto* slots = (const int32_t*)packed(a[5], "slots", at::kInt, dev, {n});
    return unlocked(p_append, c, k.p, k.ld, v.p, v.ld, slots, n, stream_of(a[0]));
}

// stream, dev, cache, q, block_table, seq_lens, scale (or None), out, lse (or None), workspace: a
// tensor, None, or True: allocated here, on the current stream, which has to be `stream`
int64_t paged_attention(PyObject* const* a) {
    const int64_t dev = integer(a[1]);
    const auto* c = (const qmm_kv_cache*)(uintptr_t)integer(a[2]);
    const int64_t d = c->head_dim, batch = length(a[5], "seq_lens", dev);
    const at::Tensor& qt = tensor(a[3], "q", at::kFloat, dev);
    const int64_t n_q = qt.dim() == 3 ? qt.size(1) : qt.dim() == 2 && d > 0 ? qt.size(1) / d : 0;
    const Rows q = rows(a[3], "q", dev, batch, n_q * d, n_q), out = rows(a[7], "out", dev, batch, n_q * d, n_q);
    const Table t = table_of(a[4], dev, batch);
    const auto* lens = (const int32_t*)packed(a[5], "seq_lens", at::kInt, dev, {batch});
    auto* lse = a[8] == Py_None ? nullptr : (float*)packed(a[8], "lse", at::kFloat, dev, {batch, n_q});
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : real(a[6]);
    at::Tensor own;
    void* ws = nullptr;
    int64_t ws_bytes = 0;
    if (a[9] == Py_True) {
        const int64_t need = p_workspace(batch, n_q, c->n_kv, d, t.width, c->page_size);
        if (need > 0) {
            own = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (at::DeviceIndex)dev));
            ws = own.data_ptr();
            ws_bytes = need;
        }
    } else if (a[9] != Py_None) {
        if (!THPVariable_Check(a[9])) refuse(PyExc_TypeError, "workspace must be 'auto', None or a device (cuda/hip) tensor");
        const at::Tensor& w = tensor(a[9], "workspace", THPVariable_Unpack(a[9]).scalar_type(), dev);
        if (!w.is_contiguous()) misshapen(w, "workspace", "contiguous");
        ws = w.data_ptr();
        ws_bytes = w.numel() * w.element_size();
    }
    return unlocked(p_attention, out.p, out.ld, lse, q.p, q.ld, c, t.p, t.ld, lens, batch, n_q, t.width, scale, ws,
                    ws_bytes, stream_of(a[0]));
}

// n and k of x, which both norms take
std::pair<int64_t, int64_t> extents(PyObject* o, int64_t dev) {
    const at::Tensor& x = tensor(o, "x", at::kFloat, dev);
    if (x.dim() != 2) misshapen(x, "x", "two-dimensional");
    return {x.size(0), x.size(1)};
}

// stream, dev, x, weight, residual (or None), eps, y, h (or None)
int64_t add_rmsnorm(PyObject* const* a) {
    const int64_t dev = integer(a[1]);
    const auto [n, k] = extents(a[2], dev);
    const Rows x = rows(a[2], "x", dev, n, k), r = rows_or_none(a[4], "residual", dev, n, k);
    const Rows y = rows(a[6], "y", dev, n, k), h = rows_or_none(a[7], "h", dev, n, k);
    const auto* w = (const float*)packed(a[3], "weight", at::kFloat, dev, {k});
    return unlocked(p_norm, y.p, y.ld, h.p, h.ld, x.p, x.ld, r.p, r.ld, w, n, k, real(a[5]), stream_of(a[0]));
}

// stream, dev, x, weight, residual (or None), eps, q, d, h (or None)
int64_t add_rmsnorm_q8(PyObject* const* a) {
    const int64_t dev = integer(a[1]);
    const auto [n, k] = extents(a[2], dev);
    const Rows x = rows(a[2], "x", dev, n, k), r = rows_or_none(a[4], "residual", dev, n, k);
    const Rows h = rows_or_none(a[8], "h", dev, n, k);
    auto* q = (int8_t*)packed(a[6], "q", at::kChar, dev, {n, k});
    auto* d = (float*)packed(a[7], "d", at::kFloat, dev, {n, k / 32});
    const auto* w = (const float*)packed(a[3], "weight", at::kFloat, dev, {k});
    return unlocked(p_norm_q8, q, d, h.p, h.ld, x.p, x.ld, r.p, r.ld, w, n, k, real(a[5]), stream_of(a[0]));
}

template <int64_t (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef def(const char* name) {
    return PyMethodDef{name, (PyCFunction)(void (*)())method<F, N>, METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {def<bind, 6>("bind"),
                           def<device, 2>("device"),
                           def<paged_extend, 12>("paged_extend"),
                           def<kv_append, 6>("kv_append"),
                           def<paged_attention, 10>("paged_attention"),
                           def<add_rmsnorm, 8>("add_rmsnorm"),
                           def<add_rmsnorm_q8, 9>("add_rmsnorm_q8"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_step", "Decode step calls of libqmm", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&g_module); }
