// binding.cpp -- the verification pass's calls from Python, on torch tensors.
//
// A target model makes these calls for every layer of every step, on tensors that a ctypes
// call checks and unpacks in 10 us, several times what the small kernels take.  Here the
// same checks (type, shape, contiguity, device) take about 1 us.  Nothing is computed or kept;
// the calls go to libdspark.so's C entry points, whose addresses bind() hands over.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <initializer_list>

#include "../../include/dspark.h"

namespace {

decltype(&dspark_verify_layout) g_layout = nullptr;
decltype(&dspark_qk_norm_rope_store) g_norm = nullptr;
decltype(&dspark_verify_attention) g_attention = nullptr;

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *format, const char *name,
                        const std::string &more = "")
{
    PyErr_Format(type, format, name, more.c_str());
    throw Raised{};
}

std::string text(at::IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

const at::Tensor &cuda_tensor(PyObject *o, const char *name, at::ScalarType type)
{
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, "%s must be torch %s", name,
              std::string(c10::toString(type)) + ", got " + c10::toString(t.scalar_type()));
    return t;
}

// A tensor whose sizes the call's own sizes come from.
const at::Tensor &leading(PyObject *o, const char *name, at::ScalarType type, int64_t dims)
{
    const at::Tensor &t = cuda_tensor(o, name, type);
    if (t.dim() != dims)
        raise(PyExc_ValueError, "%s must have %s dimensions", name, std::to_string(dims));
    return t;
}

struct Call {
    c10::DeviceIndex device = c10::cuda::current_device();   // where the library launches

    void check_device(const at::Tensor &t, const char *name) const
    {
        if (t.get_device() != device)
            raise(PyExc_ValueError, "%s is on %s", name,
                  t.device().str() + ", the current device is cuda:" + std::to_string(device));
    }
    void *ptr(PyObject *o, const char *name, at::ScalarType type,
              std::initializer_list<int64_t> shape) const
    {
        const at::Tensor &t = cuda_tensor(o, name, type);
        const at::IntArrayRef want(shape.begin(), shape.size());
        if (t.sizes() != want)
            raise(PyExc_ValueError, "%s must have shape %s", name,
                  text(want) + ", got " + text(t.sizes()));
        if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
        check_device(t, name);
        return t.data_ptr();
    }
    void *optional(PyObject *o, const char *name, at::ScalarType type,
                   std::initializer_list<int64_t> shape) const
    {
        return o == Py_None ? nullptr : ptr(o, name, type, shape);
    }
    dspark_stream_t stream(PyObject *o) const
    {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
        void *p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) throw Raised{};
        return static_cast<dspark_stream_t>(p);
    }
};

int size(int64_t v, const char *name)
{
    if (v < INT_MIN || v > INT_MAX) raise(PyExc_ValueError, "%s is out of range", name);
    return static_cast<int>(v);
}

int integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return size(v, name);
}

float number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}

// Runs `body`, which returns a status, with `count` arguments and every exception turned into
// Python's.
template <class Body>
PyObject *guarded(Py_ssize_t given, Py_ssize_t count, Body body)
{
    if (given != count) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", count, given);
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

constexpr at::ScalarType kI32 = at::kInt, kBf16 = at::kBFloat16, kF32 = at::kFloat;

template <class F>
int released(F f)
{
    int st;
    Py_BEGIN_ALLOW_THREADS st = f();
    Py_END_ALLOW_THREADS return st;
}

PyObject *verify_layout(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 17, [&] {
        enum { L, CONTEXT, ROWS, PAGES, HELD, FREE, COUNT, START, POSITION, SLOT, PS, GAMMA, ANCHOR,
               X, TOKEN, ACCEPTED, STREAM };
        if ((a[ANCHOR] == Py_None) != (a[TOKEN] == Py_None) ||
            (a[X] == Py_None) != (a[TOKEN] == Py_None))
            raise(PyExc_ValueError, "%s", "anchor, x and token go together");
        const at::Tensor &pages = leading(a[PAGES], "pages", kI32, 2);
        const int64_t B = pages.size(0), width = pages.size(1);
        const int64_t cap = leading(a[POSITION], "position", kI32, 1).size(0);
        const int64_t num = leading(a[FREE], "free_pages", kI32, 1).size(0);
        const int ps = integer(a[PS], "page_size"), gamma = integer(a[GAMMA], "gamma");
        const Call c;
        auto i32 = [&](int i, const char *name, std::initializer_list<int64_t> shape) {
            return static_cast<int32_t *>(c.optional(a[i], name, kI32, shape));
        };
        auto need = [&](int i, const char *name, std::initializer_list<int64_t> shape) {
            return static_cast<int32_t *>(c.ptr(a[i], name, kI32, shape));
        };
        int32_t *l = need(L, "L", {B}), *ctx = need(CONTEXT, "context", {B});
        int32_t *rows = need(ROWS, "rows", {B}), *tab = need(PAGES, "pages", {B, width});
        int32_t *held = need(HELD, "held", {B}), *fp = need(FREE, "free_pages", {num});
        int32_t *fc = need(COUNT, "free_count", {1}), *rs = need(START, "row_start", {B + 1});
        int32_t *pos = need(POSITION, "position", {cap}), *slot = need(SLOT, "slot", {cap});
        int32_t *anchor = i32(ANCHOR, "anchor", {B}), *x = i32(X, "x", {B, gamma});
        int32_t *token = i32(TOKEN, "token", {cap}), *acc = i32(ACCEPTED, "accepted", {B});
        const int b = size(B, "B"), w = size(width, "max_pages"), np = size(num, "num_pages");
        const int rc = size(cap, "row_capacity");
        const dspark_stream_t s = c.stream(a[STREAM]);
        return released([&] {
            return g_layout(l, anchor, x, acc, ctx, rows, tab, held, fp, fc, b, gamma, ps, w, np, rc,
                            rs, pos, slot, token, s);
        });
    });
}

PyObject *qk_norm_rope_store(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 14, [&] {
        enum { QKV, POSITION, SLOT, ROWS, Q, K, V, QW, KW, EPS, INV, INTERLEAVED, SCALE, STREAM };
        const at::Tensor &q = leading(a[Q], "q_out", kBf16, 3);
        const at::Tensor &k = leading(a[K], "k_cache", kBf16, 4);
        const at::Tensor &qkv = leading(a[QKV], "qkv", kBf16, 2);
        const int64_t cap = q.size(0), Hq = q.size(1), D = q.size(2);
        const int64_t num = k.size(0), Hkv = k.size(1), ps = k.size(2);
        const int64_t width = (Hq + 2 * Hkv) * D;
        const Call c;
        if (qkv.size(0) != cap || qkv.size(1) != width)
            raise(PyExc_ValueError, "%s must have shape %s", "qkv",
                  text({cap, width}) + ", got " + text(qkv.sizes()));
        if (width > 1 && qkv.stride(1) != 1)
            raise(PyExc_ValueError, "%s must be contiguous along its channels", "qkv");
        c.check_device(qkv, "qkv");
        const int64_t pairs =
            a[INV] == Py_None ? 0 : leading(a[INV], "inv_freq", kF32, 1).size(0);
        const void *qw = c.optional(a[QW], "q_weight", kBf16, {D});
        const void *kw = c.optional(a[KW], "k_weight", kBf16, {D});
        auto *inv = static_cast<const float *>(c.optional(a[INV], "inv_freq", kF32, {pairs}));
        auto i32 = [&](int i, const char *name, int64_t count) {
            return static_cast<const int32_t *>(c.ptr(a[i], name, kI32, {count}));
        };
        const int32_t *pos = i32(POSITION, "position", cap), *slot = i32(SLOT, "slot", cap);
        const int32_t *rows = i32(ROWS, "n_rows", 1);
        void *qo = c.ptr(a[Q], "q_out", kBf16, {cap, Hq, D});
        void *kc = c.ptr(a[K], "k_cache", kBf16, {num, Hkv, ps, D});
        void *vc = c.ptr(a[V], "v_cache", kBf16, {num, Hkv, ps, D});
        const float eps = number(a[EPS]), scale = number(a[SCALE]);
        const int inter = PyObject_IsTrue(a[INTERLEAVED]);
        if (inter < 0) throw Raised{};
        const int rot = size(2 * pairs, "inv_freq"), rc = size(cap, "row_capacity");
        const int hq = size(Hq, "Hq"), hkv = size(Hkv, "Hkv"), d = size(D, "D");
        const int p = size(ps, "page_size"), np = size(num, "num_pages");
        const int64_t stride = cap > 1 ? qkv.stride(0) : width;
        const dspark_stream_t s = c.stream(a[STREAM]);
        const void *from = qkv.data_ptr();
        return released([&] {
            return g_norm(from, stride, qw, kw, eps, inv, rot, inter, scale, pos, slot, rows, rc, hq,
                          hkv, d, p, np, qo, kc, vc, s);
        });
    });
}

PyObject *verify_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        enum { Q, K, V, PAGES, CONTEXT, START, OUT, WS, SCALE, STREAM };
        const at::Tensor &q = leading(a[Q], "q", kBf16, 3);
        const at::Tensor &k = leading(a[K], "k_cache", kBf16, 4);
        const at::Tensor &pages = leading(a[PAGES], "pages", kI32, 2);
        const int64_t bytes = leading(a[WS], "workspace", at::kByte, 1).size(0);
        const int64_t cap = q.size(0), Hq = q.size(1), D = q.size(2);
        const int64_t num = k.size(0), Hkv = k.size(1), ps = k.size(2);
        const int64_t B = pages.size(0), width = pages.size(1);
        const Call c;
        const void *qp = c.ptr(a[Q], "q", kBf16, {cap, Hq, D});
        const void *kc = c.ptr(a[K], "k_cache", kBf16, {num, Hkv, ps, D});
        const void *vc = c.ptr(a[V], "v_cache", kBf16, {num, Hkv, ps, D});
        auto i32 = [&](int i, const char *name, std::initializer_list<int64_t> shape) {
            return static_cast<const int32_t *>(c.ptr(a[i], name, kI32, shape));
        };
        const int32_t *tab = i32(PAGES, "pages", {B, width}), *ctx = i32(CONTEXT, "context", {B});
        const int32_t *rs = i32(START, "row_start", {B + 1});
        void *out = c.ptr(a[OUT], "out", kBf16, {cap, Hq, D});
        void *ws = c.ptr(a[WS], "workspace", at::kByte, {bytes});
        const float scale = number(a[SCALE]);
        const int b = size(B, "B"), rc = size(cap, "row_capacity"), hq = size(Hq, "Hq");
        const int hkv = size(Hkv, "Hkv"), d = size(D, "D"), p = size(ps, "page_size");
        const int w = size(width, "max_pages"), np = size(num, "num_pages");
        const dspark_stream_t s = c.stream(a[STREAM]);
        return released([&] {
            return g_attention(qp, kc, vc, tab, ctx, rs, b, rc, hq, hkv, d, p, w, np, scale, out, ws,
                               static_cast<size_t>(bytes), s);
        });
    });
}

PyObject *bind(PyObject *, PyObject *args)
{
    unsigned long long layout, norm, attention;
    if (!PyArg_ParseTuple(args, "KKK", &layout, &norm, &attention)) return nullptr;
    g_layout = reinterpret_cast<decltype(g_layout)>(layout);
    g_norm = reinterpret_cast<decltype(g_norm)>(norm);
    g_attention = reinterpret_cast<decltype(g_attention)>(attention);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t))
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__dspark_calls()
{
    static PyMethodDef methods[] = {
        {"bind", bind, METH_VARARGS, "addresses of libdspark.so's entry points"},
        {"verify_layout", fast(verify_layout), METH_FASTCALL, nullptr},
        {"qk_norm_rope_store", fast(qk_norm_rope_store), METH_FASTCALL, nullptr},
        {"verify_attention", fast(verify_attention), METH_FASTCALL, nullptr},
        {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dspark_calls", nullptr, -1, methods};
    return PyModule_Create(&module);
}
