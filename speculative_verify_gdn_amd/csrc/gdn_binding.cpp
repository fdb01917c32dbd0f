// gdn_binding.cpp -- the argument marshalling of the paged cache and window
// attention calls, as a Python extension (_gdn_binding, imported by gdn.py).
//
// Nothing is computed here: each function checks its torch tensors (on the
// device, dense, of the right type and shape), and passes their pointers and
// sizes to the C entry point of the same name.  The calls are short (a few
// microseconds on the GPU) and take up to ten tensors; with the checks and the
// conversions in Python a call costs 6 to 14 us of host time before anything is
// launched, here below 1.
//
// Every function takes the handle of a loaded libgdn (ctypes' _handle), the
// stream as an integer (None: torch's current one), then its tensors; it returns the C status code, or
// raises ValueError / TypeError before the library is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <dlfcn.h>

#include <cmath>
#include <cstdarg>
#include <deque>
#include <exception>
#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdn.h"

namespace {

// a raised Python exception on its way out
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Raised{};
}

// the entry points of one loaded library
struct Lib {
    decltype(&gdn_kv_reserve) kv_reserve;
    decltype(&gdn_kv_append) kv_append;
    decltype(&gdn_kv_rollback_tree) kv_rollback_tree;
    decltype(&gdn_kv_free) kv_free;
    decltype(&gdn_kv_fork) kv_fork;
    decltype(&gdn_kv_compact) kv_compact;
    decltype(&gdn_kv_copy) kv_copy;
    decltype(&gdn_attn_verify) attn_verify;
    void* handle = nullptr;
};

// the builds seen so far (a library is never closed, and a deque's elements stay where they are)
std::deque<Lib> g_libs;

template <typename F>
void symbol(void* handle, F& f, const char* name)
{
    f = reinterpret_cast<F>(dlsym(handle, name));
    if (!f) raise(PyExc_RuntimeError, "libgdn has no %s", name);
}

const Lib& lib_of(PyObject* o)
{
    void* h = PyLong_AsVoidPtr(o);
    if (!h) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "libgdn handle is null");
        throw Raised{};
    }
    for (const Lib& l : g_libs)
        if (l.handle == h) return l;
    Lib n;
    symbol(h, n.kv_reserve, "gdn_kv_reserve");
    symbol(h, n.kv_append, "gdn_kv_append");
    symbol(h, n.kv_rollback_tree, "gdn_kv_rollback_tree");
    symbol(h, n.kv_free, "gdn_kv_free");
    symbol(h, n.kv_fork, "gdn_kv_fork");
    symbol(h, n.kv_compact, "gdn_kv_compact");
    symbol(h, n.kv_copy, "gdn_kv_copy");
    symbol(h, n.attn_verify, "gdn_attn_verify");
    n.handle = h;
    g_libs.push_back(n);
    return g_libs.back();
}

PyObject* g_raw_stream;  // torch's current stream of a device, as an integer

// Where a call is launched: the device of `on`, an argument that is checked already, made current for the call (the
// library launches on the current one), and the stream given, or (None) torch's current one there.  Asked for and
// switched only where there are several: setting and restoring the same one cost 0.25 us a call.
struct Launch {
    c10::OptionalDeviceGuard guard;
    void* stream;

    Launch(PyObject* o, PyObject* on)
    {
        const c10::Device device = THPVariable_Unpack(on).device();
        const c10::impl::VirtualGuardImpl gpu(device.type());
        static const int devices = gpu.deviceCount();
        if (devices > 1 && gpu.getDevice() != device) guard.reset_device(device);
        if (o == Py_None) {
            PyObject* i = PyLong_FromLong(device.index());
            o = i ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
            Py_XDECREF(i);
            if (!o) throw Raised{};
            stream = PyLong_AsVoidPtr(o);
            Py_DECREF(o);
        } else {
            stream = PyLong_AsVoidPtr(o);
        }
        if (!stream && PyErr_Occurred()) throw Raised{};
    }
};

// the tensors of a call are on one device
void same_device(PyObject* const* a, Py_ssize_t n)
{
    int device = -1;
    for (Py_ssize_t i = 2; i < n; ++i) {
        if (a[i] == Py_None || PyLong_Check(a[i]) || !THPVariable_Check(a[i])) continue;
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda()) continue;   // (turned down by name, where it is taken)
        if (device >= 0 && t.get_device() != device)
            raise(PyExc_ValueError, "libgdn takes tensors of one device (here of %d and %d)", device, (int)t.get_device());
        device = t.get_device();
    }
}

// a tensor argument (never None)
const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

const at::Tensor& dense(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) raise(PyExc_ValueError, "libgdn takes device tensors (%s)", name);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "libgdn takes contiguous tensors (%s)", name);
    return t;
}

int dtype_of(const at::Tensor& t, const char* name)
{
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    raise(PyExc_TypeError, "unsupported dtype of %s", name);
}

int small(int64_t n, const char* what)
{
    if (n > 0x7fffffff) raise(PyExc_ValueError, "%s = %lld passes 2^31", what, (long long)n);
    return (int)n;
}

int int_of(PyObject* o, const char* name)
{
    int past = 0;
    const long v = PyLong_AsLongAndOverflow(o, &past);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (past || v > 0x7fffffff || v < -0x7fffffff) raise(PyExc_ValueError, "%s does not fit in 32 bits", name);
    return (int)v;
}

// an int32 array of a shape; None gives nullptr where it may
int32_t* ints(PyObject* o, const char* name, std::initializer_list<int64_t> shape, bool optional = false)
{
    if (optional && o == Py_None) return nullptr;
    const at::Tensor& t = dense(o, name);
    if (t.scalar_type() != at::kInt) raise(PyExc_TypeError, "%s must be int32", name);
    if (t.sizes() != at::IntArrayRef(shape)) raise(PyExc_ValueError, "%s has the wrong shape", name);
    return static_cast<int32_t*>(t.data_ptr());
}

struct Table {
    int32_t* p;
    int B, P;
};

Table table_of(PyObject* o)
{
    const at::Tensor& t = dense(o, "table");
    if (t.scalar_type() != at::kInt) raise(PyExc_TypeError, "table must be int32");
    if (t.dim() != 2) raise(PyExc_ValueError, "table must be [rows][P]");
    return Table{static_cast<int32_t*>(t.data_ptr()), small(t.size(0), "rows"), small(t.size(1), "P")};
}

struct Pages {
    void* p;
    int planes, n_pages, Hkv, page, D, dtype;
};

Pages pages_of(PyObject* o, const char* name, int dims)
{
    const at::Tensor& t = dense(o, name);
    if (t.dim() != dims)
        raise(PyExc_ValueError, dims == 5 ? "%s must be [planes][n_pages][Hkv][page][D]"
                                          : "%s must be a plane [n_pages][Hkv][page][D]", name);
    const int k = dims - 4;
    return Pages{t.data_ptr(), dims == 5 ? small(t.size(0), "planes") : 1, small(t.size(k), "n_pages"),
                 small(t.size(k + 1), "Hkv"), small(t.size(k + 2), "page"), small(t.size(k + 3), "D"),
                 dtype_of(t, name)};
}

Pages plane_pair(PyObject* k, PyObject* v, void** v_pages)
{
    const Pages a = pages_of(k, "k_pages", 4), b = pages_of(v, "v_pages", 4);
    if (a.n_pages != b.n_pages || a.Hkv != b.Hkv || a.page != b.page || a.D != b.D || a.dtype != b.dtype)
        raise(PyExc_ValueError, "k_pages and v_pages must be planes of one shape and type");
    *v_pages = b.p;
    return a;
}

// elements between the tokens of x [B][K][H][D], which may be a slice of wider rows (dense heads)
long long token_stride(const at::Tensor& x, const char* name, int64_t B, int64_t K, int64_t H, int64_t D, int dtype)
{
    if (!x.is_cuda()) raise(PyExc_ValueError, "libgdn takes device tensors (%s)", name);
    if (x.sizes() != at::IntArrayRef({B, K, H, D}) || dtype_of(x, name) != dtype)
        raise(PyExc_ValueError, "%s must be [%lld][%lld][%lld][%lld] of the cache's type", name, (long long)B,
              (long long)K, (long long)H, (long long)D);
    if (x.numel() == 0 || x.is_contiguous()) return H * D;
    const int64_t s = K > 1 ? x.stride(1) : x.stride(0);
    if ((D > 1 && x.stride(3) != 1) || (H > 1 && x.stride(2) != D) || (B > 1 && x.stride(0) != K * s) || s < H * D)
        raise(PyExc_ValueError, "%s must have dense heads and evenly spaced tokens", name);
    return s;
}

void want(Py_ssize_t n, Py_ssize_t count)
{
    if (n != count) raise(PyExc_TypeError, "%zd arguments, not %zd", count, n);
}

int do_reserve(PyObject* const* a, Py_ssize_t n)
{
    want(n, 8);  // lib stream lens add table ref granted page
    const Lib& lib = lib_of(a[0]);
    const Table t = table_of(a[4]);
    const at::Tensor& ref = dense(a[5], "ref");
    const int page = int_of(a[7], "page");
    const Launch where(a[1], a[4]);
    return lib.kv_reserve(ints(a[2], "lens", {t.B}), ints(a[3], "add", {t.B}), t.p, ints(a[5], "ref", {ref.numel()}),
                          ints(a[6], "granted", {t.B}), t.B, t.P, small(ref.numel(), "n_pages"), page, where.stream);
}

int do_append(PyObject* const* a, Py_ssize_t n)
{
    want(n, 9);  // lib stream k v k_pages v_pages lens count table
    const Lib& lib = lib_of(a[0]);
    void* vp;
    const Pages g = plane_pair(a[4], a[5], &vp);
    const Table t = table_of(a[8]);
    const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    if (k.dim() != 4) raise(PyExc_ValueError, "k must be [B][K][Hkv][D]");
    const int64_t K = k.size(1);
    const long long s = token_stride(k, "k", t.B, K, g.Hkv, g.D, g.dtype);
    if (token_stride(v, "v", t.B, K, g.Hkv, g.D, g.dtype) != s)
        raise(PyExc_ValueError, "k and v must have the same token stride");
    const Launch where(a[1], a[8]);
    return lib.kv_append(k.data_ptr(), v.data_ptr(), s, g.p, vp, ints(a[6], "lens", {t.B}),
                         ints(a[7], "count", {t.B}, true), t.p, t.B, small(K, "K"), g.Hkv, g.D, g.page, g.n_pages, t.P,
                         g.dtype, where.stream);
}

int do_rollback(PyObject* const* a, Py_ssize_t n)
{
    want(n, 11);  // lib stream node parent lens count table ref pool lens_out N
    const Lib& lib = lib_of(a[0]);
    const Pages g = pages_of(a[8], "pool", 5);
    const Table t = table_of(a[6]);
    int N;
    if (a[3] == Py_None) {
        if (a[10] == Py_None) raise(PyExc_ValueError, "a chain (parent=None) needs its window length N");
        N = int_of(a[10], "N");
    } else {
        const at::Tensor& p = dense(a[3], "parent");
        if (p.dim() != 2) raise(PyExc_ValueError, "parent must be [B][N]");
        N = small(p.size(1), "N");
    }
    const Launch where(a[1], a[6]);
    return lib.kv_rollback_tree(ints(a[2], "node", {t.B}), ints(a[3], "parent", {t.B, N}, true),
                                ints(a[4], "lens", {t.B}), ints(a[5], "count", {t.B}, true), t.p,
                                ints(a[7], "ref", {g.n_pages}), g.p, ints(a[9], "lens_out", {t.B}), t.B, N, t.P,
                                g.planes, g.n_pages, g.Hkv, g.page, g.D, g.dtype, where.stream);
}

int do_free(PyObject* const* a, Py_ssize_t n)
{
    want(n, 6);  // lib stream rows lens table ref
    const Lib& lib = lib_of(a[0]);
    const Table t = table_of(a[4]);
    const int64_t rows = dense(a[2], "rows").numel(), pages = dense(a[5], "ref").numel();
    const Launch where(a[1], a[4]);
    return lib.kv_free(ints(a[2], "rows", {rows}), ints(a[3], "lens", {t.B}), t.p, ints(a[5], "ref", {pages}),
                       small(rows, "n"), t.B, t.P, small(pages, "n_pages"), where.stream);
}

int do_fork(PyObject* const* a, Py_ssize_t n)
{
    want(n, 9);  // lib stream src dst lens table ref pool granted
    const Lib& lib = lib_of(a[0]);
    const Pages g = pages_of(a[7], "pool", 5);
    const Table t = table_of(a[5]);
    const int64_t forks = dense(a[2], "src").numel();
    const Launch where(a[1], a[5]);
    return lib.kv_fork(ints(a[2], "src", {forks}), ints(a[3], "dst", {forks}), ints(a[4], "lens", {t.B}), t.p,
                       ints(a[6], "ref", {g.n_pages}), g.p, ints(a[8], "granted", {forks}), small(forks, "n"), t.B, t.P,
                       g.planes, g.n_pages, g.Hkv, g.page, g.D, g.dtype, where.stream);
}

int do_compact(PyObject* const* a, Py_ssize_t n)
{
    want(n, 8);  // lib stream table ref pool table_out ref_out workspace
    const Lib& lib = lib_of(a[0]);
    const Pages g = pages_of(a[4], "pool", 5);
    const at::Tensor &t = dense(a[2], "table"), &to = dense(a[5], "table_out"), &w = dense(a[7], "workspace");
    if (t.scalar_type() != at::kInt || to.scalar_type() != at::kInt)
        raise(PyExc_TypeError, "table and table_out must be int32");
    if (t.sizes() != to.sizes()) raise(PyExc_ValueError, "table_out must have table's shape");
    const Launch where(a[1], a[2]);
    return lib.kv_compact(static_cast<int32_t*>(t.data_ptr()), ints(a[3], "ref", {g.n_pages}), g.p,
                          static_cast<int32_t*>(to.data_ptr()), ints(a[6], "ref_out", {g.n_pages}), w.data_ptr(),
                          w.nbytes(), t.numel(), g.planes, g.n_pages, g.Hkv, g.page, g.D, g.dtype, where.stream);
}

int do_copy(PyObject* const* a, Py_ssize_t n)
{
    want(n, 5);  // lib stream src dst pool
    const Lib& lib = lib_of(a[0]);
    const Pages g = pages_of(a[4], "pool", 5);
    const int64_t pairs = dense(a[2], "src").numel();
    const Launch where(a[1], a[2]);
    return lib.kv_copy(ints(a[2], "src", {pairs}), ints(a[3], "dst", {pairs}), g.p, small(pairs, "n"), g.planes,
                       g.n_pages, g.Hkv, g.page, g.D, g.dtype, where.stream);
}

int do_attn(PyObject* const* a, Py_ssize_t n)
{
    want(n, 14);  // lib stream q k_pages v_pages lens count parent table o lse workspace prefix_len scale
    const Lib& lib = lib_of(a[0]);
    void* vp;
    const Pages g = plane_pair(a[3], a[4], &vp);
    const Table t = table_of(a[8]);
    const at::Tensor& q = tensor(a[2], "q");
    if (q.dim() != 4) raise(PyExc_ValueError, "q must be [B][K][Hq][D]");
    const int64_t K = q.size(1), Hq = q.size(2);
    const long long s = token_stride(q, "q", t.B, K, Hq, g.D, g.dtype);
    if (a[11] == Py_None) raise(PyExc_ValueError, "attn_verify needs a workspace (attn_workspace)");
    const at::Tensor &o = dense(a[9], "o"), &w = dense(a[11], "workspace");
    if (o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type())
        raise(PyExc_ValueError, "o must have q's shape and type");
    float* lse = nullptr;
    if (a[10] != Py_None) {
        const at::Tensor& l = dense(a[10], "lse");
        if (l.scalar_type() != at::kFloat || l.sizes() != at::IntArrayRef({t.B, K, Hq}))
            raise(PyExc_ValueError, "lse must be float32 [B][K][Hq]");
        lse = static_cast<float*>(l.data_ptr());
    }
    const int prefix = int_of(a[12], "prefix_len");
    double scale;
    if (a[13] == Py_None) {
        scale = 1.0 / std::sqrt((double)g.D);
    } else {
        scale = PyFloat_AsDouble(a[13]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    const Launch where(a[1], a[8]);
    return lib.attn_verify(q.data_ptr(), s, g.p, vp, ints(a[5], "lens", {t.B}), ints(a[6], "count", {t.B}, true),
                           ints(a[7], "parent", {t.B, K}, true), t.p, o.data_ptr(), lse, w.data_ptr(), w.nbytes(), t.B,
                           small(K, "K"), small(Hq, "Hq"), g.Hkv, g.D, g.page, g.n_pages, t.P, prefix,
                           (float)scale, g.dtype, where.stream);
}

// no C++ exception leaves the extension
template <int (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    try {
        same_device(args, n);
        return PyLong_FromLong(F(args, n));
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define ENTRY(name, f, doc) {name, (PyCFunction)(void (*)())&entry<f>, METH_FASTCALL, doc}
PyMethodDef methods[] = {
    ENTRY("kv_reserve", do_reserve, "lib stream lens add table ref granted page"),
    ENTRY("kv_append", do_append, "lib stream k v k_pages v_pages lens count table"),
    ENTRY("kv_rollback_tree", do_rollback, "lib stream node parent lens count table ref pool lens_out N"),
    ENTRY("kv_free", do_free, "lib stream rows lens table ref"),
    ENTRY("kv_fork", do_fork, "lib stream src dst lens table ref pool granted"),
    ENTRY("kv_compact", do_compact, "lib stream table ref pool table_out ref_out workspace"),
    ENTRY("kv_copy", do_copy, "lib stream src dst pool"),
    ENTRY("attn_verify", do_attn, "lib stream q k_pages v_pages lens count parent table o lse workspace prefix scale"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_binding", "marshalling of the libgdn cache and attention calls", -1,
                      methods};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_binding()
{
    PyObject* c = PyImport_ImportModule("torch._C");
    if (!c) return nullptr;
    g_raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
    Py_DECREF(c);
    return g_raw_stream ? PyModule_Create(&module) : nullptr;
}
