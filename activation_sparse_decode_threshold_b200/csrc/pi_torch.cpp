// pi_torch.cpp -- the attention calls of binding.py, from torch tensors to the C
// entry points (include/pi_ffn.h): checks that the tensors are what the entry
// point will take them for and passes their addresses on.  Native because these
// calls take a few microseconds on the GPU: the same checks and conversions cost
// 3 to 8 us of a call in Python (ctypes 3 us of it), here below one.
//
// Each function returns None, the entry point's status, or the text of a refusal.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>
#include <string>

#include "../../include/pi_ffn.h"

namespace {

decltype(&pi_int4_matvec) f_matvec;
decltype(&pi_kv_append) f_append;
decltype(&pi_kv_read) f_read;
decltype(&pi_paged_attention) f_attend;

struct Refused {
    std::string text;
};
struct Raised {};   // a Python exception is set

[[noreturn]] void refuse(const char *fmt, ...)
{
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    throw Refused{text};
}

template <typename F>
PyObject *guarded(F f)
{
    try {
        const pi_status st = f();
        if (st == PI_OK) Py_RETURN_NONE;
        return PyLong_FromLong(st);
    } catch (const Refused &r) {
        return PyUnicode_FromString(r.text.c_str());
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}

long long integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
void *address(PyObject *o) { return reinterpret_cast<void *>(static_cast<uintptr_t>(integer(o))); }

const at::Tensor &tensor(PyObject *o, const char *name, int device)
{
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    const at::Device on = t.device();
    if (!on.is_cuda() || on.index() != device) refuse("%s is not on cuda:%d", name, device);
    if (t.layout() != at::kStrided) refuse("%s must be a strided tensor", name);
    return t;
}

int float_code(const at::Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
    case at::kFloat: return PI_F32;
    case at::kHalf: return PI_F16;
    case at::kBFloat16: return PI_BF16;
    default: refuse("%s must be float32, float16 or bfloat16", name);
    }
}

// Row distance of a tensor [tokens, n] or [tokens, n, m] whose rows are contiguous.
int64_t token_rows(const at::Tensor &t, const char *name, int64_t tokens, int64_t n, int64_t m = 0)
{
    const int dims = m ? 3 : 2;
    if (t.dim() != dims || t.size(0) != tokens || t.size(1) != n || (m && t.size(2) != m)) {
        if (m) refuse("%s must be [%lld, %lld, %lld]", name, (long long)tokens, (long long)n, (long long)m);
        refuse("%s must be [%lld, %lld]", name, (long long)tokens, (long long)n);
    }
    if ((m && ((m != 1 && t.stride(2) != 1) || (n != 1 && t.stride(1) != m))) || (!m && n != 1 && t.stride(1) != 1))
        refuse("%s: a token's values must be contiguous", name);
    return t.stride(0);
}

const int32_t *ints(const at::Tensor &t, const char *name, int64_t n)
{
    if (t.scalar_type() != at::kInt) refuse("%s must be int32", name);
    if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) refuse("%s must be contiguous [%lld]", name, (long long)n);
    return static_cast<const int32_t *>(t.data_ptr());
}

const float *norm_weight(PyObject *o, const char *name, int device, int dim)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name, device);
    if (t.scalar_type() != at::kFloat || !t.is_contiguous() || t.numel() != dim) refuse("%s must be contiguous float32 [head_dim]", name);
    return static_cast<const float *>(t.data_ptr());
}

// None: torch's current stream of the device.
void *stream_of(PyObject *o, int device)
{
    return o == Py_None ? static_cast<void *>(c10::cuda::getCurrentCUDAStream(device).stream()) : address(o);
}

// The entry points run without the interpreter's lock, as with ctypes.
template <typename F, typename... A>
pi_status unlocked(F f, A... a)
{
    pi_status st;
    Py_BEGIN_ALLOW_THREADS st = f(a...);
    Py_END_ALLOW_THREADS return st;
}

// What the attention calls need of their handle: (handle, heads, kv_heads, head_dim, device).
struct Layer {
    pi_attn_t a;
    int64_t heads, kv_heads, dim;
    int device;
    explicit Layer(PyObject *t)
    {
        if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 5) refuse("not a layer");
        a = static_cast<pi_attn_t>(address(PyTuple_GET_ITEM(t, 0)));
        heads = integer(PyTuple_GET_ITEM(t, 1));
        kv_heads = integer(PyTuple_GET_ITEM(t, 2));
        dim = integer(PyTuple_GET_ITEM(t, 3));
        device = int(integer(PyTuple_GET_ITEM(t, 4)));
    }
};

pi_kv_table table_of(PyObject *o, int device)
{
    const at::Tensor &t = tensor(o, "table", device);
    if (t.scalar_type() != at::kInt) refuse("table must be int32");
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) refuse("table must be [sequences, pages] with contiguous rows");
    if (t.size(0) > (1 << 30) || t.size(1) > (1 << 30)) refuse("table is too large");
    pi_kv_table r;
    r.pages = static_cast<const int32_t *>(t.data_ptr());
    r.n_seqs = int(t.size(0));
    r.width = int(t.size(1));
    r.stride = t.stride(0);
    return r;
}

// The cache's tensors as they are now, of the handle's format: (dtype, page_size, layout, k, v, k_scale, v_scale).
pi_kv_cache cache_of(PyObject *o, const Layer &l)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 7) refuse("not a cache");
    const long long code = integer(PyTuple_GET_ITEM(o, 0)), page = integer(PyTuple_GET_ITEM(o, 1)), layout = integer(PyTuple_GET_ITEM(o, 2));
    const int64_t rows[2] = {layout == PI_KV_HND ? l.kv_heads : page, layout == PI_KV_HND ? page : l.kv_heads};
    const bool scaled = code == PI_I8 || code == PI_INT4G32;
    const int64_t row = code == PI_INT4G32 ? l.dim / 2 : l.dim, groups = code == PI_INT4G32 ? l.dim / 32 : 0;
    const at::ScalarType type = code == PI_F16 ? at::kHalf : code == PI_BF16 ? at::kBFloat16 : code == PI_I8 ? at::kChar : at::kByte;
    // pages x rows x `last` values (0: without the last axis)
    auto data = [&](PyObject *t, const char *name, at::ScalarType want, int64_t last, int64_t &pages) {
        const at::Tensor &x = tensor(t, name, l.device);
        if (x.scalar_type() != want) refuse("%s must be %s", name, c10::toString(want));
        const at::IntArrayRef n = x.sizes();
        if (n.size() != (last ? 4u : 3u) || n[1] != rows[0] || n[2] != rows[1] || (last && n[3] != last) || !x.is_contiguous())
            refuse(last ? "%s must be contiguous [pages, %lld, %lld, %lld]" : "%s must be contiguous [pages, %lld, %lld]", name,
                   (long long)rows[0], (long long)rows[1], (long long)last);
        if (pages < 0) pages = n[0];
        if (n[0] != pages || pages > INT32_MAX) refuse("the cache's tensors must have the same number of pages (below 2^31)");
        return x.data_ptr();
    };
    int64_t pages = -1;
    pi_kv_cache c{};
    PyObject *const *t = &PyTuple_GET_ITEM(o, 3);
    c.k = data(t[0], "cache k", type, row, pages);
    c.v = data(t[1], "cache v", type, row, pages);
    if (scaled != (t[2] != Py_None) || scaled != (t[3] != Py_None))
        refuse("a cache of %s has %s", c10::toString(type), scaled ? "k_scale and v_scale" : "no scales");
    if (scaled) {
        const at::ScalarType scale = code == PI_I8 ? at::kFloat : at::kHalf;
        c.k_scale = data(t[2], "cache k_scale", scale, groups, pages);
        c.v_scale = data(t[3], "cache v_scale", scale, groups, pages);
    }
    c.n_pages = int(pages);
    return c;
}

int token_count(const at::Tensor &pos)
{
    if (pos.dim() != 1 || pos.size(0) > (1 << 30)) refuse("pos must be contiguous [tokens]");
    return int(pos.size(0));
}

void arguments(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) refuse("%lld arguments instead of %lld", (long long)got, (long long)want);
}

// matvec(handle, rows, columns, device, x, y, add, norm_eps, stream)
PyObject *matvec(PyObject *, PyObject *const *v, Py_ssize_t nargs)
{
    return guarded([&]() -> pi_status {
        arguments(nargs, 9);
        const int device = int(integer(v[3]));
        const at::Tensor &x = tensor(v[4], "x", device), &y = tensor(v[5], "y", device);
        if (x.dim() != 2 || x.size(0) > (1 << 30)) refuse("x must be [tokens, columns]");
        const int64_t tokens = x.size(0), n = integer(v[1]), xs = token_rows(x, "x", tokens, integer(v[2])),
                      ys = token_rows(y, "y", tokens, n);
        const int xc = float_code(x, "x"), yc = float_code(y, "y");
        const void *add = nullptr;
        if (v[6] != Py_None) {
            const at::Tensor &a = tensor(v[6], "add", device);
            if ((token_rows(a, "add", tokens, n) != ys && tokens != 1) || a.scalar_type() != y.scalar_type())
                refuse("add must have y's type and row distance");
            add = a.data_ptr();
        }
        const double eps = PyFloat_AsDouble(v[7]);
        if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
        return unlocked(f_matvec, static_cast<pi_int4_t>(address(v[0])), int(tokens), pi_dtype(xc), (const void *)x.data_ptr(), xs,
                        add, pi_dtype(yc), y.data_ptr(), ys, float(eps), stream_of(v[8], device));
    });
}

// append(layer, cache, table, pos, q, k, v, q_out, seq, q_norm, k_norm, stream)
PyObject *append(PyObject *, PyObject *const *v, Py_ssize_t nargs)
{
    return guarded([&]() -> pi_status {
        arguments(nargs, 12);
        const Layer l(v[0]);
        const pi_kv_table table = table_of(v[2], l.device);
        const pi_kv_cache cache = cache_of(v[1], l);
        const at::Tensor &pos = tensor(v[3], "pos", l.device);
        const int tokens = token_count(pos);
        const int32_t *pp = ints(pos, "pos", tokens), *sp = v[8] == Py_None ? nullptr : ints(tensor(v[8], "seq", l.device), "seq", tokens);
        const at::Tensor &q = tensor(v[4], "q", l.device), &k = tensor(v[5], "k", l.device), &w = tensor(v[6], "v", l.device),
                         &o = tensor(v[7], "q_out", l.device);
        const int code = float_code(q, "q");
        if (k.scalar_type() != q.scalar_type() || w.scalar_type() != q.scalar_type() || o.scalar_type() != q.scalar_type())
            refuse("q, k, v and q_out must have one type");
        const int64_t qs = token_rows(q, "q", tokens, l.heads, l.dim), ks = token_rows(k, "k", tokens, l.kv_heads, l.dim),
                      vs = token_rows(w, "v", tokens, l.kv_heads, l.dim), os = token_rows(o, "q_out", tokens, l.heads, l.dim);
        const float *qn = norm_weight(v[9], "q_norm", l.device, int(l.dim)), *kn = norm_weight(v[10], "k_norm", l.device, int(l.dim));
        return unlocked(f_append, l.a, &cache, &table, tokens, sp, pp, pi_dtype(code), (const void *)q.data_ptr(), qs,
                        (const void *)k.data_ptr(), ks, (const void *)w.data_ptr(), vs, qn, kn, o.data_ptr(), os,
                        stream_of(v[11], l.device));
    });
}

// read(layer, cache, table, pos, k_out, v_out, seq, stream)
PyObject *read(PyObject *, PyObject *const *v, Py_ssize_t nargs)
{
    return guarded([&]() -> pi_status {
        arguments(nargs, 8);
        const Layer l(v[0]);
        const pi_kv_table table = table_of(v[2], l.device);
        const pi_kv_cache cache = cache_of(v[1], l);
        const at::Tensor &pos = tensor(v[3], "pos", l.device);
        const int tokens = token_count(pos);
        const int32_t *pp = ints(pos, "pos", tokens), *sp = v[6] == Py_None ? nullptr : ints(tensor(v[6], "seq", l.device), "seq", tokens);
        const at::Tensor &k = tensor(v[4], "k_out", l.device), &w = tensor(v[5], "v_out", l.device);
        const int code = float_code(k, "k_out");
        token_rows(k, "k_out", tokens, l.kv_heads, l.dim);
        token_rows(w, "v_out", tokens, l.kv_heads, l.dim);
        if (!k.is_contiguous() || !w.is_contiguous() || w.scalar_type() != k.scalar_type())
            refuse("k_out and v_out must be contiguous, both of one type");
        return unlocked(f_read, l.a, &cache, &table, tokens, sp, pp, pi_dtype(code), k.data_ptr(), w.data_ptr(), stream_of(v[7], l.device));
    });
}

// attend(layer, cache, table, lens, q, out, lse, stream)
PyObject *attend(PyObject *, PyObject *const *v, Py_ssize_t nargs)
{
    return guarded([&]() -> pi_status {
        arguments(nargs, 8);
        const Layer l(v[0]);
        const pi_kv_table table = table_of(v[2], l.device);
        const pi_kv_cache cache = cache_of(v[1], l);
        const int32_t *lens = ints(tensor(v[3], "lens", l.device), "lens", table.n_seqs);
        const at::Tensor &q = tensor(v[4], "q", l.device), &o = tensor(v[5], "out", l.device);
        const int code = float_code(q, "q");
        if (o.scalar_type() != q.scalar_type()) refuse("q and out must have one type");
        const int64_t qs = token_rows(q, "q", table.n_seqs, l.heads, l.dim), os = token_rows(o, "out", table.n_seqs, l.heads, l.dim);
        float *lse = nullptr;
        if (v[6] != Py_None) {
            const at::Tensor &e = tensor(v[6], "lse", l.device);
            if (e.scalar_type() != at::kFloat || e.dim() != 2 || e.size(0) != table.n_seqs || e.size(1) != l.heads || !e.is_contiguous())
                refuse("lse must be contiguous float32 [sequences, heads]");
            lse = static_cast<float *>(e.data_ptr());
        }
        return unlocked(f_attend, l.a, &cache, &table, lens, pi_dtype(code), (const void *)q.data_ptr(), qs, o.data_ptr(), os, lse,
                        stream_of(v[7], l.device));
    });
}

// init(matvec, append, read, attend): the entry points' addresses
PyObject *init(PyObject *, PyObject *const *v, Py_ssize_t nargs)
{
    return guarded([&]() -> pi_status {
        arguments(nargs, 4);
        f_matvec = reinterpret_cast<decltype(f_matvec)>(address(v[0]));
        f_append = reinterpret_cast<decltype(f_append)>(address(v[1]));
        f_read = reinterpret_cast<decltype(f_read)>(address(v[2]));
        f_attend = reinterpret_cast<decltype(f_attend)>(address(v[3]));
        return PI_OK;
    });
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(init), METH_FASTCALL, nullptr},
    {"matvec", reinterpret_cast<PyCFunction>(matvec), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(append), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(read), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(attend), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pi_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pi_torch() { return PyModule_Create(&module); }
