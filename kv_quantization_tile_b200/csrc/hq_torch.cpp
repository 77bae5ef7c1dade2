// hq_torch.cpp -- the serving operators' calls from Python (CPython extension
// kv_quantization_tile_b200._hq_torch): argument checks on torch tensors, then
// the C ABI of include/hq.h on the tensors' device and current stream.
//
// These calls are made per layer and token, where a call through ctypes costs
// several times its kernel: here a tensor is read through torch's own headers
// and nothing is built on the Python side.  What a tensor's shape, type,
// strides or device make impossible is a ValueError; codes of the library come
// back as its error class (set once by hq.py).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>
#include <string>

#include "../../include/hq.h"

namespace {

PyObject *g_error = nullptr;  // HQError(code, where)

struct PythonError {};  // a Python exception is set

void need(bool ok, const char *what)
{
    if (!ok) throw std::invalid_argument(what);
}

const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(what) + ": a tensor");
    return THPVariable_Unpack(o);
}

// None gives a null tensor
const at::Tensor *maybe(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

template <typename T>
T integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    if (v != (long long)(T)v) throw std::invalid_argument("an integer out of range");
    return (T)v;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}

hq_rows rows(const at::Tensor &t, const char *what)
{
    if (t.dim() != 3 || (t.numel() > 0 && t.size(2) > 1 && t.stride(2) != 1))
        throw std::invalid_argument(std::string(what) + ": [tokens, heads, head_dim], contiguous along head_dim");
    const auto type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) {
        PyErr_SetString(PyExc_TypeError, "bf16 or fp32 tensors only");
        throw PythonError();
    }
    return hq_rows{ t.data_ptr(), type == at::kFloat ? HQ_F32 : HQ_BF16, t.stride(0), t.stride(1) };
}

void *pointer(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

void vector(const at::Tensor &t, at::ScalarType type, int64_t n, const char *what)
{
    need(t.scalar_type() == type && t.is_contiguous() && t.numel() == n, what);
}

void status_of(const at::Tensor *t) { need(!t || (t->scalar_type() == at::kInt && t->numel() >= 1), "status: int32 [1]"); }

// Every tensor (null ones skipped) on one CUDA device; that device, made
// current for the call, and its stream (the given handle or the current one).
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;

    Place(PyObject *handle, const at::Tensor &first, std::initializer_list<const at::Tensor *> others)
    {
        need(first.is_cuda(), "CUDA tensors only");
        const auto dev = first.device();
        for (const at::Tensor *t : others) need(!t || t->device() == dev, "tensors on one device only");
        if (c10::cuda::current_device() != dev.index()) guard.set_index(dev.index());
        stream = handle == Py_None ? (void *)c10::cuda::getCurrentCUDAStream(dev.index()).stream()
                                   : (void *)(uintptr_t)integer<long long>(handle);
    }
};

PyObject *done(int code, const char *where)
{
    if (code == HQ_OK) Py_RETURN_NONE;
    if (PyObject *e = PyObject_CallFunction(g_error, "is", code, where)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// Runs f with n arguments; C++ exceptions become Python's.
template <typename F>
PyObject *call(Py_ssize_t got, Py_ssize_t n, F f)
{
    if (got != n) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const PythonError &) {
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

hq_pages pages(const at::Tensor &k, const at::Tensor &v)
{
    need(k.dim() == 4 && k.sizes() == v.sizes() && k.strides() == v.strides() && k.stride(3) == 1 &&
             k.scalar_type() == at::kBFloat16 && v.scalar_type() == at::kBFloat16,
         "pages: k, v bf16 [pages, heads, page_size, head_dim], same strides, contiguous vectors");
    need(k.size(1) <= INT32_MAX && k.size(2) <= INT32_MAX && k.size(3) <= INT32_MAX, "pages: too large");
    return hq_pages{ k.data_ptr(), v.data_ptr(), k.size(0), (int32_t)k.size(2), (int32_t)k.size(1), (int32_t)k.size(3),
                     k.stride(0), k.stride(1), k.stride(2) };
}

void check_rope(const at::Tensor &positions, const at::Tensor &turns, int rotary, int64_t tokens)
{
    vector(positions, at::kLong, tokens, "positions: contiguous int64 [tokens]");
    vector(turns, at::kLong, rotary / 2, "rope.turns: contiguous int64 [rotary_dim / 2]");
}

// rope(x, positions, turns, rotary_dim, layout, amplitude, y, inverse, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 9, [&] {
        const at::Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "positions"), &turns = tensor(a[2], "turns"),
                         &y = tensor(a[6], "y");
        const hq_rows xs = rows(x, "x"), ys = rows(y, "y");
        need(x.sizes() == y.sizes(), "y: the shape of x");
        const int rotary = integer<int>(a[3]);
        check_rope(pos, turns, rotary, x.size(0));
        need(x.size(1) <= INT32_MAX && x.size(2) <= INT32_MAX, "x: too large");
        const Place p(a[8], x, { &y, &pos, &turns });
        return done(hq_rope(&xs, &ys, x.size(0), (int)x.size(1), (int)x.size(2), (const int64_t *)pos.data_ptr(),
                            (const uint64_t *)turns.data_ptr(), rotary, integer<int>(a[4]), (float)real(a[5]),
                            integer<int>(a[7]), p.stream),
                    "hq_rope");
    });
}

// append(k, v, slots, pages k, pages v, positions, turns, rotary_dim, layout, amplitude, q, q_out, status, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 14, [&] {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                         &pk = tensor(a[3], "pages"), &pv = tensor(a[4], "pages");
        const at::Tensor *pos = maybe(a[5], "positions"), *turns = maybe(a[6], "turns"), *q = maybe(a[10], "q"),
                         *q_out = maybe(a[11], "q_out"), *status = maybe(a[12], "status");
        const hq_pages ps = pages(pk, pv);
        const hq_rows ks = rows(k, "k"), vs = rows(v, "v");
        const int64_t tokens = k.size(0);
        need(k.sizes() == v.sizes() && k.size(1) == ps.heads && k.size(2) == ps.head_dim,
             "k, v: [tokens, heads, head_dim] of the pool");
        vector(slots, at::kLong, tokens, "slots: contiguous int64 [tokens]");
        need(!q == !q_out, "q and q_out together");
        hq_rows qs{}, os{};
        int heads = 0;
        if (q) {
            qs = rows(*q, "q");
            os = rows(*q_out, "q_out");
            need(q->sizes() == q_out->sizes() && q->size(0) == tokens && q->size(2) == ps.head_dim && q->size(1) <= INT32_MAX,
                 "q, q_out: [tokens, q heads, head_dim]");
            heads = (int)q->size(1);
        }
        const int rotary = integer<int>(a[7]);
        if (turns) {
            need(pos != nullptr, "positions: contiguous int64 [tokens]");
            check_rope(*pos, *turns, rotary, tokens);
        } else {
            pos = nullptr;
        }
        status_of(status);
        const Place p(a[13], k, { &v, &slots, &pk, &pv, pos, turns, q, q_out, status });
        return done(hq_kv_append(heads ? &qs : nullptr, heads ? &os : nullptr, heads, &ks, &vs, tokens,
                                 (const int64_t *)pointer(pos), (const uint64_t *)pointer(turns), rotary, integer<int>(a[8]),
                                 (float)real(a[9]), (const int64_t *)slots.data_ptr(), &ps, p.stream, (int32_t *)pointer(status)),
                    "hq_kv_append");
    });
}

// attention(q, q_start, kv_len, pages k, pages v, table, scale, out, workspace, max_q, max_kv, causal, window, lse,
//           status, stream)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 16, [&] {
        const at::Tensor &q = tensor(a[0], "q"), &start = tensor(a[1], "q_start"), &kv = tensor(a[2], "kv_len"),
                         &pk = tensor(a[3], "pages"), &pv = tensor(a[4], "pages"), &table = tensor(a[5], "page_table"),
                         &out = tensor(a[7], "out"), &ws = tensor(a[8], "workspace");
        const at::Tensor *lse = maybe(a[13], "lse"), *status = maybe(a[14], "status");
        const hq_pages ps = pages(pk, pv);
        const hq_rows qs = rows(q, "q"), os = rows(out, "out");
        const int64_t tokens = q.size(0), heads = q.size(1), batch = kv.numel();
        need(out.sizes() == q.sizes() && q.size(2) == ps.head_dim && ps.heads > 0 && heads > 0 && heads % ps.heads == 0 &&
                 heads <= INT32_MAX,
             "q, out: [tokens, heads * group, head_dim] of the pool");
        vector(start, at::kInt, batch + 1, "q_start: contiguous int32 [batch + 1]");
        vector(kv, at::kInt, batch, "kv_len: contiguous int32 [batch]");
        need(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == batch &&
                 (table.size(1) <= 1 || batch == 0 || table.stride(1) == 1),
             "page_table: int32 [batch, pages], contiguous rows");
        need(ws.is_contiguous(), "workspace: contiguous");
        if (lse) vector(*lse, at::kFloat, tokens * heads, "lse: contiguous fp32 [tokens, heads]");
        status_of(status);
        const Place p(a[15], q, { &start, &kv, &pk, &pv, &table, &out, &ws, lse, status });
        return done(hq_paged_attention(&qs, (const int32_t *)start.data_ptr(), (const int32_t *)kv.data_ptr(), batch, tokens,
                                       integer<int64_t>(a[9]), integer<int64_t>(a[10]), (int)(heads / ps.heads), &ps,
                                       (const int32_t *)table.data_ptr(), table.size(1), table.stride(0), (float)real(a[6]),
                                       integer<int>(a[11]), integer<int64_t>(a[12]), &os, (float *)pointer(lse), ws.data_ptr(),
                                       (uint64_t)ws.nbytes(), p.stream, (int32_t *)pointer(status)),
                    "hq_paged_attention");
    });
}

// merge(a, lse_a, b, lse_b, out, lse, stream)
PyObject *merge(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(n, 7, [&] {
        const at::Tensor &x = tensor(a[0], "a"), &lx = tensor(a[1], "lse_a"), &y = tensor(a[2], "b"),
                         &ly = tensor(a[3], "lse_b"), &out = tensor(a[4], "out");
        const at::Tensor *lse = maybe(a[5], "lse");
        const hq_rows xs = rows(x, "a"), ys = rows(y, "b"), os = rows(out, "out");
        need(x.sizes() == y.sizes() && x.sizes() == out.sizes(), "a, b, out of one shape");
        const int64_t tokens = x.size(0), heads = x.size(1);
        need(heads <= INT32_MAX && x.size(2) <= INT32_MAX, "a: too large");
        vector(lx, at::kFloat, tokens * heads, "lse_a: contiguous fp32 [tokens, heads]");
        vector(ly, at::kFloat, tokens * heads, "lse_b: contiguous fp32 [tokens, heads]");
        if (lse) vector(*lse, at::kFloat, tokens * heads, "lse: contiguous fp32 [tokens, heads]");
        const Place p(a[6], x, { &y, &out, &lx, &ly, lse });
        return done(hq_attention_merge(&xs, (const float *)lx.data_ptr(), &ys, (const float *)ly.data_ptr(), tokens, (int)heads,
                                       (int)x.size(2), &os, (float *)pointer(lse), p.stream),
                    "hq_attention_merge");
    });
}

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_XINCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    { "rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, nullptr },
    { "append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr },
    { "attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr },
    { "merge", (PyCFunction)(void (*)(void))merge, METH_FASTCALL, nullptr },
    { "set_error", set_error, METH_O, nullptr },
    { nullptr, nullptr, 0, nullptr },
};

PyModuleDef module = { PyModuleDef_HEAD_INIT, "_hq_torch", "Calls of the serving operators on torch tensors.", -1, methods };

}  // namespace

PyMODINIT_FUNC PyInit__hq_torch() { return PyModule_Create(&module); }
