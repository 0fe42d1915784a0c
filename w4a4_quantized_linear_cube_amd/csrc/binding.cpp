// Native argument marshalling of the binding's small calls (dq.py).  A
// few-row product or norm runs for 4 to 15 us on the GPU, and reading six
// tensors' shapes, strides and pointers through Python takes as long.  Each
// function here takes the tensors as they are, checks what the C ABI cannot
// see (shapes, types, row strides, alignment, device), and calls the entry
// point; it returns the entry point's status, or None where the arguments are
// not such tensors, and dq.py's own checks then say what is wrong.
#include <Python.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "dq.h"

namespace {

struct Matrix {
    void* p = nullptr;
    int64_t n = 0, c = 0, ld = 0;
    c10::ScalarType type = c10::ScalarType::Undefined;
    int device = -1;
};

// A 2-D CUDA tensor with contiguous, non-overlapping rows of `align`-byte
// alignment; the stride of a single row means nothing.
bool matrix(PyObject* o, uint64_t align, Matrix* m) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != c10::kStrided || !t.is_cuda() || t.dim() != 2) return false;
    m->n = t.size(0);
    m->c = t.size(1);
    m->ld = m->n > 1 ? t.stride(0) : m->c;
    if ((t.stride(1) != 1 && m->c > 1) || m->ld < m->c) return false;
    m->type = t.scalar_type();
    m->device = (int)t.get_device();
    m->p = t.data_ptr();
    return ((uint64_t)(uintptr_t)m->p | (m->n > 1 ? (uint64_t)m->ld * t.element_size() : 0)) % align == 0;
}

bool dtype_of(c10::ScalarType t, dq_dtype* d) {
    if (t == c10::ScalarType::BFloat16) *d = DQ_BF16;
    else if (t == c10::ScalarType::Float) *d = DQ_F32;
    else return false;
    return true;
}

// Codes [n][c] and scales [n][c / 32], dense, on `device`.
bool mx8(PyObject* codes, PyObject* scales, int device, Matrix* c, Matrix* s) {
    return matrix(codes, 8, c) && matrix(scales, 1, s) && c->ld == c->c && s->ld == s->c && c->c % 32 == 0 && s->n == c->n &&
           s->c == c->c / 32 && c->device == device && s->device == device &&
           (c->type == c10::ScalarType::Float8_e4m3fn || c->type == c10::ScalarType::Byte) &&
           (s->type == c10::ScalarType::Float8_e8m0fnu || s->type == c10::ScalarType::Byte);
}

// The raw stream: an integer, or the current one of the device for None.
bool stream_of(PyObject* o, int device, void** s) {
    if (o == Py_None) {
        *s = (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
        return true;
    }
    if (!PyLong_Check(o)) return false;
    *s = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
}

// (weight handle, workspace handle, Ci, Co, device), as dq.Rows keeps it
struct Pair {
    dq_weights* w = nullptr;
    dq_rows* a = nullptr;
    int64_t Ci = 0, Co = 0;
    int device = 0;
};
bool pair_of(PyObject* o, Pair* p) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) return false;
    p->w = (dq_weights*)PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0));
    p->a = (dq_rows*)PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 1));
    p->Ci = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
    p->Co = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3));
    p->device = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 4));
    return !PyErr_Occurred();
}

bool output(PyObject* o, int64_t n, const Pair& p, Matrix* y, dq_dtype* d) {
    return matrix(o, 1, y) && y->n == n && y->c == p.Co && y->device == p.device && dtype_of(y->type, d);
}

// Other Python threads run while a call enqueues (it may wait for room in the queue).
struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
};

// Runs `body`; None where it finds the arguments unfit or torch objects to them.
template <class Body>
PyObject* guarded(Body body) {
    int status = 0;
    bool fit = false;
    try {
        fit = body(&status);
    } catch (...) {
        fit = false;
    }
    if (fit) return PyLong_FromLong(status);
    PyErr_Clear();
    Py_RETURN_NONE;
}

// linear_rows(pair, x, y, stream)
PyObject* linear_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Pair p;
        Matrix x, y;
        dq_dtype dx, dy;
        void* stream;
        if (n != 4 || !pair_of(v[0], &p) || !matrix(v[1], 16, &x) || x.c != p.Ci || x.device != p.device || !dtype_of(x.type, &dx) ||
            !output(v[2], x.n, p, &y, &dy) || !stream_of(v[3], p.device, &stream))
            return false;
        Released released;
        *status = dq_linear_rows(p.w, x.p, dx, x.ld, x.n, p.a, y.p, dy, y.ld, stream);
        return true;
    });
}

// linear_rows8(pair, codes, scales, y, stream)
PyObject* linear_rows8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Pair p;
        Matrix c, s, y;
        dq_dtype dy;
        void* stream;
        if (n != 5 || !pair_of(v[0], &p) || !mx8(v[1], v[2], p.device, &c, &s) || c.c != p.Ci || !output(v[3], c.n, p, &y, &dy) ||
            !stream_of(v[4], p.device, &stream))
            return false;
        Released released;
        *status = dq_linear_rows8(p.w, (const uint8_t*)c.p, (const uint8_t*)s.p, c.n, p.a, y.p, dy, y.ld, stream);
        return true;
    });
}

// rmsnorm8(x, gain, eps, codes, scales, residual, h, y, group, stream)
PyObject* rmsnorm8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Matrix x, c, s, more[3];
        dq_dtype dx, dg = DQ_F32;
        void *stream, *gain = nullptr;
        if (n != 10 || !matrix(v[0], 16, &x) || !dtype_of(x.type, &dx) || !PyFloat_Check(v[2]) || !PyLong_Check(v[8])) return false;
        if (v[1] != Py_None) {
            if (!THPVariable_Check(v[1])) return false;
            const at::Tensor& g = THPVariable_Unpack(v[1]);
            if (!g.defined() || !g.is_cuda() || g.dim() != 1 || g.size(0) != x.c || !g.is_contiguous() || (int)g.get_device() != x.device ||
                !dtype_of(g.scalar_type(), &dg))
                return false;
            gain = g.data_ptr();
            if ((uintptr_t)gain % 16) return false;
        }
        if ((v[3] == Py_None) != (v[4] == Py_None)) return false;
        if (v[3] != Py_None && (!mx8(v[3], v[4], x.device, &c, &s) || c.n != x.n || c.c != x.c)) return false;
        for (int i = 0; i < 3; ++i)
            if (v[5 + i] != Py_None) {
                Matrix& m = more[i];
                if (!matrix(v[5 + i], 16, &m) || m.n != x.n || m.c != x.c || m.type != x.type || m.device != x.device) return false;
            }
        const long group = PyLong_AsLong(v[8]);
        if ((group != 32 && group != 64) || !stream_of(v[9], x.device, &stream)) return false;
        Released released;
        *status = dq_rmsnorm8(x.p, x.ld, more[0].p, more[0].ld, dx, gain, dg, PyFloat_AS_DOUBLE(v[2]), x.n, x.c, (int32_t)group,
                              more[1].p, more[1].ld, (uint8_t*)c.p, (uint8_t*)s.p, more[2].p, more[2].ld, x.device, stream);
        return true;
    });
}

// Attribute `name` of a handle or description of dq.py (whose class dq.py has checked) as an address (0 for None, with *ok kept).
void* address_of(PyObject* o, const char* name, bool* ok) {
    if (o == Py_None) return nullptr;
    PyObject* v = PyObject_GetAttrString(o, name);
    void* p = v && PyLong_Check(v) ? PyLong_AsVoidPtr(v) : nullptr;
    Py_XDECREF(v);
    if (!p || PyErr_Occurred()) *ok = false;
    return p;
}
int64_t number_of(PyObject* o, const char* name, bool* ok) {
    PyObject* v = PyObject_GetAttrString(o, name);
    const int64_t n = v && PyLong_Check(v) ? PyLong_AsLongLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) *ok = false;
    return n;
}

// A contiguous 1-D gain of n values, or None.
bool gain_of(PyObject* o, int64_t n, int device, void** p, dq_dtype* d, bool* any) {
    *p = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& g = THPVariable_Unpack(o);
    dq_dtype mine;
    if (!g.defined() || g.layout() != c10::kStrided || !g.is_cuda() || g.dim() != 1 || g.size(0) != n || !g.is_contiguous() ||
        (int)g.get_device() != device || !dtype_of(g.scalar_type(), &mine) || (*any && mine != *d))
        return false;
    *d = mine;
    *any = true;
    *p = g.data_ptr();
    return (uintptr_t)*p % 16 == 0;
}

// A contiguous int32 tensor of n values (and `c` columns, where that is not 0), or None.
bool ints_of(PyObject* o, int64_t n, int64_t c, int device, const int32_t** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != c10::kStrided || !t.is_cuda() || t.scalar_type() != c10::ScalarType::Int ||
        t.dim() != (c ? 2 : 1) || t.size(0) != n || (c && t.size(1) != c) || !t.is_contiguous() || (int)t.get_device() != device)
        return false;
    *p = (const int32_t*)t.data_ptr();
    return true;
}

// The norm and rotation of a call: (norm, eps, rope, pos) with the gains' dtype.  `rope` is followed: dq.py has seen that it is a Rope or None.
bool ops_of(PyObject* norm, PyObject* eps, PyObject* rope, PyObject* pos, int64_t n, int device, dq_head_ops* ops) {
    if (!PyLong_Check(norm) || !PyFloat_Check(eps)) return false;
    const long k = PyLong_AsLong(norm);
    if (k < 0 || k > 2) return false;
    ops->norm = (dq_norm)k;
    ops->eps = PyFloat_AS_DOUBLE(eps);
    bool ok = true;
    ops->rope = (const dq_rope*)address_of(rope, "address", &ok);
    if (!ok) return false;
    if (!ops->rope) return pos == Py_None;
    if (number_of(rope, "device", &ok) != device || !ok) return false;
    return ints_of(pos, n, ops->rope->axes, device, &ops->pos_dev);
}

// norm_rope(x, heads, y, norm, gain, eps, rope, pos, stream)
PyObject* norm_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Matrix x, y;
        dq_dtype dx, dy;
        dq_head_ops ops{};
        void *stream, *gain;
        bool any = false;
        if (n != 9 || !matrix(v[0], 16, &x) || !PyLong_Check(v[1]) || !matrix(v[2], 16, &y) || !dtype_of(x.type, &dx) ||
            !dtype_of(y.type, &dy) || y.n != x.n || y.c != x.c || y.device != x.device)
            return false;
        const long heads = PyLong_AsLong(v[1]);
        if (heads < 1 || heads > x.c || x.c % heads || !ops_of(v[3], v[5], v[6], v[7], x.n, x.device, &ops)) return false;
        if ((ops.norm == DQ_NORM_NONE && v[4] != Py_None) ||
            !gain_of(v[4], ops.norm == DQ_NORM_HEAD ? x.c / heads : x.c, x.device, &gain, &ops.gain_dt, &any) ||
            !stream_of(v[8], x.device, &stream) || x.c / heads > INT32_MAX)
            return false;
        Released released;
        *status = dq_norm_rope(x.p, x.ld, dx, x.n, (int32_t)heads, (int32_t)(x.c / heads), gain, &ops, y.p, y.ld, dy, x.device, stream);
        return true;
    });
}

// kv_write(kv, seqs, k, v, q, y, norm, gain, gain_q, eps, rope, pos, stream)
PyObject* kv_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Matrix k, val, q, y;
        dq_dtype dt, dv, dq = DQ_F32, dy = DQ_F32;
        dq_head_ops ops{};
        void *stream, *gk, *gq;
        bool any = false, ok = true;
        if (n != 13) return false;
        const dq_kv* kv = (const dq_kv*)address_of(v[0], "address", &ok);
        const dq_seqs* seqs = (const dq_seqs*)address_of(v[1], "address", &ok);
        if (!ok || !kv || !seqs) return false;
        const int device = (int)number_of(v[0], "device", &ok);
        const int64_t C = (int64_t)kv->heads * kv->head_dim;
        if (number_of(v[1], "device", &ok) != device || !ok || !matrix(v[2], 16, &k) || !matrix(v[3], 16, &val) || k.c != C || val.c != C ||
            val.n != k.n || k.device != device || val.device != device || !dtype_of(k.type, &dt) || !dtype_of(val.type, &dv) || dv != dt)
            return false;
        if ((v[4] == Py_None) != (v[5] == Py_None)) return false;
        if (v[4] != Py_None && (!matrix(v[4], 16, &q) || !matrix(v[5], 16, &y) || q.n != k.n || y.n != k.n || q.c != y.c || q.c < 1 ||
                                q.c % kv->head_dim || q.device != device || y.device != device || !dtype_of(q.type, &dq) || dq != dt ||
                                !dtype_of(y.type, &dy)))
            return false;
        if (!ops_of(v[6], v[9], v[10], v[11], k.n, device, &ops)) return false;
        if ((ops.norm == DQ_NORM_NONE && (v[7] != Py_None || v[8] != Py_None)) || (v[4] == Py_None && v[8] != Py_None)) return false;
        if (!gain_of(v[7], ops.norm == DQ_NORM_HEAD ? kv->head_dim : C, device, &gk, &ops.gain_dt, &any) ||
            !gain_of(v[8], ops.norm == DQ_NORM_HEAD ? kv->head_dim : q.c, device, &gq, &ops.gain_dt, &any) ||
            !stream_of(v[12], device, &stream))
            return false;
        Released released;
        *status = dq_kv_write(kv, seqs, k.n, dt, k.p, k.ld, val.p, val.ld, gk, q.p, q.ld, (int32_t)(q.c / kv->head_dim), gq, y.p, y.ld, dy,
                              &ops, device, stream);
        return true;
    });
}

// kv_read(kv, seqs, k, v, stream)
PyObject* kv_read(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Matrix m[2];
        dq_dtype dt = DQ_F32;
        void* stream;
        bool ok = true;
        if (n != 5 || (v[2] == Py_None && v[3] == Py_None)) return false;
        const dq_kv* kv = (const dq_kv*)address_of(v[0], "address", &ok);
        const dq_seqs* seqs = (const dq_seqs*)address_of(v[1], "address", &ok);
        if (!ok || !kv || !seqs) return false;
        const int device = (int)number_of(v[0], "device", &ok);
        if (number_of(v[1], "device", &ok) != device || !ok || !stream_of(v[4], device, &stream)) return false;
        const int one = v[2] != Py_None ? 0 : 1;
        for (int i = one; i < 2; ++i)
            if (v[2 + i] != Py_None && (!matrix(v[2 + i], 16, &m[i]) || m[i].c != (int64_t)kv->heads * kv->head_dim || m[i].device != device ||
                                        !dtype_of(m[i].type, &dt) || m[i].n != m[one].n || m[i].type != m[one].type))
                return false;
        Released released;
        *status = dq_kv_read(kv, seqs, m[one].n, m[0].p, m[0].ld, m[1].p, m[1].ld, dt, device, stream);
        return true;
    });
}

// attn_rows(kv, seqs, q, a, y, scale (below 0: head_dim ** -0.5), block, window, prefix, cap, stream)
PyObject* attn_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded([&](int* status) {
        Matrix q, y;
        dq_dtype dt, dy;
        dq_attn_ops ops{};
        void* stream;
        bool ok = true;
        if (n != 11) return false;
        const dq_kv* kv = (const dq_kv*)address_of(v[0], "address", &ok);
        const dq_seqs* seqs = (const dq_seqs*)address_of(v[1], "address", &ok);
        dq_attn* a = (dq_attn*)address_of(v[3], "address", &ok);
        if (!ok || !kv || !seqs || !a) return false;
        const int device = (int)number_of(v[0], "device", &ok);
        if (number_of(v[1], "device", &ok) != device || number_of(v[3], "device", &ok) != device || !ok || !matrix(v[2], 16, &q) ||
            !matrix(v[4], 16, &y) || !dtype_of(q.type, &dt) || !dtype_of(y.type, &dy) || dy != dt || y.n != q.n || y.c != q.c || q.c < 1 ||
            q.c % ((int64_t)kv->heads * kv->head_dim) || q.device != device || y.device != device || !PyFloat_Check(v[5]) ||
            !PyLong_Check(v[6]) || !PyLong_Check(v[7]) || !PyFloat_Check(v[9]))
            return false;
        // (block and window first: what PyLong_AsLongLong cannot take raises, and the binding's own checks say so)
        ops.block = PyLong_AsLongLong(v[6]);
        ops.window = PyLong_AsLongLong(v[7]);
        if (PyErr_Occurred() || !ints_of(v[8], seqs->seqs, 0, device, &ops.prefix_dev) || !stream_of(v[10], device, &stream)) return false;
        ops.scale = PyFloat_AS_DOUBLE(v[5]);
        if (ops.scale == -1.0) ops.scale = 1.0 / std::sqrt((double)kv->head_dim);
        ops.cap = PyFloat_AS_DOUBLE(v[9]);
        Released released;
        *status = dq_attn_rows(kv, seqs, q.n, q.p, q.ld, dt, (int32_t)(q.c / kv->head_dim), &ops, a, y.p, y.ld, device, stream);
        return true;
    });
}

PyMethodDef methods[] = {
    {"linear_rows", (PyCFunction)(void (*)(void))linear_rows, METH_FASTCALL, "dq_linear_rows(pair, x, y, stream)"},
    {"linear_rows8", (PyCFunction)(void (*)(void))linear_rows8, METH_FASTCALL, "dq_linear_rows8(pair, codes, scales, y, stream)"},
    {"rmsnorm8", (PyCFunction)(void (*)(void))rmsnorm8, METH_FASTCALL,
     "dq_rmsnorm8(x, gain, eps, codes, scales, residual, h, y, group, stream)"},
    {"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, "dq_norm_rope(x, heads, y, norm, gain, eps, rope, pos, stream)"},
    {"kv_write", (PyCFunction)(void (*)(void))kv_write, METH_FASTCALL,
     "dq_kv_write(kv, seqs, k, v, q, y, norm, gain, gain_q, eps, rope, pos, stream)"},
    {"kv_read", (PyCFunction)(void (*)(void))kv_read, METH_FASTCALL, "dq_kv_read(kv, seqs, k, v, stream)"},
    {"attn_rows", (PyCFunction)(void (*)(void))attn_rows, METH_FASTCALL,
     "dq_attn_rows(kv, seqs, q, a, y, scale, block, window, prefix, cap, stream)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dqcall", "Native calls of libdq.so's small entry points", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dqcall() { return PyModule_Create(&module); }
