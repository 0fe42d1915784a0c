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

PyMethodDef methods[] = {
    {"linear_rows", (PyCFunction)(void (*)(void))linear_rows, METH_FASTCALL, "dq_linear_rows(pair, x, y, stream)"},
    {"linear_rows8", (PyCFunction)(void (*)(void))linear_rows8, METH_FASTCALL, "dq_linear_rows8(pair, codes, scales, y, stream)"},
    {"rmsnorm8", (PyCFunction)(void (*)(void))rmsnorm8, METH_FASTCALL,
     "dq_rmsnorm8(x, gain, eps, codes, scales, residual, h, y, group, stream)"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dqcall", "Native calls of libdq.so's small entry points", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dqcall() { return PyModule_Create(&module); }
