// binding.cpp -- argument checks and calls of the dense operators for Python (module
// _binding).  A decode step makes a few of these calls a layer, and checked in Python they
// cost as much as a launch (2.7 of 6.5 us); here they cost 0.3 us.
//
// It calls libseedmm.so through the addresses that `init` is given and takes streams and
// scratch memory from torch.  No computation happens here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/seedmm.h"

namespace {

decltype(&seedmm_q4_gemv) q4_gemv_fn;
decltype(&seedmm_q4_workspace_bytes) q4_bytes_fn;
decltype(&seedmm_add_norm) add_norm_fn;
decltype(&seedmm_route) route_fn;
PyObject* error_class;    // SeedmmError(status, what)

enum { kInt32 = 16, kUint32 = 17, kOther = -1 };
enum { FLOATS = 1 << SEEDMM_F32 | 1 << SEEDMM_BF16, ROWS = FLOATS | 1 << SEEDMM_I8 };

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return SEEDMM_F32;
        case at::kBFloat16: return SEEDMM_BF16;
        case at::kChar: return SEEDMM_I8;
        case at::kInt: return kInt32;
        case at::kUInt32: return kUint32;
        default: return kOther;
    }
}

const char* name_of(int types) {
    if (types == FLOATS) return "float32 or bfloat16";
    if (types == ROWS) return "float32, bfloat16 or int8";
    if (types == 1 << SEEDMM_F32) return "float32";
    return types == 1 << kInt32 ? "int32" : "uint32";
}

// A GPU tensor of one of `types` on device `dev` (-1: any).
bool gpu_tensor(PyObject* o, const char* name, int types, int dev, const at::Tensor** t, int* code) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) {
        PyErr_Format(PyExc_TypeError, "%s must be a CUDA (HIP) tensor", name);
        return false;
    }
    *t = &THPVariable_Unpack(o);
    *code = code_of((*t)->scalar_type());
    if (*code < 0 || !(types >> *code & 1)) {
        PyErr_Format(PyExc_TypeError, "%s must be one of %s, got %s", name, name_of(types),
                     c10::toString((*t)->scalar_type()));
        return false;
    }
    if (dev >= 0 && (*t)->get_device() != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on another device", name);
        return false;
    }
    return true;
}

// A row-major tensor [N][C] or [C] whose rows may be apart.
struct Rows {
    void* p = nullptr;
    int code = 0, dev = -1;
    int64_t n = 0, c = 0, ld = 0;
    bool matrix = false;

    bool take(PyObject* o, const char* name, int types, int on = -1) {
        const at::Tensor* t;
        if (!gpu_tensor(o, name, types, on, &t, &code)) return false;
        dev = t->get_device();
        p = t->data_ptr();
        matrix = t->dim() == 2;
        if (matrix) {
            n = t->size(0);
            c = t->size(1);
            ld = n > 1 ? t->stride(0) : c;
            if ((c > 1 && t->stride(1) != 1) || ld < c) {
                PyErr_Format(PyExc_ValueError,
                             "%s must be row-major with contiguous, distinct rows", name);
                return false;
            }
            return true;
        }
        if (t->dim() == 1 && (t->size(0) <= 1 || t->stride(0) == 1)) {
            n = 1;
            c = ld = t->size(0);
            return true;
        }
        PyErr_Format(PyExc_ValueError, "%s must be a row-major [N][C] or a contiguous [C] tensor", name);
        return false;
    }
};

// A contiguous tensor of at least n elements; None gives null where it is allowed.
bool flat(PyObject* o, const char* name, int types, int64_t n, int dev, void** p, int* code) {
    const at::Tensor* t;
    int c;
    if (!gpu_tensor(o, name, types, dev, &t, &c)) return false;
    if (!t->is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
        return false;
    }
    if (t->numel() < n) {
        PyErr_Format(PyExc_ValueError, "%s has %lld elements, %lld needed", name,
                     (long long)t->numel(), (long long)n);
        return false;
    }
    *p = t->data_ptr();
    if (code) *code = c;
    return true;
}

bool fits_int(int64_t v, const char* name) {
    if (v >= 0 && v <= 0x7FFFFFFF) return true;
    PyErr_Format(PyExc_ValueError, "%s = %lld is out of range", name, (long long)v);
    return false;
}

bool int_of(PyObject* o, const char* name, int64_t* v) {
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred()) && fits_int(*v, name);
}

// `handle`: a stream's handle as a Python int, or None for torch's current stream of `dev`.
bool stream_of(PyObject* handle, int dev, void** st) {
    if (handle == Py_None) {
        *st = (void*)c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
        return true;
    }
    *st = PyLong_AsVoidPtr(handle);
    return !PyErr_Occurred();
}

// The interpreter's lock given up for a scope.  What may wait for the device (a launch, for
// room in its queue; an allocation) runs so: the stream may be waiting for Python code itself.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The call, with the tensors' device current.
template <typename F>
bool call(int dev, const char* what, F f) {
    int status;
    {
        Unlocked u;
        if (c10::hip::current_device() == dev) {
            status = f();
        } else {
            c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
            status = f();
        }
    }
    if (status == SEEDMM_OK) return true;
    PyObject* e = PyObject_CallFunction(error_class, "is", status, what);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return false;
}

bool refuse(const char* text) {
    PyErr_SetString(PyExc_ValueError, text);
    return false;
}

// (weight, scales, biases, group, x, x_scale, y, workspace, M, K, stream)
bool q4_gemv(PyObject* const* a) {
    int64_t group, M, K;
    Rows x, y;
    if (!int_of(a[3], "group", &group) || !x.take(a[4], "x", ROWS)) return false;
    if (!int_of(a[8], "M", &M) || !int_of(a[9], "K", &K)) return false;
    const int dev = x.dev;
    if (x.c < K) {
        PyErr_Format(PyExc_ValueError, "x rows hold %lld elements, K = %lld", (long long)x.c, (long long)K);
        return false;
    }
    if ((group != 32 && group != 64 && group != 128) || K % group != 0) {
        PyErr_Format(PyExc_ValueError,
                     "K = %lld must be a multiple of the group, and the group 32, 64 or 128", (long long)K);
        return false;
    }
    void *w, *s, *b, *xs = nullptr;
    int sd, bd;
    if (!flat(a[0], "weight", 1 << kUint32, M * (K / 8), dev, &w, nullptr) ||
        !flat(a[1], "scales", FLOATS, M * (K / group), dev, &s, &sd) ||
        !flat(a[2], "biases", FLOATS, M * (K / group), dev, &b, &bd))
        return false;
    if (sd != bd) {
        PyErr_SetString(PyExc_TypeError, "scales and biases must have one type");
        return false;
    }
    if (x.code == SEEDMM_I8) {
        if (!flat(a[5], "x_scale", 1 << SEEDMM_F32, x.n, dev, &xs, nullptr)) return false;
    } else if (a[5] != Py_None) {
        return refuse("x_scale goes with int8 activations");
    }
    if (!y.take(a[6], "y", FLOATS, dev)) return false;
    if (y.n < x.n || y.c < M) {
        PyErr_Format(PyExc_ValueError, "y must hold [%lld][%lld]", (long long)x.n, (long long)M);
        return false;
    }
    if (!fits_int(x.n, "N") || !fits_int(x.ld, "x's row stride") || !fits_int(y.ld, "y's row stride"))
        return false;
    void* st;
    if (!stream_of(a[10], dev, &st)) return false;
    void* ws = nullptr;
    size_t bytes = 0;
    at::Tensor own;
    if (a[7] != Py_None) {
        if (!THPVariable_Check(a[7])) {
            PyErr_SetString(PyExc_TypeError, "the workspace must be a tensor");
            return false;
        }
        const at::Tensor& t = THPVariable_Unpack(a[7]);
        if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            return refuse("the workspace must be a contiguous tensor on x's device");
        ws = t.data_ptr();
        bytes = t.nbytes();
    } else if ((bytes = q4_bytes_fn(x.code, (int)group, (int)M, (int)K, (int)x.n)) != 0) {
        Unlocked u;
        own = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
        ws = own.data_ptr();
    }
    return call(dev, "seedmm_q4_gemv", [&] {
        return q4_gemv_fn((const uint32_t*)w, s, b, sd, (int)group, x.p, x.code, (int)x.ld,
                          (const float*)xs, y.p, y.code, (int)y.ld, (int)M, (int)K, (int)x.n, ws,
                          bytes, st);
    });
}

// (x, weight, delta, eps, residual, out, scale, stream)
bool add_norm(PyObject* const* a) {
    Rows x, d, r, o;
    if (!x.take(a[0], "x", FLOATS)) return false;
    const int dev = x.dev;
    void *w = nullptr, *sc = nullptr;
    int wd = SEEDMM_F32;
    if (a[2] != Py_None) {
        if (!d.take(a[2], "delta", FLOATS, dev)) return false;
        if (d.n != x.n || d.c != x.c) return refuse("delta must have x's shape");
    }
    if (a[1] != Py_None && !flat(a[1], "weight", FLOATS, x.c, dev, &w, &wd)) return false;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return false;
    if (!o.take(a[5], "out", ROWS, dev)) return false;
    if (o.n != x.n || o.c != x.c) return refuse("out must have x's shape");
    if (o.code == SEEDMM_I8) {
        if (!flat(a[6], "scale", 1 << SEEDMM_F32, x.n, dev, &sc, nullptr)) return false;
    } else if (a[6] != Py_None) {
        return refuse("scale goes with an int8 out");
    }
    if (a[4] != Py_None) {
        if (!r.take(a[4], "residual", FLOATS, dev)) return false;
        if (r.code != x.code || r.n != x.n || r.c != x.c)
            return refuse("residual must have x's shape and type");
    }
    if (!fits_int(x.n, "N") || !fits_int(x.c, "H")) return false;
    void* st;
    if (!stream_of(a[7], dev, &st)) return false;
    return call(dev, "seedmm_add_norm", [&] {
        return add_norm_fn(x.p, x.code, x.ld, a[2] == Py_None ? nullptr : d.p, d.code, d.ld, w, wd,
                           (float)eps, a[4] == Py_None ? nullptr : r.p, r.ld, o.p, o.code, o.ld,
                           (float*)sc, (int)x.n, (int)x.c, st);
    });
}

// (logits, top_k, bias, score, ids, w, stream)
bool route(PyObject* const* a) {
    Rows l;
    int64_t k, score;
    if (!l.take(a[0], "logits", FLOATS)) return false;
    if (!l.matrix) return refuse("logits must be [T][E]");
    if (!int_of(a[1], "top_k", &k) || !int_of(a[3], "score", &score)) return false;
    if (k < 1 || k > 64 || k > l.c) {
        PyErr_Format(PyExc_ValueError, "top_k = %lld must be in [1, min(E, 64)], E = %lld", (long long)k,
                     (long long)l.c);
        return false;
    }
    void *bias = nullptr, *ids, *w, *st;
    if (a[2] != Py_None && !flat(a[2], "bias", 1 << SEEDMM_F32, l.c, l.dev, &bias, nullptr)) return false;
    if (!flat(a[4], "ids", 1 << kInt32, l.n * k, l.dev, &ids, nullptr) ||
        !flat(a[5], "w", 1 << SEEDMM_F32, l.n * k, l.dev, &w, nullptr))
        return false;
    if (!fits_int(l.n, "T") || !fits_int(l.c, "E") || !stream_of(a[6], l.dev, &st)) return false;
    return call(l.dev, "seedmm_route", [&] {
        return route_fn(l.p, l.code, l.ld, (const float*)bias, (int)score, (int)l.n, (int)l.c, (int)k,
                        (int32_t*)ids, (float*)w, st);
    });
}

// C++ exceptions end here: they become Python's.
template <bool (*F)(PyObject* const*), int COUNT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != COUNT) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", COUNT, n);
        return nullptr;
    }
    try {
        if (!F(args)) return nullptr;
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

bool set_up(PyObject* const* a) {
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return false;
    }
    q4_gemv_fn = (decltype(q4_gemv_fn))p[0];
    q4_bytes_fn = (decltype(q4_bytes_fn))p[1];
    add_norm_fn = (decltype(add_norm_fn))p[2];
    route_fn = (decltype(route_fn))p[3];
    Py_INCREF(a[4]);
    Py_XDECREF(error_class);
    error_class = a[4];
    return true;
}

#define ENTRY(name, fn, count) {name, (PyCFunction)(void*)&entry<fn, count>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("init", set_up, 5), ENTRY("q4_gemv", q4_gemv, 11),
                         ENTRY("add_norm", add_norm, 8), ENTRY("route", route, 7),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
