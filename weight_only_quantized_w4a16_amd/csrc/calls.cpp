// Marshalling of the block operators' calls for ops.py: tensors to device
// addresses, the current stream, one C-ABI call.  A decode step makes many small
// calls, and the launch itself takes 2.3 us: written in Python over ctypes, the
// checks and conversions around it took another 2.5 us of every call, here 0.6.
//
// The functions are those of the libqgemm.so that ops.py has loaded (bind);
// arguments come in the C ABI's order, the stream last (None: the current one).
// Each returns the call's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <exception>

#include "../../include/qgemm.h"

namespace {

struct BadCall {};                               // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* what) {
    PyErr_SetString(type, what);
    throw BadCall{};
}

// The positional arguments of one call, in order.
class Arguments {
public:
    Arguments(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
        if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
    }
    // A contiguous GPU tensor's address, or null for None; all tensors on one device.
    void* tensor() {
        PyObject* o = a_[i_++];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, "expected a tensor or None");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) raise(PyExc_ValueError, "tensor must be on the GPU");
        const int d = t.get_device();
        if (dev_ >= 0 && d != dev_) raise(PyExc_ValueError, "tensors must be on one device");
        dev_ = d;
        if (!t.is_contiguous()) raise(PyExc_ValueError, "tensor must be contiguous");
        return t.data_ptr();
    }
    int integer() {
        const long v = PyLong_AsLong(a_[i_++]);
        if (v == -1 && PyErr_Occurred()) throw BadCall{};
        if (v < INT_MIN || v > INT_MAX) raise(PyExc_OverflowError, "integer argument out of range");
        return (int)v;
    }
    size_t size() {
        const size_t v = PyLong_AsSize_t(a_[i_++]);
        if (v == (size_t)-1 && PyErr_Occurred()) throw BadCall{};
        return v;
    }
    float real() {
        const double v = PyFloat_AsDouble(a_[i_++]);
        if (v == -1.0 && PyErr_Occurred()) throw BadCall{};
        return (float)v;
    }
    // The last argument: the given stream's handle, or the device's current stream.
    qg_stream stream() {
        PyObject* o = a_[i_++];
        if (dev_ < 0) raise(PyExc_ValueError, "no tensor was given");
        if (o == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev_).stream();
        if (attribute(o, "device_index") != dev_)
            raise(PyExc_ValueError, "the stream belongs to another device than the tensors");
        return reinterpret_cast<qg_stream>(attribute(o, "cuda_stream"));
    }
    int device() const { return dev_; }

private:
    static long long attribute(PyObject* o, const char* name) {
        PyObject* v = PyObject_GetAttrString(o, name);
        if (!v) throw BadCall{};
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred()) throw BadCall{};
        return x;
    }
    PyObject* const* a_;
    Py_ssize_t i_ = 0;
    int dev_ = -1;
};

// Lets other Python threads run: a launch may wait for room in the device's queue.
class WithoutLock {
public:
    WithoutLock() : state_(PyEval_SaveThread()) {}
    ~WithoutLock() { PyEval_RestoreThread(state_); }
    WithoutLock(const WithoutLock&) = delete;

private:
    PyThreadState* state_;
};

// Makes the tensors' device current for one call.
class OnDevice {
public:
    explicit OnDevice(int dev) {
        if (hipGetDevice(&before_) == hipSuccess && before_ != dev) moved_ = hipSetDevice(dev) == hipSuccess;
    }
    ~OnDevice() {
        if (moved_) (void)hipSetDevice(before_);
    }

private:
    int before_ = 0;
    bool moved_ = false;
};

// Everything around the library's call once its arguments are known.
struct Launch {
    explicit Launch(int dev) : on(dev) {}
    WithoutLock lock;
    OnDevice on;
};

#define QG_CALLS(X)                                                                                              \
    X(rms_norm) X(rms_norm_quant) X(rms_norm_quant_int8) X(swiglu) X(swiglu_quant) X(swiglu_quant_int8)          \
    X(qgemm_w4a16_epilogue) X(moe_dispatch) X(moe_gather) X(moe_combine) X(moe_combine_backward)       \
    X(qk_norm_rope) X(kv_append) X(paged_attention)

struct {
#define X(f) decltype(&::f) f = nullptr;
    QG_CALLS(X)
#undef X
} lib;

// bind(name, address): the library's function of that name
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    const char* name = n == 2 ? PyUnicode_AsUTF8(a[0]) : nullptr;
    void* p = name ? PyLong_AsVoidPtr(a[1]) : nullptr;
    if (!p) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind(name, address)");
        return nullptr;
    }
#define X(f)                                              \
    if (!std::strcmp(name, #f)) {                         \
        lib.f = reinterpret_cast<decltype(lib.f)>(p);     \
        Py_RETURN_NONE;                                   \
    }
    QG_CALLS(X)
#undef X
    PyErr_Format(PyExc_ValueError, "no call named %s", name);
    return nullptr;
}

// Runs body(arguments) -> status; C++ exceptions end here.
template <class Body>
PyObject* call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, Body body) {
    try {
        Arguments args(a, n, want);
        return PyLong_FromLong(body(args));
    } catch (const BadCall&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// Pointer types of the C ABI from a tensor's address.
struct Address {
    void* p;
    template <class T>
    operator T*() const { return static_cast<T*>(p); }
};

template <class F>
PyObject* norm(PyObject* const* a, Py_ssize_t n, F f) {
    return call(a, n, 11, [f](Arguments& g) {
        const Address x{g.tensor()}, r{g.tensor()}, w{g.tensor()};
        const float eps = g.real();
        const int M = g.integer(), K = g.integer();
        const Address h{g.tensor()}, y{g.tensor()}, q{g.tensor()}, s{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return f(x, r, w, eps, M, K, h, y, q, s, st);
    });
}
PyObject* py_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 9, [](Arguments& g) {
        const Address x{g.tensor()}, r{g.tensor()}, w{g.tensor()};
        const float eps = g.real();
        const int M = g.integer(), K = g.integer();
        const Address h{g.tensor()}, y{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.rms_norm(x, r, w, eps, M, K, h, y, st);
    });
}
PyObject* py_rms_norm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) { return norm(a, n, lib.rms_norm_quant); }
PyObject* py_rms_norm_quant_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return norm(a, n, lib.rms_norm_quant_int8);
}

template <class F>
PyObject* gated(PyObject* const* a, Py_ssize_t n, F f) {
    return call(a, n, 6, [f](Arguments& g) {
        const Address gu{g.tensor()};
        const int M = g.integer(), I = g.integer();
        const Address q{g.tensor()}, s{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return f(gu, M, I, q, s, st);
    });
}
PyObject* py_swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 5, [](Arguments& g) {
        const Address gu{g.tensor()};
        const int M = g.integer(), I = g.integer();
        const Address y{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.swiglu(gu, M, I, y, st);
    });
}
PyObject* py_swiglu_quant(PyObject*, PyObject* const* a, Py_ssize_t n) { return gated(a, n, lib.swiglu_quant); }
PyObject* py_swiglu_quant_int8(PyObject*, PyObject* const* a, Py_ssize_t n) { return gated(a, n, lib.swiglu_quant_int8); }

PyObject* py_qgemm_w4a16_epilogue(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 13, [](Arguments& g) {
        const Address x{g.tensor()}, w{g.tensor()}, sc{g.tensor()}, b{g.tensor()};
        const int act = g.integer();
        const Address r{g.tensor()}, y{g.tensor()};
        const int M = g.integer(), N = g.integer(), K = g.integer();
        const Address ws{g.tensor()};
        const size_t bytes = g.size();
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.qgemm_w4a16_epilogue(x, w, sc, b, act, r, y, M, N, K, ws, bytes, st);
    });
}

PyObject* py_moe_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 14, [](Arguments& g) {
        const Address ids{g.tensor()}, rows{g.tensor()}, scale{g.tensor()};
        const int B = g.integer(), k = g.integer(), E = g.integer(), width = g.integer();
        const Address offsets{g.tensor()}, row{g.tensor()}, out{g.tensor()}, scale_out{g.tensor()}, ws{g.tensor()};
        const size_t bytes = g.size();
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.moe_dispatch(ids, rows, scale, B, k, E, width, offsets, row, out, scale_out, ws, bytes, st);
    });
}
PyObject* py_moe_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 9, [](Arguments& g) {
        const Address rows{g.tensor()}, scale{g.tensor()}, row{g.tensor()};
        const int B = g.integer(), k = g.integer(), width = g.integer();
        const Address out{g.tensor()}, scale_out{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.moe_gather(rows, scale, row, B, k, width, out, scale_out, st);
    });
}
PyObject* py_moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 9, [](Arguments& g) {
        const Address rows{g.tensor()}, row{g.tensor()}, w{g.tensor()}, res{g.tensor()};
        const int B = g.integer(), k = g.integer(), K = g.integer();
        const Address y{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.moe_combine(rows, row, w, res, B, k, K, y, st);
    });
}
PyObject* py_moe_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 10, [](Arguments& g) {
        const Address dy{g.tensor()}, rows{g.tensor()}, row{g.tensor()}, w{g.tensor()};
        const int B = g.integer(), k = g.integer(), K = g.integer();
        const Address drows{g.tensor()}, dw{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.moe_combine_backward(dy, rows, row, w, B, k, K, drows, dw, st);
    });
}

PyObject* py_qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 15, [](Arguments& g) {
        const Address qkv{g.tensor()}, wq{g.tensor()}, wk{g.tensor()};
        const float eps = g.real();
        const Address pos{g.tensor()}, freq{g.tensor()};
        const int rot = g.integer(), inter = g.integer(), T = g.integer(), Hq = g.integer(), Hkv = g.integer(),
                  D = g.integer();
        const Address q{g.tensor()}, k{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.qk_norm_rope(qkv, wq, wk, eps, pos, freq, rot, inter, T, Hq, Hkv, D, q, k, st);
    });
}
PyObject* py_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 24, [](Arguments& g) {
        const Address qkv{g.tensor()}, wq{g.tensor()}, wk{g.tensor()};
        const float eps = g.real();
        const Address freq{g.tensor()};
        const int rot = g.integer(), inter = g.integer();
        const Address offsets{g.tensor()}, len{g.tensor()}, table{g.tensor()};
        const int T = g.integer(), B = g.integer(), max_pages = g.integer(), Hq = g.integer(), Hkv = g.integer(),
                  D = g.integer();
        const Address k{g.tensor()}, v{g.tensor()}, ks{g.tensor()}, vs{g.tensor()};
        const int pages = g.integer(), page = g.integer();
        const Address q{g.tensor()};
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.kv_append(qkv, wq, wk, eps, freq, rot, inter, offsets, len, table, T, B, max_pages, Hq, Hkv, D, k, v, ks,
                             vs, pages, page, q, st);
    });
}
PyObject* py_paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 26, [](Arguments& g) {
        const Address q{g.tensor()}, k{g.tensor()}, v{g.tensor()}, ks{g.tensor()}, vs{g.tensor()};
        const int pages = g.integer(), page = g.integer();
        const Address offsets{g.tensor()}, len{g.tensor()}, table{g.tensor()};
        const int T = g.integer(), B = g.integer(), max_pages = g.integer(), Hq = g.integer(), Hkv = g.integer(),
                  D = g.integer();
        const float scale = g.real();
        const int window = g.integer(), sinks = g.integer(), shared = g.integer(), max_q = g.integer();
        const Address out{g.tensor()}, lse{g.tensor()}, ws{g.tensor()};
        const size_t bytes = g.size();
        const qg_stream st = g.stream();
        const Launch launch(g.device());
        return lib.paged_attention(q, k, v, ks, vs, pages, page, offsets, len, table, T, B, max_pages, Hq, Hkv, D, scale,
                                   window, sinks, shared, max_q, out, lse, ws, bytes, st);
    });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
#define X(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&py_##f)), METH_FASTCALL, nullptr},
    QG_CALLS(X)
#undef X
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Call marshalling of ops.py.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was built with
PyMODINIT_FUNC PyInit__calls(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", QG_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
