// kda_native.cpp -- CPython marshalling of the entry points whose host time is a step's latency:
// the decode on the 8-bit state pool, the pool's store and load, and the 4-bit projections.  One
// token's kernels run a few microseconds; checking and unpacking 17 to 28 tensors attribute by
// attribute in Python took 9 to 16 us a call, here it takes about one.  Each function checks that
// every tensor is a contiguous CUDA tensor of the right type and size on one device (ValueError or
// TypeError otherwise), calls the C entry of the same name and returns its status.  What torch throws
// on the way (a tensor without storage or strides) leaves as RuntimeError.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kda.h"

namespace {

using at::ScalarType;

constexpr int64_t kHead = 128;
constexpr int kMaxWeights = 8;

// The tensors of one call; after the first failure every later take() is a no-op.
struct Call {
    int device = -2;             // of the first tensor
    bool failed = false;

    void fail(PyObject* type, const char* name, const char* what) {
        if (!failed) PyErr_Format(type, "%s: %s", name, what);
        failed = true;
    }
    const at::Tensor* tensor(PyObject* o, const char* name) {
        if (failed) return nullptr;
        if (!THPVariable_Check(o)) {
            fail(PyExc_TypeError, name, "expected a tensor");
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    // a required tensor of `type` with `numel` elements (any number when negative)
    void* take(PyObject* o, const char* name, ScalarType type, int64_t numel) {
        const at::Tensor* t = tensor(o, name);
        if (t == nullptr) return nullptr;
        if (!t->is_cuda()) {
            fail(PyExc_ValueError, name, "expected a CUDA tensor");
            return nullptr;
        }
        if (device == -2) device = t->get_device();
        if (t->scalar_type() != type) {
            failed = true;
            PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(type),
                         c10::toString(t->scalar_type()));
        } else if (t->get_device() != device) {
            failed = true;
            PyErr_Format(PyExc_ValueError, "%s: expected a tensor on cuda:%d, got cuda:%d", name,
                         device, (int)t->get_device());
        } else if (!t->is_contiguous()) {
            fail(PyExc_ValueError, name, "expected a contiguous tensor");
        } else if (numel >= 0 && t->numel() != numel) {
            failed = true;
            PyErr_Format(PyExc_ValueError, "%s: expected %lld elements, got %lld", name,
                         (long long)numel, (long long)t->numel());
        }
        return failed ? nullptr : t->data_ptr();
    }
    void* maybe(PyObject* o, const char* name, ScalarType type, int64_t numel) {
        return o == Py_None ? nullptr : take(o, name, type, numel);
    }
    int64_t integer(PyObject* o) {
        if (failed) return 0;
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) failed = true;
        // sizes past 2^30 cannot be valid and would overflow the products below
        if (!failed && (v < -(1LL << 30) || v > (1LL << 30))) fail(PyExc_ValueError, "a size", "out of range");
        return v;
    }
    float real(PyObject* o) {
        if (failed) return 0.0f;
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) failed = true;
        return (float)v;
    }
    // the stream handle: an int, or None for torch's current stream of the tensors' device
    void* stream(PyObject* o) {
        if (failed) return nullptr;
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        void* p = PyLong_AsVoidPtr(o);
        if (p == nullptr && PyErr_Occurred()) failed = true;
        return p;
    }
    // KDA_DTYPE_* of a tensor that may be f32 or bf16
    ScalarType float_type(PyObject* o, const char* name, int* dtype) {
        const at::Tensor* t = tensor(o, name);
        if (t == nullptr) return ScalarType::Float;
        const ScalarType s = t->scalar_type();
        if (s != ScalarType::Float && s != ScalarType::BFloat16) {
            fail(PyExc_TypeError, name, "expected float32 or bfloat16");
            return ScalarType::Float;
        }
        *dtype = s == ScalarType::BFloat16 ? KDA_DTYPE_BF16 : KDA_DTYPE_F32;
        return s;
    }
    // format, slots and data of a pool's codes [P, H, Dv, 128]
    void* pool(PyObject* o, int64_t H, int64_t Dv, int* format, int64_t* P) {
        const at::Tensor* t = tensor(o, "codes");
        if (t == nullptr) return nullptr;
        const ScalarType s = t->scalar_type();
        if (s != ScalarType::Char && s != ScalarType::Float8_e4m3fn) {
            fail(PyExc_TypeError, "codes", "expected int8 or float8_e4m3fn");
            return nullptr;
        }
        if (t->dim() != 4 || t->size(1) != H || t->size(2) != Dv || t->size(3) != kHead) {
            fail(PyExc_ValueError, "codes", "expected a [slots, H, Dv, 128] tensor");
            return nullptr;
        }
        *format = s == ScalarType::Char ? KDA_Q8_INT8 : KDA_Q8_E4M3;
        *P = t->size(0);
        if (*P > 0x7fffffff) fail(PyExc_ValueError, "codes", "more than 2^31 - 1 slots");
        return take(o, "codes", s, -1);
    }
};

// The C entries run without the interpreter's lock, as through ctypes: a launch may wait for room in
// the stream's queue.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename Call>
PyObject* status(const Call& entry) {
    int rc;
    {
        const Unlocked unlocked;
        rc = entry();
    }
    return PyLong_FromLong(rc);
}

bool arity(const char* name, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, n);
    return false;
}

// (state, codes, scales, state_rows, slots, N, H, Dv, ring, ring_pool, stream)
template <bool STORE>
PyObject* state_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(STORE ? "state_store_q8" : "state_load_q8", n, 11)) return nullptr;
    Call c;
    const int64_t N = c.integer(a[5]), H = c.integer(a[6]), Dv = c.integer(a[7]);
    int format = 0;
    int64_t P = 0, S = 0, ring_row = 0;
    void* codes = c.pool(a[1], H, Dv, &format, &P);
    if (const at::Tensor* t = c.tensor(a[0], "state")) {
        if (t->dim() != 4 || t->size(1) != H || t->size(2) != Dv || t->size(3) != kHead)
            c.fail(PyExc_ValueError, "state", "expected a [rows, H, Dv, 128] tensor");
        S = t->size(0);
    }
    void* state = c.take(a[0], "state", ScalarType::Float, -1);
    void* scales = c.take(a[2], "scales", ScalarType::Float, P * H * Dv);
    void* rows = c.maybe(a[3], "state rows", ScalarType::Int, N);
    void* slots = c.maybe(a[4], "slots", ScalarType::Int, N);
    void *ring = nullptr, *ring_pool = nullptr;
    if ((a[8] == Py_None) != (a[9] == Py_None)) {
        c.fail(PyExc_ValueError, "ring, ring_pool", "both or neither");
    } else if (a[8] != Py_None) {
        const at::Tensor* r = c.tensor(a[8], "ring");
        const at::Tensor* p = c.tensor(a[9], "ring_pool");
        if (r != nullptr && p != nullptr) {
            if (r->dim() < 2 || p->dim() < 2 || r->size(0) != S || p->size(0) != P)
                c.fail(PyExc_ValueError, "ring, ring_pool", "expected one row for each state and slot");
            else
                ring_row = S > 0 ? r->numel() / S : (P > 0 ? p->numel() / P : 0);
        }
        ring = c.take(a[8], "ring", ScalarType::Float, S * ring_row);
        ring_pool = c.take(a[9], "ring_pool", ScalarType::Float, P * ring_row);
    }
    void* stream = c.stream(a[10]);
    if (c.failed) return nullptr;
    return status([&] {
        return STORE ? kda_state_store_q8((float*)state, codes, (float*)scales, format, (int*)rows,
                                          (int*)slots, (int)S, (int)P, (int)N, (int)H, (int)kHead, (int)Dv,
                                          (float*)ring, (float*)ring_pool, ring_row, stream)
                     : kda_state_load_q8(codes, (float*)scales, (float*)state, format, (int*)slots,
                                         (int*)rows, (int)P, (int)S, (int)N, (int)H, (int)kHead, (int)Dv,
                                         (float*)ring_pool, (float*)ring, ring_row, stream);
    });
}

// (q_raw, k_raw, v_raw, conv_w, ring_pool, f_raw, dt_bias, a_log, beta_raw, codes, scales, norm_w,
//  gate_raw, y, slots, slots_out, keep, N, T, H, Hk, Dv, K, gate_mode, gate_lb, l2_eps, scale,
//  rms_eps, stream)
PyObject* decode_fused_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("decode_fused_q8", n, 29)) return nullptr;
    Call c;
    const int64_t N = c.integer(a[17]), T = c.integer(a[18]), H = c.integer(a[19]), Hk = c.integer(a[20]);
    const int64_t Dv = c.integer(a[21]), K = c.integer(a[22]), mode = c.integer(a[23]);
    const float gate_lb = c.real(a[24]), l2_eps = c.real(a[25]), scale = c.real(a[26]), rms_eps = c.real(a[27]);
    int format = 0, raw_dtype = 0;
    int64_t P = 0;
    const ScalarType f32 = ScalarType::Float, i32 = ScalarType::Int;
    const ScalarType raw = c.float_type(a[0], "q_raw", &raw_dtype);
    void* codes = c.pool(a[9], H, Dv, &format, &P);
    // (sizes the C entry refuses give sums here that match no tensor, or an empty one)
    const int64_t rows = N * T, qk = Hk * kHead, v = H * Dv, channels = 2 * qk + v;
    const int64_t gate = (mode & KDA_GATE_PER_HEAD) != 0 ? H : H * kHead;
    void* q = c.take(a[0], "q_raw", raw, rows * qk);
    void* k = c.take(a[1], "k_raw", raw, rows * qk);
    void* vr = c.take(a[2], "v_raw", raw, rows * v);
    void* conv_w = c.take(a[3], "conv_w", f32, channels * K);
    void* ring = c.take(a[4], "ring_pool", f32, P * channels * (K - 1));
    void* f = c.take(a[5], "f_raw", f32, rows * gate);
    void* dt = c.take(a[6], "dt_bias", f32, gate);
    void* a_log = c.take(a[7], "a_log", f32, H);
    void* beta = c.take(a[8], "beta_raw", f32, rows * H);
    void* scales = c.take(a[10], "scales", f32, P * v);
    void* norm_w = c.take(a[11], "norm_w", f32, Dv);
    void* z = c.take(a[12], "gate_raw", f32, rows * v);
    void* y = c.take(a[13], "y", f32, rows * v);
    void* slots = c.maybe(a[14], "slots", i32, N);
    void* slots_out = c.maybe(a[15], "slots_out", i32, N);
    void* keep = c.maybe(a[16], "keep", i32, N);
    void* stream = c.stream(a[28]);
    if (c.failed) return nullptr;
    return status([&] {
        return kda_decode_fused_q8(
            q, k, vr, raw_dtype, (float*)conv_w, (float*)ring, (float*)f, (float*)dt, (float*)a_log,
            (int)mode, gate_lb, (float*)beta, codes, (float*)scales, format, (int*)slots, (int*)slots_out,
            (int*)keep, (float*)norm_w, (float*)z, (float*)y, (int)P, (int)N, (int)T, (int)H, (int)Hk,
            (int)kHead, (int)Dv, (int)K, l2_eps, scale, rms_eps, stream);
    });
}

// (x, weights, scales, zeros or None, outs, group, workspace or None, stream)
PyObject* proj_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("proj_w4", n, 8)) return nullptr;
    Call c;
    int x_dtype = 0, scale_dtype = 0;
    const ScalarType xt = c.float_type(a[0], "x", &x_dtype);
    int64_t t = 0, in_f = 0;
    if (const at::Tensor* x = c.tensor(a[0], "x")) {
        if (x->dim() != 2) c.fail(PyExc_ValueError, "x", "expected a [t, in_f] tensor");
        else t = x->size(0), in_f = x->size(1);
        if (t > (1 << 30) || in_f > (1 << 30)) c.fail(PyExc_ValueError, "x", "too large");
    }
    void* x = c.take(a[0], "x", xt, -1);
    const int64_t group = c.integer(a[5]);
    if (!c.failed && group <= 0) c.fail(PyExc_ValueError, "group", "expected 32, 64 or 128");
    if (c.failed) return nullptr;
    PyObject* lists[4] = {a[1], a[2], a[4], a[3]};          // weights, scales, outs, zeros
    static const char* const names[4] = {"weights", "scales", "outs", "zeros"};
    const int parts = a[3] == Py_None ? 3 : 4;
    Py_ssize_t nw = 0;
    for (int i = 0; i < parts; ++i) {
        if (!PyList_Check(lists[i]) && !PyTuple_Check(lists[i])) {
            c.fail(PyExc_TypeError, names[i], "expected a list of tensors");
            return nullptr;
        }
        const Py_ssize_t len = PySequence_Fast_GET_SIZE(lists[i]);
        if (i == 0) nw = len;
        if (len != nw || nw > kMaxWeights) {
            c.fail(PyExc_ValueError, names[i], "expected one entry for each of at most 8 weights");
            return nullptr;
        }
    }
    const void *w[kMaxWeights] = {}, *s[kMaxWeights] = {}, *z[kMaxWeights] = {};
    float* o[kMaxWeights] = {};
    int rows[kMaxWeights] = {};
    ScalarType st = ScalarType::Float;
    for (Py_ssize_t i = 0; i < nw; ++i) {
        PyObject* wo = PySequence_Fast_GET_ITEM(lists[0], i);
        PyObject* so = PySequence_Fast_GET_ITEM(lists[1], i);
        const at::Tensor* wt = c.tensor(wo, "weights");
        if (wt == nullptr) return nullptr;
        if (wt->dim() != 2 || wt->size(1) != in_f / 2 || wt->size(0) > 0x7fffffff) {
            c.fail(PyExc_ValueError, "weights", "expected [rows, in_f / 2] tensors");
            return nullptr;
        }
        const int64_t r = wt->size(0);
        rows[i] = (int)r;
        if (i == 0) st = c.float_type(so, "scales", &scale_dtype);
        w[i] = c.take(wo, "weights", ScalarType::Byte, -1);
        s[i] = c.take(so, "scales", st, r * (in_f / group));
        o[i] = (float*)c.take(PySequence_Fast_GET_ITEM(lists[2], i), "outs", ScalarType::Float, t * r);
        if (parts == 4)
            z[i] = c.take(PySequence_Fast_GET_ITEM(lists[3], i), "zeros", st, r * (in_f / group));
        if (c.failed) return nullptr;
    }
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[6] != Py_None) {
        ws = c.take(a[6], "workspace", ScalarType::Byte, -1);
        if (ws != nullptr) ws_bytes = (size_t)THPVariable_Unpack(a[6]).numel();
    }
    void* stream = c.stream(a[7]);
    if (c.failed) return nullptr;
    return status([&] {
        return kda_proj_w4(x, x_dtype, (int)t, (int)in_f, (int)nw, w, s, parts == 4 ? z : nullptr,
                           scale_dtype, (int)group, rows, o, ws, ws_bytes, stream);
    });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

// No C++ exception passes the interpreter's C frames: that would end the process.
template <Fast F>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyMethodDef methods[] = {
    {"state_store_q8", (PyCFunction)(void (*)(void))guarded<state_q8<true>>, METH_FASTCALL, nullptr},
    {"state_load_q8", (PyCFunction)(void (*)(void))guarded<state_q8<false>>, METH_FASTCALL, nullptr},
    {"decode_fused_q8", (PyCFunction)(void (*)(void))guarded<decode_fused_q8>, METH_FASTCALL, nullptr},
    {"proj_w4", (PyCFunction)(void (*)(void))guarded<proj_w4>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_native(void) { return PyModule_Create(&module); }
