// kda_native.cpp -- CPython marshalling of the entry points whose host time is a step's latency:
// the decode on the 8-bit state pool, the pool's store and load, the 4-bit projections, linear
// attention, the verification of drafts and the norms around a block.  One
// token's kernels run a few microseconds; checking and unpacking 17 to 28 tensors attribute by
// attribute in Python took 9 to 16 us a call, here it takes about one.  Each function checks that
// every tensor is a CUDA tensor of the right type and size on one device, contiguous but for what may
// have its rows apart (linear attention's q, k and v, the probabilities) (ValueError or TypeError
// otherwise), calls the C entry of the same name and returns its status.  What torch throws
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
    // a required [rows, width] tensor of `type` whose rows may lie apart; *stride: elements between them
    void* rows2d(PyObject* o, const char* name, ScalarType type, int64_t rows, int64_t width, long* stride) {
        const at::Tensor* t = tensor(o, name);
        if (t == nullptr) return nullptr;
        *stride = (long)width;
        if (!t->is_cuda()) {
            fail(PyExc_ValueError, name, "expected a CUDA tensor");
        } else if (t->scalar_type() != type) {
            failed = true;
            PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(type),
                         c10::toString(t->scalar_type()));
        } else if (t->dim() != 2 || t->size(0) != rows || t->size(1) != width) {
            failed = true;
            PyErr_Format(PyExc_ValueError, "%s: expected a [%lld, %lld] tensor", name, (long long)rows,
                         (long long)width);
        } else if (width > 1 && t->stride(1) != 1) {
            fail(PyExc_ValueError, name, "expected rows of adjacent elements");
        } else {
            if (device == -2) device = t->get_device();
            if (t->get_device() != device) {
                failed = true;
                PyErr_Format(PyExc_ValueError, "%s: expected a tensor on cuda:%d, got cuda:%d", name, device,
                             (int)t->get_device());
            }
            if (rows > 1) *stride = (long)t->stride(0);
        }
        return failed ? nullptr : t->data_ptr();
    }
    // a required [a, b, width] tensor whose a * b rows lie evenly apart; *stride: elements between them
    void* rows3d(PyObject* o, const char* name, ScalarType type, int64_t a, int64_t b, int64_t width,
                 long* stride) {
        const at::Tensor* t = tensor(o, name);
        if (t == nullptr) return nullptr;
        if (t->dim() != 3 || t->size(0) != a || t->size(1) != b || t->size(2) != width) {
            failed = true;
            PyErr_Format(PyExc_ValueError, "%s: expected a [%lld, %lld, %lld] tensor", name, (long long)a,
                         (long long)b, (long long)width);
            return nullptr;
        }
        if (!t->is_cuda()) {
            fail(PyExc_ValueError, name, "expected a CUDA tensor");
            return nullptr;
        }
        if (device == -2) device = t->get_device();
        const int64_t row = b > 1 ? t->stride(1) : a > 1 ? t->stride(0) : width;
        if (t->scalar_type() != type) {
            failed = true;
            PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, c10::toString(type),
                         c10::toString(t->scalar_type()));
        } else if (t->get_device() != device) {
            fail(PyExc_ValueError, name, "expected a tensor on the other tensors' device");
        } else if ((width > 1 && t->stride(2) != 1) || (a > 1 && b > 1 && t->stride(0) != b * row)) {
            fail(PyExc_ValueError, name, "expected rows of adjacent elements, evenly apart");
        }
        *stride = (long)row;
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

// What the linear attention calls share: q, k, v rows and their strides.
struct LinRows {
    int dtype = 0;
    long qs = 0, ks = 0, vs = 0;
    void *q, *k, *v;
    LinRows(Call& c, PyObject* const* a, int64_t rows, int64_t H, int64_t Hk, int64_t Dv) {
        const ScalarType t = c.float_type(a[0], "q", &dtype);
        q = c.rows2d(a[0], "q", t, rows, Hk * kHead, &qs);
        k = c.rows2d(a[1], "k", t, rows, Hk * kHead, &ks);
        v = c.rows2d(a[2], "v", t, rows, H * Dv, &vs);
    }
};

// (q, k, v, log_decay, state_in or None, state_out, o, workspace or None, cu_seqlens or None,
//  cu_seqlens_host or None, N, T, H, Hk, Dv, scale, algo, stream); T: tokens of each sequence without
// cu_seqlens, ignored with it; algo: KDA_ALGO_AUTO or KDA_ALGO_SEQ
PyObject* linattn_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("linattn_prefill", n, 18)) return nullptr;
    Call c;
    int64_t N = c.integer(a[10]), T = c.integer(a[11]);
    const int64_t H = c.integer(a[12]), Hk = c.integer(a[13]), Dv = c.integer(a[14]);
    const float scale = c.real(a[15]);
    const int64_t algo = c.integer(a[16]);
    if (!c.failed && algo != KDA_ALGO_AUTO && algo != KDA_ALGO_SEQ) return PyLong_FromLong(KDA_ERR_ENUM);
    const bool varlen = a[8] != Py_None;
    int64_t rows = N * T;
    const int* cu_host = nullptr;
    if (varlen) {
        const at::Tensor* h = c.tensor(a[9], "cu_seqlens_host");
        if (h != nullptr && (h->is_cuda() || h->scalar_type() != ScalarType::Int || !h->is_contiguous() ||
                             h->numel() < 1))
            c.fail(PyExc_ValueError, "cu_seqlens_host", "expected a contiguous int32 CPU tensor [N + 1]");
        if (c.failed) return nullptr;
        cu_host = h->data_ptr<int>();
        N = h->numel() - 1;
        rows = cu_host[N];
        // (before any size follows from them)
        for (int64_t i = 0; i < N; ++i)
            if (cu_host[i + 1] < cu_host[i]) return PyLong_FromLong(KDA_ERR_CU_SEQLENS);
        if (cu_host[0] != 0) return PyLong_FromLong(KDA_ERR_CU_SEQLENS);
    }
    const LinRows r(c, a, rows, H, Hk, Dv);
    void* g = c.take(a[3], "log_decay", ScalarType::Float, H);
    void* s_in = c.maybe(a[4], "state_in", ScalarType::Float, N * H * Dv * kHead);
    void* s_out = c.take(a[5], "state_out", ScalarType::Float, N * H * Dv * kHead);
    void* o = c.take(a[6], "o", ScalarType::Float, rows * H * Dv);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[7] != Py_None) {
        ws = c.take(a[7], "workspace", ScalarType::Byte, -1);
        if (ws != nullptr) ws_bytes = (size_t)THPVariable_Unpack(a[7]).numel();
    }
    void* cu = varlen ? c.take(a[8], "cu_seqlens", ScalarType::Int, N + 1) : nullptr;
    void* stream = c.stream(a[17]);
    if (c.failed) return nullptr;
    const int dtype = algo == KDA_ALGO_SEQ ? r.dtype | KDA_LINATTN_SEQ : r.dtype;
    return status([&] {
        return varlen ? kda_linattn_prefill_varlen(r.q, r.qs, r.k, r.ks, r.v, r.vs, dtype, (float*)g,
                                                   (float*)s_in, (float*)s_out, (float*)o, (int*)cu, cu_host,
                                                   (int)N, (int)rows, (int)H, (int)Hk, (int)kHead, (int)Dv,
                                                   scale, ws, ws_bytes, stream)
                      : kda_linattn_prefill(r.q, r.qs, r.k, r.ks, r.v, r.vs, dtype, (float*)g,
                                            (float*)s_in, (float*)s_out, (float*)o, (int)N, (int)T, (int)H,
                                            (int)Hk, (int)kHead, (int)Dv, scale, ws, ws_bytes, stream);
    });
}

// (q, k, v, log_decay, pool, o, slots, slots_out, keep, N, T, H, Hk, Dv, scale, stream)
PyObject* linattn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("linattn_decode", n, 16)) return nullptr;
    Call c;
    const int64_t N = c.integer(a[9]), T = c.integer(a[10]), H = c.integer(a[11]), Hk = c.integer(a[12]);
    const int64_t Dv = c.integer(a[13]);
    const float scale = c.real(a[14]);
    const LinRows r(c, a, N * T, H, Hk, Dv);
    int64_t P = 0;
    if (const at::Tensor* t = c.tensor(a[4], "pool")) {
        if (t->dim() != 4 || t->size(1) != H || t->size(2) != Dv || t->size(3) != kHead ||
            t->size(0) > 0x7fffffff)
            c.fail(PyExc_ValueError, "pool", "expected a [slots, H, Dv, 128] tensor");
        else
            P = t->size(0);
    }
    void* g = c.take(a[3], "log_decay", ScalarType::Float, H);
    void* pool = c.take(a[4], "pool", ScalarType::Float, -1);
    void* o = c.take(a[5], "o", ScalarType::Float, N * T * H * Dv);
    void* slots = c.maybe(a[6], "slots", ScalarType::Int, N);
    void* slots_out = c.maybe(a[7], "slots_out", ScalarType::Int, N);
    void* keep = c.maybe(a[8], "keep", ScalarType::Int, N);
    void* stream = c.stream(a[15]);
    if (c.failed) return nullptr;
    return status([&] {
        return kda_linattn_decode(r.q, r.qs, r.k, r.ks, r.v, r.vs, r.dtype, (float*)g, (float*)pool,
                                  (int*)slots, (int*)slots_out, (int*)keep, (float*)o, (int)P, (int)N,
                                  (int)T, (int)H, (int)Hk, (int)kHead, (int)Dv, scale, stream);
    });
}

// (target, tokens, u, r, keep, out_tokens, draft or None, n_draft or None, stream)
PyObject* draft_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("draft_accept", n, 9)) return nullptr;
    Call c;
    int dtype = 0;
    const ScalarType pt = c.float_type(a[0], "target", &dtype);
    int64_t N = 0, T = 0, V = 0;
    if (const at::Tensor* t = c.tensor(a[0], "target")) {
        if (t->dim() != 3 || t->size(0) > (1 << 30) || t->size(1) > (1 << 30) || t->size(2) > 0x7fffffff)
            c.fail(PyExc_ValueError, "target", "expected a [N, T, V] tensor");
        else
            N = t->size(0), T = t->size(1), V = t->size(2);
    }
    if (!c.failed && T < 1) c.fail(PyExc_ValueError, "target", "expected at least one row a sequence");
    if (c.failed) return nullptr;
    long ts = 0, ds = 0;
    void* target = c.rows3d(a[0], "target", pt, N, T, V, &ts);
    void* draft = a[6] == Py_None ? nullptr : c.rows3d(a[6], "draft", pt, N, T - 1, V, &ds);
    void* tokens = c.take(a[1], "tokens", ScalarType::Int, N * (T - 1));
    void* u = c.take(a[2], "u", ScalarType::Float, N * (T - 1));
    void* r = c.take(a[3], "r", ScalarType::Float, N);
    void* keep = c.take(a[4], "keep", ScalarType::Int, N);
    void* out = c.take(a[5], "out_tokens", ScalarType::Int, N * T);
    void* nd = c.maybe(a[7], "n_draft", ScalarType::Int, N);
    void* stream = c.stream(a[8]);
    if (c.failed) return nullptr;
    return status([&] {
        return kda_draft_accept(target, ts, draft, ds, dtype, (int*)tokens, (float*)u, (float*)r, (int*)nd,
                                (int*)keep, (int*)out, (int)N, (int)T, (int)V, stream);
    });
}

// (residual, block or None, h or None, z or None, norm_w or None, block_w or None, gate or None,
//  gate_act, res_scale, block_scale, eps, stream)
PyObject* residual_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity("residual_rmsnorm", n, 12)) return nullptr;
    Call c;
    int rt = 0, bt = 0, zt = 0, per_row = 0;
    const ScalarType res_t = c.float_type(a[0], "residual", &rt);
    const ScalarType blk_t = a[1] == Py_None ? res_t : c.float_type(a[1], "block", &bt);
    const ScalarType z_t = a[3] == Py_None ? res_t : c.float_type(a[3], "z", &zt);
    int64_t rows = 0, F = 0;
    if (const at::Tensor* t = c.tensor(a[0], "residual")) {
        if (t->dim() != 2 || t->size(0) > 0x7fffffff || t->size(1) > 0x7fffffff)
            c.fail(PyExc_ValueError, "residual", "expected a [rows, F] tensor");
        else
            rows = t->size(0), F = t->size(1);
    }
    const int64_t act = c.integer(a[7]);
    const float rs = c.real(a[8]), bs = c.real(a[9]), eps = c.real(a[10]);
    const ScalarType f32 = ScalarType::Float;
    void* res = c.take(a[0], "residual", res_t, -1);
    void* blk = c.maybe(a[1], "block", blk_t, rows * F);
    void* h = c.maybe(a[2], "h", res_t, rows * F);
    void* z = c.maybe(a[3], "z", z_t, rows * F);
    void* nw = c.maybe(a[4], "norm_w", f32, F);
    void* bw = c.maybe(a[5], "block_w", f32, F);
    void* gate = nullptr;
    if (a[6] != Py_None) {
        if (const at::Tensor* t = c.tensor(a[6], "gate")) {
            per_row = t->dim() != 1;
            gate = c.take(a[6], "gate", per_row ? blk_t : f32, per_row ? rows * F : F);
        }
    }
    void* stream = c.stream(a[11]);
    if (c.failed) return nullptr;
    return status([&] {
        return kda_residual_rmsnorm(res, rt, blk, bt, (float*)bw, gate, per_row, (int)act, rs, bs, (float*)nw,
                                    h, z, zt, (long)rows, (int)F, eps, stream);
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
    {"linattn_prefill", (PyCFunction)(void (*)(void))guarded<linattn_prefill>, METH_FASTCALL, nullptr},
    {"linattn_decode", (PyCFunction)(void (*)(void))guarded<linattn_decode>, METH_FASTCALL, nullptr},
    {"draft_accept", (PyCFunction)(void (*)(void))guarded<draft_accept>, METH_FASTCALL, nullptr},
    {"residual_rmsnorm", (PyCFunction)(void (*)(void))guarded<residual_rmsnorm>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_native(void) { return PyModule_Create(&module); }
