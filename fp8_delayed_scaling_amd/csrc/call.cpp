// call.cpp -- the block operators' calls from Python without per-argument work in Python.
//
// Each function here takes a binding's arguments as they are and, when every one is what the call
// wants (dense tensors on the GPU of the right type and shape, None where that may be), calls the C
// entry point and returns True.  Arguments that do not fit, and those that the entry point refuses
// before it launches anything, give False: the binding then goes through its own checks, which name
// what is wrong.  A HIP error may come after a launch, so that call is not made again: it raises the
// binding's error from here.
//
// What it saves: a four-row norm takes 20 arguments, which ctypes and the checks in Python took 10.2 us
// for, the launch included; here the whole call takes 4.0 us on the host, 0.4 of them for the arguments,
// and the kernel runs 4.2.
#include <hip/hip_runtime_api.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "../../include/fp8ds.h"

namespace {

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat;
constexpr auto kU8 = at::kByte, kI32 = at::kInt;

// The arguments in order; ok turns false at the first that does not fit.
struct Args {
    PyObject *const *a;
    bool ok;
    Args(PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : a(args), ok(n == want) {}

    const at::Tensor *tensor(int i, at::ScalarType type) {
        if (!ok || !THPVariable_Check(a[i])) return fail();
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        return t.is_cuda() && t.scalar_type() == type ? &t : fail();
    }
    const at::Tensor *fail() {
        ok = false;
        return nullptr;
    }
    // a dense tensor of this shape, or None
    template <class T>
    T *dense(int i, at::ScalarType type, std::initializer_list<int64_t> shape, bool required = false) {
        if (!ok) return nullptr;
        if (a[i] == Py_None) {
            ok = !required;
            return nullptr;
        }
        const at::Tensor *t = tensor(i, type);
        if (t == nullptr) return nullptr;
        ok = t->is_contiguous() && t->sizes() == c10::IntArrayRef(shape);
        return static_cast<T *>(t->data_ptr());
    }
    // a dense tensor of at least n elements, or None
    template <class T>
    T *some(int i, at::ScalarType type, int64_t n) {
        if (!ok || a[i] == Py_None) return nullptr;
        const at::Tensor *t = tensor(i, type);
        if (t == nullptr) return nullptr;
        ok = t->is_contiguous() && t->numel() >= n;
        return static_cast<T *>(t->data_ptr());
    }
    // workspace: any dense tensor or None
    void *workspace(int i, size_t &bytes) {
        bytes = 0;
        if (!ok || a[i] == Py_None) return nullptr;
        if (!THPVariable_Check(a[i])) return fail(), nullptr;
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        ok = t.is_cuda() && t.is_contiguous();
        bytes = t.nbytes();
        return t.data_ptr();
    }
    int64_t integer(int i) {
        if (!ok) return 0;
        if (!PyLong_Check(a[i])) return fail(), 0;
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    // as the bindings' int(): what a C int holds
    int small(int i) {
        const int64_t v = integer(i);
        if (v != (int)v) ok = false;
        return (int)v;
    }
    int truth(int i) {
        if (!ok) return 0;
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v > 0;
    }
    float real(int i) {
        if (!ok) return 0.f;
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return (float)v;
    }
    // None: the current stream; a torch stream; a handle
    hipStream_t stream(int i) {
        if (!ok) return nullptr;
        if (a[i] == Py_None) return c10::hip::getCurrentHIPStream().stream();
        void *p = nullptr;
        if (PyLong_Check(a[i])) {
            p = PyLong_AsVoidPtr(a[i]);
        } else {
            PyObject *handle = PyObject_GetAttrString(a[i], "cuda_stream");
            if (handle != nullptr) p = PyLong_AsVoidPtr(handle);
            Py_XDECREF(handle);
        }
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<hipStream_t>(p);
    }
    // [T, H, D] bfloat16 with strides of its own, the elements of a head one behind the other; or None
    fp8ds_heads heads(int i, int64_t T, int64_t H, int64_t D, bool required = true) {
        fp8ds_heads h{nullptr, D, D};
        if (!ok) return h;
        if (a[i] == Py_None) {
            ok = !required;
            return h;
        }
        const at::Tensor *t = tensor(i, kBf16);
        if (t == nullptr) return h;
        ok = t->sizes() == c10::IntArrayRef({T, H, D}) && (t->numel() == 0 || t->stride(2) == 1);
        if (!ok) return h;
        h.data = static_cast<uint16_t *>(t->data_ptr());
        if (T > 1) h.token_stride = t->stride(0);      // of a single token or head a stride says nothing
        if (H > 1) h.head_stride = t->stride(1);
        return h;
    }
    // gate [G, H] with G dividing the rows, or None
    const uint16_t *gate(int i, int64_t rows, int64_t width, int64_t &n) {
        n = 0;
        if (!ok || a[i] == Py_None) return nullptr;
        const at::Tensor *t = tensor(i, kBf16);
        if (t == nullptr) return nullptr;
        ok = t->is_contiguous() && t->dim() == 2 && t->size(1) == width && t->size(0) >= 1 && rows % t->size(0) == 0;
        if (ok) n = t->size(0);
        return static_cast<const uint16_t *>(t->data_ptr());
    }
};

PyObject *done(bool ok) { return PyBool_FromLong(ok); }
// Makes the call with the interpreter's lock released, as ctypes does: a launch waits while the GPU's
// queue is full.
template <class Call> PyObject *done_with(Call call) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    if (status != FP8DS_ERR_HIP) return done(status == FP8DS_OK);
    PyObject *package = PyImport_ImportModule("fp8_delayed_scaling_amd");
    PyObject *never = package != nullptr ? PyObject_CallMethod(package, "_check", "i", status) : nullptr;      // raises
    Py_XDECREF(package);
    return never;
}

PyObject *norm_fwd(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 20);
    if (!a.ok) return done(false);
    const at::Tensor *ref = a.tensor(args[0] == Py_None ? 4 : 0, kBf16);
    if (ref == nullptr || ref->dim() != 2) return done(false);
    const int64_t M = ref->size(0), H = ref->size(1);
    const int kind = a.small(17);
    const int64_t stats = kind == FP8DS_NORM_LAYER ? 2 * M : M;
    const auto *o = a.dense<uint16_t>(0, kBf16, {M, H});
    const auto *w_post = a.dense<uint16_t>(1, kBf16, {H}), *b_post = a.dense<uint16_t>(2, kBf16, {H});
    int64_t G;
    const auto *gate = a.gate(3, M, H, G);
    const auto *resid = a.dense<uint16_t>(4, kBf16, {M, H});
    const float alpha = a.real(5);
    auto *x = a.dense<uint16_t>(6, kBf16, {M, H}, o != nullptr);
    auto *post = a.some<float>(7, kF32, stats);
    const auto *w_pre = a.dense<uint16_t>(8, kBf16, {H}), *b_pre = a.dense<uint16_t>(9, kBf16, {H});
    auto *pre = a.some<float>(10, kF32, stats);
    auto *h = a.dense<uint16_t>(11, kBf16, {M, H});
    auto *h8 = a.dense<uint8_t>(12, kU8, {M, H});
    const auto *scale = a.some<float>(13, kF32, 1);
    const int fmt = a.small(14);
    auto *sinv = a.some<float>(15, kF32, 1), *amax = a.some<float>(16, kF32, 1);
    const float eps = a.real(18);
    const hipStream_t st = a.stream(19);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_norm_residual_fwd(o, w_post, b_post, gate, G, resid, alpha, x, post, w_pre, b_pre, pre, h, h8, scale,
                                     fmt, sinv, amax, kind, eps, M, H, st);
    });
}

PyObject *norm_bwd(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 21);
    if (!a.ok) return done(false);
    const at::Tensor *ref = a.tensor(args[0] != Py_None ? 0 : 1, kBf16);
    if (ref == nullptr || ref->dim() != 2) return done(false);
    const int64_t M = ref->size(0), H = ref->size(1);
    const int kind = a.small(19);
    const int64_t stats = kind == FP8DS_NORM_LAYER ? 2 * M : M;
    const auto *dh = a.dense<uint16_t>(0, kBf16, {M, H}), *dx = a.dense<uint16_t>(1, kBf16, {M, H});
    const auto *o = a.dense<uint16_t>(2, kBf16, {M, H});
    const auto *w_post = a.dense<uint16_t>(3, kBf16, {H}), *b_post = a.dense<uint16_t>(4, kBf16, {H});
    int64_t G;
    const auto *gate = a.gate(5, M, H, G);
    const float alpha = a.real(6);
    const auto *x = a.dense<uint16_t>(7, kBf16, {M, H});
    const auto *post = a.some<float>(8, kF32, stats);
    const auto *w_pre = a.dense<uint16_t>(9, kBf16, {H});
    const auto *pre = a.some<float>(10, kF32, stats);
    auto *d_block = a.dense<uint16_t>(11, kBf16, {M, H}), *d_resid = a.dense<uint16_t>(12, kBf16, {M, H});
    auto *dw_post = a.dense<float>(13, kF32, {H}), *db_post = a.dense<float>(14, kF32, {H});
    auto *dgate = a.dense<float>(15, kF32, {G > 1 ? G : 1, H});
    auto *dw_pre = a.dense<float>(16, kF32, {H}), *db_pre = a.dense<float>(17, kF32, {H});
    size_t bytes;
    void *ws = a.workspace(18, bytes);
    const hipStream_t st = a.stream(20);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_norm_residual_bwd(dh, dx, o, w_post, b_post, gate, G, alpha, x, post, w_pre, pre, d_block, d_resid,
                                     dw_post, db_post, dgate, dw_pre, db_pre, ws, bytes, kind, M, H, st);
    });
}

PyObject *moe_plan(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 8);
    const at::Tensor *e = a.tensor(0, kI32), *s = a.ok ? a.tensor(4, kI32) : nullptr;
    if (!a.ok || e->dim() != 2) return done(false);
    const int64_t T = e->size(0), k = e->size(1), E = a.integer(1), align = a.integer(2), cap = s->numel();
    const auto *experts = a.dense<int32_t>(0, kI32, {T, k});
    auto *offsets = a.dense<int32_t>(3, kI32, {E + 1}, true);
    auto *src = a.some<int32_t>(4, kI32, cap);
    auto *slot = a.dense<int32_t>(5, kI32, {T, k}, true);
    size_t bytes;
    void *ws = a.workspace(6, bytes);
    const hipStream_t st = a.stream(7);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_moe_plan(experts, T, k, E, align, cap, offsets, src, slot, ws, bytes, st);
    });
}

PyObject *moe_sort_cast(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 11);
    const at::Tensor *t = a.tensor(0, kBf16), *s = a.ok ? a.tensor(1, kI32) : nullptr;
    if (!a.ok || t->dim() != 2) return done(false);
    const int64_t T = t->size(0), H = t->size(1), cap = s->numel(), top = a.integer(2);
    const auto *x = a.dense<uint16_t>(0, kBf16, {T, H});
    const auto *src = a.some<int32_t>(1, kI32, cap);
    const auto *w = a.dense<float>(3, kF32, {T, top});
    const auto *scale = a.some<float>(4, kF32, 1);
    const int fmt = a.small(5);
    auto *out = a.dense<uint8_t>(6, kU8, {cap, H}, true), *out_t = a.dense<uint8_t>(7, kU8, {H, cap});
    auto *sinv = a.some<float>(8, kF32, 1), *amax = a.some<float>(9, kF32, 1);
    const hipStream_t st = a.stream(10);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_moe_sort_cast(x, T, src, cap, top, w, scale, fmt, out, out_t, sinv, amax, H, st);
    });
}

PyObject *moe_sort_codes(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 6);
    const at::Tensor *t = a.tensor(0, kU8), *s = a.ok ? a.tensor(1, kI32) : nullptr;
    if (!a.ok || t->dim() != 2) return done(false);
    const int64_t T = t->size(0), H = t->size(1), cap = s->numel(), top = a.integer(2);
    const auto *x = a.dense<uint8_t>(0, kU8, {T, H});
    const auto *src = a.some<int32_t>(1, kI32, cap);
    auto *out = a.dense<uint8_t>(3, kU8, {cap, H}, true), *out_t = a.dense<uint8_t>(4, kU8, {H, cap});
    const hipStream_t st = a.stream(5);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_moe_sort_codes(x, T, src, cap, top, out, out_t, H, st);
    });
}

PyObject *moe_combine(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 5);
    const at::Tensor *t = a.tensor(0, kBf16), *s = a.ok ? a.tensor(1, kI32) : nullptr;
    if (!a.ok || t->dim() != 2 || s->dim() != 2) return done(false);
    const int64_t cap = t->size(0), H = t->size(1), T = s->size(0), k = s->size(1);
    const auto *ys = a.dense<uint16_t>(0, kBf16, {cap, H});
    const auto *slot = a.dense<int32_t>(1, kI32, {T, k});
    const auto *w = a.dense<float>(2, kF32, {T, k});
    auto *y = a.dense<uint16_t>(3, kBf16, {T, H}, true);
    const hipStream_t st = a.stream(4);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_moe_combine(ys, cap, slot, w, T, k, y, H, st);
    });
}

PyObject *moe_weight_grad(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 5);
    const at::Tensor *t = a.tensor(1, kBf16), *s = a.ok ? a.tensor(2, kI32) : nullptr;
    if (!a.ok || t->dim() != 2 || s->dim() != 2) return done(false);
    const int64_t cap = t->size(0), H = t->size(1), T = s->size(0), k = s->size(1);
    const auto *dy = a.dense<uint16_t>(0, kBf16, {T, H}, true);
    const auto *ys = a.dense<uint16_t>(1, kBf16, {cap, H});
    const auto *slot = a.dense<int32_t>(2, kI32, {T, k});
    auto *dw = a.dense<float>(3, kF32, {T, k}, true);
    const hipStream_t st = a.stream(4);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_moe_weight_grad(dy, ys, cap, slot, T, k, dw, H, st);
    });
}

// Output of the experts' products: its type, with unit stride along the rows.
const at::Tensor *output(Args &a, int i, int &dtype) {
    if (!a.ok || !THPVariable_Check(a.a[i])) return a.fail();
    const at::Tensor &t = THPVariable_Unpack(a.a[i]);
    dtype = t.scalar_type() == kBf16 ? FP8DS_OUT_BF16 : FP8DS_OUT_FP32;
    return t.is_cuda() && (t.scalar_type() == kBf16 || t.scalar_type() == kF32) ? &t : a.fail();
}
bool rows_dense(const at::Tensor *t) { return t->numel() == 0 || t->stride(-1) == 1; }

PyObject *grouped_gemm(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 9);
    const at::Tensor *A = a.tensor(0, kU8), *B = a.ok ? a.tensor(3, kU8) : nullptr;
    int dtype = 0;
    const at::Tensor *D = output(a, 7, dtype);
    if (!a.ok || A->dim() != 2 || B->dim() != 3 || D->dim() != 2 || A->size(1) != B->size(2)) return done(false);
    const int64_t cap = A->size(0), K = A->size(1), E = B->size(0), N = B->size(1);
    if (D->size(0) != cap || D->size(1) != N || !rows_dense(A) || !rows_dense(B) || !rows_dense(D)) return done(false);
    const int fa = a.small(1), fb = a.small(4);
    const auto *sa = a.some<float>(2, kF32, 1), *sb = a.some<float>(5, kF32, 1);
    const auto *off = a.dense<int32_t>(6, kI32, {E + 1}, true);
    const hipStream_t st = a.stream(8);
    if (!a.ok) return done(false);
    const auto *pa = static_cast<const uint8_t *>(A->data_ptr()), *pb = static_cast<const uint8_t *>(B->data_ptr());
    void *pd = D->data_ptr();
    return done_with([&] {
        return fp8_grouped_gemm(pa, fa, sa, A->stride(0), pb, fb, sb, B->stride(1), B->stride(0), off, E, pd,
                                D->stride(0), dtype, cap, N, K, st);
    });
}

PyObject *grouped_wgrad(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 9);
    const at::Tensor *A = a.tensor(0, kU8), *B = a.ok ? a.tensor(3, kU8) : nullptr;
    const at::Tensor *off = a.ok ? a.tensor(6, kI32) : nullptr;
    int dtype = 0;
    const at::Tensor *D = output(a, 7, dtype);
    if (!a.ok || A->dim() != 2 || B->dim() != 2 || A->size(1) != B->size(1) || off->numel() < 1 || !off->is_contiguous()) return done(false);
    const int64_t N = A->size(0), cap = A->size(1), K = B->size(0), E = off->numel() - 1;
    if (!rows_dense(A) || !rows_dense(B) || !D->is_contiguous() || D->sizes() != c10::IntArrayRef({E, N, K})) return done(false);
    const int fa = a.small(1), fb = a.small(4);
    const auto *sa = a.some<float>(2, kF32, 1), *sb = a.some<float>(5, kF32, 1);
    const hipStream_t st = a.stream(8);
    if (!a.ok) return done(false);
    const auto *pa = static_cast<const uint8_t *>(A->data_ptr()), *pb = static_cast<const uint8_t *>(B->data_ptr());
    const auto *po = static_cast<const int32_t *>(off->data_ptr());
    void *pd = D->data_ptr();
    return done_with([&] {
        return fp8_grouped_wgrad(pa, fa, sa, A->stride(0), pb, fb, sb, B->stride(0), po, E, pd, dtype, cap, N, K, st);
    });
}

// q [Tq, Hq, D] and k [Tk, Hkv, D] give an attention's sizes, the offsets (both or neither) its sequences.
struct AttentionSizes {
    int64_t Tq = 0, Hq = 0, D = 0, Tk = 0, Hkv = 0, B = 0;
    const int32_t *off_q = nullptr, *off_k = nullptr;
    AttentionSizes(Args &a, int q, int k, int offsets_q, int offsets_k, int batch) {
        const at::Tensor *tq = a.tensor(q, kBf16), *tk = a.ok ? a.tensor(k, kBf16) : nullptr;
        if (!a.ok || tq->dim() != 3 || tk->dim() != 3) {
            a.ok = false;
            return;
        }
        Tq = tq->size(0), Hq = tq->size(1), D = tq->size(2), Tk = tk->size(0), Hkv = tk->size(1);
        if (a.a[offsets_q] == Py_None) {
            B = a.integer(batch);
            a.ok = a.ok && a.a[offsets_k] == Py_None;
            return;
        }
        const at::Tensor *o = a.tensor(offsets_q, kI32);
        if (o == nullptr) return;
        B = o->numel() - 1;
        off_q = a.dense<int32_t>(offsets_q, kI32, {B + 1}, true);
        off_k = a.dense<int32_t>(offsets_k, kI32, {B + 1}, true);
    }
    float scale(Args &a, int i) const { return a.ok && a.a[i] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : a.real(i); }
};

PyObject *attention_fwd(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 18);
    if (!a.ok) return done(false);
    const AttentionSizes z(a, 0, 1, 5, 6, 7);
    const fp8ds_heads q = a.heads(0, z.Tq, z.Hq, z.D), k = a.heads(1, z.Tk, z.Hkv, z.D), v = a.heads(2, z.Tk, z.Hkv, z.D);
    const fp8ds_heads out = a.heads(3, z.Tq, z.Hq, z.D, false);
    auto *lse = a.dense<float>(4, kF32, {z.Hq, z.Tq});
    const int causal = a.truth(8);
    const int64_t window = a.integer(9);
    const float scale = z.scale(a, 10);
    auto *out8 = a.dense<uint8_t>(11, kU8, {z.Tq, z.Hq * z.D});
    const auto *s8 = a.some<float>(12, kF32, 1);
    const int fmt = a.small(13);
    auto *sinv = a.some<float>(14, kF32, 1), *amax = a.some<float>(15, kF32, 1);
    size_t bytes;
    void *ws = a.workspace(16, bytes);
    const hipStream_t st = a.stream(17);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_attention_fwd(q, k, v, out, lse, out8, s8, fmt, sinv, amax, z.off_q, z.off_k, z.B, z.Tq, z.Tk, z.Hq, z.Hkv,
                                 z.D, scale, causal, window, ws, bytes, st);
    });
}

PyObject *attention_bwd(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 17);
    if (!a.ok) return done(false);
    const AttentionSizes z(a, 1, 2, 10, 11, 12);
    const fp8ds_heads dout = a.heads(0, z.Tq, z.Hq, z.D), q = a.heads(1, z.Tq, z.Hq, z.D), k = a.heads(2, z.Tk, z.Hkv, z.D);
    const fp8ds_heads v = a.heads(3, z.Tk, z.Hkv, z.D), out = a.heads(4, z.Tq, z.Hq, z.D);
    const auto *lse = a.dense<float>(5, kF32, {z.Hq, z.Tq}, true);
    const fp8ds_heads dq = a.heads(6, z.Tq, z.Hq, z.D), dk = a.heads(7, z.Tk, z.Hkv, z.D), dv = a.heads(8, z.Tk, z.Hkv, z.D);
    size_t bytes;
    void *ws = a.workspace(9, bytes);
    const int causal = a.truth(13);
    const int64_t window = a.integer(14);
    const float scale = z.scale(a, 15);
    const hipStream_t st = a.stream(16);
    if (!a.ok) return done(false);
    return done_with([&] {
        return fp8_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, z.off_q, z.off_k, z.B, z.Tq, z.Tk, z.Hq, z.Hkv, z.D, scale,
                                 causal, window, ws, bytes, st);
    });
}

// Rows of logits: float32 or bfloat16, [T, E], unit stride along a row.
const at::Tensor *logits_of(Args &a, int i, int &dtype) {
    const at::Tensor *t = output(a, i, dtype);
    if (t == nullptr) return nullptr;
    return t->dim() == 2 && (t->size(1) <= 1 || rows_dense(t)) ? t : a.fail();
}
int64_t row_stride(const at::Tensor *t) { return t->size(0) > 1 ? t->stride(0) : t->size(1); }

PyObject *moe_route(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 10);
    int dtype = 0;
    const at::Tensor *l = logits_of(a, 0, dtype), *x = a.ok ? a.tensor(1, kI32) : nullptr;
    if (!a.ok || x->dim() != 2) return done(false);
    const int64_t T = l->size(0), E = l->size(1), top = x->size(1);
    auto *experts = a.dense<int32_t>(1, kI32, {T, top}, true);
    auto *weights = a.dense<float>(2, kF32, {T, top}, true), *lse = a.dense<float>(3, kF32, {T}, true);
    auto *counts = a.dense<int32_t>(4, kI32, {E + 1}, true);
    auto *prob_sum = a.dense<float>(5, kF32, {E}, true), *loss = a.some<float>(6, kF32, 1);
    size_t bytes;
    void *ws = a.workspace(7, bytes);
    const int normalise = a.truth(8);
    const hipStream_t st = a.stream(9);
    if (!a.ok) return done(false);
    const void *pl = l->data_ptr();
    return done_with([&] {
        return fp8_moe_route(pl, dtype, row_stride(l), T, E, top, normalise, experts, weights, lse, counts, prob_sum, loss, ws, bytes, st);
    });
}

PyObject *moe_route_bwd(PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 10);
    int dtype = 0, dtype_d = 0;
    const at::Tensor *l = logits_of(a, 0, dtype), *x = a.ok ? a.tensor(1, kI32) : nullptr, *d = logits_of(a, 7, dtype_d);
    if (!a.ok || x->dim() != 2 || dtype != dtype_d || l->sizes() != d->sizes()) return done(false);
    const int64_t T = l->size(0), E = l->size(1), top = x->size(1);
    const auto *experts = a.dense<int32_t>(1, kI32, {T, top}, true);
    const auto *weights = a.dense<float>(2, kF32, {T, top}, true), *lse = a.dense<float>(3, kF32, {T}, true);
    const auto *counts = a.dense<int32_t>(4, kI32, {E + 1}, true);
    const auto *dweights = a.dense<float>(5, kF32, {T, top}), *dloss = a.some<float>(6, kF32, 1);
    const int normalise = a.truth(8);
    const hipStream_t st = a.stream(9);
    if (!a.ok) return done(false);
    const void *pl = l->data_ptr();
    void *pd = d->data_ptr();
    return done_with([&] {
        return fp8_moe_route_bwd(pl, dtype, row_stride(l), T, E, top, normalise, experts, weights, lse, counts, dweights, dloss, pd,
                                 row_stride(d), st);
    });
}

// PyTorch raises C++ exceptions for tensors without storage or strides, and where there is no GPU to
// have a current stream.  None may leave a function that C calls: the binding's checks raise them again.
template <PyObject *(*call)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) noexcept {
    try {
        return call(args, n);
    } catch (...) {
        PyErr_Clear();
        return done(false);
    }
}

#define FP8DS_CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8DS_CALL(norm_fwd),      FP8DS_CALL(norm_bwd),    FP8DS_CALL(moe_plan),        FP8DS_CALL(moe_sort_cast),
                         FP8DS_CALL(moe_sort_codes), FP8DS_CALL(moe_combine), FP8DS_CALL(moe_weight_grad), FP8DS_CALL(grouped_gemm),
                         FP8DS_CALL(grouped_wgrad), FP8DS_CALL(attention_fwd), FP8DS_CALL(attention_bwd), FP8DS_CALL(moe_route),
                         FP8DS_CALL(moe_route_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "The block operators' calls.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call(void) { return PyModule_Create(&module); }
