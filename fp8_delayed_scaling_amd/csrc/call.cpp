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
                         FP8DS_CALL(grouped_wgrad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "The block operators' calls.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call(void) { return PyModule_Create(&module); }
