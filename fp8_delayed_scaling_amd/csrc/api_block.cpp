// api_block.cpp -- the extern "C" boundary of the operators around the linear layer: the block
// norms, the sort of tokens by expert, the experts' products (declared in include/fp8ds.h).
//
// As in api.cpp: arguments are checked on the host before anything is launched, nothing here
// allocates device memory, copies between host and device or synchronises.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/fp8ds.h"
#include "launch.h"

namespace {

inline bool is_aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// every pointer (nullptr included) on a multiple of n
template <class... P> bool all_aligned(uintptr_t n, P... p) { return (is_aligned(p, n) && ...); }
inline bool valid_fmt(int f) { return f == FP8DS_E4M3 || f == FP8DS_E5M2; }
inline bool valid_out(int d) { return d == FP8DS_OUT_BF16 || d == FP8DS_OUT_FP32; }
inline bool valid_norm(int k) { return k == FP8DS_NORM_RMS || k == FP8DS_NORM_LAYER; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? FP8DS_OK : FP8DS_ERR_HIP; }
inline bool size_ok(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return false;
    return rows == 0 || cols == 0 || rows <= (INT64_C(1) << 40) / cols;
}

// Shapes that the two norm calls share.
int check_norm_shape(int64_t rows, int64_t width, const uint16_t *gate, int64_t n_gates) {
    if (!size_ok(rows, width) || rows > INT_MAX || width > fp8ds::kNormMaxWidth) return FP8DS_ERR_SHAPE;
    if (n_gates < 0 || (width > 0 && (gate == nullptr) != (n_gates == 0))) return FP8DS_ERR_SHAPE;
    if (n_gates > 0 && (rows % n_gates != 0 || (rows == 0 && n_gates > fp8ds::kNormMaxGates))) return FP8DS_ERR_SHAPE;
    return FP8DS_OK;
}

// T tokens with `top` choices each, in 32-bit numbers.
inline bool choices_ok(int64_t T, int64_t top) { return T >= 0 && top >= 1 && top <= INT_MAX && T <= INT_MAX / top; }

int check_sort(const void *x, int64_t T, const int32_t *src, int64_t cap, int64_t top, const void *out, int64_t width) {
    if (!choices_ok(T, top) || cap < 0 || cap > INT_MAX || cap % 16 != 0) return FP8DS_ERR_SHAPE;
    if (width < 0 || width > INT_MAX / 2 || width % 16 != 0 || !size_ok(cap, width) || !size_ok(T, width))
        return FP8DS_ERR_SHAPE;
    if (cap == 0 || width == 0) return FP8DS_OK;
    if (((cap + 63) / 64) * ((width + 63) / 64) > INT_MAX) return FP8DS_ERR_SHAPE;
    if ((x == nullptr && T > 0) || src == nullptr || out == nullptr) return FP8DS_ERR_NULL;
    if (!all_aligned(16, x, static_cast<const void *>(src), out)) return FP8DS_ERR_ALIGN;
    return FP8DS_OK;
}

int check_back(const uint16_t *ys, int64_t cap, const int32_t *slot, int64_t T, int64_t top, int64_t width) {
    if (!choices_ok(T, top) || cap < 0 || cap > INT_MAX) return FP8DS_ERR_SHAPE;
    if (width < 0 || width > INT_MAX / 2 || width % 16 != 0 || !size_ok(cap, width) || !size_ok(T, width))
        return FP8DS_ERR_SHAPE;
    if (T == 0 || width == 0) return FP8DS_OK;
    if ((ys == nullptr && cap > 0) || slot == nullptr) return FP8DS_ERR_NULL;
    if (!is_aligned(ys, 16) || !is_aligned(slot, 4)) return FP8DS_ERR_ALIGN;
    return FP8DS_OK;
}

int check_grouped(const uint8_t *A, int fa, const float *a_sinv, int64_t lda, int64_t rows_a, const uint8_t *B, int fb,
                  const float *b_sinv, int64_t ldb, int64_t rows_b, const int32_t *offsets, int64_t E, const void *D,
                  int out_dtype, int64_t cap, int64_t N, int64_t K, int64_t inner) {
    if (!valid_fmt(fa) || !valid_fmt(fb) || !valid_out(out_dtype)) return FP8DS_ERR_FORMAT;
    if (E < 0 || cap < 0 || N < 0 || K < 0 || E > INT_MAX || cap > INT_MAX || N > INT_MAX || K > INT_MAX)
        return FP8DS_ERR_SHAPE;
    if (inner % 16 != 0) return FP8DS_ERR_SHAPE;
    if (inner > 0) {                                   // an empty contraction reads neither operand
        if (lda < inner || ldb < inner || lda >= fp8ds::kGroupedMaxLd || ldb >= fp8ds::kGroupedMaxLd)
            return FP8DS_ERR_SHAPE;
        if (!size_ok(rows_a, lda) || !size_ok(rows_b, ldb)) return FP8DS_ERR_SHAPE;
        if (lda % 16 != 0 || ldb % 16 != 0) return FP8DS_ERR_ALIGN;
    }
    if (!all_aligned(16, A, B) || !all_aligned(4, a_sinv, b_sinv) || !is_aligned(offsets, 4) ||
        !is_aligned(D, out_dtype == FP8DS_OUT_BF16 ? 2 : 4))
        return FP8DS_ERR_ALIGN;
    return FP8DS_OK;
}

}  // namespace

extern "C" {

int fp8_norm_residual_fwd(const uint16_t *block_out, const uint16_t *w_post, const uint16_t *b_post,
                          const uint16_t *gate, int64_t n_gates, const uint16_t *resid, float alpha, uint16_t *x,
                          float *post_stats, const uint16_t *w_pre, const uint16_t *b_pre, float *pre_stats,
                          uint16_t *h, uint8_t *h8, const float *scale, int fmt, float *scale_inv_out,
                          float *amax_slot, int kind, float eps, int64_t rows, int64_t width, hipStream_t stream) {
    if (!valid_norm(kind) || !valid_fmt(fmt)) return FP8DS_ERR_FORMAT;
    if (int st = check_norm_shape(rows, width, gate, n_gates); st != FP8DS_OK) return st;
    if (!(eps >= 0.f) || eps > 3.4e38f) return FP8DS_ERR_ARG;
    if (rows == 0 || width == 0) return FP8DS_OK;      // an empty buffer's pointer may be NULL
    if (kind == FP8DS_NORM_RMS && (b_post != nullptr || b_pre != nullptr)) return FP8DS_ERR_ARG;
    if (block_out == nullptr && (w_post != nullptr || gate != nullptr || x != nullptr || w_pre == nullptr))
        return FP8DS_ERR_ARG;
    if (w_post == nullptr && b_post != nullptr) return FP8DS_ERR_ARG;
    if (w_pre == nullptr && (b_pre != nullptr || h != nullptr || h8 != nullptr)) return FP8DS_ERR_ARG;
    if (block_out == nullptr ? resid == nullptr : x == nullptr) return FP8DS_ERR_NULL;
    if (w_pre != nullptr && h == nullptr && h8 == nullptr) return FP8DS_ERR_NULL;
    if (h8 != nullptr && scale == nullptr) return FP8DS_ERR_NULL;
    if (!all_aligned(16, block_out, w_post, b_post, gate, resid, x, w_pre, b_pre, h) || !is_aligned(h8, 16) ||
        !all_aligned(4, post_stats, pre_stats, scale_inv_out, amax_slot) || !is_aligned(scale, 4))
        return FP8DS_ERR_ALIGN;
    fp8ds::NormFwd a{};
    a.block_out = block_out; a.w_post = w_post; a.b_post = b_post; a.gate = gate; a.resid = resid;
    a.w_pre = w_pre; a.b_pre = b_pre; a.x = x; a.h = h; a.h8 = h8;
    a.post_stats = post_stats; a.pre_stats = pre_stats;
    a.scale = scale; a.sinv = scale_inv_out; a.amax = amax_slot;
    a.alpha = alpha; a.eps = eps;
    a.rows = rows; a.width = (int)width;
    a.rows_per_gate = n_gates > 0 ? rows / n_gates : rows;
    return hip_status(fp8ds::launch_norm_fwd(a, kind == FP8DS_NORM_LAYER, fmt, stream));
}

size_t fp8_norm_residual_workspace_bytes(int64_t rows, int64_t width, int64_t n_gates) {
    if (!size_ok(rows, width) || width > fp8ds::kNormMaxWidth || n_gates < 0) return 0;
    return fp8ds::norm_workspace_bytes(rows, width, n_gates);
}

int fp8_norm_residual_bwd(const uint16_t *dh, const uint16_t *dx, const uint16_t *block_out, const uint16_t *w_post,
                          const uint16_t *b_post, const uint16_t *gate, int64_t n_gates, float alpha,
                          const uint16_t *x, const float *post_stats, const uint16_t *w_pre, const float *pre_stats,
                          uint16_t *d_block, uint16_t *d_resid, float *dw_post, float *db_post, float *dgate,
                          float *dw_pre, float *db_pre, void *workspace, size_t workspace_bytes, int kind,
                          int64_t rows, int64_t width, hipStream_t stream) {
    if (!valid_norm(kind)) return FP8DS_ERR_FORMAT;
    if (int st = check_norm_shape(rows, width, gate, n_gates); st != FP8DS_OK) return st;
    if (kind == FP8DS_NORM_RMS && (b_post != nullptr || db_post != nullptr || db_pre != nullptr)) return FP8DS_ERR_ARG;
    if (width == 0) return FP8DS_OK;
    if (gate == nullptr && dgate != nullptr) return FP8DS_ERR_ARG;
    if (w_post == nullptr && (b_post != nullptr || dw_post != nullptr || db_post != nullptr)) return FP8DS_ERR_ARG;
    if (rows > 0) {                                    // without rows an empty buffer's pointer may be NULL
        if (dh == nullptr && (dw_pre != nullptr || db_pre != nullptr)) return FP8DS_ERR_ARG;
        if (block_out == nullptr && (w_post != nullptr || gate != nullptr || d_block != nullptr)) return FP8DS_ERR_ARG;
        if (dh == nullptr && dx == nullptr) return FP8DS_ERR_NULL;
        if (dh != nullptr && (x == nullptr || w_pre == nullptr || pre_stats == nullptr)) return FP8DS_ERR_NULL;
        if (w_post != nullptr && post_stats == nullptr) return FP8DS_ERR_NULL;
        if (block_out == nullptr ? d_resid == nullptr : d_block == nullptr) return FP8DS_ERR_NULL;
        const size_t need = fp8ds::norm_workspace_bytes(rows, width, n_gates);
        if (workspace == nullptr || workspace_bytes < need) return FP8DS_ERR_WORKSPACE;
    }
    if (!all_aligned(16, dh, dx, block_out, w_post, b_post, gate, x, w_pre) || !all_aligned(16, d_block, d_resid) ||
        !is_aligned(workspace, 16) || !all_aligned(4, post_stats, pre_stats) ||
        !all_aligned(16, dw_post, db_post, dgate, dw_pre, db_pre))
        return FP8DS_ERR_ALIGN;
    fp8ds::NormBwd a{};
    a.dh = dh; a.dx = dx; a.block_out = block_out; a.w_post = w_post; a.b_post = b_post; a.gate = gate;
    a.x = x; a.w_pre = w_pre; a.post_stats = post_stats; a.pre_stats = pre_stats;
    a.d_block = d_block; a.d_resid = d_resid;
    a.dw_post = dw_post; a.db_post = db_post; a.dgate = dgate; a.dw_pre = dw_pre; a.db_pre = db_pre;
    a.alpha = block_out != nullptr ? alpha : 1.f;
    a.rows = rows; a.width = (int)width;
    return hip_status(fp8ds::launch_norm_bwd(a, kind == FP8DS_NORM_LAYER, n_gates, workspace, stream));
}

int64_t fp8_moe_capacity(int64_t T, int64_t top, int64_t E, int64_t align) {
    if (!choices_ok(T, top) || E < 1 || E > fp8ds::kMoeMaxExperts || align < 16 || align > 1024 || align % 16 != 0) return -1;
    const int64_t n = T * top;
    return (n + (n < E ? n : E) * (align - 1)) / align * align;
}

size_t fp8_moe_workspace_bytes(int64_t T, int64_t top, int64_t E) {
    if (!choices_ok(T, top) || E < 1 || E > fp8ds::kMoeMaxExperts) return 0;
    return fp8ds::moe_workspace_bytes(T * top, E);
}

int fp8_moe_plan(const int32_t *experts, int64_t T, int64_t top, int64_t E, int64_t align, int64_t cap,
                 int32_t *offsets, int32_t *src, int32_t *slot, void *workspace, size_t workspace_bytes,
                 hipStream_t stream) {
    const int64_t need_rows = fp8_moe_capacity(T, top, E, align);
    if (need_rows < 0 || need_rows > INT_MAX || cap > INT_MAX || cap < need_rows || cap % 16 != 0) return FP8DS_ERR_SHAPE;
    if (offsets == nullptr || (T > 0 && (experts == nullptr || slot == nullptr)) || (cap > 0 && src == nullptr))
        return FP8DS_ERR_NULL;
    if (!is_aligned(experts, 4) || !all_aligned(4, offsets, src, slot) || !is_aligned(workspace, 4)) return FP8DS_ERR_ALIGN;
    const size_t need = fp8ds::moe_workspace_bytes(T * top, E);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8DS_ERR_WORKSPACE;
    return hip_status(fp8ds::launch_moe_plan(experts, T * top, E, align, cap, offsets, src, slot, workspace, stream));
}

int fp8_moe_sort_cast(const uint16_t *x, int64_t T, const int32_t *src, int64_t cap, int64_t top,
                      const float *weights, const float *scale, int fmt, uint8_t *out, uint8_t *out_t,
                      float *scale_inv_out, float *amax_slot, int64_t width, hipStream_t stream) {
    if (!valid_fmt(fmt)) return FP8DS_ERR_FORMAT;
    if (int st = check_sort(x, T, src, cap, top, out, width); st != FP8DS_OK) return st;
    if (cap == 0 || width == 0) return FP8DS_OK;
    if (scale == nullptr) return FP8DS_ERR_NULL;
    if (!is_aligned(out_t, 16) || !all_aligned(4, weights, scale) || !all_aligned(4, scale_inv_out, amax_slot))
        return FP8DS_ERR_ALIGN;
    const fp8ds::MoeSort a{x, src, weights, scale, out, out_t, scale_inv_out, amax_slot, cap, (int)width, (int)top,
                           (int)(T * top)};
    return hip_status(fp8ds::launch_moe_sort(a, fmt == FP8DS_E4M3 ? fp8ds::kSortE4M3 : fp8ds::kSortE5M2, stream));
}

int fp8_moe_sort_codes(const uint8_t *x8, int64_t T, const int32_t *src, int64_t cap, int64_t top, uint8_t *out,
                       uint8_t *out_t, int64_t width, hipStream_t stream) {
    if (int st = check_sort(x8, T, src, cap, top, out, width); st != FP8DS_OK) return st;
    if (cap == 0 || width == 0) return FP8DS_OK;
    if (!is_aligned(out_t, 16)) return FP8DS_ERR_ALIGN;
    const fp8ds::MoeSort a{x8, src, nullptr, nullptr, out, out_t, nullptr, nullptr, cap, (int)width, (int)top,
                           (int)(T * top)};
    return hip_status(fp8ds::launch_moe_sort(a, fp8ds::kSortCodes, stream));
}

int fp8_moe_sort_bf16(const uint16_t *x, int64_t T, const int32_t *src, int64_t cap, int64_t top,
                      const float *weights, uint16_t *out, int64_t width, hipStream_t stream) {
    if (int st = check_sort(x, T, src, cap, top, out, width); st != FP8DS_OK) return st;
    if (cap == 0 || width == 0) return FP8DS_OK;
    if (!is_aligned(weights, 4)) return FP8DS_ERR_ALIGN;
    const fp8ds::MoeSort a{x, src, weights, nullptr, out, nullptr, nullptr, nullptr, cap, (int)width, (int)top,
                           (int)(T * top)};
    return hip_status(fp8ds::launch_moe_sort(a, fp8ds::kSortBf16, stream));
}

int fp8_moe_combine(const uint16_t *ys, int64_t cap, const int32_t *slot, const float *weights, int64_t T,
                    int64_t top, uint16_t *y, int64_t width, hipStream_t stream) {
    if (int st = check_back(ys, cap, slot, T, top, width); st != FP8DS_OK) return st;
    if (T == 0 || width == 0) return FP8DS_OK;
    if (y == nullptr) return FP8DS_ERR_NULL;
    if (!is_aligned(y, 16) || !is_aligned(weights, 4)) return FP8DS_ERR_ALIGN;
    return hip_status(fp8ds::launch_moe_combine(ys, slot, weights, y, T, top, width, cap, stream));
}

int fp8_moe_weight_grad(const uint16_t *dy, const uint16_t *ys, int64_t cap, const int32_t *slot, int64_t T,
                        int64_t top, float *dweights, int64_t width, hipStream_t stream) {
    if (int st = check_back(ys, cap, slot, T, top, width); st != FP8DS_OK) return st;
    if (T == 0) return FP8DS_OK;
    if (dweights == nullptr || slot == nullptr || (dy == nullptr && width > 0)) return FP8DS_ERR_NULL;
    if (!is_aligned(dy, 16) || !is_aligned(dweights, 4) || !is_aligned(slot, 4)) return FP8DS_ERR_ALIGN;
    return hip_status(fp8ds::launch_moe_weight_grad(dy, ys, slot, dweights, T, top, width, cap, stream));
}

int fp8_grouped_gemm(const uint8_t *A, int fa, const float *a_scale_inv, int64_t lda, const uint8_t *B, int fb,
                     const float *b_scale_inv, int64_t ldb, int64_t stride_b, const int32_t *offsets, int64_t E,
                     void *D, int64_t ldd, int out_dtype, int64_t cap, int64_t N, int64_t K, hipStream_t stream) {
    if (int st = check_grouped(A, fa, a_scale_inv, lda, cap, B, fb, b_scale_inv, ldb, N, offsets, E, D, out_dtype, cap, N,
                               K, K);
        st != FP8DS_OK)
        return st;
    if (ldd < N || ldd >= fp8ds::kGroupedMaxLd || !size_ok(cap, ldd) || (K > 0 && !size_ok(E, stride_b))) return FP8DS_ERR_SHAPE;
    if (K > 0 && stride_b % 16 != 0) return FP8DS_ERR_ALIGN;
    if (!fp8ds::grouped_gemm_fits(cap, E, N)) return FP8DS_ERR_SHAPE;
    if (cap == 0 || N == 0 || E == 0) return FP8DS_OK;
    if (offsets == nullptr || D == nullptr || a_scale_inv == nullptr || b_scale_inv == nullptr) return FP8DS_ERR_NULL;
    if (K > 0 && (A == nullptr || B == nullptr)) return FP8DS_ERR_NULL;
    // without a contraction the strides are unchecked and stand for nothing: none reaches an offset
    if (K == 0) lda = ldb = stride_b = 0;
    const fp8ds::Grouped g{A, B, a_scale_inv, b_scale_inv, offsets, D, lda, ldb, stride_b, ldd, 0, (int)cap, (int)E,
                           (int)N, (int)K};
    return hip_status(fp8ds::launch_grouped_gemm(g, fa, fb, out_dtype, stream));
}

int fp8_grouped_wgrad(const uint8_t *At, int fa, const float *a_scale_inv, int64_t lda, const uint8_t *Bt, int fb,
                      const float *b_scale_inv, int64_t ldb, const int32_t *offsets, int64_t E, void *dW,
                      int out_dtype, int64_t cap, int64_t N, int64_t K, hipStream_t stream) {
    if (int st = check_grouped(At, fa, a_scale_inv, lda, N, Bt, fb, b_scale_inv, ldb, K, offsets, E, dW, out_dtype, cap, N,
                               K, cap);
        st != FP8DS_OK)
        return st;
    if (!size_ok(N, K) || K >= fp8ds::kGroupedMaxLd || !size_ok(E, N * K) || !fp8ds::grouped_wgrad_fits(E, N, K)) return FP8DS_ERR_SHAPE;
    if (N == 0 || K == 0 || E == 0) return FP8DS_OK;
    if (offsets == nullptr || dW == nullptr || a_scale_inv == nullptr || b_scale_inv == nullptr) return FP8DS_ERR_NULL;
    if (cap > 0 && (At == nullptr || Bt == nullptr)) return FP8DS_ERR_NULL;
    if (cap == 0) lda = ldb = 0;                       // as above
    const fp8ds::Grouped g{At, Bt, a_scale_inv, b_scale_inv, offsets, dW, lda, ldb, 0, K, N * K, (int)cap, (int)E,
                           (int)N, (int)K};
    return hip_status(fp8ds::launch_grouped_wgrad(g, fa, fb, out_dtype, stream));
}

}  // extern "C"
