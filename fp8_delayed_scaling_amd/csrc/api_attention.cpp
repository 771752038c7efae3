// api_attention.cpp -- the extern "C" boundary of attention and of the router in front of the sort by
// expert (declared in include/fp8ds.h).
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
inline int hip_status(hipError_t e) { return e == hipSuccess ? FP8DS_OK : FP8DS_ERR_HIP; }
inline bool size_ok(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return false;
    return rows == 0 || cols == 0 || rows <= (INT64_C(1) << 40) / cols;
}
// T tokens with `top` choices each, in 32-bit numbers.
inline bool choices_ok(int64_t T, int64_t top) { return T >= 0 && top >= 1 && top <= INT_MAX && T <= INT_MAX / top; }

// lse / softmax_scale and softmax_scale * log2(e) stay finite
constexpr float kScaleMin = 1e-30f, kScaleMax = 1e30f;

// Tokens of heads at strides of their own.  `group`: heads of neighbouring tokens that a kernel reaches from one base, by byte
// offsets below 2^31 (up to 34 tokens on).
int check_heads(const fp8ds_heads &h, int64_t T, int64_t H, int64_t D, bool output, int64_t group) {
    if (T == 0) return FP8DS_OK;
    if (h.token_stride < 0 || h.head_stride < 0) return FP8DS_ERR_SHAPE;
    if (T > 1 && (h.token_stride < D || h.token_stride >= fp8ds::kAttnMaxStride)) return FP8DS_ERR_SHAPE;
    if (output && H > 1 && h.head_stride < D) return FP8DS_ERR_SHAPE;
    if (!size_ok(T, h.token_stride) || !size_ok(H, h.head_stride)) return FP8DS_ERR_SHAPE;
    if (group > 1 && h.head_stride > (INT64_C(1) << 30) / group - 34 * (T > 1 ? h.token_stride : 0) / group - D) return FP8DS_ERR_SHAPE;
    if (h.data == nullptr) return FP8DS_ERR_NULL;
    if (h.token_stride % 8 != 0 || h.head_stride % 8 != 0 || !is_aligned(h.data, 16)) return FP8DS_ERR_ALIGN;
    return FP8DS_OK;
}

int check_attention(const int32_t *offsets_q, const int32_t *offsets_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                    int64_t Hkv, int64_t D, float softmax_scale, int64_t window, int causal) {
    if (B < 0 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || B > INT_MAX) return FP8DS_ERR_SHAPE;
    if (D < 8 || D > fp8ds::kAttnMaxHead || D % 8 != 0) return FP8DS_ERR_SHAPE;
    if (Tq > fp8ds::kAttnMaxRows / Hq || Tk > fp8ds::kAttnMaxRows / Hkv) return FP8DS_ERR_SHAPE;
    if ((offsets_q == nullptr) != (offsets_k == nullptr)) return FP8DS_ERR_NULL;
    if (offsets_q == nullptr && B > 0 && (Tq % B != 0 || Tk % B != 0)) return FP8DS_ERR_SHAPE;
    if (!(softmax_scale >= kScaleMin && softmax_scale <= kScaleMax) || window < 0 || (window > 0 && causal == 0)) return FP8DS_ERR_ARG;
    if (!all_aligned(4, offsets_q, offsets_k)) return FP8DS_ERR_ALIGN;
    return fp8ds::attention_fits(Tq, Tk, B, Hq, Hkv, offsets_q != nullptr) ? FP8DS_OK : FP8DS_ERR_SHAPE;
}

// of a single token the stride says nothing; the kernels take a row's extent from it
fp8ds::Heads heads_of(const fp8ds_heads &h, int64_t T, int64_t D) { return fp8ds::Heads{h.data, T > 1 ? h.token_stride : D, h.head_stride}; }

int check_route(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t top) {
    if (!valid_out(dtype)) return FP8DS_ERR_FORMAT;
    if (E < 1 || E > fp8ds::kMoeMaxExperts || top < 1 || top > E || !choices_ok(T, top) || ld < E || !size_ok(T, ld)) return FP8DS_ERR_SHAPE;
    if (logits == nullptr && T > 0) return FP8DS_ERR_NULL;
    return is_aligned(logits, dtype == FP8DS_OUT_BF16 ? 2 : 4) ? FP8DS_OK : FP8DS_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t fp8_attention_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
    if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || D > fp8ds::kAttnMaxHead) return 0;
    if (Tq > fp8ds::kAttnMaxRows / Hq || Tk > fp8ds::kAttnMaxRows / Hkv) return 0;
    if (Tq == 0) return 0;
    // enough for offsets and for equal sequences, with an amax and without
    const size_t n = fp8ds::attention_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, true, true);
    const size_t m = Tq % B == 0 && Tk % B == 0 ? fp8ds::attention_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, false, true) : 0;
    return n > m ? n : m;
}

int fp8_attention_fwd(fp8ds_heads q, fp8ds_heads k, fp8ds_heads v, fp8ds_heads out, float *lse, uint8_t *out8,
                      const float *scale, int fmt, float *scale_inv_out, float *amax_slot, const int32_t *offsets_q,
                      const int32_t *offsets_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D,
                      float softmax_scale, int causal, int64_t window, void *workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    if (!valid_fmt(fmt)) return FP8DS_ERR_FORMAT;
    if (int st = check_attention(offsets_q, offsets_k, B, Tq, Tk, Hq, Hkv, D, softmax_scale, window, causal); st != FP8DS_OK) return st;
    if (B == 0 || Tq == 0) return FP8DS_OK;
    if (out.data == nullptr && out8 == nullptr) return FP8DS_ERR_NULL;
    if (out8 != nullptr && scale == nullptr) return FP8DS_ERR_NULL;
    if (int st = check_heads(q, Tq, Hq, D, false, Hq / Hkv); st != FP8DS_OK) return st;
    if (int st = check_heads(k, Tk, Hkv, D, false, 1); st != FP8DS_OK) return st;
    if (int st = check_heads(v, Tk, Hkv, D, false, 1); st != FP8DS_OK) return st;
    if (out.data != nullptr)
        if (int st = check_heads(out, Tq, Hq, D, true, 1); st != FP8DS_OK) return st;
    if (!is_aligned(out8, 16) || !all_aligned(4, lse, scale_inv_out, amax_slot) || !is_aligned(scale, 4) || !is_aligned(workspace, 16))
        return FP8DS_ERR_ALIGN;
    const size_t need = fp8ds::attention_workspace_bytes(Tq, Tk, B, Hq, Hkv, D, offsets_q != nullptr, out8 != nullptr && amax_slot != nullptr);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8DS_ERR_WORKSPACE;
    fp8ds::Attention a{};
    a.q = heads_of(q, Tq, D); a.k = heads_of(k, Tk, D); a.v = heads_of(v, Tk, D); a.out = heads_of(out, Tq, D);
    a.offsets_q = offsets_q; a.offsets_k = offsets_k;
    a.lse = lse; a.out8 = out8; a.scale = scale; a.sinv = scale_inv_out; a.amax = amax_slot;
    a.softmax_scale = softmax_scale; a.fmt = fmt; a.causal = causal != 0;
    a.window = window < Tk ? (int)window : 0;
    a.B = (int)B; a.Tq = (int)Tq; a.Tk = (int)Tk; a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.G = (int)(Hq / Hkv); a.D = (int)D;
    return hip_status(fp8ds::launch_attention_fwd(a, workspace, stream));
}

size_t fp8_attention_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
    if (B < 1 || Tq < 0 || Tk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || Tq > fp8ds::kAttnMaxRows / Hq) return 0;
    return fp8ds::attention_bwd_workspace_bytes(Tq, Hq);
}

int fp8_attention_bwd(fp8ds_heads dout, fp8ds_heads q, fp8ds_heads k, fp8ds_heads v, fp8ds_heads out, const float *lse,
                      fp8ds_heads dq, fp8ds_heads dk, fp8ds_heads dv, const int32_t *offsets_q, const int32_t *offsets_k,
                      int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hkv, int64_t D, float softmax_scale, int causal,
                      int64_t window, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (int st = check_attention(offsets_q, offsets_k, B, Tq, Tk, Hq, Hkv, D, softmax_scale, window, causal); st != FP8DS_OK) return st;
    if (B == 0 || (Tq == 0 && Tk == 0)) return FP8DS_OK;
    if (lse == nullptr && Tq > 0) return FP8DS_ERR_NULL;
    for (const fp8ds_heads *h : {&dout, &q})
        if (int st = check_heads(*h, Tq, Hq, D, false, Hq / Hkv); st != FP8DS_OK) return st;
    for (const fp8ds_heads *h : {&k, &v})
        if (int st = check_heads(*h, Tk, Hkv, D, false, 1); st != FP8DS_OK) return st;
    if (int st = check_heads(out, Tq, Hq, D, false, 1); st != FP8DS_OK) return st;
    if (int st = check_heads(dq, Tq, Hq, D, true, 1); st != FP8DS_OK) return st;
    for (const fp8ds_heads *h : {&dk, &dv})
        if (int st = check_heads(*h, Tk, Hkv, D, true, 1); st != FP8DS_OK) return st;
    if (!is_aligned(lse, 4) || !is_aligned(workspace, 16)) return FP8DS_ERR_ALIGN;
    const size_t need = fp8ds::attention_bwd_workspace_bytes(Tq, Hq);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8DS_ERR_WORKSPACE;
    fp8ds::Attention a{};
    a.q = heads_of(q, Tq, D); a.k = heads_of(k, Tk, D); a.v = heads_of(v, Tk, D); a.out = heads_of(out, Tq, D); a.dout = heads_of(dout, Tq, D);
    a.dq = heads_of(dq, Tq, D); a.dk = heads_of(dk, Tk, D); a.dv = heads_of(dv, Tk, D);
    a.offsets_q = offsets_q; a.offsets_k = offsets_k;
    a.lse = const_cast<float *>(lse);
    a.softmax_scale = softmax_scale; a.causal = causal != 0;
    a.window = window < Tk ? (int)window : 0;
    a.B = (int)B; a.Tq = (int)Tq; a.Tk = (int)Tk; a.Hq = (int)Hq; a.Hkv = (int)Hkv; a.G = (int)(Hq / Hkv); a.D = (int)D;
    return hip_status(fp8ds::launch_attention_bwd(a, workspace, stream));
}

size_t fp8_moe_route_workspace_bytes(int64_t T, int64_t E) {
    if (T < 0 || E < 1 || E > fp8ds::kMoeMaxExperts) return 0;
    return fp8ds::moe_route_workspace_bytes(T, E);
}

int fp8_moe_route(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t top, int normalise, int32_t *experts,
                  float *weights, float *lse, int32_t *counts, float *prob_sum, float *loss, void *workspace,
                  size_t workspace_bytes, hipStream_t stream) {
    if (int st = check_route(logits, dtype, ld, T, E, top); st != FP8DS_OK) return st;
    if ((T > 0 && (experts == nullptr || weights == nullptr || lse == nullptr)) || counts == nullptr || prob_sum == nullptr || loss == nullptr)
        return FP8DS_ERR_NULL;
    if (!all_aligned(4, experts, counts) || !all_aligned(4, weights, lse, prob_sum, loss) || !is_aligned(workspace, 8)) return FP8DS_ERR_ALIGN;
    const size_t need = fp8ds::moe_route_workspace_bytes(T, E);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FP8DS_ERR_WORKSPACE;
    fp8ds::Route a{};
    a.logits = logits; a.ld = ld; a.T = T; a.E = (int)E; a.top = (int)top; a.bf16 = dtype == FP8DS_OUT_BF16; a.normalise = normalise != 0;
    a.experts = experts; a.weights = weights; a.lse = lse; a.counts = counts; a.prob_sum = prob_sum; a.loss = loss;
    return hip_status(fp8ds::launch_moe_route(a, workspace, stream));
}

int fp8_moe_route_bwd(const void *logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t top, int normalise,
                      const int32_t *experts, const float *weights, const float *lse, const int32_t *counts,
                      const float *dweights, const float *dloss, void *dlogits, int64_t ld_d, hipStream_t stream) {
    if (int st = check_route(logits, dtype, ld, T, E, top); st != FP8DS_OK) return st;
    if (ld_d < E || !size_ok(T, ld_d)) return FP8DS_ERR_SHAPE;
    if (T == 0) return FP8DS_OK;
    if (lse == nullptr || dlogits == nullptr) return FP8DS_ERR_NULL;
    if (dweights != nullptr && (experts == nullptr || weights == nullptr)) return FP8DS_ERR_NULL;
    if (dloss != nullptr && counts == nullptr) return FP8DS_ERR_NULL;
    if (!all_aligned(4, experts, counts) || !all_aligned(4, weights, lse, dweights, dloss) || !is_aligned(dlogits, dtype == FP8DS_OUT_BF16 ? 2 : 4))
        return FP8DS_ERR_ALIGN;
    fp8ds::Route a{};
    a.logits = logits; a.ld = ld; a.T = T; a.E = (int)E; a.top = (int)top; a.bf16 = dtype == FP8DS_OUT_BF16; a.normalise = normalise != 0;
    a.experts = const_cast<int32_t *>(experts); a.weights = const_cast<float *>(weights); a.lse = const_cast<float *>(lse);
    a.counts = const_cast<int32_t *>(counts); a.dweights = dweights; a.dloss = dloss; a.dlogits = dlogits; a.ld_d = ld_d;
    return hip_status(fp8ds::launch_moe_route_bwd(a, stream));
}

}  // extern "C"
