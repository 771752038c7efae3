// launch.h -- internal launchers behind the C ABI (host side; arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8ds {

hipError_t launch_cast_amax(const uint16_t *x, int64_t n, const float *scale, int fmt, uint8_t *out,
                            float *sinv_out, float *amax_slot, const float *noop, hipStream_t st);
hipError_t launch_cast_transpose(const uint16_t *x, int64_t rows, int64_t cols, const float *scale, int fmt,
                                 uint8_t *out, uint8_t *out_t, float *sinv_out, float *amax_slot,
                                 const float *noop, hipStream_t st);
// x0 and x1 cast+transposed (out_t may be nullptr: codes only) by one launch when both take the
// same code path, else by two; one FP8 format for both.
hipError_t launch_cast_transpose_pair(const uint16_t *x0, int64_t rows0, int64_t cols0, const float *scale0,
                                      uint8_t *out0, uint8_t *out_t0, float *sinv0, float *amax0, const float *noop0,
                                      const uint16_t *x1, int64_t rows1, int64_t cols1, const float *scale1,
                                      uint8_t *out1, uint8_t *out_t1, float *sinv1, float *amax1, const float *noop1,
                                      int fmt, hipStream_t st);
size_t dbias_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_dbias_cast_transpose(const uint16_t *dy, int64_t rows, int64_t cols, const float *scale,
                                       int fmt, uint8_t *out, uint8_t *out_t, float *sinv_out,
                                       float *amax_slot, float *dbias, void *ws, hipStream_t st);

hipError_t launch_fp8_transpose(const uint8_t *in, int64_t rows, int64_t cols, uint8_t *out_t, const float *noop,
                                hipStream_t st);

constexpr int kMaxScaleTensors = 4096;
hipError_t launch_scale_update(float *hist, int64_t L, int64_t T, float *scale, float *scale_inv,
                               const int32_t *fmts_host, int32_t margin, hipStream_t st);

// out_dtype: 0 bfloat16, 1 float32, 2 E4M3, 3 E5M2 (the last two use d_scale, d_sinv_out, d_amax).
hipError_t launch_gemm_bias(const uint8_t *A, int fa, const float *a_sinv, int64_t lda, const uint8_t *B, int fb,
                            const float *b_sinv, int64_t ldb, const uint16_t *bias, void *D, int64_t ldd,
                            int out_dtype, int64_t M, int64_t N, int64_t K, const float *d_scale,
                            float *d_sinv_out, float *d_amax, hipStream_t st);

// The forward of a small layer (casts of x and W, GEMM + bias, bfloat16 y) in one launch, with
// the results of the cast-pair launch + GEMM launch; linear_fwd_small_ok says when it applies.
bool linear_fwd_small_ok(int64_t M, int64_t N, int64_t K, const uint8_t *x8_t);
hipError_t launch_linear_fwd_small(const uint16_t *x, const uint16_t *w, const uint16_t *bias, int64_t M, int64_t N,
                                   int64_t K, const float *x_scale, float *x_amax, uint8_t *x8, float *x_scale_inv,
                                   const float *w_scale, float *w_amax, uint8_t *w8, uint8_t *w8_t,
                                   float *w_scale_inv, const float *w_noop, uint16_t *y, hipStream_t st);

// The norms around a block (norm.hip).  Pointers that are nullptr leave their part out.
struct NormFwd {
    const uint16_t *block_out, *w_post, *b_post, *gate, *resid, *w_pre, *b_pre;
    uint16_t *x, *h;
    uint8_t *h8;
    float *post_stats, *pre_stats;
    const float *scale;
    float *sinv, *amax;
    float alpha, eps;
    int64_t rows, rows_per_gate;
    int width;
};
struct NormBwd {
    const uint16_t *dh, *dx, *block_out, *w_post, *b_post, *gate, *x, *w_pre;
    const float *post_stats, *pre_stats;
    uint16_t *d_block, *d_resid;
    float *dw_post, *db_post, *dgate, *dw_pre, *db_pre;
    float alpha;
    int64_t rows;
    int width;
    // set by the launcher: how the rows are shared out, and the workspace
    int64_t rows_per_gate, unit_rows, units_per_gate, units;
    bool gated;              // more gates than blocks: the partials hold the gate already, dgate is finished
    float *part[4];
};
constexpr int64_t kNormMaxWidth = 16384;
constexpr int64_t kNormMaxGates = 65531;   // with the weights' and biases' sums, one grid row each
size_t norm_workspace_bytes(int64_t rows, int64_t width, int64_t n_gates);
hipError_t launch_norm_fwd(const NormFwd &a, int layer, int fmt, hipStream_t st);
hipError_t launch_norm_bwd(NormBwd a, int layer, int64_t n_gates, void *ws, hipStream_t st);

// Tokens sorted by expert and back (moe.hip).
constexpr int64_t kMoeMaxExperts = 1024;
size_t moe_workspace_bytes(int64_t n, int64_t E);
hipError_t launch_moe_plan(const int32_t *experts, int64_t n, int64_t E, int64_t align, int64_t cap, int32_t *offsets,
                           int32_t *src, int32_t *slot, void *ws, hipStream_t st);
// in_codes: x holds FP8 codes that are moved; otherwise bfloat16, cast with fmt (or, out_bf16,
// rounded back to bfloat16)
struct MoeSort {
    const void *x;
    const int32_t *src;
    const float *weights, *scale;
    void *out;
    uint8_t *out_t;
    float *sinv, *amax;
    int64_t cap;
    int width, top, choices;
};
enum { kSortCodes = 0, kSortE4M3 = 1, kSortE5M2 = 2, kSortBf16 = 3 };
hipError_t launch_moe_sort(const MoeSort &a, int what, hipStream_t st);
hipError_t launch_moe_combine(const uint16_t *ys, const int32_t *slot, const float *weights, uint16_t *y, int64_t T,
                              int64_t k, int64_t width, int64_t cap, hipStream_t st);
hipError_t launch_moe_weight_grad(const uint16_t *dy, const uint16_t *ys, const int32_t *slot, float *dweights,
                                  int64_t T, int64_t k, int64_t width, int64_t cap, hipStream_t st);

// The experts' products over sorted rows (grouped.hip).
struct Grouped {
    const uint8_t *A, *B;
    const float *a_sinv, *b_sinv;
    const int32_t *offsets;
    void *D;
    int64_t lda, ldb, stride_b, ldd, stride_d;
    int cap, E, N, K;
};
constexpr int64_t kGroupedMaxLd = INT64_C(1) << 23;
// whether a launch can number the call's tiles
bool grouped_gemm_fits(int64_t cap, int64_t E, int64_t N);
bool grouped_wgrad_fits(int64_t E, int64_t N, int64_t K);
hipError_t launch_grouped_gemm(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st);
hipError_t launch_grouped_wgrad(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st);

// Attention between the QKV layer and the projection (attention.hip).  A tensor of heads: elements of a
// head follow each other, tokens and heads lie ts and hs elements apart.
struct Heads {
    uint16_t *p;
    int64_t ts, hs;
};
struct Attention {
    Heads q, k, v, out, dout, dq, dk, dv;
    const int32_t *offsets_q, *offsets_k;    // both nullptr: B sequences of equal lengths
    float *lse;
    uint8_t *out8;
    const float *scale;
    float *sinv, *amax;
    float softmax_scale;
    int fmt, causal, window;                 // window 0: none
    int B, Tq, Tk, Hq, Hkv, G, D;
    // set by the launcher: splits of the keys, their sums or the backward's row values; the waves' largest
    // outputs with their rows, and what is needed to compute the largest of all again (nullptr: not wanted)
    int splits, tops;
    float *part, *top_part;
    uint32_t *top;
    int32_t *top_row;
    int32_t *top_done;
};
constexpr int64_t kAttnMaxHead = 128;
constexpr int64_t kAttnMaxStride = INT64_C(1) << 23;     // between tokens: 64 rows' offsets stay below 2^31
constexpr int64_t kAttnMaxRows = INT64_C(1) << 28;       // tokens x heads
bool attention_fits(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, bool ragged);
// of a batch with offsets (ragged) or of equal sequences, with the amax of its output or without
size_t attention_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, bool ragged, bool amax);
size_t attention_bwd_workspace_bytes(int64_t Tq, int64_t Hq);
hipError_t launch_attention_fwd(Attention a, void *ws, hipStream_t st);
hipError_t launch_attention_bwd(Attention a, void *ws, hipStream_t st);

// The choice of experts from the router's logits (router.hip).
struct Route {
    const void *logits;
    int64_t ld, T;
    int E, top, bf16, normalise;
    int32_t *experts;
    float *weights, *lse;
    int32_t *counts;
    float *prob_sum, *loss;
    // backward
    const float *dweights, *dloss;
    void *dlogits;
    int64_t ld_d;
    // set by the launcher: the blocks' sums and counts, and their live rows
    unsigned int __attribute__((ext_vector_type(2))) *part, *part_loss;
    int32_t *part_live;
};
size_t moe_route_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_moe_route(Route a, void *ws, hipStream_t st);
hipError_t launch_moe_route_bwd(const Route &a, hipStream_t st);

}  // namespace fp8ds
