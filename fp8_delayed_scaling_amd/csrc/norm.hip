// norm.hip -- the norms before and after a block, fused with the block's gate and the residual
// scale, forward and backward, on gfx950.
//
//   n = norm(o) * w_post + b_post       the block's output, normalised
//   x = bf16(alpha * resid + gate * n)  the residual stream
//   h = norm(x) * w_pre + b_pre         the next block's input: bfloat16 and / or FP8 codes
//
// norm is RMS (v * rstd) or layer ((v - mean) * rstd).  Both directions are HBM-streaming
// kernels: a row is read once into registers, the row statistics come from one reduction (RMS) or
// two (layer: the mean first, then the squared deviations, which keeps rows with a large mean
// exact), and everything that depends on them leaves in the same pass.  All arithmetic is float32;
// values round where they are stored (x, h, the codes, the gradients).  The second norm reads the
// rounded x, which is what the backward reads.
//
// A row belongs to a team of TPR threads, 8 V columns each, held as raw bfloat16 pairs.  VEC
// (width % 8 == 0): thread t holds the 16-byte chunks t, t + TPR, ...; otherwise (odd widths, rows
// only 2-byte aligned) columns t, t + TPR, ... one at a time, still coalesced.
#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

template <int TPR, int V, bool VEC>
struct Row {
    static constexpr int kElems = 8 * V;
    static __device__ __forceinline__ int col(int t, int i) {
        return VEC ? (t + (i >> 3) * TPR) * 8 + (i & 7) : t + i * TPR;
    }
    // raw[i / 2] holds elements i (low half) and i + 1; columns past the width read as zero
    static __device__ __forceinline__ void load(const uint16_t *__restrict__ p, int H, int t, uint32_t (&raw)[4 * V]) {
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                u32x4 q = {0u, 0u, 0u, 0u};
                if ((t + v * TPR) * 8 < H) q = *reinterpret_cast<const u32x4 *>(p + (t + v * TPR) * 8);
                raw[4 * v] = q.x; raw[4 * v + 1] = q.y; raw[4 * v + 2] = q.z; raw[4 * v + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) {
                const int c0 = t + 2 * j * TPR, c1 = c0 + TPR;
                const uint32_t lo = c0 < H ? p[c0] : 0u, hi = c1 < H ? p[c1] : 0u;
                raw[j] = lo | (hi << 16);
            }
        }
    }
    static __device__ __forceinline__ float get(const uint32_t (&raw)[4 * V], int i) {
        return (i & 1) ? bf16_hi(raw[i >> 1]) : bf16_lo(raw[i >> 1]);
    }
    static __device__ __forceinline__ void store(uint16_t *__restrict__ p, int H, int t, const uint32_t (&raw)[4 * V]) {
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((t + v * TPR) * 8 < H)
                    *reinterpret_cast<u32x4 *>(p + (t + v * TPR) * 8) =
                        u32x4{raw[4 * v], raw[4 * v + 1], raw[4 * v + 2], raw[4 * v + 3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) {
                const int c0 = t + 2 * j * TPR, c1 = c0 + TPR;
                if (c0 < H) p[c0] = (uint16_t)raw[j];
                if (c1 < H) p[c1] = (uint16_t)(raw[j] >> 16);
            }
        }
    }
    // float32 columns (partial sums)
    static __device__ __forceinline__ void store_f32(float *__restrict__ p, int H, int t, const float (&v)[8 * V]) {
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < 2 * V; ++q) {
                const int c = col(t, 4 * q);
                if (c < H) *reinterpret_cast<f32x4 *>(p + c) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8 * V; ++i)
                if (col(t, i) < H) p[col(t, i)] = v[i];
        }
    }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Sums over a row's team, every thread receiving them.  `red` holds two buffers of 2 floats per
// wave, used in turn: a buffer is written again only after the next call's barrier, which every
// thread reaches after its reads of this call.
template <int TPR>
struct TeamSum {
    float (*red)[2][TPR / 64];
    int turn = 0;
    __device__ __forceinline__ void operator()(float &a, float &b) {
        a = wave_sum(a);
        b = wave_sum(b);
        if constexpr (TPR > 64) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) { red[turn][0][wave] = a; red[turn][1][wave] = b; }
            __syncthreads();
            a = red[turn][0][0]; b = red[turn][1][0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) { a += red[turn][0][w]; b += red[turn][1][w]; }
            turn ^= 1;
        }
    }
    __device__ __forceinline__ void operator()(float &a) {
        a = wave_sum(a);
        if constexpr (TPR > 64) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) red[turn][0][wave] = a;
            __syncthreads();
            a = red[turn][0][0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) a += red[turn][0][w];
            turn ^= 1;
        }
    }
};

// Mean and 1 / standard deviation of the row in v (columns past the width hold zero).
template <int TPR, int V, bool VEC, bool LN>
__device__ __forceinline__ void row_stats(const float (&v)[8 * V], int H, int t, float eps, TeamSum<TPR> &sum,
                                          float &rstd, float &mean) {
    const float inv = 1.0f / (float)H;
    mean = 0.f;
    float ss = 0.f;
    if constexpr (LN) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) s += v[i];
        sum(s);
        mean = s * inv;
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) {
            const float d = Row<TPR, V, VEC>::col(t, i) < H ? v[i] - mean : 0.f;
            ss += d * d;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) ss += v[i] * v[i];
    }
    sum(ss);
    rstd = 1.0f / sqrtf(ss * inv + eps);
}

}  // namespace

// ------------------------------------------------------------------------------------------
// Forward: a team per row, rows taken in a grid-stride loop.
// ------------------------------------------------------------------------------------------
template <int TPR, int V, bool VEC, bool LN, int FMT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_fwd(const NormFwd a) {
    constexpr int NT = TPR < 256 ? 256 : TPR, TEAMS = NT / TPR;
    using R = Row<TPR, V, VEC>;
    __shared__ float red[2][2][TPR / 64];
    __shared__ uint32_t ared[NT / 64];
    TeamSum<TPR> sum{red};
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int H = a.width;
    const float s = a.h8 != nullptr ? *a.scale : 0.f;
    uint32_t amag = 0;
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + team; row < a.rows; row += (int64_t)gridDim.x * TEAMS) {
        const int64_t base = row * H;
        uint32_t xr[4 * V];
        float v[8 * V];
        float rstd, mean;
        if (a.block_out != nullptr) {
            uint32_t orw[4 * V], rr[4 * V], wr[4 * V], br[4 * V], gr[4 * V];
            R::load(a.block_out + base, H, t, orw);
            if (a.resid != nullptr) R::load(a.resid + base, H, t, rr);
#pragma unroll
            for (int i = 0; i < 8 * V; ++i) v[i] = R::get(orw, i);
            if (a.w_post != nullptr) {
                R::load(a.w_post, H, t, wr);
                if constexpr (LN) if (a.b_post != nullptr) R::load(a.b_post, H, t, br);
                row_stats<TPR, V, VEC, LN>(v, H, t, a.eps, sum, rstd, mean);
                if (t == 0 && a.post_stats != nullptr) {
                    a.post_stats[row] = rstd;
                    if constexpr (LN) a.post_stats[a.rows + row] = mean;
                }
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) {
                    v[i] = (v[i] - mean) * rstd * R::get(wr, i);
                    if constexpr (LN) if (a.b_post != nullptr) v[i] += R::get(br, i);
                }
            }
            if (a.gate != nullptr) {
                R::load(a.gate + row / a.rows_per_gate * H, H, t, gr);
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) v[i] *= R::get(gr, i);
            }
            if (a.resid != nullptr) {
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) v[i] = __builtin_fmaf(a.alpha, R::get(rr, i), v[i]);
            }
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) xr[j] = f32x2_to_bf16x2_rne(v[2 * j], v[2 * j + 1]);
            R::store(a.x + base, H, t, xr);
        } else {
            R::load(a.resid + base, H, t, xr);
        }
        if (a.w_pre == nullptr) continue;
        // columns past the width hold zero: their x is made of zero loads, except a gate or bias
        // (also loaded as zero there)
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) v[i] = R::get(xr, i);
        uint32_t wr[4 * V], br[4 * V];
        R::load(a.w_pre, H, t, wr);
        if constexpr (LN) if (a.b_pre != nullptr) R::load(a.b_pre, H, t, br);
        row_stats<TPR, V, VEC, LN>(v, H, t, a.eps, sum, rstd, mean);
        if (t == 0 && a.pre_stats != nullptr) {
            a.pre_stats[row] = rstd;
            if constexpr (LN) a.pre_stats[a.rows + row] = mean;
        }
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) {
            v[i] = (v[i] - mean) * rstd * R::get(wr, i);
            if constexpr (LN) if (a.b_pre != nullptr) v[i] += R::get(br, i);
        }
        if (a.h != nullptr) {
            uint32_t hr[4 * V];
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) hr[j] = f32x2_to_bf16x2_rne(v[2 * j], v[2 * j + 1]);
            R::store(a.h + base, H, t, hr);
        }
        if (a.h8 != nullptr) {
#pragma unroll
            for (int i = 0; i < 8 * V; ++i)
                if (R::col(t, i) < H) amag = max(amag, __float_as_uint(v[i]) & 0x7FFFFFFFu);
            if constexpr (VEC) {
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const u32x2 c = {encode4<FMT>(v[8 * q] * s, v[8 * q + 1] * s, v[8 * q + 2] * s, v[8 * q + 3] * s),
                                     encode4<FMT>(v[8 * q + 4] * s, v[8 * q + 5] * s, v[8 * q + 6] * s, v[8 * q + 7] * s)};
                    if (R::col(t, 8 * q) < H) *reinterpret_cast<u32x2 *>(a.h8 + base + R::col(t, 8 * q)) = c;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8 * V; ++i)
                    if (R::col(t, i) < H) a.h8[base + R::col(t, i)] = (uint8_t)encode_exact<FMT>(v[i] * s);
            }
        }
    }
    if (a.h8 != nullptr) {
        const uint32_t bm = block_max_u32<NT>(amag, ared);
        if (threadIdx.x == 0) {
            fold_amax_bits(a.amax, bm);
            if (blockIdx.x == 0 && a.sinv != nullptr) *a.sinv = 1.0f / s;
        }
    }
}

// ------------------------------------------------------------------------------------------
// Backward.  With hat = (x - mean) rstd and q = dh * w_pre:
//   d      = dx + rstd (q - [mean of q] - hat [mean of q hat])     gradient of x
//   d_resid = alpha d;  dn = gate d;  dgate = sum over a gate's rows of d n
//   d_block = the same form over o with dn * w_post
//   dw_pre = sum dh hat, db_pre = sum dh, dw_post = sum dn ohat, db_post = sum dn
// ([mean of q] for layer norms only).  Column sums: a block takes `units` (row ranges inside one
// gate's rows) one after the other, each thread summing its own columns in registers over its
// rows; one partial per block (weights, biases) or per unit (gate) goes to the workspace and
// k_norm_cols adds the partials in a fixed order, so the sums are the same run to run.
// ------------------------------------------------------------------------------------------
template <int TPR, int V, bool VEC, bool LN>
__global__ __launch_bounds__(TPR) void k_norm_bwd(const NormBwd a) {
    using R = Row<TPR, V, VEC>;
    __shared__ float red[2][2][TPR / 64];
    TeamSum<TPR> sum{red};
    const int t = threadIdx.x;
    const int H = a.width;
    const float inv = 1.0f / (float)H;
    float dwq[8 * V], dbq[8 * V], dwp[8 * V], dbp[8 * V];
#pragma unroll
    for (int i = 0; i < 8 * V; ++i) dwq[i] = dbq[i] = dwp[i] = dbp[i] = 0.f;
    const int64_t u0 = a.units * blockIdx.x / gridDim.x, u1 = a.units * (blockIdx.x + 1) / gridDim.x;
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t gi = u / a.units_per_gate, part = u - gi * a.units_per_gate;
        const int64_t r0 = gi * a.rows_per_gate + part * a.unit_rows;
        const int64_t left = a.rows_per_gate - part * a.unit_rows;
        const int64_t r1 = r0 + (left < a.unit_rows ? left : a.unit_rows);
        uint32_t gr[4 * V];
        if (a.gate != nullptr) R::load(a.gate + gi * H, H, t, gr);
        float dg[8 * V];
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) dg[i] = 0.f;
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t base = row * H;
            uint32_t raw[4 * V], wr[4 * V];
            float d[8 * V], hat[8 * V];
#pragma unroll
            for (int i = 0; i < 8 * V; ++i) d[i] = 0.f;
            if (a.dh != nullptr) {
                uint32_t dr[4 * V];
                R::load(a.dh + base, H, t, dr);
                R::load(a.x + base, H, t, raw);
                R::load(a.w_pre, H, t, wr);
                const float rstd = a.pre_stats[row], mean = LN ? a.pre_stats[a.rows + row] : 0.f;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) {
                    const float dy = R::get(dr, i);
                    hat[i] = (R::get(raw, i) - mean) * rstd;
                    d[i] = dy * R::get(wr, i);          // zero past the width
                    dwq[i] += dy * hat[i];
                    if constexpr (LN) { dbq[i] += dy; s0 += d[i]; }
                    s1 += d[i] * hat[i];
                }
                if constexpr (LN) sum(s1, s0); else sum(s1);
                s0 *= inv; s1 *= inv;
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) d[i] = rstd * (d[i] - s0 - hat[i] * s1);
            }
            if (a.dx != nullptr) {
                R::load(a.dx + base, H, t, raw);
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) d[i] += R::get(raw, i);
            }
            if (a.d_resid != nullptr) {
#pragma unroll
                for (int j = 0; j < 4 * V; ++j) raw[j] = f32x2_to_bf16x2_rne(a.alpha * d[2 * j], a.alpha * d[2 * j + 1]);
                R::store(a.d_resid + base, H, t, raw);
            }
            if (a.block_out == nullptr) continue;
            R::load(a.block_out + base, H, t, raw);
            if (a.w_post != nullptr) {
                uint32_t br[4 * V];
                R::load(a.w_post, H, t, wr);
                if constexpr (LN) if (a.b_post != nullptr) R::load(a.b_post, H, t, br);
                const float rstd = a.post_stats[row], mean = LN ? a.post_stats[a.rows + row] : 0.f;
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) {
                    hat[i] = (R::get(raw, i) - mean) * rstd;
                    const float w = R::get(wr, i);
                    if (a.gate != nullptr) {
                        float n = hat[i] * w;
                        if constexpr (LN) if (a.b_post != nullptr) n += R::get(br, i);
                        dg[i] += d[i] * n;
                        d[i] *= R::get(gr, i);
                    }
                    dwp[i] += d[i] * hat[i];
                    if constexpr (LN) dbp[i] += d[i];
                    d[i] *= w;                          // zero past the width
                    if constexpr (LN) s0 += d[i];
                    s1 += d[i] * hat[i];
                }
                if constexpr (LN) sum(s1, s0); else sum(s1);
                s0 *= inv; s1 *= inv;
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) d[i] = rstd * (d[i] - s0 - hat[i] * s1);
            } else if (a.gate != nullptr) {
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) {
                    dg[i] += d[i] * R::get(raw, i);
                    d[i] *= R::get(gr, i);
                }
            }
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) raw[j] = f32x2_to_bf16x2_rne(d[2 * j], d[2 * j + 1]);
            R::store(a.d_block + base, H, t, raw);
        }
        // the gate's partial of this unit; a gate of one unit is finished here
        if (a.dgate != nullptr)
            R::store_f32((a.units_per_gate == 1 ? a.dgate : a.gate_part) + u * H, H, t, dg);
    }
    const int64_t at = (int64_t)blockIdx.x * H;
    if (a.dw_pre != nullptr) R::store_f32(a.col_part[0] + at, H, t, dwq);
    if (a.dw_post != nullptr) R::store_f32(a.col_part[1] + at, H, t, dwp);
    if constexpr (LN) {
        if (a.db_pre != nullptr) R::store_f32(a.col_part[2] + at, H, t, dbq);
        if (a.db_post != nullptr) R::store_f32(a.col_part[3] + at, H, t, dbp);
    }
}

// Column sums of the partials: block (c, y) owns 64 columns of output y (0..3 the weights and
// biases over all blocks' partials, 4 + g gate g over its units).  Thread (r = t / 64, c = t % 64)
// takes partials r, r + 16, ...; the 16 sums are then added in a fixed tree.
__global__ __launch_bounds__(1024) void k_norm_cols(const NormBwd a, int nblk) {
    __shared__ float part[16][64];
    const int r = threadIdx.x >> 6, c = threadIdx.x & 63;
    const int H = a.width;
    const int64_t j = (int64_t)blockIdx.x * 64 + c;
    const int y = blockIdx.y;
    float *out;
    const float *p;
    int64_t n;
    if (y < 4) {
        out = y == 0 ? a.dw_pre : y == 1 ? a.dw_post : y == 2 ? a.db_pre : a.db_post;
        p = y == 0 ? a.col_part[0] : y == 1 ? a.col_part[1] : y == 2 ? a.col_part[2] : a.col_part[3];
        n = nblk;
    } else {
        out = a.dgate + (int64_t)(y - 4) * H;
        p = a.gate_part + (int64_t)(y - 4) * a.units_per_gate * H;
        n = a.units_per_gate;
    }
    if (out == nullptr) return;   // block-uniform
    float acc = 0.f;
    if (j < H)
        for (int64_t i = r; i < n; i += 16) acc += p[i * H + j];
    part[r][c] = acc;
    __syncthreads();
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        if (r < w) part[r][c] += part[r + w][c];
        __syncthreads();
    }
    if (r == 0 && j < H) out[j] = part[0][c];
}

namespace {
constexpr int64_t kNormBlocks = 2048;      // forward: blocks of the grid-stride loop
constexpr int64_t kNormBwdBlocks = 512;    // backward: blocks, each with its partial column sums

// Rows a unit holds: the rows shared evenly over the blocks, never more than one gate's.
void norm_units(int64_t rows, int64_t n_gates, int64_t &unit_rows, int64_t &per_gate, int64_t &units) {
    const int64_t g = n_gates > 0 ? n_gates : 1, rpg = rows / g;
    unit_rows = (rows + kNormBwdBlocks - 1) / kNormBwdBlocks;
    if (unit_rows > rpg) unit_rows = rpg;
    if (unit_rows < 1) unit_rows = 1;
    per_gate = (rpg + unit_rows - 1) / unit_rows;
    units = per_gate * g;
}
}  // namespace

size_t norm_workspace_bytes(int64_t rows, int64_t width, int64_t n_gates) {
    if (rows <= 0 || width <= 0) return 0;
    int64_t ur, pg, units;
    norm_units(rows, n_gates, ur, pg, units);
    const int64_t nblk = units < kNormBwdBlocks ? units : kNormBwdBlocks;
    return (size_t)((4 * nblk + (pg > 1 ? units : 0)) * width) * sizeof(float);
}

hipError_t launch_norm_fwd(const NormFwd &a, int layer, int fmt, hipStream_t st) {
    const bool vec = a.width % 8 == 0;
#define FP8DS_NF(TPR, V, VEC_, LN_, FMT_)                                                                  \
    do {                                                                                                   \
        constexpr int64_t teams = TPR < 256 ? 256 / TPR : 1;                                               \
        const int64_t need = (a.rows + teams - 1) / teams;                                                 \
        k_norm_fwd<TPR, V, VEC_, LN_, FMT_>                                                                \
            <<<dim3((unsigned)(need < kNormBlocks ? need : kNormBlocks)), TPR < 256 ? 256 : TPR, 0, st>>>(a); \
    } while (0)
#define FP8DS_NF_F(TPR, V, VEC_, LN_)                                                                      \
    do { if (fmt == FP8DS_E4M3) FP8DS_NF(TPR, V, VEC_, LN_, kE4M3); else FP8DS_NF(TPR, V, VEC_, LN_, kE5M2); } while (0)
#define FP8DS_NF_L(TPR, V, VEC_)                                                                           \
    do { if (layer) FP8DS_NF_F(TPR, V, VEC_, true); else FP8DS_NF_F(TPR, V, VEC_, false); } while (0)
#define FP8DS_NF_V(TPR, V)                                                                                 \
    do { if (vec) FP8DS_NF_L(TPR, V, true); else FP8DS_NF_L(TPR, V, false); } while (0)
    if (a.width <= 512) FP8DS_NF_V(64, 1);
    else if (a.width <= 1024) FP8DS_NF_V(64, 2);
    else if (a.width <= 2048) FP8DS_NF_V(256, 1);
    else if (a.width <= 4096) FP8DS_NF_V(256, 2);
    else if (a.width <= 8192) FP8DS_NF_V(512, 2);
    else FP8DS_NF_V(1024, 2);
#undef FP8DS_NF_V
#undef FP8DS_NF_L
#undef FP8DS_NF_F
#undef FP8DS_NF
    return hipGetLastError();
}

hipError_t launch_norm_bwd(NormBwd a, int layer, int64_t n_gates, void *ws, hipStream_t st) {
    norm_units(a.rows, n_gates, a.unit_rows, a.units_per_gate, a.units);   // no rows: no units, the sums are zero
    a.rows_per_gate = a.rows / (n_gates > 0 ? n_gates : 1);
    const int64_t nblk = a.units < kNormBwdBlocks ? a.units : kNormBwdBlocks;
    float *w = static_cast<float *>(ws);
    for (int i = 0; i < 4; ++i) a.col_part[i] = w + i * nblk * a.width;
    a.gate_part = w + 4 * nblk * a.width;
    const bool vec = a.width % 8 == 0;
#define FP8DS_NB(TPR, V)                                                                                   \
    do {                                                                                                   \
        const dim3 grid((unsigned)nblk);                                                                   \
        if (vec && layer) k_norm_bwd<TPR, V, true, true><<<grid, TPR, 0, st>>>(a);                         \
        else if (vec) k_norm_bwd<TPR, V, true, false><<<grid, TPR, 0, st>>>(a);                            \
        else if (layer) k_norm_bwd<TPR, V, false, true><<<grid, TPR, 0, st>>>(a);                          \
        else k_norm_bwd<TPR, V, false, false><<<grid, TPR, 0, st>>>(a);                                    \
    } while (0)
    if (a.rows == 0) {}
    else if (a.width <= 512) FP8DS_NB(64, 1);
    else if (a.width <= 2048) FP8DS_NB(256, 1);
    else if (a.width <= 4096) FP8DS_NB(256, 2);
    else if (a.width <= 8192) FP8DS_NB(512, 2);
    else if (a.width <= 12288) FP8DS_NB(512, 3);
    else FP8DS_NB(512, 4);
#undef FP8DS_NB
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int64_t gates = a.dgate != nullptr && a.units_per_gate != 1 ? n_gates : 0;
    if (gates > 0 || a.dw_pre != nullptr || a.dw_post != nullptr || a.db_pre != nullptr || a.db_post != nullptr)
        k_norm_cols<<<dim3((unsigned)((a.width + 63) / 64), (unsigned)(4 + gates)), 1024, 0, st>>>(a, (int)nblk);
    return hipGetLastError();
}

}  // namespace fp8ds
