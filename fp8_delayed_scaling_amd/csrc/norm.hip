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
// A row belongs to a team of TPR threads, 8 V columns each, held as raw bfloat16 pairs: thread t holds
// the 16-byte chunks t, t + TPR, ...  VEC: width % 8 == 0, every chunk is whole and aligned; otherwise
// the same chunks are loaded and stored at whatever address they have (gfx950 takes 16-byte accesses
// at any) and the row's last, partial chunk one column at a time.
#include "../../include/fp8ds.h"
#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

typedef u32x4 u32x4_any __attribute__((aligned(2)));      // at any bfloat16's address
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

template <int TPR, int V, bool VEC>
struct Row {
    static __device__ __forceinline__ int col(int t, int i) { return (t + (i >> 3) * TPR) * 8 + (i & 7); }
    // chunk v of thread t; columns past the width read as zero
    static __device__ __forceinline__ u32x4 chunk(const uint16_t *__restrict__ p, int H, int t, int v) {
        const int c = (t + v * TPR) * 8;
        u32x4 q = {0u, 0u, 0u, 0u};
        if (c + 8 <= H) {
            q = *reinterpret_cast<const u32x4_any *>(p + c);
        } else if (!VEC && c < H) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (c + i < H) q[i >> 1] |= (uint32_t)p[c + i] << (16 * (i & 1));
        }
        return q;
    }
    // raw[i / 2] holds elements i (low half) and i + 1
    static __device__ __forceinline__ void load(const uint16_t *__restrict__ p, int H, int t, uint32_t (&raw)[4 * V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const u32x4 q = chunk(p, H, t, v);
            raw[4 * v] = q.x; raw[4 * v + 1] = q.y; raw[4 * v + 2] = q.z; raw[4 * v + 3] = q.w;
        }
    }
    static __device__ __forceinline__ float get(const uint32_t (&raw)[4 * V], int i) {
        return (i & 1) ? bf16_hi(raw[i >> 1]) : bf16_lo(raw[i >> 1]);
    }
    static __device__ __forceinline__ void store_chunk(uint16_t *__restrict__ p, int H, int t, int v, u32x4 q) {
        const int c = (t + v * TPR) * 8;
        if (c + 8 <= H) {
            *reinterpret_cast<u32x4_any *>(p + c) = q;
        } else if (!VEC && c < H) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (c + i < H) p[c + i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
        }
    }
    static __device__ __forceinline__ void store(uint16_t *__restrict__ p, int H, int t, const uint32_t (&raw)[4 * V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) store_chunk(p, H, t, v, u32x4{raw[4 * v], raw[4 * v + 1], raw[4 * v + 2], raw[4 * v + 3]});
    }
    // float32 columns (partial sums)
    static __device__ __forceinline__ void store_f32(float *__restrict__ p, int H, int t, const float (&v)[8 * V]) {
#pragma unroll
        for (int q = 0; q < 2 * V; ++q) {
            const int c = col(t, 4 * q);
            if (c + 4 <= H) {
                *reinterpret_cast<f32x4_any *>(p + c) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            } else if (!VEC) {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (c + i < H) p[c + i] = v[4 * q + i];
            }
        }
    }
};

// Sum over the wave's lanes, by moves inside the vector unit, the same order always.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xf>(v);       // from 1, 2, 4, 8 lanes below inside 16
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);       // lane 15 of each 16 to the next 16, lane 31 to the upper half
    v = dpp_add<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Barrier that waits for this wave's LDS accesses only: global loads and stores stay in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
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
            lds_barrier();
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
            lds_barrier();
            a = red[turn][0][0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) a += red[turn][0][w];
            turn ^= 1;
        }
    }
};

// Mean and 1 / standard deviation of the row in v, whose columns past the width hold zero; v becomes its
// deviations from the mean, and those columns stay zero: an infinite (0 - mean) * rstd there would turn
// the next norm's sums into NaN.
template <int TPR, int V, bool VEC, bool LN>
__device__ __forceinline__ void row_stats(float (&v)[8 * V], int H, int t, float eps, TeamSum<TPR> &sum,
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
            v[i] = Row<TPR, V, VEC>::col(t, i) < H ? v[i] - mean : 0.f;
            ss += v[i] * v[i];
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
// Forward: a team per row, rows taken in a grid-stride loop.  Bound by HBM: [8192, 4096] RMS with
// bfloat16 and FP8 output 65.6 us for 302 MB (4.6 TB/s; a plain copy 5.1), [2051, 1001] layer norm
// 9.3 us (20.5 with one column at a time; its teams of one wave are two on a SIMD, which hide little of
// two dependent sums a norm), four rows of 4096 4.2 us, two row sums' latency.
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
                    v[i] = v[i] * rstd * R::get(wr, i);
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
            v[i] = v[i] * rstd * R::get(wr, i);
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
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const u32x2 c = {encode4<FMT>(v[8 * q] * s, v[8 * q + 1] * s, v[8 * q + 2] * s, v[8 * q + 3] * s),
                                 encode4<FMT>(v[8 * q + 4] * s, v[8 * q + 5] * s, v[8 * q + 6] * s, v[8 * q + 7] * s)};
                const int col = R::col(t, 8 * q);
                if (col + 8 <= H) {
                    *reinterpret_cast<u32x2_any *>(a.h8 + base + col) = c;
                } else if (!VEC) {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (col + i < H) a.h8[base + col + i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
                }
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
//   d_resid = alpha d;  dn = gate d
//   d_block = the same form over o with dn * w_post
//   dw_pre = sum dh hat, db_pre = sum dh, dw_post = sum dn ohat, db_post = sum dn, dgate = sum d n
// ([mean of q] for layer norms only).  Inside one gate's rows the gate is a constant, so that the
// sums S1 = sum d ohat and S0 = sum d give all of the last three:
//   dw_post = sum over gates of gate S1, db_post of gate S0, dgate = w_post S1 + b_post S0.
//
// A block takes a unit: a range of rows inside one gate's.  Each thread sums its own columns in
// registers over the rows, one partial per unit goes to the workspace, and k_norm_cols adds the
// partials in a fixed order, so the sums are the same run to run.  MULTI: with more gates than
// blocks a unit is one gate's rows and a block takes several, finishes dgate itself and keeps
// dw_post and db_post in registers too.
//
// VEC: the row's four inputs go straight into LDS (each thread reads back what it loaded itself),
// the next row's as soon as this row's are used, so that a block per CU keeps HBM busy across the
// two sums that every row waits for.  Other widths are loaded into registers.  ([2048, 12288]
// layer norm: the kernel and k_norm_cols took 303 + 33 us with five column sums, spilled registers
// and no loads ahead; they take 85 + 19 us.)  The waits count loads only: the stores issued between
// them make each wait stricter than the load it is for.
//
// Forms that spill registers, with bytes of scratch a thread (VEC / other widths): layer norms past
// 8192 columns (0 / 484) and past 12288 (236 / 420), RMS norms there (0 / 68, 0 / 400); with MULTI layer
// norms past 4096 (12 / 160), 8192 (448 / 1244) and 12288 (440 / 652), RMS norms past 8192 (0 / 124) and
// 12288 (160 / 588).
// ------------------------------------------------------------------------------------------
namespace {
// Uniform statistics by scalar loads: nothing waits behind the row loads and stores in flight.
__device__ __forceinline__ float scalar_at(const float *p, int64_t i) {
    return reinterpret_cast<const __attribute__((address_space(4))) float *>(reinterpret_cast<uint64_t>(p))[i];
}
__device__ __forceinline__ float bf16_of(const u32x4 &q, int i) { return (i & 1) ? bf16_hi(q[i >> 1]) : bf16_lo(q[i >> 1]); }

// A column's mean: zero past the width, where the row was loaded as zero, so that its normalised value
// is zero too ((0 - mean) * rstd may be infinite, and its product with a zero NaN).  The launcher gives
// rows of two chunks a thread and more to teams that they fill at least half: no bound to compare there.
template <int TPR, int V, bool VEC, bool LN>
__device__ __forceinline__ float mean_of(float mean, int H, int t, int v, int i) {
    if (!LN || 2 * (v + 1) <= V) return mean;
    return Row<TPR, V, VEC>::col(t, 8 * v + (VEC ? 0 : i)) < H ? mean : 0.f;
}

// One of a row's inputs: chunk v of the thread in LDS or in registers.
template <int TPR, int V, bool VEC>
struct RowInput {
    u32x4 *lds;
    u32x4 reg[VEC ? 1 : V];
    __device__ __forceinline__ void load(const uint16_t *p, int H, int t) {
        if constexpr (VEC) {
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, H * 2, 0x00020000);
            const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
#pragma unroll
            for (int v = 0; v < V; ++v)      // past the width: out of the buffer's bound, zeros
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)(lds + v * TPR + wave * 64), 16,
                                                         (uint32_t)((t + v * TPR) * 16), 0, 0, 0);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) reg[v] = Row<TPR, V, VEC>::chunk(p, H, t, v);
        }
    }
    __device__ __forceinline__ u32x4 get(int t, int v) const {
        if constexpr (VEC) return lds[v * TPR + t];
        else return reg[v];
    }
};
// Waits for all row loads but the `later` inputs issued last (V loads each; 0 to 3), and for any
// stores between: the compiler does not tie a load into LDS to the reads of it.
template <int V>
__device__ __forceinline__ void wait_inputs(int later) {
    auto wait = [](auto n) {
        constexpr int kVm = waitcnt_vm(decltype(n)::value);
        static_assert(vm_of_waitcnt(kVm) == decltype(n)::value);     // 18 for three inputs of six loads
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kVm);
        asm volatile("" ::: "memory");
    };
    if (later == 3) wait(std::integral_constant<int, 3 * V>{});
    else if (later == 2) wait(std::integral_constant<int, 2 * V>{});
    else if (later == 1) wait(std::integral_constant<int, V>{});
    else wait(std::integral_constant<int, 0>{});
}
// LDS reads are done: their chunks may be loaded anew.
__device__ __forceinline__ void lds_read_done() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}
}  // namespace

template <int TPR, int V, bool VEC, bool LN, bool MULTI>
__global__ __launch_bounds__(TPR) void k_norm_bwd(const NormBwd a) {
    using R = Row<TPR, V, VEC>;
    __shared__ float red[2][2][(TPR + 63) / 64];
    __shared__ u32x4 l_dh[VEC ? TPR * V : 1], l_x[VEC ? TPR * V : 1], l_dx[VEC ? TPR * V : 1], l_o[VEC ? TPR * V : 1];
    RowInput<TPR, V, VEC> i_dh{l_dh}, i_x{l_x}, i_dx{l_dx}, i_o{l_o};
    TeamSum<TPR> sum{red};
    const int t = threadIdx.x;
    const int H = a.width;
    const float inv = 1.0f / (float)H;
    float p1[8 * V], p0[LN ? 8 * V : 1], s1[8 * V], s0[LN ? 8 * V : 1];      // sums of dh hat, dh, d ohat, d
    float w1[MULTI ? 8 * V : 1], w0[MULTI && LN ? 8 * V : 1];                // of gate s1, gate s0
#pragma unroll
    for (int i = 0; i < 8 * V; ++i) {
        p1[i] = 0.f;
        if constexpr (LN) p0[i] = 0.f;
        if constexpr (MULTI) w1[i] = 0.f;
        if constexpr (MULTI && LN) w0[i] = 0.f;
    }
    uint32_t wq[4 * V] = {}, wp[4 * V] = {}, gr[4 * V];
#pragma unroll
    for (int j = 0; j < 4 * V; ++j) gr[j] = 0x3F803F80u;      // without a gate: 1
    if (a.dh != nullptr) R::load(a.w_pre, H, t, wq);
    if (a.w_post != nullptr) R::load(a.w_post, H, t, wp);
    const int has_dh = a.dh != nullptr ? 2 : 0, has_dx = a.dx != nullptr ? 1 : 0, has_o = a.block_out != nullptr ? 1 : 0;
    const int64_t u0 = MULTI ? a.units * blockIdx.x / gridDim.x : blockIdx.x;
    const int64_t u1 = MULTI ? a.units * (blockIdx.x + 1) / gridDim.x : u0 + 1;
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t gi = u / a.units_per_gate, part = u - gi * a.units_per_gate;
        const int64_t r0 = gi * a.rows_per_gate + part * a.unit_rows;
        const int64_t left = a.rows_per_gate - part * a.unit_rows;
        const int64_t r1 = r0 + (left < a.unit_rows ? left : a.unit_rows);
#pragma unroll
        for (int i = 0; i < 8 * V; ++i) {
            s1[i] = 0.f;
            if constexpr (LN) s0[i] = 0.f;
        }
        if (a.gate != nullptr) R::load(a.gate + gi * H, H, t, gr);
        if (VEC && r0 < r1) {
            lds_read_done();
            if (a.dh != nullptr) { i_dh.load(a.dh + r0 * H, H, t); i_x.load(a.x + r0 * H, H, t); }
            if (a.dx != nullptr) i_dx.load(a.dx + r0 * H, H, t);
            if (a.block_out != nullptr) i_o.load(a.block_out + r0 * H, H, t);
        }
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t base = row * H, next = base + H;
            const bool more = row + 1 < r1;
            if constexpr (!VEC) {
                if (a.dh != nullptr) { i_dh.load(a.dh + base, H, t); i_x.load(a.x + base, H, t); }
                if (a.dx != nullptr) i_dx.load(a.dx + base, H, t);
                if (a.block_out != nullptr) i_o.load(a.block_out + base, H, t);
            }
            // opaque in every row: the weights stay packed, two to a register
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) asm volatile("" : "+v"(wq[j]), "+v"(wp[j]), "+v"(gr[j]));
            int tc = t;                       // opaque too: the columns' bounds are compared anew, not kept
            if constexpr (LN) asm volatile("" : "+v"(tc));
            float d[8 * V];
            if (a.dh != nullptr) {
                const float rstd = scalar_at(a.pre_stats, row), mean = LN ? scalar_at(a.pre_stats, a.rows + row) : 0.f;
                float m0 = 0.f, m1 = 0.f;
                if constexpr (VEC) wait_inputs<V>(has_dx + has_o);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 dq = i_dh.get(t, v), xq = i_x.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 8 * v + i;
                        const float dy = bf16_of(dq, i), hat = (bf16_of(xq, i) - mean_of<TPR, V, VEC, LN>(mean, H, tc, v, i)) * rstd;
                        d[k] = dy * R::get(wq, k);          // zero past the width
                        p1[k] += dy * hat;
                        if constexpr (LN) { p0[k] += dy; m0 += d[k]; }
                        m1 += d[k] * hat;
                    }
                }
                if constexpr (LN) sum(m1, m0); else sum(m1);
                m0 *= inv; m1 *= inv;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 xq = i_x.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 8 * v + i;
                        const float hat = (bf16_of(xq, i) - mean_of<TPR, V, VEC, LN>(mean, H, tc, v, i)) * rstd;
                        d[k] = rstd * (d[k] - m0 - hat * m1);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8 * V; ++i) d[i] = 0.f;
            }
            if (a.dx != nullptr) {
                if constexpr (VEC) wait_inputs<V>(has_o);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 q = i_dx.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[8 * v + i] += bf16_of(q, i);
                }
            }
            if (VEC && more) {
                lds_read_done();
                if (a.dh != nullptr) { i_dh.load(a.dh + next, H, t); i_x.load(a.x + next, H, t); }
                if (a.dx != nullptr) i_dx.load(a.dx + next, H, t);
            }
            if (a.d_resid != nullptr) {
                uint32_t raw[4 * V];
#pragma unroll
                for (int j = 0; j < 4 * V; ++j) raw[j] = f32x2_to_bf16x2_rne(a.alpha * d[2 * j], a.alpha * d[2 * j + 1]);
                R::store(a.d_resid + base, H, t, raw);
            }
            if (a.block_out == nullptr) continue;
            uint32_t raw[4 * V];
            if constexpr (VEC) wait_inputs<V>(more ? has_dh + has_dx : 0);
            if (a.w_post != nullptr) {
                const float rstd = scalar_at(a.post_stats, row), mean = LN ? scalar_at(a.post_stats, a.rows + row) : 0.f;
                float m0 = 0.f, m1 = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 q = i_o.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 8 * v + i;
                        const float hat = (bf16_of(q, i) - mean_of<TPR, V, VEC, LN>(mean, H, tc, v, i)) * rstd;
                        s1[k] += d[k] * hat;
                        if constexpr (LN) s0[k] += d[k];
                        d[k] = d[k] * R::get(gr, k) * R::get(wp, k);      // zero past the width
                        if constexpr (LN) m0 += d[k];
                        m1 += d[k] * hat;
                    }
                }
                if constexpr (LN) sum(m1, m0); else sum(m1);
                m0 *= inv; m1 *= inv;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 q = i_o.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 8 * v + i;
                        const float hat = (bf16_of(q, i) - mean_of<TPR, V, VEC, LN>(mean, H, tc, v, i)) * rstd;
                        d[k] = rstd * (d[k] - m0 - hat * m1);
                    }
                }
            } else if (a.gate != nullptr) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const u32x4 q = i_o.get(t, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s1[8 * v + i] += d[8 * v + i] * bf16_of(q, i);
                        d[8 * v + i] *= R::get(gr, 8 * v + i);
                    }
                }
            }
            if (VEC && more) {
                lds_read_done();
                i_o.load(a.block_out + next, H, t);
            }
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) raw[j] = f32x2_to_bf16x2_rne(d[2 * j], d[2 * j + 1]);
            R::store(a.d_block + base, H, t, raw);
        }
        if constexpr (MULTI) {
            // this gate's gradient is complete; its rows' share of the weights' and biases'
            uint32_t br[4 * V];
            if (LN && a.b_post != nullptr) R::load(a.b_post, H, t, br);
            float dg[8 * V];
#pragma unroll
            for (int i = 0; i < 8 * V; ++i) {
                dg[i] = a.w_post != nullptr ? s1[i] * R::get(wp, i) : s1[i];
                if constexpr (LN) if (a.b_post != nullptr) dg[i] += s0[i] * R::get(br, i);
                w1[i] += R::get(gr, i) * s1[i];
                if constexpr (LN) w0[i] += R::get(gr, i) * s0[i];
            }
            if (a.dgate != nullptr) R::store_f32(a.dgate + gi * H, H, t, dg);
        }
    }
    const int64_t at = (int64_t)blockIdx.x * H;
    if (a.dw_pre != nullptr) R::store_f32(a.part[0] + at, H, t, p1);
    if (a.dw_post != nullptr || (!MULTI && a.dgate != nullptr)) {
        if constexpr (MULTI) R::store_f32(a.part[1] + at, H, t, w1);
        else R::store_f32(a.part[1] + at, H, t, s1);
    }
    if constexpr (LN) {
        if (a.db_pre != nullptr) R::store_f32(a.part[2] + at, H, t, p0);
        if (a.db_post != nullptr || (!MULTI && a.dgate != nullptr && a.b_post != nullptr)) {
            if constexpr (MULTI) R::store_f32(a.part[3] + at, H, t, w0);
            else R::store_f32(a.part[3] + at, H, t, s0);
        }
    }
}

// Column sums of the n units' partials: block (c, y) owns CW columns of dw_pre and db_pre (y = 0),
// dw_post and db_post (1) or of gate y - 2.  Thread (r = t / CW, c = t % CW) takes partials r,
// r + 1024 / CW, ...; those sums are then added in a fixed tree.
template <int CW>
__global__ __launch_bounds__(1024) void k_norm_cols(const NormBwd a, int n) {
    constexpr int R = 1024 / CW;
    __shared__ float sums[2][R][CW];
    const int r = threadIdx.x / CW, c = threadIdx.x % CW;
    const int H = a.width;
    const int64_t j = (int64_t)blockIdx.x * CW + c;
    const int y = blockIdx.y;
    float *out1 = y == 0 ? a.dw_pre : y == 1 ? a.dw_post : a.dgate, *out0 = y == 0 ? a.db_pre : y == 1 ? a.db_post : nullptr;
    if (out1 == nullptr && out0 == nullptr) return;   // block-uniform
    const bool second = out0 != nullptr || (y >= 2 && a.b_post != nullptr);
    const float *q1 = a.part[y == 0 ? 0 : 1], *q0 = a.part[y == 0 ? 2 : 3];
    const int per = (int)a.units_per_gate, lo = y < 2 ? 0 : (y - 2) * per, hi = y < 2 ? n : lo + per;
    const bool gated = y == 1 && a.gate != nullptr && !a.gated;
    float v1 = 0.f, v0 = 0.f;
    if (j < H) {
#pragma unroll 4
        for (int i = lo + r; i < hi; i += R) {
            float f = 1.f;
            if (gated) f = __uint_as_float((uint32_t)a.gate[(int64_t)(i / per) * H + j] << 16);
            if (out1 != nullptr) v1 += f * q1[(int64_t)i * H + j];
            if (second) v0 += f * q0[(int64_t)i * H + j];
        }
    }
    sums[0][r][c] = v1;
    sums[1][r][c] = v0;
    __syncthreads();
#pragma unroll
    for (int w = R / 2; w >= 1; w >>= 1) {
        if (r < w) {
            sums[0][r][c] += sums[0][r + w][c];
            sums[1][r][c] += sums[1][r + w][c];
        }
        __syncthreads();
    }
    if (r != 0 || j >= H) return;
    v1 = sums[0][0][c];
    v0 = sums[1][0][c];
    if (y < 2) {
        if (out1 != nullptr) out1[j] = v1;
        if (out0 != nullptr) out0[j] = v0;
    } else {
        if (a.w_post != nullptr) v1 *= __uint_as_float((uint32_t)a.w_post[j] << 16);
        if (a.b_post != nullptr) v1 += v0 * __uint_as_float((uint32_t)a.b_post[j] << 16);
        out1[(int64_t)(y - 2) * H + j] = v1;
    }
}

namespace {
constexpr int64_t kNormBlocks = 2048;      // forward: blocks of the grid-stride loop

// Backward blocks: what a CU holds beside each other of the width's teams (4 KB to 128 KB of LDS), so
// that about as many bytes are in flight at any width, in 256 CUs.
int64_t norm_bwd_blocks(int64_t width) {
    return 256 * (width <= 1024 ? 8 : width <= 2048 ? 4 : width <= 4096 ? 2 : 1);
}
// The rows in units inside one gate's: as many as there are blocks, of four rows at least where that
// leaves one for every CU (a unit writes up to four rows of float32 partials); with more gates than
// blocks one for each gate.
void norm_units(int64_t rows, int64_t width, int64_t n_gates, NormBwd &a) {
    const int64_t g = n_gates > 0 ? n_gates : 1, most = norm_bwd_blocks(width);
    a.rows_per_gate = rows / g;
    const int64_t share = g >= most ? 1 : most / g;              // units of a gate, at most
    a.unit_rows = (a.rows_per_gate + share - 1) / share;
    if (a.unit_rows < 4 && rows >= 4 * 256) a.unit_rows = 4;
    if (a.unit_rows > a.rows_per_gate) a.unit_rows = a.rows_per_gate;
    if (a.unit_rows < 1) a.unit_rows = 1;
    a.units_per_gate = (a.rows_per_gate + a.unit_rows - 1) / a.unit_rows;
    a.units = a.units_per_gate * g;
    a.gated = g > most;
}
}  // namespace

size_t norm_workspace_bytes(int64_t rows, int64_t width, int64_t n_gates) {
    if (rows <= 0 || width <= 0) return 0;
    NormBwd a{};
    norm_units(rows, width, n_gates, a);
    const int64_t n = a.gated ? norm_bwd_blocks(width) : a.units;
    return (size_t)(4 * n * width) * sizeof(float);
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
    norm_units(a.rows, a.width, n_gates, a);              // no rows: no units, the sums are zero
    const int64_t n = a.gated ? norm_bwd_blocks(a.width) : a.units;
    for (int i = 0; i < 4; ++i) a.part[i] = static_cast<float *>(ws) + i * n * a.width;
    const bool vec = a.width % 8 == 0;
#define FP8DS_NB(LN, TPR, V)                                                                               \
    do {                                                                                                   \
        const dim3 grid((unsigned)n);                                                                      \
        if (vec && a.gated) k_norm_bwd<TPR, V, true, LN, true><<<grid, TPR, 0, st>>>(a);                   \
        else if (vec) k_norm_bwd<TPR, V, true, LN, false><<<grid, TPR, 0, st>>>(a);                        \
        else if (a.gated) k_norm_bwd<TPR, V, false, LN, true><<<grid, TPR, 0, st>>>(a);                    \
        else k_norm_bwd<TPR, V, false, LN, false><<<grid, TPR, 0, st>>>(a);                                \
    } while (0)
    // the widest rows: teams whose column sums stay in registers (layer norms keep twice as many:
    // [2048, 12288] 110 us with 256 threads, 128 with 768; rms norms 91 and 84).  Two chunks a thread and
    // more only for widths past half of the team's columns, which the kernel builds on.
    if (a.rows == 0) {}
    else if (a.width <= 512) { if (layer) FP8DS_NB(true, 64, 1); else FP8DS_NB(false, 64, 1); }
    else if (a.width <= 1024) { if (layer) FP8DS_NB(true, 128, 1); else FP8DS_NB(false, 128, 1); }
    else if (a.width <= 2048) { if (layer) FP8DS_NB(true, 256, 1); else FP8DS_NB(false, 256, 1); }
    else if (a.width <= 4096) { if (layer) FP8DS_NB(true, 256, 2); else FP8DS_NB(false, 256, 2); }
    else if (a.width <= 8192) { if (layer) FP8DS_NB(true, 512, 2); else FP8DS_NB(false, 512, 2); }
    else if (a.width <= 12288) { if (layer) FP8DS_NB(true, 256, 6); else FP8DS_NB(false, 768, 2); }
    else { if (layer) FP8DS_NB(true, 1024, 2); else FP8DS_NB(false, 512, 4); }
#undef FP8DS_NB
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int64_t gates = a.dgate != nullptr && !(a.gated && a.rows > 0) ? n_gates : 0;
    if (gates > 0 || a.dw_pre != nullptr || a.dw_post != nullptr || a.db_pre != nullptr || a.db_post != nullptr) {
        const int parts = a.rows > 0 ? (int)n : 0;
        // narrow rows have many partials and few columns: more threads to a column
        if (a.width > 2048) k_norm_cols<64><<<dim3((unsigned)((a.width + 63) / 64), (unsigned)(2 + gates)), 1024, 0, st>>>(a, parts);
        else k_norm_cols<16><<<dim3((unsigned)((a.width + 15) / 16), (unsigned)(2 + gates)), 1024, 0, st>>>(a, parts);
    }
    return hipGetLastError();
}

}  // namespace fp8ds
