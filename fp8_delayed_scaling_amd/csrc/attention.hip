// attention.hip -- attention between the QKV layer and the projection, forward and backward, on gfx950.
//
// Forward, one pass over the keys with a running reference m and sum l of each query row (scores in units of log2):
//   S^T = K Q^T,  P = exp2(S scale log2(e) - m),  O^T += V^T P^T,  l += sum P;   out = O / l, lse = (m + log2 l) ln 2
// The reference moves, and O and l are rescaled, only where a score passes it by 2^8: all quotients stay what they are.
// Backward, from lse, without a sum over the row:
//   P = exp2((S - lse / scale) scale log2(e)),  dS = P (dO V^T - <dO, O>)
//   dQ = scale dS K (k_attn_dq, by query rows);  dV = P^T dO,  dK = scale dS^T Q (k_attn_dkv, by keys)
// in two kernels, so that every sum has one owner and a fixed order; S and dP are computed in both (7 products, not 5).
// P and dS are rounded to bfloat16 as operands: the gradients are off by 0.0023 .. 0.0025 of their norm, 0.0017 of which is their
// own rounding to bfloat16 and as much that of the operands.  In two parts each they take ten products for seven: 4 x 2048
// tokens 725 us for 467, 1 x 8192 2630 for 1660.
//
// Products are 32 x 32 x 16 matrix instructions with the scores transposed: a lane owns one query row (in k_attn_dkv one
// key) and 16 of 32 scores, so a row's maximum and sum take one exchange between the wave's halves, and the 16 values,
// rounded to bfloat16, are the next product's operand as they lie: the contraction runs over the rows in the order in
// which the lanes hold them, and the other operand is read from LDS in that order by transposing reads.  Query rows are
// numbered token by token, the heads of a key/value head's group side by side, so that a tile of keys serves the whole
// group, and the keys' gradients sum over the group inside one block.
//
// What bounds long ones: the matrix units, in use for 59 % (k_attn_dkv) and 64 % (k_attn_dq) of the cycles at 1 x 8192, and
// the power that they draw; shorter ones, 4 x 2048 with 52, 51 and 40 % (k_attn_fwd), the blocks' starts and ends, tiles that
// are half masked, and the waits inside a step.  A loop of these instructions from registers, with random bits, sustains
// 1.75 PFLOP/s on this card, the forward of 1 x 8192 tokens of 32 heads (8 of keys) of 128 1.03 (532 us causal), its backward
// 0.82 of five products, 1.15 of the seven (1684 us); with zeros as inputs, and all else the same, 394 and 1232 us: the
// clock falls from 2.4 to 1.6 .. 1.95 GHz under load.  No single part of a step bounds it: with the loads and barriers left
// out the forward took 9 % less, without the exponentials 8 %, without the reads of LDS 9 %.
#include <climits>

#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kRows = 128;                   // query rows (or keys) of a block, 32 to a wave
constexpr int kFewRows = 32;                 // query rows of a block whose waves share the keys instead
constexpr int kKeys = 64;                    // keys of a step
constexpr int kStepRows = 64;                // query rows of a step
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every descriptor's bound
constexpr int kBufDesc3 = 0x00020000;        // raw buffer descriptor, bounds checked in bytes
constexpr int kMostSplits = 64;              // of the keys
constexpr int kTops = 16, kTopParts = 32;     // rows that are computed again for the amax, shares of their keys
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

#define FP8DS_WAIT_VM(n) __builtin_amdgcn_s_waitcnt(waitcnt_vm(n))
#define FP8DS_WAIT_LGKM() __builtin_amdgcn_s_waitcnt(0xC07F)
#define FP8DS_WAIT_ALL() __builtin_amdgcn_s_waitcnt(0x0070)     // vmcnt(0) lgkmcnt(0)
#define FP8DS_BARRIER()                          \
    do {                                         \
        asm volatile("" ::: "memory");           \
        __builtin_amdgcn_s_barrier();            \
        asm volatile("" ::: "memory");           \
    } while (0)

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// What follows from v is computed where it is used, not ahead of a loop that has no registers to keep it.
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The lane's number, computed where it is used.
__device__ __forceinline__ int lane_now() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}
__device__ __forceinline__ float uniform_value(float v) { return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v))); }
// an offset, past every bound where left is negative
__device__ __forceinline__ uint32_t held(uint32_t off, int left) { return off | ((uint32_t)left & kOutside); }

// ---------------------------------------------------------------------------------- sequences
struct Span {
    int64_t begin;
    int len;
};
// Sequence b's tokens, held to [0, T) whatever the offsets are.
__device__ __forceinline__ Span span_of(const int32_t *off, int b, int T, int B) {
    if (off == nullptr) {
        const int len = T / B;
        return Span{(int64_t)b * len, len};
    }
    const int lo = min(max(off[b], 0), T), hi = min(max(off[b + 1], lo), T);
    return Span{lo, hi - lo};
}

// Tile t of the sequences' rows (`group` rows a token, `height` rows a tile): its sequence and its number in it,
// the last tile of a sequence first.  False past the last.
__device__ __forceinline__ bool find_tile(const int32_t *off, int T, int B, int group, int height, int t, int &b, int &tile) {
    if (off == nullptr) {
        const int n = (T / B * group + height - 1) / height;
        b = t % B;
        tile = n - 1 - t / B;
        return tile >= 0;
    }
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const int i = b0 + lane;
        int n = 0;
        if (i < B) n = (int)(((int64_t)span_of(off, i, T, B).len * group + height - 1) / height);
        int64_t upto = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t v = __shfl_up(upto, d, 64);
            if (lane >= d) upto += v;
        }
        const uint64_t past = __ballot(before + upto > t);
        if (past != 0) {
            const int first = __ffsll((unsigned long long)past) - 1;
            b = uniform(b0 + first);
            const int64_t end = before + __shfl(upto, first, 64);
            tile = uniform((int)(end - 1 - t));
            return true;
        }
        before += __shfl(upto, 63, 64);
    }
    return false;
}

// ------------------------------------------------------------------------------------- tiles
// A tile in LDS holds rows of PITCH bytes in 16-byte pieces; piece c of a row lies at c ^ swz(row), so that reading one
// piece of many rows and reading 4 rows of the transposed form both reach all banks.
template <int DB> struct Shape {                 // DB: head size in blocks of 32
    static constexpr int pitch = DB <= 2 ? 128 : 256;
    static constexpr int pieces = pitch / 16;
    static constexpr int rows_a_load = 1024 / pitch;     // rows that one load of a wave fills
    static constexpr int ks = 2 * DB;                    // steps of 16 along the head
    static __device__ __forceinline__ int swz(int row) {
        return pitch == 256 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
    }
};

// A lane's addresses in a tile.  row[ks]: row l % 32, elements 16 ks + 8 (l / 32) .. + 7, an operand whose contraction
// runs along the head.  tr[d][s]: the transposed read of elements 32 d + l % 32 of the rows 8 s + 4 (l / 32) .. + 3, an
// operand whose contraction runs over the rows.
template <int DB> struct Reader {
    uint32_t row[2 * DB], tr[DB][2];
    __device__ __forceinline__ explicit Reader(int lane) {
        using S = Shape<DB>;
        const int r = lane & 31, h = lane >> 5;
#pragma unroll
        for (int k = 0; k < S::ks; ++k) row[k] = r * S::pitch + ((2 * k + h) ^ S::swz(r)) * 16;
        const int i = lane & 15;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int tr_row = 8 * s + 4 * h + (i >> 2), c = 4 * d + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1);
                tr[d][s] = tr_row * S::pitch + (c ^ S::swz(tr_row)) * 16 + (i & 1) * 8;
            }
    }
};
__device__ __forceinline__ bf16x8 read_row(const uint8_t *p) { return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p)); }
__device__ __forceinline__ i16x4 read_tr4(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)p);
}
// rows s .. of block d: 16 rows of the contraction, in the order in which the products leave them (rows 4 h .. + 3, then
// 8 + 4 h .. + 3 for lane half h)
template <int DB> __device__ __forceinline__ bf16x8 read_tr(const uint8_t *p, const Reader<DB> &rd, int d) {
    const i16x4 a = read_tr4(p + rd.tr[d][0]), b = read_tr4(p + rd.tr[d][1]);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
// The same addresses from three registers: the pieces' numbers enter by exclusive or.  In the kernels with 200 and more
// registers in use these instructions cost less than the 13 registers (k_attn_dkv spills with a Reader; the forward and
// k_attn_dq take the same time with either).
template <int DB> struct Walker {
    uint32_t row0, tr0, tr1;
    __device__ __forceinline__ explicit Walker(int lane) {
        const Reader<DB> rd(lane);
        row0 = rd.row[0], tr0 = rd.tr[0][0], tr1 = rd.tr[0][1];
    }
    // keeps the addresses from being computed ahead of the loop, into registers
    __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(row0), "+v"(tr0), "+v"(tr1)); }
    __device__ __forceinline__ uint32_t row(int k) const { return row0 ^ (k * 32); }
    __device__ __forceinline__ bf16x8 tr(const uint8_t *p, int d) const {
        const i16x4 a = read_tr4(p + (tr0 ^ (d * 64))), b = read_tr4(p + (tr1 ^ (d * 64)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};
__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
// eight of the 16 values that a lane holds of a 32 x 32 product, as an operand of the next
__device__ __forceinline__ bf16x8 pack8(const f32x16 &v, int s) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)v[8 * s + i];
    return r;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const void *p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)(uint32_t)uniform((int)a) | (uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(u), (short)0, uniform((int)bytes), kBufDesc3);
}
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rs, uint8_t *to, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)to, 16, off, 0, 0, 0);
}

// Loads of ROWS consecutive rows (tokens) by WAVES waves, rows and pieces past the end as zeros.
template <int DB, int ROWS, int WAVES> struct RowLoads {
    using S = Shape<DB>;
    static constexpr int n = ROWS / (S::rows_a_load * WAVES);                    // loads of a wave
    static constexpr int variants = S::rows_a_load * WAVES >= 16 ? 1 : 16 / (S::rows_a_load * WAVES);
    uint32_t off[variants];
    uint32_t step;                                                               // bytes from variant to variant's next turn
    int wave;
    __device__ __forceinline__ RowLoads(int lane, int wave_, int D, int64_t ts) : wave(wave_) {
#pragma unroll
        for (int i = 0; i < variants; ++i) {
            const int row = (i * WAVES + wave) * S::rows_a_load + lane / S::pieces, c = (lane % S::pieces) ^ S::swz(row);
            off[i] = c * 8 < D ? (uint32_t)(row * (int)ts * 2 + c * 16) : kOutside;
        }
        step = (uint32_t)(variants * WAVES * S::rows_a_load * (int)ts * 2);
    }
    // `first`: the first row; `left`: rows there are (at least one)
    __device__ __forceinline__ void operator()(const uint16_t *first, int64_t ts, int left, uint8_t *tile) const {
        const auto rs = bounded(first, (uint32_t)min(left, ROWS) * (uint32_t)ts * 2u);
#pragma unroll
        for (int i = 0; i < n; ++i) load_lds(rs, tile + (i * WAVES + wave) * 1024, off[i % variants] + (i / variants) * step);
    }
};

__device__ __forceinline__ float both_halves_max(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float both_halves_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
// A lane's values 8 s .. 8 s + 7 of a product [32 x 32] whose columns are lanes, turned into 8 consecutive rows:
// 16 s + 8 (l / 32) .. + 7.
__device__ __forceinline__ void consecutive8(const f32x16 &v, int s, float (&o)[8]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[8 * s + u]), __float_as_uint(v[8 * s + 4 + u]), false, false);
        o[u] = __uint_as_float(p[0]);
        o[4 + u] = __uint_as_float(p[1]);
    }
}
__device__ __forceinline__ u32x4 to_bf16(const float (&v)[8]) {
    return u32x4{f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]), f32x2_to_bf16x2_rne(v[4], v[5]), f32x2_to_bf16x2_rne(v[6], v[7])};
}

// Eight values of one output row: bfloat16, codes, the largest magnitude.
struct Emit {
    float scale;
    uint64_t best = 0;                           // the largest magnitude's bits, then the row's complement: ties to the lowest
    __device__ __forceinline__ explicit Emit(const Attention &a) : scale(a.out8 != nullptr ? *a.scale : 1.f) {}
    __device__ __forceinline__ void operator()(const Attention &a, int64_t token, int head, int d, const float (&v)[8]) {
        if (a.out.p != nullptr) *reinterpret_cast<u32x4 *>(a.out.p + token * a.out.ts + head * a.out.hs + d) = to_bf16(v);
        if (a.out8 == nullptr) return;
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        const uint64_t mine = (uint64_t)amax << 32 | (uint32_t)~(uint32_t)(token * a.Hq + head);
        best = best > mine ? best : mine;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * scale;
        u32x2 w;
        if (a.fmt == kE4M3) w = u32x2{encode4<kE4M3>(y[0], y[1], y[2], y[3]), encode4<kE4M3>(y[4], y[5], y[6], y[7])};
        else w = u32x2{encode4<kE5M2>(y[0], y[1], y[2], y[3]), encode4<kE5M2>(y[4], y[5], y[6], y[7])};
        *reinterpret_cast<u32x2 *>(a.out8 + (token * a.Hq + head) * a.D + d) = w;
    }
    // Every lane of the wave takes part.  Outputs made of rounded probabilities leave the wave's largest with its row,
    // for k_attn_amax; exact ones go straight into the slot.
    __device__ __forceinline__ void finish(const Attention &a) {
        if (a.out8 == nullptr || a.amax == nullptr) return;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const uint64_t other = __shfl_xor((unsigned long long)best, o, 64);
            best = best > other ? best : other;
        }
        if ((threadIdx.x & 63) != 0) return;
        if (a.top == nullptr) {
            fold_amax_bits(a.amax, (uint32_t)(best >> 32));
        } else {
            a.top[blockIdx.x * kWaves + (threadIdx.x >> 6)] = (uint32_t)(best >> 32);
            a.top_row[blockIdx.x * kWaves + (threadIdx.x >> 6)] = (int32_t)~(uint32_t)best;
        }
    }
};
__device__ __forceinline__ void write_inverse(const Attention &a) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.out8 != nullptr && a.sinv != nullptr) *a.sinv = 1.0f / *a.scale;
    if (blockIdx.x == 0 && threadIdx.x < kTops && a.top != nullptr) a.top_done[threadIdx.x] = 0;      // k_attn_amax counts there
}

// Keys that query row `pos` of a sequence may see: [lo, hi).
struct Seen {
    int lo, hi;
};
__device__ __forceinline__ Seen seen(const Attention &a, int pos, int lq, int lk) {
    if (!a.causal) return Seen{0, lk};
    const int at = pos + (lk - lq);              // the row's own key
    return Seen{a.window > 0 ? max(0, at - a.window + 1) : 0, min(lk, at + 1)};
}

// The running reference of a row's sums, in units of log2 (m; ref: 0 for none).  An exponential is exp2(fma(score, s2, -ref)), and
// ref a rounding of score * s2 for the largest: where that passes 2^30, half a step of it is 32 and more, and the largest
// exponential would be 0 or an infinity.  Such a row takes the power of two below s2, with which the product is exact: scores a
// step apart are then 2^-32 and less of each other with either.  Nothing changes for all other rows, nor in time (1 x 8192 524
// us with and without; (score - m) * s2 for every score instead, one instruction more, 549).
constexpr float kFar = 0x1p30f;
constexpr float kFarLse = 0x1p24f;               // beyond it no digit of exp(score - lse) is left of a float32 lse
struct Reference {
    float m = -kInf, ref = 0.f, s2;
    __device__ __forceinline__ explicit Reference(float all) : s2(all) {}
    // from the largest score so far: what the sums are to be multiplied by
    __device__ __forceinline__ float move(float top, float all) {
        const float mx = top * all, mn = fmaxf(m, mx), al = mn == -kInf ? 1.f : __builtin_amdgcn_exp2f(m - mn);
        if (mx > m) {
            s2 = fabsf(mx) > kFar ? __uint_as_float(__float_as_uint(all) & 0xFF800000u) : all;
            ref = top * s2;
        }
        m = mn;
        return al;
    }
};

// The running softmax of k_attn_fwd_few, 32 keys a step.  Its probabilities enter the second product as three bfloat16, which
// hold all 24 bits: bytes and not products are the bound there, so exact ones cost nothing (k_attn_fwd rounds them to one).
template <int DB> struct Softmax {
    f32x16 o[DB];
    Reference r;
    float l = 0.f;                               // of this lane's keys only
    __device__ __forceinline__ explicit Softmax(float s2) : r(s2) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    }
    __device__ __forceinline__ void step(const uint8_t *sk, const uint8_t *sv, const Reader<DB> &rd, const bf16x8 (&qf)[2 * DB],
                                         float s2, bool masked, int key0, Seen see, int lane) {
        using S = Shape<DB>;
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
        for (int k = 0; k < S::ks; ++k) s = mfma(read_row(sk + rd.row[k]), qf[k], s);
        if (masked) {
            const int h4 = key0 + 4 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = h4 + (i >> 2) * 8 + (i & 3);
                s[i] = key >= see.lo && key < see.hi ? s[i] : -kInf;
            }
        }
        float mx = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
        mx = both_halves_max(mx);
        if (__any(mx * s2 > r.m + 8.f)) {        // no lane past 2^8 of its reference: the sums are kept as they are
            const float al = r.move(mx, s2);
            l *= al;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= al;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], r.s2, -r.ref));
            l += s[i];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            f32x16 left;
            const bf16x8 p = pack8(s, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) left[i] = s[8 * x + i] - (float)p[i];
            const bf16x8 p2 = pack8(left, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) left[i] -= (float)p2[i];
            const bf16x8 p3 = pack8(left, 0);
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const bf16x8 v = read_tr<DB>(sv + x * 16 * S::pitch, rd, d);
                o[d] = mfma(v, p, o[d]);
                o[d] = mfma(v, p2, o[d]);
                o[d] = mfma(v, p3, o[d]);
            }
        }
    }
};

// The lane's row as an operand: elements 16 k + 8 (l / 32) .. + 7, zeros past the head or where there is no row.  Without
// a branch: what is not there is read from `any`, a row that is.
template <int DB>
__device__ __forceinline__ void load_query(bf16x8 (&f)[2 * DB], const uint16_t *row, const uint16_t *any, bool there, int D, int half) {
    const uint16_t *from = there ? row : any;
    u32x4 v[2 * DB];
#pragma unroll
    for (int k = 0; k < 2 * DB; ++k) v[k] = *reinterpret_cast<const u32x4 *>(from + (k * 16 + half * 8 < D ? k * 16 + half * 8 : 0));
#pragma unroll
    for (int k = 0; k < 2 * DB; ++k) {
        const bool in = there && k * 16 + half * 8 < D;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[k][u] = in ? v[k][u] : 0u;
        f[k] = __builtin_bit_cast(bf16x8, v[k]);
    }
}

// What a part's sums count in the whole: about its reference m, against the whole's.  Without a key that counts l is 0, or NaN
// where the scores were, and stays one.
__device__ __forceinline__ float part_weight(float m, float l, float whole) { return m == -kInf ? l * 0.f : __builtin_amdgcn_exp2f(m - whole); }

__device__ __forceinline__ float *part_sums(const Attention &a, int split) { return a.part + ((int64_t)split * a.Tq * a.Hq) * a.D; }
__device__ __forceinline__ float *part_stats(const Attention &a, int split) {
    return a.part + (int64_t)a.splits * a.Tq * a.Hq * a.D + (int64_t)split * a.Tq * a.Hq * 2;
}

}  // namespace

// A block: 128 query rows of one key/value head, 32 to each wave; all waves read the same 64 keys a step, from two turns of
// LDS (64 KB, two blocks to a CU, so that one block's barrier and exponentials lie beside the other's products).  A wave none
// of whose rows sees a step computes it all the same: a branch around it would have the sums copied.  The probabilities are
// rounded to bfloat16 (off by up to 2^-8 of each term, as the output itself): the matrix instruction's type.  The output is
// off by 0.0023 of its norm, in two parts, with twice the products for the sums, by 0.0017, its own rounding: 204 us for 152
// at 4 x 2048 without an amax, 729 for 525 at 1 x 8192.
// 4 x 2048 tokens, 32 heads, 8 of keys, of 128, causal: 168 .. 180 us, 0.8 PFLOP/s (half of a tile at the diagonal counts for
// nothing, and a block's start and end take 4 us of 45); without a mask 280 us, 0.98; 1 x 16384 causal 1.07; 1 x 8192 with a
// window of 1024 and the amax 175.  What a head size that fills no block of 32 costs: 72 is computed as 96 (1 x 2048 41 us; as
// 128 46, and 2 x 4096 of 96 237 and 263 us), sizes up to 56 as 64.
template <int DB>
__global__ __launch_bounds__(kThreads, 2) void k_attn_fwd(const Attention a) {
    using S = Shape<DB>;
    constexpr int kTile = kKeys * S::pitch, kRun = 2 * DB, kAhead = 3;
    // two turns of K and V: arrays of their own, so that reading one does not wait for the loads into the other
    __shared__ __align__(1024) uint8_t k0[kTile], k1[kTile], v0[kTile], v1[kTile];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    write_inverse(a);
    const int kvh = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, split = rest % a.splits;
    int b, tile;
    if (!find_tile(a.offsets_q, a.Tq, a.B, a.G, kRows, rest / a.splits, b, tile)) {
        if (a.top != nullptr && a.splits == 1 && lane == 0) a.top[blockIdx.x * kWaves + wave] = 0;
        return;
    }
    const Span sq = span_of(a.offsets_q, b, a.Tq, a.B), sk = span_of(a.offsets_k, b, a.Tk, a.B);
    const int rows = sq.len * a.G, r0 = tile * kRows, last = min(r0 + kRows, rows) - 1;
    const int r0w = r0 + wave * 32, r = r0w + (lane & 31);
    const int pos = r / a.G, head = kvh * a.G + r - pos * a.G;
    const bool there = r < rows;
    const int64_t token = sq.begin + pos;
    bf16x8 qf[S::ks];
    load_query<DB>(qf, a.q.p + token * a.q.ts + head * a.q.hs, a.q.p, there, a.D, lane >> 5);

    // keys of the block, of the wave, of the lane
    int lo = seen(a, r0 / a.G, sq.len, sk.len).lo & ~(kKeys - 1), hi = seen(a, last / a.G, sq.len, sk.len).hi;
    if (a.splits > 1) {
        const int steps = (max(hi - lo, 0) + kKeys - 1) / kKeys, each = (steps + a.splits - 1) / a.splits;
        lo += split * each * kKeys;
        hi = min(hi, lo + each * kKeys);
    }
    const int wf = min(r0w, last) / a.G, wl = min(r0w + 31, last) / a.G;
    const Seen first = seen(a, wf, sq.len, sk.len), end = seen(a, wl, sq.len, sk.len);
    const Seen see = seen(a, pos, sq.len, sk.len);         // rows past the last compute what is never written

    const RowLoads<DB, kKeys, kWaves> loads_k(lane, wave, a.D, a.k.ts), loads_v(lane, wave, a.D, a.v.ts);
    const uint16_t *kp = a.k.p + sk.begin * a.k.ts + kvh * a.k.hs, *vp = a.v.p + sk.begin * a.v.ts + kvh * a.v.hs;
    Walker<DB> rd(lane);
    const float s2 = uniform_value(a.softmax_scale * kLog2e);
    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    Reference row(s2);
    float l = 0.f;                               // of this lane's keys only
    if (lo < hi) {
        loads_k(kp + (int64_t)lo * a.k.ts, a.k.ts, sk.len - lo, k0);
        loads_v(vp + (int64_t)lo * a.v.ts, a.v.ts, sk.len - lo, v0);
    }
    auto turn = [&](int j, const uint8_t *tk, const uint8_t *tv, uint8_t *next_k, uint8_t *next_v) __attribute__((always_inline)) {
        FP8DS_WAIT_ALL();
        FP8DS_BARRIER();
        const int next = j + kKeys;
        if (next < hi) {
            loads_k(kp + (int64_t)next * a.k.ts, a.k.ts, sk.len - next, next_k);
            loads_v(vp + (int64_t)next * a.v.ts, a.v.ts, sk.len - next, next_v);
        }
        const bool masked = next > first.hi || j < end.lo;
        // Four runs of products, kRun each: the scores of 32 keys, of the next 32, and the sums over either.  The first
        // 32 keys' exponentials go beside the second run, the others' beside the third; operands are read kAhead ahead.
        // The exponentials are taken about the reference as it is, and again where a score proves to be past 2^8 of it.
        f32x16 s[2];
        bf16x8 f[kAhead], p[2][2];
        float part[2], mx;
        auto read = [&](int n) __attribute__((always_inline)) {
            if (n < 2 * kRun) return read_row(tk + (n / kRun) * 32 * S::pitch + rd.row(n % kRun));
            const int kb = n / kRun - 2, x = (n % kRun) / DB, d = n % DB;
            return rd.tr(tv + (kb * 32 + x * 16) * S::pitch, d);
        };
        auto mask = [&](int kb) __attribute__((always_inline)) {
            if (!masked) return;
            const int key0 = j + kb * 32 + 4 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = key0 + (i >> 2) * 8 + (i & 3);
                s[kb][i] = key >= see.lo && key < see.hi ? s[kb][i] : -kInf;
            }
        };
        // share n of kRun of the exponentials of a run's scores; the last packs them
        auto values = [&](int kb, int n) __attribute__((always_inline)) {
            if (n == 0) mx = s[kb][0], part[kb] = 0.f;
#pragma unroll
            for (int i = n * 16 / kRun; i < (n + 1) * 16 / kRun; ++i) {
                mx = fmaxf(mx, s[kb][i]);
                float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], row.s2, -row.ref));
                asm volatile("" : "+v"(e));          // here, not behind the branch that they might not reach
                part[kb] += e;
                p[kb][i / 8][i % 8] = (__bf16)e;
            }
        };
        auto settle = [&](int kb) __attribute__((always_inline)) {
            mx = both_halves_max(mx);
            if (__any(mx * s2 > row.m + 8.f)) {
                const float al = row.move(mx, s2);
                l *= al;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= al;
#pragma unroll
                for (int n = 0; n < kRun; ++n) values(kb, n);
            }
            l += part[kb];
        };
        rd.fresh();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[0][i] = s[1][i] = 0.f;
#pragma unroll
        for (int n = 0; n < kAhead; ++n) f[n] = read(n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kRun; ++n) {
            const bf16x8 now = f[n % kAhead];
            f[n % kAhead] = read(n + kAhead);
            s[0] = mfma(now, qf[n], s[0]);
            __builtin_amdgcn_sched_barrier(0);
        }
        mask(0);
        rd.fresh();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kRun; ++n) {
            const bf16x8 now = f[(n + kRun) % kAhead];
            f[(n + kRun) % kAhead] = read(n + kRun + kAhead);
            s[1] = mfma(now, qf[n], s[1]);
            values(0, n);
            __builtin_amdgcn_sched_barrier(0);
        }
        settle(0);
        mask(1);
        rd.fresh();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kRun; ++n) {
            const bf16x8 now = f[(n + 2 * kRun) % kAhead];
            f[(n + 2 * kRun) % kAhead] = read(n + 2 * kRun + kAhead);
            o[n % DB] = mfma(now, p[0][n / DB], o[n % DB]);
            values(1, n);
            __builtin_amdgcn_sched_barrier(0);
        }
        settle(1);
        rd.fresh();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kRun; ++n) {
            const bf16x8 now = f[(n + 3 * kRun) % kAhead];
            if (n + kAhead < kRun) f[(n + 3 * kRun) % kAhead] = read(n + 3 * kRun + kAhead);
            o[n % DB] = mfma(now, p[1][n / DB], o[n % DB]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // a branch around a step, or out of the loop between two, would have the sums copied at each
    int j = lo;
    for (; j + kKeys < hi; j += 2 * kKeys) {
        turn(j, k0, v0, k1, v1);
        turn(j + kKeys, k1, v1, k0, v0);
    }
    if (j < hi) turn(j, k0, v0, k1, v1);
    l = both_halves_sum(l);
    if (a.splits > 1) {
        if (!there) return;
        const int64_t at_row = token * a.Hq + head;
        if (lane < 32) {
            float *st = part_stats(a, split) + at_row * 2;
            st[0] = row.m;
            st[1] = l;
        }
        float *to = part_sums(a, split) + at_row * a.D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = d * 32 + i * 8 + (lane >> 5) * 4;
                if (at < a.D) *reinterpret_cast<f32x4 *>(to + at) = f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
            }
        return;
    }
    const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;       // a NaN stays one
    if (there && lane < 32 && a.lse != nullptr) a.lse[(int64_t)head * a.Tq + token] = l == 0.f ? -kInf : (row.m + __builtin_amdgcn_logf(l)) * kLn2;
    // The rows go out through LDS, kLanes lanes to a row and 8 elements to a lane, so that the casts are one short loop: as
    // straight code from the registers they took more of the instruction cache than all else.
    constexpr int kLanes = DB == 2 ? 8 : 16, kPieces = 2 * kLanes;   // 16-byte pieces of a row; lane l's row keeps them at p ^ l
    FP8DS_WAIT_ALL();
    FP8DS_BARRIER();
    uint8_t *const stage = wave == 0 ? k0 : wave == 1 ? k1 : wave == 2 ? v0 : v1;
    static_assert(kTile >= 32 * kPieces * 16, "an array holds a wave's rows");
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = lane & 31, piece = (8 * d + 2 * i + (lane >> 5)) ^ (x & (kPieces - 1));
            *reinterpret_cast<f32x4 *>(stage + (x * kPieces + piece) * 16) = f32x4{o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
        }
    FP8DS_WAIT_LGKM();
    asm volatile("" ::: "memory");
    Emit emit(a);
    const int at = lane % kLanes * 8;
#pragma unroll 1
    for (int x = lane / kLanes; x < 32; x += 64 / kLanes) {
        const int rr = r0w + x, p = rr / a.G;
        if (rr >= rows || at >= a.D) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 y = *reinterpret_cast<const f32x4 *>(stage + (x * kPieces + ((at / 4 + i) ^ (x & (kPieces - 1)))) * 16);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[4 * i + u] = y[u];
        }
        emit(a, sq.begin + p, kvh * a.G + rr - p * a.G, at, v);
    }
    emit.finish(a);
}

// A block: up to 32 query rows of one key/value head; its waves share the keys, 32 to a wave, each with two turns of LDS of
// its own and no barrier until the end.  Bound by the bytes of K and V: 16 sequences of up to 4096 keys, 8 key heads of 128,
// 170 MB in 33.5 us, 5.0 TB/s, what a copy reaches; k_attn_join behind it 5.0 us.
template <int DB>
__global__ __launch_bounds__(kThreads, 1) void k_attn_fwd_few(const Attention a) {
    using S = Shape<DB>;
    constexpr int kTile = 32 * S::pitch, kPitch = 32 * DB + 4;       // floats of an output row in LDS
    // each wave's K and V, two turns; afterwards the waves' sums
    constexpr int kPart = kWaves * kTile;
    static_assert(kPart >= 32 * kPitch * 4, "an array holds one wave's sums");
    __shared__ __align__(1024) uint8_t k0[kPart], k1[kPart], v0[kPart], v1[kPart];
    __shared__ float stats[kWaves][32][2];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    write_inverse(a);
    const int kvh = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv, split = rest % a.splits;
    int b, tile;
    if (!find_tile(a.offsets_q, a.Tq, a.B, a.G, kFewRows, rest / a.splits, b, tile)) return;
    const Span sq = span_of(a.offsets_q, b, a.Tq, a.B), sk = span_of(a.offsets_k, b, a.Tk, a.B);
    const int rows = sq.len * a.G, r0 = tile * kFewRows, last = min(r0 + kFewRows, rows) - 1;
    const int r = r0 + (lane & 31), pos = r / a.G, head = kvh * a.G + r - pos * a.G;
    const bool there = r < rows;
    bf16x8 qf[S::ks];
    load_query<DB>(qf, a.q.p + (sq.begin + pos) * a.q.ts + head * a.q.hs, a.q.p, there, a.D, lane >> 5);
    const Seen first = seen(a, r0 / a.G, sq.len, sk.len), end = seen(a, last / a.G, sq.len, sk.len);
    const Seen see = seen(a, pos, sq.len, sk.len);         // rows past the last compute what is never written
    constexpr int kStep = kWaves * 32;
    int lo = first.lo & ~31, hi = end.hi;
    if (a.splits > 1) {
        const int steps = (max(hi - lo, 0) + kStep - 1) / kStep, each = (steps + a.splits - 1) / a.splits;
        lo += split * each * kStep;
        hi = min(hi, lo + each * kStep);
    }
    const RowLoads<DB, 32, 1> loads_k(lane, 0, a.D, a.k.ts), loads_v(lane, 0, a.D, a.v.ts);
    const uint16_t *kp = a.k.p + sk.begin * a.k.ts + kvh * a.k.hs, *vp = a.v.p + sk.begin * a.v.ts + kvh * a.v.hs;
    const Reader<DB> rd(lane);
    const float s2 = a.softmax_scale * kLog2e;
    Softmax<DB> sm(s2);
    const int mine = wave * kTile;
    int j = lo + wave * 32;
    if (j < hi) {
        loads_k(kp + (int64_t)j * a.k.ts, a.k.ts, sk.len - j, k0 + mine);
        loads_v(vp + (int64_t)j * a.v.ts, a.v.ts, sk.len - j, v0 + mine);
    }
    auto turn = [&](int at, const uint8_t *tk, const uint8_t *tv, uint8_t *next_k, uint8_t *next_v) __attribute__((always_inline)) {
        const int next = at + kStep;
        FP8DS_WAIT_LGKM();                                           // the reads of the tile that is overwritten next
        asm volatile("" ::: "memory");
        if (next < hi) {
            loads_k(kp + (int64_t)next * a.k.ts, a.k.ts, sk.len - next, next_k + mine);
            loads_v(vp + (int64_t)next * a.v.ts, a.v.ts, sk.len - next, next_v + mine);
            FP8DS_WAIT_VM(2 * decltype(loads_k)::n);
        } else {
            FP8DS_WAIT_VM(0);
        }
        asm volatile("" ::: "memory");
        const bool masked = at + 32 > first.hi || at < end.lo;
        sm.step(tk + mine, tv + mine, rd, qf, s2, masked, at, see, lane);
    };
    for (; j + kStep < hi; j += 2 * kStep) {
        turn(j, k0, v0, k1, v1);
        turn(j + kStep, k1, v1, k0, v0);
    }
    if (j < hi) turn(j, k0, v0, k1, v1);
    // the four waves' sums, joined in order
    const float l = both_halves_sum(sm.l);
    if (lane < 32) {
        stats[wave][lane][0] = sm.r.m;
        stats[wave][lane][1] = l;
    }
    __syncthreads();
    const uint8_t *const sums[kWaves] = {k0, k1, v0, v1};
    uint8_t *own = wave == 0 ? k0 : wave == 1 ? k1 : wave == 2 ? v0 : v1;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4 *>(own + ((lane & 31) * kPitch + d * 32 + i * 8 + (lane >> 5) * 4) * 4) =
                f32x4{sm.o[d][4 * i], sm.o[d][4 * i + 1], sm.o[d][4 * i + 2], sm.o[d][4 * i + 3]};
    __syncthreads();
    Emit emit(a);
    constexpr int kPer = 4 * DB;                                     // threads of a row, 8 elements each
    for (int w = threadIdx.x; w < (last - r0 + 1) * kPer; w += kThreads) {
        const int x = w / kPer, d = w % kPer * 8, rr = r0 + x, p = rr / a.G, hd = kvh * a.G + rr - p * a.G;
        if (d >= a.D) continue;
        float m = -kInf, sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kWaves; ++i) m = fmaxf(m, stats[i][x][0]);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float wt = part_weight(stats[i][x][0], stats[i][x][1], m);
            sum += stats[i][x][1] * wt;
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] += reinterpret_cast<const float *>(sums[i])[x * kPitch + d + u] * wt;
        }
        const int64_t token = sq.begin + p, row = token * a.Hq + hd;
        if (a.splits > 1) {
            float *to = part_sums(a, split) + row * a.D + d;
            *reinterpret_cast<f32x4 *>(to) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4 *>(to + 4) = f32x4{v[4], v[5], v[6], v[7]};
            if (d == 0) {
                float *st = part_stats(a, split) + row * 2;
                st[0] = m;
                st[1] = sum;
            }
            continue;
        }
        const float inv = sum > 0.f ? 1.0f / sum : sum == 0.f ? 0.f : sum;
        if (d == 0 && a.lse != nullptr) a.lse[(int64_t)hd * a.Tq + token] = sum == 0.f ? -kInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= inv;
        emit(a, token, hd, d, v);
    }
    if (a.splits == 1) emit.finish(a);
}

// The splits' sums of each row, joined in order.  16 threads a row; rows of no sequence stay as they are.  Bound by the
// latency of two dependent rounds of loads (5 us), then by the parts' bytes: 8192 rows of 8 parts, 34 MB, 8.7 us.
__global__ __launch_bounds__(kThreads) void k_attn_join(const Attention a) {
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int d = (threadIdx.x & 15) * 8;
    const int64_t token = row / a.Hq;
    const int head = (int)(row - token * a.Hq);
    bool there = token < a.Tq;
    if (there && a.offsets_q != nullptr) {
        // the last sequence that begins at or before the token
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.offsets_q[mid] <= token) lo = mid;
            else hi = mid;
        }
        there = a.offsets_q[lo] <= token && token < a.offsets_q[lo + 1];
    }
    Emit emit(a);
    if (there) {
        // lane l of the row takes the stats of the splits l, l + 16, ...
        constexpr int kTurns = kMostSplits / 16;
        float w[kTurns], m = -kInf, sum = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        float2 st[kTurns];
#pragma unroll
        for (int n = 0; n < kTurns; ++n) {
            const int i = n * 16 + (threadIdx.x & 15);
            st[n] = i < a.splits ? *reinterpret_cast<const float2 *>(part_stats(a, i) + row * 2) : make_float2(-kInf, 0.f);
            m = fmaxf(m, st[n].x);
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 16));
#pragma unroll
        for (int n = 0; n < kTurns; ++n) {
            w[n] = part_weight(st[n].x, st[n].y, m);
            sum += st[n].y * w[n];
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 16);
        const float *from = part_sums(a, 0) + row * a.D + (d < a.D ? d : 0);
        const int64_t next = (int64_t)a.Tq * a.Hq * a.D;
#pragma unroll
        for (int n = 0; n < kTurns; ++n)
#pragma unroll 8
            for (int i = n * 16; i < min(a.splits, n * 16 + 16); ++i) {
                const float wt = __shfl(w[n], i & 15, 16);
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(from + i * next), hi = *reinterpret_cast<const f32x4 *>(from + i * next + 4);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    v[u] += lo[u] * wt;
                    v[4 + u] += hi[u] * wt;
                }
            }
        const float inv = sum > 0.f ? 1.0f / sum : sum == 0.f ? 0.f : sum;
        if (d == 0 && a.lse != nullptr) a.lse[(int64_t)head * a.Tq + token] = sum == 0.f ? -kInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= inv;
        if (d < a.D) emit(a, token, head, d, v);
    }
    emit.finish(a);
}

// The amax.  An output made of rounded probabilities is off by up to 2^-8 sum p |v|, so the largest of them only tells which
// rows are likely to hold it: of each wave's rows (32 of k_attn_fwd, 4 of k_attn_join) the largest, of those within 1/64 of
// the largest of all the kTops largest.  These are computed again with probabilities of 32 bits.  What is left is a row
// that its own rounding put below another, of the same wave or by more than 1/64 where values cancel: the amax is off by
// 2^-7 max(sum p |v|) at most, two roundings, and by float32 roundings alone where no two rows are that near.  (Unrounded
// probabilities for every row, in two operands, would take 204 us for 152 at 4 x 2048, and 117 for 80 at 2 x 256 on 8192 keys.)
// kTopParts blocks take a row, and the last of a row to come joins their sums in order.  The sums pass between the blocks by
// accesses of their own to memory that all XCDs see: a fence would write a whole L2 back (17 us at 4 x 2048 with fences, 13
// in two launches).  10.6 .. 11.7 us: three dependent rounds of reads, of the waves' maxima by every block, of keys, of values.
__device__ __forceinline__ void shared_store(float *p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float shared_load(const float *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__global__ __launch_bounds__(kThreads) void k_attn_amax(const Attention a) {
    constexpr int kChunk = kThreads;                                 // keys at a time
    __shared__ uint32_t red[kWaves], value[kThreads];
    __shared__ uint64_t red2[kWaves];
    __shared__ float fred[kWaves], prob[kChunk], q[128], acc[16][128];
    __shared__ int found[kThreads], rows[kTops], all, last;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    // the waves' outputs, four to a load (a.tops % 4 == 0), the first kHeld of a thread kept
    constexpr int kHeld = 8;
    const u32x4 *const tops = reinterpret_cast<const u32x4 *>(a.top);
    const int n = a.tops / 4;
    u32x4 held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = t + i * kThreads < n ? tops[t + i * kThreads] : u32x4{0, 0, 0, 0};
    uint32_t top = 0;
    auto largest = [&](const u32x4 &x) __attribute__((always_inline)) { top = max(max(max(x.x, x.y), max(x.z, x.w)), top); };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) largest(held[i]);
#pragma unroll 8
    for (int i = t + kHeld * kThreads; i < n; i += kThreads) largest(tops[i]);
    top = block_max_u32<kThreads>(top, red);
    if (t == 0) red[0] = top;
    if (t == 0) all = 0;
    __syncthreads();
    top = red[0];
    if (top == 0 || top >= 0x7F800000u) {                            // nothing, or an infinity or NaN, which no rounding made
        if (blockIdx.x == 0 && t == 0) fold_amax_bits(a.amax, top);
        return;
    }
    // the kTops largest candidates, of equal ones the first in the order of the waves: listed as they are found and ranked, or, of
    // more than a list holds, one by one, each the largest behind the one before (not unrolled: the longer code between what
    // runs before and after it made calls that never take it 1.2 us slower)
    const uint32_t least = max(__float_as_uint(__uint_as_float(top) * (1.f - 1.f / 64)), 1u);
    auto find = [&](const u32x4 &x, int i) __attribute__((always_inline)) {
        if (max(max(x.x, x.y), max(x.z, x.w)) < least) return;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (x[u] >= least) {
                const int at = atomicAdd(&all, 1);
                if (at < kThreads) found[at] = 4 * i + u, value[at] = x[u];
            }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) find(held[i], t + i * kThreads);
#pragma unroll 8
    for (int i = t + kHeld * kThreads; i < n; i += kThreads) find(tops[i], i);
    __syncthreads();
    if (all <= kThreads) {
        if (t < all) {
            int before = 0;
            for (int i = 0; i < all; ++i) before += value[i] > value[t] || (value[i] == value[t] && found[i] < found[t]);
            if (before < kTops) rows[before] = a.top_row[found[t]];
        }
    } else {
        uint64_t last_one = ~UINT64_C(0);                            // its value, then the complement of its number
        for (int r = 0; r < kTops; ++r) {
            uint64_t best = 0;
            auto most = [&](const u32x4 &x, int i) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint64_t mine = (uint64_t)x[u] << 32 | (uint32_t)~(4 * i + u);
                    best = mine < last_one && mine > best ? mine : best;
                }
            };
#pragma unroll 1
            for (int i = t; i < n; i += kThreads) most(tops[i], i);
#pragma unroll 1
            for (int o = 32; o >= 1; o >>= 1) {
                const uint64_t other = __shfl_xor((unsigned long long)best, o, 64);
                best = best > other ? best : other;
            }
            if (lane == 0) red2[wave] = best;
            __syncthreads();
            last_one = max(max(red2[0], red2[1]), max(red2[2], red2[3]));
            if (t == 0) rows[r] = a.top_row[~(uint32_t)last_one];
            __syncthreads();
        }
    }
    __syncthreads();
    const int c = blockIdx.x / kTopParts, part = blockIdx.x % kTopParts;
    if (c >= min(all, kTops)) return;
    const int row = rows[c], token = row / a.Hq, head = row - token * a.Hq, kvh = head / a.G;
    int b;
    if (a.offsets_q == nullptr) {
        b = token / (a.Tq / a.B);
    } else {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.offsets_q[mid] <= token) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    const Span sq = span_of(a.offsets_q, b, a.Tq, a.B), sk = span_of(a.offsets_k, b, a.Tk, a.B);
    const Seen see = seen(a, token - (int)sq.begin, sq.len, sk.len);
    const int share = (max(see.hi - see.lo, 0) + kTopParts - 1) / kTopParts;
    const int k_first = see.lo + part * share, k_end = min(see.hi, k_first + share);
    if (t < 128) q[t] = t < a.D ? bf16_lo(a.q.p[(int64_t)token * a.q.ts + head * a.q.hs + t]) : 0.f;
    __syncthreads();
    const float s2 = a.softmax_scale * kLog2e;
    const uint16_t *kp = a.k.p + sk.begin * a.k.ts + kvh * a.k.hs, *vp = a.v.p + sk.begin * a.v.ts + kvh * a.v.hs;
    // o: elements 8 (t % 16) .. + 7 over every 16th key
    const int d8 = (t & 15) * 8;
    float m = -kInf, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = k_first; j < k_end; j += kChunk) {
        float s = -kInf;
        if (j + t < k_end) {
            const uint16_t *row_k = kp + (int64_t)(j + t) * a.k.ts;
            s = 0.f;
            u32x4 x[16];
#pragma unroll
            for (int d = 0; d < 16; ++d) x[d] = d * 8 < a.D ? *reinterpret_cast<const u32x4 *>(row_k + d * 8) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = __builtin_fmaf(q[d * 8 + 2 * i + 1], bf16_hi(x[d][i]), __builtin_fmaf(q[d * 8 + 2 * i], bf16_lo(x[d][i]), s));
        }
        float mx = s;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
        if (lane == 0) fred[wave] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(m, fmaxf(fred[0], fred[1])), fmaxf(fred[2], fred[3])), ref = mn == -kInf ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f((m - ref) * s2), p = __builtin_amdgcn_exp2f((s - ref) * s2);
        m = mn;
        l = l * al + p;
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] *= al;
        prob[t] = p;
        __syncthreads();
        u32x4 x[kChunk / 16];
#pragma unroll
        for (int i = 0; i < kChunk / 16; ++i) {
            const int key = j + (t >> 4) + 16 * i;
            x[i] = key < k_end && d8 < a.D ? *reinterpret_cast<const u32x4 *>(vp + (int64_t)key * a.v.ts + d8) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kChunk / 16; ++i) {
            const float p = prob[(t >> 4) + 16 * i];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                o[2 * u] = __builtin_fmaf(p, bf16_lo(x[i][u]), o[2 * u]);
                o[2 * u + 1] = __builtin_fmaf(p, bf16_hi(x[i][u]), o[2 * u + 1]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) acc[t >> 4][d8 + u] = o[u];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, 64);
    if (lane == 0) fred[wave] = l;
    __syncthreads();
    float *mine_part = a.top_part + (int64_t)blockIdx.x * 130;
    if (t < 128) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += acc[i][t];
        shared_store(mine_part + t, sum);
    }
    if (t == 128) {
        shared_store(mine_part + 128, m);
        shared_store(mine_part + 129, fred[0] + fred[1] + fred[2] + fred[3]);
    }
    FP8DS_WAIT_VM(0);                                                // this wave's stores have arrived
    __syncthreads();
    if (t == 0) last = __hip_atomic_fetch_add(&a.top_done[c], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (last != kTopParts - 1 || t >= 128) return;
    const float *parts = a.top_part + (int64_t)c * kTopParts * 130;
    float pm[kTopParts], pl[kTopParts], pv[kTopParts], sum = 0.f, v = 0.f;
    m = -kInf;
#pragma unroll
    for (int i = 0; i < kTopParts; ++i) pm[i] = shared_load(parts + i * 130 + 128), pl[i] = shared_load(parts + i * 130 + 129), pv[i] = shared_load(parts + i * 130 + t);
#pragma unroll
    for (int i = 0; i < kTopParts; ++i) m = fmaxf(m, pm[i]);
#pragma unroll
    for (int i = 0; i < kTopParts; ++i) {
        const float w = pm[i] == -kInf ? 0.f : __builtin_amdgcn_exp2f((pm[i] - m) * s2);
        sum += w * pl[i];
        v += w * pv[i];
    }
    const uint32_t best = wave_max_u32(sum > 0.f ? __float_as_uint(v / sum) & 0x7FFFFFFFu : 0u);
    if (lane == 0) fold_amax_bits(a.amax, best);
}

// ---------------------------------------------------------------------------------- backward
// Rows of the group's heads, 64 at a time, for 4 waves: row r is token r / G, head r % G of the group.  A lane's loads of a
// tile lie `turn` = 16 or 32 rows apart, its tiles 128 (two sets of waves).  EVEN: G divides `turn`, so that a lane keeps
// its head and its offset, and only the bases move; otherwise the rows are walked, not divided.  (1 x 4096 tokens, 32 heads, 8
// of keys, of 128: backward 559 us, walked 650: the walk's instructions at each load, and k_attn_dkv spills; heads of 64, where
// it does not: 336 and 343.)
template <int DB, bool EVEN> struct GroupLoads {
    using S = Shape<DB>;
    static constexpr int turn = S::rows_a_load * kWaves, n = kStepRows / turn;       // loads of a wave for one tile
    int p, g;                                                        // token after p0 and head of the lane's row of the next tile
    int first, p0, g0;                                               // that tile's first row, its token and head
    uint32_t off_q, off_o;                                           // EVEN: the lane's offsets; else off_q: its byte in a row
    int wave;
    __device__ __forceinline__ GroupLoads(int lane, int wave_, int D, int G, int first_, int q_ts, int q_hs, int o_ts, int o_hs)
        : first(first_), wave(wave_) {
        const int row = wave * S::rows_a_load + lane / S::pieces, r = first + row;
        const int c = (lane % S::pieces) ^ S::swz(row);              // the same piece in all loads
        p0 = first / G, g0 = first - p0 * G;
        p = r / G, g = r - p * G;
        p -= p0;
        off_q = c * 8 < D ? c * 16 : kOutside;                       // past the head: past every bound, whatever is added
        off_o = off_q + (EVEN ? (uint32_t)(__mul24(p, o_ts) + g * o_hs) * 2u : 0u);
        if (EVEN) off_q += (uint32_t)(__mul24(p, q_ts) + g * q_hs) * 2u;
    }
    // Q's and dO's rows; the bases: the sequence's first token at the group's first head
    __device__ __forceinline__ void operator()(const uint16_t *q, int q_ts, int q_hs, const uint16_t *o, int o_ts, int o_hs, int G, int rows,
                                               uint8_t *tq, uint8_t *to) {
        const auto rq = bounded(q + (int64_t)p0 * q_ts, 0x7FFFFFFFu), ro = bounded(o + (int64_t)p0 * o_ts, 0x7FFFFFFFu);
        const int dp = turn / G, dg = turn - dp * G;                 // uniform
        // rows there are, less one, behind the lane's first
        const int left = rows - 1 - first - wave * S::rows_a_load - lane_now() / S::pieces;
        int x = p, y = g;
        off_q = (uint32_t)opaque((int)off_q), off_o = (uint32_t)opaque((int)off_o);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            uint32_t oq = off_q + (uint32_t)(EVEN ? i * dp * q_ts : __mul24(x, q_ts) + y * q_hs) * 2u;
            uint32_t oo = (EVEN ? off_o : off_q) + (uint32_t)(EVEN ? i * dp * o_ts : __mul24(x, o_ts) + y * o_hs) * 2u;
            load_lds(rq, tq + (i * kWaves + wave) * 1024, held(oq, left - i * turn));
            load_lds(ro, to + (i * kWaves + wave) * 1024, held(oo, left - i * turn));
            if constexpr (!EVEN) {
                y += dg, x += dp;
                if (y >= G) y -= G, ++x;
            }
        }
        first += 2 * kStepRows;
        const int tp = 2 * kStepRows / G, tg = 2 * kStepRows - tp * G;
        if constexpr (EVEN) {
            p0 += tp;
        } else {
            // the lane's row and the tile's first, 128 rows on
            g += tg, p += tp;
            if (g >= G) g -= G, ++p;
            g0 += tg;
            const int moved = tp + (g0 >= G);
            if (g0 >= G) g0 -= G;
            p0 += moved, p -= moved;
        }
    }
};

// A block: 128 keys of one key/value head over all query rows of its group that see them.  Two sets of four waves take
// turns at the steps of 64 rows, 32 keys to each wave of a set; the second set's sums are added to the first's at the end.  A
// wave's K and V stay in registers, its dK and dV in accumulators: with heads of 128 that is 192 of the 256 registers that
// two waves a SIMD leave to each, so that what else a step keeps is counted (addresses by exclusive or, operands one or two
// products ahead; a spilled register's reload waits for the loads in flight as well: 400 us with spills, 331 without).  Above
// heads of 96 the walked rows of GroupLoads still spill four (20 bytes): they take two registers more.
// 4 x 2048 tokens, 32 heads, 8 of keys, of 128, causal: 272 .. 323 us, 0.85 .. 1.0 PFLOP/s of its four products; 1 x 8192
// 1103 us, 1.0.  The matrix units are in use for 59 % of the cycles at the clock that the power leaves.
template <int DB, bool EVEN>
__global__ __launch_bounds__(2 * kThreads, 2) void k_attn_dkv(const Attention a) {
    using S = Shape<DB>;
    constexpr int kTile = kStepRows * S::pitch, kAhead = DB < 4 ? 3 : EVEN ? 2 : 1, kRun = 2 * DB;
    __shared__ __align__(1024) uint8_t q0[2 * kTile], q1[2 * kTile], o0[2 * kTile], o1[2 * kTile];     // Q and dO of each set, two turns
    __shared__ __align__(256) float st0[2][2 * kStepRows], st1[2][2 * kStepRows];    // the rows' -lse / scale, then -delta
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6 & 3), set = uniform(threadIdx.x >> 8);
    const int kvh = blockIdx.x % a.Hkv;
    int b, tile;
    if (!find_tile(a.offsets_k, a.Tk, a.B, 1, kRows, blockIdx.x / a.Hkv, b, tile)) return;
    const Span sq = span_of(a.offsets_q, b, a.Tq, a.B), sk = span_of(a.offsets_k, b, a.Tk, a.B);
    if (a.causal) tile = (sk.len + kRows - 1) / kRows - 1 - tile;    // the keys that most rows see first
    const int G = a.G, rows = sq.len * G, j0 = tile * kRows, past = sk.len - sq.len;
    const int jw = j0 + wave * 32, key = jw + (lane & 31);
    bf16x8 kf[S::ks], vf[S::ks];
    load_query<DB>(kf, a.k.p + (sk.begin + key) * a.k.ts + kvh * a.k.hs, a.k.p, key < sk.len, a.D, lane >> 5);
    load_query<DB>(vf, a.v.p + (sk.begin + key) * a.v.ts + kvh * a.v.hs, a.v.p, key < sk.len, a.D, lane >> 5);

    // query rows that see key j: [(j - past) G, (j - past + window) G)
    auto from = [&](int j) { return a.causal ? (int)min(max((int64_t)(j - past) * G, (int64_t)0), (int64_t)rows) : 0; };
    auto until = [&](int j) {
        return a.causal && a.window > 0 ? (int)min(max(((int64_t)j - past + a.window) * G, (int64_t)0), (int64_t)rows) : rows;
    };
    const int lo = from(j0) & ~(kStepRows - 1), hi = until(min(j0 + kRows, sk.len) - 1);
    const int w_first = from(jw), w_end = until(jw + 31);            // rows that any key of the wave sees
    const int all_from = from(jw + 31), all_until = until(jw);       // rows that every key of the wave sees

    GroupLoads<DB, EVEN> loads(lane, wave, a.D, G, lo + set * kStepRows, (int)a.q.ts, (int)a.q.hs, (int)a.dout.ts, (int)a.dout.hs);
    const uint16_t *qp = a.q.p + sq.begin * a.q.ts + (int64_t)kvh * G * a.q.hs;
    const uint16_t *dp = a.dout.p + sq.begin * a.dout.ts + (int64_t)kvh * G * a.dout.hs;
    const int64_t all = (int64_t)a.Tq * a.Hq, row0 = ((int64_t)kvh * a.Tq + sq.begin) * G;
    const auto rs_stats = bounded(a.part, (uint32_t)(all * 8));
    auto load = [&](int r, uint8_t *tq, uint8_t *to, float (*ts)[2 * kStepRows]) __attribute__((always_inline)) {
        loads(qp, (int)a.q.ts, (int)a.q.hs, dp, (int)a.dout.ts, (int)a.dout.hs, G, rows, tq + set * kTile, to + set * kTile);
        if (wave < 2)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_stats, (__attribute__((address_space(3))) void *)(ts[set] + wave * kStepRows), 4,
                                                     held((uint32_t)(row0 + r + lane_now() + wave * all) * 4u, rows - 1 - r - lane_now()), 0, 0, 0);
    };
    Walker<DB> rd(lane);
    const float s2 = uniform_value(a.softmax_scale * kLog2e);
    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.f;
    // r0: the first set's rows; the second's lie 64 behind
    if (lo + set * kStepRows < hi) load(lo + set * kStepRows, q0, o0, st0);
    auto turn = [&](int r0, const uint8_t *step_q, const uint8_t *step_o, const float (*step_st)[2 * kStepRows], uint8_t *next_q,
                    uint8_t *next_o, float (*next_st)[2 * kStepRows]) __attribute__((always_inline)) {
        FP8DS_WAIT_ALL();
        FP8DS_BARRIER();
        r0 += set * kStepRows;
        if (r0 + 2 * kStepRows < hi) load(r0 + 2 * kStepRows, next_q, next_o, next_st);
#pragma unroll
        for (int part = 0; part < kStepRows / 32; ++part) {
            const int r = r0 + part * 32;
            if (r >= w_end || r + 32 <= w_first) continue;
            const uint8_t *tq = step_q + set * kTile + part * 32 * S::pitch, *td = step_o + set * kTile + part * 32 * S::pitch;
            const float *st = step_st[set] + part * 32 + 4 * (lane >> 5);
            // Four runs of products, kRun each: s and p (dP) along the head, then the sums of dV and dK over the rows.  Their
            // operands are read kAhead products ahead, and each product takes its share of the other instructions with
            // it: the exponentials go beside p, the slopes beside dV.
            f32x16 s, p;
            bf16x8 f[kAhead];
            auto read = [&](int n) __attribute__((always_inline)) {
                if (n < kRun) return read_row(tq + rd.row(n));
                if (n < 2 * kRun) return read_row(td + rd.row(n - kRun));
                const int x = (n % kRun) / DB, d = n % DB;
                return rd.tr((n < 3 * kRun ? td : tq) + x * 16 * S::pitch, d);
            };
            auto start = [&](f32x16 &v, const float *from, int i) __attribute__((always_inline)) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(from + 8 * i);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[4 * i + u] = x[u];
            };
            rd.fresh();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; ++i) start(s, st, i);
#pragma unroll
            for (int n = 0; n < kAhead; ++n) f[n] = read(n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                const bf16x8 now = f[n % kAhead];
                f[n % kAhead] = read(n + kAhead);
                s = mfma(now, kf[n], s);
                if (n >= kRun - 4) start(p, st + kStepRows, n - (kRun - 4));
                __builtin_amdgcn_sched_barrier(0);
            }
            if (r < all_from || r + 32 > all_until) {
                const int l = lane_now(), k = jw + (l & 31), mine_from = from(k), mine_until = until(k);
                const float none = __uint_as_float((uint32_t)opaque((int)0xFF800000u));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = r + (i >> 2) * 8 + 4 * (l >> 5) + (i & 3);
                    s[i] = at >= mine_from && at < mine_until ? s[i] : none;
                }
            }
            rd.fresh();
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 pf[2], sf[2];
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                const bf16x8 now = f[(n + kRun) % kAhead];
                f[(n + kRun) % kAhead] = read(n + kRun + kAhead);
                p = mfma(now, vf[n], p);
#pragma unroll
                for (int i = n * 16 / kRun; i < (n + 1) * 16 / kRun; ++i) s[i] = __builtin_amdgcn_exp2f(s[i] * s2);
                if (n == kRun - 1) pf[0] = pack8(s, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            rd.fresh();
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                const bf16x8 now = f[(n + 2 * kRun) % kAhead];
                f[(n + 2 * kRun) % kAhead] = read(n + 2 * kRun + kAhead);
                dv[n % DB] = mfma(now, pf[n / DB], dv[n % DB]);
                if (n == DB - 1) pf[1] = pack8(s, 1);
                // the last of p's products has to be through before its values are used
                if (n >= 2 && n < 6 && kRun >= 8) {
#pragma unroll
                    for (int i = (n - 2) * 4; i < (n - 1) * 4; ++i) p[i] *= s[i];
                }
                if (kRun < 8 && n >= 1) {
#pragma unroll
                    for (int i = (n - 1) * 16 / (kRun - 1); i < n * 16 / (kRun - 1); ++i) p[i] *= s[i];
                }
                if (n == kRun - 2) sf[0] = pack8(p, 0);
                if (n == kRun - 1) sf[1] = pack8(p, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            rd.fresh();
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                const bf16x8 now = f[(n + 3 * kRun) % kAhead];
                if (n + kAhead < kRun) f[(n + 3 * kRun) % kAhead] = read(n + 3 * kRun + kAhead);
                dk[n % DB] = mfma(now, sf[n / DB], dk[n % DB]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    for (int r = lo; r < hi; r += 4 * kStepRows) {
        turn(r, q0, o0, st0, q1, o1, st1);
        if (r + 2 * kStepRows >= hi) break;
        turn(r + 2 * kStepRows, q1, o1, st1, q0, o0, st0);
    }
    // the second set's sums
    FP8DS_WAIT_ALL();
    __syncthreads();
    static_assert(sizeof(q0) >= 2 * DB * 16 * 64 * 4, "an array holds a wave's sums");
    float *mine = reinterpret_cast<float *>(wave == 0 ? q0 : wave == 1 ? q1 : wave == 2 ? o0 : o1) + lane_now();
    if (set == 1) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                mine[(d * 16 + i) * 64] = dk[d][i];
                mine[((DB + d) * 16 + i) * 64] = dv[d][i];
            }
    }
    __syncthreads();
    if (set == 1) return;
    const int l = lane_now(), out = jw + (l & 31);
    const bool there = out < sk.len;
    const int64_t token = sk.begin + out;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            dk[d][i] += mine[(d * 16 + i) * 64];
            dv[d][i] += mine[((DB + d) * 16 + i) * 64];
        }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float x[8], y[8];
            consecutive8(dk[d], s, x);
            consecutive8(dv[d], s, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= a.softmax_scale;
            const int at = d * 32 + s * 16 + (l >> 5) * 8;
            if (there && at < a.D) {
                *reinterpret_cast<u32x4 *>(a.dk.p + token * a.dk.ts + kvh * a.dk.hs + at) = to_bf16(x);
                *reinterpret_cast<u32x4 *>(a.dv.p + token * a.dv.ts + kvh * a.dv.hs + at) = to_bf16(y);
            }
        }
}

// A block: 128 query rows, 32 to each wave, over the keys that they see, as the forward.  It also leaves what the keys'
// gradients need of each row in the workspace, in the order [key/value head, token, head of the group].
// <dout, out> of the rounded output is off by e, up to 2^-8 of its terms.  The slopes P (dP - <dout, out>) of a row then have
// the sum -e instead of 0: that goes into what the keys' gradients take, and dQ lacks -e sum P k.  Heads of up to 96 keep
// sum P k beside dQ, one more product of dQ's operands: 4 x 2048 of 64 292 us for 272 with both kernels, 1 x 8192 of 96 (16 heads,
// 4 of keys; two registers spill, nine where operands are read three products ahead, in the same time) 960 for 904.
// Above 96 there are no registers for it: blocks of up to 256 keys, where e counts most, go over their keys twice, for the
// sum first (8 x 256 of 128 65 us for 56; window 128 at 4 x 2048 186 for 168), others leave e in dQ.  Error of all gradients
// against 64 bits, their own rounding being 0.0017: with e 0.0025 (2048 keys) .. 0.0028 (window 5), without it 0.0023 .. 0.0024.
// 4 x 2048 tokens, 32 heads, 8 of keys, of 128, causal: 215 .. 251 us, 0.8 .. 0.95 PFLOP/s of its three products; 1 x 8192
// 750 .. 791 us, 1.0.
template <int DB>
__global__ __launch_bounds__(kThreads, 2) void k_attn_dq(const Attention a) {
    using S = Shape<DB>;
    constexpr int kTile = kKeys * S::pitch, kRun = 2 * DB, kAhead = DB == 3 ? 2 : 3;
    constexpr bool kWithKeys = DB <= 3;          // sum P k is kept
    constexpr int kTwice = 256;                  // keys of a block that goes over them twice instead
    __shared__ __align__(1024) uint8_t k0[kTile], k1[kTile], v0[kTile], v1[kTile];      // as in the forward
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int kvh = blockIdx.x % a.Hkv;
    int b, tile;
    if (!find_tile(a.offsets_q, a.Tq, a.B, a.G, kRows, blockIdx.x / a.Hkv, b, tile)) return;
    const Span sq = span_of(a.offsets_q, b, a.Tq, a.B), sk = span_of(a.offsets_k, b, a.Tk, a.B);
    const int rows = sq.len * a.G, r0 = tile * kRows, last = min(r0 + kRows, rows) - 1;
    const int r0w = r0 + wave * 32, r = r0w + (lane & 31);
    const int pos = r / a.G, head = kvh * a.G + r - pos * a.G;
    const bool there = r < rows;
    const int64_t token = sq.begin + pos;
    bf16x8 qf[S::ks], df[S::ks];
    load_query<DB>(qf, a.q.p + token * a.q.ts + head * a.q.hs, a.q.p, there, a.D, lane >> 5);
    load_query<DB>(df, a.dout.p + token * a.dout.ts + head * a.dout.hs, a.dout.p, there, a.D, lane >> 5);
    const float s2 = uniform_value(a.softmax_scale * kLog2e);
    // -lse / scale, -inf where the row has no probabilities to compute again, and -<dout, out> of the row
    float low = -kInf, delta = 0.f, slope_sum = 0.f;
    {
        bf16x8 of[S::ks];
        load_query<DB>(of, a.out.p + token * a.out.ts + head * a.out.hs, a.out.p, there, a.D, lane >> 5);
#pragma unroll
        for (int k = 0; k < S::ks; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) delta -= (float)df[k][i] * (float)of[k][i];
        delta = both_halves_sum(delta);
    }
    if (there) {
        const float lse = a.lse[(int64_t)head * a.Tq + token];
        low = fabsf(lse) >= kFarLse ? -kInf : -lse / a.softmax_scale;
        if (lane < 32) a.part[((int64_t)kvh * a.Tq + sq.begin) * a.G + r] = low;
        low *= s2;
    }
    const int lo = seen(a, r0 / a.G, sq.len, sk.len).lo & ~(kKeys - 1), hi = seen(a, last / a.G, sq.len, sk.len).hi;
    const Seen first = seen(a, min(r0w, last) / a.G, sq.len, sk.len), end = seen(a, min(r0w + 31, last) / a.G, sq.len, sk.len);
    const Seen see = seen(a, pos, sq.len, sk.len);         // rows past the last compute what is never written
    const RowLoads<DB, kKeys, kWaves> loads_k(lane, wave, a.D, a.k.ts), loads_v(lane, wave, a.D, a.v.ts);
    const uint16_t *kp = a.k.p + sk.begin * a.k.ts + kvh * a.k.hs, *vp = a.v.p + sk.begin * a.v.ts + kvh * a.v.hs;
    Walker<DB> rd(lane);
    auto load = [&](int j, uint8_t *tk, uint8_t *tv) __attribute__((always_inline)) {
        if (j >= hi) return;
        loads_k(kp + (int64_t)j * a.k.ts, a.k.ts, sk.len - j, tk);
        loads_v(vp + (int64_t)j * a.v.ts, a.v.ts, sk.len - j, tv);
    };
    auto hide = [&](f32x16 &s, int key0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int key = key0 + 4 * (lane >> 5) + (i >> 2) * 8 + (i & 3);
            s[i] = key >= see.lo && key < see.hi ? s[i] : -kInf;
        }
    };
    load(lo, k0, v0);
    if (!kWithKeys && hi - lo <= kTwice) {       // the sum of the slopes first
        auto sums = [&](int j, const uint8_t *tk, const uint8_t *tv, uint8_t *next_k, uint8_t *next_v) __attribute__((always_inline)) {
            FP8DS_WAIT_ALL();
            FP8DS_BARRIER();
            load(j + kKeys, next_k, next_v);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                f32x16 s, p;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.f, p[i] = delta;
#pragma unroll
                for (int k = 0; k < kRun; ++k) {
                    s = mfma(read_row(tk + kb * 32 * S::pitch + rd.row(k)), qf[k], s);
                    p = mfma(read_row(tv + kb * 32 * S::pitch + rd.row(k)), df[k], p);
                }
                hide(s, j + kb * 32);
#pragma unroll
                for (int i = 0; i < 16; ++i) slope_sum += __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], s2, low)) * p[i];
            }
        };
        for (int j = lo; j < hi; j += 2 * kKeys) {
            sums(j, k0, v0, k1, v1);
            if (j + kKeys >= hi) break;
            sums(j + kKeys, k1, v1, k0, v0);
        }
        delta -= both_halves_sum(slope_sum);
        slope_sum = 0.f;
        FP8DS_WAIT_ALL();
        FP8DS_BARRIER();                                             // every wave has read the tiles
        load(lo, k0, v0);
    }
    f32x16 dq[DB], pk[kWithKeys ? DB : 1];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[d][i] = 0.f;
#pragma unroll
    for (int d = 0; d < (kWithKeys ? DB : 1); ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[d][i] = 0.f;
    auto turn = [&](int j, const uint8_t *tk, const uint8_t *tv, uint8_t *next_k, uint8_t *next_v) __attribute__((always_inline)) {
        FP8DS_WAIT_ALL();
        FP8DS_BARRIER();
        const int next = j + kKeys;
        load(next, next_k, next_v);
        if (j >= end.hi || next <= first.lo) return;
        const bool masked = next > first.hi || j < end.lo;
        // Six runs of products, kRun each: scores and dP of 32 keys, of the next 32, and the sums over either.  As in the keys'
        // gradients: operands kAhead products ahead, the exponentials beside dP, the slopes beside the run after it.
        f32x16 s[2], p[2];
        bf16x8 f[kAhead], sf[2][2], pf[2][2];
        auto read = [&](int n) __attribute__((always_inline)) {
            const int run = n / kRun, i = n % kRun;
            if (run < 4) return read_row((run & 1 ? tv : tk) + (run >> 1) * 32 * S::pitch + rd.row(i));
            return rd.tr(tk + ((run - 4) * 32 + i / DB * 16) * S::pitch, i % DB);
        };
        auto step = [&](int n) __attribute__((always_inline)) {      // the operand of product n; the one kAhead on is read
            const bf16x8 now = f[n % kAhead];
            if (n + kAhead < 6 * kRun) f[n % kAhead] = read(n + kAhead);
            return now;
        };
        auto slopes = [&](int kb, int n) __attribute__((always_inline)) {     // from the third product on: dP's last is through
            if (n >= 2) {
#pragma unroll
                for (int i = (n - 2) * 16 / (kRun - 2); i < (n - 1) * 16 / (kRun - 2); ++i) {
                    p[kb][i] *= s[kb][i];
                    slope_sum += p[kb][i];
                }
            }
            if (n == kRun - 1) sf[kb][0] = pack8(p[kb], 0), sf[kb][1] = pack8(p[kb], 1);
            if (kWithKeys && n == kRun - 1) pf[kb][0] = pack8(s[kb], 0), pf[kb][1] = pack8(s[kb], 1);
        };
        rd.fresh();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[kb][i] = 0.f;
                p[kb][i] = delta;
            }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) f[n] = read(n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                s[kb] = mfma(step(2 * kb * kRun + n), qf[n], s[kb]);
                if (kb == 1) slopes(0, n);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (masked) hide(s[kb], j + kb * 32);
            rd.fresh();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                p[kb] = mfma(step((2 * kb + 1) * kRun + n), df[n], p[kb]);
#pragma unroll
                for (int i = n * 16 / kRun; i < (n + 1) * 16 / kRun; ++i) s[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], s2, low));
                __builtin_amdgcn_sched_barrier(0);
            }
            rd.fresh();
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int n = 0; n < kRun; ++n) {
                const bf16x8 now = step((4 + kb) * kRun + n);
                dq[n % DB] = mfma(now, sf[kb][n / DB], dq[n % DB]);
                if constexpr (kWithKeys) pk[n % DB] = mfma(now, pf[kb][n / DB], pk[n % DB]);
                if (kb == 0) slopes(1, n);
                __builtin_amdgcn_sched_barrier(0);
            }
            rd.fresh();
        }
    };
    for (int j = lo; j < hi; j += 2 * kKeys) {
        turn(j, k0, v0, k1, v1);
        if (j + kKeys >= hi) break;
        turn(j + kKeys, k1, v1, k0, v0);
    }
    slope_sum = both_halves_sum(slope_sum);
    if (there && lane < 32) a.part[(int64_t)a.Tq * a.Hq + ((int64_t)kvh * a.Tq + sq.begin) * a.G + r] = delta - slope_sum;
    if constexpr (kWithKeys) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[d][i] = __builtin_fmaf(-slope_sum, pk[d][i], dq[d][i]);
    }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float x[8];
            consecutive8(dq[d], s, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= a.softmax_scale;
            const int at = d * 32 + s * 16 + (lane >> 5) * 8;
            if (there && at < a.D) *reinterpret_cast<u32x4 *>(a.dq.p + token * a.dq.ts + head * a.dq.hs + at) = to_bf16(x);
        }
}

// ---------------------------------------------------------------------------------- launches
namespace {
constexpr int kCUs = 256;
constexpr int64_t kMostBlocks = (INT64_C(1) << 32) / (2 * kThreads) - 1;

int64_t most_tiles(int64_t T, int64_t B, int64_t group, int64_t height, bool ragged) {
    return ragged ? T * group / height + B : B * ((T / B * group + height - 1) / height);
}
struct Plan {
    bool few;
    int64_t blocks, splits;
};
// Few query rows to a sequence (32 at the mean: one block of 32): the waves share the keys.  8 key heads, 4 rows to each of 16
// sequences of 4096 keys: 46.5 us and 48 with blocks of 128 rows, 32 rows to each of 4 of 8192 keys 29.7 and 32.2.  Up to 64
// rows, two blocks that read the same keys, as long as these blocks are one round (64 rows to each of 16 of 4096 keys 50
// and 54, to one of 8192 19 and 21.5, to one of 2882 15.6 and 19.5; to each of 64 of 1024, four rounds, 88 and 49; 128 rows to
// each of 16 53 and 39).
// Fewer blocks than the GPU holds at a time (one block of few rows to a CU, two of the others): the keys are split, into as
// many parts as bring the blocks nearest to that.  16 sequences of up to 4096 keys, 8 key heads, 144 blocks: 44.4 us whole,
// 37.7 in two parts, 40.5 in three, 39.9 in four, 49 in eight, each over the same cache time after time, of which part stays
// on the chip (over others in between 46 in two parts).  Parts no shorter than 512 keys of blocks of 128 rows (one sequence of
// 2048 keys, 256 tokens: 28 us, with 256 keys 31.6, with 1024 30.6), of 256 of the others: of the keys that there are at the
// mean.  What a window leaves of them is not counted, so its parts are shorter and some empty (one token on 8192 keys, window
// 1024: 32 parts of which 8 have keys, 18.5 us), nor that one sequence may be longer than the others.  The places are those
// of heads of 128, as are nearly all figures; of 64 a CU holds three blocks of 128 rows by registers, two of few rows by LDS.
Plan fwd_plan(int64_t Tq, int64_t Tk, int64_t B, int64_t Hkv, int64_t G, bool ragged) {
    Plan p;
    p.few = Tq * G <= kFewRows * B || (Tq * G <= 2 * kFewRows * B && most_tiles(Tq, B, G, kFewRows, ragged) * Hkv <= kCUs);
    const int64_t tiles = most_tiles(Tq, B, G, p.few ? kFewRows : kRows, ragged) * Hkv;
    const int64_t slots = p.few ? kCUs : 2 * kCUs, shortest = p.few ? 256 : 512;
    int64_t s = tiles > 0 ? (slots + tiles / 2) / tiles : 1;
    const int64_t most = Tk / B / shortest;
    if (s > most) s = most;
    p.splits = s < 1 ? 1 : s > kMostSplits ? kMostSplits : s;
    p.blocks = tiles * p.splits;
    return p;
}
}  // namespace

bool attention_fits(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, bool ragged) {
    if (B == 0) return true;
    return fwd_plan(Tq, Tk, B, Hkv, Hq / Hkv, ragged).blocks <= kMostBlocks && most_tiles(Tq, B, Hq / Hkv, kRows, ragged) * Hkv <= kMostBlocks &&
           most_tiles(Tk, B, 1, kRows, ragged) * Hkv <= kMostBlocks;
}

// The forward's workspace: the splits' sums and stats, then what the amax takes.
struct Room {
    size_t sums, stats, top, top_row, top_part, top_done, bytes;
    int64_t tops;
    Room(const Plan &p, int64_t Tq, int64_t Hq, int64_t D, bool amax) {
        const auto up = [](size_t n) { return (n + 15) & ~(size_t)15; };
        const size_t rows = (size_t)(Tq * Hq), split = p.splits > 1 ? (size_t)p.splits : 0;
        tops = p.few || !amax ? 0 : (p.splits > 1 ? (int64_t)(rows + 15) / 16 : p.blocks) * kWaves;
        sums = 0;
        stats = split * rows * D * 4;                                // D % 8 == 0
        top = stats + up(split * rows * 8);
        top_row = top + up((size_t)tops * 4);
        top_part = top_row + up((size_t)tops * 4);
        top_done = top_part + (tops > 0 ? kTops * kTopParts * 130 * 4 : 0);
        bytes = top_done + (tops > 0 ? kTops * 4 : 0);
    }
};

size_t attention_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, bool ragged, bool amax) {
    return Room(fwd_plan(Tq, Tk, B, Hkv, Hq / Hkv, ragged), Tq, Hq, D, amax).bytes;
}
size_t attention_bwd_workspace_bytes(int64_t Tq, int64_t Hq) { return (size_t)(Tq * Hq * 8); }

#define FP8DS_BY_HEAD(KERNEL, BLOCKS, THREADS)                                                                \
    do {                                                                                               \
        const dim3 grid((unsigned)(BLOCKS));                                                           \
        if (a.D <= 64) KERNEL<2><<<grid, THREADS, 0, st>>>(a);                                        \
        else if (a.D <= 96) KERNEL<3><<<grid, THREADS, 0, st>>>(a);                                   \
        else KERNEL<4><<<grid, THREADS, 0, st>>>(a);                                                  \
    } while (0)

hipError_t launch_attention_fwd(Attention a, void *ws, hipStream_t st) {
    const Plan p = fwd_plan(a.Tq, a.Tk, a.B, a.Hkv, a.G, a.offsets_q != nullptr);
    const Room room(p, a.Tq, a.Hq, a.D, a.out8 != nullptr && a.amax != nullptr);
    uint8_t *const base = static_cast<uint8_t *>(ws);
    a.splits = (int)p.splits;
    a.part = reinterpret_cast<float *>(base);
    if (room.tops > 0) {
        a.tops = (int)room.tops;
        a.top = reinterpret_cast<uint32_t *>(base + room.top);
        a.top_row = reinterpret_cast<int32_t *>(base + room.top_row);
        a.top_part = reinterpret_cast<float *>(base + room.top_part);
        a.top_done = reinterpret_cast<int32_t *>(base + room.top_done);
    }
    if (p.few) FP8DS_BY_HEAD(k_attn_fwd_few, p.blocks, kThreads);
    else FP8DS_BY_HEAD(k_attn_fwd, p.blocks, kThreads);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.splits > 1) {
        k_attn_join<<<(unsigned)(((int64_t)a.Tq * a.Hq + 15) / 16), kThreads, 0, st>>>(a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (a.top != nullptr) {
        k_attn_amax<<<kTops * kTopParts, kThreads, 0, st>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_attention_bwd(Attention a, void *ws, hipStream_t st) {
    const bool ragged = a.offsets_q != nullptr;
    a.part = static_cast<float *>(ws);
    if (a.Tq > 0) FP8DS_BY_HEAD(k_attn_dq, most_tiles(a.Tq, a.B, a.G, kRows, ragged) * a.Hkv, kThreads);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (a.Tk > 0) {
        const dim3 grid((unsigned)(most_tiles(a.Tk, a.B, 1, kRows, ragged) * a.Hkv));
        const bool even = (a.D <= 64 ? GroupLoads<2, true>::turn : GroupLoads<4, true>::turn) % a.G == 0;
        if (a.D <= 64) even ? k_attn_dkv<2, true><<<grid, 2 * kThreads, 0, st>>>(a) : k_attn_dkv<2, false><<<grid, 2 * kThreads, 0, st>>>(a);
        else if (a.D <= 96) even ? k_attn_dkv<3, true><<<grid, 2 * kThreads, 0, st>>>(a) : k_attn_dkv<3, false><<<grid, 2 * kThreads, 0, st>>>(a);
        else even ? k_attn_dkv<4, true><<<grid, 2 * kThreads, 0, st>>>(a) : k_attn_dkv<4, false><<<grid, 2 * kThreads, 0, st>>>(a);
    }
    return hipGetLastError();
}

}  // namespace fp8ds
