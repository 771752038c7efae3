// router.hip -- the choice of experts from the router's logits, with the balance loss, and its gradient, on gfx950.
//
// One read of the logits: the first choice is the row's maximum, which the softmax is taken about; every further choice is a
// maximum over what is left.  A block adds its rows' probabilities and choices up, and a second launch joins the blocks
// in order.  Bound by latency up to some thousand rows (8192 of 64 experts, 4 choices: 8.8 us, a launch of 5.3 and one of
// 4.0), then by the instructions of the choices: 32768 rows of 256 experts, 8 choices, 22 us for 19 MB.
// Backward: with g_j = dweights_j, c_e = dloss E counts_e / (choices * rows), w the weights
//   dp = c + g at the choices (normalised: (g - <w, g>) / sum of p),  dlogits = p (dp - <p, dp>)
#include <climits>

#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMostBlocks = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Reductions over the wave, the same in every lane.  The steps go 1, 2, 4, 8 lanes inside rows of 16, then from row to row;
// lanes that a step does not reach take the neutral 0.
#define FP8DS_DPP(v, ctrl, rows) __builtin_amdgcn_update_dpp(0, (int)(v), ctrl, rows, 0xf, false)
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x111, 0xf));
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x112, 0xf));
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x114, 0xf));
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x118, 0xf));
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x142, 0xa));
    v = max(v, (uint32_t)FP8DS_DPP(v, 0x143, 0xc));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x111, 0xf));
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x112, 0xf));
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x114, 0xf));
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x118, 0xf));
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x142, 0xa));
    v += __uint_as_float((uint32_t)FP8DS_DPP(__float_as_uint(v), 0x143, 0xc));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Keys that order as the logits do, as whole numbers, so that a step of a maximum is one instruction.  0: never chosen (-inf
// or NaN).  A bfloat16 logit leaves room for its expert's complement: the key then finds the expert too.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);     // -0 becomes 0: they are equal
    return x > -kInf ? u ^ (uint32_t)(((int)u >> 31) | (int)0x80000000) : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key ^ ((int)key < 0 ? 0x80000000u : 0xFFFFFFFFu)); }

template <bool BF16> __device__ __forceinline__ float logit(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else return static_cast<const float *>(p)[i];
}

// `both`: the experts' counts times their summed probabilities.
__device__ __forceinline__ float loss_of(int E, float both, int all, int live) { return (float)E * (both / (float)max(all, 1)) / (float)max(live, 1); }

// The balance loss from the experts' counts and summed probabilities (in LDS); one block.
__device__ __forceinline__ void finish_loss(const Route &a, const float *sums, const int *counts, float *red) {
    float both = 0.f;
    int all = 0;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        both += (float)counts[e] * sums[e];
        all += counts[e];
    }
    both = wave_sum(both);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o, 64);
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = both;
        reinterpret_cast<int *>(red)[kWaves + (threadIdx.x >> 6)] = all;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    both = 0.f;
    all = 0;
    for (int w = 0; w < kWaves; ++w) {
        both += red[w];
        all += reinterpret_cast<const int *>(red)[kWaves + w];
    }
    *a.loss = loss_of(a.E, both, all, counts[a.E]);
}

// A block's sums (of its waves, added in order) and counts (cnt[N]: rows): its part, or, of the only block, all there is.
template <int N> __device__ __forceinline__ void block_parts(const Route &a, float (*sums)[N], int *cnt, float *red) {
    const int nb = gridDim.x;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += sums[w][e];
        if (nb == 1) {
            a.prob_sum[e] = s;
            a.counts[e] = cnt[e];
            sums[0][e] = s;
        } else {
            a.part[(int64_t)blockIdx.x * a.E + e] = u32x2{__float_as_uint(s), (uint32_t)cnt[e]};
        }
    }
    if (nb > 1) {
        if (threadIdx.x == 0) a.part_live[blockIdx.x] = cnt[N];
        return;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.counts[a.E] = cnt[N];
        cnt[a.E] = cnt[N];
    }
    __syncthreads();
    finish_loss(a, sums[0], cnt, red);
}

}  // namespace

// A wave takes a row, lane l its experts l, l + 64, ...  Bound by the instructions of the choices: each takes a maximum over
// the wave, the expert that holds it, and its removal.
template <bool BF16, int V>
__global__ __launch_bounds__(kThreads) void k_moe_route(const Route a) {
    __shared__ int cnt[64 * V + 1];
    __shared__ float sums[kWaves][64 * V];
    __shared__ float red[2 * kWaves];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    for (int e = threadIdx.x; e <= 64 * V; e += kThreads) cnt[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    int live = 0;
    const int64_t step = (int64_t)gridDim.x * kWaves;
    float next[V];
    auto load = [&](int64_t t) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < V; ++v) next[v] = v * 64 + lane < a.E && t < a.T ? logit<BF16>(a.logits, t * a.ld + v * 64 + lane) : -kInf;
    };
    load((int64_t)blockIdx.x * kWaves + wave);
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += step) {
        float x[V];
        uint32_t key[V];
        bool nan = false;
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = next[v];
        load(t + step);                                              // the wave's next row comes in beside this one's choices
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            nan |= x[v] != x[v];
            key[v] = key_of(x[v]);
            if (BF16) key[v] = key[v] != 0 ? (key[v] & 0xFFFF0000u) | (uint32_t)(0xFFFF - e) : 0u;
        }
        const bool any_nan = __any(nan);
        // Choice j goes to lane j % 64, 64 at a time; the largest logit is the first.
        float mx = 0.f, inv = 0.f, total = 0.f, held = 0.f;
        int held_e = -1;
        bool dead = false;
        float chosen = 0.f;                                          // sum of the chosen ones' exp(x - mx)
        for (int j = 0; j < a.top; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = max(best, key[v]);
            best = wave_max(best);
            int e = -1;
            if (BF16) {
                if (best != 0) e = 0xFFFF - (int)(best & 0xFFFFu);
            } else {
#pragma unroll
                for (int v = V - 1; v >= 0; --v) {
                    const uint64_t at = __ballot(key[v] == best);
                    e = at != 0 ? v * 64 + __ffsll((unsigned long long)at) - 1 : e;
                }
                e = best != 0 ? e : -1;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = e == v * 64 + lane ? 0u : key[v];
            // (of a negative bfloat16 the key's low bits were ones)
            const float value = logit_of(!BF16 ? best : (int)best < 0 ? best & 0xFFFF0000u : best | 0xFFFFu);
            if (j == 0) {
                dead = best == 0 && !any_nan;
                mx = best != 0 ? value : -kInf;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = dead || v * 64 + lane >= a.E ? 0.f : __builtin_amdgcn_exp2f((x[v] - mx) * kLog2e);
                    total += x[v];
                }
                total = wave_sum(total);
                inv = dead ? 0.f : 1.0f / total;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += x[v] * inv;
                live += !dead;
            }
            held = lane == (j & 63) ? value : held;
            held_e = lane == (j & 63) ? e : held_e;
            if ((j & 63) == 63 || j == a.top - 1) {
                const int j0 = j & ~63;
                float w = 0.f;
                if (j0 + lane <= j) {
                    if (held_e >= 0) {
                        w = __builtin_amdgcn_exp2f((held - mx) * kLog2e);
                        if (mx != mx || total != total) w = total;   // a NaN in the row
                        atomicAdd(&cnt[held_e], 1);
                    }
                    a.experts[t * a.top + j0 + lane] = held_e;
                }
                chosen += wave_sum(w);
                // normalised weights need all choices' sum: those of earlier turns are gone over again
                const float each = a.normalise ? (chosen > 0.f || chosen != chosen ? 1.0f / chosen : 0.f) : inv;
                const bool last = j == a.top - 1;
                if (j0 + lane <= j) a.weights[t * a.top + j0 + lane] = a.normalise && !last ? w : w * each;
                if (a.normalise && last)
                    for (int i = lane; i < j0; i += 64) a.weights[t * a.top + i] *= each;
            }
        }
        if (lane == 0) a.lse[t] = dead ? -kInf : mx + __builtin_amdgcn_logf(total) * kLn2;
    }
    if (lane == 0 && live != 0) atomicAdd(&cnt[64 * V], live);
#pragma unroll
    for (int v = 0; v < V; ++v) sums[wave][v * 64 + lane] = acc[v];
    __syncthreads();
    block_parts<64 * V>(a, sums, cnt, red);
}

// Up to 256 experts: a wave takes four rows, 16 lanes to a row, lane l of them the experts l, l + 16, ...  No step leaves
// the 16 lanes, so that a choice costs a row a quarter of the wave's instructions.  32768 rows of 256 experts, 8 choices:
// 25.4 us, with a wave to a row 35.2; of 8192 rows, for half of the waves, 15.6 and 15.8; of 1024 14.3 and 11.4.  The rows go
// round the blocks: in runs of 64 to a block three blocks of four had none (8192 rows 18.7, 128 17.2 for 13.2).  More experts do
// not fit a lane's registers: V logits, keys, sums and the next row's logits.
template <int CTRL> __device__ __forceinline__ uint32_t max16(uint32_t v) { return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true)); }
__device__ __forceinline__ uint32_t row_max(uint32_t v) { return max16<0x121>(max16<0x122>(max16<0x124>(max16<0x128>(v)))); }      // row_ror 8, 4, 2, 1
template <int CTRL> __device__ __forceinline__ float add16(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float v) { return add16<0x121>(add16<0x122>(add16<0x124>(add16<0x128>(v)))); }

template <bool BF16, int V>
__global__ __launch_bounds__(kThreads) void k_moe_route_rows(const Route a) {
    __shared__ int cnt[16 * V + 1];
    __shared__ float sums[kWaves][16 * V];
    __shared__ float red[2 * kWaves];
    const int lane = threadIdx.x & 63, l = lane & 15, group = lane >> 4, wave = uniform(threadIdx.x >> 6);
    for (int e = threadIdx.x; e <= 16 * V; e += kThreads) cnt[e] = 0;
    __syncthreads();
    float acc[V], next[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    int live = 0;
    const int64_t step = (int64_t)gridDim.x * kWaves * 4;
    auto load = [&](int64_t t) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < V; ++v) next[v] = v * 16 + l < a.E && t < a.T ? logit<BF16>(a.logits, t * a.ld + v * 16 + l) : -kInf;
    };
    const int64_t first = ((int64_t)wave * gridDim.x + blockIdx.x) * 4;      // every block has rows before one has more
    load(first + group);
    for (int64_t t0 = first; t0 < a.T; t0 += step) {
        const int64_t t = t0 + group;
        const bool row = t < a.T;
        float x[V];
        uint32_t key[V];
        bool nan = false;
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = next[v];
        load(t + step);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nan |= x[v] != x[v];
            key[v] = key_of(x[v]);
            if (BF16) key[v] = key[v] != 0 ? (key[v] & 0xFFFF0000u) | (uint32_t)(0xFFFF - (v * 16 + l)) : 0u;
        }
        const bool any_nan = (__ballot(nan) >> (lane & 48) & 0xFFFF) != 0;
        float mx = 0.f, inv = 0.f, total = 0.f, held = 0.f, chosen = 0.f;
        int held_e = -1;
        bool dead = false;
        for (int j = 0; j < a.top; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = max(best, key[v]);
            best = row_max(best);
            int e = 0xFFFF - (int)(best & 0xFFFFu);
            if (BF16) {
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = key[v] == best ? 0u : key[v];       // the expert is part of the key
            } else {
                uint32_t low = 0;                                    // the complement of the lane's first expert that has it
#pragma unroll
                for (int v = V - 1; v >= 0; --v) low = key[v] == best ? (uint32_t)(0xFFFF - (v * 16 + l)) : low;
                e = 0xFFFF - (int)row_max(low);
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = e == v * 16 + l ? 0u : key[v];
            }
            e = best != 0 ? e : -1;
            const float value = logit_of(!BF16 ? best : (int)best < 0 ? best & 0xFFFF0000u : best | 0xFFFFu);
            if (j == 0) {
                dead = best == 0 && !any_nan;
                mx = best != 0 ? value : -kInf;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = dead || v * 16 + l >= a.E ? 0.f : __builtin_amdgcn_exp2f((x[v] - mx) * kLog2e);
                    total += x[v];
                }
                total = row_sum(total);
                inv = dead ? 0.f : 1.0f / total;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += x[v] * inv;
                live += !dead;
            }
            held = l == (j & 15) ? value : held;
            held_e = l == (j & 15) ? e : held_e;
            if ((j & 15) == 15 || j == a.top - 1) {                  // 16 choices at a time
                const int j0 = j & ~15;
                const bool mine = row && j0 + l <= j;
                float w = 0.f;
                if (mine) {
                    if (held_e >= 0) {
                        w = __builtin_amdgcn_exp2f((held - mx) * kLog2e);
                        if (total != total) w = total;               // a NaN in the row
                        atomicAdd(&cnt[held_e], 1);
                    }
                    a.experts[t * a.top + j0 + l] = held_e;
                }
                chosen += row_sum(w);
                const float each = a.normalise ? (chosen > 0.f || chosen != chosen ? 1.0f / chosen : 0.f) : inv;
                const bool last = j == a.top - 1;
                if (mine) a.weights[t * a.top + j0 + l] = a.normalise && !last ? w : w * each;
                if (a.normalise && last && row)
                    for (int i = l; i < j0; i += 16) a.weights[t * a.top + i] *= each;
            }
        }
        if (row && l == 0) a.lse[t] = dead ? -kInf : mx + __builtin_amdgcn_logf(total) * kLn2;
    }
    if (l == 0 && live != 0) atomicAdd(&cnt[16 * V], live);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        acc[v] += __shfl_xor(acc[v], 16, 64);
        acc[v] += __shfl_xor(acc[v], 32, 64);
        if (group == 0) sums[wave][v * 16 + l] = acc[v];
    }
    __syncthreads();
    block_parts<16 * V>(a, sums, cnt, red);
}

// The blocks' counts and sums, 64 experts to a block: 16 threads an expert take every 16th block's, and are added in order.
// (One CU reads 50 GB/s: by itself it took 10 us for 256 blocks of 256 experts.)  With one block the loss is finished here,
// else by k_moe_route_loss from each block's part of it.
__global__ __launch_bounds__(kThreads) void k_moe_route_join(const Route a, int nb) {
    __shared__ float sums[kThreads];
    __shared__ int cnt[kThreads];
    const int t = threadIdx.x, lane = t & 63, e = blockIdx.x * 64 + lane;
    float s = 0.f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 16
        for (int b = t >> 6; b < nb; b += kWaves) {
            const u32x2 p = a.part[(int64_t)b * a.E + e];
            s += __uint_as_float(p.x);
            c += (int)p.y;
        }
    }
    sums[t] = s;
    cnt[t] = c;
    int live = 0;
    if (t < 64) {
        for (int b = t; b < nb; b += 64) live += a.part_live[b];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) live += __shfl_xor(live, o, 64);
    }
    __syncthreads();
    if (t >= 64) return;
    s = 0.f;
    c = 0;
#pragma unroll
    for (int g = 0; g < kWaves; ++g) {
        s += sums[g * 64 + t];
        c += cnt[g * 64 + t];
    }
    if (e < a.E) {
        a.prob_sum[e] = s;
        a.counts[e] = c;
    }
    const float both = wave_sum((float)c * s);
    int all = c;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o, 64);
    if (t != 0) return;
    if (blockIdx.x == 0) a.counts[a.E] = live;
    if (gridDim.x == 1) *a.loss = loss_of(a.E, both, all, live);
    else a.part_loss[blockIdx.x] = u32x2{__float_as_uint(both), (uint32_t)all};
}

__global__ __launch_bounds__(64) void k_moe_route_loss(const Route a, int blocks) {
    if (threadIdx.x != 0) return;
    float both = 0.f;
    int all = 0;
    for (int b = 0; b < blocks; ++b) {
        const u32x2 p = a.part_loss[b];
        both += __uint_as_float(p.x);
        all += (int)p.y;
    }
    *a.loss = loss_of(a.E, both, all, a.counts[a.E]);
}

// dlogits[e] = p_e (c_e - s) + the chosen experts' own part; a wave to a row.  p is exp(logit - lse) by its sum over the row: of
// logits far from zero lse has no digits behind the point (all at -1e9, as padding may be: exp would be 1 for each).  Bound by
// latency: 8192 rows of 64 experts 4.7 us, 5 MB.
template <bool BF16, int V>
__global__ __launch_bounds__(256) void k_moe_route_bwd(const Route a) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    // d loss / d p_e: the same for every row
    float c[V];
    int all = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane, n = a.dloss != nullptr && e < a.E ? a.counts[e] : 0;
        all += n;
        c[v] = (float)n;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) all += __shfl_xor(all, o, 64);
    if (a.dloss != nullptr) {
        const float f = *a.dloss * (float)a.E / (float)max(all, 1) / (float)max(a.counts[a.E], 1);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] *= f;
    }
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += step) {
        const float lse = a.lse[t];
        const bool dead = lse == -kInf;
        float p[V], d[V], s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            p[v] = e < a.E && !dead ? __builtin_amdgcn_exp2f((logit<BF16>(a.logits, t * a.ld + e) - lse) * kLog2e) : 0.f;
            s0 += p[v];
            s1 += p[v] * c[v];
        }
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        const float inv = dead ? 0.f : 1.0f / s0;
        s1 *= inv;
        float s2 = 0.f;
        if (a.dweights != nullptr) {
            for (int j = lane; j < a.top; j += 64) {
                const int e = a.experts[t * a.top + j];
                if (e >= 0 && e < a.E) s2 += a.weights[t * a.top + j] * a.dweights[t * a.top + j];
            }
            s2 = wave_sum(s2);
        }
        const float all_of = s1 + (a.normalise ? 0.f : s2), each = a.normalise ? s2 : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = dead ? 0.f : p[v] * inv * (c[v] - all_of);
        if (a.dweights != nullptr && !dead)
            for (int j = 0; j < a.top; ++j) {
                const int e = uniform(a.experts[t * a.top + j]);
                const float g = a.weights[t * a.top + j] * (a.dweights[t * a.top + j] - each);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (e == v * 64 + lane && e < a.E) d[v] += g;
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            if (e >= a.E) continue;
            if constexpr (BF16) static_cast<uint16_t *>(a.dlogits)[t * a.ld_d + e] = f32_to_bf16_rne(d[v]);
            else static_cast<float *>(a.dlogits)[t * a.ld_d + e] = d[v];
        }
    }
}

namespace {
// Rows that one block takes in one turn (64 of up to 256 experts, 16 of more) it finishes by itself, in one launch; more rows
// are spread, and joined in a second.  us with one block and with several, bfloat16: 64 rows of 64 experts, 4 choices 5.3
// and 8.1, 128 rows 7.4 and 6.6 .. 8.0; 64 rows of 256, 8 choices 11.8 and 15.1, 128 rows 18.8 and 13.2; 64 rows of 1024 (four
// turns) 25.1 and 14.4.  256 blocks, one to a CU, at most: 32768 rows of 256 experts 25.4, with 128 blocks 39.2, with 512
// 31.0 (the second block of a CU waits for the first's LDS); 8192 rows of 64 8.9, 10.4 and 13.4.
int64_t route_blocks(int64_t T, int64_t E) {
    if (T <= (E <= 256 ? 4 : 1) * kWaves) return 1;
    const int64_t n = (T + kWaves - 1) / kWaves;
    return n < kMostBlocks ? n : kMostBlocks;
}
}  // namespace

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
    const int64_t nb = route_blocks(T, E);
    return nb > 1 ? (size_t)(nb * (2 * E + 1) * 4 + kMoeMaxExperts / 64 * 8) : 0;
}

#define FP8DS_BY_TYPE(KERNEL, V, BLOCKS, THREADS)                                                   \
    do {                                                                                             \
        if (a.bf16) KERNEL<true, V><<<(unsigned)(BLOCKS), THREADS, 0, st>>>(a);                      \
        else KERNEL<false, V><<<(unsigned)(BLOCKS), THREADS, 0, st>>>(a);                            \
    } while (0)

hipError_t launch_moe_route(Route a, void *ws, hipStream_t st) {
    const int64_t nb = route_blocks(a.T, a.E);
    a.part = static_cast<u32x2 *>(ws);
    a.part_loss = a.part + nb * a.E;
    a.part_live = reinterpret_cast<int32_t *>(a.part_loss + kMoeMaxExperts / 64);
    if (a.E <= 16) FP8DS_BY_TYPE(k_moe_route_rows, 1, nb, kThreads);
    else if (a.E <= 64) FP8DS_BY_TYPE(k_moe_route_rows, 4, nb, kThreads);
    else if (a.E <= 128) FP8DS_BY_TYPE(k_moe_route_rows, 8, nb, kThreads);
    else if (a.E <= 256) FP8DS_BY_TYPE(k_moe_route_rows, 16, nb, kThreads);
    else if (a.E <= 512) FP8DS_BY_TYPE(k_moe_route, 8, nb, kThreads);
    else FP8DS_BY_TYPE(k_moe_route, 16, nb, kThreads);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || nb == 1) return e;
    const int blocks = (a.E + 63) / 64;
    k_moe_route_join<<<blocks, kThreads, 0, st>>>(a, (int)nb);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || blocks == 1) return e;
    k_moe_route_loss<<<1, 64, 0, st>>>(a, blocks);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const Route &a, hipStream_t st) {
    const int64_t rows = (a.T + 3) / 4, nb = rows < 2048 ? rows : 2048;
    if (a.E <= 64) FP8DS_BY_TYPE(k_moe_route_bwd, 1, nb, 256);
    else if (a.E <= 128) FP8DS_BY_TYPE(k_moe_route_bwd, 2, nb, 256);
    else if (a.E <= 256) FP8DS_BY_TYPE(k_moe_route_bwd, 4, nb, 256);
    else if (a.E <= 512) FP8DS_BY_TYPE(k_moe_route_bwd, 8, nb, 256);
    else FP8DS_BY_TYPE(k_moe_route_bwd, 16, nb, 256);
    return hipGetLastError();
}

}  // namespace fp8ds
