// router.hip -- the choice of experts from the router's logits, with the balance loss, and its gradient, on gfx950.
#include <climits>

#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMostBlocks = 256;
constexpr int64_t kOneBlock = 128;           // rows that one block takes, finishing them itself
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int CTRL, int ROWS> __device__ __forceinline__ float dpp(float old, float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(old), (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}
// over the wave, the same in every lane; a NaN is passed over by the maximum
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0x111, 0xf>(v, v));     // row_shr 1, 2, 4, 8 inside 16 lanes, then across
    v = fmaxf(v, dpp<0x112, 0xf>(v, v));
    v = fmaxf(v, dpp<0x114, 0xf>(v, v));
    v = fmaxf(v, dpp<0x118, 0xf>(v, v));
    v = fmaxf(v, dpp<0x142, 0xa>(v, v));
    v = fmaxf(v, dpp<0x143, 0xc>(v, v));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0x111, 0xf>(0.f, v);
    v += dpp<0x112, 0xf>(0.f, v);
    v += dpp<0x114, 0xf>(0.f, v);
    v += dpp<0x118, 0xf>(0.f, v);
    v += dpp<0x142, 0xa>(0.f, v);
    v += dpp<0x143, 0xc>(0.f, v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

template <bool BF16> __device__ __forceinline__ float logit(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else return static_cast<const float *>(p)[i];
}

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
    *a.loss = (float)a.E * (both / (float)max(all, 1)) / (float)max(counts[a.E], 1);
}

}  // namespace

// A wave takes a row, lane l its experts l, l + 64, ...
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
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += step) {
        float x[V], p[V];
        float mx = -kInf;
        bool nan = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            x[v] = e < a.E ? logit<BF16>(a.logits, t * a.ld + e) : -kInf;
            mx = fmaxf(mx, x[v]);
            nan |= x[v] != x[v];
        }
        mx = wave_max(mx);
        const bool dead = mx == -kInf && !__any(nan);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[v] = dead ? 0.f : __builtin_amdgcn_exp2f((x[v] - mx) * kLog2e);
            if (v * 64 + lane >= a.E) p[v] = 0.f;
            sum += p[v];
        }
        sum = wave_sum(sum);
        const float inv = dead ? 0.f : 1.0f / sum;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += p[v] * inv;
        live += !dead;
        // the largest logit left, ties to the lowest expert
        float chosen_sum = 0.f, mine_w = 0.f;
        int mine_e = -1;
        for (int j = 0; j < a.top; ++j) {
            float best = -kInf;
#pragma unroll
            for (int v = 0; v < V; ++v) best = fmaxf(best, x[v]);
            best = wave_max(best);
            int e = -1;
            if (best > -kInf) {
#pragma unroll
                for (int v = V - 1; v >= 0; --v) {
                    const uint64_t at = __ballot(x[v] == best);
                    if (at != 0) e = v * 64 + __ffsll((unsigned long long)at) - 1;
                }
            }
            float w = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (e == v * 64 + lane) {
                    w = p[v];
                    x[v] = -kInf;
                }
            if (e >= 0) {
                w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(w), e & 63));
                chosen_sum += w;
                if (lane == 0) atomicAdd(&cnt[e], 1);
            }
            if (lane == (j & 63)) {
                mine_e = e;
                mine_w = w;
            }
            if ((j & 63) == 63 || j == a.top - 1) {                  // 64 choices at a time
                const int j0 = j & ~63;
                if (j0 + lane <= j) {
                    a.experts[t * a.top + j0 + lane] = mine_e;
                    a.weights[t * a.top + j0 + lane] = a.normalise ? mine_w : mine_w * inv;
                }
            }
        }
        if (a.normalise) {
            const float each = chosen_sum > 0.f || chosen_sum != chosen_sum ? 1.0f / chosen_sum : 0.f;
            for (int j = lane; j < a.top; j += 64) a.weights[t * a.top + j] *= each;
        }
        if (lane == 0) a.lse[t] = dead ? -kInf : mx + __builtin_amdgcn_logf(sum) * kLn2;
    }
    if (lane == 0 && live != 0) atomicAdd(&cnt[64 * V], live);
#pragma unroll
    for (int v = 0; v < V; ++v) sums[wave][v * 64 + lane] = acc[v];
    __syncthreads();
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
            a.part_sum[(int64_t)blockIdx.x * a.E + e] = s;
            a.part_cnt[(int64_t)blockIdx.x * (a.E + 1) + e] = cnt[e];
        }
    }
    if (nb > 1) {
        if (threadIdx.x == 0) a.part_cnt[(int64_t)blockIdx.x * (a.E + 1) + a.E] = cnt[64 * V];
        return;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.counts[a.E] = cnt[64 * V];
        cnt[a.E] = cnt[64 * V];
    }
    __syncthreads();
    finish_loss(a, sums[0], cnt, red);
}

// The blocks' counts and sums: `groups` threads an expert take every groups-th block, the groups are added in order.
__global__ __launch_bounds__(kThreads) void k_moe_route_join(const Route a, int nb, int log2_e) {
    __shared__ float sums[kThreads];
    __shared__ int cnt[kThreads + 1];
    __shared__ float red[2 * kWaves];
    const int t = threadIdx.x, e = t & ((1 << log2_e) - 1), groups = kThreads >> log2_e;
    float s = 0.f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int b = t >> log2_e; b < nb; b += groups) {
            s += a.part_sum[(int64_t)b * a.E + e];
            c += a.part_cnt[(int64_t)b * (a.E + 1) + e];
        }
    }
    sums[t] = s;
    cnt[t] = c;
    int live = 0;
    if (t < 64) {
        for (int b = t; b < nb; b += 64) live += a.part_cnt[(int64_t)b * (a.E + 1) + a.E];
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) live += __shfl_xor(live, o, 64);
    }
    __syncthreads();
    if (t < a.E) {
        s = 0.f;
        c = 0;
        for (int g = 0; g < groups; ++g) {
            s += sums[(g << log2_e) + t];
            c += cnt[(g << log2_e) + t];
        }
        a.prob_sum[t] = s;
        a.counts[t] = c;
    }
    __syncthreads();
    if (t < a.E) {
        sums[t] = s;
        cnt[t] = c;
    }
    if (t == 0) {
        a.counts[a.E] = live;
        cnt[a.E] = live;
    }
    __syncthreads();
    finish_loss(a, sums, cnt, red);
}

// dlogits[e] = p_e (c_e - s) + the chosen experts' own part; a wave to a row.
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
        float p[V], d[V], s1 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            p[v] = e < a.E && !dead ? __builtin_amdgcn_exp2f((logit<BF16>(a.logits, t * a.ld + e) - lse) * kLog2e) : 0.f;
            s1 += p[v] * c[v];
        }
        s1 = wave_sum(s1);
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
        for (int v = 0; v < V; ++v) d[v] = p[v] * (c[v] - all_of);
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
int64_t route_blocks(int64_t T) {
    if (T <= kOneBlock) return 1;
    const int64_t n = (T + kWaves - 1) / kWaves;
    return n < kMostBlocks ? n : kMostBlocks;
}
}  // namespace

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
    const int64_t nb = route_blocks(T);
    return nb > 1 ? (size_t)(nb * (2 * E + 1) * 4) : 0;
}

#define FP8DS_BY_EXPERTS(KERNEL, BLOCKS, THREADS)                                                    \
    do {                                                                                             \
        const dim3 grid((unsigned)(BLOCKS));                                                         \
        if (a.bf16) {                                                                                \
            if (a.E <= 64) KERNEL<true, 1><<<grid, THREADS, 0, st>>>(a);                             \
            else if (a.E <= 128) KERNEL<true, 2><<<grid, THREADS, 0, st>>>(a);                       \
            else if (a.E <= 256) KERNEL<true, 4><<<grid, THREADS, 0, st>>>(a);                       \
            else KERNEL<true, 16><<<grid, THREADS, 0, st>>>(a);                                      \
        } else {                                                                                     \
            if (a.E <= 64) KERNEL<false, 1><<<grid, THREADS, 0, st>>>(a);                            \
            else if (a.E <= 128) KERNEL<false, 2><<<grid, THREADS, 0, st>>>(a);                      \
            else if (a.E <= 256) KERNEL<false, 4><<<grid, THREADS, 0, st>>>(a);                      \
            else KERNEL<false, 16><<<grid, THREADS, 0, st>>>(a);                                     \
        }                                                                                            \
    } while (0)

hipError_t launch_moe_route(Route a, void *ws, hipStream_t st) {
    const int64_t nb = route_blocks(a.T);
    a.part_sum = static_cast<float *>(ws);
    a.part_cnt = static_cast<int32_t *>(ws) + nb * a.E;
    FP8DS_BY_EXPERTS(k_moe_route, nb, kThreads);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || nb == 1) return e;
    int log2_e = 0;
    while ((1 << log2_e) < a.E) ++log2_e;
    k_moe_route_join<<<1, kThreads, 0, st>>>(a, (int)nb, log2_e);
    return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const Route &a, hipStream_t st) {
    const int64_t n = (a.T + 3) / 4;
    FP8DS_BY_EXPERTS(k_moe_route_bwd, n < 2048 ? n : 2048, 256);
    return hipGetLastError();
}

}  // namespace fp8ds
