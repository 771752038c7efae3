// moe.hip -- tokens sorted by expert and back, with the router's weights, on gfx950.
//
// A choice i = t * top + j sends token t to expert experts[i].  The plan is a stable counting sort
// of the choices by expert: expert e owns the sorted rows [offsets[e], offsets[e + 1]), its
// choices first, in order, then rows that hold none (src = -1) up to a multiple of `align`, so
// that every expert's rows start where the FP8 products' 16-byte loads can start.  src[row] is the
// choice a sorted row holds, slot[choice] its row (-1 for a choice that goes nowhere).
//
//   sort     out[row] = x[src[row] / top] (times weights[src[row]]), zeros where src is -1
//   combine  y[t] = sum_j weights[t, j] * ys[slot[t, j]]        (float32, j ascending)
//   weights' gradient  dweights[t, j] = <dy[t], ys[slot[t, j]]>
//
// The gradient of sort is combine without weights, the gradient of combine is sort with weights
// (applied to dy) plus the weights' gradient.  Everything but the plan is bound by HBM: rows are
// moved in 16-byte pieces, and the FP8 forms write the transposed copy (the weight gradient's
// operand) from the same pass.  8192 tokens x 4 choices, width 4096: codes sorted with their
// transpose 58 us for 302 MB (5.2 TB/s, what a plain copy reaches), combine 61 us for 336 MB; 5000 x
// 6, width 2048: weighted FP8 gradients with their transpose 40 us, the weights' gradient 28 us; the
// plan of 32768 choices 4.7 + 4.9 us, of 32 choices 3.7, launches and latency.  Indices are checked in
// the kernels: a src or slot out of range counts as -1, so no content of the index buffers makes an
// access out of bounds.
#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

// ------------------------------------------------------------------------------------------
// Plan.  Blocks of 1024 threads take `rounds` times 1024 consecutive choices.  With more than one
// block, k_moe_hist counts each block's choices per expert first; k_moe_plan then starts every
// expert's rows from the counts of all blocks (each block adds them up for itself), and ranks its
// choices: inside a wave by ballots over the bits of the expert number, across the block's waves
// by a running position per expert.  Integer sums only, so the plan is the same every time.
// ------------------------------------------------------------------------------------------
namespace {
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int64_t kPlanOneBlock = 4096;       // choices that one block takes without a histogram launch
constexpr int64_t kPlanBlocks = 64;           // blocks beyond which each takes more rounds

void plan_shape(int64_t n, int &nb, int &rounds) {
    if (n <= kPlanOneBlock) {
        nb = 1;
        rounds = (int)((n + kPlanThreads - 1) / kPlanThreads);
        return;
    }
    rounds = (int)((n + kPlanThreads * kPlanBlocks - 1) / (kPlanThreads * kPlanBlocks));
    nb = (int)((n + (int64_t)rounds * kPlanThreads - 1) / ((int64_t)rounds * kPlanThreads));
}
}  // namespace

__global__ __launch_bounds__(kPlanThreads) void k_moe_hist(const int32_t *__restrict__ experts, int64_t n, int E,
                                                           int rounds, int32_t *__restrict__ hist) {
    __shared__ int32_t cnt[kMoeMaxExperts];
    const int t = threadIdx.x;
    cnt[t] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * rounds * kPlanThreads + t;
    for (int r = 0; r < rounds; ++r) {
        const int64_t i = i0 + (int64_t)r * kPlanThreads;
        if (i < n) {
            const int32_t e = experts[i];
            if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
        }
    }
    __syncthreads();
    if (t < E) hist[(int64_t)blockIdx.x * E + t] = cnt[t];
}

__global__ __launch_bounds__(kPlanThreads) void k_moe_plan(const int32_t *__restrict__ experts, int64_t n, int E,
                                                           int align, int64_t cap, int rounds,
                                                           const int32_t *__restrict__ hist,
                                                           int32_t *__restrict__ offsets, int32_t *__restrict__ src,
                                                           int32_t *__restrict__ slot) {
    __shared__ int32_t base[kMoeMaxExperts];
    __shared__ int32_t wcnt[kPlanWaves][kMoeMaxExperts];
    __shared__ int32_t wsum[kPlanWaves + 1], ahead[kMoeMaxExperts];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, nb = gridDim.x;
    const int64_t i0 = (int64_t)blockIdx.x * rounds * kPlanThreads + t;

    // choices of expert t: all, and those in the blocks before this one
    int32_t total = 0, before = 0;
    if (nb == 1) {
        base[t] = 0;
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            const int64_t i = i0 + (int64_t)r * kPlanThreads;
            if (i < n) {
                const int32_t e = experts[i];
                if (e >= 0 && e < E) atomicAdd(&base[e], 1);
            }
        }
        __syncthreads();
        total = base[t];
    } else {
        // all threads read the histograms, 1024 / (E rounded up to a power of two) blocks' at a time
        base[t] = ahead[t] = 0;
        __syncthreads();
        const int log2 = E > 1 ? 32 - __builtin_clz(E - 1) : 0, e = t & ((1 << log2) - 1);
        int32_t all = 0, mine = 0;
        if (e < E) {
#pragma unroll 4
            for (int b = t >> log2; b < nb; b += kPlanThreads >> log2) {
                const int32_t h = hist[(int64_t)b * E + e];
                all += h;
                mine += b < (int)blockIdx.x ? h : 0;
            }
        }
        if (all != 0) atomicAdd(&base[e], all);
        if (mine != 0) atomicAdd(&ahead[e], mine);
        __syncthreads();
        total = base[t];
        before = ahead[t];
    }
    // first row of expert t: exclusive sum of the padded counts
    const int32_t padded = (total + align - 1) / align * align;
    int32_t incl = padded;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int32_t first = incl - padded, end = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        const int32_t v = wsum[w];
        if (w < wave) first += v;
        end += v;
    }
    base[t] = first + before;
    if (blockIdx.x == 0) {
        if (t < E) offsets[t] = first;
        if (t == 0) offsets[E] = end;
    }
    // rows without a choice: behind each expert's own (experts dealt to the blocks) and at the end
    if (t < E && t % nb == (int)blockIdx.x)
        for (int32_t p = first + total; p < first + padded; ++p) src[p] = -1;
    for (int64_t p = end + (int64_t)blockIdx.x * kPlanThreads + t; p < cap; p += (int64_t)nb * kPlanThreads) src[p] = -1;

    const int bits = 32 - __builtin_clz(E);   // expert numbers 0 .. E, E standing for "none"
    for (int r = 0; r < rounds; ++r) {
        const int64_t i = i0 + (int64_t)r * kPlanThreads;
        const int32_t e = i < n ? experts[i] : -1;
        const bool valid = e >= 0 && e < E;
        const int key = valid ? e : E;
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const bool bit = (key >> b) & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1ull));
        for (int c = lane; c < E; c += 64) wcnt[wave][c] = 0;
        __builtin_amdgcn_wave_barrier();
        if (valid && rank == 0) wcnt[wave][key] = __popcll(same);
        __syncthreads();
        if (t < E) {
            int32_t pos = base[t];
#pragma unroll
            for (int w = 0; w < kPlanWaves; ++w) {
                const int32_t c = wcnt[w][t];
                wcnt[w][t] = pos;
                pos += c;
            }
            base[t] = pos;
        }
        __syncthreads();
        if (valid) {
            const int32_t p = wcnt[wave][key] + rank;
            slot[i] = p;
            src[p] = (int32_t)i;
        } else if (i < n) {
            slot[i] = -1;
        }
        __syncthreads();
    }
}

size_t moe_workspace_bytes(int64_t n, int64_t E) {
    int nb, rounds;
    plan_shape(n, nb, rounds);
    return nb > 1 ? (size_t)nb * (size_t)E * sizeof(int32_t) : 0;
}

hipError_t launch_moe_plan(const int32_t *experts, int64_t n, int64_t E, int64_t align, int64_t cap, int32_t *offsets,
                           int32_t *src, int32_t *slot, void *ws, hipStream_t st) {
    int nb, rounds;
    plan_shape(n, nb, rounds);
    int32_t *hist = static_cast<int32_t *>(ws);
    if (nb > 1) {
        k_moe_hist<<<nb, kPlanThreads, 0, st>>>(experts, n, (int)E, rounds, hist);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    k_moe_plan<<<nb, kPlanThreads, 0, st>>>(experts, n, (int)E, (int)align, cap, rounds, hist, offsets, src, slot);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------------
// Sort.  Eight or sixteen consecutive columns of a sorted row: the values (token row times
// weight, float32), their amax, and their codes.
// ------------------------------------------------------------------------------------------
namespace {
// Token row of a sorted row's choice, -1 for none.
__device__ __forceinline__ int token_of(int32_t src, int choices, int top) {
    return (uint32_t)src < (uint32_t)choices ? src / top : -1;
}
__device__ __forceinline__ uint32_t amax4(uint32_t acc, float a, float b, float c, float d) {
    acc = max(acc, __float_as_uint(a) & 0x7FFFFFFFu);
    acc = max(acc, __float_as_uint(b) & 0x7FFFFFFFu);
    acc = max(acc, __float_as_uint(c) & 0x7FFFFFFFu);
    return max(acc, __float_as_uint(d) & 0x7FFFFFFFu);
}
}  // namespace

// Row-major output only: TX threads per row, 16 columns each step.
template <int WHAT>
__global__ __launch_bounds__(256) void k_moe_rows(const MoeSort a, int tx_log2, int64_t first) {
    __shared__ uint32_t red[4];
    const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
    const int64_t row = ((first + blockIdx.x) << (8 - tx_log2)) + ty;
    constexpr bool kCast = WHAT == kSortE4M3 || WHAT == kSortE5M2;
    constexpr int FMT = WHAT == kSortE5M2 ? kE5M2 : kE4M3;
    float s = 0.f;
    if constexpr (kCast) s = *a.scale;
    uint32_t amag = 0;
    if (row < a.cap) {
        const int32_t sv = a.src[row];
        const int tok = token_of(sv, a.choices, a.top);
        float w = 1.f;
        if (a.weights != nullptr && tok >= 0) w = a.weights[sv];
        const int n16 = a.width >> 4;
        for (int c = tx; c < n16; c += 1 << tx_log2) {
            const int64_t in = (int64_t)tok * a.width + c * 16, at = row * a.width + c * 16;
            if constexpr (WHAT == kSortCodes) {
                u32x4 v = {0u, 0u, 0u, 0u};
                if (tok >= 0) v = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(a.x) + in);
                __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(a.out) + at));
            } else {
                u32x4 p = {0u, 0u, 0u, 0u}, q = {0u, 0u, 0u, 0u};
                if (tok >= 0) {
                    const u32x4 *x = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + in);
                    p = x[0];
                    q = x[1];
                }
                const uint32_t r[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                float v[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) { v[2 * i] = bf16_lo(r[i]) * w; v[2 * i + 1] = bf16_hi(r[i]) * w; }
                if (tok < 0)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.f;
                if constexpr (kCast) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        amag = amax4(amag, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        o[i] = tok < 0 ? 0u : encode4<FMT>(v[4 * i] * s, v[4 * i + 1] * s, v[4 * i + 2] * s, v[4 * i + 3] * s);
                    }
                    __builtin_nontemporal_store(u32x4{o[0], o[1], o[2], o[3]},
                                                reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(a.out) + at));
                } else {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
                    u32x4 *y = reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + at);
                    __builtin_nontemporal_store(u32x4{o[0], o[1], o[2], o[3]}, y);
                    __builtin_nontemporal_store(u32x4{o[4], o[5], o[6], o[7]}, y + 1);
                }
            }
        }
    }
    if constexpr (kCast) {
        const uint32_t bm = block_max_u32<256>(amag, red);
        if (threadIdx.x == 0) {
            fold_amax_bits(a.amax, bm);
            if (blockIdx.x == 0 && a.sinv != nullptr) *a.sinv = 1.0f / s;
        }
    }
}

// Codes and their transpose: TS x TS tiles, 8 x 8 codes per thread, the transposed copy through
// LDS (slot rb of transposed row c at rb ^ (c / 8): conflict-free writes, 16-byte reads), as the
// cast + transpose kernel does; here the tile's rows come from the tokens that src names.
template <int WHAT, int TS>
__global__ __launch_bounds__((TS / 8) * (TS / 8)) void k_moe_sort_t(const MoeSort a, int tiles_c, int first) {
    constexpr int NRB = TS / 8, NT = NRB * NRB, CH = TS / 16;
    constexpr int FMT = WHAT == kSortE5M2 ? kE5M2 : kE4M3;
    __shared__ __align__(16) uint8_t tT[TS * TS];
    __shared__ uint32_t red[NT / 64];
    const int t = threadIdx.x, rb = t / NRB, cb = t % NRB;
    const int tile = first + (int)blockIdx.x, tile_r = (uint32_t)tile / (uint32_t)tiles_c, tile_c = tile - tile_r * tiles_c;
    const int64_t r0 = (int64_t)tile_r * TS, row = r0 + rb * 8;
    const int c0 = tile_c * TS, col = c0 + cb * 8;
    const int H = a.width;
    float s = 0.f;
    if constexpr (WHAT != kSortCodes) s = *a.scale;
    uint32_t amag = 0;
    uint32_t orow[8][2];
    const bool in = row < a.cap && col < H;    // cap and the width are multiples of 16: whole micro-tiles
    int32_t sv[8];
    if (in) {
        const u32x4 p = *reinterpret_cast<const u32x4 *>(a.src + row), q = *reinterpret_cast<const u32x4 *>(a.src + row + 4);
        sv[0] = p.x; sv[1] = p.y; sv[2] = p.z; sv[3] = p.w; sv[4] = q.x; sv[5] = q.y; sv[6] = q.z; sv[7] = q.w;
    } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) sv[r] = -1;
    }
    if constexpr (WHAT == kSortCodes) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int tok = token_of(sv[r], a.choices, a.top);
            u32x2 v = {0u, 0u};
            if (tok >= 0) v = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(a.x) + (int64_t)tok * H + col);
            orow[r][0] = v.x;
            orow[r][1] = v.y;
        }
    } else {
        u32x4 x[8];
        float w[8];
        bool live[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int tok = token_of(sv[r], a.choices, a.top);
            live[r] = tok >= 0;
            x[r] = u32x4{0u, 0u, 0u, 0u};
            w[r] = 1.f;
            if (live[r]) {
                x[r] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.x) + (int64_t)tok * H + col);
                if (a.weights != nullptr) w[r] = a.weights[sv[r]];
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t q[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = live[r] ? bf16_lo(q[i]) * w[r] : 0.f;
                v[2 * i + 1] = live[r] ? bf16_hi(q[i]) * w[r] : 0.f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                amag = amax4(amag, v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
                orow[r][h] = live[r] ? encode4<FMT>(v[4 * h] * s, v[4 * h + 1] * s, v[4 * h + 2] * s, v[4 * h + 3] * s) : 0u;
            }
        }
    }
    if (in) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
            __builtin_nontemporal_store(u32x2{orow[r][0], orow[r][1]},
                                        reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + (row + r) * H + col));
    }
    uint32_t ocol[8][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        tr4(orow[0][h], orow[1][h], orow[2][h], orow[3][h], ocol[4 * h][0], ocol[4 * h + 1][0], ocol[4 * h + 2][0],
            ocol[4 * h + 3][0]);
        tr4(orow[4][h], orow[5][h], orow[6][h], orow[7][h], ocol[4 * h][1], ocol[4 * h + 1][1], ocol[4 * h + 2][1],
            ocol[4 * h + 3][1]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int tc = cb * 8 + c;
        *reinterpret_cast<u32x2 *>(&tT[tc * TS + ((rb ^ ((tc >> 3) & (NRB - 1))) << 3)]) = u32x2{ocol[c][0], ocol[c][1]};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (TS * TS / 16) / NT; ++i) {
        const int q = t + NT * i;
        const int tr = q / CH, part = q % CH;
        const int g = (tr >> 3) & (NRB - 1);
        u32x4 v = *reinterpret_cast<const u32x4 *>(&tT[tr * TS + ((part ^ (g >> 1)) << 4)]);
        if (g & 1) v = v.zwxy;
        const int64_t oc = r0 + part * 16;
        if (c0 + tr < H && oc < a.cap)
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(a.out_t + (int64_t)(c0 + tr) * a.cap + oc));
    }
    if constexpr (WHAT != kSortCodes) {
        const uint32_t bm = block_max_u32<NT>(amag, red);
        if (t == 0) {
            fold_amax_bits(a.amax, bm);
            if (blockIdx.x == 0 && a.sinv != nullptr) *a.sinv = 1.0f / s;
        }
    }
}

// ------------------------------------------------------------------------------------------
// Combine: a thread sums eight columns of a token's rows; four rows are loaded before any is used.
// A choice without a row contributes nothing, whatever its weight holds.
// ------------------------------------------------------------------------------------------
template <bool WEIGHTED>
__global__ __launch_bounds__(256) void k_moe_combine(const uint16_t *__restrict__ ys, const int32_t *__restrict__ slot,
                                                     const float *__restrict__ weights, uint16_t *__restrict__ y,
                                                     int64_t T, int k, int H, int64_t cap, int tx_log2, int64_t first) {
    const int tx = threadIdx.x & ((1 << tx_log2) - 1), ty = threadIdx.x >> tx_log2;
    const int64_t tok = ((first + blockIdx.x) << (8 - tx_log2)) + ty;
    if (tok >= T) return;
    for (int c = tx; c < (H >> 3); c += 1 << tx_log2) {
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int j0 = 0; j0 < k; j0 += 4) {
            u32x4 v[4];
            float w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] = u32x4{0u, 0u, 0u, 0u};
                w[u] = 0.f;
                if (j0 + u < k) {
                    const int32_t p = slot[tok * k + j0 + u];
                    if (p >= 0 && p < cap) {
                        v[u] = *reinterpret_cast<const u32x4 *>(ys + (int64_t)p * H + c * 8);
                        w[u] = WEIGHTED ? weights[tok * k + j0 + u] : 1.f;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t q[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = __builtin_fmaf(w[u], bf16_lo(q[i]), acc[2 * i]);
                    acc[2 * i + 1] = __builtin_fmaf(w[u], bf16_hi(q[i]), acc[2 * i + 1]);
                }
            }
        }
        __builtin_nontemporal_store(u32x4{f32x2_to_bf16x2_rne(acc[0], acc[1]), f32x2_to_bf16x2_rne(acc[2], acc[3]),
                                          f32x2_to_bf16x2_rne(acc[4], acc[5]), f32x2_to_bf16x2_rne(acc[6], acc[7])},
                                    reinterpret_cast<u32x4 *>(y + tok * H + c * 8));
    }
}

// Weights' gradient: one wave per choice.
__global__ __launch_bounds__(256) void k_moe_weight_grad(const uint16_t *__restrict__ dy, const uint16_t *__restrict__ ys,
                                                         const int32_t *__restrict__ slot, float *__restrict__ dweights,
                                                         int64_t n, int k, int H, int64_t cap, int64_t first) {
    const int lane = threadIdx.x & 63;
    const int64_t i = (first + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (i >= n) return;
    const int32_t p = slot[i];
    float acc = 0.f;
    if (p >= 0 && p < cap) {
        const uint16_t *a = dy + i / k * H, *b = ys + (int64_t)p * H;
        for (int c = lane; c < (H >> 3); c += 64) {
            const u32x4 u = *reinterpret_cast<const u32x4 *>(a + c * 8), v = *reinterpret_cast<const u32x4 *>(b + c * 8);
            const uint32_t q[4] = {u.x, u.y, u.z, u.w}, r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc = __builtin_fmaf(bf16_lo(q[j]), bf16_lo(r[j]), acc);
                acc = __builtin_fmaf(bf16_hi(q[j]), bf16_hi(r[j]), acc);
            }
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
    if (lane == 0) dweights[i] = acc;
}

namespace {
// Threads per row for `pieces` 16-byte pieces: a power of two up to the block.
int row_threads_log2(int64_t pieces) {
    int l = 0;
    while (l < 8 && (INT64_C(1) << l) < pieces) ++l;
    return l;
}
constexpr int64_t kSortBigTiles = 256;    // 256 x 256 tiles from one per CU on, else 64 x 64

// A launch numbers its threads in 32 bits, and one of more runs what is left modulo 2^32 without an
// error: larger grids go in pieces, each told its first block.
constexpr int64_t kMostThreads = INT64_C(1) << 31;
template <class Launch> hipError_t in_pieces(int64_t blocks, int threads, Launch launch) {
    const int64_t most = kMostThreads / threads;
    for (int64_t first = 0; first < blocks; first += most) {
        launch(dim3((unsigned)(blocks - first < most ? blocks - first : most)), first);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}
}  // namespace

hipError_t launch_moe_sort(const MoeSort &a, int what, hipStream_t st) {
    if (a.out_t != nullptr) {
        const int64_t big = ((a.cap + 255) / 256) * (((int64_t)a.width + 255) / 256);
        const int ts = big >= kSortBigTiles ? 256 : 64;
        const int tiles_c = (a.width + ts - 1) / ts;
        return in_pieces((a.cap + ts - 1) / ts * tiles_c, ts == 256 ? 1024 : 64, [&](dim3 grid, int64_t first) {
#define FP8DS_SORT_T(W_)                                                                                   \
    do {                                                                                                   \
        if (ts == 256) k_moe_sort_t<W_, 256><<<grid, 1024, 0, st>>>(a, tiles_c, (int)first);               \
        else k_moe_sort_t<W_, 64><<<grid, 64, 0, st>>>(a, tiles_c, (int)first);                            \
    } while (0)
            switch (what) {
                case kSortCodes: FP8DS_SORT_T(kSortCodes); break;
                case kSortE4M3: FP8DS_SORT_T(kSortE4M3); break;
                default: FP8DS_SORT_T(kSortE5M2); break;
            }
#undef FP8DS_SORT_T
        });
    }
    const int l = row_threads_log2(a.width >> 4);
    return in_pieces((a.cap + (256 >> l) - 1) / (256 >> l), 256, [&](dim3 grid, int64_t first) {
        switch (what) {
            case kSortCodes: k_moe_rows<kSortCodes><<<grid, 256, 0, st>>>(a, l, first); break;
            case kSortE4M3: k_moe_rows<kSortE4M3><<<grid, 256, 0, st>>>(a, l, first); break;
            case kSortE5M2: k_moe_rows<kSortE5M2><<<grid, 256, 0, st>>>(a, l, first); break;
            default: k_moe_rows<kSortBf16><<<grid, 256, 0, st>>>(a, l, first); break;
        }
    });
}

hipError_t launch_moe_combine(const uint16_t *ys, const int32_t *slot, const float *weights, uint16_t *y, int64_t T,
                              int64_t k, int64_t width, int64_t cap, hipStream_t st) {
    const int l = row_threads_log2(width >> 3);
    return in_pieces((T + (256 >> l) - 1) / (256 >> l), 256, [&](dim3 grid, int64_t first) {
        if (weights != nullptr)
            k_moe_combine<true><<<grid, 256, 0, st>>>(ys, slot, weights, y, T, (int)k, (int)width, cap, l, first);
        else
            k_moe_combine<false><<<grid, 256, 0, st>>>(ys, slot, weights, y, T, (int)k, (int)width, cap, l, first);
    });
}

hipError_t launch_moe_weight_grad(const uint16_t *dy, const uint16_t *ys, const int32_t *slot, float *dweights,
                                  int64_t T, int64_t k, int64_t width, int64_t cap, hipStream_t st) {
    const int64_t n = T * k;
    return in_pieces((n + 3) / 4, 256, [&](dim3 grid, int64_t first) {
        k_moe_weight_grad<<<grid, 256, 0, st>>>(dy, ys, slot, dweights, n, (int)k, (int)width, cap, first);
    });
}

}  // namespace fp8ds
