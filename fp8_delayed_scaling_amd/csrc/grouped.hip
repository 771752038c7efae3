// grouped.hip -- the experts' FP8 products over tokens sorted by expert, on gfx950 matrix cores.
//
//   forward / input gradient   D[r, :] = A[r, :] B[e]^T * a_scale_inv * b_scale_inv   for the rows r of expert e
//   weight gradient            D[e] = A[:, rows of e] B[:, rows of e]^T * (the same)
//
// offsets[e] .. offsets[e + 1] are expert e's rows, read on the device: the host never learns
// them, so the grid covers the largest number of tiles any routing can give and the blocks past
// the actual tiles end at once.  Both operands are K-contiguous and accumulate in float32; the one
// product order per output is fixed, so results do not depend on the routing of other experts.
// Offsets are held to [0, cap] and to multiples of 16 as they are read, so no content of the
// buffer makes an access out of bounds.
#include <climits>

#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

constexpr int kT = 128;                      // tile rows and columns
constexpr int kStep = 128;                   // K bytes per step
constexpr int kThreads = 256;
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ int offset_at(const Grouped &g, int e) {
    return min(max(g.offsets[e], 0), g.cap) & ~15;
}

// The expert and first row of row tile `tile`, counting every expert's tiles of `tm` rows in
// order: each wave sums 64 experts' tile counts at a time.  False past the last tile.
__device__ __forceinline__ bool find_tile(const Grouped &g, int tile, int tm, int &e, int &row, int &end) {
    const int lane = threadIdx.x & 63;
    int seen = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
        const int i = e0 + lane;
        int lo = 0, hi = 0;
        if (i < g.E) {
            lo = offset_at(g, i);
            hi = offset_at(g, i + 1);
        }
        const int n = hi > lo ? (hi - lo + tm - 1) / tm : 0;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if (lane >= off) incl += v;
        }
        const uint64_t past = __ballot(seen + incl > tile);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            e = __builtin_amdgcn_readfirstlane(e0 + l);
            row = __builtin_amdgcn_readfirstlane(__shfl(lo + (tile - seen - (incl - n)) * tm, l, 64));
            end = __builtin_amdgcn_readfirstlane(__shfl(hi, l, 64));
            return true;
        }
        seen += __shfl(incl, 63, 64);
    }
    return false;
}

// One 128 x 128 tile of A B^T: rows_a / rows_b rows are inside, K a multiple of 16 (the rest of
// the last step counts as zero codes).  Four waves of 64 x 64.
template <int FA, int FB, int OUT>
__device__ __forceinline__ void tile_product(const uint8_t *__restrict__ A, int64_t lda, int rows_a,
                                             const uint8_t *__restrict__ B, int64_t ldb, int rows_b, int K, float sa,
                                             float sb, void *__restrict__ D, int64_t ldd) {
    __shared__ __align__(16) uint8_t lds[2][2][kT * kStep];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int lrow = tid >> 3, part = tid & 7;    // rows lrow + 32 i, 16-byte piece `part`
    u32x4 ra[4], rb[4];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = lrow + 32 * i;
            ra[i] = rb[i] = u32x4{0u, 0u, 0u, 0u};
            if (k0 + part * 16 < K) {
                ra[i] = *reinterpret_cast<const u32x4 *>(A + (int64_t)min(r, rows_a - 1) * lda + k0 + part * 16);
                rb[i] = *reinterpret_cast<const u32x4 *>(B + (int64_t)min(r, rows_b - 1) * ldb + k0 + part * 16);
            }
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = lrow + 32 * i;
            *reinterpret_cast<u32x4 *>(&lds[buf][0][r * kStep + ((part ^ swz(r)) << 4)]) = ra[i];
            *reinterpret_cast<u32x4 *>(&lds[buf][1][r * kStep + ((part ^ swz(r)) << 4)]) = rb[i];
        }
    };
    const int r16 = lane & 15, g = lane >> 4;
    auto frag = [&](const uint8_t *p, int r) -> i32x8 {
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(p + r * kStep + (((2 * g) ^ swz(r)) << 4));
        const u32x4 hi = *reinterpret_cast<const u32x4 *>(p + r * kStep + (((2 * g + 1) ^ swz(r)) << 4));
        i32x8 v;
        v[0] = (int)lo.x; v[1] = (int)lo.y; v[2] = (int)lo.z; v[3] = (int)lo.w;
        v[4] = (int)hi.x; v[5] = (int)hi.y; v[6] = (int)hi.z; v[7] = (int)hi.w;
        return v;
    };
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int nk = (K + kStep - 1) / kStep;
    if (nk > 0) {
        load(0);
        stash(0);
    }
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        if (kt + 1 < nk) load((kt + 1) * kStep);
        const uint8_t *as = lds[kt & 1][0], *bs = lds[kt & 1][1];
        i32x8 fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[i] = frag(as, wm * 64 + i * 16 + r16);
            fb[i] = frag(bs, wn * 64 + i * 16 + r16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i], acc[i][j], FB, FA, 0, 0, 0, 0);
        if (kt + 1 < nk) stash((kt + 1) & 1);
        __syncthreads();
    }
    // lane l holds D[16 i + l % 16][16 j + 4 (l / 16) + u] in element u of acc[i][j]
    constexpr int kEsz = OUT == 0 ? 2 : 4;
    const bool vec4 = ((reinterpret_cast<uintptr_t>(D) & (uintptr_t)(4 * kEsz - 1)) == 0) && (ldd % 4 == 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = wm * 64 + i * 16 + r16;
        if (row >= rows_a) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = wn * 64 + j * 16 + g * 4;
            float v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = dequant_bias(acc[i][j][u], sa, sb, 0.f);
            const int64_t o = (int64_t)row * ldd + col;
            if (vec4 && col + 3 < rows_b) {
                if constexpr (OUT == 0)
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(D) + o) =
                        u32x2{f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3])};
                else
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(D) + o) = f32x4{v[0], v[1], v[2], v[3]};
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (col + u < rows_b) {
                        if constexpr (OUT == 0) static_cast<uint16_t *>(D)[o + u] = f32_to_bf16_rne(v[u]);
                        else static_cast<float *>(D)[o + u] = v[u];
                    }
            }
        }
    }
}

}  // namespace

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(kThreads) void k_grouped_gemm(const Grouped g, int tiles_n) {
    const int tile = blockIdx.x / tiles_n, tn = blockIdx.x - tile * tiles_n;
    int e, row, end;
    if (!find_tile(g, tile, kT, e, row, end)) return;
    constexpr int kEsz = OUT == 0 ? 2 : 4;
    tile_product<FA, FB, OUT>(g.A + (int64_t)row * g.lda, g.lda, min(kT, end - row),
                              g.B + (int64_t)e * g.stride_b + (int64_t)tn * kT * g.ldb, g.ldb, min(kT, g.N - tn * kT), g.K,
                              *g.a_sinv, *g.b_sinv,
                              static_cast<uint8_t *>(g.D) + ((int64_t)row * g.ldd + tn * kT) * kEsz, g.ldd);
}

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(kThreads) void k_grouped_wgrad(const Grouped g, int tiles_m, int tiles_n) {
    const int per = tiles_m * tiles_n, e = blockIdx.x / per, in = blockIdx.x - e * per;
    const int tm = in / tiles_n, tn = in - tm * tiles_n;
    const int lo = offset_at(g, e), len = max(0, offset_at(g, e + 1) - lo);
    constexpr int kEsz = OUT == 0 ? 2 : 4;
    tile_product<FA, FB, OUT>(g.A + (int64_t)tm * kT * g.lda + lo, g.lda, min(kT, g.N - tm * kT),
                              g.B + (int64_t)tn * kT * g.ldb + lo, g.ldb, min(kT, g.K - tn * kT), len, *g.a_sinv,
                              *g.b_sinv,
                              static_cast<uint8_t *>(g.D) + ((int64_t)e * g.stride_d + (int64_t)tm * kT * g.ldd + tn * kT) * kEsz,
                              g.ldd);
}

#define FP8DS_GROUPED_SWITCH(CALL)                                                                         \
    switch ((fa * 2 + fb) * 2 + out_dtype) {                                                               \
        case 0: CALL(kE4M3, kE4M3, 0); break;                                                              \
        case 1: CALL(kE4M3, kE4M3, 1); break;                                                              \
        case 2: CALL(kE4M3, kE5M2, 0); break;                                                              \
        case 3: CALL(kE4M3, kE5M2, 1); break;                                                              \
        case 4: CALL(kE5M2, kE4M3, 0); break;                                                              \
        case 5: CALL(kE5M2, kE4M3, 1); break;                                                              \
        case 6: CALL(kE5M2, kE5M2, 0); break;                                                              \
        default: CALL(kE5M2, kE5M2, 1); break;                                                             \
    }

// The largest number of row tiles: every expert with rows adds at most one partial tile.
static int64_t most_row_tiles(int64_t cap, int64_t E, int64_t tm) {
    const int64_t used = (cap + 15) / 16;
    return cap / tm + (E < used ? E : used);
}
bool grouped_gemm_fits(int64_t cap, int64_t E, int64_t N) {
    return most_row_tiles(cap, E, kT) <= INT_MAX / ((N + kT) / kT);
}
bool grouped_wgrad_fits(int64_t E, int64_t N, int64_t K) {
    const int64_t per = ((N + kT) / kT) * ((K + kT) / kT);   // at most 2^48
    return E <= INT_MAX / per;
}

hipError_t launch_grouped_gemm(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st) {
    const int tiles_n = (g.N + kT - 1) / kT;
    const dim3 grid((unsigned)(most_row_tiles(g.cap, g.E, kT) * tiles_n));
#define FP8DS_GG(FA_, FB_, O_) k_grouped_gemm<FA_, FB_, O_><<<grid, kThreads, 0, st>>>(g, tiles_n)
    FP8DS_GROUPED_SWITCH(FP8DS_GG)
#undef FP8DS_GG
    return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st) {
    const int tiles_m = (g.N + kT - 1) / kT, tiles_n = (g.K + kT - 1) / kT;
    const dim3 grid((unsigned)((int64_t)g.E * tiles_m * tiles_n));
#define FP8DS_GW(FA_, FB_, O_) k_grouped_wgrad<FA_, FB_, O_><<<grid, kThreads, 0, st>>>(g, tiles_m, tiles_n)
    FP8DS_GROUPED_SWITCH(FP8DS_GW)
#undef FP8DS_GW
    return hipGetLastError();
}

}  // namespace fp8ds
