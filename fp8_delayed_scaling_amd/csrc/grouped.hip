// grouped.hip -- the experts' FP8 products over tokens sorted by expert, on gfx950 matrix cores.
//
//   forward / input gradient   D[r, :] = A[r, :] B[e]^T * a_scale_inv * b_scale_inv   for the rows r of expert e
//   weight gradient            D[e] = A[:, rows of e] B[:, rows of e]^T * (the same)
//
// offsets[e] .. offsets[e + 1] are expert e's rows, read on the device: the host never learns
// them.  Both operands are K-contiguous and accumulate in float32; the one product order per output
// is fixed, so results do not depend on the routing of other experts.  Offsets are held to [0, cap]
// and to multiples of 16 as they are read, and the number of tiles to what offsets in order can give, so
// no content of the buffer makes an access out of bounds or a search without end.
//
// Two kernels, both of four waves (2 x 2, each up to 128 x 128 made of v_mfma_f32_16x16x128_f8f6f4
// tiles) that take one tile after the other, the first loads of a tile in flight while the tile
// before is written:
//   Wide    up to 256 rows of A by 256 rows of B, one block on each CU: the fewest bytes per product
//   Paired  up to 128 rows by 256, two blocks on each CU, which fill each other's waits: for short
//           contractions, small problems and few rows per expert
// Measured: 64 experts, [2048, 4096], 32768 rows: evenly routed forward 239 us (2.3 PFLOP/s; a dense
// product of that size 197), unevenly 262-268 (2.1, bound by the products and by the 537 MB of
// weights in turn), weight gradient 496-504 (1.07 GB of output), 64 rows 54-57 us (341 MB, 6.2 TB/s).
// An expert's rows are shared evenly among its tiles, in steps of 32 (16 for each row of waves); a
// tile runs only the 16-row blocks it has.  All loads are buffer loads into LDS whose bound is the
// tile's extent: rows past it, and the 16-byte pieces past K (their offset is moved out of the bound),
// arrive as zeros without touching memory.  The bound is compared with the lane's offset after the
// scalar offset is taken off it, so the scalar offset stays inside the tile's K bytes too.
#include <climits>
#include <type_traits>

#include "../../include/fp8ds.h"
#include "device_common.h"
#include "launch.h"

namespace fp8ds {

namespace {

constexpr int kWide = 256, kPaired = 128;    // most rows of a tile
constexpr int kTn = 256;                     // its columns (rows of B)
constexpr int kStep = 128;                   // K bytes per step
constexpr int kThreads = 256;
constexpr int kCUs = 256;
constexpr int kXcds = 8;                     // blocks are dealt round-robin to the XCDs
constexpr int kLog2Run = 3;                  // tiles that follow each other on one XCD, in the forward
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every tile's extent (below 2^31 bytes)
constexpr int kStreaming = 2;                // nontemporal
constexpr int kBufDesc3 = 0x00020000;        // raw buffer descriptor, bounds checked in bytes

// vmcnt-only wait, and a workgroup barrier without a fence (a fenced one would wait for every load
// in flight); the empty asm statements keep memory accesses on their side.
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

// Division by a number that is the same for all tiles: opaque, so that no reciprocal is kept from one
// tile to the next in a register (there is none to spare, and a reload would wait for all stores).
__device__ __forceinline__ int divide(int n, int d) {
    asm volatile("" : "+s"(d));
    return (int)((uint32_t)n / (uint32_t)d);
}
__device__ __forceinline__ int divide_any(int n, int d) { return (int)((uint32_t)n / (uint32_t)d); }
__device__ __forceinline__ int modulo(int n, int d) { return n - divide(n, d) * d; }

// Rows of each of the tiles of at most tm rows (32, 64, 128 or 256) that share n rows: ceil(n / tm)
// tiles, the same multiple of 32 each (the last may have fewer, never none).
__host__ __device__ inline int tile_rows(int n, int tm) {
    const int tiles = (n + tm - 1) / tm, blocks = (n + 31) / 32;
    return tiles > 0 ? (blocks + tiles - 1) / tiles * 32 : 0;
}

// The largest number of row tiles of at most tm rows that offsets in order can give: every expert with
// rows adds at most one partial tile.
__host__ __device__ inline int64_t most_row_tiles(int64_t cap, int64_t E, int64_t tm) {
    const int64_t used = (cap + 15) / 16;
    return cap / tm + (E < used ? E : used);
}

// A tile's operands and output, uniform over the block.
struct Tile {
    const uint8_t *A, *B;
    void *D;
    int rows, cols, K;
};

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);      // row_shr:1, 2, 4, 8 inside 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);      // row_bcast:15, then 31
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

// The forward's tiles, an expert's ceil(rows / tile height) * tiles_n with its row tiles running fastest.
// Among 64 experts, tall tiles come first (in every expert all tiles but the last have one height).
// The tiles are taken in rounds, runs of 8 (single ones, where an XCD has fewer blocks) dealt to the
// XCDs forwards and backwards in turn, a run to blocks of one XCD: they share B's rows, which come
// from HBM once, and A's.  Every block so takes a like mixture of heights, and half of the blocks take
// theirs from the last round to the first: tall tiles, bound by the products, run beside low ones, bound
// by B's bytes.  (Unevenly routed forward of 64 experts, half of which have under 1 % of the rows, when
// this was chosen: in the experts' order 330 us, tall tiles first 286, this way 275.)
template <int OUT>
struct RowTiles {
    const Grouped &g;
    int log2_tm, tiles_n, log2_run, total, deals, round, e0, before;      // before: tiles before those of the experts e0 .. e0 + 63
    __device__ __forceinline__ RowTiles(const Grouped &g_, int log2_tm_, int tiles_n_)
        : g(g_), log2_tm(log2_tm_), tiles_n(tiles_n_), log2_run(gridDim.x >= kXcds << kLog2Run ? kLog2Run : 0), total(0), round(0), e0(0), before(0) {
        // Offsets that fall may count rows for several experts, without end: past what offsets in order
        // can give, nothing is computed.  So every number of tiles below fits in 31 bits.
        const uint32_t most = (uint32_t)most_row_tiles(g.cap, g.E, 1 << log2_tm);
        uint32_t all = 0;
        int lo, hi;
        for (int e = 0; e < g.E; e += 64) all = min(all + row_tiles(e, lo, hi), most + 1);
        total = uniform(all <= most ? (int)all * tiles_n : 0);
        deals = (total + (kXcds << log2_run) - 1) / (kXcds << log2_run);
    }
    __device__ __forceinline__ int tiles_of(int n) const { return (n + (1 << log2_tm) - 1) >> log2_tm; }
    // row tiles of the experts e .. e + 63 (below 2^31), and the rows of the lane's among them
    __device__ __forceinline__ uint32_t row_tiles(int e, int &lo, int &hi) const {
        const int i = e + (threadIdx.x & 63);
        lo = hi = 0;
        if (i < g.E) {
            lo = min(max(g.offsets[i], 0), g.cap) & ~15;
            hi = max(lo, min(max(g.offsets[i + 1], 0), g.cap) & ~15);
        }
        return (uint32_t)uniform(__builtin_amdgcn_readlane(wave_scan(tiles_of(hi - lo)), 63));
    }
    __device__ __forceinline__ int count(int e, int &lo, int &hi) const { return (int)row_tiles(e, lo, hi) * tiles_n; }
    // the block's next tile; false when there is none
    __device__ __forceinline__ bool operator()(Tile &t) {
        const int slots = gridDim.x / kXcds, slot = blockIdx.x / kXcds, xcd = blockIdx.x % kXcds;
        const int rounds = divide((deals << log2_run) + slots - 1, slots);
        int tile;
        for (;; ++round) {
            if (round >= rounds) return false;
            const int r = (slot >> log2_run) & 1 ? rounds - 1 - round : round;
            const int l = r * slots + (r & 1 ? slots - 1 - slot : slot), deal = l >> log2_run;
            tile = ((deal * kXcds + (deal & 1 ? kXcds - 1 - xcd : xcd)) << log2_run) + (l & ((1 << log2_run) - 1));
            if (tile < total) break;
        }
        ++round;
        int lo, hi, n = count(e0, lo, hi);
        while (tile < before) {
            e0 -= 64;
            n = count(e0, lo, hi);
            before -= n;
        }
        while (tile >= before + n) {
            before += n;
            e0 += 64;
            n = count(e0, lo, hi);
        }
        int at = tile - before, h = 1 << (log2_tm - 5);
        const int blocks = (hi - lo + 31) >> 5, n_tiles = tiles_of(hi - lo);
        int mine = 0;                      // the lane's expert's height: its 32-row blocks shared by its tiles
        if (n_tiles > 0) mine = divide_any(blocks + n_tiles - 1, n_tiles);
        for (; h > 1; --h) {
            const int of_h = uniform(__builtin_amdgcn_readlane(wave_scan(mine == h ? tiles_of(hi - lo) : 0), 63)) * tiles_n;
            if (at < of_h) break;
            at -= of_h;
        }
        const int tiles = mine == h ? tiles_of(hi - lo) : 0, incl = wave_scan(tiles);
        const int k = __builtin_ctzll(__ballot(incl * tiles_n > at)), e = e0 + k;
        const int first = __builtin_amdgcn_readlane(lo, k), end = __builtin_amdgcn_readlane(hi, k);
        const int row_tiles = __builtin_amdgcn_readlane(tiles, k), in = at - __builtin_amdgcn_readlane(incl - tiles, k) * tiles_n;
        const int tn = divide(in, row_tiles), row = first + (in - tn * row_tiles) * h * 32;
        constexpr int kEsz = OUT == 0 ? 2 : 4;
        t = Tile{g.A + (int64_t)row * g.lda, g.B + (int64_t)e * g.stride_b + (int64_t)tn * kTn * g.ldb,
                 static_cast<uint8_t *>(g.D) + ((int64_t)row * g.ldd + tn * kTn) * kEsz, min(h * 32, end - row),
                 min(kTn, g.N - tn * kTn), g.K};
        return true;
    }
};

// Scalar loads: the offsets are not written while the kernel runs, and a vector load would wait
// for every store in flight before it.
__device__ __forceinline__ int offset_at(const Grouped &g, int e) {
    const auto *o = reinterpret_cast<const __attribute__((address_space(4))) int32_t *>(reinterpret_cast<uint64_t>(g.offsets));
    return min(max(o[uniform(e)], 0), g.cap) & ~15;
}

// The weight gradient's tiles.  Every XCD takes an eighth of each expert's tiles, whatever the
// routing, so that it reads few of the operands' rows and keeps them in its L2: half of the row
// tiles by a quarter of the columns where the row tiles are even (547 us with all row tiles by an
// eighth, 535 this way), else all by an eighth.  Which eighth moves with the expert, so that
// remainders spread.  Where two to four experts' eighths fill
// an XCD's blocks, those form as many groups, and each expert goes to the group that has the least
// work so far (a tile costs its K steps and about three for its output); else the tiles are taken
// in order, shifted by some blocks in every round.
template <int OUT>
struct ExpertTiles {
    const Grouped &g;
    int tiles_m, tiles_n, h, per, chunk, slots, groups, next;      // next: round, or expert with groups
    int work[4];
    __device__ __forceinline__ ExpertTiles(const Grouped &g_, int tiles_m_, int tiles_n_)
        : g(g_), tiles_m(tiles_m_), tiles_n(tiles_n_), h(tile_rows(g_.N, kPaired)), next(0) {
        per = tiles_m * tiles_n;
        chunk = (per + kXcds - 1) / kXcds;
        slots = gridDim.x / kXcds;
        groups = slots / chunk;
        if (groups < 2 || groups > 4 || groups * chunk * 10 < slots * 9) groups = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) work[i] = i < groups ? 0 : INT_MAX;
    }
    __device__ __forceinline__ bool operator()(Tile &t) {
        const int slot = blockIdx.x / kXcds, xcd = blockIdx.x % kXcds;
        int e, in;
        if (groups > 0) {
            const int mine = divide(slot, chunk);
            for (;; ++next) {
                if (next >= g.E || mine >= groups) return false;
                const int cost = (max(0, offset_at(g, next + 1) - offset_at(g, next)) + kStep - 1) / kStep + 3;
                int least = 0, w = work[0];
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    if (work[i] < w) { w = work[i]; least = i; }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i == least) work[i] += cost;
                e = next;
                in = slot - mine * chunk + (xcd + e) % kXcds * chunk;
                if (least == mine && in < per) break;
            }
            ++next;
        } else {
            const int total = g.E * chunk;                             // 31 bits
            for (;; ++next) {
                if (next * slots >= total) return false;
                const int at = next * slots + modulo(slot + next * 11, slots);
                e = divide(at, chunk);
                in = at - e * chunk + (xcd + e) % kXcds * chunk;
                if (at < total && in < per) break;
            }
            ++next;
        }
        const int stripe = tiles_m % 2 == 0 ? tiles_m / 2 : tiles_m, s = divide(in, stripe * tiles_n), q = in - s * stripe * tiles_n;
        const int tn = divide(q, stripe), tm = s * stripe + q - tn * stripe;
        const int lo = offset_at(g, e), len = max(0, offset_at(g, e + 1) - lo);
        constexpr int kEsz = OUT == 0 ? 2 : 4;
        t = Tile{g.A + (int64_t)tm * h * g.lda + lo, g.B + (int64_t)tn * kTn * g.ldb + lo,
                 static_cast<uint8_t *>(g.D) + ((int64_t)e * g.stride_d + (int64_t)tm * h * g.ldd + tn * kTn) * kEsz,
                 min(h, g.N - tm * h), min(kTn, g.K - tn * kTn), len};
        return true;
    }
};

// The 16-byte piece c of row r of a slot sits at piece c ^ swz(r) of its 128 bytes, so that the 16
// lanes of one phase of a fragment read (lanes 0-3, 12-15, 20-23, 24-27 and so on: two K groups) hit
// distinct banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// B's rows lie in a slot in the order that the output wants.  Row 128 n + 16 q + m is row m of wave
// column n's fragment q and holds the column col_of(q, m) of its 128: a lane, which has one m, then
// has 16 bytes of consecutive columns of a row in its accumulators of 8 (bfloat16) or 4 (float32)
// fragments, and 16 lanes have 256, which one store instruction writes for each of four rows.
template <int OUT> __device__ __forceinline__ int col_of(int q, int m) {
    return OUT == 0 ? 8 * m + q : 64 * (q >> 2) + 4 * m + (q & 3);
}

// What both kernels share: the loads, the fragments and the output.
template <int FA, int FB, int OUT, bool STREAM>
struct Work {
    int64_t ldd;
    float sa, sb;
    int lda, ldb, wave, wm, wn;

    explicit __device__ __forceinline__ Work(const Grouped &gr)
        : ldd(gr.ldd), sa(*gr.a_sinv), sb(*gr.b_sinv), lda((int)gr.lda), ldb((int)gr.ldb) {
        wave = uniform((int)threadIdx.x >> 6);
        wm = wave >> 1; wn = wave & 1;
    }
    // The lane, as a value the compiler cannot see through: what depends on it is formed anew for
    // each tile, not kept in registers (or worse, in memory) from one to the next.
    static __device__ __forceinline__ int fresh_lane() {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        return lane;
    }
    // Load i of a slot: wave w fills its 1 KB block 4 i + w, rows 32 i + 8 w .. + 7; lane l row l / 8,
    // stored piece l % 8.
    struct Loads {
        int k;                   // K byte of the lane's piece inside a step
        uint32_t va, vb;         // the lane's offset in a slot's first load
    };
    __device__ __forceinline__ Loads loads_of(int lane) const {
        const int row = wave * 8 + (lane >> 3), k = ((lane & 7) ^ swz(row)) * 16;
        return Loads{k, (uint32_t)(row * lda + k), (uint32_t)(col_of<OUT>(row >> 4, row & 15) * ldb + k)};
    }
    // Tiles' extents are below 2^31 bytes.  The descriptor has to be in scalar registers.
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const uint8_t *p, int64_t bytes) {
        const uint64_t a = reinterpret_cast<uint64_t>(p);
        const uint64_t u = (uint64_t)(uint32_t)uniform((int)a) | (uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32;
        return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(u), (short)0, uniform((int)bytes), kBufDesc3);
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint8_t *slot, int i, uint32_t off, int k0) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)(slot + (i * 4 + wave) * 1024), 16, off,
                                                 (uint32_t)k0, 0, 0);
    }
    // K byte of step j's first piece: the loads' scalar offset, the last step's for one past it (all its
    // pieces are outside)
    static __device__ __forceinline__ int first_byte(int nk, int j) { return uniform(min(j, nk - 1) * kStep); }
    static __device__ __forceinline__ uint32_t outside(const Tile &t, int j, int piece) {
        return j * kStep + piece < t.K ? 0u : kOutside;
    }
    static __device__ __forceinline__ i32x8 frag(const uint8_t *p, int o0, int o1) {
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(p + o0);
        const u32x4 hi = *reinterpret_cast<const u32x4 *>(p + o1);
        i32x8 v;
        v[0] = (int)lo.x; v[1] = (int)lo.y; v[2] = (int)lo.z; v[3] = (int)lo.w;
        v[4] = (int)hi.x; v[5] = (int)hi.y; v[6] = (int)hi.z; v[7] = (int)hi.w;
        return v;
    }

    // row of B, after the lane's in the first load, that load i takes: slot rows 32 i .. are fragments 2 i and 2 i + 1
    static __device__ __forceinline__ constexpr int row_b(int i) { return (i >> 2) * 128 + (OUT == 0 ? 2 * (i & 3) : 64 * ((i >> 1) & 1) + 2 * (i & 1)); }
    static __device__ __forceinline__ int steps(const Tile &t) { return max(1, (uniform(t.K) + kStep - 1) / kStep); }   // K = 0: one of zeros
    // lane l holds row 32 i + 16 wm + 4 (l / 16) + u, column col_of(q, l % 16), in element u of acc[i][q]
    template <int NB>
    __device__ __forceinline__ void store(const Tile &t, const f32x4 (&acc)[NB][8]) const {
        constexpr int kEsz = OUT == 0 ? 2 : 4, kPer = 16 / kEsz;      // elements of a 16-byte store
        const bool vec = (reinterpret_cast<uintptr_t>(t.D) & 15) == 0 && ldd % kPer == 0 && t.cols % kPer == 0;
        const int lane = fresh_lane(), col0 = wn * 128 + col_of<OUT>(0, lane & 15), row0 = wm * 16 + (lane >> 4) * 4;
        const uint32_t at = (uint32_t)((row0 * (int)ldd + col0) * kEsz);      // 32 rows are less than 2^30 bytes
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const auto rs = bounded(static_cast<const uint8_t *>(t.D) + (int64_t)(i * 32) * ldd * kEsz, 0x7fffffff);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t here = i * 32 + row0 + u < t.rows ? at + (uint32_t)(u * (int)ldd * kEsz) : kOutside;
#pragma unroll
                for (int p = 0; p < 8 / kPer; ++p) {
                    u32x4 w;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if constexpr (OUT == 0)
                            w[h] = f32x2_to_bf16x2_rne(dequant_bias(acc[i][2 * h][u], sa, sb, 0.f), dequant_bias(acc[i][2 * h + 1][u], sa, sb, 0.f));
                        else
                            w[h] = __float_as_uint(dequant_bias(acc[i][4 * p + h][u], sa, sb, 0.f));
                    }
                    if (vec) {
                        const uint32_t off = col0 + p * 64 < t.cols ? here + (uint32_t)(p * 64 * kEsz) : kOutside;
                        __builtin_amdgcn_raw_buffer_store_b128(w, rs, (int)off, 0, STREAM ? kStreaming : 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const uint32_t off = col0 + p * 64 + e < t.cols ? here + (uint32_t)((p * 64 + e) * kEsz) : kOutside;
                            if constexpr (OUT == 0)
                                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w[e >> 1] >> (16 * (e & 1))), rs, (int)off, 0, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b32(w[e], rs, (int)off, 0, 0);
                        }
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Wide.  LDS holds two K steps of A and three of B, 160 KB in all.  Step j
// multiplies A_j, its fragments read one 16-row block ahead of the MFMAs, by B_j, whose fragments
// were read into registers during step j - 1; it reads the fragments of B_{j+1}, loads B_{j+3} into
// B_j's slot, before its last block waits for A_{j+1} and B_{j+2}, and in that block loads A_{j+2}
// into A_j's slot.  So A_j, B_j and B_{j+1} have arrived in every wave's part before step j begins:
// for step 0 by the wait at the tile's start.  A is read by several tiles at a time and comes from
// L2, B from HBM.
template <int FA, int FB, int OUT, bool STREAM>
struct Wide : Work<FA, FB, OUT, STREAM> {
    using W = Work<FA, FB, OUT, STREAM>;
    using Loads = typename W::Loads;
    using W::loads_of;
    using W::fresh_lane;
    using W::bounded;
    using W::load;
    using W::outside;
    using W::first_byte;
    using W::frag;
    using W::row_b;
    using W::steps;
    using W::lda;
    using W::ldb;
    using W::wm;
    using W::wn;
    using W::store;
    uint8_t *sa0, *sa1, *sb0, *sb1, *sb2;
    __device__ __forceinline__ Wide(const Grouped &g, uint8_t *a0, uint8_t *a1, uint8_t *b0, uint8_t *b1, uint8_t *b2)
        : W(g), sa0(a0), sa1(a1), sb0(b0), sb1(b1), sb2(b2) {}
    // The steps' slots and registers repeat with period 6; a tile starts at the phase that lets its
    // last step be the sixth.
    static __device__ __forceinline__ int phase(int nk) { return (6 - nk % 6) % 6; }
    static __device__ __forceinline__ uint8_t *pick(bool c, uint8_t *x, uint8_t *y) { return c ? x : y; }
    __device__ __forceinline__ uint8_t *slot_a(int p) const { return pick(p & 1, sa1, sa0); }
    __device__ __forceinline__ uint8_t *slot_b(int p) const { return pick(p % 3 == 0, sb0, pick(p % 3 == 1, sb1, sb2)); }

    // A tile's first loads, all five slots, in the order of their waits: A_0, B_0 and B_1, which
    // step 0 reads, then A_1 and B_2, which it waits for itself (kLater loads).
    static constexpr int kLater = 16;
    __device__ __forceinline__ void first_loads(const Tile &t) const {
        const int nk = steps(t), p = phase(nk);
        const Loads ld = loads_of(fresh_lane());
        const auto rs_a = bounded(t.A, (int64_t)t.rows * lda), rs_b = bounded(t.B, (int64_t)t.cols * ldb);
        auto load_a = [&](int j) {
            const uint32_t out = outside(t, j, ld.k);
            uint8_t *const a = slot_a(p + j);
            const int k0 = first_byte(nk, j);
#pragma unroll
            for (int i = 0; i < 8; ++i) load(rs_a, a, i, (ld.va | out) + i * 32 * lda, k0);
        };
        auto load_b = [&](int j) {
            const uint32_t out = outside(t, j, ld.k);
            uint8_t *const b = slot_b(p + j);
            const int k0 = first_byte(nk, j);
#pragma unroll
            for (int i = 0; i < 8; ++i) load(rs_b, b, i, (ld.vb | out) + row_b(i) * ldb, k0);
        };
        load_a(0);
        load_b(0);
        load_b(1);
        __builtin_amdgcn_sched_barrier(0);
        load_a(1);
        load_b(2);
        __builtin_amdgcn_sched_barrier(0);
    }

    // Waits for all loads but the last N before `stores` (at least that many) output stores: those
    // may be in flight too.
    template <int N>
    static __device__ __forceinline__ void wait_before_stores(int stores) {
        asm volatile("" ::: "memory");
        if (stores >= 32) FP8DS_WAIT_VM(N + 32);
        else if (stores >= 16) FP8DS_WAIT_VM(N + 16);
        else FP8DS_WAIT_VM(N);
    }

    // Products of a tile of at most 32 NB rows, then the next tile's first loads, then the output.
    // `stores`: those of the tile before, still in flight.  Returns this tile's.
    template <int NB, class Tiles>
    __device__ __forceinline__ int run(const Tile &t, Tiles &tiles, Tile &next, bool &more, int stores) const {
        f32x4 acc[NB][8];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int nk = steps(t);
        const int lane = fresh_lane(), r16 = lane & 15, g = lane >> 4;
        const Loads ld = loads_of(lane);
        // fragments: the second piece of the lane's 32 bytes is the first's neighbour
        const int o = r16 * kStep + (((2 * g) ^ swz(r16)) << 4), oa = wm * 16 * kStep + o, ob = wn * 128 * kStep + o;
        auto frag_a = [&](const uint8_t *slot, int i) { return frag(slot + i * 32 * kStep, oa, oa ^ 16); };
        auto frag_b = [&](const uint8_t *slot, int q) { return frag(slot + q * 16 * kStep, ob, ob ^ 16); };
        const auto rs_a = bounded(t.A, (int64_t)t.rows * lda), rs_b = bounded(t.B, (int64_t)t.cols * ldb);
        i32x8 fb0[8], fb1[8], fa[2];
        constexpr int kBlocks = NB - 1;
        auto mfma = [&](int i, const i32x8 &a, const i32x8 (&b)[8]) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                acc[i][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[q], acc[i][q], FA, FB, 0, 0, 0, 0);
        };
        auto interleave = [](int n) {
#pragma unroll
            for (int q = 0; q < n; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            }
        };
        // P: the phase's parity; block i's A fragment is fa[(P NB + i) % 2]
        auto step = [&](auto pc, int j, uint8_t *a_cur, uint8_t *a_nxt, uint8_t *b_nxt, uint8_t *b_free, const i32x8 (&fbc)[8],
                        i32x8 (&fbn)[8]) {
            constexpr int P = decltype(pc)::value;
            const uint32_t out_b = outside(t, j + 3, ld.k);
            const int k_b = first_byte(nk, j + 3);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                fa[(P * NB + i + 1) & 1] = frag_a(a_cur, i + 1);
#pragma unroll
                for (int q = 8 * i / kBlocks; q < 8 * (i + 1) / kBlocks; ++q) {
                    fbn[q] = frag_b(b_nxt, q);
                    load(rs_b, b_free, q, (ld.vb | out_b) + row_b(q) * ldb, k_b);
                }
                mfma(i, fa[(P * NB + i) & 1], fbc);
                interleave(8);
                __builtin_amdgcn_sched_barrier(0);
            }
            // In flight: B_{j+3}, loaded above.  In step 0 its eight loads follow the stores of the tile
            // before, which follow A_1 and B_2.
            if (j == 0) wait_before_stores<8>(stores);
            else FP8DS_WAIT_VM(8);
            FP8DS_WAIT_LGKM();
            FP8DS_BARRIER();
            __builtin_amdgcn_sched_barrier(0);
            const i32x8 last = fa[(P * NB + NB - 1) & 1];
            fa[(P * NB + NB) & 1] = frag_a(a_nxt, 0);
            const uint32_t out_a = outside(t, j + 2, ld.k);
            const int k_a = first_byte(nk, j + 2);
#pragma unroll
            for (int n = 0; n < NB; ++n) load(rs_a, a_cur, n, (ld.va | out_a) + n * 32 * lda, k_a);
            mfma(NB - 1, last, fbc);
            interleave(8);
            __builtin_amdgcn_sched_barrier(0);
        };
        const int p = phase(nk);
        wait_before_stores<kLater>(stores);                  // A_0, B_0 and B_1; in flight: A_1, B_2, the stores
        FP8DS_BARRIER();
        {
            const uint8_t *b = slot_b(p), *a = slot_a(p);
#pragma unroll
            for (int q = 0; q < 8; ++q) fb0[q] = fb1[q] = frag_b(b, q);
            fa[0] = fa[1] = frag_a(a, 0);
        }
        FP8DS_WAIT_LGKM();
        FP8DS_BARRIER();
        __builtin_amdgcn_sched_barrier(0);
        const std::integral_constant<int, 0> even{};
        const std::integral_constant<int, 1> odd{};
        int j = -p;
        do {
            if (j >= 0) step(even, j, sa0, sa1, sb1, sb0, fb0, fb1);
            if (j + 1 >= 0) step(odd, j + 1, sa1, sa0, sb2, sb1, fb1, fb0);
            if (j + 2 >= 0) step(even, j + 2, sa0, sa1, sb0, sb2, fb0, fb1);
            if (j + 3 >= 0) step(odd, j + 3, sa1, sa0, sb1, sb0, fb1, fb0);
            if (j + 4 >= 0) step(even, j + 4, sa0, sa1, sb2, sb1, fb0, fb1);
            step(odd, j + 5, sa1, sa0, sb0, sb2, fb1, fb0);
            j += 6;
        } while (j < nk);
        FP8DS_WAIT_ALL();                                    // every load into the slots has landed
        FP8DS_BARRIER();
        __builtin_amdgcn_sched_barrier(0);
        more = tiles(next);                                  // nothing is in flight that its loads would wait for
        if (more) first_loads(next);
        this->template store<NB>(t, acc);
        return NB * (OUT == 0 ? 4 : 8);
    }

};

// Paired.  LDS holds one K step of A and two of B, 80 KB: two blocks share a
// CU.  Step j waits for A_j and B_j, reads all their fragments into registers, and after a barrier
// loads A_{j+1} and B_{j+2} into the slots so freed while its MFMAs run; the other block's MFMAs
// fill the time of the reads and waits, and its loads that of the output.  A is read by several
// tiles at a time and comes from L2; B, from HBM, has two steps to arrive.
template <int FA, int FB, int OUT, bool STREAM>
struct Paired : Work<FA, FB, OUT, STREAM> {
    using W = Work<FA, FB, OUT, STREAM>;
    using Loads = typename W::Loads;
    using W::loads_of;
    using W::fresh_lane;
    using W::bounded;
    using W::load;
    using W::outside;
    using W::first_byte;
    using W::frag;
    using W::row_b;
    using W::steps;
    using W::lda;
    using W::ldb;
    using W::wm;
    using W::wn;
    using W::store;
    uint8_t *sa0, *sb0, *sb1;
    __device__ __forceinline__ Paired(const Grouped &g, uint8_t *a0, uint8_t *b0, uint8_t *b1) : W(g), sa0(a0), sb0(b0), sb1(b1) {}
    // B's slots alternate; a tile starts with the one that lets its last step use the second.
    __device__ __forceinline__ uint8_t *slot_b(int p) const {
        uint8_t *const x = sb0, *const y = sb1;
        return p & 1 ? y : x;
    }

    // A tile's first loads: B_0 and A_0, then B_1.
    __device__ __forceinline__ void first_loads(const Tile &t) const {
        const int nk = steps(t), p = nk & 1;
        const Loads ld = loads_of(fresh_lane());
        const auto rs_a = bounded(t.A, (int64_t)t.rows * lda), rs_b = bounded(t.B, (int64_t)t.cols * ldb);
        const uint32_t out0 = outside(t, 0, ld.k), out1 = outside(t, 1, ld.k);
        const int k1 = first_byte(nk, 1);
        uint8_t *b0 = slot_b(p), *b1 = slot_b(p + 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) load(rs_b, b0, i, (ld.vb | out0) + row_b(i) * ldb, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) load(rs_a, sa0, i, (ld.va | out0) + i * 32 * lda, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) load(rs_b, b1, i, (ld.vb | out1) + row_b(i) * ldb, k1);
        __builtin_amdgcn_sched_barrier(0);
    }

    // Products of a tile of at most 32 NB rows, then the next tile's first loads, then the output.
    template <int NB, class Tiles>
    __device__ __forceinline__ int run(const Tile &t, Tiles &tiles, Tile &next, bool &more, int) const {
        f32x4 acc[NB][8];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[i][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int nk = steps(t);
        const int lane = fresh_lane(), r16 = lane & 15, g = lane >> 4;
        const Loads ld = loads_of(lane);
        // fragments: the second piece of the lane's 32 bytes is the first's neighbour
        const int o = r16 * kStep + (((2 * g) ^ swz(r16)) << 4), oa = wm * 16 * kStep + o, ob = wn * 128 * kStep + o;
        const auto rs_a = bounded(t.A, (int64_t)t.rows * lda), rs_b = bounded(t.B, (int64_t)t.cols * ldb);
        auto step = [&](int j, uint8_t *b) {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            FP8DS_WAIT_VM(8);                                // in flight: B_{j+1}, or stores of the tile before
            FP8DS_BARRIER();
            __builtin_amdgcn_sched_barrier(0);
            i32x8 fa[NB], fb[8];
#pragma unroll
            for (int i = 0; i < NB; ++i) fa[i] = frag(sa0 + i * 32 * kStep, oa, oa ^ 16);
#pragma unroll
            for (int q = 0; q < 8; ++q) fb[q] = frag(b + q * 16 * kStep, ob, ob ^ 16);
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            FP8DS_WAIT_LGKM();
            FP8DS_BARRIER();
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t out_a = outside(t, j + 1, ld.k), out_b = outside(t, j + 2, ld.k);
            const int k_a = first_byte(nk, j + 1), k_b = first_byte(nk, j + 2);
#pragma unroll
            for (int i = 0; i < NB; ++i) load(rs_a, sa0, i, (ld.va | out_a) + i * 32 * lda, k_a);
            __builtin_amdgcn_sched_barrier(0x7cf);           // loads into LDS stay in this order
#pragma unroll
            for (int i = 0; i < 8; ++i) load(rs_b, b, i, (ld.vb | out_b) + row_b(i) * ldb, k_b);
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    acc[i][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[i], fb[q], acc[i][q], FA, FB, 0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < 8 + NB; ++n) {
                __builtin_amdgcn_sched_group_barrier(0x008, NB > 1 ? 2 : 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        int j = -(nk & 1);
        do {
            if (j >= 0) step(j, sb0);
            step(j + 1, sb1);
            j += 2;
        } while (j < nk);
        FP8DS_WAIT_ALL();                                    // every load into the slots has landed
        FP8DS_BARRIER();
        __builtin_amdgcn_sched_barrier(0);
        more = tiles(next);
        if (more) first_loads(next);
        this->template store<NB>(t, acc);
        return 0;
    }

};

template <int FA, int FB, int OUT, bool STREAM, class Tiles>
__device__ __forceinline__ void run_wide(const Grouped &g, Tiles &&tiles) {
    __shared__ __align__(16) uint8_t sa0[256 * kStep];
    __shared__ __align__(16) uint8_t sa1[256 * kStep];
    __shared__ __align__(16) uint8_t sb0[256 * kStep];
    __shared__ __align__(16) uint8_t sb1[256 * kStep];
    __shared__ __align__(16) uint8_t sb2[256 * kStep];
    Tile t, next;
    if (!tiles(t)) return;
    const Wide<FA, FB, OUT, STREAM> w(g, sa0, sa1, sb0, sb1, sb2);
    w.first_loads(t);
    int stores = 0;
    for (bool more = true; more; t = next) {
        const int nb = (t.rows + 31) / 32;
        if (nb <= 2) stores = w.template run<2>(t, tiles, next, more, stores);
        else if (nb <= 4) stores = w.template run<4>(t, tiles, next, more, stores);
        else if (nb == 5) stores = w.template run<5>(t, tiles, next, more, stores);
        else if (nb == 6) stores = w.template run<6>(t, tiles, next, more, stores);
        else if (nb == 7) stores = w.template run<7>(t, tiles, next, more, stores);
        else stores = w.template run<8>(t, tiles, next, more, stores);
    }
}

template <int FA, int FB, int OUT, bool STREAM, class Tiles>
__device__ __forceinline__ void run_paired(const Grouped &g, Tiles &&tiles) {
    __shared__ __align__(16) uint8_t sa0[128 * kStep];
    __shared__ __align__(16) uint8_t sb0[256 * kStep];
    __shared__ __align__(16) uint8_t sb1[256 * kStep];
    Tile t, next;
    if (!tiles(t)) return;
    const Paired<FA, FB, OUT, STREAM> w(g, sa0, sb0, sb1);
    w.first_loads(t);
    for (bool more = true; more; t = next) {
        const int nb = (t.rows + 31) / 32;
        if (nb == 1) w.template run<1>(t, tiles, next, more, 0);
        else if (nb == 2) w.template run<2>(t, tiles, next, more, 0);
        else if (nb == 3) w.template run<3>(t, tiles, next, more, 0);
        else w.template run<4>(t, tiles, next, more, 0);
    }
}

}  // namespace

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(kThreads, 1) void k_grouped_gemm_wide(const Grouped g, int tiles_n) {
    run_wide<FA, FB, OUT, true>(g, RowTiles<OUT>(g, 8, tiles_n));
}
template <int FA, int FB, int OUT>
__global__ __launch_bounds__(kThreads, 2) void k_grouped_gemm_paired(const Grouped g, int log2_tm, int tiles_n) {
    run_paired<FA, FB, OUT, true>(g, RowTiles<OUT>(g, log2_tm, tiles_n));
}
template <int FA, int FB, int OUT, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void k_grouped_wgrad(const Grouped g, int tiles_m, int tiles_n) {
    run_paired<FA, FB, OUT, STREAM>(g, ExpertTiles<OUT>(g, tiles_m, tiles_n));
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

// Tiles are numbered in 31 bits, positions up to a round of blocks past the last.
bool grouped_gemm_fits(int64_t cap, int64_t E, int64_t N) {
    return most_row_tiles(cap, E, 32) <= (INT_MAX - (1 << 16)) / ((N + kTn) / kTn);
}
bool grouped_wgrad_fits(int64_t E, int64_t N, int64_t K) {
    const int64_t per = ((N + kPaired) / kPaired) * ((K + kTn) / kTn) + kXcds;   // at most 2^48
    return E <= (INT_MAX - (1 << 16)) / per;
}
// One or two blocks per CU, fewer for fewer tiles: a multiple of `unit`, so that no XCD has more tiles
// than blocks where others have fewer (unit: the XCDs, times a run where runs are dealt).
static unsigned blocks_for(int64_t tiles, int64_t most, int64_t unit) {
    return (unsigned)(tiles < most ? (tiles + unit - 1) / unit * unit : most);
}
static unsigned forward_blocks(int64_t tiles, int64_t most) {
    return blocks_for(tiles, most, tiles >= kXcds << kLog2Run ? kXcds << kLog2Run : kXcds);
}
// Wide tiles from 192 rows for each expert on and two rounds of them on all CUs.
static bool wide_preferred(const Grouped &g, int tiles_n) {
    return g.cap / g.E >= 192 && (int64_t)g.cap / kWide * tiles_n >= 2 * kCUs;
}

// Paired tiles are at most 128 rows high, lower where even routing would give fewer than one for
// every other CU: more blocks then share the rows (7872 rows over 6 experts, [400, 3056]: 35 us with
// tiles of 32 rows, 24 of 64; 2704 over 4, [240, 3392]: 18.5 and 20.6).
static int paired_log2(const Grouped &g, int tiles_n) {
    int l = 7;
    while (l > 5 && ((int64_t)g.cap >> l) * tiles_n < kCUs / 2) --l;
    return l;
}

// Weight gradients that no cache holds leave L2 first (nontemporal stores): 64 experts' [2048, 4096]
// of 512 rows each, 1.07 GB, 542 us without and 405 with; 270 MB of short rows that do not fill
// their cache lines (64 x [608, 3472], 16 rows each) 60 and 97, 4 MB 19 and 22.  The forward's
// output always does (input gradient of 6002 rows, [2560, 1424]: 60 us without, 54 with).
static bool wgrad_streams(const Grouped &g, int out_dtype) {
    return (int64_t)g.E * g.N * g.K * (out_dtype == FP8DS_OUT_BF16 ? 2 : 4) >= (INT64_C(512) << 20);
}

hipError_t launch_grouped_gemm(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st) {
    const int tiles_n = (g.N + kTn - 1) / kTn;
    const bool wide = wide_preferred(g, tiles_n);
    const int l = paired_log2(g, tiles_n);
    const unsigned grid = wide ? forward_blocks(most_row_tiles(g.cap, g.E, kWide) * tiles_n, kCUs)
                               : forward_blocks(most_row_tiles(g.cap, g.E, 1 << l) * tiles_n, 2 * kCUs);
#define FP8DS_GG(FA_, FB_, O_)                                                                 \
    do {                                                                                       \
        if (wide) k_grouped_gemm_wide<FA_, FB_, O_><<<grid, kThreads, 0, st>>>(g, tiles_n);       \
        else k_grouped_gemm_paired<FA_, FB_, O_><<<grid, kThreads, 0, st>>>(g, l, tiles_n);       \
    } while (0)
    FP8DS_GROUPED_SWITCH(FP8DS_GG)
#undef FP8DS_GG
    return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const Grouped &g, int fa, int fb, int out_dtype, hipStream_t st) {
    const bool stream = wgrad_streams(g, out_dtype);
    const int tiles_m = (g.N + kPaired - 1) / kPaired, tiles_n = (g.K + kTn - 1) / kTn;
    // an XCD's places: an eighth of each expert's tiles, rounded up
    const int64_t places = (int64_t)g.E * (((int64_t)tiles_m * tiles_n + kXcds - 1) / kXcds);
    const unsigned grid = blocks_for(places * kXcds, 2 * kCUs, kXcds);
#define FP8DS_GW(FA_, FB_, O_)                                                                            \
    do {                                                                                                  \
        if (stream) k_grouped_wgrad<FA_, FB_, O_, true><<<grid, kThreads, 0, st>>>(g, tiles_m, tiles_n);   \
        else k_grouped_wgrad<FA_, FB_, O_, false><<<grid, kThreads, 0, st>>>(g, tiles_m, tiles_n);         \
    } while (0)
    FP8DS_GROUPED_SWITCH(FP8DS_GW)
#undef FP8DS_GW
    return hipGetLastError();
}

}  // namespace fp8ds
