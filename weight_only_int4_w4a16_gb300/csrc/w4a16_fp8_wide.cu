// The 8-bit linear for many tokens (the operation of w4a16_fp8.cu):
//
//   y[m, n] = sum_b sx[m, b] sw[n / 128, b] * (sum_{k in block b} x[m, k] w[n, k])
//
// MMA shape: a pair of CTAs (cta_group::2) computes 256 tokens x 256 weight rows,
// the tokens as the MMA's M = 256 (128 per CTA, a token per tensor-memory lane),
// the weight rows as its N = 256 (each CTA loads half of them, the tensor cores
// read both halves): per block of 128 k a CTA loads 32 KB for 8.4 MFLOP, two thirds
// of what a CTA alone would for a tile of 128 x 256.  A lane is a token, so a block's
// scale is one number per thread and 128-column half, sx sw, and adding a block to
// the sums costs one multiply-add per element.
//
//   Roles (640 threads per CTA): warps 0..15 (lane = token, warp / 4 = quarter of
//   the 256 columns) scale and add the blocks' sums and write y; warp 16 streams the
//   CTA's 128 rows of x and its 128 rows of w per block by TMA; warp 17 of the
//   leading CTA issues the pair's products; warps 18 and 19 bring the scales of four
//   blocks at a time to shared memory (loaded by the sum warps themselves, their
//   latency held up the tensor-memory loads).  Two block sums of 256 columns fill the
//   tensor memory: while the tensor cores run one, the other is read.
//
//   Outputs go through shared memory to TMA stores (boxes of 32 tokens x 64
//   columns), where the residual was loaded by TMA before; where N or an address
//   does not allow TMA, the warps copy the same boxes row by row.
//
//   Work: few tiles are split along K between the pairs of a cluster, which exchange
//   their sums through distributed shared memory.  Otherwise whole tiles in turn
//   while every pair has one; what remains beyond the last full round (and that
//   round with it) is cut into equal runs of blocks ("stream-K"), so that no pair
//   waits.  A run is then at least as long as a tile, so a tile has at most two
//   pieces, and the pair that comes last adds the other's: the order of two terms
//   does not change their sum.
//
//   Bound by the turn of the two block sums: a block takes about 900 cycles where its
//   products alone would take 512 (4.80 PFLOP/s over the GPU).  From a block's commit
//   through the tensor-memory loads and multiply-adds of its 256 columns to the next
//   product into the same columns is a chain of about 1500 cycles, and two buffers are
//   all that the tensor memory holds; the operands' and the loads' shared-memory
//   traffic takes the rest.  M 4096, N 34816, K 5120: 563 to 574 us, 2.5 to 2.6 PFLOP/s,
//   136 to 138% of the measured bf16 rate.  From an earlier state that took 580 to 590 us:
//   the same with eight sum warps of 128 columns each; not kept were four buffers of 128
//   columns (650 us), packed multiply-adds (730), three stages (630), five (no change).
//   65 to 256 tokens take a whole tile's time (N 34816, K 5120: 45 to 46 us at 72 to 256
//   tokens, where the weights' bytes would take 27 to 29): two rounds of 40 blocks.
//
// Every mbarrier wait is bounded, as in w4a16_fp8.cu, and the sum warps come to the
// barriers of split tiles whether or not their waits were met.  The cluster barriers
// (after the setup, before the exchange, before the exit) are reached by every
// thread: all that comes before them ends.
#include <cstring>

#include "w4a16_fp8_common.cuh"
#include "w4a16_internal.h"
#include "w4a16_tcgen05.cuh"

namespace w4a16 {
namespace {

using namespace dev;

constexpr int kTileM = 256, kTileN = 256;      // of a pair
constexpr int kHalf = 128;                     // rows of x, and of w, per CTA
constexpr int kStageX = kHalf * kGroup, kStageW = kHalf * kGroup;
constexpr int kStage = kStageX + kStageW;      // 32 KB
constexpr int kStages = 4;
constexpr int kSumWarps = 16;
constexpr int kCols = 64;                      // columns per sum warp
constexpr int kTmaWarp = 16, kMmaWarp = 17;     // 18 and 19 load scales
constexpr int kScaleSlots = 3;                 // batches of four blocks' scales
constexpr int kScaleSlot = kHalf * 16 + 32;    // the tokens' four each, then the two weight blocks'
constexpr int kThreads = 640;                  // five warpgroups
// registers per thread: the launch's, split between the warpgroups
constexpr int kLaunchRegs = 96, kSumRegs = 104, kOtherRegs = 64;
static_assert(4 * kSumRegs + kOtherRegs <= 5 * kLaunchRegs, "the launch's registers");
constexpr int kDBufs = 2;                      // block sums in tensor memory
constexpr int kTmemCols = 512;
constexpr int kMaxSplit = 4;                   // pairs of a cluster
constexpr int kStoreCols = 64;                 // columns per TMA store (a 128-byte row)
constexpr int kStoreBytes = 32 * kStoreCols * 2;  // a warp's staging: 4 KB
static_assert(kStoreCols == kCols, "a warp's outputs are one box");
constexpr int kGroupM = 16;                    // token tiles that share a pass over the weights
constexpr int kBarBytes = (2 * kStages + 2 * kDBufs + kSumWarps + 2 * kScaleSlots) * 8 + 16;
constexpr int kSmem = 1024 + kStages * kStage + kSumWarps * kStoreBytes +
                      kScaleSlots * kScaleSlot + kBarBytes;
constexpr uint32_t kIdesc =  // D f32, A and B e4m3 (0), N = 256, M = 256
    (1u << 4) | ((uint32_t)(kTileN >> 3) << 17) | ((uint32_t)(kTileM >> 4) << 24);

static_assert(kHalf * kTileN * 4 <= kStages * kStage, "a split tile's sums fit the stages");

struct WideParams {
    CUtensorMap xmap;  // x: (K bytes, M rows), box {128, 128}, 128-byte swizzle
    CUtensorMap wmap;  // w: (K bytes, N rows), the same
    CUtensorMap ymap;  // y: (N, M) of 16 bits, box {64, 32}, 128-byte swizzle (kTma)
    CUtensorMap rmap;  // the residual, the same
    const float *xs, *ws;
    const uint16_t *residual;
    uint16_t *y;
    float *partials;     // [2 * pairs][2 CTAs][256 columns][128 tokens] fp32
    unsigned *counters;  // [split tiles][2 CTAs], zero between launches
    int *status;
    int M, N, G, NB;
    int tiles_m, tiles_n;
    int whole;           // tiles that pairs take whole, in turn
    long long split;     // blocks of the other tiles, cut into equal runs
    int ksplit;          // pairs of a cluster that split each tile along K (1: none)
    int scales16;        // four blocks' scales of a row are one aligned 16-byte load
};

// A pair's work, in order: segments (tile t, blocks [j0, j1)).
struct Walk {
    int tile, pairs, pair;
    long long pos, end;
    __device__ __forceinline__ Walk(const WideParams &p)
        : pairs(gridDim.x / 2), pair(blockIdx.x / 2) {
        if (p.ksplit > 1) {  // the pair's part of its cluster's tile
            tile = p.whole;
            const int i = pair % p.ksplit;
            pos = (long long)(pair / p.ksplit) * p.G;
            end = pos + (i + 1) * p.G / p.ksplit;
            pos += i * p.G / p.ksplit;
        } else {
            tile = pair;
            pos = begin(p, pair);
            end = begin(p, pair + 1);
        }
    }
    __device__ __forceinline__ long long begin(const WideParams &p, int b) const {
        return (long long)b * p.split / pairs;
    }
    // the pair whose run holds block i of the split tiles
    __device__ __forceinline__ int owner(const WideParams &p, long long i) const {
        return (int)(((i + 1) * (long long)pairs - 1) / p.split);
    }
    __device__ __forceinline__ bool next(const WideParams &p, int &t, int &j0, int &j1) {
        if (tile < p.whole) {
            t = tile;
            j0 = 0;
            j1 = p.G;
            tile += pairs;
            return true;
        }
        if (pos >= end) return false;
        const int i = (int)(pos / p.G);
        const long long t0 = (long long)i * p.G;
        t = p.whole + i;
        j0 = (int)(pos - t0);
        j1 = (int)((t0 + p.G < end ? t0 + p.G : end) - t0);
        pos = t0 + j1;
        return true;
    }
};

// Tile t's first token and first weight row: groups of kGroupM token tiles pass
// over the weights together, so that a weight tile is read from memory once per
// group and x's rows stay in L2.
__device__ __forceinline__ void tile_at(const WideParams &p, int t, int &m0, int &n0) {
    const int per = kGroupM * p.tiles_n, g = t / per, r = t - g * per;
    const int gm = min(kGroupM, p.tiles_m - g * kGroupM);
    const int n = r / gm;
    m0 = (g * kGroupM + r - n * gm) * kTileM;
    n0 = n * kTileN;
}

// a row's scales of blocks j .. j + 3 (those past the end are not used)
__device__ __forceinline__ float4 load4(const WideParams &p, const float *row, int j) {
    if (p.scales16) return __ldg(reinterpret_cast<const float4 *>(row + j));
    const int e = p.G - 1;
    return make_float4(__ldg(row + j), __ldg(row + min(j + 1, e)), __ldg(row + min(j + 2, e)),
                       __ldg(row + min(j + 3, e)));
}

__device__ __forceinline__ void prefetch_l2(const void *address) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(address));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {  // one rounding each
    if constexpr (kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Rows m .. m + 31, columns n .. n + 63 of the residual into a warp's staging (kIn), or
// of y out of it, for rows that TMA cannot address: 32-bit words where N is even and
// the address allows it, else single elements, 4 rows at a time (their loads together;
// 8 spill more: 1240 tokens, N 33533, K 1440 113 us for 84).
template <bool kIn>
__device__ __forceinline__ void copy_rows(const WideParams &p, uint8_t *staging, int lane, int m,
                                          int n) {
    const bool words = p.N % 2 == 0 && ((uintptr_t)(kIn ? p.residual : p.y) & 3) == 0;
    const int rows = min(32, p.M - m), cols = min(kStoreCols, p.N - n);
    // element (r, c) of the staging, 128-byte swizzled
    auto at = [&](int r, int c) {
        return staging + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2;
    };
    constexpr int kRows = 4;
    __syncwarp();
    for (int r0 = 0; r0 < rows; r0 += kRows) {
        const size_t o = (size_t)(m + r0) * p.N + n;
        if (words) {
            const int c = 2 * lane;
            if (c >= cols) continue;
            uint32_t v[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (r0 + r < rows) {
                    if constexpr (kIn)
                        v[r] = *reinterpret_cast<const uint32_t *>(
                            p.residual + o + (size_t)r * p.N + c);
                    else
                        v[r] = *reinterpret_cast<const uint32_t *>(at(r0 + r, c));
                }
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (r0 + r < rows) {
                    if constexpr (kIn) *reinterpret_cast<uint32_t *>(at(r0 + r, c)) = v[r];
                    else *reinterpret_cast<uint32_t *>(p.y + o + (size_t)r * p.N + c) = v[r];
                }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = lane + 32 * h;
                if (c >= cols) continue;
                uint16_t v[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r0 + r < rows) {
                        if constexpr (kIn) v[r] = p.residual[o + (size_t)r * p.N + c];
                        else v[r] = *reinterpret_cast<const uint16_t *>(at(r0 + r, c));
                    }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r0 + r < rows) {
                        if constexpr (kIn) *reinterpret_cast<uint16_t *>(at(r0 + r, c)) = v[r];
                        else p.y[o + (size_t)r * p.N + c] = v[r];
                    }
            }
        }
    }
    __syncwarp();
}

// 32 tokens' kC columns of y (8 or 16), m = the warp's first token, n = the first
// column: the sums at `sums` (this lane's token, columns kHalf apart) of the CTAs of
// this rank in the cluster's up to kS pairs, loaded all at once and added in K order,
// + residual, one rounding each.  Rows that 16-byte accesses do not fit go through
// `staging` (1 KB of the warp's own), so that they are read and written along the rows.
template <bool kBf16, bool kTma, int kC, int kS>
__device__ __forceinline__ void exchange(const WideParams &p, const float *sums, uint4 *staging,
                                         uint32_t rank, int lane, int m, int n) {
    constexpr int kQ = kC / 8;      // 16-byte pieces per row
    constexpr int kStep = 32 / kC;  // rows per step of the copies along the rows
    const int rows = min(32, p.M - m), cols = min(kC, p.N - n);
    const size_t o = (size_t)(m + lane) * p.N + n;
    uint16_t *cells = reinterpret_cast<uint16_t *>(staging);  // [32 tokens][kC columns]
    const int row0 = lane / kC, col = lane % kC;
    uint4 r[kQ];
    if (p.residual) {
        if constexpr (kTma) {
#pragma unroll
            for (int h = 0; h < kQ; ++h) {
                r[h] = make_uint4(0, 0, 0, 0);
                if (lane < rows && 8 * h < cols)
                    r[h] = *reinterpret_cast<const uint4 *>(p.residual + o + 8 * h);
            }
        } else {
            uint16_t c[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i)
                if (kStep * i + row0 < rows && col < cols)
                    c[i] = p.residual[(size_t)(m + kStep * i + row0) * p.N + n + col];
#pragma unroll
            for (int i = 0; i < kC; ++i) cells[(kStep * i + row0) * kC + col] = c[i];
            __syncwarp();
#pragma unroll
            for (int h = 0; h < kQ; ++h) r[h] = staging[kQ * lane + h];
            __syncwarp();
        }
    }
    float v[kS][kC];
#pragma unroll
    for (int q = 0; q < kS; ++q)
        if (q < p.ksplit) {
            const uint32_t from = map_to_rank(smem_u32(sums), 2 * q + rank);
            // only what is stored below (the staging takes everything): a load that
            // nothing waits for could be on its way when the other CTA has left
#pragma unroll
            for (int i = 0; i < kC; ++i)
                v[q][i] = !kTma || (lane < rows && (i & ~7) < cols)
                              ? ld_cluster(from + i * kHalf * 4) : 0.f;
        }
    uint32_t out[kC / 2];
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
        float lo = v[0][2 * i], hi = v[0][2 * i + 1];
#pragma unroll
        for (int q = 1; q < kS; ++q)
            if (q < p.ksplit) {
                lo += v[q][2 * i];
                hi += v[q][2 * i + 1];
            }
        if (p.residual) {
            const uint4 w = r[i / 4];
            const uint32_t e = i % 4 == 0 ? w.x : i % 4 == 1 ? w.y : i % 4 == 2 ? w.z : w.w;
            lo += half_bits_to_float((uint16_t)e, kBf16);
            hi += half_bits_to_float((uint16_t)(e >> 16), kBf16);
        }
        out[i] = pack16<kBf16>(lo, hi);
    }
#pragma unroll
    for (int h = 0; h < kQ; ++h) {
        const uint4 y = make_uint4(out[4 * h], out[4 * h + 1], out[4 * h + 2], out[4 * h + 3]);
        if constexpr (!kTma)
            staging[kQ * lane + h] = y;
        else if (lane < rows && 8 * h < cols)  // what allows TMA allows 16-byte stores
            *reinterpret_cast<uint4 *>(p.y + o + 8 * h) = y;
    }
    if constexpr (!kTma) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kC; ++i)
            if (kStep * i + row0 < rows && col < cols)
                p.y[(size_t)(m + kStep * i + row0) * p.N + n + col] =
                    cells[(kStep * i + row0) * kC + col];
        __syncwarp();
    }
}

// kTma: y (and the residual) can go by TMA.  The copies of the other case stay out of
// this one's registers: in one kernel they cost its products 17%.
template <bool kBf16, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_wide_kernel(const __grid_constant__ WideParams p) {
    extern __shared__ uint8_t smem_raw[];
    // the same offsets in both CTAs: the products read both shared memories at
    // the leader's addresses
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sm_store = smem + kStages * kStage;
    uint8_t *sm_scales = sm_store + kSumWarps * kStoreBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_scales + kScaleSlots * kScaleSlot);
    uint64_t *empty = full + kStages;      // this CTA's stage read
    uint64_t *d_full = empty + kStages;    // a block's sums ready
    uint64_t *d_empty = d_full + kDBufs;   // (leader) read by both CTAs
    uint64_t *r_full = d_empty + kDBufs;   // [sum warp] its residual landed
    uint64_t *sc_full = r_full + kSumWarps;  // [scale slot]
    uint64_t *sc_empty = sc_full + kScaleSlots;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sc_empty + kScaleSlots);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_last = const_cast<int *>(abort + 1);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1, leader = crank & ~1u;

    grid_dependents_launch();
    if (threadIdx.x == kTmaWarp * 32) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), 1);
        }
        for (int i = 0; i < kDBufs; ++i) {
            mbar_init(smem_u32(d_full + i), 1);
            mbar_init(smem_u32(d_empty + i), 2 * kSumWarps);
        }
        for (int i = 0; i < kSumWarps; ++i) mbar_init(smem_u32(r_full + i), 1);
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(smem_u32(sc_full + i), 64);
            mbar_init(smem_u32(sc_empty + i), kSumWarps);
        }
        *abort = 0;
        mbar_init_fence();
        prefetch_tensormap(&p.xmap);
        prefetch_tensormap(&p.wmap);
        if (kTma) prefetch_tensormap(&p.ymap);
        if (kTma && p.residual) prefetch_tensormap(&p.rmap);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a split tile's sums, [256 columns][128 tokens], over the stages
    float *sums = reinterpret_cast<float *>(smem);
    auto fail = [&](int code) {
        *abort = 1;
        atomicOr(p.status, code);
    };

    Walk walk(p);
    int t, j0, j1, m0, n0;
    if (warp >= kSumWarps) {
        regs_dec<kOtherRegs>();
        if (warp == kTmaWarp) {
            // ------------------------------------------------ producer
            grid_dependency_wait();
            if (lane == 0) {
                const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
                int c = 0;
                bool ok = true;
                while (ok && walk.next(p, t, j0, j1)) {
                    tile_at(p, t, m0, n0);
                    const int mr = m0 + (int)rank * kHalf, nr = n0 + (int)rank * kHalf;
                    for (int j = j0; j < j1; ++j, ++c) {
                        const int s = c % kStages;
                        if (c >= kStages &&
                            !mbar_wait(smem_u32(empty + s), ((c / kStages) - 1) & 1, abort)) {
                            fail(kErrSlotWait);
                            ok = false;
                            break;
                        }
                        const uint32_t st = smem_u32(smem + s * kStage);
                        // both CTAs' bytes count at the leader's barrier
                        const uint32_t bar = map_to_rank(smem_u32(full + s), leader);
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(full + s), 2 * kStage);
                        tma_load_2d_pair(st, &p.xmap, j * kGroup, mr, bar, pol_x);
                        tma_load_2d_pair(st + kStageX, &p.wmap, j * kGroup, nr, bar, pol_w);
                    }
                }
                // every load issued must have landed before the CTA exits: the leader
                // sees both CTAs' (the other waits for it at the last cluster barrier)
                if (rank == 0)
                    for (int i = c - kStages > 0 ? c - kStages : 0; i < c; ++i)
                        if (!mbar_wait_drain(smem_u32(full + i % kStages), (i / kStages) & 1))
                            atomicOr(p.status, kErrDrain);
                // and so must the leader's arrivals at this CTA's barriers (after an
                // abort the products that were to bring them may not have been issued)
                for (int i = c - kStages > 0 ? c - kStages : 0; ok && i < c; ++i)
                    ok = mbar_wait(smem_u32(empty + i % kStages), (i / kStages) & 1, abort);
                if (!ok && !*abort) fail(kErrDrain);
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------ products
            if (rank == 0) {
                const uint32_t stages = uniform(smem_u32(smem));
                const uint32_t bars = uniform(smem_u32(full));
                const uint32_t tm = uniform(tmem);
                const uint16_t both = (uint16_t)(3u << leader);
                int c = 0;
                bool ok = true;
                while (ok && walk.next(p, t, j0, j1)) {
                    for (int j = j0; j < j1; ++j, ++c) {
                        const int s = c % kStages, d = c % kDBufs;
                        if (!mbar_wait_all(bars + 8 * s, (c / kStages) & 1, abort)) {
                            if (lane == 0) fail(kErrStageWait);
                            ok = false;
                            break;
                        }
                        if (c >= kDBufs && !mbar_wait_all(bars + 8 * (2 * kStages + kDBufs + d),
                                                          ((c / kDBufs) - 1) & 1, abort)) {
                            if (lane == 0) fail(kErrSumWait);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t a = smem_desc_sw128(stages + s * kStage);
                            mma_f8_block_pair(tm + d * kTileN, a, a + (kStageX >> 4), kIdesc);
                            mma_commit_pair(bars + 8 * (2 * kStages + d), both);
                            mma_commit_pair(bars + 8 * (kStages + s), both);
                        }
                    }
                }
                // the products issued complete before the tensor memory is freed
                if (lane == 0)
                    for (int i = c - kDBufs > 0 ? c - kDBufs : 0; i < c; ++i)
                        if (!mbar_wait_drain(smem_u32(d_full + i % kDBufs), (i / kDBufs) & 1))
                            atomicOr(p.status, kErrDrain);
                // as have the arrivals from the other CTA's sum warps
                for (int i = c - kDBufs > 0 ? c - kDBufs : 0; ok && i < c; ++i)
                    ok = mbar_wait_all(smem_u32(d_empty + i % kDBufs), (i / kDBufs) & 1, abort);
                if (!ok && !*abort && lane == 0) fail(kErrDrain);
            }
        } else if (warp > kMmaWarp) {
            // ------------------------------------------------ scales
            // (rows and columns past the end take the last one's: they are not stored)
            grid_dependency_wait();
            const int i = (warp - kMmaWarp - 1) * 32 + lane;  // tokens i and i + 64
            int c = 0;                                        // batches
            bool ok = true;
            while (ok && walk.next(p, t, j0, j1)) {
                tile_at(p, t, m0, n0);
                const int mr = m0 + (int)rank * kHalf + i;
                const float *x0 = p.xs + (size_t)min(mr, p.M - 1) * p.G;
                const float *x1 = p.xs + (size_t)min(mr + 64, p.M - 1) * p.G;
                const float *w0 = p.ws + (size_t)min(n0 / kGroup + i, p.NB - 1) * p.G;
                for (int j = j0 & ~3; j < j1; j += 4, ++c) {
                    const int s = c % kScaleSlots;
                    const float4 a = load4(p, x0, j), b = load4(p, x1, j);
                    float4 w = a;
                    if (i < 2) w = load4(p, w0, j);
                    if (c >= kScaleSlots && !mbar_wait_all(smem_u32(sc_empty + s),
                                                           ((c / kScaleSlots) - 1) & 1, abort)) {
                        if (lane == 0) fail(kErrSlotWait);
                        ok = false;
                        break;
                    }
                    float4 *slot = reinterpret_cast<float4 *>(sm_scales + s * kScaleSlot);
                    slot[i] = a;
                    slot[i + 64] = b;
                    if (i < 2) slot[kHalf + i] = w;
                    mbar_arrive(smem_u32(sc_full + s));
                }
            }
        }
        __syncwarp();
        if (p.ksplit > 1) cluster_sync();  // with the sum warps', before the exchange
    } else {
        // ------------------------------------------------ sums and outputs
        regs_inc<kSumRegs>();
        grid_dependency_wait();
        const int quarter = warp & 3, col = (warp >> 2) * kCols;  // its 64 columns
        const int r = quarter * 32 + lane;  // token within the CTA's 128
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + col;
        uint8_t *stage_out = sm_store + warp * kStoreBytes;
        const uint32_t bar_full = smem_u32(d_full);
        const uint32_t bar_empty = map_to_rank(smem_u32(d_empty), leader);
        const uint32_t bar_res = smem_u32(r_full + warp);
        uint32_t res_asked = 0, res_taken = 0;  // residual tiles
        // the scale products of four blocks 4 i .. 4 i + 3, from the slot
        int sc = 0;  // batches
        auto take_scales = [&](float4 &f) {
            const int s = sc % kScaleSlots;
            if (!mbar_wait_all(smem_u32(sc_full + s), (sc / kScaleSlots) & 1, abort)) return false;
            const float4 *slot = reinterpret_cast<const float4 *>(sm_scales + s * kScaleSlot);
            const float4 a = slot[r], b = slot[kHalf + col / kGroup];
            f = make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(sc_empty + s));
            ++sc;
            return true;
        };
        // the warp's 32 tokens x 64 columns of the residual, into its staging
        auto ask_residual = [&](int n, int mw) {
            if (lane == 0) {
                tma_store_wait_read();  // the staging is free
                mbar_arrive_expect_tx(bar_res, kStoreBytes);
                tma_load_2d(smem_u32(stage_out), &p.rmap, n, mw, bar_res, policy_evict_first());
            }
            ++res_asked;
        };
        const bool staged_res = kTma && p.residual;
        int c = 0;
        // ok: false once a wait has given up.  Then the warp computes and stores nothing
        // more, but walks on to the next tile that is split, where all sum warps meet
        bool ok = true, more = walk.next(p, t, j0, j1);
        while (more) {
            tile_at(p, t, m0, n0);
            const int mw = m0 + (int)rank * kHalf + quarter * 32;
            const int nc = n0 + col, tt = t, end = j1;
            const bool whole = j0 == 0 && j1 == p.G;
            if (ok && whole && staged_res) ask_residual(nc, mw);
            if constexpr (!kTma) {
                // the residual's rows on their way to L2 meanwhile (a row's 128 bytes
                // are in at most two lines): 1240 tokens, N 33532, K 1440 156 us for 177 (132
                // in the present state of the kernel)
                if (whole && p.residual && mw + lane < p.M && nc < p.N) {
                    const uint16_t *row = p.residual + (size_t)(mw + lane) * p.N;
                    prefetch_l2(row + nc);
                    prefetch_l2(row + nc + min(kStoreCols, p.N - nc) - 1);
                }
            }
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
            for (int j = j0 & ~3, begin = j0; j < end && ok; j += 4) {
                float4 f;
                ok = take_scales(f);
                if (!ok) break;
                const float sb[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j + u < begin) continue;
                    if (j + u >= end) break;
                    const uint32_t from = taddr + (c % kDBufs) * kTileN;
                    ok = mbar_wait_all(bar_full + 8 * (c % kDBufs), (c / kDBufs) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    // 16 columns a load, the next on its way while one is added
                    uint32_t v[2][16];
                    tmem_ld(from, v[0]);
#pragma unroll
                    for (int q = 0; q < kCols / 16; ++q) {
                        tmem_wait_ld(v[q & 1]);
                        if (q + 1 < kCols / 16) {
                            tmem_ld(from + 16 * (q + 1), v[(q + 1) & 1]);
                        } else {  // all read: the tensor cores may write again
                            tc_fence_before();
                            if (lane == 0) mbar_arrive_remote(bar_empty + 8 * (c % kDBufs));
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * q + i] =
                                fmaf(__uint_as_float(v[q & 1][i]), sb[u], acc[16 * q + i]);
                    }
                    ++c;
                }
            }
            if (!ok && lane == 0) fail(kErrSumWait);
            more = walk.next(p, t, j0, j1);
            if (p.ksplit > 1) {
                // the cluster's tile: the sums wait in this CTA's stages, which
                // nothing uses any more, for the exchange below
#pragma unroll
                for (int i = 0; i < kCols; ++i) sums[(col + i) * kHalf + r] = acc[i];
                break;
            }
            if (!whole) {
                // part of a tile: if the other piece is in its pair's slot by now, it
                // is added to this one; else this one goes to this pair's slot (0: the
                // run begins inside the tile, 1: the tile begins inside the run), and
                // whoever of the two sees the other's there finishes the tile
                const long long tile0 = (long long)(tt - p.whole) * p.G;
                const int b0 = walk.owner(p, tile0), b1 = walk.owner(p, tile0 + p.G - 1);
                const int b = walk.pair == b0 ? b1 : b0;
                auto slot = [&](int pair) {
                    const int s = 2 * pair + (walk.begin(p, pair) > tile0 ? 0 : 1);
                    return p.partials + ((size_t)(2 * s + rank) * kTileN + col) * kHalf + r;
                };
                unsigned *there = p.counters + 2 * (tt - p.whole) + rank;  // pieces in slots
                if (threadIdx.x == 0) *s_last = atomicAdd(there, 0u) != 0u;
                ok = barrier_all(1, kSumWarps * 32, ok);
                if (!ok) break;  // all of them
                if (!*s_last) {
                    float *part = slot(walk.pair);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) part[(size_t)i * kHalf] = acc[i];
                    __threadfence();
                    asm volatile("bar.sync 1, %0;" ::"r"(kSumWarps * 32) : "memory");
                    if (threadIdx.x == 0) *s_last = atomicAdd(there, 1u) != 0u;
                    asm volatile("bar.sync 1, %0;" ::"r"(kSumWarps * 32) : "memory");
                }
                const bool last = *s_last != 0;
                if (last) {
                    __threadfence();
                    if (threadIdx.x == 0) *there = 0u;  // ready for the next launch
                    if (staged_res) ask_residual(nc, mw);
                    const float *src = slot(b);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {  // a round trip each
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __ldcg(src + (size_t)(32 * q + i) * kHalf);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[32 * q + i] += v[i];
                    }
                }
                // s_last is written again only after every thread has read it
                asm volatile("bar.sync 1, %0;" ::"r"(kSumWarps * 32) : "memory");
                if (!last) continue;
            }
            if (!ok) continue;
            // y[m][nc .. nc + 63] = sums (+ residual), one rounding each, by way of the
            // warp's staging: the residual comes there, and the outputs leave from
            // there, by TMA or (rows that TMA cannot address) by the warp's own copies
            if (staged_res) {
                ok = mbar_wait_all(bar_res, res_taken & 1, abort);
                if (!ok) {
                    if (lane == 0) fail(kErrStageWait);
                    continue;
                }
                ++res_taken;
            } else if constexpr (kTma) {
                if (lane == 0) tma_store_wait_read();  // the staging is free
                __syncwarp();
            } else if (p.residual) {
                copy_rows<true>(p, stage_out, lane, mw, nc);
            }
            uint8_t *row = stage_out + lane * 128;
#pragma unroll
            for (int q = 0; q < 8; ++q) {  // 8 columns, 16 bytes, at the swizzled chunk
                uint4 *at = reinterpret_cast<uint4 *>(row + ((q ^ (lane & 7)) << 4));
                float *v = acc + q * 8;
                if (p.residual) {
                    const uint4 u = *at;
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] += half_bits_to_float((uint16_t)w[i], kBf16);
                        v[2 * i + 1] += half_bits_to_float((uint16_t)(w[i] >> 16), kBf16);
                    }
                }
                *at = make_uint4(pack16<kBf16>(v[0], v[1]), pack16<kBf16>(v[2], v[3]),
                                 pack16<kBf16>(v[4], v[5]), pack16<kBf16>(v[6], v[7]));
            }
            if constexpr (kTma) {
                fence_async_shared();
                __syncwarp();
                if (lane == 0 && nc < p.N && mw < p.M)
                    tma_store_2d(&p.ymap, nc, mw, smem_u32(stage_out));
            } else {
                copy_rows<false>(p, stage_out, lane, mw, nc);
            }
        }
        // what was asked for lands, what was stored is written, before the exit
        if (res_asked != res_taken && lane == 0 && !mbar_wait_drain(bar_res, res_taken & 1))
            atomicOr(p.status, kErrDrain);
        tma_store_wait();
        __syncwarp();
        if (p.ksplit > 1) {
            // the exchange: the cluster's CTAs of these 128 tokens share out the tile's
            // columns, in groups of 16 (two pairs) or 8; a warp takes a group for 32
            // tokens (lane = token).  It stays with these warps: the others keep few
            // registers.
            cluster_sync();
            if (!*abort) {
                const int S = p.ksplit, width = S == 2 ? 16 : 8;
                uint4 *own = reinterpret_cast<uint4 *>(stage_out);
                tile_at(p, blockIdx.x / (2 * S), m0, n0);
                for (int u = warp;; u += kSumWarps) {
                    const int qu = u & 3, c = ((u >> 2) * S + (int)(crank >> 1)) * width;
                    const int m = m0 + (int)rank * kHalf + qu * 32, n = n0 + c;
                    if (c >= kTileN || n >= p.N || m >= p.M) break;
                    const float *from = sums + c * kHalf + qu * 32 + lane;
                    if (S == 2) exchange<kBf16, kTma, 16, 2>(p, from, own, rank, lane, m, n);
                    else exchange<kBf16, kTma, 8, kMaxSplit>(p, from, own, rank, lane, m, n);
                }
            }
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    // No CTA's shared or tensor memory goes while another uses it.  Everything read of
    // the others' has been stored by now, and every arrival at a barrier of theirs has
    // been waited for there, so all of it has landed; the barrier orders execution only.
    cluster_arrive_relaxed();
    cluster_wait();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

void config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int pairs, int ksplit,
            cudaStream_t stream) {
    cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2u * ksplit, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

// clusters of k pairs that run at the same time, found by fp8_wide_init (before it, as
// many as the SMs hold; there may be none of some size)
int g_clusters[kMaxSplit + 1];
bool g_found;
int clusters(int k, const DeviceInfo &dev) {
    return g_found ? g_clusters[k] : dev.sm_count / (2 * k);
}

}  // namespace

Fp8WidePlan plan_fp8_wide(int M, int N, int K, const DeviceInfo &dev, const Workspace &ws) {
    Fp8WidePlan pl{};
    pl.G = (K + kGroup - 1) / kGroup;
    pl.tiles_m = (M + kTileM - 1) / kTileM;
    pl.tiles_n = (int)(((long long)N + kTileN - 1) / kTileN);  // N up to 2^31 - 1
    const long long tiles = (long long)pl.tiles_m * pl.tiles_n;
    const int pairs = dev.sm_count / 2;
    pl.pairs = (int)(tiles < pairs ? tiles : pairs);
    pl.whole = (int)tiles;
    pl.ksplit = 1;
    // few tiles: the largest cluster that keeps every tile in one wave (M 256, N 5120:
    // K 5120 23.2 us, 27.3 unsplit; K 17408 37.5, 68.3), with at least eight blocks of
    // K per pair (M 256, N 1024, K 1024: 12.9 us, 15.0 with four; K 1536 the same).
    // Two are enough where rows do not go by TMA: the exchange shares out their copies
    // too (M 300, N 1021, K 1024 with a residual 10.3 us, 13.3 with four, 19.1 with
    // eight; without 9.8, 10.2, 11.6).  More than four pairs lose: M 512, N 1024,
    // K 5120 19.1 us with eight, 12.8 with four.
    const int least = N % 8 == 0 ? 8 : 2;
    for (int k = kMaxSplit; k > 1; --k)
        if (tiles <= clusters(k, dev) && pl.G >= least * k) {
            pl.ksplit = k;
            pl.pairs = (int)tiles * k;
            pl.whole = 0;
            return pl;
        }
    // an unfinished last round: it and the full round before it are cut into equal
    // runs where that saves more than the pieces cost, about 24 blocks and, in long
    // tiles, a third of a round.  M 512, microseconds, whole against equal runs:
    //   empty blocks per pair, of a round's
    //   N 10240, K 2048    15 of 16    27.3   28.1
    //   N 16896, K 5120    11 of 40    47.7   56.0
    //   N 14592, K 5120    20 of 40    47.7   47.7
    //   N 20480, K 5120    36 of 40    66.2   62.0
    //   N 16896, K 17408   36 of 136  129.7  138.1
    //   N 14592, K 17408   68 of 136  129.7  117.4
    const long long rest = tiles % pairs, empty = (pairs - rest) * pl.G;
    if (tiles < pairs || rest == 0 || empty < 24ll * pairs || (pairs - rest) * 3 < pairs) return pl;
    const long long split = pairs + rest;
    if ((size_t)2 * pairs * 2 * kTileN * kHalf * sizeof(float) > ws.partial_bytes ||
        2 * split > ws.n_counters - kMmaSchedWords)
        return pl;
    pl.whole = (int)(tiles - split);
    pl.split = split * pl.G;
    return pl;
}

cudaError_t launch_fp8_wide(const Fp8Args &a, const Fp8WidePlan &plan, const Workspace &ws,
                            cudaStream_t stream) {
    WideParams p;
    memset(&p, 0, sizeof(p));
    if (!encode_fp8_rows(&p.xmap, a.x, a.M, a.K, kHalf) ||
        !encode_fp8_rows(&p.wmap, a.w, a.N, a.K, kHalf))
        return cudaErrorInvalidValue;
    const bool tma = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0 &&
                     ((uintptr_t)a.residual & 15) == 0;
    if (tma && (!encode_rows16(&p.ymap, a.y, a.M, a.N, 32, kStoreCols) ||
                (a.residual && !encode_rows16(&p.rmap, a.residual, a.M, a.N, 32, kStoreCols))))
        return cudaErrorInvalidValue;
    p.xs = a.xs;
    p.ws = a.ws;
    p.residual = a.residual;
    p.y = a.y;
    p.partials = ws.partials;
    p.counters = ws.counters;
    p.status = ws.status;
    p.M = a.M;
    p.N = a.N;
    p.G = plan.G;
    p.NB = (int)(((long long)a.N + kGroup - 1) / kGroup);
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.scales16 = plan.G % 4 == 0 && ((uintptr_t)a.xs & 15) == 0 && ((uintptr_t)a.ws & 15) == 0;
    p.whole = plan.whole;
    p.ksplit = plan.ksplit;
    p.split = plan.split;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(cfg, attr, plan.pairs, plan.ksplit, stream);
    if (tma) return a.bf16 ? cudaLaunchKernelEx(&cfg, fp8_wide_kernel<true, true>, p)
                           : cudaLaunchKernelEx(&cfg, fp8_wide_kernel<false, true>, p);
    return a.bf16 ? cudaLaunchKernelEx(&cfg, fp8_wide_kernel<true, false>, p)
                  : cudaLaunchKernelEx(&cfg, fp8_wide_kernel<false, false>, p);
}

cudaError_t fp8_wide_init(const DeviceInfo &) {
    const void *kernels[] = {
        (const void *)fp8_wide_kernel<false, false>, (const void *)fp8_wide_kernel<false, true>,
        (const void *)fp8_wide_kernel<true, false>, (const void *)fp8_wide_kernel<true, true>};
    cudaError_t e = cudaSuccess;
    for (const void *k : kernels) {
        // the sum warps wait for registers that the launch has to have: a build that gives
        // the kernel fewer than the split counts on would never get past that
        cudaFuncAttributes attr;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, k);
        if (e == cudaSuccess && attr.numRegs < kLaunchRegs) e = cudaErrorLaunchOutOfResources;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    }
    for (int k = 2; k <= kMaxSplit && e == cudaSuccess; ++k) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(cfg, attr, k, k, nullptr);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&g_clusters[k], fp8_wide_kernel<true, true>, &cfg);
    }
    g_found = e == cudaSuccess;
    return e;
}

}  // namespace w4a16
