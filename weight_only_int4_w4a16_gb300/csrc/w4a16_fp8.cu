// The 8-bit linear for up to 64 tokens (more: w4a16_fp8_wide.cu):
// y [M, N] = x [M, K] w [N, K]^T (+ residual) for e4m3 rows x with one fp32 scale
// per 128 elements and e4m3 weights with one fp32 scale per block of 128 x 128
// (forum.sourcefind.cn thread "vLLM on Hygon Z100", section
// 六: FP8 checkpoints, dequantised to 16 bits at load there because the GPU has
// no FP8 arithmetic; here the tensor cores take the 8-bit data):
//
//   y[m, n] = sum_b sx[m, b] sw[n / 128, b] * (sum_{k in block b} x[m, k] w[n, k])
//
// The scales change every 128 elements of K, so the tensor cores' accumulator
// holds one block's sum only: per block b a fresh product of 128 weight rows by
// T tokens lands in tensor memory, and the sum warps add it, times sx sw, to fp32
// sums in registers (one fused multiply-add per element and block).  A product of two
// e4m3 numbers is exact, the tensor cores add 128 of them in fp32; a block's addition
// rounds once, and y once, to its 16 bits.
//
//   MMA shape (swap AB): the MMA's M = 128 weight rows of one tile, its N = T
//   tokens (16, 32 or 64; missing tokens are zero rows of x), K = 32 per
//   instruction, four instructions per block.  A partial last block is filled
//   with zeros by TMA.
//
//   Roles (one CTA per SM): four sum warps, eight from 32 tokens on (thread = weight
//   row), scale and add the blocks and write y; the next warp streams two blocks of
//   weights and of x per stage by TMA (128-byte swizzled, K-major; 256 consecutive
//   bytes of each weight row), its lanes copy the blocks' scales next to them; the
//   last warp issues the products.
//
//   Work: few tiles (a small N) are split along K between the CTAs of a cluster,
//   which exchange their sums through distributed shared memory.  More take whole
//   tiles in turn; where that would leave much of the last wave empty, the (tile,
//   block) sequence is cut into equal runs, one per CTA ("stream-K"), and a tile
//   split between CTAs is summed by the last of them from global memory.  Pieces are
//   added in K order either way: results do not depend on which CTA came last.
//
//   Bound by the weights' bytes and, in short calls, by the start (about 3 us to the
//   first weights) and the exchange of split tiles (about 2 us); from 32 tokens on the
//   sum warps' turn per block shows too (64 tokens, multiply-adds switched off: 20.1 us
//   for 22.3).  N 34816, K 5120 (178 MB) at 8 tokens: 28.3 to 29.1 us, 6.1 to 6.3 TB/s,
//   90 to 93% of the measured copy rate, at 64 tokens 38.0; N 5120, K 17408 (89 MB) at
//   64 tokens: 22.6 us, 4.0 TB/s; N 8192, K 5120 (42 MB) at 1 token: 10.4 us, 4.0 TB/s.
//
// Every mbarrier wait is bounded; on expiry the kernel records an error code in
// the device status word, drains what it has in flight, frees its tensor memory
// and exits.  The barriers of split tiles have no limit of their own: every sum warp
// comes to the first one, whether or not its waits were met, and there they agree on
// whether to go on (barrier_all).
#include <cstring>

#include "w4a16_fp8_common.cuh"
#include "w4a16_internal.h"
#include "w4a16_tcgen05.cuh"

namespace w4a16 {
namespace {

using namespace dev;

constexpr int kTileN = 128;                   // weight rows per tile (MMA M)
constexpr int kSub = 2;                       // blocks per stage
constexpr int kBlockW = kTileN * kGroup;      // 16 KB of weights per block
constexpr int kMaxStages = 6;
constexpr int kSmemBudget = 220 * 1024;       // the stages
constexpr int kDBufs = 2;                     // stages' sums in tensor memory
constexpr int kTmemCols = 512;
constexpr int kMaxCluster = 8;

struct Fp8Params {
    CUtensorMap wmap;  // w: (K bytes, N rows), box {128, 128}, 128-byte swizzle
    CUtensorMap xmap;  // x: (K bytes, M rows), box {128, T}
    const float *xs, *ws;
    const uint16_t *residual;
    uint16_t *y;
    float *partials;     // [2 * grid][T][128] fp32
    unsigned *counters;  // [tiles], zero between launches
    int *status;
    int M, N, G;
    long long total;     // blocks of all tiles
    int tiles;
    int streamk;
    int ksplit;          // CTAs of a cluster that split each tile along K (1: none)
    int bf16;
};

template <int T>
struct Cfg {
    // warps that add the sums: a quarter of the rows each, and from 32 tokens on
    // half of the tokens, so that a tile's outputs are written by twice the threads
    // (64 tokens, N 20480: K 2048 23.2 us against 25.2 with four warps, K 5120 43.3
    // against 43.6, K 17408 119.4 against 116.2; sixteen warps: no change)
    static constexpr int kSumWarps = T >= 32 ? 8 : 4;
    static constexpr int kCols = T / (kSumWarps / 4);  // tokens per thread
    static constexpr int kTmaWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
    static constexpr int kThreads = (kSumWarps + 2) * 32;
    static constexpr int kBlockX = T * kGroup;
    static constexpr int kStage = kSub * (kBlockW + kBlockX);  // weights, then x
    // floats per stage: per block T scales of x, then per block the weights'
    static constexpr int kScales = kSub * T + 4;
    static constexpr uint32_t kIdesc =     // D f32, A and B e4m3 (0), N = T, M = 128
        (1u << 4) | ((uint32_t)(T >> 3) << 17) | ((uint32_t)(kTileN >> 4) << 24);
    static constexpr int kFit = kSmemBudget / (kStage + kScales * 4);
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    // slack for the 1024-byte alignment, the stages, their scales, the
    // barriers, the tensor-memory address, abort and last flags
    static constexpr int kSmem =
        1024 + kStages * (kStage + kScales * 4) + (2 * kStages + 2 * kDBufs) * 8 + 16;
};

// The CTA's work: segments (a tile and a run of its blocks), in order.
struct Walk {
    long long pos, end;
    __device__ __forceinline__ Walk(const Fp8Params &p) {
        if (p.ksplit > 1) {  // the CTA's part of its cluster's tile
            const int r = blockIdx.x % p.ksplit;
            const long long t0 = (long long)(blockIdx.x / p.ksplit) * p.G;
            pos = t0 + r * p.G / p.ksplit;
            end = t0 + (r + 1) * p.G / p.ksplit;
        } else if (p.streamk) {
            pos = begin(p, blockIdx.x);
            end = begin(p, blockIdx.x + 1);
        } else {
            pos = (long long)blockIdx.x * p.G;
            end = p.total;
        }
    }
    static __device__ __forceinline__ long long begin(const Fp8Params &p, int b) {
        return (long long)b * p.total / gridDim.x;
    }
    // the CTA whose run holds block i
    static __device__ __forceinline__ int owner(const Fp8Params &p, long long i) {
        return (int)(((i + 1) * (long long)gridDim.x - 1) / p.total);
    }
    // next segment: blocks [j0, j1) of tile t
    __device__ __forceinline__ bool next(const Fp8Params &p, int &t, int &j0, int &j1) {
        if (pos >= end) return false;
        t = (int)(pos / p.G);
        const long long t0 = (long long)t * p.G;
        j0 = (int)(pos - t0);
        if (p.streamk || p.ksplit > 1) {
            j1 = (int)((t0 + p.G < end ? t0 + p.G : end) - t0);
            pos = t0 + j1;
        } else {
            j1 = p.G;
            pos += (long long)gridDim.x * p.G;
        }
        return true;
    }
};

// The partial-sum slot of CTA b for the tile whose first block is tile0: its
// first one when the run begins inside the tile, its second when the tile
// begins inside the run.
__device__ __forceinline__ int slot_of(const Fp8Params &p, int b, long long tile0) {
    return 2 * b + (Walk::begin(p, b) > tile0 ? 0 : 1);
}

// y[m0 .. m0 + 15][n] = v (+ residual), one rounding each.  The residual may be
// y itself: its 16 values are read before any of the 16 outputs is written.
__device__ __forceinline__ void store16(const Fp8Params &p, int m0, int n, const float *v) {
    float r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        r[i] = p.residual && m0 + i < p.M
                   ? half_bits_to_float(p.residual[(size_t)(m0 + i) * p.N + n], p.bf16)
                   : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (m0 + i < p.M) p.y[(size_t)(m0 + i) * p.N + n] = float_to_half_bits(v[i] + r[i], p.bf16);
}

// four rows' residual of token m (zeros without one, or past N), and their outputs;
// vec: rows in fours and 8-byte aligned
__device__ __forceinline__ float4 residual4(const Fp8Params &p, int m, int n, bool vec) {
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.residual) {
        const uint16_t *src = p.residual + (size_t)m * p.N + n;
        if (vec) {
            if (n < p.N) {
                const uint2 u = *reinterpret_cast<const uint2 *>(src);
                r[0] = half_bits_to_float((uint16_t)u.x, p.bf16);
                r[1] = half_bits_to_float((uint16_t)(u.x >> 16), p.bf16);
                r[2] = half_bits_to_float((uint16_t)u.y, p.bf16);
                r[3] = half_bits_to_float((uint16_t)(u.y >> 16), p.bf16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < p.N) r[i] = half_bits_to_float(src[i], p.bf16);
        }
    }
    return make_float4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store4(const Fp8Params &p, int m, int n, bool vec, float4 v) {
    const uint16_t h[4] = {float_to_half_bits(v.x, p.bf16), float_to_half_bits(v.y, p.bf16),
                           float_to_half_bits(v.z, p.bf16), float_to_half_bits(v.w, p.bf16)};
    uint16_t *dst = p.y + (size_t)m * p.N + n;
    if (vec) {
        if (n < p.N)
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2((uint32_t)h[0] | (uint32_t)h[1] << 16,
                           (uint32_t)h[2] | (uint32_t)h[3] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.N) dst[i] = h[i];
    }
}

template <int T>
__global__ void __launch_bounds__(Cfg<T>::kThreads, 1)
    fp8_kernel(const __grid_constant__ Fp8Params p) {
    using C = Cfg<T>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int NS = C::kStages;
    float *sm_scales = reinterpret_cast<float *>(smem + (size_t)NS * C::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_scales + NS * C::kScales);
    uint64_t *empty = full + NS;
    uint64_t *d_full = empty + NS;
    uint64_t *d_empty = d_full + kDBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(d_empty + kDBufs);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_last = const_cast<int *>(abort + 1);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    grid_dependents_launch();
    if (threadIdx.x == C::kTmaWarp * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(full + i), 1 + 32);  // the TMA bytes, each lane's scales
            // the products, each reader of the scales
            mbar_init(smem_u32(empty + i), 1 + C::kSumWarps);
        }
        for (int i = 0; i < kDBufs; ++i) {
            mbar_init(smem_u32(d_full + i), 1);
            mbar_init(smem_u32(d_empty + i), C::kSumWarps);
        }
        *abort = 0;
        mbar_init_fence();
        prefetch_tensormap(&p.wmap);
        prefetch_tensormap(&p.xmap);
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    float *sums = reinterpret_cast<float *>(smem);  // [T][128], once the stages are done
    auto fail = [&](int code) {
        *abort = 1;
        atomicOr(p.status, code);
    };

    Walk walk(p);
    int t, j0, j1;
    if (warp == C::kTmaWarp) {
        // ------------------------------------------------ producer
        grid_dependency_wait();
        const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
        int c = 0;  // stages
        bool ok = true;
        while (ok && walk.next(p, t, j0, j1)) {
            for (int j = j0; j < j1; j += kSub, ++c) {
                const int s = c % NS, nb = min(kSub, j1 - j);
                if (c >= NS && !mbar_wait_all(smem_u32(empty + s), ((c / NS) - 1) & 1, abort)) {
                    if (lane == 0) fail(kErrSlotWait);
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(full + s);
                if (lane == 0) {
                    const uint32_t st = smem_u32(smem + (size_t)s * C::kStage);
                    mbar_arrive_expect_tx(bar, nb * (kBlockW + C::kBlockX));
                    for (int b = 0; b < nb; ++b)
                        tma_load_2d(st + b * kBlockW, &p.wmap, (j + b) * kGroup, t * kTileN, bar,
                                    pol_w);
                    for (int b = 0; b < nb; ++b)
                        tma_load_2d(st + kSub * kBlockW + b * C::kBlockX, &p.xmap, (j + b) * kGroup,
                                    0, bar, pol_x);
                }
                const uint32_t sc = smem_u32(sm_scales + s * C::kScales);
#pragma unroll
                for (int i = 0; i < (T + 31) / 32; ++i) {
                    const int tt = lane + 32 * i;
                    const bool live = tt < p.M;
                    const float *src = live ? p.xs + (size_t)tt * p.G + j : p.xs;
#pragma unroll
                    for (int b = 0; b < kSub; ++b)
                        if (tt < T)
                            cp_async4(sc + 4 * (b * T + tt), live && b < nb ? src + b : p.xs,
                                      live && b < nb ? 4u : 0u);
                }
                if (lane < nb)
                    cp_async4(sc + 4 * (kSub * T + lane), p.ws + (size_t)t * p.G + j + lane, 4u);
                cp_async_arrive(bar);
            }
        }
        // every copy issued must have landed before the CTA exits
        if (lane == 0)
            for (int i = c - NS > 0 ? c - NS : 0; i < c; ++i)
                if (!mbar_wait_drain(smem_u32(full + i % NS), (i / NS) & 1))
                    atomicOr(p.status, kErrDrain);
        cp_async_wait_all();
    } else if (warp == C::kMmaWarp) {
        // ------------------------------------------------ products
        const uint32_t stages = uniform(smem_u32(smem)), bars = uniform(smem_u32(full));
        const uint32_t tm = uniform(tmem);
        int c = 0;
        bool ok = true;
        while (ok && walk.next(p, t, j0, j1)) {
            for (int j = j0; j < j1; j += kSub, ++c) {
                const int s = c % NS, d = c % kDBufs, nb = min(kSub, j1 - j);
                if (!mbar_wait_all(bars + 8 * s, (c / NS) & 1, abort)) {
                    if (lane == 0) fail(kErrStageWait);
                    ok = false;
                    break;
                }
                if (c >= kDBufs && !mbar_wait_all(bars + 8 * (2 * NS + kDBufs + d),
                                                  ((c / kDBufs) - 1) & 1, abort)) {
                    if (lane == 0) fail(kErrSumWait);
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t st = stages + s * C::kStage;
                    const uint64_t a = smem_desc_sw128(st);
                    const uint64_t b = smem_desc_sw128(st + kSub * kBlockW);
                    mma_f8_block(tm + d * kSub * T, a, b, C::kIdesc);
                    if (nb > 1)
                        mma_f8_block(tm + (d * kSub + 1) * T, a + (kBlockW >> 4),
                                     b + (C::kBlockX >> 4), C::kIdesc);
                    mma_commit(bars + 8 * (2 * NS + d));
                    mma_commit(bars + 8 * (NS + s));
                }
            }
        }
        // the products issued complete before the tensor memory is freed, and the last
        // arrivals land before the CTA exits (after an abort the sum warps' may not come)
        if (lane == 0) {
            for (int i = c - kDBufs > 0 ? c - kDBufs : 0; i < c; ++i)
                if (!mbar_wait_drain(smem_u32(d_full + i % kDBufs), (i / kDBufs) & 1))
                    atomicOr(p.status, kErrDrain);
            const int e = c - 1;
            if (ok && c > 0 && !mbar_wait(smem_u32(empty + e % NS), (e / NS) & 1, abort) &&
                !*abort)
                fail(kErrDrain);
        }
    } else {
        // ------------------------------------------------ sums and outputs
        grid_dependency_wait();
        constexpr int kCols = C::kCols;
        const int r = (warp & 3) * 32 + lane;   // row within the tile
        const int cb = (warp >> 2) * kCols;     // first token within the tile
        const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + cb;
        int c = 0;
        // false once a wait has given up: then the warp computes and stores nothing more,
        // but walks on to the next tile that is split, where all sum warps meet
        bool ok = true;
        while (walk.next(p, t, j0, j1)) {
            const int n = t * kTileN + r, mt = p.M - cb;  // this thread's tokens: i < mt
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
            for (int j = j0; j < j1 && ok; j += kSub, ++c) {
                const int s = c % NS, d = c % kDBufs;
                const bool two = j + 1 < j1;
                const float *sc = sm_scales + s * C::kScales;
                // the scale products of block b of the stage
                auto factors = [&](int b, float (&f)[kCols]) {
                    const float sw = sc[kSub * T + b];
#pragma unroll
                    for (int i = 0; i < kCols; i += 4) {
                        const float4 sx = *reinterpret_cast<const float4 *>(sc + b * T + cb + i);
                        f[i] = sx.x * sw;
                        f[i + 1] = sx.y * sw;
                        f[i + 2] = sx.z * sw;
                        f[i + 3] = sx.w * sw;
                    }
                };
                // the stage's barrier shows its scales, the sums' its products; the first
                // block's factors come while the tensor cores are still at work, the
                // second's while its sums are on their way
                float f[kCols];
                uint32_t u[kCols], v[kCols];
                const uint32_t from = taddr + d * kSub * T;
                ok = mbar_wait_all(smem_u32(full + s), (c / NS) & 1, abort);
                if (ok) {
                    factors(0, f);
                    ok = mbar_wait_all(smem_u32(d_full + d), (c / kDBufs) & 1, abort);
                }
                if (!ok) {
                    if (lane == 0) fail(kErrSumWait);
                    break;
                }
                tc_fence_after();
                tmem_ld(from, u);
                tmem_wait_ld(u);
                if (two) tmem_ld(from + T, v);
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    acc[i] = fmaf(__uint_as_float(u[i]), f[i], acc[i]);
                if (two) {
                    factors(1, f);
                    tmem_wait_ld(v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(d_empty + d));
                    mbar_arrive(smem_u32(empty + s));
                }
                if (two) {
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        acc[i] = fmaf(__uint_as_float(v[i]), f[i], acc[i]);
                }
            }
            if (j0 == 0 && j1 == p.G) {  // a whole tile
                if (ok && n < p.N) {
#pragma unroll
                    for (int i = 0; i < kCols; i += 16) store16(p, cb + i, n, acc + i);
                }
                continue;
            }
            if (p.ksplit > 1) {
                // the cluster's tile: the sums wait in this CTA's stages, which
                // nothing uses any more, for the exchange below
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    if (i < mt) sums[(cb + i) * kTileN + r] = acc[i];
                break;
            }
            // part of a tile: the sums go to this CTA's slot, and the last CTA
            // of the tile adds the slots in K order
            const long long tile0 = (long long)t * p.G;
            const size_t mine = (size_t)cb * kTileN + r;
            float *part = p.partials + (size_t)slot_of(p, blockIdx.x, tile0) * T * kTileN + mine;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                if (i < mt) part[(size_t)i * kTileN] = acc[i];
            __threadfence();
            ok = barrier_all(1, C::kSumWarps * 32, ok);
            if (!ok) break;  // all of them
            const int b0 = Walk::owner(p, tile0), b1 = Walk::owner(p, tile0 + p.G - 1);
            if (threadIdx.x == 0)
                *s_last = atomicAdd(p.counters + t, 1u) == (unsigned)(b1 - b0) ? 1 : 0;
            asm volatile("bar.sync 1, %0;" ::"r"(C::kSumWarps * 32) : "memory");
            if (*s_last) {
                __threadfence();
                if (threadIdx.x == 0) p.counters[t] = 0u;  // ready for the next launch
                // a piece's loads all at once: a round trip per piece
#pragma unroll
                for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
                for (int b = b0; b <= b1; ++b) {
                    const float *src =
                        p.partials + (size_t)slot_of(p, b, tile0) * T * kTileN + mine;
                    float v[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        v[i] = i < mt ? __ldcg(src + (size_t)i * kTileN) : 0.f;
#pragma unroll
                    for (int i = 0; i < kCols; ++i) acc[i] += v[i];
                }
                if (n < p.N) {
#pragma unroll
                    for (int i = 0; i < kCols; i += 16) store16(p, cb + i, n, acc + i);
                }
            }
            // s_last is written again only after every thread has read it
            asm volatile("bar.sync 1, %0;" ::"r"(C::kSumWarps * 32) : "memory");
        }
    }
    if (p.ksplit > 1) {
        // the exchange: CTA r of the cluster takes every ksplit-th token of the tile,
        // adds the CTAs' sums in K order (which is rank order) and writes y; a warp
        // takes a token's 128 rows, four per lane, and four tokens at a time
        __syncthreads();
        cluster_sync();
        if (!*abort) {
            const int S = p.ksplit, n = (int)(blockIdx.x / S) * kTileN + 4 * lane;
            const bool vec = p.N % 4 == 0 && ((uintptr_t)p.y & 7) == 0 &&
                             ((uintptr_t)p.residual & 7) == 0;
            const uint32_t mine = smem_u32(sums + 4 * lane);
            constexpr int kBatch = 4, kWarps = C::kSumWarps + 2;
            for (int i0 = cluster_rank() + S * warp; i0 < p.M; i0 += kBatch * kWarps * S) {
                float4 v[kBatch][kMaxCluster], res[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int m = i0 + i * kWarps * S;
                    res[i] = m < p.M ? residual4(p, m, n, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q)
                        if (q < S && m < p.M)
                            v[i][q] =
                                ld4_cluster(map_to_rank(mine, q) + (uint32_t)(m * kTileN * 4));
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int m = i0 + i * kWarps * S;
                    if (m >= p.M) break;
                    float4 sum = v[i][0];
#pragma unroll
                    for (int q = 1; q < kMaxCluster; ++q)
                        if (q < S) {
                            sum.x += v[i][q].x;
                            sum.y += v[i][q].y;
                            sum.z += v[i][q].z;
                            sum.w += v[i][q].w;
                        }
                    store4(p, m, n, vec, make_float4(sum.x + res[i].x, sum.y + res[i].y,
                                                          sum.z + res[i].z, sum.w + res[i].w));
                }
            }
        }
        // no CTA leaves while another reads its sums: the arrival comes after the
        // stores of what was read, and orders execution only
        cluster_arrive_relaxed();
        cluster_wait();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int T>
void config_t(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int grid, int ksplit,
              cudaStream_t stream) {
    cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Cfg<T>::kThreads);
    cfg.dynamicSmemBytes = Cfg<T>::kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ksplit, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = ksplit > 1 ? 2 : 1;
}

template <int T>
cudaError_t launch_t(const Fp8Params &p, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config_t<T>(cfg, attr, grid, p.ksplit, stream);
    return cudaLaunchKernelEx(&cfg, fp8_kernel<T>, p);
}

// clusters of k CTAs that run at the same time, found by fp8_init (before it, as many as
// the SMs hold; there may be none of some size)
int g_clusters[kMaxCluster + 1];
bool g_found;
int clusters(int k, const DeviceInfo &dev) { return g_found ? g_clusters[k] : dev.sm_count / k; }

}  // namespace

Fp8Plan plan_fp8(int M, int N, int K, const DeviceInfo &dev, const Workspace &ws) {
    Fp8Plan pl{};
    pl.T = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    pl.G = (K + kGroup - 1) / kGroup;
    pl.tiles = (int)(((long long)N + kTileN - 1) / kTileN);  // N up to 2^31 - 1
    pl.ksplit = 1;
    pl.grid = pl.tiles < dev.sm_count ? pl.tiles : dev.sm_count;
    // few tiles: the largest cluster that keeps every tile in one wave (N 5120: M 8,
    // K 5120 15.0 us against 19.1 in equal runs; M 64, K 17408 29.3 against 33.4), with
    // at least two blocks of K per CTA (M 8, N 512, K 1024: 8.8 us, 10.9 with four)
    for (int k = kMaxCluster; k > 1; --k)
        if (pl.tiles <= clusters(k, dev) && pl.G >= 2 * k) {
            pl.ksplit = k;
            pl.grid = pl.tiles * k;
            return pl;
        }
    // whole tiles in turn, or equal runs of blocks.  Whole tiles leave the last wave
    // partly empty, equal runs add and read back the pieces of split tiles, which
    // costs what about 20 blocks do.  Microseconds, whole against equal runs:
    //   empty blocks per CTA   M 8           M 64
    //   N 20480, K 2048   15   19.1   21.1   23.2   23.2
    //   N 34048, K 5120   10   37.5   41.6   43.6   45.7
    //   N 29184, K 5120   20   37.5   35.5   43.6   39.5
    //   N 20480, K 5120   38   35.7   30.4   43.3   34.2
    //   N 10752, K 17408  61   49.8   45.7   64.1   49.2
    const int waves = (pl.tiles + dev.sm_count - 1) / dev.sm_count;
    const long long empty = ((long long)waves * dev.sm_count - pl.tiles) * pl.G;
    const size_t need = (size_t)2 * dev.sm_count * pl.T * kTileN * sizeof(float);
    if (empty >= 20ll * dev.sm_count && (long long)pl.tiles * pl.G >= 4ll * dev.sm_count &&
        need <= ws.partial_bytes && pl.tiles <= ws.n_counters - kMmaSchedWords) {
        pl.streamk = true;
        pl.grid = dev.sm_count;
    }
    return pl;
}

cudaError_t launch_fp8(const Fp8Args &a, const Fp8Plan &plan, const Workspace &ws,
                       cudaStream_t stream) {
    Fp8Params p;
    memset(&p, 0, sizeof(p));
    if (!encode_fp8_rows(&p.wmap, a.w, a.N, a.K, kTileN) ||
        !encode_fp8_rows(&p.xmap, a.x, a.M, a.K, plan.T))
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
    p.tiles = plan.tiles;
    p.total = (long long)plan.tiles * plan.G;
    p.streamk = plan.streamk;
    p.ksplit = plan.ksplit;
    p.bf16 = a.bf16;
    switch (plan.T) {
        case 16: return launch_t<16>(p, plan.grid, stream);
        case 32: return launch_t<32>(p, plan.grid, stream);
        default: return launch_t<64>(p, plan.grid, stream);
    }
}

cudaError_t fp8_init(const DeviceInfo &) {
    if (!tensor_map_encoder()) return cudaErrorSymbolNotFound;
    const struct { const void *f; int smem; } fns[] = {
        {(const void *)fp8_kernel<16>, Cfg<16>::kSmem},
        {(const void *)fp8_kernel<32>, Cfg<32>::kSmem},
        {(const void *)fp8_kernel<64>, Cfg<64>::kSmem}};
    for (const auto &k : fns) {
        cudaError_t e =
            cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
        if (e != cudaSuccess) return e;
    }
    // one CTA per SM whatever T, so one kernel answers for all
    for (int k = 2; k <= kMaxCluster; ++k) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config_t<64>(cfg, attr, k, k, nullptr);
        attr[0] = attr[1];
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&g_clusters[k], fp8_kernel<64>, &cfg);
        if (e != cudaSuccess) return e;
    }
    g_found = true;
    return cudaSuccess;
}

}  // namespace w4a16
