// The 8-bit linear: y [M, N] = x [M, K] w [N, K]^T (+ residual) for e4m3 rows x
// with one fp32 scale per 128 elements and e4m3 weights with one fp32 scale per
// block of 128 x 128 (forum.sourcefind.cn thread "vLLM on Hygon Z100", section
// 六: FP8 checkpoints, dequantised to 16 bits at load there because the GPU has
// no FP8 arithmetic; here the tensor cores take the 8-bit data):
//
//   y[m, n] = sum_b sx[m, b] sw[n / 128, b] * (sum_{k in block b} x[m, k] w[n, k])
//
// The scales change every 128 elements of K, so the tensor cores' accumulator
// holds one block's sum only: per block b a fresh product of 128 weight rows by
// T tokens lands in tensor memory, and four warps add it, times sx sw, to fp32
// sums in registers (one fused multiply-add per element and block).
//
//   MMA shape (swap AB): the MMA's M = 128 weight rows of one tile, its N = T
//   tokens (16, 32, 64 or 128; missing tokens are zero rows of x), K = 32 per
//   instruction, four instructions per block.  A partial last block is filled
//   with zeros by TMA.
//
//   Roles (one CTA per SM, 192 threads): warps 0..3 (thread = weight row) scale
//   and add the blocks and write y; warp 4 streams a block of weights and of x
//   per stage by TMA (128-byte swizzled, K-major), its lanes copy the block's
//   scales next to them; warp 5 issues the products.
//
//   Work: the (tile, block) sequence is cut into equal runs, one per CTA
//   ("stream-K"); a tile split between CTAs is summed by the last of them in K
//   order, so results do not depend on which CTA came last.
//
// Every mbarrier wait is bounded; on expiry the kernel records an error code in
// the device status word, drains what it has in flight, frees its tensor memory
// and exits.
#include <cstring>

#include "w4a16_fp8_common.cuh"
#include "w4a16_internal.h"
#include "w4a16_tcgen05.cuh"

namespace w4a16 {
namespace {

using namespace dev;

constexpr int kTileN = 128;                   // weight rows per tile (MMA M)
constexpr int kStageW = kTileN * kGroup;      // 16 KB of weights per block
constexpr int kEpiWarps = 4;
constexpr int kTmaWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kThreads = 192;
constexpr int kMaxStages = 12;
constexpr int kSmemBudget = 216 * 1024;       // the stages
constexpr int kDBufs = 4;                     // block sums in tensor memory
constexpr int kTmemCols = 512;

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
    int tiles_m;         // token tiles; tile = n_tile * tiles_m + m_tile
    long long total;     // blocks of all tiles
    int tiles;
    int streamk;
    int stages;
    int bf16;
};

template <int T>
struct Cfg {
    static constexpr int kStageX = T * kGroup;
    static constexpr int kStage = kStageW + kStageX;
    static constexpr int kScales = T + 4;  // floats per stage: T of x, then the weight block's
    static constexpr uint32_t kIdesc =     // D f32, A and B e4m3 (0), N = T, M = 128
        (1u << 4) | ((uint32_t)(T >> 3) << 17) | ((uint32_t)(kTileN >> 4) << 24);
    static int stages() {
        const int n = kSmemBudget / (kStage + kScales * 4);
        return n < kMaxStages ? n : kMaxStages;
    }
    // slack for the 1024-byte alignment, the stages, their scales, the
    // barriers, the tensor-memory address, abort and last flags
    static int smem(int stages) {
        return 1024 + stages * (kStage + kScales * 4) + (2 * kMaxStages + 2 * kDBufs) * 8 + 16;
    }
};

// The CTA's work: segments (a tile and a run of its blocks), in order.
struct Walk {
    long long pos, end;
    __device__ __forceinline__ Walk(const Fp8Params &p) {
        if (p.streamk) {
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
        if (p.streamk) {
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

template <int T>
__global__ void __launch_bounds__(kThreads, 1) fp8_kernel(const __grid_constant__ Fp8Params p) {
    using C = Cfg<T>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int NS = p.stages;
    float *sm_scales = reinterpret_cast<float *>(smem + (size_t)NS * C::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_scales + NS * C::kScales);
    uint64_t *empty = full + kMaxStages;
    uint64_t *d_full = empty + kMaxStages;
    uint64_t *d_empty = d_full + kDBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(d_empty + kDBufs);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_last = const_cast<int *>(abort + 1);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    grid_dependents_launch();
    if (threadIdx.x == kTmaWarp * 32) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(full + i), 1 + 32);          // the TMA bytes, each lane's scales
            mbar_init(smem_u32(empty + i), 1 + kEpiWarps);  // the products, each reader of the scales
        }
        for (int i = 0; i < kDBufs; ++i) {
            mbar_init(smem_u32(d_full + i), 1);
            mbar_init(smem_u32(d_empty + i), kEpiWarps);
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
    auto fail = [&](int code) {
        *abort = 1;
        atomicOr(p.status, code);
    };

    Walk walk(p);
    int t, j0, j1;
    if (warp == kTmaWarp) {
        // ------------------------------------------------ producer
        grid_dependency_wait();
        const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
        int c = 0;
        bool ok = true;
        while (ok && walk.next(p, t, j0, j1)) {
            const int nt = t / p.tiles_m, m0 = (t - nt * p.tiles_m) * T;
            for (int j = j0; j < j1; ++j, ++c) {
                const int s = c % NS;
                if (c >= NS && !__all_sync(0xffffffffu, mbar_wait(smem_u32(empty + s),
                                                                  ((c / NS) - 1) & 1, abort))) {
                    if (lane == 0) fail(kErrSlotWait);
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(full + s);
                if (lane == 0) {
                    const uint32_t st = smem_u32(smem + (size_t)s * C::kStage);
                    mbar_arrive_expect_tx(bar, C::kStage);
                    tma_load_2d(st, &p.wmap, j * kGroup, nt * kTileN, bar, pol_w);
                    tma_load_2d(st + kStageW, &p.xmap, j * kGroup, m0, bar, pol_x);
                }
                const uint32_t sc = smem_u32(sm_scales + s * C::kScales);
#pragma unroll
                for (int i = 0; i < (T + 31) / 32; ++i) {
                    const int tt = lane + 32 * i;
                    const bool live = tt < T && m0 + tt < p.M;
                    if (tt < T)
                        cp_async4(sc + 4 * tt, live ? p.xs + (size_t)(m0 + tt) * p.G + j : p.xs,
                                  live ? 4u : 0u);
                }
                if (lane == 0) cp_async4(sc + 4 * T, p.ws + (size_t)nt * p.G + j, 4u);
                cp_async_arrive(bar);
            }
        }
        // every copy issued must have landed before the CTA exits
        if (lane == 0)
            for (int i = c - NS > 0 ? c - NS : 0; i < c; ++i)
                if (!mbar_wait_drain(smem_u32(full + i % NS), (i / NS) & 1))
                    atomicOr(p.status, kErrDrain);
        cp_async_wait_all();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ products
        const uint32_t stages = uniform(smem_u32(smem)), bars = uniform(smem_u32(full));
        const uint32_t tm = uniform(tmem);
        int c = 0;
        bool ok = true;
        while (ok && walk.next(p, t, j0, j1)) {
            for (int j = j0; j < j1; ++j, ++c) {
                const int s = c % NS, d = c % kDBufs;
                if (!mbar_wait_all(bars + 8 * s, (c / NS) & 1, abort)) {
                    if (lane == 0) fail(kErrStageWait);
                    ok = false;
                    break;
                }
                if (c >= kDBufs && !mbar_wait_all(bars + 8 * (2 * kMaxStages + kDBufs + d),
                                                  ((c / kDBufs) - 1) & 1, abort)) {
                    if (lane == 0) fail(kErrSumWait);
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t a = smem_desc_sw128(stages + s * C::kStage);
                    mma_f8_block(tm + d * T, a, a + (kStageW >> 4), C::kIdesc);
                    mma_commit(bars + 8 * (2 * kMaxStages + d));
                    mma_commit(bars + 8 * (kMaxStages + s));
                }
            }
        }
        // the products issued complete before the tensor memory is freed
        if (lane == 0)
            for (int i = c - kDBufs > 0 ? c - kDBufs : 0; i < c; ++i)
                if (!mbar_wait_drain(smem_u32(d_full + i % kDBufs), (i / kDBufs) & 1))
                    atomicOr(p.status, kErrDrain);
    } else {
        // ------------------------------------------------ sums and outputs
        grid_dependency_wait();
        const int r = warp * 32 + lane;  // row within the tile
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        int c = 0;
        bool ok = true;
        while (ok && walk.next(p, t, j0, j1)) {
            const int nt = t / p.tiles_m, m0 = (t - nt * p.tiles_m) * T;
            const int n = nt * kTileN + r;
            float acc[T];
#pragma unroll
            for (int i = 0; i < T; ++i) acc[i] = 0.f;
            for (int j = j0; j < j1; ++j, ++c) {
                const int s = c % NS, d = c % kDBufs;
                // the stage's barrier shows its scales, the sum's its products
                if (!__all_sync(0xffffffffu,
                                mbar_wait(smem_u32(full + s), (c / NS) & 1, abort) &&
                                    mbar_wait(smem_u32(d_full + d), (c / kDBufs) & 1, abort))) {
                    if (lane == 0) fail(kErrSumWait);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *sc = sm_scales + s * C::kScales;
                const float sw = sc[T];
#pragma unroll
                for (int i0 = 0; i0 < T; i0 += 16) {
                    uint32_t u[16];
                    float v[16];
                    tmem_ld(tmem + lanes + d * T + i0, u);
                    tmem_wait_ld(u);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 sx = *reinterpret_cast<const float4 *>(sc + i0 + i);
                        acc[i0 + i] = fmaf(v[i], sx.x * sw, acc[i0 + i]);
                        acc[i0 + i + 1] = fmaf(v[i + 1], sx.y * sw, acc[i0 + i + 1]);
                        acc[i0 + i + 2] = fmaf(v[i + 2], sx.z * sw, acc[i0 + i + 2]);
                        acc[i0 + i + 3] = fmaf(v[i + 3], sx.w * sw, acc[i0 + i + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(d_empty + d));
                    mbar_arrive(smem_u32(empty + s));
                }
            }
            if (!ok) break;
            if (j0 == 0 && j1 == p.G) {  // a whole tile
                if (n < p.N) {
#pragma unroll
                    for (int i = 0; i < T; i += 16) store16(p, m0 + i, n, acc + i);
                }
                continue;
            }
            // part of a tile: the sums go to this CTA's slot, and the last CTA
            // of the tile adds the slots in K order
            const long long tile0 = (long long)t * p.G;
            float *part = p.partials + (size_t)slot_of(p, blockIdx.x, tile0) * T * kTileN + r;
            const int mt = min(T, p.M - m0);
#pragma unroll
            for (int i = 0; i < T; ++i)
                if (i < mt) part[(size_t)i * kTileN] = acc[i];
            __threadfence();
            asm volatile("bar.sync 1, %0;" ::"r"(kEpiWarps * 32) : "memory");
            const int b0 = Walk::owner(p, tile0), b1 = Walk::owner(p, tile0 + p.G - 1);
            if (threadIdx.x == 0)
                *s_last = atomicAdd(p.counters + t, 1u) == (unsigned)(b1 - b0) ? 1 : 0;
            asm volatile("bar.sync 1, %0;" ::"r"(kEpiWarps * 32) : "memory");
            if (*s_last) {
                __threadfence();
                for (int i0 = 0; i0 < mt; i0 += 16) {
                    float sum[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[i] = 0.f;
                    for (int b = b0; b <= b1; ++b) {
                        const float *src = p.partials +
                                           ((size_t)slot_of(p, b, tile0) * T + i0) * kTileN + r;
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            v[i] = i0 + i < mt ? __ldcg(src + (size_t)i * kTileN) : 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[i] += v[i];
                    }
                    if (n < p.N) store16(p, m0 + i0, n, sum);
                }
                if (threadIdx.x == 0) p.counters[t] = 0u;  // ready for the next launch
            }
            // s_last is written again only after every thread has read it
            asm volatile("bar.sync 1, %0;" ::"r"(kEpiWarps * 32) : "memory");
        }
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
cudaError_t launch_t(const Fp8Params &p, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<T>::smem(p.stages);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8_kernel<T>, p);
}

int stages_of(int T) {
    switch (T) {
        case 16: return Cfg<16>::stages();
        case 32: return Cfg<32>::stages();
        case 64: return Cfg<64>::stages();
        default: return Cfg<128>::stages();
    }
}

}  // namespace

Fp8Plan plan_fp8(int M, int N, int K, const DeviceInfo &dev, const Workspace &ws) {
    Fp8Plan pl{};
    pl.T = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    pl.G = (K + kGroup - 1) / kGroup;
    pl.tiles_m = (M + pl.T - 1) / pl.T;
    pl.tiles = (long long)pl.tiles_m * ((N + kTileN - 1) / kTileN);
    const long long total = pl.tiles * pl.G;
    // whole tiles when they fill the last wave; else equal runs of blocks, of
    // at least four blocks each
    const long long waves = (pl.tiles + dev.sm_count - 1) / dev.sm_count;
    pl.streamk = pl.tiles * 100 < waves * dev.sm_count * 95;
    pl.grid = (int)(pl.tiles < dev.sm_count ? pl.tiles : dev.sm_count);
    if (pl.streamk) {
        long long g = total / 4 < dev.sm_count ? total / 4 : dev.sm_count;
        if (g > pl.grid) pl.grid = (int)g;
        pl.ws_bytes = (size_t)2 * pl.grid * pl.T * kTileN * sizeof(float);
        if (pl.grid == pl.tiles || pl.ws_bytes > ws.partial_bytes ||
            pl.tiles > ws.n_counters - kMmaSchedWords) {
            pl.streamk = false;
            pl.ws_bytes = 0;
            pl.grid = (int)(pl.tiles < dev.sm_count ? pl.tiles : dev.sm_count);
        }
    }
    pl.stages = stages_of(pl.T);
    return pl;
}

cudaError_t launch_fp8(const Fp8Args &a, const Fp8Plan &plan, const Workspace &ws,
                       cudaStream_t stream) {
    Fp8Params p;
    memset(&p, 0, sizeof(p));
    if (!encode_fp8_rows(&p.wmap, a.w, a.N, a.K, kTileN) || !encode_fp8_rows(&p.xmap, a.x, a.M, a.K, plan.T))
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
    p.tiles_m = plan.tiles_m;
    p.tiles = (int)plan.tiles;
    p.total = plan.tiles * plan.G;
    p.streamk = plan.streamk;
    p.stages = plan.stages;
    p.bf16 = a.bf16;
    switch (plan.T) {
        case 16: return launch_t<16>(p, plan.grid, stream);
        case 32: return launch_t<32>(p, plan.grid, stream);
        case 64: return launch_t<64>(p, plan.grid, stream);
        default: return launch_t<128>(p, plan.grid, stream);
    }
}

cudaError_t fp8_init(const DeviceInfo &) {
    if (!tensor_map_encoder()) return cudaErrorSymbolNotFound;
    const struct { const void *f; int smem; } fns[] = {
        {(const void *)fp8_kernel<16>, Cfg<16>::smem(Cfg<16>::stages())},
        {(const void *)fp8_kernel<32>, Cfg<32>::smem(Cfg<32>::stages())},
        {(const void *)fp8_kernel<64>, Cfg<64>::smem(Cfg<64>::stages())},
        {(const void *)fp8_kernel<128>, Cfg<128>::smem(Cfg<128>::stages())}};
    for (const auto &k : fns) {
        cudaError_t e =
            cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace w4a16
