// Low-rank adapters of many requests beside a shared projection:
//
//   y[m] = residual[m] + scale_l * B_l (A_l x[m]),   l = ids[m]
//
// with the projection's columns in parts (q, k, v; gate, up), each with R rows of A of its
// own: t[m, p R + r] = sum_k x[m, k] a[l, p R + r, k], y[m, n] += scale_l * sum_r
// t[m, p(n) R + r] b[l, n, r].  (forum.sourcefind.cn thread "vLLM on Hygon Z100", section
// 二, lists the projections of a decoder layer; their adapters are products of the same
// rows, read beside them.)
//
// Three kernels: plan groups the rows by adapter, shrink computes t, expand y.
//   * plan: one CTA counts the rows of each adapter and cuts them into tall tiles of 128
//     rows, or one low tile if they are at most 16.  The order of the rows within an
//     adapter is that of an atomic counter and changes no result: all tiles of an adapter
//     are of one kind, and a row's sums do not depend on its place in a tile.
//   * shrink: a tile of 128 rows and 128 rows of A through shared memory, or a tile of up to
//     16 rows and 32 rows of A straight from memory (each of their weights is used once);
//     K in slices where there are few tiles, whose sums expand adds in order.
//   * expand: a tile and a run of columns; t of the tile as the MMA's M from shared memory.
// All are bound by the bytes of x, y and the adapters (the products are 2 R of each byte
// of y), so the products run on the warp MMA, whose fragments hold 16 contiguous bytes of a
// row of y once the columns of four 8-column tiles are interleaved.
//
// t is fp32; as expand's operand it is split into two values of the 16-bit type, the value
// rounded and the rest rounded, of a row first scaled by a power of two to at most 2: 16
// bits (bf16) or 22 (fp16) of it enter the product, at twice the MMAs, which are not the
// bound up to rank 64.
#include "w4a16_fp8_common.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTall = 128;   // rows of a tall tile
constexpr int kLow = 16;     // and of a low one, at most
constexpr int kPlanThreads = 1024;
constexpr int kTallRanks = 128;  // rows of A of a shrink unit of a tall tile
constexpr int kLowRanks = 32;    // and of a low one
constexpr int kSpan = 128;       // columns of a step of expand, tall tiles
constexpr int kLowSpan = 256;    // and low ones
constexpr int kShrinkStages = 3;
constexpr int kShrinkStage = (kTall + kTallRanks) * 128;  // bytes: 64 k of x and A
constexpr int kShrinkSmem = kShrinkStages * kShrinkStage;

struct Tile {
    int adapter, first, count, pad;
};
// the plan in the scratch: counts, tiles (tall, then low, then those without an adapter),
// then the rows by adapter
struct Plan {
    int tall, low, none, pad;
};

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes to shared memory, the first n from memory, the others zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(p));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
    return v;
}
template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void chain_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ const Plan *plan_of(const LoraArgs &a) {
    return static_cast<const Plan *>(a.scratch);
}
__device__ __forceinline__ const Tile *tiles_of(const LoraArgs &a) {
    return reinterpret_cast<const Tile *>(static_cast<const Plan *>(a.scratch) + 1);
}
__device__ __forceinline__ const int *order_of(const LoraArgs &a) {
    return reinterpret_cast<const int *>(tiles_of(a) + lora_max_tiles(a.M, a.L));
}
__device__ __forceinline__ float *sums_of(const LoraArgs &a) {
    return reinterpret_cast<float *>(static_cast<char *>(a.scratch) + lora_plan_bytes(a.M, a.L));
}
__device__ __forceinline__ int rank_of(const LoraArgs &a, int l) {
    if (l >= a.L) return 0;
    return a.ranks ? min(max(a.ranks[l], 0), a.R) : a.R;
}

// K slices of a tall and of a low tile, the same in shrink and expand: so that the units
// are about as many as CTAs
struct Slices {
    int tall, tall_k, low, low_k;  // slices, and elements of each (a multiple of 64)
};
__device__ __forceinline__ Slices slices_of(const LoraArgs &a, const Plan &p) {
    const int q = a.parts * a.R;
    Slices s;
    const int tu = max(1, p.tall * ((q + kTallRanks - 1) / kTallRanks));
    s.tall = max(1, min(min(a.max_slices, a.K / 256), a.ctas / 2 / tu));
    s.tall_k = ((a.K + s.tall - 1) / s.tall + 63) / 64 * 64;
    s.tall = (a.K + s.tall_k - 1) / s.tall_k;
    const int lu = max(1, p.low * ((q + kLowRanks - 1) / kLowRanks));
    s.low = max(1, min(min(a.max_slices, a.K / 256), a.ctas / lu));
    s.low_k = ((a.K + s.low - 1) / s.low + 63) / 64 * 64;
    s.low = (a.K + s.low_k - 1) / s.low_k;
    return s;
}

// ---------------------------------------------------------------------------
// plan: one CTA.  Bin l < L: the rows of adapter l; bin L: those without one.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(LoraArgs a) {
    __shared__ int count[kMaxAdapters + 1], sums[3][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    chain_start();
    Plan *plan = static_cast<Plan *>(a.scratch);
    Tile *tiles = const_cast<Tile *>(tiles_of(a));
    int *order = const_cast<int *>(order_of(a));
    for (int l = tid; l <= a.L; l += kPlanThreads) count[l] = 0;
    __syncthreads();
    // whole warps take each step together, for the matches
    const int rounds = (a.M + kPlanThreads - 1) / kPlanThreads;
    for (int i = 0; i < rounds; ++i) {
        const int m = i * kPlanThreads + tid;
        int l = m < a.M ? a.ids[m] : -1;
        if ((unsigned)l >= (unsigned)a.L || rank_of(a, l) == 0) l = a.L;
        const unsigned same = __match_any_sync(0xffffffffu, m < a.M ? l : -1);
        if (m < a.M && lane == __ffs(same) - 1) atomicAdd(&count[l], __popc(same));
    }
    __syncthreads();
    // scans over the adapters (one per thread) of rows, tall and low tiles
    const int n = tid < a.L ? count[tid] : 0;
    int v[3] = {n, n > kLow ? (n + kTall - 1) / kTall : 0, n > 0 && n <= kLow};
    const int own[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int u = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += u;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 3; ++i) sums[i][warp] = v[i];
    __syncthreads();
    int all[3] = {0, 0, 0};
    for (int w = 0; w < 32; ++w)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (w < warp) v[i] += sums[i][w];
            all[i] += sums[i][w];
        }
    const int none = a.M - all[0], none_tiles = (none + kTall - 1) / kTall;
    if (tid == 0) *plan = {all[1], all[2], none_tiles, 0};
    const int first = v[0] - own[0];
    for (int i = 0; i < own[1]; ++i)
        tiles[v[1] - own[1] + i] = {tid, first + i * kTall, min(kTall, n - i * kTall), 0};
    if (own[2]) tiles[all[1] + v[2] - 1] = {tid, first, n, 0};
    for (int i = tid; i < none_tiles; i += kPlanThreads)
        tiles[all[1] + all[2] + i] = {a.L, all[0] + i * kTall, min(kTall, none - i * kTall), 0};
    if (tid < a.L) count[tid] = first;
    if (tid == 0) count[a.L] = all[0];
    __syncthreads();
    for (int i = 0; i < rounds; ++i) {
        const int m = i * kPlanThreads + tid;
        int l = m < a.M ? a.ids[m] : -1;
        if ((unsigned)l >= (unsigned)a.L || rank_of(a, l) == 0) l = a.L;
        const unsigned same = __match_any_sync(0xffffffffu, m < a.M ? l : -1);
        const int lead = __ffs(same) - 1;
        int at = 0;
        if (m < a.M && lane == lead) at = atomicAdd(&count[l], __popc(same));
        at = __shfl_sync(0xffffffffu, at, lead);
        if (m < a.M) order[at + __popc(same & ((1u << lane) - 1))] = m;
    }
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// A tile of up to 128 rows, rows q0 .. q0 + 127 of A, k0 <= k < k1.  Warps 4 x 2: 32 rows,
// every other 8 rows of A.
template <bool kBf16>
__device__ void shrink_tall(const LoraArgs &a, const Tile &t, int q0, int k0, int k1, int slice,
                            uint8_t *smem) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int wm = warp >> 1, wn = warp & 1;
    const int Q = a.parts * a.R, rank = rank_of(a, t.adapter);
    const uint32_t base = smem_of(smem);
    const int *order = order_of(a) + t.first;
    // this thread's 16 bytes of four rows of x and of A, per stage
    const int col = tid & 7, r0 = tid >> 3;
    const uint16_t *xp[4], *ap[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i, q = q0 + r;
        xp[i] = r < t.count ? a.x + (size_t)order[r] * a.K : nullptr;
        ap[i] = q < Q && q % a.R < rank ? a.a + ((size_t)t.adapter * Q + q) * a.K : nullptr;
    }
    const int ranks = min(kTallRanks, Q - q0);
    auto issue = [&](int s) {
        const uint32_t st = base + s % kShrinkStages * kShrinkStage;
        const int k = k0 + s * 64 + col * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i;
            const uint32_t at = (r << 7) + ((col ^ ((r & 1) << 2)) << 4);
            if (r < t.count) copy16(st + at, k < k1 ? xp[i] + k : a.x, k < k1 ? 16 : 0);
            if (r < ranks)
                copy16(st + kTall * 128 + at, ap[i] && k < k1 ? ap[i] + k : a.a,
                       ap[i] && k < k1 ? 16 : 0);
        }
    };
    const int steps = (k1 - k0 + 63) / 64;
    const int tiles_n = (ranks + 7) / 8;
    float acc[2][8][4] = {};
#pragma unroll
    for (int s = 0; s < kShrinkStages - 1; ++s) {
        if (s < steps) issue(s);
        commit_copies();
    }
    for (int s = 0; s < steps; ++s) {
        wait_copies<kShrinkStages - 2>();
        __syncthreads();
        if (s + kShrinkStages - 1 < steps) issue(s + kShrinkStages - 1);
        commit_copies();
        const uint32_t st = base + s % kShrinkStages * kShrinkStage;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = (((h * 4 + c) ^ ((g & 1) << 2)) << 4);
            uint4 x[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    x[i][u] = lds128(st + ((wm * 32 + i * 16 + u * 8 + g) << 7) + at);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (2 * n + wn >= tiles_n) break;
                const uint4 w = lds128(st + kTall * 128 + (((2 * n + wn) * 8 + g) << 7) + at);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma<kBf16>(acc[i][n], x[i][0].x, x[i][1].x, x[i][0].y, x[i][1].y, w.x, w.y);
                    mma<kBf16>(acc[i][n], x[i][0].z, x[i][1].z, x[i][0].w, x[i][1].w, w.z, w.w);
                }
            }
        }
    }
    wait_copies<0>();
    __syncthreads();  // the next unit fills the stages
    float *sums = sums_of(a) + (size_t)slice * a.M * Q;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = wm * 32 + i * 16 + u * 8 + g;
            if (r >= t.count) continue;
            float *row = sums + (size_t)order[r] * Q;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int q = q0 + (2 * n + wn) * 8 + c * 2;
                if (q < Q)
                    *reinterpret_cast<float2 *>(row + q) =
                        make_float2(acc[i][n][2 * u], acc[i][n][2 * u + 1]);
            }
        }
}

// A tile of up to 16 rows, rows q0 .. q0 + 31 of A, k0 <= k < k1, every warp its own 64 k
// in turn.
template <bool kBf16>
__device__ void shrink_low(const LoraArgs &a, const Tile &t, int q0, int k0, int k1, int slice,
                           uint8_t *smem) {
    constexpr int NT = kLowRanks / 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int Q = a.parts * a.R, rank = rank_of(a, t.adapter);
    const int *order = order_of(a) + t.first;
    const uint16_t *x0 = a.x + (size_t)order[min(g, t.count - 1)] * a.K,
                   *x1 = a.x + (size_t)order[min(g + 8, t.count - 1)] * a.K;
    const uint16_t *w[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int q = q0 + n * 8 + g;
        w[n] = q < Q && q % a.R < rank ? a.a + ((size_t)t.adapter * Q + q) * a.K : nullptr;
    }
    float acc[NT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int k = k0 + warp * 64; k < k1; k += kWarps * 64) {
        uint4 xv[2][2], wv[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kk = k + h * 32 + c * 8;
            const bool in = kk < k1;
            xv[h][0] = in ? *reinterpret_cast<const uint4 *>(x0 + kk) : zero;
            xv[h][1] = in ? *reinterpret_cast<const uint4 *>(x1 + kk) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                wv[n][h] = in && w[n] ? *reinterpret_cast<const uint4 *>(w[n] + kk) : zero;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma<kBf16>(acc[n], xv[h][0].x, xv[h][1].x, xv[h][0].y, xv[h][1].y, wv[n][h].x,
                           wv[n][h].y);
                mma<kBf16>(acc[n], xv[h][0].z, xv[h][1].z, xv[h][0].w, xv[h][1].w, wv[n][h].z,
                           wv[n][h].w);
            }
    }
    // the warps' sums, in order
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[(warp * kLow + g + (i >> 1) * 8) * (kLowRanks + 8) + n * 8 + c * 2 + (i & 1)] =
                acc[n][i];
    __syncthreads();
    float *sums = sums_of(a) + (size_t)slice * a.M * Q;
    for (int i = tid; i < t.count * kLowRanks; i += kThreads) {
        const int r = i / kLowRanks, q = i % kLowRanks;
        if (q0 + q >= Q) continue;
        float v = 0.f;
        for (int u = 0; u < kWarps; ++u) v += red[(u * kLow + r) * (kLowRanks + 8) + q];
        sums[(size_t)order[r] * Q + q0 + q] = v;
    }
    __syncthreads();
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(LoraArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    chain_start();
    const Plan p = *plan_of(a);
    const Slices sl = slices_of(a, p);
    const int Q = a.parts * a.R;
    const int tq = (Q + kTallRanks - 1) / kTallRanks, lq = (Q + kLowRanks - 1) / kLowRanks;
    const int tall = p.tall * tq * sl.tall, units = tall + p.low * lq * sl.low;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        if (u < tall) {
            const int q = u % tq, s = u / tq % sl.tall;
            const Tile t = tiles_of(a)[u / tq / sl.tall];
            shrink_tall<kBf16>(a, t, q * kTallRanks, s * sl.tall_k, min(a.K, (s + 1) * sl.tall_k),
                               s, smem);
        } else {
            const int v = u - tall, q = v % lq, s = v / lq % sl.low;
            const Tile t = tiles_of(a)[p.tall + v / lq / sl.low];
            shrink_low<kBf16>(a, t, q * kLowRanks, s * sl.low_k, min(a.K, (s + 1) * sl.low_k), s,
                              smem);
        }
    }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
// bytes of a row of R values in shared memory: whole 16s, an odd number of 32 bytes so that
// rows next to each other lie in other banks
__host__ __device__ constexpr int row_pitch(int R) {
    return (((R + 15) / 16) | 1) * 32;
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
    return (uint32_t)float_to_half_bits(lo, bf16) | (uint32_t)float_to_half_bits(hi, bf16) << 16;
}

// Row m's t of a part (the sum of its slices) -> its two halves in shared memory and the
// factor that undoes their scaling, by one warp.  Zeros from the adapter's rank on.
template <bool kBf16>
__device__ __forceinline__ void stage_row(const LoraArgs &a, int m, int part, int rank, int slices,
                                          uint8_t *hi, uint8_t *lo, float *factor) {
    const int lane = threadIdx.x & 31, Q = a.parts * a.R;
    const float *row = sums_of(a) + (size_t)m * Q + part * a.R;
    const int padded = (a.R + 15) / 16 * 16;
    float v[kMaxRank / 64][2];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxRank / 64; ++i) {
        const int r = i * 64 + lane * 2;
        v[i][0] = v[i][1] = 0.f;
        if (r < rank) {  // R is even, and so are the addresses
            for (int s = 0; s < slices; ++s) {
                const float2 u = *reinterpret_cast<const float2 *>(row + (size_t)s * a.M * Q + r);
                v[i][0] += u.x, v[i][1] += u.y;
            }
            if (r + 1 >= rank) v[i][1] = 0.f;
        }
        most = fmaxf(most, fmaxf(fabsf(v[i][0]), fabsf(v[i][1])));
    }
    // (a NaN does not count here, and an Inf leaves the row as it is)
    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(most)) >> 23;
    const int e = top >= 255 || top == 0 ? 127 : min(max((int)top, 2), 252);
    const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
    if (lane == 0) *factor = __uint_as_float((uint32_t)e << 23);
#pragma unroll
    for (int i = 0; i < kMaxRank / 64; ++i) {
        const int r = i * 64 + lane * 2;
        if (r >= padded) continue;
        float h[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float w = v[i][j] * down;
            h[j] = half_bits_to_float(float_to_half_bits(w, kBf16), kBf16);
            l[j] = isfinite(h[j]) ? w - h[j] : 0.f;
        }
        *reinterpret_cast<uint32_t *>(hi + r * 2) = pack16(h[0], h[1], kBf16);
        *reinterpret_cast<uint32_t *>(lo + r * 2) = pack16(l[0], l[1], kBf16);
    }
}

// 8 columns of a row of y: v + residual, of which `n` exist.  No adapter: the residual
// itself.
template <bool kBf16, bool kVec>
struct Cells {
    uint4 r;
    __device__ __forceinline__ void load(const LoraArgs &a, size_t at, int n) {
        r = make_uint4(0, 0, 0, 0);
        if (!a.residual) return;
        if constexpr (kVec) {
            if (n > 0) r = *reinterpret_cast<const uint4 *>(a.residual + at);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) w[i >> 1] |= (uint32_t)a.residual[at + i] << (16 * (i & 1));
            r = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ void store(const LoraArgs &a, size_t at, int n, const float (&v)[8],
                                          bool adapted) {
        uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if (adapted)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack16(half_bits_to_float((uint16_t)w[i], kBf16) + v[2 * i],
                              half_bits_to_float((uint16_t)(w[i] >> 16), kBf16) + v[2 * i + 1],
                              kBf16);
        if constexpr (kVec) {
            if (n > 0) *reinterpret_cast<uint4 *>(a.y + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) a.y[at + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
};

// where column j of 32 lies among the rows of four 8-column MMA tiles so that a lane's
// results are 8 neighbours: MMA tile (j >> 1) & 3, its column (j >> 3) * 2 + (j & 1)
__device__ __forceinline__ int interleaved(int j) {
    return (j >> 1 & 3) * 8 + (j >> 3) * 2 + (j & 1);
}

// 16 rows from `a_hi`, 32 columns: the warp's sums; b(n, k16) gives the fragment of 8-column
// tile n
template <bool kBf16, typename B>
__device__ __forceinline__ void product32(float (&acc)[4][4], uint32_t a_hi, uint32_t a_lo,
                                          int pitch, int ksteps, B b) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int k = 0; k < ksteps; ++k) {
        const uint32_t at = g * pitch + k * 32 + c * 8;
        const uint2 h0 = lds64(a_hi + at), h1 = lds64(a_hi + at + 8 * pitch),
                    l0 = lds64(a_lo + at), l1 = lds64(a_lo + at + 8 * pitch);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const uint2 w = b(n, k);
            mma<kBf16>(acc[n], h0.x, h1.x, h0.y, h1.y, w.x, w.y);
            mma<kBf16>(acc[n], l0.x, l1.x, l0.y, l1.y, w.x, w.y);
        }
    }
}

// A tall tile, columns n0 <= n < n1 of a part: every warp 16 rows.
template <bool kBf16, bool kVec>
__device__ void expand_tall(const LoraArgs &a, const Tile &t, int part, int n0, int n1, int slices,
                            uint8_t *smem) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int rank = rank_of(a, t.adapter), pitch = row_pitch(a.R), ksteps = (rank + 15) / 16;
    const int *order = order_of(a) + t.first;
    uint8_t *hi = smem, *lo = smem + kTall * pitch, *bs = smem + 2 * kTall * pitch;
    __shared__ float factor[kTall];
    const bool adapted = rank > 0;
    if (!adapted && a.residual == a.y) return;
    auto issue = [&](int n, int stage) {  // columns n .. n + 127 of B
        const int chunks = ksteps * 2;
        for (int i = tid; i < kSpan * chunks; i += kThreads) {
            const int j = i / chunks, r = i % chunks * 8;
            const bool valid = n + j < n1 && r < rank;
            copy16(smem_of(bs) + stage * kSpan * pitch +
                       ((j & ~31) + interleaved(j & 31)) * pitch + r * 2,
                   valid ? a.b + ((size_t)t.adapter * a.N + n + j) * a.R + r : a.b,
                   valid ? min(2 * (rank - r), 16) : 0);
        }
    };
    if (adapted) {
        issue(n0, 0);
        commit_copies();
        for (int i = 0; i < kLow; ++i) {
            const int r = warp * kLow + i;
            if (r < t.count)
                stage_row<kBf16>(a, order[r], part, rank, slices, hi + r * pitch, lo + r * pitch,
                                 factor + r);
        }
        __syncwarp();
    }
    const int r[2] = {warp * kLow + g, warp * kLow + g + 8};
    const bool in[2] = {r[0] < t.count, r[1] < t.count};
    const size_t at[2] = {in[0] ? (size_t)order[r[0]] * a.N : 0,
                          in[1] ? (size_t)order[r[1]] * a.N : 0};
    const float scale = adapted ? a.scales[t.adapter] : 0.f;
    const float f[2] = {adapted && in[0] ? scale * factor[r[0]] : 0.f,
                        adapted && in[1] ? scale * factor[r[1]] : 0.f};
    for (int n = n0, stage = 0; n < n1; n += kSpan, stage ^= 1) {
        Cells<kBf16, kVec> cell[4][2];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int col = n + s * 32 + c * 8;
                cell[s][u].load(a, at[u] + col, in[u] ? n1 - col : 0);
            }
        if (adapted) {
            wait_copies<0>();
            __syncthreads();  // this step's columns are there, the last one's are free
            if (n + kSpan < n1) issue(n + kSpan, stage ^ 1);
            commit_copies();
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (n + s * 32 >= n1) break;
            float acc[4][4];
            const uint32_t b0 = smem_of(bs) + (stage * kSpan + s * 32 + g) * pitch + c * 8;
            product32<kBf16>(acc, smem_of(hi) + warp * kLow * pitch,
                             smem_of(lo) + warp * kLow * pitch, pitch, ksteps,
                             [&](int j, int k) { return lds64(b0 + j * 8 * pitch + k * 32); });
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) v[2 * j + i] = acc[j][2 * u + i] * f[u];
                const int col = n + s * 32 + c * 8;
                cell[s][u].store(a, at[u] + col, in[u] ? n1 - col : 0, v, adapted);
            }
        }
    }
    wait_copies<0>();
    __syncthreads();  // the next unit fills the same memory
}

// A low tile, columns n0 <= n < n1 of a part: every warp 32 columns, B from memory (each of
// its weights is used once).
template <bool kBf16, bool kVec>
__device__ void expand_low(const LoraArgs &a, const Tile &t, int part, int n0, int n1, int slices,
                           uint8_t *smem) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int rank = rank_of(a, t.adapter), pitch = row_pitch(a.R), ksteps = (rank + 15) / 16;
    const int *order = order_of(a) + t.first;
    uint8_t *hi = smem, *lo = smem + kLow * pitch;
    __shared__ float factor[kLow];
    for (int i = warp; i < t.count; i += kWarps)
        stage_row<kBf16>(a, order[i], part, rank, slices, hi + i * pitch, lo + i * pitch,
                         factor + i);
    __syncthreads();
    const int r[2] = {g, g + 8};
    const bool in[2] = {r[0] < t.count, r[1] < t.count};
    const size_t at[2] = {in[0] ? (size_t)order[r[0]] * a.N : 0,
                          in[1] ? (size_t)order[r[1]] * a.N : 0};
    const float scale = a.scales[t.adapter];
    const float f[2] = {in[0] ? scale * factor[r[0]] : 0.f, in[1] ? scale * factor[r[1]] : 0.f};
    for (int n = n0 + warp * 32; n < n1; n += kWarps * 32) {
        Cells<kBf16, kVec> cell[2];
        const int col = n + c * 8;
#pragma unroll
        for (int u = 0; u < 2; ++u) cell[u].load(a, at[u] + col, in[u] ? n1 - col : 0);
        // lane g's column of MMA tile j
        const uint16_t *w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = n + (g >> 1) * 8 + j * 2 + (g & 1);
            w[j] = m < n1 ? a.b + ((size_t)t.adapter * a.N + m) * a.R + c * 4 : nullptr;
        }
        float acc[4][4];
        product32<kBf16>(acc, smem_of(hi), smem_of(lo), pitch, ksteps, [&](int j, int k) {
            uint2 v = make_uint2(0, 0);
            const int left = rank - (k * 16 + c * 4);
            if (w[j] && left > 0) {
                v = *reinterpret_cast<const uint2 *>(w[j] + k * 16);
                if (left < 4) {  // nothing beyond the rank
                    v.x &= left == 1 ? 0xffffu : ~0u;
                    v.y &= left == 3 ? 0xffffu : 0u;
                }
            }
            return v;
        });
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) v[2 * j + i] = acc[j][2 * u + i] * f[u];
            cell[u].store(a, at[u] + col, in[u] ? n1 - col : 0, v, true);
        }
    }
    __syncthreads();  // the next unit fills the same memory
}

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) expand_kernel(LoraArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    chain_start();
    const Plan p = *plan_of(a);
    const Slices sl = slices_of(a, p);
    // runs of columns: whole steps, about four units per CTA, never past a part's end
    int steps = 0, low_steps = 0;
    for (int i = 0; i < a.parts; ++i) {
        steps += (a.part[i] + kSpan - 1) / kSpan;
        low_steps += (a.part[i] + kLowSpan - 1) / kLowSpan;
    }
    const int tall_tiles = p.tall + p.none;
    const int run = min(max((int)((long long)tall_tiles * steps / (4 * (int)gridDim.x)), 1), 16) *
                    kSpan;
    const int low_run =
        min(max((int)((long long)p.low * low_steps / (4 * (int)gridDim.x)), 1), 16) * kLowSpan;
    int runs = 0, low_runs = 0;
    for (int i = 0; i < a.parts; ++i) {
        runs += (a.part[i] + run - 1) / run;
        low_runs += (a.part[i] + low_run - 1) / low_run;
    }
    const long long tall = (long long)tall_tiles * runs,
                    units = tall + (long long)p.low * low_runs;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const bool is_low = u >= tall;
        const int per = is_low ? low_runs : runs, width = is_low ? low_run : run;
        const long long v = is_low ? u - tall : u;
        int tile = (int)(v / per), i = (int)(v % per), part = 0, first = 0;
        for (; i >= (a.part[part] + width - 1) / width; ++part) {
            i -= (a.part[part] + width - 1) / width;
            first += a.part[part];
        }
        const int n0 = first + i * width, n1 = min(n0 + width, first + a.part[part]);
        if (is_low) {
            const Tile t = tiles_of(a)[p.tall + tile];
            expand_low<kBf16, kVec>(a, t, part, n0, n1, sl.low, smem);
        } else {
            if (tile >= p.tall) tile += p.low;
            const Tile t = tiles_of(a)[tile];
            expand_tall<kBf16, kVec>(a, t, part, n0, n1, sl.tall, smem);
        }
    }
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), int grid, int threads, int smem,
                           cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int expand_smem(int R) { return (2 * kTall + 2 * kSpan) * row_pitch(R); }

template <bool kBf16>
cudaError_t launch_type(const LoraArgs &a, bool vec, cudaStream_t stream) {
    cudaError_t e = launch_chained(plan_kernel, 1, kPlanThreads, 0, stream, a);
    if (e == cudaSuccess)
        e = launch_chained(shrink_kernel<kBf16>, a.ctas, kThreads, kShrinkSmem, stream, a);
    if (e != cudaSuccess) return e;
    return vec ? launch_chained(expand_kernel<kBf16, true>, a.ctas, kThreads, expand_smem(a.R),
                                stream, a)
               : launch_chained(expand_kernel<kBf16, false>, a.ctas, kThreads, expand_smem(a.R),
                                stream, a);
}

}  // namespace

cudaError_t launch_lora(LoraArgs a, bool bf16, const DeviceInfo &dev, cudaStream_t stream) {
    a.ctas = 2 * dev.sm_count;
    a.max_slices = lora_max_slices(a.M);
    // 16-byte accesses of y and the residual
    bool vec = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.residual & 15) == 0;
    for (int i = 0; i < a.parts; ++i) vec = vec && a.part[i] % 8 == 0;
    return bf16 ? launch_type<true>(a, vec, stream) : launch_type<false>(a, vec, stream);
}

cudaError_t lora_init() {
    const struct { const void *f; int bytes; } kernels[] = {
        {(const void *)shrink_kernel<true>, kShrinkSmem},
        {(const void *)shrink_kernel<false>, kShrinkSmem},
        {(const void *)expand_kernel<true, true>, expand_smem(kMaxRank)},
        {(const void *)expand_kernel<true, false>, expand_smem(kMaxRank)},
        {(const void *)expand_kernel<false, true>, expand_smem(kMaxRank)},
        {(const void *)expand_kernel<false, false>, expand_smem(kMaxRank)}};
    for (const auto &k : kernels) {
        cudaError_t e =
            cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.bytes);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace w4a16
