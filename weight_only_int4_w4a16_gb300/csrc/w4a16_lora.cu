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
// The rows are grouped by adapter, those of an adapter in tall tiles of 128 rows, or in one
// low tile if they are at most 16.  All tiles of an adapter are of one kind, and a row's
// sums do not depend on its place in a tile, so the order within an adapter changes no
// result.  Up to 1024 rows each CTA groups for itself in shared memory; more are grouped by
// a kernel of one CTA before (plan_kernel).
//   * shrink: t, a cluster of 8 CTAs per tile and block of A's rows, each with an eighth of
//     K, whose sums meet through distributed shared memory (one CTA per SM walking all of
//     K would leave most SMs idle: a tall tile's x is 1.3 MB at K 5120, and there are few).
//     A tall tile and 128 rows of A go through shared memory; a low one and 32 rows of A
//     come straight from memory, since each of their weights is used once.
//   * expand: y.  All steps (64 columns of a tall tile, 32 of a low one for each warp) are
//     one sequence of which every CTA takes an equal run; B and the residual come through
//     rings of asynchronous copies, which start before shrink has ended.
// Both are bound by the bytes of x, y and the adapters (R products per byte of y read and
// written), so they run on the warp MMA, whose fragments hold 16 contiguous bytes of a row
// of y once the columns of four 8-column tiles are interleaved.
//
// t is fp32; as expand's operand it is split into two values of the 16-bit type, the value
// rounded and the rest rounded, of a row first scaled by a power of two to at most 2: 16
// bits (bf16) or 22 (fp16) of it enter the product, at twice the MMAs, which are not the
// bound up to rank 64.
#include "w4a16_routed.cuh"

namespace w4a16 {
namespace {

using namespace routed;

constexpr int kTall = 128;   // rows of a tall tile
constexpr int kLow = 16;     // and of a low one, at most
constexpr int kPlanThreads = 1024;
constexpr int kCluster = 8;      // CTAs that share a shrink unit's K
constexpr int kTallRanks = 128;  // rows of A of a shrink unit of a tall tile
constexpr int kLowRanks = 32;    // and of a low one
constexpr int kShrinkStages = 3;
constexpr int kShrinkStage = (kTall + kTallRanks) * 128;  // bytes: 64 k of x and A
constexpr int kShrinkSmem = kShrinkStages * kShrinkStage;
constexpr int kTallCols = 64;  // columns of a step of expand, tall tiles
constexpr int kLowCols = 32;   // low ones

struct Tile {
    uint16_t adapter, first, count, pad;
};
// tall tiles, then low ones, then those of rows without an adapter (as high as tall ones)
struct Counts {
    int tall, low, none, pad;
};
struct Plan {
    Counts n;
    const Tile *tiles;
    const uint16_t *order;  // the rows by adapter
};
// a CTA's own, of up to kMaxRows rows
struct LocalPlan {
    Counts n;
    Tile tiles[kMaxRows + kMaxRows / kTall + 2];
    uint16_t order[kMaxRows];
};
static_assert(sizeof(Counts) == 16 && sizeof(Tile) == 8, "as lora_plan_bytes counts them");
static_assert(kMaxRows == kLoraLocalRows, "as lora_kernels counts them");
static_assert(kMaxAdapters + 1 <= kMaxBins, "the sort holds every adapter and none");

__device__ __forceinline__ int rank_of(const LoraArgs &a, int l) {
    if (l >= a.L) return 0;
    return a.ranks ? min(max(a.ranks[l], 0), a.R) : a.R;
}
// the row's adapter, L for none
__device__ __forceinline__ int bin_of(const LoraArgs &a, int m) {
    const int l = a.ids[m];
    return (unsigned)l < (unsigned)a.L && rank_of(a, l) > 0 ? l : a.L;
}
__device__ __forceinline__ int tall_tiles(int n) {
    return n > kLow ? (n + kTall - 1) / kTall : 0;
}
__device__ __forceinline__ void put_tiles(Tile *tiles, int l, int first, int n) {
    for (int i = 0; i < n; i += kTall)
        tiles[i / kTall] = {(uint16_t)l, (uint16_t)(first + i), (uint16_t)min(kTall, n - i), 0};
}

__device__ Counts *shared_counts(const LoraArgs &a) { return static_cast<Counts *>(a.scratch); }
__device__ __forceinline__ float *sums_of(const LoraArgs &a) {
    return reinterpret_cast<float *>(static_cast<char *>(a.scratch) + lora_plan_bytes(a.M, a.L));
}
__device__ __forceinline__ Plan shared_plan(const LoraArgs &a) {
    Plan p;
    p.tiles = reinterpret_cast<const Tile *>(shared_counts(a) + 1);
    p.order = reinterpret_cast<const uint16_t *>(p.tiles + lora_max_tiles(a.M, a.L));
    return p;
}

// The plan of the call; `space` is free again afterwards.
__device__ Plan make_plan(const LoraArgs &a, LocalPlan &own, void *space) {
    Plan p = shared_plan(a);
    if (a.M > kMaxRows) {
        p.n = *shared_counts(a);
        return p;
    }
    group_rows(
        *static_cast<RowSort *>(space), own.order, a.M, a.L + 1,
        [&](int m) { return bin_of(a, m); },
        [&](int l, int n) {  // rows, tall tiles << 11, low tiles << 21
            if (l == a.L) return (unsigned)n;
            return (unsigned)n | (unsigned)tall_tiles(n) << 11 |
                   (unsigned)(n > 0 && n <= kLow) << 21;
        },
        [&](int l, int n, unsigned at, unsigned total) {
            const int tall = total >> 11 & 1023, low = total >> 21, first = at & 2047;
            if (l == a.L) {
                own.n = {tall, low, (n + kTall - 1) / kTall, 0};
                put_tiles(own.tiles + tall + low, l, first, n);
            } else if (n > 0) {
                put_tiles(own.tiles + (n <= kLow ? tall + (at >> 21) : at >> 11 & 1023), l, first,
                          n);
            }
        });
    p.n = own.n;
    p.tiles = own.tiles;
    p.order = own.order;
    return p;
}

// ---------------------------------------------------------------------------
// plan: one CTA, more than kMaxRows rows.  Bin l < L: the rows of adapter l; bin L: those
// without one.  The order within a bin is that of an atomic counter.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(LoraArgs a) {
    __shared__ int count[kMaxAdapters + 1], sums[3][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_last();
    launch_next();
    const Plan plan = shared_plan(a);
    Tile *tiles = const_cast<Tile *>(plan.tiles);
    uint16_t *order = const_cast<uint16_t *>(plan.order);
    for (int l = tid; l <= a.L; l += kPlanThreads) count[l] = 0;
    __syncthreads();
    // whole warps take each step together, for the matches
    const int rounds = (a.M + kPlanThreads - 1) / kPlanThreads;
    for (int i = 0; i < rounds; ++i) {
        const int m = i * kPlanThreads + tid;
        const int l = m < a.M ? bin_of(a, m) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, l);
        if (l >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[l], __popc(same));
    }
    __syncthreads();
    // scans over the adapters (one per thread) of rows, tall and low tiles
    const int n = tid < a.L ? count[tid] : 0;
    int v[3] = {n, tall_tiles(n), n > 0 && n <= kLow};
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
    const int none = a.M - all[0], first = v[0] - own[0];
    if (tid == 0) {
        *shared_counts(a) = {all[1], all[2], (none + kTall - 1) / kTall, 0};
        count[a.L] = all[0];
    }
    put_tiles(tiles + (own[2] ? all[1] + v[2] - own[2] : v[1] - own[1]), tid, first, n);
    for (int i = tid * kTall; i < none; i += kPlanThreads * kTall)
        put_tiles(tiles + all[1] + all[2] + i / kTall, a.L, all[0] + i, min(kTall, none - i));
    if (tid < a.L) count[tid] = first;
    __syncthreads();
    for (int i = 0; i < rounds; ++i) {
        const int m = i * kPlanThreads + tid;
        const int l = m < a.M ? bin_of(a, m) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, l);
        const int lead = __ffs(same) - 1;
        int at = 0;
        if (l >= 0 && lane == lead) at = atomicAdd(&count[l], __popc(same));
        at = __shfl_sync(0xffffffffu, at, lead);
        if (l >= 0) order[at + __popc(same & ((1u << lane) - 1))] = (uint16_t)m;
    }
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// All threads of the cluster's CTAs come to each of these, whatever their share of the work:
// these waits have no limit of their own, but nothing before them waits.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float4 load_peer(uint32_t at, int rank) {
    float4 v;
    uint32_t peer;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer)
                 : "memory");
    return v;
}

// The CTAs' sums of `rows` rows and `ranks` (a multiple of 4) rows of A, [row][pitch] fp32 at
// the start of each one's shared memory -> t, in the order of K: every CTA writes an eighth
// of the rows.
__device__ void join_sums(const LoraArgs &a, const uint16_t *order, int rows, int q0, int ranks,
                          int pitch, uint32_t smem) {
    const int Q = a.parts * a.R, quads = ranks / 4;
    cluster_sync();
    const int share = (rows + kCluster - 1) / kCluster, first = (int)cluster_rank() * share;
    const int n = max(0, min(share, rows - first)) * quads;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int r = first + i / quads, q = i % quads * 4;
        float4 v[kCluster];
#pragma unroll
        for (int u = 0; u < kCluster; ++u) v[u] = load_peer(smem + (r * pitch + q) * 4, u);
#pragma unroll
        for (int u = 1; u < kCluster; ++u)
            v[0].x += v[u].x, v[0].y += v[u].y, v[0].z += v[u].z, v[0].w += v[u].w;
        *reinterpret_cast<float4 *>(sums_of(a) + (size_t)order[r] * Q + q0 + q) = v[0];
    }
    cluster_sync();  // the others have read this CTA's
}

// A tile of up to 128 rows, rows q0 .. q0 + 127 of A, k0 <= k < k1.  Warps 4 x 2: 32 rows,
// every other 8 rows of A.
template <bool kBf16>
__device__ void shrink_tall(const LoraArgs &a, const uint16_t *order, const Tile &t, int q0, int k0,
                            int k1, uint8_t *smem) {
    constexpr int kPitch = kTallRanks + 4;
    static_assert(kTall * kPitch * 4 <= kShrinkSmem, "the sums fit the stages");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int wm = warp >> 1, wn = warp & 1;
    const int Q = a.parts * a.R, rank = rank_of(a, t.adapter);
    const uint32_t base = smem_of(smem);
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
        const int k = k0 + s * 64 + col * 8, in = k < k1 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i;
            // piece c of row r is at c ^ 4 in odd rows: lanes of neighbouring rows read
            // other banks
            const uint32_t at = (r << 7) + ((col ^ ((r & 1) << 2)) << 4);
            if (xp[i]) copy16(st + at, in ? xp[i] + k : a.x, in);
            if (r < ranks)
                copy16(st + kTall * 128 + at, ap[i] && in ? ap[i] + k : a.a, ap[i] ? in : 0);
        }
    };
    const int steps = k1 > k0 ? (k1 - k0 + 63) / 64 : 0;
    const int tiles_n = ranks / 8;
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
    __syncthreads();  // the sums go where the stages were
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float *row = red + (wm * 32 + i * 16 + u * 8 + g) * kPitch + c * 2;
#pragma unroll
            for (int n = 0; n < 8; ++n)
                *reinterpret_cast<float2 *>(row + (2 * n + wn) * 8) =
                    make_float2(acc[i][n][2 * u], acc[i][n][2 * u + 1]);
        }
    join_sums(a, order, t.count, q0, ranks, kPitch, base);
}

// A tile of up to 16 rows, rows q0 .. q0 + 31 of A, k0 <= k < k1, an eighth for each warp.
template <bool kBf16>
__device__ void shrink_low(const LoraArgs &a, const uint16_t *order, const Tile &t, int q0, int k0,
                           int k1, uint8_t *smem) {
    constexpr int NT = kLowRanks / 8, kPitch = kLowRanks + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int Q = a.parts * a.R, rank = rank_of(a, t.adapter);
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
    const int per = (max(k1 - k0, 0) + 8 * kWarps - 1) / (8 * kWarps) * 8;
    const int end = min(k1, k0 + (warp + 1) * per);
#pragma unroll 3
    for (int k = k0 + warp * per; k < end; k += 32) {
        const int kk = k + c * 8;
        const bool in = kk < end;
        const uint4 xv0 = in ? *reinterpret_cast<const uint4 *>(x0 + kk) : zero,
                    xv1 = in ? *reinterpret_cast<const uint4 *>(x1 + kk) : zero;
        uint4 wv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            wv[n] = in && w[n] ? *reinterpret_cast<const uint4 *>(w[n] + kk) : zero;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma<kBf16>(acc[n], xv0.x, xv1.x, xv0.y, xv1.y, wv[n].x, wv[n].y);
            mma<kBf16>(acc[n], xv0.z, xv1.z, xv0.w, xv1.w, wv[n].z, wv[n].w);
        }
    }
    // the warps' sums, in order, then the CTAs'
    float *sum = reinterpret_cast<float *>(smem), *red = sum + kLow * kPitch;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            red[(warp * kLow + g + (i >> 1) * 8) * kPitch + n * 8 + c * 2 + (i & 1)] = acc[n][i];
    __syncthreads();
    for (int i = tid; i < kLow * kLowRanks; i += kThreads) {
        const int r = i / kLowRanks, q = i % kLowRanks;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[(u * kLow + r) * kPitch + q];
        sum[r * kPitch + q] = v;
    }
    join_sums(a, order, t.count, q0, min(kLowRanks, Q - q0), kPitch, smem_of(smem));
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(LoraArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocalPlan own;
    wait_for_last();
    launch_next();
    const Plan p = make_plan(a, own, smem);
    const int Q = a.parts * a.R;
    const int tq = (Q + kTallRanks - 1) / kTallRanks, lq = (Q + kLowRanks - 1) / kLowRanks;
    const int tall = p.n.tall * tq, units = tall + p.n.low * lq;
    const int slice = (a.K + kCluster * 8 - 1) / (kCluster * 8) * 8;
    const int k0 = (int)cluster_rank() * slice, k1 = min(a.K, k0 + slice);
    for (int u = blockIdx.x / kCluster; u < units; u += gridDim.x / kCluster) {
        const bool is_tall = u < tall;
        const int v = is_tall ? u : u - tall, per = is_tall ? tq : lq;
        const Tile t = p.tiles[(is_tall ? 0 : p.n.tall) + v / per];
        const uint16_t *order = p.order + t.first;
        if (is_tall)
            shrink_tall<kBf16>(a, order, t, v % per * kTallRanks, k0, k1, smem);
        else
            shrink_low<kBf16>(a, order, t, v % per * kLowRanks, k0, k1, smem);
    }
}

// ---------------------------------------------------------------------------
// expand.  RK: 16s of rank that the kernel holds.
// ---------------------------------------------------------------------------
// bytes of a row of B in shared memory: an odd number of 32 bytes, so that rows next to each
// other lie in other banks
constexpr int row_pitch(int RK) { return (RK | 1) * 32; }
constexpr int tall_stages(int RK) { return RK == 1 ? 5 : RK == 2 ? 4 : RK == 4 ? 3 : 2; }
constexpr int low_stages(int RK) { return 8 / RK; }
constexpr int tall_stage(int RK) { return kTall * kTallCols * 2 + kTallCols * row_pitch(RK); }
constexpr int low_stage(int RK) { return kLowCols * row_pitch(RK); }
constexpr int max_of(int a, int b) { return a > b ? a : b; }
constexpr int expand_smem(int RK) {
    return max_of(max_of(tall_stages(RK) * tall_stage(RK), kWarps * low_stages(RK) * low_stage(RK)),
                  (int)sizeof(RowSort));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
    return (uint32_t)float_to_half_bits(lo, bf16) | (uint32_t)float_to_half_bits(hi, bf16) << 16;
}

// where column j of 32 lies among the rows of four 8-column MMA tiles so that a lane's
// results are 8 neighbours: MMA tile (j >> 1) & 3, its column (j >> 3) * 2 + (j & 1)
__device__ __forceinline__ int interleaved(int j) {
    return (j >> 1 & 3) * 8 + (j >> 3) * 2 + (j & 1);
}

// Two rows of 16 (g, g + 8) as a lane holds them: t in two halves, where their y lies, and
// the factor of their products.
template <bool kBf16, int RK>
struct Rows {
    uint32_t hi[RK][4], lo[RK][4];
    float factor[2];

    // m: the rows, or -1
    __device__ __forceinline__ void load(const LoraArgs &a, const int (&m)[2], int part, int rank,
                                         float scale) {
        const int c = threadIdx.x & 3, Q = a.parts * a.R;
        float4 v[2][RK];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float *row = sums_of(a) + (size_t)max(m[u], 0) * Q + part * a.R + c * 4;
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                const int left = m[u] < 0 ? 0 : rank - (k * 16 + c * 4);
                v[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (left > 0) v[u][k] = __ldcg(reinterpret_cast<const float4 *>(row + k * 16));
                if (left < 4) v[u][k].w = 0.f;
                if (left < 3) v[u][k].z = 0.f;
                if (left < 2) v[u][k].y = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float most = 0.f;  // (a NaN does not count)
#pragma unroll
            for (int k = 0; k < RK; ++k)
                most = fmaxf(fmaxf(most, fmaxf(fabsf(v[u][k].x), fabsf(v[u][k].y))),
                             fmaxf(fabsf(v[u][k].z), fabsf(v[u][k].w)));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // a row of zeros, or with an Inf, stays as it is
            const int top = __float_as_uint(most) >> 23;
            const int e = top >= 255 || top == 0 ? 127 : min(max(top, 2), 252);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
            factor[u] = __uint_as_float((uint32_t)e << 23) * scale;
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                const float w[4] = {v[u][k].x * down, v[u][k].y * down, v[u][k].z * down,
                                    v[u][k].w * down};
                float h[4], l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = half_bits_to_float(float_to_half_bits(w[i], kBf16), kBf16);
                    l[i] = isfinite(h[i]) ? w[i] - h[i] : 0.f;
                }
                hi[k][u] = pack16(h[0], h[1], kBf16), hi[k][2 + u] = pack16(h[2], h[3], kBf16);
                lo[k][u] = pack16(l[0], l[1], kBf16), lo[k][2 + u] = pack16(l[2], l[3], kBf16);
            }
        }
    }

    // 32 columns whose rows of B (interleaved) start at b: v[u] are 8 neighbours of row u
    __device__ __forceinline__ void product(float (&v)[2][8], uint32_t b, int ksteps) const {
        const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        float acc[4][4] = {};
        b += g * row_pitch(RK) + c * 8;
#pragma unroll
        for (int k = 0; k < RK; ++k) {
            if (k >= ksteps) break;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint2 w = lds64(b + n * 8 * row_pitch(RK) + k * 32);
                mma<kBf16>(acc[n], hi[k][0], hi[k][1], hi[k][2], hi[k][3], w.x, w.y);
                mma<kBf16>(acc[n], lo[k][0], lo[k][1], lo[k][2], lo[k][3], w.x, w.y);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) v[u][2 * n + i] = acc[n][2 * u + i] * factor[u];
    }
};

// 8 columns of a row, of which n exist
template <bool kVec>
__device__ __forceinline__ uint4 load_cells(const uint16_t *p, int n) {
    if constexpr (kVec) return n > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool kVec>
__device__ __forceinline__ void store_cells(uint16_t *p, int n, uint4 v) {
    if constexpr (kVec) {
        if (n > 0) *reinterpret_cast<uint4 *>(p) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
}
template <bool kBf16>
__device__ __forceinline__ uint4 add_cells(uint4 r, const float (&v)[8]) {
    uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack16(half_bits_to_float((uint16_t)w[i], kBf16) + v[2 * i],
                      half_bits_to_float((uint16_t)(w[i] >> 16), kBf16) + v[2 * i + 1], kBf16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows without an adapter: columns n0 <= n < n1 of the residual, or zeros.
template <bool kVec>
__device__ void copy_rows(const LoraArgs &a, const uint16_t *order, const Tile &t, int n0, int n1) {
    if (a.residual == a.y) return;
    const int cells = (n1 - n0 + 7) / 8;
    for (int i = threadIdx.x; i < t.count * cells; i += kThreads) {
        const int r = i / cells, n = n0 + i % cells * 8;
        const size_t at = (size_t)order[r] * a.N + n;
        store_cells<kVec>(a.y + at, n1 - n,
                          a.residual ? load_cells<kVec>(a.residual + at, n1 - n)
                                     : make_uint4(0, 0, 0, 0));
    }
}

// A tall tile, columns n0 <= n < n1 of a part: every warp 16 rows.  A stage is 64 columns of
// B and (kVec) of the tile's residual.
template <bool kBf16, int RK, bool kVec>
__device__ void expand_tall(const LoraArgs &a, const uint16_t *order, const Tile &t, int part,
                            int n0, int n1, uint8_t *smem) {
    constexpr int kStages = tall_stages(RK), kBytes = tall_stage(RK), kRes = kTall * kTallCols * 2;
    constexpr int kPieces = 2 * RK;  // of 16 bytes in a row of B
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int rank = rank_of(a, t.adapter), ksteps = (rank + 15) / 16;
    const uint32_t base = smem_of(smem);
    const bool staged = kVec && a.residual;
    // this thread's 16 bytes of four rows of the residual, per stage
    const int col = tid & 7, r0 = tid >> 3;
    const uint16_t *rp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        rp[i] = staged && r < t.count ? a.residual + (size_t)order[r] * a.N + col * 8 : nullptr;
    }
    const uint16_t *b = a.b + (size_t)t.adapter * a.N * a.R;
    auto issue = [&](int n, int stage) {
        const uint32_t st = base + stage * kBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i, in = n + col * 8 < n1 ? 16 : 0;
            if (rp[i])
                copy16(st + (r << 7) + ((col ^ ((r & 1) << 2)) << 4), in ? rp[i] + n : a.residual,
                       in);
        }
#pragma unroll
        for (int i = 0; i < (kTallCols * kPieces + kThreads - 1) / kThreads; ++i) {
            const int q = tid + i * kThreads, j = q / kPieces, r = q % kPieces * 8;
            if (j >= kTallCols) break;
            const int in = n + j < n1 ? max(0, min(2 * (rank - r), 16)) : 0;
            copy16(st + kRes + ((j & ~31) + interleaved(j & 31)) * row_pitch(RK) + r * 2,
                   in ? b + (size_t)(n + j) * a.R + r : a.b, in);
        }
    };
    int next = n0;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s, next += kTallCols) {
        if (next < n1) issue(next, s);
        commit_copies();
    }
    const int r[2] = {warp * 16 + g, warp * 16 + g + 8};
    const int m[2] = {r[0] < t.count ? order[r[0]] : -1, r[1] < t.count ? order[r[1]] : -1};
    const size_t at[2] = {(size_t)max(m[0], 0) * a.N, (size_t)max(m[1], 0) * a.N};
    const float scale = a.scales[t.adapter];
    Rows<kBf16, RK> rows;
    wait_for_last();  // t
    rows.load(a, m, part, rank, scale);
    int stage = 0, free = kStages - 1;
    for (int n = n0; n < n1; n += kTallCols, next += kTallCols) {
        wait_copies<kStages - 2>();
        __syncthreads();  // this stage is there, the one before is free
        if (next < n1) issue(next, free);
        commit_copies();
        const uint32_t st = base + stage * kBytes;
#pragma unroll
        for (int s = 0; s < kTallCols / 32; ++s) {
            float v[2][8];
            rows.product(v, st + kRes + s * 32 * row_pitch(RK), ksteps);
            const int cc = n + s * 32 + c * 8;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int cells = m[u] >= 0 ? n1 - cc : 0;
                uint4 res = make_uint4(0, 0, 0, 0);
                if (staged)
                    res = lds128(st + (r[u] << 7) + (((s * 4 + c) ^ ((r[u] & 1) << 2)) << 4));
                else if (a.residual)
                    res = load_cells<kVec>(a.residual + at[u] + cc, cells);
                store_cells<kVec>(a.y + at[u] + cc, cells, add_cells<kBf16>(res, v[u]));
            }
        }
        free = stage;
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    wait_copies<0>();
    __syncthreads();  // what comes next fills the same memory
}

// A low tile, columns n0 <= n < n1 of a part: every warp 32 of them in turn, with a ring of
// its own for B.
template <bool kBf16, int RK, bool kVec>
__device__ void expand_low(const LoraArgs &a, const uint16_t *order, const Tile &t, int part,
                           int n0, int n1, uint8_t *smem) {
    constexpr int kStages = low_stages(RK), kBytes = low_stage(RK), kPieces = 2 * RK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int rank = rank_of(a, t.adapter), ksteps = (rank + 15) / 16;
    const uint32_t base = smem_of(smem) + warp * kStages * kBytes;
    const uint16_t *b = a.b + (size_t)t.adapter * a.N * a.R;
    auto issue = [&](int n, int stage) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int q = lane + i * 32, j = q / kPieces, r = q % kPieces * 8;
            const int in = n + j < n1 ? max(0, min(2 * (rank - r), 16)) : 0;
            copy16(base + stage * kBytes + interleaved(j) * row_pitch(RK) + r * 2,
                   in ? b + (size_t)(n + j) * a.R + r : a.b, in);
        }
    };
    constexpr int kStride = kWarps * kLowCols;
    int n = n0 + warp * kLowCols, next = n;
#pragma unroll
    for (int s = 0; s < kStages; ++s, next += kStride) {
        if (next < n1) issue(next, s);
        commit_copies();
    }
    const int m[2] = {g < t.count ? order[g] : -1, g + 8 < t.count ? order[g + 8] : -1};
    const size_t at[2] = {(size_t)max(m[0], 0) * a.N + c * 8, (size_t)max(m[1], 0) * a.N + c * 8};
    uint4 res[2];
    auto fetch = [&](int n) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            res[u] = a.residual && n < n1 && m[u] >= 0
                         ? load_cells<kVec>(a.residual + at[u] + n, n1 - n - c * 8)
                         : make_uint4(0, 0, 0, 0);
    };
    fetch(n);
    const float scale = a.scales[t.adapter];
    Rows<kBf16, RK> rows;
    wait_for_last();  // t
    rows.load(a, m, part, rank, scale);
    for (int stage = 0; n < n1; n += kStride, next += kStride) {
        wait_copies<kStages - 1>();
        __syncwarp();
        float v[2][8];
        rows.product(v, base + stage * kBytes, ksteps);
        uint4 out[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) out[u] = add_cells<kBf16>(res[u], v[u]);
        __syncwarp();  // all lanes have read the stage
        if (next < n1) issue(next, stage);
        commit_copies();
        stage = stage == kStages - 1 ? 0 : stage + 1;
        fetch(n + kStride);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            store_cells<kVec>(a.y + at[u] + n, m[u] >= 0 ? n1 - n - c * 8 : 0, out[u]);
    }
    wait_copies<0>();
    __syncthreads();  // what comes next fills the same memory
}

// The steps from, .. , to - 1 of (tile, part, step of `cols` columns), in runs of one tile and part
template <typename Run>
__device__ __forceinline__ void walk(const LoraArgs &a, int cols, long long from, long long to,
                                     Run run) {
    int per = 0;
    for (int i = 0; i < a.parts; ++i) per += (a.part[i] + cols - 1) / cols;
    while (from < to) {
        const int tile = (int)(from / per);
        int s = (int)(from - (long long)tile * per), part = 0, first = 0, steps;
        for (;; ++part) {
            steps = (a.part[part] + cols - 1) / cols;
            if (s < steps) break;
            s -= steps;
            first += a.part[part];
        }
        const int n = (int)min((long long)(steps - s), to - from);
        run(tile, part, first + s * cols, min(first + (s + n) * cols, first + a.part[part]));
        from += n;
    }
}

template <bool kBf16, int RK, bool kVec>
__global__ void __launch_bounds__(kThreads, RK == 8 ? 1 : 2) expand_kernel(LoraArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocalPlan own;
    launch_next();
    // shrink has let this kernel start after all that came before shrink had ended: the plan,
    // B and the residual may be read before shrink's own results
    const Plan p = make_plan(a, own, smem);
    int tall_steps = 0, low_steps = 0;
    for (int i = 0; i < a.parts; ++i) {
        tall_steps += (a.part[i] + kTallCols - 1) / kTallCols;
        low_steps += (a.part[i] + kLowCols - 1) / kLowCols;
    }
    const auto share = [&](long long steps, int i) { return steps * i / (int)gridDim.x; };
    const long long tall = (long long)(p.n.tall + p.n.none) * tall_steps,
                    low = (long long)p.n.low * low_steps;
    walk(a, kTallCols, share(tall, blockIdx.x), share(tall, blockIdx.x + 1),
         [&](int tile, int part, int n0, int n1) {
             const Tile t = p.tiles[tile < p.n.tall ? tile : tile + p.n.low];
             if (t.adapter == a.L)
                 copy_rows<kVec>(a, p.order + t.first, t, n0, n1);
             else
                 expand_tall<kBf16, RK, kVec>(a, p.order + t.first, t, part, n0, n1, smem);
         });
    walk(a, kLowCols, share(low, blockIdx.x), share(low, blockIdx.x + 1),
         [&](int tile, int part, int n0, int n1) {
             const Tile t = p.tiles[p.n.tall + tile];
             expand_low<kBf16, RK, kVec>(a, p.order + t.first, t, part, n0, n1, smem);
         });
    wait_for_last();  // (for those without a step: what follows this kernel waits for it alone)
}

template <bool kBf16, int RK, bool kVec>
cudaError_t launch_expand(const LoraArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    return launch_chained(expand_kernel<kBf16, RK, kVec>, dim3((RK == 8 ? 1 : 2) * dev.sm_count),
                          kThreads, expand_smem(RK), 1, stream, a);
}
template <bool kBf16, bool kVec>
cudaError_t launch_expand_rank(const LoraArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    if (a.R <= 16) return launch_expand<kBf16, 1, kVec>(a, dev, stream);
    if (a.R <= 32) return launch_expand<kBf16, 2, kVec>(a, dev, stream);
    if (a.R <= 64) return launch_expand<kBf16, 4, kVec>(a, dev, stream);
    return launch_expand<kBf16, 8, kVec>(a, dev, stream);
}

template <bool kBf16>
cudaError_t launch_type(const LoraArgs &a, bool vec, const DeviceInfo &dev, cudaStream_t stream) {
    if (a.M > kMaxRows) {
        const cudaError_t e = launch_chained(plan_kernel, dim3(1), kPlanThreads, 0, 1, stream, a);
        if (e != cudaSuccess) return e;
    }
    // as many clusters as there can be units, or as run at once
    const long long units = (long long)lora_max_tiles(a.M, a.L) *
                            ((a.parts * a.R + kLowRanks - 1) / kLowRanks);
    const int most = 2 * dev.sm_count / kCluster;
    const int clusters = units < most ? (int)units : most;
    const cudaError_t e = launch_chained(shrink_kernel<kBf16>, dim3(clusters * kCluster), kThreads,
                                         kShrinkSmem, kCluster, stream, a);
    if (e != cudaSuccess) return e;
    return vec ? launch_expand_rank<kBf16, true>(a, dev, stream)
               : launch_expand_rank<kBf16, false>(a, dev, stream);
}

template <bool kBf16, int RK>
cudaError_t init_expand() {
    const void *kernels[] = {(const void *)expand_kernel<kBf16, RK, true>,
                             (const void *)expand_kernel<kBf16, RK, false>};
    for (const void *k : kernels) {
        cudaError_t e =
            cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, expand_smem(RK));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool kBf16>
cudaError_t init_type() {
    cudaError_t e = cudaFuncSetAttribute((const void *)shrink_kernel<kBf16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kShrinkSmem);
    if (e == cudaSuccess) e = init_expand<kBf16, 1>();
    if (e == cudaSuccess) e = init_expand<kBf16, 2>();
    if (e == cudaSuccess) e = init_expand<kBf16, 4>();
    if (e == cudaSuccess) e = init_expand<kBf16, 8>();
    return e;
}

}  // namespace

cudaError_t launch_lora(const LoraArgs &a, bool bf16, const DeviceInfo &dev, cudaStream_t stream) {
    // 16-byte accesses of y and the residual
    bool vec = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.residual & 15) == 0;
    for (int i = 0; i < a.parts; ++i) vec = vec && a.part[i] % 8 == 0;
    return bf16 ? launch_type<true>(a, vec, dev, stream) : launch_type<false>(a, vec, dev, stream);
}

cudaError_t lora_init() {
    const cudaError_t e = init_type<true>();
    return e == cudaSuccess ? init_type<false>() : e;
}

}  // namespace w4a16
