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
// low tile if they are at most 16; in calls of up to 128 rows, decode steps mostly, in low
// tiles whatever their number.  All tiles of an adapter are of one kind, and a row's sums do
// not depend on its place in a tile, so the order within an adapter changes no result.  Up to
// 1024 rows each CTA groups for itself in shared memory; more are grouped by a kernel of one
// CTA before (plan_kernel).
//   * shrink: t, a cluster of 8 CTAs per tile and block of A's rows, each with an eighth of
//     K, whose sums meet through distributed shared memory (a tall tile's x is 1.3 MB at
//     K 5120, and there are few tiles: without the split most SMs would idle).  A tall tile
//     and 128 rows of A go through shared memory; a low one and 32 rows of A come straight
//     from memory, since each of their weights is used once.
//   * expand: y.  All steps (128 columns of a tall tile, 32 of a low one for each warp) are
//     one sequence of which every CTA takes an equal run; B and the residual come through
//     rings of asynchronous copies.  In calls of few rows its CTAs start wherever shrink leaves
//     an SM room (two of shrink's CTAs take all its registers), so that their grouping and
//     first copies are done when shrink ends.
// Tall tiles run on tcgen05 (M = 128 rows of the tile), low ones on the warp MMA with the rows
// as its M = 16, straight from what the asynchronous copies bring.
//
// What bounds it (one GB300, calls in a row in a graph).  Few rows: the chain of two kernels
// and their dependent loads, 7.1 us for one row, rank 16, beside qkv (0.8 MB), of which the
// grouping is 1, the loads of A 1.5, the sums' meeting 1.5, t and the outputs 1.5; 64 rows of
// 32 adapters beside gate+up 21.7 us, of which the adapters' 46 MB are 7 to 8.  Many rows:
// the bytes of y, 150 us for 4096 rows, rank 64, beside gate+up (643 MB, 4.3 TB/s): the
// grouping, shrink 20, then expand 122, where copies alone would take about 105 and products and
// outputs alone about 90, which one CTA per SM, in step at a barrier per 128 columns, overlaps
// in part.  With the tall tiles on the warp MMA the same call took 189 to 221 us.  Columns that
// are not multiples of 8 (or addresses of 2 bytes) are read and written 2 bytes a lane, the
// residual with nothing ahead: the same call with 17405 + 17403 columns takes 602 us.
//
// t is fp32; as expand's operand it is split into two values of the 16-bit type, of a row first
// scaled by a power of two: the value cut to the type and the rest rounded.  16 bits (bf16) or
// 22 (fp16) of it enter the product, at twice the MMAs, which are not the bound.  Both halves
// have t's sign and neither is zero unless t is, so that an infinite weight times them is what
// it is times t (a rest of zero, or of the other sign, would make it NaN).
//
// Every wait for a product is bounded; one that expires sets a status bit, and the kernel
// goes on to its end without further products or waits, but for one at the end, bounded too,
// for those in flight, before the tensor memory is freed.
#include "w4a16_routed.cuh"
#include "w4a16_tcgen05.cuh"

namespace w4a16 {
namespace {

using namespace routed;

constexpr int kTall = 128;   // rows of a tall tile
constexpr int kLow = 16;     // and of a low one, at most
constexpr int kFewRows = 128;    // calls of up to so many rows have low tiles only
constexpr int kLocalRows = kLoraLocalRows;  // and up to so many every CTA groups for itself
constexpr int kPlanThreads = 1024;
constexpr int kShrinkThreads = 256;
constexpr int kCluster = 8;      // CTAs that share a shrink unit's K
constexpr int kTallRanks = 128;  // rows of A of a shrink unit of a tall tile
constexpr int kLowRanks = 32;    // and of a low one
constexpr int kShrinkStage = (kTall + kTallRanks) * 128;  // bytes: 64 k of x and A
// Its kernel's kind: calls of few rows, with low tiles only, in small shared memory; calls
// whose tall units are no more than the clusters of one CTA per SM that run at once, with six
// stages each (1000 rows beside o: 29.5 us for 31.3 with three); others, two CTAs per SM
// (4096 rows beside gate+up: 152 us for 160 with the one of six stages)
enum Kind { kFew, kDeep, kMany };
constexpr int shrink_stages(Kind kind) { return kind == kDeep ? 6 : 3; }
constexpr int kMaxShrinkStages = 6;
constexpr int kTallCols = 128;  // columns of a step of expand, tall tiles
constexpr int kLowCols = 32;    // low ones
constexpr int kLowPitch = kLowRanks + 8;  // of a low unit's sums in shared memory
constexpr int max_of(int a, int b) { return a > b ? a : b; }
constexpr int kShrinkTmem = 128, kExpandTmem = 256;  // columns: a tile's sums; two steps'
constexpr int kExpandBars = 2;
constexpr int kErrProducts = 1 << 21;  // device status bit: a wait for products expired

struct Tile {
    uint16_t adapter, first, count, pad;
};
struct Counts {
    int tall, low;      // tiles
    int rows, none;     // with an adapter, and without (those come last)
};
// a CTA's own, of up to kRows rows; tall tiles from the front, low ones from the back, as
// adapter << 17 | first << 7 | count - 1
template <int kRows>
struct LocalPlan {
    static constexpr int kTiles = kRows + kRows / kLow;
    Counts n;
    uint32_t tiles[kTiles];
    uint16_t order[kRows];
};
struct Plan {
    Counts n;
    const Tile *shared;      // tall tiles, then low ones; null: the CTA's own
    const uint32_t *own;
    int own_tiles;
    const uint16_t *order;   // the rows by adapter

    static __device__ __forceinline__ Tile unpack(uint32_t t) {
        return {(uint16_t)(t >> 17), (uint16_t)(t >> 7 & 1023), (uint16_t)((t & 127) + 1), 0};
    }
    __device__ __forceinline__ Tile tall(int i) const { return shared ? shared[i] : unpack(own[i]); }
    __device__ __forceinline__ Tile low(int i) const {
        return shared ? shared[n.tall + i] : unpack(own[own_tiles - 1 - i]);
    }
};
static_assert(sizeof(Counts) == 16 && sizeof(Tile) == 8, "as lora_plan_bytes counts them");
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
// the tiles of an adapter with n rows: tall ones, low ones
__device__ __forceinline__ int tall_tiles(int n, bool few) {
    return !few && n > kLow ? (n + kTall - 1) / kTall : 0;
}
__device__ __forceinline__ int low_tiles(int n, bool few) {
    return few || n <= kLow ? (n + kLow - 1) / kLow : 0;
}
__device__ Counts *shared_counts(const LoraArgs &a) { return static_cast<Counts *>(a.scratch); }
__device__ __forceinline__ float *sums_of(const LoraArgs &a) {
    return reinterpret_cast<float *>(static_cast<char *>(a.scratch) + lora_plan_bytes(a.M, a.L));
}
__device__ __forceinline__ Plan shared_plan(const LoraArgs &a) {
    Plan p{};
    p.shared = reinterpret_cast<const Tile *>(shared_counts(a) + 1);
    p.order = reinterpret_cast<const uint16_t *>(p.shared + lora_max_tiles(a.M, a.L));
    return p;
}

// The plan of the call; `space` is free again afterwards.  kRows: of calls that the CTA
// groups for itself.
template <int kCta, int kRows>
__device__ Plan make_plan(const LoraArgs &a, LocalPlan<kRows> &own, void *space) {
    constexpr bool few = kRows == kFewRows;
    Plan p = shared_plan(a);
    if (a.M > kRows) {
        p.n = *shared_counts(a);
        return p;
    }
    // a pack: rows, tall tiles << 11, low tiles << 21; bin L (no adapter), the last, has none
    group_rows<kCta>(
        *static_cast<RowSort<kRows> *>(space), own.order, a.M, a.L + 1,
        [&](int m) { return bin_of(a, m); },
        [&](int l, int n) {
            return l == a.L ? 0u
                            : (unsigned)n | (unsigned)tall_tiles(n, few) << 11 |
                                  (unsigned)low_tiles(n, few) << 21;
        },
        [&](int l, int n, unsigned at) {
            if (l == a.L) return;
            const bool tall = tall_tiles(n, few) > 0;
            const int height = tall ? kTall : kLow;
            int i = tall ? (int)(at >> 11 & 1023)
                         : LocalPlan<kRows>::kTiles - 1 - (int)(at >> 21);
            for (int r = 0; r < n; r += height, i += tall ? 1 : -1)
                own.tiles[i] = (uint32_t)l << 17 | ((at & 2047) + r) << 7 |
                               (min(height, n - r) - 1);
        },
        [&](unsigned total) {
            const int rows = total & 2047;
            own.n = {(int)(total >> 11 & 1023), (int)(total >> 21), rows, a.M - rows};
        });
    p.n = own.n;
    p.shared = nullptr;
    p.own = own.tiles;
    p.own_tiles = LocalPlan<kRows>::kTiles;
    p.order = own.order;
    return p;
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    return reinterpret_cast<uint8_t *>(((uintptr_t)p + 1023) & ~(uintptr_t)1023);
}

// ---------------------------------------------------------------------------
// products of tall tiles: tensor memory, the barriers that tell of their ends
// ---------------------------------------------------------------------------
struct ProductSpace {
    uint64_t done[kMaxShrinkStages];
    uint32_t tmem;
    int abort;
};
struct Products {
    ProductSpace *sp;
    int *status;
    uint32_t tmem;
    unsigned count;   // committed so far, by barrier in turn
    unsigned issued;  // warp 0, which issues them: the same, but for those left out
    bool ok;          // none of this warp's waits has given up; warp 0 issues none after one

    // all threads, before the next kernel may start: its CTAs take tensor memory too
    template <int kCols>
    __device__ __forceinline__ void begin(ProductSpace *space, int *status_word) {
        sp = space, status = status_word, count = issued = 0, ok = true;
        if (threadIdx.x == 0) {
            for (int i = 0; i < kMaxShrinkStages; ++i) dev::mbar_init(smem_of(&sp->done[i]), 1);
            dev::mbar_init_fence();
            sp->abort = 0;
        }
        __syncwarp();
        if (threadIdx.x < 32) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_of(&sp->tmem)),
                         "r"(kCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        dev::tc_fence_before();
        __syncthreads();
        dev::tc_fence_after();
        tmem = sp->tmem;
    }
    // kBars: as wait's
    template <int kCols, int kBars>
    __device__ __forceinline__ void end() {
        dev::tc_fence_before();
        __syncthreads();
        if (threadIdx.x < 32) {
            if (!ok)
                for (unsigned n = issued > kBars ? issued - kBars : 0; n < issued; ++n) {
                    dev::mbar_wait_drain(bar(n, kBars), n / kBars & 1);
                    __syncwarp();
                }
            dev::tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(kCols)
                         : "memory");
        }
    }
    // the barrier of products n, of `bars` in turn
    __device__ __forceinline__ uint32_t bar(unsigned n, int bars) const {
        return smem_of(&sp->done[n % bars]);
    }
    // products n (counted from 0) and all before are done; whole warps wait, and go on together
    __device__ __forceinline__ void wait(unsigned n, int bars) {
        volatile int *abort = &sp->abort;
        if (!dev::mbar_wait_all(bar(n, bars), n / bars & 1, abort)) {
            ok = false;
            if (!*abort) {
                *abort = 1;
                atomicOr(status, kErrProducts);
            }
        }
        __syncwarp();
    }
};
// D[tensor memory] (+)= A B^T over 16 k, both 128-byte swizzled in shared memory.  Issued by
// the elected lane of a warp whose control flow and operands are uniform: by one thread of a
// diverged warp each took about 220 cycles.
__device__ __forceinline__ void product16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// M = 128, N = n (a multiple of 16), fp32 sums
template <bool kBf16>
__device__ __forceinline__ uint32_t product_desc(int n) {
    return (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTall >> 4) << 24);
}
// where 16-byte piece c of a 128-byte row r lies in the swizzled layout
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)(r << 7) + (uint32_t)((c ^ (r & 7)) << 4);
}

// The plan to where the expanding kernel reads it.
__device__ void share_plan(const LoraArgs &a, const Plan &p) {
    const Plan to = shared_plan(a);
    Tile *tiles = const_cast<Tile *>(to.shared);
    uint16_t *order = const_cast<uint16_t *>(to.order);
    for (int i = threadIdx.x; i < p.n.tall + p.n.low; i += kShrinkThreads)
        tiles[i] = i < p.n.tall ? p.tall(i) : p.low(i - p.n.tall);
    for (int i = threadIdx.x; i < a.M; i += kShrinkThreads) order[i] = p.order[i];
    if (threadIdx.x == 0) *shared_counts(a) = p.n;
}

// ---------------------------------------------------------------------------
// plan: one CTA, more than kLocalRows rows.  Bin l < L: the rows of adapter l; bin L: those
// without one.  The order within a bin is that of an atomic counter.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(LoraArgs a) {
    __shared__ int count[kMaxAdapters + 1], sums[3][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_last();
    launch_next();
    const Plan plan = shared_plan(a);
    Tile *tiles = const_cast<Tile *>(plan.shared);
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
    int v[3] = {n, tall_tiles(n, false), low_tiles(n, false)};
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
    const int first = v[0] - own[0];
    if (tid == 0) {
        *shared_counts(a) = {all[1], all[2], all[0], a.M - all[0]};
        count[a.L] = all[0];
    }
    for (int i = 0; i < own[1]; ++i)
        tiles[v[1] - own[1] + i] = {(uint16_t)tid, (uint16_t)(first + i * kTall),
                                    (uint16_t)min(kTall, n - i * kTall), 0};
    if (own[2]) tiles[all[1] + v[2] - 1] = {(uint16_t)tid, (uint16_t)first, (uint16_t)n, 0};
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
    __syncwarp();
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
    for (int i = threadIdx.x; i < n; i += kShrinkThreads) {
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

// A tile of up to 128 rows, rows q0 .. q0 + 127 of A, k0 <= k < k1: the products of a stage
// of 64 k are issued once it is there, and its slot is filled again once they are done.
template <bool kBf16, int kShrinkStages>
__device__ void shrink_tall(const LoraArgs &a, const uint16_t *order, const Tile &t, int q0, int k0,
                            int k1, uint8_t *smem, Products &pr) {
    constexpr int kPitch = kTallRanks + 4;
    static_assert(kTall * kPitch * 4 <= kShrinkStages * kShrinkStage, "the sums fit the stages");
    const int tid = threadIdx.x, lane = tid & 31, warp = (int)dev::uniform(tid >> 5);
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
        const uint32_t st = base + (pr.count + s) % kShrinkStages * kShrinkStage;
        const int k = k0 + s * 64 + col * 8, in = k < k1 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 32 * i;
            const uint32_t at = swizzled(r, col);
            if (xp[i]) copy16(st + at, in ? xp[i] + k : a.x, in);
            if (r < ranks)
                copy16(st + kTall * 128 + at, ap[i] && in ? ap[i] + k : a.a, ap[i] ? in : 0);
        }
    };
    const int steps = k1 > k0 ? (k1 - k0 + 63) / 64 : 0;
    const uint32_t idesc = dev::uniform(product_desc<kBf16>((ranks + 15) / 16 * 16)),
                   tmem = dev::uniform(pr.tmem);
#pragma unroll
    for (int s = 0; s < kShrinkStages - 1; ++s) {
        if (s < steps) issue(s);
        commit_copies();
    }
    for (int s = 0; s < steps; ++s) {
        wait_copies<kShrinkStages - 2>();
        dev::fence_async_shared();
        __syncthreads();
        if (warp == 0 && pr.ok) {
            dev::tc_fence_after();
            const uint32_t st =
                dev::uniform(base + (pr.count + s) % kShrinkStages * kShrinkStage);
            const uint64_t x = dev::smem_desc_sw128(st), w = dev::smem_desc_sw128(st + kTall * 128);
            const uint32_t bar = dev::uniform(pr.bar(pr.count + s, kShrinkStages));
            if (dev::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    product16(tmem, x + 2 * k, w + 2 * k, idesc, s + k > 0);
                dev::mma_commit(bar);
            }
            __syncwarp();
            pr.issued = pr.count + s + 1;
        }
        if (s + kShrinkStages - 1 < steps) {
            if (s > 0) pr.wait(pr.count + s - 1, kShrinkStages);
            issue(s + kShrinkStages - 1);
        }
        commit_copies();
    }
    if (steps > 0) pr.wait(pr.count + steps - 1, kShrinkStages);
    pr.count += steps;
    dev::tc_fence_after();
    __syncthreads();  // the sums go where the stages were
    // a warp's 32 rows (its quarter of the tensor memory's lanes), half of A's rows
    const int r = (warp & 3) * 32 + lane, q = (warp >> 2) * 64;
    float *row = reinterpret_cast<float *>(smem) + r * kPitch + q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t v[32] = {};
        if (steps > 0) {
            dev::tmem_ld(pr.tmem + ((uint32_t)(warp & 3) << 21) + q + h * 32, v);
            dev::tmem_wait_ld(v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(row + h * 32 + i * 4) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    dev::tc_fence_before();
    join_sums(a, order, t.count, q0, ranks, kPitch, base);
}

// A tile of up to 16 rows, rows q0 .. q0 + 31 of A, k0 <= k < k1, an eighth for each warp.
template <bool kBf16>
__device__ void shrink_low(const LoraArgs &a, const uint16_t *order, const Tile &t, int q0, int k0,
                           int k1, uint8_t *smem) {
    constexpr int NT = kLowRanks / 8, kPitch = kLowPitch, kWarps = kShrinkThreads / 32;
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
    for (int i = tid; i < kLow * kLowRanks; i += kShrinkThreads) {
        const int r = i / kLowRanks, q = i % kLowRanks;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[(u * kLow + r) * kPitch + q];
        sum[r * kPitch + q] = v;
    }
    join_sums(a, order, t.count, q0, min(kLowRanks, Q - q0), kPitch, smem_of(smem));
}

constexpr int shrink_smem(Kind kind) {
    return kind == kFew ? max_of((kShrinkThreads / 32 + 1) * kLow * kLowPitch * 4,
                         (int)sizeof(RowSort<kFewRows>))
                : shrink_stages(kind) * kShrinkStage + 1024;  // (to align them)
}

template <bool kBf16, Kind kKind>
__global__ void __launch_bounds__(kShrinkThreads, kKind == kDeep ? 1 : 2) shrink_kernel(LoraArgs a) {
    constexpr bool few = kKind == kFew;
    constexpr int kRows = few ? kFewRows : kLocalRows;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = few ? smem_raw : align1024(smem_raw);
    __shared__ LocalPlan<kRows> own;
    __shared__ ProductSpace space;
    Products pr;
    // tensor memory is taken once the kernels before have ended: others of the library let this
    // one start before they have taken theirs, all 512 columns, and would wait for these
    // without end if their shared memory left room beside it
    wait_for_last();
    if constexpr (!few) pr.begin<kShrinkTmem>(&space, a.status);
    launch_next();
    const Plan p = make_plan<kShrinkThreads, kRows>(a, own, smem);
    if (!few && a.M <= kRows && blockIdx.x == 0) share_plan(a, p);
    const int Q = a.parts * a.R;
    const int tq = (Q + kTallRanks - 1) / kTallRanks, lq = (Q + kLowRanks - 1) / kLowRanks;
    const int tall = p.n.tall * tq, units = tall + p.n.low * lq;
    const int slice = (a.K + kCluster * 8 - 1) / (kCluster * 8) * 8;
    const int k0 = (int)cluster_rank() * slice, k1 = min(a.K, k0 + slice);
    for (int u = blockIdx.x / kCluster; u < units; u += gridDim.x / kCluster) {
        if (!few && u < tall) {
            const Tile t = p.tall(u / tq);
            if constexpr (!few)
                shrink_tall<kBf16, shrink_stages(kKind)>(a, p.order + t.first, t, u % tq * kTallRanks, k0, k1, smem, pr);
        } else {
            const int v = u - tall;
            const Tile t = p.low(v / lq);
            shrink_low<kBf16>(a, p.order + t.first, t, v % lq * kLowRanks, k0, k1, smem);
        }
    }
    if constexpr (!few) pr.end<kShrinkTmem, shrink_stages(kKind)>();
}

// ---------------------------------------------------------------------------
// expand.  RK: 16s of rank that the kernel holds.
// ---------------------------------------------------------------------------
// bytes of a row of B in shared memory (low tiles): an odd number of 32 bytes, so that rows
// next to each other lie in other banks
constexpr int row_pitch(int RK) { return (RK | 1) * 32; }
// Calls of few rows: two CTAs of 8 warps per SM, small enough to start beside one of shrink's
// while it runs (two take the SM's registers).  Others: one of 16 warps with all of the SM.
constexpr int expand_threads(bool few) { return few ? 256 : 512; }
constexpr int kResidualStage = kTall * kTallCols * 2;
constexpr int blocks64(int RK) { return RK > 4 ? 2 : 1; }  // of 64 of the rank
constexpr int b_stage(int RK) { return blocks64(RK) * kTallCols * 128; }
constexpr int t_half(int RK) { return blocks64(RK) * kTall * 128; }
constexpr int residual_stages(int RK) { return RK > 4 ? 2 : 4; }
constexpr int b_stages(int RK) { return RK > 4 ? 2 : 3; }
constexpr int low_residual = kLow * kLowCols * 2;
constexpr int low_stage(int RK) { return kLowCols * row_pitch(RK) + low_residual; }
constexpr int low_stages(int RK, bool few) {
    return few ? (RK == 1 ? 4 : RK == 2 ? 2 : 1) : (RK == 1 ? 6 : RK == 2 ? 3 : RK == 4 ? 2 : 1);
}
constexpr int expand_smem(int RK, bool few) {
    const int low = expand_threads(few) / 32 * low_stages(RK, few) * low_stage(RK);
    return few ? max_of(low, (int)sizeof(RowSort<kFewRows>))
               : 1024 + max_of(2 * t_half(RK) + residual_stages(RK) * kResidualStage +
                                   b_stages(RK) * b_stage(RK),
                               low);
}

// two values rounded to the 16-bit type (nearest even), or cut to it; and back
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t d;
    if constexpr (kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t cut16(float lo, float hi) {
    uint32_t d;
    if constexpr (kBf16) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
    if constexpr (kBf16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
// the power of two (its exponent field) that scales a row whose largest finite value is `most`
// below 8 (bf16) or 2^15 (fp16, whose smallest number is then 2^-38 of the largest)
template <bool kBf16>
__device__ __forceinline__ int row_exponent(float most) {
    return min(max((int)(__float_as_uint(most) >> 23) - (kBf16 ? 0 : 14), 2), 252);
}
__device__ __forceinline__ float scale_down(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }
__device__ __forceinline__ float scale_up(int e) { return __uint_as_float((uint32_t)e << 23); }
// the larger of a row's largest finite value so far and |v|
__device__ __forceinline__ float larger(float most, float v) {
    return isfinite(v) ? fmaxf(most, fabsf(v)) : most;
}
// the larger magnitude (NaN stays) with x's sign
__device__ __forceinline__ float at_least(float v, float least, float x) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(v)), "f"(least));
    return copysignf(d, x);
}
// x * down and y * down as the sum of two pairs of the 16-bit type, hi cut and lo rounded.
// Where one would be zero though the value is not, it is the least number of its sign: in the
// scaled row 2^-38 (fp16) or less of the largest.
template <bool kBf16>
__device__ __forceinline__ void split(float x, float y, float down, uint32_t &hi, uint32_t &lo) {
    constexpr float kLeast = kBf16 ? 0x1p-126f : 0x1p-24f;  // (bf16: the smallest normal one)
    const float lx = x != 0.f ? kLeast : 0.f, ly = y != 0.f ? kLeast : 0.f;
    const float u = at_least(x * down, lx, x), v = at_least(y * down, ly, y);
    hi = cut16<kBf16>(u, v);
    const float2 h = unpack16<kBf16>(hi);
    // (fmaxf takes the number: the rest of an Inf is the least one, that of a NaN does not matter)
    lo = pack16<kBf16>(copysignf(fmaxf(fabsf(u - h.x), lx), x),
                       copysignf(fmaxf(fabsf(v - h.y), ly), y));
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
            float most = 0.f;
#pragma unroll
            for (int k = 0; k < RK; ++k)
                most = larger(larger(larger(larger(most, v[u][k].x), v[u][k].y), v[u][k].z),
                              v[u][k].w);
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int e = row_exponent<kBf16>(most);
            const float down = scale_down(e);
            factor[u] = scale_up(e) * scale;
#pragma unroll
            for (int k = 0; k < RK; ++k) {
                split<kBf16>(v[u][k].x, v[u][k].y, down, hi[k][u], lo[k][u]);
                split<kBf16>(v[u][k].z, v[u][k].w, down, hi[k][2 + u], lo[k][2 + u]);
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
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<kBf16>(w[i]);
        w[i] = pack16<kBf16>(f.x + v[2 * i], f.y + v[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows without an adapter: all columns of the residual, or zeros, 1024 at a time for each warp
// of the grid in turn.
template <int kCta, bool kVec>
__device__ void copy_rows(const LoraArgs &a, const uint16_t *rows, int n) {
    if (a.residual == a.y) return;
    constexpr int kCols = 1024;
    const int lane = threadIdx.x & 31, pieces = (a.N + kCols - 1) / kCols;
    const long long all = (long long)n * pieces;
    for (long long i = (long long)blockIdx.x * (kCta / 32) + (threadIdx.x >> 5); i < all;
         i += (long long)gridDim.x * (kCta / 32)) {
        const int r = (int)(i / pieces), c = (int)(i - (long long)r * pieces) * kCols + lane * 8;
        const size_t at = (size_t)rows[r] * a.N + c;
        uint4 v[kCols / 256];
#pragma unroll
        for (int j = 0; j < kCols / 256; ++j)
            v[j] = a.residual ? load_cells<kVec>(a.residual + at + j * 256, a.N - c - j * 256)
                              : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kCols / 256; ++j)
            store_cells<kVec>(a.y + at + j * 256, a.N - c - j * 256, v[j]);
    }
}

// A tall tile, columns n0 <= n < n1 of a part, 128 at a time: the products of a step are
// issued a step ahead of its outputs.  The residual lies in the stage where the outputs
// take its place, row by row, and leave in whole sectors.  (Steps of 64 columns, 128 bytes of
// a row at a time, in two CTAs of 8 warps per SM: 189 us for 160, 4096 rows beside gate+up.
// Without the barrier per step, each warp with its own cells of the residual, 64 bytes of a
// row, and a further warp for B and the products: 160 for 149.)
template <bool kBf16, int RK, bool kVec>
__device__ void expand_tall(const LoraArgs &a, const uint16_t *order, const Tile &t, int part,
                            int n0, int n1, uint8_t *smem, Products &pr) {
    constexpr int kCta = expand_threads(false), kRs = residual_stages(RK), kBs = b_stages(RK);
    constexpr int kBlocks = blocks64(RK), kPieces = kBlocks * 8;  // of 16 bytes in a row of B
    // a step's copies are two groups, residual and B: at a step's start B of the next and the
    // residual of this one have to be there, and all younger groups may still be under way
    constexpr int kPending = kBs > 2 ? 2 : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = (int)dev::uniform(tid >> 5);
    const int rank = rank_of(a, t.adapter), ksteps = (int)dev::uniform((rank + 15) / 16);
    const uint32_t t_hi = smem_of(smem), t_lo = t_hi + t_half(RK), res0 = t_hi + 2 * t_half(RK),
                   b0 = res0 + kRs * kResidualStage;
    __shared__ float factor[kTall];
    const bool staged = kVec && a.residual;
    // this thread's 16 bytes of four rows of the residual, per stage
    const int col = tid & 15, r0 = tid >> 4;
    const uint16_t *rp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        rp[i] = staged && r < t.count ? a.residual + (size_t)order[r] * a.N + n0 + col * 8 : nullptr;
    }
    const uint16_t *b = a.b + ((size_t)t.adapter * a.N + n0) * a.R;
    const int steps = (n1 - n0 + kTallCols - 1) / kTallCols;
    // where 8 columns c of a row of a residual stage lie: two halves of 64 columns
    const auto cell = [](int r, int c) { return (uint32_t)(c >> 3) * (kTall * 128) + swizzled(r, c & 7); };
    // (a thread's rows are multiples of 8 apart, so their swizzle is the same)
    const int bj = tid / kPieces, bc = tid % kPieces;
    constexpr int kBRows = kCta / kPieces;  // rows of B between a thread's pieces
    static_assert(kBRows % 8 == 0, "the same swizzle");
    const uint32_t b_at = (bc >> 3) * kTallCols * 128 + swizzled(bj, bc & 7), r_at = cell(r0, col);
    const int b_size = bc < 2 * ksteps ? max(0, min(2 * (rank - bc * 8), 16)) : -1;
    const uint16_t *bp = b + (size_t)bj * a.R + bc * 8;
    auto issue_b = [&](int s) {
        if (b_size < 0) return;
        const uint32_t st = b0 + s % kBs * b_stage(RK) + b_at;
        const int n = s * kTallCols + bj;
#pragma unroll
        for (int i = 0; i < kTallCols / kBRows; ++i)
            copy16(st + i * kBRows * 128, bp + (size_t)(s * kTallCols + i * kBRows) * a.R,
                   n0 + n + i * kBRows < n1 ? b_size : 0);
    };
    auto issue_residual = [&](int s) {
        const uint32_t st = res0 + s % kRs * kResidualStage + r_at;
        const int n = s * kTallCols, in = n0 + n + col * 8 < n1 ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (rp[i]) copy16(st + i * 32 * 128, rp[i] + n, in);
    };
#pragma unroll
    for (int s = 0; s < kBs; ++s) {
        if (s < steps) issue_b(s);
        commit_copies();
    }
#pragma unroll
    for (int s = 0; s < kRs - 1; ++s) {
        if (s < steps) issue_residual(s);
        commit_copies();
    }
    const float scale = a.scales[t.adapter];
    wait_for_last();  // t
    {
        // four threads per row of t, a quarter of its part each
        constexpr int kQuads = kBlocks * 4;
        const int r = tid >> 2, quarter = tid & 3;
        const bool mine = r < t.count;
        const float *row = sums_of(a) + (mine ? (size_t)order[r] * a.parts * a.R + part * a.R : 0);
        float4 v[kQuads];
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int k = (quarter * kQuads + i) * 4, left = mine ? rank - k : 0;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (left > 0) v[i] = __ldcg(reinterpret_cast<const float4 *>(row + k));
            if (left < 4) v[i].w = 0.f;
            if (left < 3) v[i].z = 0.f;
            if (left < 2) v[i].y = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            most = larger(larger(larger(larger(most, v[i].x), v[i].y), v[i].z), v[i].w);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int e = row_exponent<kBf16>(most);
        const float down = scale_down(e);
        if (quarter == 0) factor[r] = scale_up(e) * scale;
#pragma unroll
        for (int i = 0; i < kQuads; i += 2) {
            uint32_t h[4], l[4];
            split<kBf16>(v[i].x, v[i].y, down, h[0], l[0]);
            split<kBf16>(v[i].z, v[i].w, down, h[1], l[1]);
            split<kBf16>(v[i + 1].x, v[i + 1].y, down, h[2], l[2]);
            split<kBf16>(v[i + 1].z, v[i + 1].w, down, h[3], l[3]);
            const int c = (quarter * kQuads + i) / 2;  // piece of 8
            const uint32_t at = (c >> 3) * kTall * 128 + swizzled(r, c & 7);
            sts128(t_hi + at, make_uint4(h[0], h[1], h[2], h[3]));
            sts128(t_lo + at, make_uint4(l[0], l[1], l[2], l[3]));
        }
    }
    const uint32_t idesc = product_desc<kBf16>(kTallCols), tmem = dev::uniform(pr.tmem);
    const uint32_t u_hi = dev::uniform(t_hi), u_lo = dev::uniform(t_lo), u_b = dev::uniform(b0);
    auto products = [&](int s) {  // warp 0
        if (!pr.ok) return;
        dev::tc_fence_after();
        const unsigned n = dev::uniform(pr.count + s);
        const uint32_t st = u_b + s % kBs * b_stage(RK), d = tmem + (n & 1) * kTallCols;
        const uint32_t bar = dev::uniform(pr.bar(n, kExpandBars));
        if (dev::elect_one()) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < kBlocks * 4; ++k)
                    if (k < ksteps)
                        product16(d,
                                  dev::smem_desc_sw128((h ? u_lo : u_hi) + (k >> 2) * kTall * 128) +
                                      2 * (k & 3),
                                  dev::smem_desc_sw128(st + (k >> 2) * kTallCols * 128) + 2 * (k & 3),
                                  idesc, h + k > 0);
            dev::mma_commit(bar);
        }
        __syncwarp();
        pr.issued = n + 1;
    };
    // outputs: a warp's 32 rows (its quarter of the tensor memory's lanes) and 32 columns;
    // out[i]: where row i * 8 + lane / 4 of them lies in y
    const int quarter = (warp & 3) * 32, side = (warp >> 2) * 32;
    const int mine = quarter + lane;
    uint16_t *out[4];
    bool there[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = quarter + i * 8 + (lane >> 2);
        there[i] = r < t.count;
        out[i] = a.y + (there[i] ? (size_t)order[r] * a.N : 0) + n0 + side + (lane & 3) * 8;
    }
    // in a residual stage (whose address is a multiple of 1024): piece i of the lane's row is at
    // own ^ i * 16, its piece of row i * 8 + lane / 4 at shared + i * 1024
    const uint32_t own = cell(mine, side >> 3),
                   shared = cell(quarter + (lane >> 2), (side >> 3) + (lane & 3));
    wait_copies<kBs - 1 + kRs - 1>();  // the first step's B
    dev::fence_async_shared();
    __syncthreads();
    const float f = factor[mine];
    if (warp == 0) products(0);
    for (int s = 0; s < steps; ++s) {
        wait_copies<kPending>();
        dev::fence_async_shared();
        __syncthreads();
        if (warp == 0 && s + 1 < steps) products(s + 1);
        if (s + kRs - 1 < steps) issue_residual(s + kRs - 1);
        commit_copies();
        const uint32_t st = res0 + s % kRs * kResidualStage;
        const int n = s * kTallCols + side, left = n1 - n0 - n;
        if constexpr (!kVec) {
            if (a.residual)
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    const int r = quarter + i;
                    uint16_t v = 0;
                    if (r < t.count && lane < left)
                        v = a.residual[(size_t)order[r] * a.N + n0 + n + lane];
                    sts16(st + cell(r, (side + lane) >> 3) + (lane & 7) * 2, v);
                }
            __syncwarp();
        }
        pr.wait(pr.count + s, kExpandBars);
        dev::tc_fence_after();
        // this step's products are done: its B makes room
        if (s + kBs < steps) issue_b(s + kBs);
        commit_copies();
        uint32_t v[32];
        dev::tmem_ld(pr.tmem + ((pr.count + s) & 1) * kTallCols + ((uint32_t)quarter << 16) + side,
                     v);
        dev::tmem_wait_ld(v);
        dev::tc_fence_before();
        uint4 r[4];  // (all loads, then the arithmetic: their latency shows)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = a.residual ? lds128((st + own) ^ (i << 4)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(v[8 * i + j]) * f;
            r[i] = add_cells<kBf16>(r[i], w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sts128((st + own) ^ (i << 4), r[i]);
        __syncwarp();
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = lds128(st + shared + i * 1024);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (there[i] && (lane & 3) * 8 < left)
                    *reinterpret_cast<uint4 *>(out[i] + s * kTallCols) = r[i];
        } else {
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const int r = quarter + i;
                const uint16_t w = lds16(st + cell(r, (side + lane) >> 3) + (lane & 7) * 2);
                if (r < t.count && lane < left)
                    a.y[(size_t)order[r] * a.N + n0 + n + lane] = w;
            }
        }
    }
    pr.count += steps;
    wait_copies<0>();
    __syncthreads();  // what comes next fills the same memory
}

// A low tile, columns n0 <= n < n1 of a part: every warp 32 of them in turn, with a ring of
// its own for B and (kVec) the residual.
template <bool kBf16, int RK, bool kVec, bool few>
__device__ void expand_low(const LoraArgs &a, const uint16_t *order, const Tile &t, int part,
                           int n0, int n1, uint8_t *smem) {
    constexpr int kStages = low_stages(RK, few), kBytes = low_stage(RK), kPieces = 2 * RK;
    constexpr int kStride = expand_threads(few) / 32 * kLowCols;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int rank = rank_of(a, t.adapter), ksteps = (rank + 15) / 16;
    const uint32_t base = smem_of(smem) + warp * kStages * kBytes;
    const uint16_t *b = a.b + (size_t)t.adapter * a.N * a.R;
    const bool staged = kVec && a.residual;
    const int m[2] = {g < t.count ? order[g] : -1, g + 8 < t.count ? order[g + 8] : -1};
    const size_t at[2] = {(size_t)max(m[0], 0) * a.N + c * 8, (size_t)max(m[1], 0) * a.N + c * 8};
    auto issue = [&](int n, int stage) {
        const uint32_t st = base + stage * kBytes;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int q = lane + i * 32, j = q / kPieces, r = q % kPieces * 8;
            const int in = n + j < n1 ? max(0, min(2 * (rank - r), 16)) : 0;
            copy16(st + interleaved(j) * row_pitch(RK) + r * 2,
                   in ? b + (size_t)(n + j) * a.R + r : a.b, in);
        }
        if (staged)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (m[u] >= 0 && n + c * 8 < n1)
                    copy16(st + kLowCols * row_pitch(RK) + (u * 8 + g) * (kLowCols * 2) + c * 16,
                           a.residual + at[u] + n, 16);
    };
    int n = n0 + warp * kLowCols, next = n;
#pragma unroll
    for (int s = 0; s < kStages; ++s, next += kStride) {
        if (next < n1) issue(next, s);
        commit_copies();
    }
    uint4 res[2];
    auto fetch = [&](int n) {  // the residual from memory, a step ahead
#pragma unroll
        for (int u = 0; u < 2; ++u)
            res[u] = a.residual && n < n1 && m[u] >= 0
                         ? load_cells<kVec>(a.residual + at[u] + n, n1 - n - c * 8)
                         : make_uint4(0, 0, 0, 0);
    };
    if constexpr (!kVec) fetch(n);
    const float scale = a.scales[t.adapter];
    Rows<kBf16, RK> rows;
    wait_for_last();  // t
    rows.load(a, m, part, rank, scale);
    for (int stage = 0; n < n1; n += kStride, next += kStride) {
        wait_copies<kStages - 1>();
        __syncwarp();
        const uint32_t st = base + stage * kBytes;
        float v[2][8];
        rows.product(v, st, ksteps);
        uint4 out[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (kVec)
                res[u] = staged ? lds128(st + kLowCols * row_pitch(RK) +
                                         (u * 8 + g) * (kLowCols * 2) + c * 16)
                                : make_uint4(0, 0, 0, 0);
            out[u] = add_cells<kBf16>(res[u], v[u]);
        }
        __syncwarp();  // all lanes have read the stage
        if (next < n1) issue(next, stage);
        commit_copies();
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (!kVec) fetch(n + kStride);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            store_cells<kVec>(a.y + at[u] + n, m[u] >= 0 ? n1 - n - c * 8 : 0, out[u]);
    }
    wait_copies<0>();
    __syncthreads();  // what comes next fills the same memory
}

// This CTA's share of `tiles` tiles' steps of `cols` columns, the parts' steps in turn: equal
// runs of the sequence, each piece of one tile and part to `run`
template <typename Run>
__device__ __forceinline__ void walk(const LoraArgs &a, int cols, int tiles, Run run) {
    int per = 0;
    for (int i = 0; i < a.parts; ++i) per += (a.part[i] + cols - 1) / cols;
    const int G = gridDim.x, i = blockIdx.x, all = tiles * per;
    int from = all / G * i + min(i, all % G);
    const int to = from + all / G + (i < all % G);
    int tile = from / per, s = from - tile * per;
    while (from < to) {
        int part = 0, first = 0, steps, at = s;
        for (;; ++part) {
            steps = (a.part[part] + cols - 1) / cols;
            if (at < steps) break;
            at -= steps;
            first += a.part[part];
        }
        const int n = min(steps - at, to - from);
        run(tile, part, first + at * cols, min(first + (at + n) * cols, first + a.part[part]));
        from += n, s += n;
        if (s == per) ++tile, s = 0;
    }
}

template <bool kBf16, int RK, bool kVec, bool few>
__global__ void __launch_bounds__(expand_threads(few), few ? 2 : 1) expand_kernel(LoraArgs a) {
    constexpr int kCta = expand_threads(few);
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = few ? smem_raw : align1024(smem_raw);
    __shared__ LocalPlan<kFewRows> own;
    __shared__ ProductSpace space;
    Products pr;
    if constexpr (!few) pr.begin<kExpandTmem>(&space, a.status);
    launch_next();
    Plan p;
    if constexpr (few) {
        // shrink has let this kernel start after all that came before shrink had ended: the
        // ids, B and the residual may be read before shrink's own results
        p = make_plan<kCta, kFewRows>(a, own, smem);
    } else {
        wait_for_last();  // (its shared memory lets it start only beside the last of shrink)
        p = shared_plan(a);
        p.n = *shared_counts(a);
    }
    if constexpr (!few)
        walk(a, kTallCols, p.n.tall, [&](int tile, int part, int n0, int n1) {
            const Tile t = p.tall(tile);
            expand_tall<kBf16, RK, kVec>(a, p.order + t.first, t, part, n0, n1, smem, pr);
        });
    walk(a, kLowCols, p.n.low, [&](int tile, int part, int n0, int n1) {
        const Tile t = p.low(tile);
        expand_low<kBf16, RK, kVec, few>(a, p.order + t.first, t, part, n0, n1, smem);
    });
    copy_rows<kCta, kVec>(a, p.order + p.n.rows, p.n.none);
    wait_for_last();  // (for those without a step: what follows this kernel waits for it alone)
    if constexpr (!few) pr.end<kExpandTmem, kExpandBars>();
}

template <bool kBf16, int RK, bool kVec, bool few>
cudaError_t launch_expand(const LoraArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    return launch_chained(expand_kernel<kBf16, RK, kVec, few>, dim3((few ? 2 : 1) * dev.sm_count),
                          expand_threads(few), expand_smem(RK, few), 1, stream, a);
}
template <bool kBf16, bool kVec, bool few>
cudaError_t launch_expand_rank(const LoraArgs &a, const DeviceInfo &dev, cudaStream_t stream) {
    if (a.R <= 16) return launch_expand<kBf16, 1, kVec, few>(a, dev, stream);
    if (a.R <= 32) return launch_expand<kBf16, 2, kVec, few>(a, dev, stream);
    if (a.R <= 64) return launch_expand<kBf16, 4, kVec, few>(a, dev, stream);
    return launch_expand<kBf16, 8, kVec, few>(a, dev, stream);
}

constexpr int kRounds = 4;
int resident_clusters[3];  // of shrink_kernel's kinds, that run at once (set by lora_init)

Kind kind_of(int M, int R, int parts) {
    if (M <= kFewRows) return kFew;
    const int units = (M + kTall - 1) / kTall * ((parts * R + kTallRanks - 1) / kTallRanks);
    return units <= resident_clusters[kDeep] ? kDeep : kMany;
}
// Shrink's clusters: one for each unit that there can be, up to some rounds of those that run
// at once (just those, each with all its units, 166 us for 152 at 4096 rows beside gate+up).
// Calls of few rows cut every adapter into low tiles, so they have up to M / 16 more of them
// than adapters (128 rows of one adapter beside qkv, K 5120, rank 16: 13.1 us, 22.6 with the
// bound of the others; 100 rows beside o 11.4 for 27.5).
int clusters_of(int M, int L, int R, int parts, Kind kind) {
    const int adapters = M < L ? M : L;
    const long long tiles = kind != kFew              ? lora_max_tiles(M, L)
                            : adapters + M / kLow < M ? adapters + M / kLow
                                                      : M;
    const long long units = tiles * ((parts * R + kLowRanks - 1) / kLowRanks);
    const int most = kRounds * resident_clusters[kind];
    return units < most ? (int)units : most;
}

template <bool kBf16, Kind kKind>
cudaError_t launch_calls(const LoraArgs &a, bool vec, const DeviceInfo &dev, cudaStream_t stream) {
    constexpr bool few = kKind == kFew;
    if (a.M > kLocalRows) {
        const cudaError_t e = launch_chained(plan_kernel, dim3(1), kPlanThreads, 0, 1, stream, a);
        if (e != cudaSuccess) return e;
    }
    const int clusters = clusters_of(a.M, a.L, a.R, a.parts, kKind);
    const cudaError_t e =
        launch_chained(shrink_kernel<kBf16, kKind>, dim3(clusters * kCluster), kShrinkThreads,
                       shrink_smem(kKind), kCluster, stream, a);
    if (e != cudaSuccess) return e;
    return vec ? launch_expand_rank<kBf16, true, few>(a, dev, stream)
               : launch_expand_rank<kBf16, false, few>(a, dev, stream);
}

cudaError_t set_smem(const void *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <bool kBf16, bool few, int RK>
cudaError_t init_expand() {
    const cudaError_t e =
        set_smem((const void *)expand_kernel<kBf16, RK, true, few>, expand_smem(RK, few));
    return e != cudaSuccess ? e
                            : set_smem((const void *)expand_kernel<kBf16, RK, false, few>,
                                       expand_smem(RK, few));
}
template <bool kBf16, Kind kKind>
cudaError_t init_shrink() {
    cudaError_t e = set_smem((const void *)shrink_kernel<kBf16, kKind>, shrink_smem(kKind));
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kCluster);
        cfg.blockDim = dim3(kShrinkThreads);
        cfg.dynamicSmemBytes = shrink_smem(kKind);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, shrink_kernel<kBf16, kKind>, &cfg);
        if (e == cudaSuccess && n < 1) e = cudaErrorInvalidConfiguration;
        resident_clusters[kKind] = n;
    }
    return e;
}
template <bool kBf16>
cudaError_t init_calls() {
    cudaError_t e = init_shrink<kBf16, kFew>();
    if (e == cudaSuccess) e = init_shrink<kBf16, kDeep>();
    if (e == cudaSuccess) e = init_shrink<kBf16, kMany>();
    if (e == cudaSuccess) e = init_expand<kBf16, true, 1>();
    if (e == cudaSuccess) e = init_expand<kBf16, false, 1>();
    if (e == cudaSuccess) e = init_expand<kBf16, true, 2>();
    if (e == cudaSuccess) e = init_expand<kBf16, false, 2>();
    if (e == cudaSuccess) e = init_expand<kBf16, true, 4>();
    if (e == cudaSuccess) e = init_expand<kBf16, false, 4>();
    if (e == cudaSuccess) e = init_expand<kBf16, true, 8>();
    if (e == cudaSuccess) e = init_expand<kBf16, false, 8>();
    return e;
}

}  // namespace

cudaError_t launch_lora(const LoraArgs &a, bool bf16, const DeviceInfo &dev, cudaStream_t stream) {
    // 16-byte accesses of y and the residual
    bool vec = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.residual & 15) == 0;
    for (int i = 0; i < a.parts; ++i) vec = vec && a.part[i] % 8 == 0;
    switch (kind_of(a.M, a.R, a.parts)) {
        case kFew:
            return bf16 ? launch_calls<true, kFew>(a, vec, dev, stream)
                        : launch_calls<false, kFew>(a, vec, dev, stream);
        case kDeep:
            return bf16 ? launch_calls<true, kDeep>(a, vec, dev, stream)
                        : launch_calls<false, kDeep>(a, vec, dev, stream);
        default:
            return bf16 ? launch_calls<true, kMany>(a, vec, dev, stream)
                        : launch_calls<false, kMany>(a, vec, dev, stream);
    }
}

void lora_plan(int M, int L, int R, int parts, int32_t *info) {
    const Kind kind = kind_of(M, R, parts);
    info[0] = kind;
    info[1] = clusters_of(M, L, R, parts, kind);
    info[2] = lora_kernels(M);
}

cudaError_t lora_init() {
    const cudaError_t e = init_calls<true>();
    return e == cudaSuccess ? init_calls<false>() : e;
}

}  // namespace w4a16
