// A layer of experts whose weights come in 8 bits, for the few tokens of a decode step:
//
//   h[s] = silu(gate_e x[t]) * up_e x[t],   out[t] = sum_j weights[t, j] * down_e h[s]
//
// with slot s = t k + j the token's j-th choice and e = ids[t, j].  (forum.sourcefind.cn
// thread "vLLM on Hygon Z100", section 七: tokens regrouped by expert, an expert small-M
// product, the weighted sum; section 六: FP8 checkpoints.)  Weights are e4m3 with a scale
// per block of 128 x 128, activations 16 bits.
//
// Three kernels: gate and up with silu-and-mul, down, the weighted sum.  Both products are
// one kernel, experts_kernel.  A tile is up to 8 NT columns of one expert, a slot each (of
// down two, see below); a unit is a tile and 16 * 8 / KS rows of the expert's weights, whose K
// a CTA walks in stages of KS blocks of 128: a warp has 16 rows (for gate and up: 8 gate rows
// and their 8 up rows, so that a lane holds a gate sum and its up sum) and one of the stage's
// KS blocks, and the KS warps of the same rows add their sums at the unit's end.  So every stage brings 16 KB of
// weights in runs of 128 KS bytes of a row, and a unit is small (KS 8) where there are few
// tiles.  The weights are the warp MMA's M, the tokens its N: a decode step's experts see
// one to a few tokens each, and the bytes of the weights bound the layer, not the products
// (8 tokens need 1/16 of what the warp MMA can do while the weights arrive).
//
// e4m3 codes become the 16-bit type exactly (through fp16, which holds all of them); the
// products of a block are summed in fp32, scaled once and added in fp32.  h enters down as two
// bf16 values, the value rounded and the rest rounded, whatever the layer's type: 16 bits of
// it at fp32's range (fp16 would end at 65504).  They are two neighbouring columns of down's
// tile, whose sums one lane holds; so a tile of few slots costs no further products.  down's
// sums stay fp32 up to the one rounding of out.
//
// Every CTA groups the slots itself (a stable counting sort in shared memory, or one warp's
// work up to 32 slots), which costs it no launch and no pass through memory.
//
// What bounds it (one GB300, calls in a row in a graph; 128 experts, 8 each, 2048 -> 2 x 768
// -> 2048).  64 tokens, bf16: 113 us, 595 MB at 5.3 TB/s, 78% of the measured copy rate; the
// issue slots (the codes' way to bf16 is four instructions a pair, for fp16 one) and the
// barrier per stage (with the products switched off, h in one value, 99 us).  8 tokens, fp16:
// 48.9 us, 5.0 TB/s.  One token: 14.2 us for 38 MB, of which the weights' stream is 6; the rest
// are the ids' load, the grouping and the first weights' latency, twice, and the sum.
// With h rounded once to the 16-bit type these took 109, 46.9 and 13.9 us, and out's error was
// 1.4 to 1.5 times that of h in fp32 (now the same to four digits); with the two values in
// tiles of their own 114, 50.5 and 14.4.
// Tried and not kept, with h in one value: bf16 activations scaled to fp16 in the stage (30% fewer instructions,
// but on every stage's critical path: 124 us at 64 tokens for 115), five or six stages (no
// change: the bytes in flight are enough), one CTA per SM (205), the sum by the last of down's
// units (one token 15.1 for 13.9).
#include <math.h>

#include "w4a16_routed.cuh"

namespace w4a16 {
namespace {

using namespace routed;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 4;
constexpr int kStageWeights = 16 << 10;  // bytes

// two e4m3 codes -> two 16-bit values, exact
template <bool kBf16>
__device__ __forceinline__ uint32_t widen(uint16_t codes) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(codes));
    if constexpr (kBf16) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&d);
        const __nv_bfloat162 b = __floats2bfloat162_rn(__low2float(h), __high2float(h));
        d = *reinterpret_cast<const uint32_t *>(&b);
    }
    return d;
}
struct Tables {
    uint16_t slot[kFp8MoeMaxSlots];         // slots by expert, in order
    uint16_t tile_expert[kFp8MoeMaxSlots];  // a tile: slots tile_first .. + tile_count
    uint16_t tile_first[kFp8MoeMaxSlots];
    uint8_t tile_count[kFp8MoeMaxSlots];
    int tiles;
};
using Sort = RowSort<kFp8MoeMaxSlots>;
// columns of a tile: 8 NT, fewer where a stage of KS blocks leaves no room for them
template <int NT, int KS>
constexpr int kCap = 8 * NT * KS <= 32 ? 8 * NT : 32 / KS;
// bytes of a stage: the weights, the columns' activations, the scales
template <int NT, int KS>
constexpr int kStageBytes = kStageWeights + kCap<NT, KS> * 256 * KS + 128;
// The kernel's dynamic shared memory: the stages, where the slots are sorted before.  No more
// than that, so that two CTAs share an SM: NT 2, KS 2 with its 15 KB of tables and sums, too
// (40 tokens, 2 of 8 experts, 2048 -> 2 x 1024 -> 2048: 20.4 us, with 100 KB for every cut 27.6).
template <int NT, int KS>
constexpr int kRingBytes = kStages * kStageBytes<NT, KS> > (int)sizeof(Sort)
                               ? kStages * kStageBytes<NT, KS>
                               : (int)sizeof(Sort);
static_assert(kMaxMoeExperts <= kMaxBins, "the sort holds every expert");

// The slots by expert, in tiles of up to cap slots; how many tiles.  An id outside [0, E)
// leaves its slot out; one other than -1 is reported.
__device__ int make_tiles(Tables &tb, Sort &sp, const int32_t *ids, int S, int E, int cap,
                          int *status) {
    group_rows<kThreads>(
        sp, tb.slot, S, E,
        [&](int s) {
            const int e = ids[s];
            if ((unsigned)e >= (unsigned)E && e != -1 && status && blockIdx.x == 0)
                atomicOr(status, kErrMoeIds);
            return e;
        },
        [&](int, int n) { return (unsigned)n | (unsigned)(n + cap - 1) / cap << 11; },
        [&](int e, int n, unsigned at) {
            int tile = at >> 11, first = at & 2047;
            for (; n > 0; n -= cap, first += cap, ++tile) {
                tb.tile_expert[tile] = (uint16_t)e;
                tb.tile_first[tile] = (uint16_t)first;
                tb.tile_count[tile] = (uint8_t)min(cap, n);
            }
        },
        [&](unsigned total) { tb.tiles = total >> 11; });
    return tb.tiles;
}

// silu(g) u = g u / (1 + e^-g).  Far below zero, where 1 + e^-g is e^-g to fp32's last bit and
// leaves its range soon, it is g p u p with p = e^(g/2), in an order that neither overflows nor
// underflows before the result does.  -Inf gives NaN, as the quotient does.
__device__ __forceinline__ float silu_mul(float g, float u) {
    if (g < -80.f) {
        const float p = expf(0.5f * g);
        return g * p * u * p;
    }
    return g / (1.f + expf(-g)) * u;
}

// v as two bf16 values; the largest finite ones, whose nearest bf16 is Inf, stay finite
__device__ __forceinline__ void halves(float v, uint16_t &hi, uint16_t &lo) {
    __nv_bfloat16 h = __float2bfloat16_rn(v);
    float rest = v - __bfloat162float(h);
    if (__hisinf(h)) {
        h = __float2bfloat16_rz(v);  // (of Inf Inf)
        rest = isinf(v) ? 0.f : __bfloat162float(__float2bfloat16_rz(v - __bfloat162float(h)));
    }
    hi = __bfloat16_as_ushort(h);
    lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
}

// kSilu: gate and up, x by token, h by slot; else down, h by slot, o (fp32) by slot.  h is
// two rows of bf16 per slot, the values and the rests.
template <bool kBf16, int NT, int KS, bool kSilu>
__global__ void __launch_bounds__(kThreads, 2) experts_kernel(Fp8ExpertsArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Tables tb;
    __shared__ float red[kWarps * 32 * NT * 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int S = a.T * a.k, cap = a.cap;

    if constexpr (kSilu) wait_for_last();
    launch_next();
    const int n_tiles = make_tiles(tb, *reinterpret_cast<Sort *>(ring), a.ids, S, a.E, cap,
                                   kSilu ? a.status : nullptr);

    constexpr int ks_log = KS == 8 ? 3 : KS == 4 ? 2 : KS == 2 ? 1 : 0;
    constexpr int per = (kSilu ? 64 : 128) / KS;  // rows of results of a unit
    constexpr int x_bytes = kCap<NT, KS> * 256 * KS, stage_bytes = kStageBytes<NT, KS>;
    const int blocks = (a.rows + per - 1) / per, units = n_tiles * blocks;
    const int ksteps = (a.K + 128 * KS - 1) / (128 * KS);
    const int mine = blockIdx.x < units ? (units - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    const int steps = mine * ksteps;
    const uint32_t ring0 = smem_of(ring);
    const int Gk = (a.K + kGroup - 1) / kGroup;

    // Copies walk the units' stages in order.  Per unit each thread keeps where its 16-byte
    // pieces of weights (four), activations (kX) and its scale come from.
    constexpr int kW = kStageWeights / 16 / kThreads;
    constexpr int kX = (kCap<NT, KS> * 16 * KS + kThreads - 1) / kThreads;
    const int wc = tid & (8 * KS - 1), wr = tid >> (3 + ks_log);     // piece of a row, row
    const int xc = tid & (16 * KS - 1), xr = tid >> (4 + ks_log);
    struct Cursor {
        int unit, kstep, stage;
    };
    const uint8_t *wp[kW];
    const uint16_t *xp[kX];
    const float *sp = a.s;
    int w_size[kW] = {};  // 16, or 0 for a piece of a row that does not exist
    auto enter_weights = [&](int unit) {
        const int tile = unit / blocks, row0 = (unit - tile * blocks) * per;
        const size_t e = tb.tile_expert[tile];
        const uint8_t *w = a.w + e * a.w_rows * a.K + wc * 16;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int r = wr + i * (32 >> ks_log);
            int row = row0 + r, j = row;
            if constexpr (kSilu) {
                j = row0 + (r >> 4) * 8 + (r & 7);
                row = j + (r & 8 ? a.rows : 0);
            }
            wp[i] = w + (size_t)row * a.K;
            w_size[i] = j < a.rows ? 16 : 0;
        }
        if (tid < 2 * kWarps) {
            const int rg = (tid >> 1) >> ks_log;
            int row;
            if constexpr (kSilu)
                row = min(row0 + rg * 8, a.rows - 1) + (tid & 1 ? a.rows : 0);
            else
                row = min(row0 + rg * 16 + (tid & 1 ? 8 : 0), a.rows - 1);
            sp = a.s + (e * ((a.w_rows + kGroup - 1) / kGroup) + row / kGroup) * Gk;
        }
    };
    auto enter_x = [&](int unit) {
        const int tile = unit / blocks, first = tb.tile_first[tile], n = tb.tile_count[tile];
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int r = xr + i * (16 >> ks_log), tok = kSilu ? r : r >> 1;
            xp[i] = nullptr;
            if (tok < n) {
                const int s = tb.slot[first + tok];
                xp[i] = a.x + (size_t)(kSilu ? s / a.k : 2 * s + (r & 1)) * a.K + xc * 8;
            }
        }
    };
    auto copy_weights = [&](const Cursor &cu) {
        // piece c of row r is at c ^ 4 in odd rows, so that lanes of neighbouring rows read
        // other banks (this thread's rows are all odd or all even)
        const uint32_t st = (ring0 + cu.stage * stage_bytes + tid * 16) ^ ((wr & 1) << 6);
        const int k = cu.kstep * KS * kGroup;
        const int in = k + wc * 16 < a.K ? 16 : 0;
#pragma unroll
        for (int i = 0; i < kW; ++i)  // (no bytes are read where the size is 0)
            copy16(st + i * kThreads * 16, wp[i] + k, min(in, w_size[i]));
        if (tid < 2 * kWarps)
            copy4(ring0 + cu.stage * stage_bytes + kStageWeights + x_bytes + tid * 4,
                  sp + min(cu.kstep * KS + ((tid >> 1) & (KS - 1)), Gk - 1));
    };
    auto copy_x = [&](const Cursor &cu) {
        const uint32_t st = ring0 + cu.stage * stage_bytes + kStageWeights;
        const int k = cu.kstep * KS * kGroup;
        const int in = k + xc * 8 < a.K ? 16 : 0;
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int r = xr + i * (16 >> ks_log);
            if (xp[i])
                copy16(st + (r << (8 + ks_log)) + ((xc ^ (r & 1)) << 4), xp[i] + k, in);
        }
    };
    auto advance = [&](Cursor &cu) {
        cu.stage = cu.stage == kStages - 1 ? 0 : cu.stage + 1;
        if (++cu.kstep == ksteps) {
            cu.kstep = 0;
            cu.unit += gridDim.x;
        }
    };

    Cursor in = {(int)blockIdx.x, 0, 0};
    if constexpr (!kSilu) {
        // the weights do not depend on the kernel before
        for (int i = 0; i < kStages - 1 && i < steps; ++i) {
            if (in.kstep == 0) enter_weights(in.unit);
            copy_weights(in);
            advance(in);
        }
        in = {(int)blockIdx.x, 0, 0};
        wait_for_last();
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < steps) {
            if (kSilu && in.kstep == 0) enter_weights(in.unit);
            if (in.kstep == 0) enter_x(in.unit);
            if (kSilu) copy_weights(in);
            copy_x(in);
            advance(in);
        }
        commit_copies();  // (down: the first group holds the weights of all)
    }

    const int rg = warp >> ks_log, ks = warp & (KS - 1);
    float tot[NT][4] = {};
    Cursor at = {(int)blockIdx.x, 0, 0};
    for (int step = 0; step < steps; ++step, advance(at)) {
        wait_copies<kStages - 2>();
        __syncthreads();  // the stage is there, and the one before it is free
        if (step + kStages - 1 < steps) {
            if (in.kstep == 0) enter_weights(in.unit), enter_x(in.unit);
            copy_weights(in);
            copy_x(in);
            advance(in);
        }
        commit_copies();
        const uint32_t st = ring0 + at.stage * stage_bytes;
        float acc[NT][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t wp = st + ((rg * 16 + g) << (7 + ks_log)) +
                                (((ks * 8 + h * 4 + c) ^ ((g & 1) << 2)) << 4);
            const uint4 lo = lds128(wp), hi = lds128(wp + (8 << (7 + ks_log)));
            const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
            uint32_t b[NT][8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int col = min(n * 8 + g, kCap<NT, KS> - 1);
                const uint32_t xp = st + kStageWeights + (col << (8 + ks_log));
                const int c16 = ks * 16 + h * 8 + c * 2;
                const uint4 b0 = lds128(xp + ((c16 ^ (col & 1)) << 4)),
                            b1 = lds128(xp + (((c16 + 1) ^ (col & 1)) << 4));
                b[n][0] = b0.x, b[n][1] = b0.y, b[n][2] = b0.z, b[n][3] = b0.w;
                b[n][4] = b1.x, b[n][5] = b1.y, b[n][6] = b1.z, b[n][7] = b1.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a0 = widen<kBf16>((uint16_t)wl[j]),
                               a2 = widen<kBf16>((uint16_t)(wl[j] >> 16)),
                               a1 = widen<kBf16>((uint16_t)wh[j]),
                               a3 = widen<kBf16>((uint16_t)(wh[j] >> 16));
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma<kBf16>(acc[n], a0, a1, a2, a3, b[n][2 * j], b[n][2 * j + 1]);
            }
        }
        const float *sc = reinterpret_cast<const float *>(ring + at.stage * stage_bytes +
                                                          kStageWeights + x_bytes) + warp * 2;
        const float s0 = sc[0], s1 = sc[1];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            tot[n][0] = fmaf(s0, acc[n][0], tot[n][0]);
            tot[n][1] = fmaf(s0, acc[n][1], tot[n][1]);
            tot[n][2] = fmaf(s1, acc[n][2], tot[n][2]);
            tot[n][3] = fmaf(s1, acc[n][3], tot[n][3]);
        }
        if (at.kstep != ksteps - 1) continue;

        // the unit's end: the warps of the same rows add up, in the order of their blocks
        if (ks != 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[((warp * NT + n) * 4 + i) * 32 + lane] = tot[n][i];
        }
        __syncthreads();
        if (ks == 0) {
            for (int w = 1; w < KS; ++w)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tot[n][i] += red[(((warp + w) * NT + n) * 4 + i) * 32 + lane];
            const int tile = at.unit / blocks, row0 = (at.unit - tile * blocks) * per;
            const int first = tb.tile_first[tile], count = tb.tile_count[tile];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if constexpr (kSilu) {
                    const int j = row0 + rg * 8 + g;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int tok = n * 8 + c * 2 + i;
                        if (tok >= count || j >= a.rows) continue;
                        uint16_t *h = a.h + 2 * (size_t)tb.slot[first + tok] * a.rows + j;
                        halves(silu_mul(tot[n][i], tot[n][2 + i]), h[0], h[a.rows]);
                    }
                } else {
                    const int tok = n * 4 + c, j = row0 + rg * 16 + g;
                    if (tok >= count) continue;
                    float *o = a.o + (size_t)tb.slot[first + tok] * a.rows + j;
                    if (j < a.rows) o[0] = tot[n][0] + tot[n][1];
                    if (j + 8 < a.rows) o[8] = tot[n][2] + tot[n][3];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[n][i] = 0.f;
    }
}

// out[t] = sum_j weights[t, j] * o[t k + j], j in order, without the choices that are none
template <bool kBf16>
__global__ void __launch_bounds__(256) combine_kernel(const float *o, const int32_t *ids,
                                                      const float *weights, int T, int k, int E,
                                                      int N, uint16_t *out) {
    launch_next();
    wait_for_last();
    const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float v = 0.f;
    for (int j = 0; j < k; ++j) {
        const int s = t * k + j;
        if ((unsigned)ids[s] < (unsigned)E) v = fmaf(weights[s], o[(size_t)s * N + n], v);
    }
    out[(size_t)t * N + n] = float_to_half_bits(v, kBf16);
}

// How a product is cut: NT by which columns of an expert share a tile, KS by which a stage's
// blocks are split among the warps.
struct Cut {
    int nt, ks;
};
// The cut of the smallest cost: the units of the busiest CTA, each its weights' bytes, its
// activations' and 8 KB for its start and end, a tenth more for each further 8 columns of a
// tile.  The choices are on the device, so the tiles are those of even choices: `used`
// experts with `each` slots, each so many columns.  (64 tokens, 4 of 16 experts, 2048 -> 2 x
// 768 -> 2048, bf16: gate and up by NT 2, KS 1 36.9 us, by 1, 1 46.3, by 4, 1 42.2; down by
// 4, 1 36.9, by 2, 1 38.4, by 1, 1 42.5.  Of twelve such sizes, 1 to 64 tokens and 8 to 128
// experts, the choice is at most 7% behind the best: 64 tokens, 4 of 8, 34.0 for 31.8.)
Cut cut_of(double used, double each, int T, int columns, int rows_per_unit, int rows, int K,
           int grid) {
    Cut best{1, 1};
    double least = INFINITY;
    for (int nt = 1; nt <= 4; nt *= 2) {
        const int most = 8 / columns * nt, cap = T < most ? T : most;  // slots
        const double tiles = used * (cap == T || each <= 0.6 * cap ? 1.0 : each / cap + 0.5);
        for (int ks = 1; ks * columns * cap <= 32 && ks * nt <= (nt == 1 ? 8 : 4); ks *= 2) {
            const int per = rows_per_unit / ks;
            const double units = tiles * ((rows + per - 1) / per);
            const double cost = ceil(units / grid) * (0.9 + 0.1 * nt) *
                                (128.0 / ks * K + 2.0 * columns * fmin(cap, each) * K + 8192);
            if (cost < least) least = cost, best = {nt, ks};
        }
        if (T <= most) break;
    }
    return best;
}

template <bool kBf16, bool kSilu, int NT, int KS>
cudaError_t launch_cut(Fp8ExpertsArgs &p, int grid, cudaStream_t stream) {
    constexpr int most = (kSilu ? 8 : 4) * NT;
    p.cap = p.T < most ? p.T : most;
    return launch_chained(experts_kernel<kBf16, NT, KS, kSilu>, dim3(grid), kThreads,
                          kRingBytes<NT, KS>, 1, stream, p);
}
template <bool kBf16, bool kSilu>
cudaError_t launch_product(Fp8ExpertsArgs p, Cut cut, int grid, cudaStream_t stream) {
    switch (cut.nt * 16 + cut.ks) {
        case 1 * 16 + 1: return launch_cut<kBf16, kSilu, 1, 1>(p, grid, stream);
        case 1 * 16 + 2: return launch_cut<kBf16, kSilu, 1, 2>(p, grid, stream);
        case 1 * 16 + 4: return launch_cut<kBf16, kSilu, 1, 4>(p, grid, stream);
        case 1 * 16 + 8: return launch_cut<kBf16, kSilu, 1, 8>(p, grid, stream);
        case 2 * 16 + 1: return launch_cut<kBf16, kSilu, 2, 1>(p, grid, stream);
        case 2 * 16 + 2: return launch_cut<kBf16, kSilu, 2, 2>(p, grid, stream);
        default: return launch_cut<kBf16, kSilu, 4, 1>(p, grid, stream);
    }
}

struct Plan {
    Cut gate_up, down;
    int grid;
};
Plan plan_of(int T, int k, int E, int K, int I, int N, const DeviceInfo &dev) {
    const int grid = 2 * dev.sm_count;
    const double used = E * (1.0 - pow(1.0 - fmin(1.0, (double)k / E), T)), each = T * k / used;
    return {cut_of(used, each, T, 1, 64, I, K, grid), cut_of(used, each, T, 2, 128, N, I, grid),
            grid};
}

template <bool kBf16>
cudaError_t launch_type(const Fp8MoeArgs &a, const DeviceInfo &dev, int *status,
                        cudaStream_t stream) {
    const Plan plan = plan_of(a.T, a.k, a.E, a.K, a.I, a.N, dev);
    uint16_t *h = static_cast<uint16_t *>(a.scratch);
    float *o = reinterpret_cast<float *>(static_cast<char *>(a.scratch) +
                                         fp8_moe_h_bytes(a.T, a.k, a.I));
    cudaError_t e = launch_product<kBf16, true>(
        {a.x, a.w1, a.s1, a.ids, h, nullptr, status, a.T, a.k, a.E, a.K, a.I, 2 * a.I, 0},
        plan.gate_up, plan.grid, stream);
    if (e != cudaSuccess) return e;
    e = launch_product<true, false>(
        {h, a.w2, a.s2, a.ids, nullptr, o, status, a.T, a.k, a.E, a.I, a.N, a.N, 0},
        plan.down, plan.grid, stream);
    if (e != cudaSuccess) return e;
    return launch_chained(combine_kernel<kBf16>, dim3((a.N + 255) / 256, a.T), 256, 0, 1, stream,
                          (const float *)o, a.ids, a.weights, a.T, a.k, a.E, a.N, a.out);
}

// CTAs of each cut's kernels that an SM holds at once, the fewest of both types (set by
// fp8_moe_init)
int resident[2][5][9];  // [gate and up][NT][KS]

template <bool kBf16, bool kSilu, int NT, int KS>
cudaError_t init_cut() {
    const auto kernel = experts_kernel<kBf16, NT, KS, kSilu>;
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRingBytes<NT, KS>);
    int n = 0;
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, kRingBytes<NT, KS>);
    int &r = resident[kSilu][NT][KS];
    if (e == cudaSuccess && (r == 0 || n < r)) r = n;
    return e;
}
template <bool kBf16, bool kSilu>
cudaError_t init_product() {
    cudaError_t e = init_cut<kBf16, kSilu, 1, 1>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 1, 2>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 1, 4>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 1, 8>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 2, 1>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 2, 2>();
    if (e == cudaSuccess) e = init_cut<kBf16, kSilu, 4, 1>();
    return e;
}

}  // namespace

cudaError_t launch_fp8_moe(const Fp8MoeArgs &a, bool bf16, const DeviceInfo &dev, int *status,
                           cudaStream_t stream) {
    return bf16 ? launch_type<true>(a, dev, status, stream)
                : launch_type<false>(a, dev, status, stream);
}

cudaError_t fp8_moe_init() {
    cudaError_t e = init_product<true, true>();
    if (e == cudaSuccess) e = init_product<false, true>();
    if (e == cudaSuccess) e = init_product<true, false>();
    return e;
}

void fp8_moe_plan(int T, int k, int E, int K, int I, int N, const DeviceInfo &dev, int32_t *info) {
    const Plan p = plan_of(T, k, E, K, I, N, dev);
    info[0] = p.gate_up.nt, info[1] = p.gate_up.ks;
    info[2] = p.down.nt, info[3] = p.down.ks;
    info[4] = p.grid;
    const int a = resident[1][p.gate_up.nt][p.gate_up.ks], b = resident[0][p.down.nt][p.down.ks];
    info[5] = a < b ? a : b;
}

}  // namespace w4a16
