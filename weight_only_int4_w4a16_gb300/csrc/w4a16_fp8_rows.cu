// The steps around the 8-bit linear of w4a16_fp8.cu that are done row by row:
//
//   rmsnorm   h = x + residual,  v = h / sqrt(mean(h^2) + eps) * weight
//   quant     v = x,  or  v = silu(x[:, :n]) * x[:, n:],  silu(g) = g / (1 + e^-g)
//
// (forum.sourcefind.cn thread "vLLM on Hygon Z100", section 二, names RMSNorm
// and SiLU-and-mul among the operators between a decoder layer's linears), with
// v written in 16 bits (rmsnorm) or as an 8-bit row: per group of 128
// consecutive elements one scale s = max(a, 2^-100) / 448, a the group's
// largest finite magnitude, and per element e4m3(v / s), nearest even.
//
// Everything before the stores is fp32; the sum h is rounded to 16 bits only
// where it is stored (the norm reads the unrounded sum), v once where it is
// stored.  v / s is the correctly rounded fp32 quotient, from the correctly
// rounded reciprocal r = 1 / s and one correction (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): q0 = v r,
// q = q0 + (v - q0 s) r, so a tie of e4m3 falls as it does for IEEE division.
// Inf and NaN elements do not enter a and become e4m3's NaN, so that one of
// them does not take its group with it.
//
// Layout: a lane holds 8 consecutive elements (a 16-byte load), so 16 lanes
// hold a group and four shuffles give its largest magnitude.  Rows whose width
// or address does not allow 16-byte accesses are read and written element by
// element (kVec false), the lanes of a group on neighbours.  In the norm they then
// change hands in shared memory (kStaged), so that a lane adds the same squares and a
// row has the same bits; the quantisation has no sums, and its lanes keep every 16th
// element.
#include <float.h>

#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr int kLaneElems = 8;                             // elements of a row per lane and step
constexpr int kGroupLanes = kGroup / kLaneElems;          // 16 lanes hold a scale group
constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.8886090522101180541e-31f;  // 2^-100

// lets the next kernel's CTAs start while this one drains, then waits for the
// kernel before (whose outputs this one may read)
__device__ __forceinline__ void chain_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Two fp32 values in one 64-bit register: the packed instructions round each as the
// scalar ones do and take half their issue slots, which is what bounds these kernels
// beside memory.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float lo, float hi) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
__device__ __forceinline__ float lo(f2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(f2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 neg2(f2 a) { return a ^ 0x8000000080000000ull; }

template <bool kBf16>
__device__ __forceinline__ float to_float(uint16_t h) {
    if constexpr (kBf16) return __uint_as_float((uint32_t)h << 16);
    else return __half2float(__ushort_as_half(h));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t to_16(float v) {  // nearest, ties to even
    if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else return __half_as_ushort(__float2half_rn(v));
}

// Where the two groups of a warp change hands: 128 elements each, the second in other
// banks than the first.
constexpr int kStageGroup = kGroup + 16;
constexpr int kStageWarp = 2 * kStageGroup;  // 16-bit words
// The group's part of a warp's stage, and its lane's first element there and in the
// row when the lanes take neighbours; element i of the lane is 16 i further.
__device__ __forceinline__ uint16_t *group_stage(uint16_t *stage) {
    return stage + (threadIdx.x & kGroupLanes ? kStageGroup : 0);
}
__device__ __forceinline__ int neighbour(int c) {
    return (c & ~(kGroup - 1)) + (threadIdx.x & (kGroupLanes - 1));
}

// Elements c .. c + 7 of a row (zeros past its n elements), in pairs; with neither kVec
// nor kStaged every 16th of its group.  All lanes of the warp call it together (and
// store8); stage is the warp's own.
template <bool kBf16, bool kVec, bool kStaged>
__device__ __forceinline__ void load8(const uint16_t *row, int c, int n, f2 (&v)[4],
                                      uint16_t *stage) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if constexpr (kVec) {  // n is a multiple of 8
        if (c < n) u = *reinterpret_cast<const uint4 *>(row + c);
    } else {
        const int e = neighbour(c);
        uint16_t h[kLaneElems];
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i)
            h[i] = e + kGroupLanes * i < n ? row[e + kGroupLanes * i] : (uint16_t)0;
        if constexpr (kStaged) {
            uint16_t *own = group_stage(stage);
#pragma unroll
            for (int i = 0; i < kLaneElems; ++i) own[e % kGroup + kGroupLanes * i] = h[i];
            __syncwarp();
            u = *reinterpret_cast<const uint4 *>(own + c % kGroup);
            __syncwarp();
        } else {
            u = make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16,
                           h[4] | (uint32_t)h[5] << 16, h[6] | (uint32_t)h[7] << 16);
        }
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pack(to_float<kBf16>((uint16_t)w[i]), to_float<kBf16>((uint16_t)(w[i] >> 16)));
}

template <bool kBf16, bool kVec>
__device__ __forceinline__ void store8(uint16_t *row, int c, int n, const f2 (&v)[4],
                                       uint16_t *stage) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)to_16<kBf16>(lo(v[i])) | (uint32_t)to_16<kBf16>(hi(v[i])) << 16;
    const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (kVec) {
        if (c < n) *reinterpret_cast<uint4 *>(row + c) = u;
    } else {
        const int e = neighbour(c);
        uint16_t *own = group_stage(stage);
        *reinterpret_cast<uint4 *>(own + c % kGroup) = u;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i)
            if (e + kGroupLanes * i < n)
                row[e + kGroupLanes * i] = own[e % kGroup + kGroupLanes * i];
        __syncwarp();
    }
}

// two fp32 values -> two e4m3 codes (lo in the low byte), nearest even
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// max(a, |b|) where NaN wins
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}
// the largest of the 16 lanes of a group
__device__ __forceinline__ float group_max(float a) {
#pragma unroll
    for (int o = kGroupLanes / 2; o > 0; o >>= 1)
        a = max_abs_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// silu(g) * u = g / (1 + e^-g) * u for a 16-bit g.  e^-g = 2^(-g L), L = log2(e) =
// H + R with H the leading bits of L, as many as make -g H exact in fp32 (13 beside
// fp16's 11, 16 beside bf16's 8): the exponential's argument carries no rounding error,
// which |g| would magnify.  2^(-g R) = 1 + y (+ y^2 / 2 in fp16), y = -g R ln 2: where the
// exponential counts, |y| is at most 4.2e-3 in fp16 and 4.3e-4 in bf16, and the terms left
// out 1.3e-8 and 9.2e-8 (where g is large and positive it is zero and the sum 1).
// The quotient is corrected like quant8's.
//
// From about g = -86.6 down the sum comes near the end of fp32's range, where its
// reciprocal would vanish, while u can still lift the result to any size.  kScale makes
// e^-g y overflow there, so that the result is NaN: a warp with Inf or NaN leaves the
// common path anyway (quant8), and takes silu_mul_deep for them.  Of 4096 x 17408: bf16
// 59.5 us as with neither, fp16 61.5 (59.4 without its y^2 / 2); 70.7 when every warp has
// such a gate (a test of each lane's gates instead cost every call 7 us).
template <bool kBf16>
__device__ __forceinline__ f2 silu_mul(f2 g, f2 u) {
    constexpr float kH = kBf16 ? 1.44268798828125f : 1.442626953125f;
    constexpr float kRLn2 = kBf16 ? 4.888495152e-06f : 4.719484150e-05f;
    constexpr float kScale = kBf16 ? 16384.f : 2048.f;
    const f2 t = mul2(g, both(-kH)), y = mul2(g, both(-kRLn2 * kScale));
    float e0, e1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(lo(t)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(hi(t)));
    const f2 e = pack(e0, e1);
    const f2 w = kBf16 ? both(-1.f / kScale)
                       : fma2(y, both(-0.5f / (kScale * kScale)), both(-1.f / kScale));
    const f2 s = fma2(e, both(-1.f), fma2(mul2(e, y), w, both(-1.f)));  // -(1 + e^-g)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(-lo(s)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(-hi(s)));
    const f2 r = pack(r0, r1), q = mul2(g, r);
    return mul2(fma2(fma2(s, q, g), r, q), u);
}
// The same where 1 + e^-g is e^-g to fp32's last bit: g p u p with p = e^(g/2), in an
// order that neither overflows nor underflows before the result does.  -Inf gives NaN,
// as the quotient does.
__device__ __forceinline__ f2 silu_mul_deep(f2 g, f2 u) {
    constexpr float kH = 1.442626953125f, kRLn2 = 4.719484150e-05f;
    const f2 t = mul2(g, both(0.5f * kH)), y = mul2(g, both(0.5f * kRLn2));
    float e0, e1;  // subnormal ones too
    asm("ex2.approx.f32 %0, %1;" : "=f"(e0) : "f"(lo(t)));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e1) : "f"(hi(t)));
    f2 p = pack(e0, e1);
    p = fma2(mul2(p, y), fma2(y, both(0.5f), both(1.f)), p);
    return mul2(mul2(mul2(g, p), u), p);
}
// v where it is a number, else d
__device__ __forceinline__ f2 number_or(f2 v, f2 d) {
    return pack(isnan(lo(v)) ? lo(d) : lo(v), isnan(hi(v)) ? hi(d) : hi(v));
}

// A lane's 8 elements of its group -> 8 codes of row q and, from the group's
// first lane, the group's scale.  All lanes of the warp call it together.  Where one of
// the warp's elements is Inf or NaN, `again` may first compute them another way.
template <bool kVec, bool kStaged, typename Again>
__device__ __forceinline__ void quant8(f2 (&v)[4], uint8_t *q, float *scale, int c, int n,
                                       uint16_t *stage, Again again) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max_abs_nan(max_abs_nan(a, lo(v[i])), hi(v[i]));
    a = group_max(a);
    if (__any_sync(0xffffffffu, !(a <= FLT_MAX))) {
        // an Inf or NaN in one of the warp's groups: make it NaN, and the largest
        // magnitude that of the others
        again(v);
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = add2(v[i], add2(v[i], neg2(v[i])));
            a = fmaxf(fmaxf(a, fabsf(lo(v[i]))), fabsf(hi(v[i])));  // fmaxf passes over NaN
        }
        a = group_max(a);
    }
    const float s = __fdiv_rn(fmaxf(a, kScaleFloor), kE4m3Max);
    const f2 r = both(__frcp_rn(s)), ns = both(-s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 q0 = mul2(v[i], r);
        v[i] = fma2(fma2(q0, ns, v[i]), r, q0);
    }
    if (c < n && c % kGroup == 0) *scale = s;
    const uint32_t c0 = e4m3x2(lo(v[0]), hi(v[0])) | e4m3x2(lo(v[1]), hi(v[1])) << 16;
    const uint32_t c1 = e4m3x2(lo(v[2]), hi(v[2])) | e4m3x2(lo(v[3]), hi(v[3])) << 16;
    if constexpr (kVec) {
        if (c < n) *reinterpret_cast<uint2 *>(q + c) = make_uint2(c0, c1);
    } else {
        const int e = neighbour(c);
        uint8_t *own = reinterpret_cast<uint8_t *>(group_stage(stage));
        if constexpr (kStaged) {
            *reinterpret_cast<uint2 *>(own + c % kGroup) = make_uint2(c0, c1);
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kLaneElems; ++i)
            if (e + kGroupLanes * i < n)
                q[e + kGroupLanes * i] = kStaged ? own[e % kGroup + kGroupLanes * i]
                                                 : (uint8_t)((i < 4 ? c0 : c1) >> (8 * (i & 3)));
        if constexpr (kStaged) __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// rmsnorm: a CTA per row, V steps of 8 elements per thread, the row in
// registers between the sum of squares and the outputs (one pass over memory).
// Bound by memory: 8192 rows of 5120 with the residual's sum, bf16 to 8 bits, take
// 43.7 us (6.75 TB/s, 99% of the measured copy rate; 45.7 with scalar arithmetic);
// rows of 5119, in 2-byte accesses, 110 us (142 with a lane's own elements in turn).
// ---------------------------------------------------------------------------
template <bool kBf16, bool kVec, int V>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a) {
    __shared__ float warp_sums[32];
    __shared__ __align__(16) uint16_t stages[kVec ? 8 : 32 * kStageWarp];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint16_t *stage = stages + (kVec ? 0 : warp * kStageWarp);
    const size_t row = blockIdx.x;
    const uint16_t *x = a.x + row * a.H;
    chain_start();
    f2 h[V][4], sums = both(0.f);
#pragma unroll
    for (int s = 0; s < V; ++s) {
        const int c = (s * (int)blockDim.x + (int)threadIdx.x) * kLaneElems;
        load8<kBf16, kVec, true>(x, c, a.H, h[s], stage);
        if (a.residual) {
            f2 r[4];
            load8<kBf16, kVec, true>(a.residual + row * a.H, c, a.H, r, stage);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[s][i] = add2(h[s][i], r[i]);
        }
    }
#pragma unroll
    for (int s = 0; s < V; ++s) {
        const int c = (s * (int)blockDim.x + (int)threadIdx.x) * kLaneElems;
        if (a.sum_out) store8<kBf16, kVec>(a.sum_out + row * a.H, c, a.H, h[s], stage);
#pragma unroll
        for (int i = 0; i < 4; ++i) sums = fma2(h[s][i], h[s][i], sums);
    }
    float sum = lo(sums) + hi(sums);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) warp_sums[warp] = sum;
    __syncthreads();
    // every warp adds the warps' sums in the same tree
    sum = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, (float)a.H) + a.eps));
#pragma unroll
    for (int s = 0; s < V; ++s) {
        const int c = (s * (int)blockDim.x + (int)threadIdx.x) * kLaneElems;
        f2 w[4];  // every row's: it comes from L1 or L2
        load8<kBf16, kVec, true>(a.weight, c, a.H, w, stage);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[s][i] = mul2(mul2(h[s][i], both(rstd)), w[i]);
        if (a.y) store8<kBf16, kVec>(a.y + row * a.H, c, a.H, h[s], stage);
        if (a.q)
            quant8<kVec, true>(h[s], a.q + row * a.H,
                         a.scales + row * ((a.H + kGroup - 1) / kGroup) + c / kGroup, c, a.H,
                         stage, [](f2 (&)[4]) {});
    }
}

// ---------------------------------------------------------------------------
// quant: 16 lanes per (row, group), two groups each, both loaded before either is
// computed; a CTA has 16 consecutive groups of a row.  Bound by memory: silu-and-mul
// of 4096 x 17408 takes 57.6 us (6.23 TB/s, 92% of the measured copy rate; with scalar
// arithmetic 60.3, then 67.1 with 256 threads and one group each, 63.9 with 256 and
// two); of 4096 x 17405, in 2-byte accesses, 90 us (104 with a lane's own elements in
// turn).
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 128;
constexpr int kQuantU = 2;

template <bool kBf16, bool kVec, bool kSilu>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(QuantArgs a) {
    constexpr int U = kQuantU;
    chain_start();
    const size_t row = blockIdx.y;
    const uint16_t *x = a.x + row * (kSilu ? 2 * (size_t)a.N : (size_t)a.N);
    const int first = (int)(blockIdx.x * U * kQuantThreads + threadIdx.x) * kLaneElems;
    f2 v[U][4], u[U][4];
#pragma unroll
    for (int s = 0; s < U; ++s) {  // all loads, then the arithmetic
        const int c = first + s * kQuantThreads * kLaneElems;
        load8<kBf16, kVec, false>(x, c, a.N, v[s], nullptr);
        if constexpr (kSilu) load8<kBf16, kVec, false>(x + a.N, c, a.N, u[s], nullptr);
    }
#pragma unroll
    for (int s = 0; s < U; ++s) {
        const int c = first + s * kQuantThreads * kLaneElems;
        if constexpr (kSilu) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[s][i] = silu_mul<kBf16>(v[s][i], u[s][i]);
        }
        // gates far below zero: their rows once more, from the cache
        auto again = [&](f2 (&w)[4]) {
            if constexpr (kSilu) {
                f2 g[4], up[4];
                load8<kBf16, kVec, false>(x, c, a.N, g, nullptr);
                load8<kBf16, kVec, false>(x + a.N, c, a.N, up, nullptr);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = number_or(w[i], silu_mul_deep(g[i], up[i]));
            }
        };
        quant8<kVec, false>(v[s], a.q + row * a.N, a.scales + row * a.G + c / kGroup, c, a.N,
                            nullptr, again);
    }
}

cudaLaunchConfig_t chained(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

template <bool kBf16, bool kVec>
cudaError_t launch_norm_v(const NormArgs &a, int steps, int threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = chained(dim3(a.M), threads, stream, attr);
    switch (steps) {
        case 1: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kBf16, kVec, 1>, a);
        case 2: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kBf16, kVec, 2>, a);
        default: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kBf16, kVec, 4>, a);
    }
}

template <bool kBf16, bool kVec>
cudaError_t launch_quant_v(const QuantArgs &a, bool silu, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    constexpr int per = kQuantThreads * kLaneElems * kQuantU;
    const cudaLaunchConfig_t cfg =
        chained(dim3((a.N + per - 1) / per, a.M), kQuantThreads, stream, attr);
    return silu ? cudaLaunchKernelEx(&cfg, quant_kernel<kBf16, kVec, true>, a)
                : cudaLaunchKernelEx(&cfg, quant_kernel<kBf16, kVec, false>, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, bool bf16, cudaStream_t stream) {
    const bool vec = a.H % kLaneElems == 0 && aligned16(a.x) && aligned16(a.residual) &&
                     aligned16(a.weight) && aligned16(a.sum_out) && aligned16(a.y) &&
                     aligned16(a.q);
    const int lanes = (a.H + kLaneElems - 1) / kLaneElems;
    // up to four steps per thread before more than 128 threads: small CTAs keep more
    // rows in flight (8192 rows of 5120, with scalar arithmetic: 61.3 us in one step,
    // 49.1 in two, 45.7 in four; of 2048: 23.7 in one step, 19.9 in two)
    int steps = 1;
    while (steps < 4 && lanes > 128 * steps) steps *= 2;
    const int threads = ((lanes + steps - 1) / steps + 31) / 32 * 32;
    if (vec) return bf16 ? launch_norm_v<true, true>(a, steps, threads, stream)
                         : launch_norm_v<false, true>(a, steps, threads, stream);
    return bf16 ? launch_norm_v<true, false>(a, steps, threads, stream)
                : launch_norm_v<false, false>(a, steps, threads, stream);
}

cudaError_t launch_quant(const QuantArgs &a, bool bf16, bool silu, cudaStream_t stream) {
    const bool vec = a.N % kLaneElems == 0 && aligned16(a.x) && aligned16(a.q);
    if (vec) return bf16 ? launch_quant_v<true, true>(a, silu, stream)
                         : launch_quant_v<false, true>(a, silu, stream);
    return bf16 ? launch_quant_v<true, false>(a, silu, stream)
                : launch_quant_v<false, false>(a, silu, stream);
}

}  // namespace w4a16
