// The choice of experts: for each row of a router's logits the k largest in falling
// order (equal ones by index) and their weights,
//
//   p = softmax(row) or 1 / (1 + e^-logit),  weight = scale * p (/ sum of the chosen p)
//
// (forum.sourcefind.cn thread "vLLM on Hygon Z100", section 七: a router picks k of E
// experts per token, whose outputs are summed with the router's weights.)
//
// A NaN counts as -Inf; the p of -Inf is 0, so a switched-off expert that has to be
// chosen all the same weighs nothing; the p of equal +Inf are equal shares (softmax) or
// 1.  Everything is fp32: the exponentials' arguments are differences to the row's
// largest, and the sums are over p of at most 1.  Sigmoids that are renormalised count in
// units of e^top where the row's largest is negative, so that their shares outlive their p;
// below l = -745, where binary64 has no e^l either, p is 0.
//
// A warp has a row, each lane every 32nd logit as an integer key that orders as the number
// does (in registers up to 256 logits a row, in local memory above).  A step finds the largest
// key and the lowest index that holds it (two warp-wide integer reductions), and its lane
// strikes it out.  8192 rows of 256 logits, k 8, take 9.1 us in a row in a graph (their 8.9 MB
// would take 1.3): 829 instructions a row, 5.4 us if every cycle issued one; 61% do, and the
// others wait for the half-rate integer pipe, for fixed latencies and for the logits, in about
// equal parts.  One row takes 2.1, a launch.  (Holders by a vote, with the second reduction
// only for ties: 10.2.)
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kKeyMinusInf = 0x007fffffu;  // the key of -Inf; struck out or no logit: 0

__device__ __forceinline__ uint32_t key_of(float v) {
    v = isnan(v) ? -INFINITY : v + 0.f;  // -0 counts as +0
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <int kType>
__device__ __forceinline__ float load_logit(const void *row, size_t i) {
    if constexpr (kType == kLogitsF32) return static_cast<const float *>(row)[i];
    const uint16_t h = static_cast<const uint16_t *>(row)[i];
    if constexpr (kType == kDtypeBf16) return __uint_as_float((uint32_t)h << 16);
    else return __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// e^(v - top) with top the row's largest: 1 for the largest itself, which may be
// infinite, and 0 for -Inf
__device__ __forceinline__ float share(uint32_t key, uint32_t top) {
    if (key <= kKeyMinusInf) return 0.f;
    return key == top ? 1.f : expf(value_of(key) - value_of(top));
}

// 1 / (1 + e^-v) in units of e^unit (unit <= 0, and v <= unit where v is negative): e^(v - unit)
// / (1 + e^v) there
__device__ __forceinline__ float sigmoid(float v, float unit) {
    if (v >= 0.f) return 1.f / (1.f + expf(-v));
    return v > -745.f ? expf(v - unit) / (1.f + expf(v)) : 0.f;
}

template <int kType, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= a.T) return;
    uint32_t key[V], most = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < a.E ? key_of(load_logit<kType>(a.logits, (size_t)t * a.E + e)) : 0u;
        most = max(most, key[i]);
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, most);
    float total = 1.f;  // of all p; where the weights are renormalised it would cancel
    if (!a.sigmoid && !a.renormalize) {
        total = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) total += share(key[i], top);
        total = warp_sum(total);
    }
    uint32_t mine = 0;  // lane j: the j-th choice
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, most);
        unsigned at = ~0u;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == m) at = lane + 32 * i;
        at = __reduce_min_sync(0xffffffffu, at);
        if (lane == j) mine = m, chosen = (int)at;
        if (lane == (int)(at & 31)) {
            most = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i == (int)(at >> 5)) key[i] = 0;
                most = max(most, key[i]);
            }
        }
    }
    float p = 0.f;
    if (lane < a.k && mine > kKeyMinusInf)
        p = a.sigmoid ? sigmoid(value_of(mine), a.renormalize ? fminf(value_of(top), 0.f) : 0.f)
                      : share(mine, top) / total;
    if (a.renormalize) {
        const float sum = warp_sum(p);
        p = sum > 0.f ? p / sum : 0.f;
    }
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = chosen;
        a.weights[(size_t)t * a.k + lane] = p * a.scale;
    }
}

template <int kType, int V>
cudaError_t launch(const RouteArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.T + kRouteWarps - 1) / kRouteWarps);
    cfg.blockDim = dim3(kRouteWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel<kType, V>, a);
}

template <int kType>
cudaError_t launch_type(const RouteArgs &a, cudaStream_t stream) {
    if (a.E <= 64) return launch<kType, 2>(a, stream);
    if (a.E <= 128) return launch<kType, 4>(a, stream);
    if (a.E <= 256) return launch<kType, 8>(a, stream);
    if (a.E <= 512) return launch<kType, 16>(a, stream);
    return launch<kType, 32>(a, stream);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, int type, cudaStream_t stream) {
    switch (type) {
        case kLogitsF32: return launch_type<kLogitsF32>(a, stream);
        case kDtypeBf16: return launch_type<kDtypeBf16>(a, stream);
        default: return launch_type<kDtypeF16>(a, stream);
    }
}

}  // namespace w4a16
