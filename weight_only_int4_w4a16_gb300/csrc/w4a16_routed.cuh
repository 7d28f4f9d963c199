// Shared by the products whose weights a row chooses (layers of 8-bit experts, low-rank
// adapters): asynchronous copies, the warp MMA, and the grouping of rows by what they chose.
#pragma once

#include "w4a16_fp8_common.cuh"

namespace w4a16 {
namespace routed {

__device__ __forceinline__ uint32_t smem_of(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes to shared memory, the first n from memory, the others zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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
                 : "r"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint16_t lds16(uint32_t p) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t p, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(v) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
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
// what follows may start (the next kernel's CTAs), and what came before has ended
__device__ __forceinline__ void launch_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_last() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- rows by bin, in one CTA ------------------------------------------------------
constexpr int kMaxBins = 1025;
template <int kRows>
struct RowSort {  // space that is free again afterwards
    uint16_t bin[kRows];
    uint8_t rank[kRows];                    // among the equal bins of the row's 32
    uint16_t before[kMaxBins + 1];          // rows of lower bins
    unsigned sums[32];
    uint16_t count[kRows / 32 * kMaxBins + 1];  // [32 rows][bin]
};

// order: the rows s < n (n <= kRows) by bin_of(s) in [0, bins), stable, those outside left
// out.  pack(bin, n) is a bin's n rows in its low 11 bits and counts of what the caller cuts
// them into above; emit(bin, n, at) gets each bin that has rows and the sum of the packs of
// the lower ones, done(total) the sum of all, before the last emit or after.  Up to 32 rows
// are one warp's work.
template <int kCta, int kRows, typename BinOf, typename Pack, typename Emit, typename Done>
__device__ void group_rows(RowSort<kRows> &sp, uint16_t *order, int n, int bins, BinOf bin_of,
                           Pack pack, Emit emit, Done done) {
    constexpr int kCtaWarps = kCta / 32;
    constexpr int kBinsPerThread = (kMaxBins + kCta - 1) / kCta;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n <= 32) {
        if (warp == 0) {
            int b = lane < n ? bin_of(lane) : -1;
            if ((unsigned)b >= (unsigned)bins) b = bins;  // sorts behind all
            int place = 0, rows = 0;
            bool first = true;
            for (int j = 0; j < n; ++j) {
                const int o = __shfl_sync(0xffffffffu, b, j);
                place += o < b || (o == b && j < lane);
                rows += o == b;
                first = first && !(o == b && j < lane);
            }
            const bool lead = first && b < bins && lane < n;
            const unsigned own = lead ? pack(b, rows) : 0u;
            unsigned at = 0, total = 0;
            for (int j = 0; j < n; ++j) {
                const int o = __shfl_sync(0xffffffffu, b, j);
                const unsigned v = __shfl_sync(0xffffffffu, own, j);
                at += o < b ? v : 0u;
                total += v;
            }
            if (b < bins) order[place] = (uint16_t)lane;
            if (lead) emit(b, rows, at);
            if (lane == 0) done(total);
        }
        __syncthreads();
        return;
    }
    const int chunks = (n + 31) / 32;
    // (the bins first, all rows' loads under way at once)
#pragma unroll 4
    for (int s = tid; s < chunks * 32; s += kCta) {
        const int b = s < n ? bin_of(s) : -1;
        sp.bin[s] = (uint16_t)((unsigned)b < (unsigned)bins ? b : 0xffff);
    }
    for (int i = tid; i < (chunks * bins + 1) / 2; i += kCta)
        reinterpret_cast<uint32_t *>(sp.count)[i] = 0;
    __syncthreads();
    for (int c = warp; c < chunks; c += kCtaWarps) {
        const int s = c * 32 + lane, b = sp.bin[s];
        const unsigned same = __match_any_sync(0xffffffffu, b);
        const int rank = __popc(same & ((1u << lane) - 1));
        sp.rank[s] = (uint8_t)rank;
        if (b != 0xffff && rank == 0) sp.count[c * bins + b] = (uint16_t)__popc(same);
    }
    __syncthreads();
    // neighbouring bins per thread: the counts of 32 rows each become what lies before
    // them, and the bins' packs are added up over the threads
    int rows[kBinsPerThread];
    unsigned own = 0;
    const int per = (bins + kCta - 1) / kCta;
#pragma unroll
    for (int i = 0; i < kBinsPerThread; ++i) {
        const int b = per * tid + i;
        rows[i] = 0;
        if (i < per && b < bins) {
            for (int c = 0; c < chunks; ++c) {
                const int v = sp.count[c * bins + b];
                sp.count[c * bins + b] = (uint16_t)rows[i];
                rows[i] += v;
            }
            own += pack(b, rows[i]);
        }
    }
    unsigned incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sp.sums[warp] = incl;
    __syncthreads();
    unsigned at = incl - own, total = 0;
#pragma unroll
    for (int w = 0; w < kCtaWarps; ++w) {
        const unsigned v = sp.sums[w];
        if (w < warp) at += v;
        total += v;
    }
    if (tid == 0) done(total);
#pragma unroll
    for (int i = 0; i < kBinsPerThread; ++i) {
        const int b = per * tid + i;
        if (i < per && b < bins) {
            sp.before[b] = (uint16_t)(at & 2047);
            if (rows[i] > 0) emit(b, rows[i], at);
            at += pack(b, rows[i]);
        }
    }
    __syncthreads();
    for (int s = tid; s < n; s += kCta) {
        const int b = sp.bin[s];
        if (b != 0xffff)
            order[sp.before[b] + sp.count[s / 32 * bins + b] + sp.rank[s]] = (uint16_t)s;
    }
    __syncthreads();
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster,
                           cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace routed
}  // namespace w4a16
