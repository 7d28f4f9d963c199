// The expired-wait path, exercised on purpose: one thread runs the bounded
// waits the warp-MMA kernels use (a completion counter that must reach a
// target, an mbarrier phase) on a counter nothing increments and an mbarrier
// nothing arrives at.  Each wait gives up after its time limit.  A second warp
// waits for an mbarrier that is arrived at, goes on, and learns at the barrier
// where the 8-bit linear's sum warps agree (barrier_all) that the first has
// given up; it reports the mbarrier wait.  Reports are ORed into the library's
// device status word, as by an expired wait in a production kernel; nothing
// faults, traps or hangs, and the context stays usable.  Given an arrival
// counter, the probe first increments it: what a split launch cut short by an
// expired wait can leave behind (an arrival counted, its block never reduced),
// so that a test can check that the report of the expiry also clears such
// counters.
#include <cuda.h>

#include "w4a16_internal.h"
#include "w4a16_mma_common.cuh"
#include "w4a16_tcgen05.cuh"

namespace w4a16 {
namespace {

using namespace warp_mma;

__device__ unsigned g_never_incremented;  // zero for the life of the module

constexpr int kProbeThreads = 64;

__global__ void __launch_bounds__(kProbeThreads) wait_probe_kernel(int *status, unsigned *stale) {
    __shared__ __align__(8) uint64_t bars[2];  // nothing arrives at the first
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        if (stale) atomicAdd(stale, 1u);
        for (int i = 0; i < 2; ++i) mbar_init(dev::smem_u32(bars + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        dev::mbar_arrive(dev::smem_u32(bars + 1));
        if (!wait_counter(&g_never_incremented, 1u)) atomicOr(status, kErrProbeCounterWait);
    }
    __syncthreads();
    const bool met = mbar_wait(dev::smem_u32(bars + warp), 0);
    const bool all = dev::barrier_all(1, kProbeThreads, met);
    if (met && !all && threadIdx.x == 32) atomicOr(status, kErrProbeBarrierWait);
}

}  // namespace

cudaError_t launch_wait_probe(int *status, unsigned *stale, cudaStream_t stream) {
    wait_probe_kernel<<<1, kProbeThreads, 0, stream>>>(status, stale);
    return cudaGetLastError();
}

}  // namespace w4a16
