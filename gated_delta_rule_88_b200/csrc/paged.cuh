// paged.cuh -- device helpers of the paged latent cache's kernels.
#pragma once

#include "common.cuh"

namespace kda {
namespace paged {

// Error word code of a bad page, length or offset of the latent cache
// (kda_get_device_error); a bad page of kda_pages_* is kErrBadSlot.
constexpr int kErrBadPage = 5;

// Offset i of a sequence's new tokens, i <= N: cu[i] clamped to the token
// axis, or i * per without offsets.
__device__ __forceinline__ int token_offset(const int32_t *cu, int i, int per, int T) {
    return cu ? min(max(cu[i], 0), T) : i * per;
}

// The sequence of token t (N if it lies behind the last one), by one warp:
// a 32-way search for the number of offsets cu[1..N] that are <= t (offsets
// do not decrease).  Every lane gets the result.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int per, int T, int t) {
    if (!cu) return t / per;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = N;                       // the answer lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;      // probes at the ends of 32 pieces
        const int at = lo + min(n, (lane + 1) * step);
        const bool below = lane * step < n && min(max(cu[at], 0), T) <= t;
        const int full = __popc(__ballot_sync(0xffffffffu, below));    // leading pieces wholly below
        const int skip = min(n, full * step);
        lo += skip;
        n = min(n - skip, step - 1);
    }
    return lo;
}

// Programmatic dependent launch: the second kernel of a pair is launched while
// the first still runs (launch_after, once the first's blocks have all called
// let_next_start or ended) and waits with wait_for_previous for its end and its
// writes, so that only the launch itself overlaps.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace paged
}  // namespace kda
