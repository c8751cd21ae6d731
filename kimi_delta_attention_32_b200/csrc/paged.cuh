// paged.cuh -- device helpers of the calls on the paged key-value cache.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "launchers.h"

namespace kda {

// Bit of the device error word: a length or page number read on the device is out of range.
constexpr unsigned int kErrIndex = 2u;

// A length read on the device, clamped to [0, most].
__device__ __forceinline__ int checked_len(int len, int most, unsigned int* err) {
    if (len >= 0 && len <= most) return len;
    atomicOr(err, kErrIndex);
    return len < 0 ? 0 : most;
}

// Element offset of (slot, head 0) of sequence n in the K and V pages, -1 when the page number is
// out of range. The slot must be below max_pages * page_size.
__device__ __forceinline__ int64_t slot_offset(const PagedCache& c, int64_t n, int slot) {
    const int page = __ldg(c.block_table + n * c.max_pages + slot / c.page_size);
    if (page < 0 || page >= c.num_pages) {
        atomicOr(c.err, kErrIndex);
        return -1;
    }
    return page * c.page_stride + (slot % c.page_size) * c.slot_stride;
}

// Programmatic dependent launch: a kernel launched with launch_after may start while the one before
// it on the stream ends; it waits here until that one has finished and its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// SMs of the current device (0 if the query fails).
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
}

// Launches a kernel that begins with grid_wait().
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Before every launch: what is set belongs to the current context (0.05 us).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace kda
