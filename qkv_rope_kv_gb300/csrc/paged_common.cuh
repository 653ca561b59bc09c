// What the paged-cache kernels share: the view of the cache that a launch carries,
// slot addressing, and each file's device status word (see qkv_check_device_error).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qkv_internal.h"

namespace qkv_paged {

constexpr unsigned int kFlagSlotRange = 1u;  // a slot outside the sequence's capacity
constexpr unsigned int kFlagIndexRange = 4u; // a page id, length or sequence index out of range

static __device__ unsigned int g_paged_status[2];  // [0] flags, [1] a bad value
static std::atomic<bool> g_launched{false};        // whether this process launched any of this file's kernels

__device__ __forceinline__ void flag_bad(unsigned int bit, int value) {
    atomicOr(&g_paged_status[0], bit);
    atomicExch(&g_paged_status[1], static_cast<unsigned int>(value));
}

// A slot's page and its row there; a table entry is asked for here and looked at by row_offset(), so that
// several can be in flight together.
struct PageRef {
    int id, in_page;
};
__device__ __forceinline__ PageRef page_ref(const PagedView& c, int seq, int slot) {
    const int pg = slot / c.page_size;
    return {c.table[static_cast<int64_t>(seq) * c.max_pages + pg], slot - pg * c.page_size};
}
// Element offset of the slot's row in the pools, or -1 (and the status flag) where the table names a page
// that is not there.  64-bit: a pool can hold more than 2^31 elements.
__device__ __forceinline__ int64_t row_offset(const PagedView& c, PageRef r) {
    if (static_cast<unsigned int>(r.id) >= static_cast<unsigned int>(c.n_pages)) {
        flag_bad(kFlagIndexRange, r.id);
        return -1;
    }
    return r.id * c.page_stride + static_cast<int64_t>(r.in_page) * c.nkt;
}

__device__ __forceinline__ int64_t row_offset(const PagedView& c, int seq, int slot) {
    return row_offset(c, page_ref(c, seq, slot));
}

// Ask for the line that holds *p.  Only L2 takes it, so this may come before what writes there has ended.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Length of sequence b, or 0 (and the status flag) where it is outside [0, capacity].
__device__ __forceinline__ int checked_len(const PagedView& c, const int32_t* lens, int b) {
    const int n = lens[b];
    if (n < 0 || n > c.max_pages * c.page_size) {
        flag_bad(kFlagIndexRange, n);
        return 0;
    }
    return n;
}

constexpr int kSms = 152;  // of a GB300: grids are sized for them

// Launch after the stream's previous kernel as a programmatic dependent (the blocks are set up while that
// one drains, and wait for it, griddep_wait, before they read anything), in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
static inline cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                                           cudaStream_t stream, int cluster, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned int>(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    g_launched.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Read and clear this file's status word (synchronises the stream); nothing has set it where nothing was launched.
static inline cudaError_t status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    if (!g_launched.load(std::memory_order_relaxed)) return cudaSuccess;
    unsigned int h[2] = {0u, 0u};
    cudaError_t e = cudaMemcpyFromSymbolAsync(h, g_paged_status, sizeof(h), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    if (h[0] != 0u) {
        const unsigned int zero[2] = {0u, 0u};
        e = cudaMemcpyToSymbolAsync(g_paged_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
        if (e != cudaSuccess) return e;
        *flags |= h[0];
        *bad = static_cast<int32_t>(h[1]);
    }
    return cudaSuccess;
}

}  // namespace qkv_paged
