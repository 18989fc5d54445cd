// zdmmv_kv.cuh -- the paged 4-bit key/value cache's layout (include/zdmmv.h,
// zdmmv_kv_cache) for the kernels that write and read it, and the launch helper
// of the attention half's kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "zdmmv.h"
#include "zdmmv_device.cuh"
#include "zdmmv_internal.h"

namespace zdmmv {

constexpr int kKvSlab = 16;  // tokens of a tile: the k extent of one m16n8k16 for the product with V

// Words that a lane of a tile holds side by side: a token's words of W blocks are
// read and written as one 128-, 64- or 32-bit access.
template <int NB> struct KvGeom {
    static constexpr int kDim = NB * kQK;
    static constexpr int kVec = NB % 4 == 0 ? 4 : (NB % 2 == 0 ? 2 : 1);
    static constexpr int kCodeBytes = 8 * kDim;   // K (or V) codes of a tile
    static constexpr int kScaleBytes = kDim;      // K (or V) scales of a tile
    static constexpr int kTileBytes = 18 * kDim;  // K codes, V codes, K scales, V scales
    static constexpr int kVAt = kCodeBytes, kKScaleAt = 2 * kCodeBytes, kVScaleAt = 2 * kCodeBytes + kScaleBytes;
    // word of token r's 8 codes of block b, dimensions 8t .. 8t+7
    __host__ __device__ static constexpr int k_word(int r, int b, int t) {
        return (((r >> 3) * (NB / kVec) + b / kVec) * 32 + (r & 7) * 4 + t) * kVec + b % kVec;
    }
    // 16-bit half of token r's 4 V codes of block b, dimensions 4g .. 4g+3
    __host__ __device__ static constexpr int v_half(int r, int b, int g) {
        return ((((r >> 3) * (NB / kVec) + b / kVec) * 32 + g * 4 + ((r & 7) >> 1)) * kVec + b % kVec) * 2 + (r & 1);
    }
    // fp16 number of token r's scale of block b
    __host__ __device__ static constexpr int scale_half(int r, int b) { return ((r >> 1) * NB + b) * 2 + (r & 1); }
};

// n / d and n % d for 0 <= n < 2^31 by a multiplication: q = n * ceil(2^p / d) >> p with p = 31 + ceil(log2 d), exact
// there (the product's error is below n / 2^p <= 1 / d).
struct FastDiv {
    uint32_t d, m, p;
    __host__ static FastDiv of(int32_t d) {
        FastDiv f{static_cast<uint32_t>(d), 0, 31};
        while ((1ull << (f.p - 31)) < f.d) ++f.p;
        f.m = static_cast<uint32_t>(((1ull << f.p) + f.d - 1) / f.d);
        return f;
    }
    __device__ __forceinline__ int div(int n) const {
        return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> p);
    }
    __device__ __forceinline__ int mod(int n, int q) const { return n - q * static_cast<int>(d); }
};

// The cache's fields that the kernels take.
struct KvView {
    uint8_t *pages;
    const int32_t *table;
    int64_t n_pages;
    int64_t page_bytes;
    int32_t n_seq, max_pages, page_tokens, n_kv_heads;
};

// Blocks of a head of a supported dimension, else 0.
int kv_blocks(int head_dim);
// The cache's argument checks (a status of zdmmv.h), and its view.
zdmmv_status kv_check(const zdmmv_kv_cache *c, KvView *out);

inline bool kv_misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// One launch with the programmatic-dependent-launch attribute (unless ZDMMV_PDL=0).
// Every kernel launched so waits (griddepcontrol.wait) before it reads or writes
// global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_block_op(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                            Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Raises KERNEL's dynamic shared-memory limit to the device's, once per device.
template <auto KERNEL> cudaError_t smem_limit_raised() {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = raise_dynamic_smem_limit(reinterpret_cast<const void *>(KERNEL), dev);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

__device__ __forceinline__ void block_op_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void block_op_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace zdmmv
