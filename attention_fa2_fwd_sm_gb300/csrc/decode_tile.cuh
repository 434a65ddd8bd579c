// decode_tile.cuh -- what the decode kernels share: the stage of 64 keys, the
// matrix instructions on it, and the programmatic launch.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "sm103_ptx.cuh"

namespace attn {
namespace dec {

constexpr int kKeysPerStage = 64;
constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr int kMaxGroup = 16;
constexpr int kChunkGranule = 64;

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                        uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                          uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// Byte address of the 16-byte unit `u` (elements 8u..8u+7) of key row `k` of a
// 64-key tile stored as D/64 chunks of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_unit_addr(uint32_t tile, int k, int u) {
    return tile + (u >> 3) * (kKeysPerStage * 128) + k * 128 + (((u & 7) ^ (k & 7)) << 4);
}

// Zero the bf16 halves of a V fragment register whose keys lie at or beyond
// `n_valid` (keys k_lo and k_lo + 1 live in the low and high halves).
__device__ __forceinline__ uint32_t mask_pair(uint32_t r, int k_lo, int n_valid) {
    if (k_lo >= n_valid) r &= 0xffff0000u;
    if (k_lo + 1 >= n_valid) r &= 0x0000ffffu;
    return r;
}

// Launch `kernel` allowing it to start before the grid ahead of it on the
// stream has finished (it must griddep_wait() before reading that grid's
// output).
template <typename... KArgs, typename... Args>
cudaError_t launch_programmatic(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dec
}  // namespace attn
