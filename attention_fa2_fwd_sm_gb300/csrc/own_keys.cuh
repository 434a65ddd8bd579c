// own_keys.cuh -- the numbering of the sequences' own cached keys by which the
// kernels of the shared-prefix decode share them out (own_keys_sm103.cu has the
// first of them, and why).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "attn_internal.h"

namespace attn {

namespace own {

// Keys: two warps of a stage.  A step of 8 KV heads of 64 keys, of 300, of 3000: with 32
// 9.6, 9.6, 11.6 us, with 64 11.0, 9.6, 10.3, with 128 13.7, 10.3, 11.0.
constexpr int kMinShare = 32;

__device__ __forceinline__ int length_of(const int *seqlens, int max_seqlen, int b) {
    return min(max(seqlens[b], 0), max_seqlen);
}

// A place in the numbering, and what is left of a share from there.
struct Place {
    int b, g, j, len;
    long long left;
    __device__ __forceinline__ int keys() const { return int(min((long long)(len - j), left)); }
    // To the segment behind this one; call only while something is left.
    __device__ __forceinline__ void next(const int *seqlens, int max_seqlen, int Hkv) {
        j = 0;
        if (++g < Hkv) return;
        g = 0;
        do {
            len = length_of(seqlens, max_seqlen, ++b);
        } while (len == 0);
    }
};

__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)(unsigned(a) / unsigned(b)) : a / b;
}

}  // namespace own
}  // namespace attn
