// decode_sm103.cu -- split-KV grouped-query decode (one query row per query
// head) and the log-sum-exp merge of the per-split partial states.
//
// kernbench2 "Fused Grouped-Query Attention": a decode step processes a
// single query position against the whole KV history, so its time is the
// time to stream the KV cache from HBM; each KV head is shared by a group of
// G query heads; the KV sequence is split and the running softmax states
// (m, l, O) of the pieces are reduced (section "Inference with Long-Context
// Length", Case 4).  Here the pieces are CTAs of one GPU and the reduction is
// a second kernel.
//
// The decode kernel itself is in decode_kernel.cuh.
//
// Ragged multi-user batches (attn_decode_varlen): one chunk size for the whole
// batch, chosen on the device from the total number of cached keys, cuts every
// sequence into chunks; a plan kernel writes the resulting work list (batch
// entry, key range) and each decode CTA takes one item of it, so a long
// sequence is spread over many CTAs however short the others are.  The
// reduction then has two levels, as in the kernbench2 decode family's
// multi-user "two-level reduce-to-root" (short-context section): the warps of
// a CTA are combined in shared memory, and one merge per (user, query head)
// reduces that user's chunks.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "attn_internal.h"
#include "decode_kernel.cuh"
#include "sm103_ptx.cuh"

namespace attn {

// Built-in scratch for attn_decode_noalloc: the split partials of callers
// that cannot hand the library a workspace.  A fixed-size array that is part
// of the library image, so every GPU that loads the library holds it until
// the process exits.  Host code must not use the symbol itself as a pointer
// (on the host it names a stand-in, not device memory); decode_noalloc_scratch
// looks up the real device address.
static __device__ __align__(256) unsigned char g_decode_noalloc_scratch[kDecodeNoAllocScratchBytes];

namespace dec {

// Merge: L = max_s lse_s, w_s = exp(lse_s - L), O = sum_s w_s O_s / sum_s w_s.
// The block stages the lse values in shared memory (one load per thread) and
// issues the partial outputs eight splits at a time, so the merge costs a few
// memory round trips instead of one per split; the sums run over s in order.
template <int D>
__global__ void __launch_bounds__(D) merge_kernel(const float *ws_o, const float *ws_lse,
                                                  __nv_bfloat16 *o, int num_splits) {
    __shared__ float lse_sh[kDecodeMaxSplits];
    __shared__ float max_sh[D / 32];
    griddep_wait();  // launched behind the decode grid, which writes the partials
    const int bh = blockIdx.x, col = threadIdx.x;
    const float *lse = ws_lse + (size_t)bh * num_splits;
    const float *po = ws_o + (size_t)bh * num_splits * D;
    float L = -INFINITY;
    for (int s = col; s < num_splits; s += D) {
        const float v = lse[s];
        lse_sh[s] = v;
        L = fmaxf(L, v);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, off));
    if ((col & 31) == 0) max_sh[col >> 5] = L;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) L = fmaxf(L, max_sh[w]);
    float wsum = 0.f, acc = 0.f;
    if (L != -INFINITY) {
        int s = 0;
        for (; s + 8 <= num_splits; s += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = po[(size_t)(s + i) * D + col];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = __expf(lse_sh[s + i] - L);
                wsum += w;
                acc += w * v[i];
            }
        }
        for (; s < num_splits; ++s) {
            const float w = __expf(lse_sh[s] - L);
            wsum += w;
            acc += w * po[(size_t)s * D + col];
        }
    }
    o[(size_t)bh * D + col] = __float2bfloat16_rn(wsum > 0.f ? acc / wsum : 0.f);
}

// Varlen plan, one CTA: total keys T = sum_b min(max(seqlens[b], 0), max_seqlen);
// chunk C = max(min_chunk, ceil(T * Hkv / target) rounded up to 64); sequence
// b gets n_b = ceil(len_b / C) items [c C, min(c C + C, len_b)), numbered
// consecutively by b.  The item count is at most ceil(target / Hkv) + B.
__global__ void __launch_bounds__(256) varlen_plan_kernel(const int *seqlens, int B, int max_seqlen, int Hkv,
                                                          long long target, int min_chunk, int *plan) {
    __shared__ long long warp_part[8];
    __shared__ int chunk_s;
    griddep_launch_dependents();  // the decode grid may be scheduled; it waits for this one
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int per = (B + 255) / 256;  // consecutive sequences per thread
    const int b0 = min(t * per, B), b1 = min(b0 + per, B);
    auto len_of = [&](int b) {
        const int n = seqlens[b];
        return n < 0 ? 0 : (n > max_seqlen ? max_seqlen : n);
    };
    // Inclusive block scan of one value per thread (warp shuffles, then the
    // eight warp totals); returns the thread's exclusive prefix and the total.
    auto block_scan = [&](long long v, long long &total) {
        long long x = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        __syncthreads();
        if (lane == 31) warp_part[w] = x;
        __syncthreads();
        long long before = 0;
        total = 0;
        for (int i = 0; i < 8; ++i) {
            if (i < w) before += warp_part[i];
            total += warp_part[i];
        }
        return before + x - v;
    };
    long long keys = 0;
    for (int b = b0; b < b1; ++b) keys += len_of(b);
    long long T = 0;
    block_scan(keys, T);
    if (t == 0) {
        long long c = (T * Hkv + target - 1) / target;
        c = (c + kChunkGranule - 1) / kChunkGranule * kChunkGranule;
        if (c < min_chunk) c = min_chunk;
        chunk_s = int(c < 0x40000000LL ? c : 0x40000000LL);
        plan[1] = chunk_s;
    }
    __syncthreads();
    const int C = chunk_s;
    long long mine = 0;  // items of this thread's sequences
    for (int b = b0; b < b1; ++b) mine += (len_of(b) + C - 1) / C;
    long long count = 0;
    int first = int(block_scan(mine, count));
    if (t == 0) plan[0] = int(count);
    int *items = plan + plan_items_offset(B);
    for (int b = b0; b < b1; ++b) {
        const int len = len_of(b);
        const int n = (len + C - 1) / C;
        plan[2 + b] = first;
        plan[2 + B + b] = n;
        for (int c = 0; c < n; ++c) {
            int *it = items + 3 * (first + c);
            it[0] = b;
            it[1] = c * C;
            it[2] = min(c * C + C, len);
        }
        first += n;
    }
}

// Varlen merge: for (b, h), the n_b partials of b's items.  n_b = 0 gives O = 0.
template <int D>
__global__ void __launch_bounds__(D) merge_varlen_kernel(const int *plan, int B, int Hq, const float *ws_o,
                                                         const float *ws_lse, __nv_bfloat16 *o) {
    griddep_wait();  // launched behind the decode grid, which writes the partials
    const int bh = blockIdx.x, col = threadIdx.x;
    const int b = bh / Hq, h = bh % Hq;
    const int f = plan[2 + b], n = plan[2 + B + b];
    float L = -INFINITY;
    for (int s = f; s < f + n; ++s) L = fmaxf(L, ws_lse[(size_t)s * Hq + h]);
    float wsum = 0.f, acc = 0.f;
    if (L != -INFINITY) {
        for (int s = f; s < f + n; ++s) {
            const float w = __expf(ws_lse[(size_t)s * Hq + h] - L);
            wsum += w;
            acc += w * ws_o[((size_t)s * Hq + h) * D + col];
        }
    }
    o[(size_t)bh * D + col] = __float2bfloat16_rn(wsum > 0.f ? acc / wsum : 0.f);
}

template <int D, int S>
int launch(const DecodeLaunch &a, cudaStream_t stream) {
    using C = Cfg<D, S>;
    CUtensorMap mk, mv;
    if (!encode_bf16_3d(&mk, a.kcache, D, uint64_t(a.max_seqlen), uint64_t(a.B) * a.Hkv, 64,
                        kKeysPerStage) ||
        !encode_bf16_3d(&mv, a.vcache, D, uint64_t(a.max_seqlen), uint64_t(a.B) * a.Hkv, 64,
                        kKeysPerStage))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (decode)");
    Params p;
    p.q = reinterpret_cast<const __nv_bfloat16 *>(a.q);
    p.seqlens = a.seqlens;
    p.o = reinterpret_cast<__nv_bfloat16 *>(a.o);
    p.ws_o = a.ws_o;
    p.ws_lse = a.ws_lse;
    p.plan = a.plan;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.max_seqlen = a.max_seqlen;
    p.num_splits = a.num_splits;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    static bool attr_set[kMaxDevices] = {};  // per instantiation and device
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(
            decode_kernel<D, S, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(decode_kernel)");
        if (dev >= 0) attr_set[dev] = true;
    }
    // The kernels after the first are launched with programmatic stream
    // serialization: each may be scheduled while the one ahead drains and
    // waits (griddep_wait) for it before touching its output.
    if (a.plan) {
        varlen_plan_kernel<<<1, 256, 0, stream>>>(a.seqlens, a.B, a.max_seqlen, a.Hkv, a.varlen_target,
                                                  a.varlen_min_chunk, a.plan);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return note_cuda_error(e, "varlen_plan_kernel launch");
        e = launch_programmatic(decode_kernel<D, S, false>, dim3(a.Hkv, a.varlen_max_items, 1), dim3(kThreads),
                                C::kSmemBytes, stream, mk, mv, p);
        if (e != cudaSuccess) return note_cuda_error(e, "decode_kernel launch (varlen)");
        e = launch_programmatic(merge_varlen_kernel<D>, dim3(a.B * a.Hq), dim3(D), 0, stream,
                                (const int *)a.plan, a.B, a.Hq, (const float *)a.ws_o, (const float *)a.ws_lse, p.o);
        return e == cudaSuccess ? 0 : note_cuda_error(e, "merge_varlen_kernel launch");
    }
    decode_kernel<D, S, false><<<dim3(a.num_splits, a.Hkv, a.B), dim3(kThreads), C::kSmemBytes, stream>>>(mk, mv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return note_cuda_error(e, "decode_kernel launch");
    if (a.num_splits > 1) {
        e = launch_programmatic(merge_kernel<D>, dim3(a.B * a.Hq), dim3(D), 0, stream, (const float *)a.ws_o,
                                (const float *)a.ws_lse, p.o, a.num_splits);
        if (e != cudaSuccess) return note_cuda_error(e, "merge_kernel launch");
    }
    return 0;
}

}  // namespace dec

int decode_launch(const DecodeLaunch &a, cudaStream_t stream) {
    // The split grid of at most one CTA per SM runs the deep ring; the varlen
    // grid (an upper bound on its work items) keeps the base ring.
    const bool deep = !a.plan && a.num_sms > 0 && (long long)a.num_splits * a.Hkv * a.B <= a.num_sms;
    if (a.d == 64) return dec::launch<64, dec::kBaseStages<64>>(a, stream);
    return deep ? dec::launch<128, dec::kDeepStages<128>>(a, stream)
                : dec::launch<128, dec::kBaseStages<128>>(a, stream);
}

cudaError_t decode_noalloc_scratch(void **ptr) {
    // One lookup per device, made with that device current; later calls reuse it.
    static void *addr[kMaxDevices] = {nullptr};
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_decode_noalloc_scratch);
        if (e != cudaSuccess) return e;
        addr[dev] = p;
    }
    *ptr = addr[dev];
    return cudaSuccess;
}

cudaError_t decode_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_decode_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_decode_status, &zero, sizeof(int));
}

}  // namespace attn
