// decode_prefix_sm103.cu -- decode for a batch whose sequences share a prefix,
// and decode that accumulates the attention weight of every cached key.
//
// Each sequence b attends the P keys of the prefix (one copy per KV head for
// the whole batch) and the len_b keys of its own cache:
//     s_j = scale <q, k_j>,  L = log sum_j exp(s_j),  o = sum_j exp(s_j - L) v_j,
//     weights[b, g, j] += sum over the group's heads of exp(s_j - L)  (own keys).
// Softmax partials over disjoint sets of keys merge exactly: (o_i, L_i) give
// L = log sum_i exp(L_i) and o = sum_i exp(L_i - L) o_i.  So three kernels:
//
//   1. Prefix: fwd_kernel<D, kMapPrefix> (fwd_kernel.cuh).  For one KV head the
//      B * G query rows are a matrix, and S = Q K^T and P V are matrix products
//      whose keys are read once for the whole batch: tcgen05, 128 rows a tile
//      whatever B * G is, since even a tile of one row outruns HBM.  Shares of
//      key blocks as in prefix_order.cuh.
//   2. Own keys: decode_kernel<D, S, true> (decode_kernel.cuh), HBM-bound; with
//      weights it also writes the scores (4 G bytes a key beside 4 d read).
//      Launched programmatically, it fills SMs as the prefix's CTAs leave.
//   3. Finish: merges the partials of every row and, with weights, turns the
//      scores into weights now that L is known.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_kernel.cuh"
#include "fwd_kernel.cuh"
#include "prefix_order.cuh"

namespace attn {

namespace {

// Own keys: about 5/3 CTAs an SM in all and no chunk below kOwnMinChunk keys, as
// the ragged decode's plan.
constexpr int kOwnMinChunk = 512;
long long own_target(int sms) { return (5LL * sms) / 3 > 0 ? (5LL * sms) / 3 : 1; }

constexpr int kFinishThreads = 128;
constexpr int kWeightKeys = 1024;  // keys of one finishing CTA

struct FinishParams {
    const int *plan;  // null: no own keys
    const float *own_o, *own_lse, *pre_o, *pre_lse, *scores;
    __nv_bfloat16 *o;
    float *lse, *weights;
    int B, Hq, Hkv, G, P, max_seqlen, subs;
    PrefixOrder po;
};

// The partials of row (b, h): those of the prefix, then those of b's own items.
struct RowParts {
    const float *pre, *own;  // log-sum-exps, log2 units
    size_t pre_stride, own_stride;
    int n_pre, n;
    __device__ __forceinline__ float lse(int i) const {
        return i < n_pre ? pre[i * pre_stride] : own[(i - n_pre) * own_stride];
    }
};

__device__ __forceinline__ RowParts row_parts(const FinishParams &p, int b, int h) {
    RowParts r;
    r.n_pre = r.n = 0;
    r.pre_stride = (size_t)p.B * p.Hq;
    r.own_stride = p.Hq;
    r.pre = p.pre_lse + (size_t)b * p.Hq + h;
    r.own = p.own_lse + h;
    if (p.P > 0) r.n = r.n_pre = prefix_parts(p.po, prefix_row(p.po, h / p.G, b / p.po.rb / 2));
    if (p.plan) {
        r.own += (size_t)p.plan[2 + b] * p.Hq;
        r.n += p.plan[2 + p.B + b];
    }
    return r;
}

// Maximum and sum of 2^(lse_i - maximum) over a row's partials, by one warp;
// w0 is 2^(lse_lane - maximum).
__device__ __forceinline__ void warp_total(const RowParts &r, int lane, float &top, float &sum, float &w0) {
    const float l0 = lane < r.n ? r.lse(lane) : -INFINITY;
    top = l0;
    for (int i = lane + 32; i < r.n; i += 32) top = fmaxf(top, r.lse(i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float ref = top == -INFINITY ? 0.f : top;
    sum = w0 = fast_exp2(l0 - ref);
    for (int i = lane + 32; i < r.n; i += 32) sum += fast_exp2(r.lse(i) - ref);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
}

template <int kCols>
struct Cols {
    float v[kCols];
};
template <int kCols>
__device__ __forceinline__ Cols<kCols> load_cols(const float *p) {
    Cols<kCols> c;
    if constexpr (kCols == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        c.v[0] = x.x, c.v[1] = x.y, c.v[2] = x.z, c.v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        c.v[0] = x.x, c.v[1] = x.y;
    }
    return c;
}

// Grid: first the rows (b, h), each by kWarps warps of a CTA; then, with
// weights, a CTA for every 1024 keys of every own item of every KV head.
// A row's chain is what bounds the merge: its counts, then its partials' L, then
// their outputs.  The outputs do not depend on the L's, so the first eight of
// each warp are loaded before L is known.  One warp a row when there are rows
// enough to fill the GPU with; four take turns of eight partials when not.
template <int D, int kWarps>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const FinishParams p) {
    constexpr int kCols = D / 32;  // columns of a lane
    constexpr int kAhead = 8;
    __shared__ float acc_sh[kWarps > 1 ? kFinishThreads / 32 : 1][D];
    __shared__ float lse_sh[dec::kMaxGroup];
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.B * p.Hq;
    constexpr int kRows = kFinishThreads / 32 / kWarps;
    const int row_ctas = (rows + kRows - 1) / kRows;
    if (int(blockIdx.x) < row_ctas) {
        const int row = blockIdx.x * kRows + warp / kWarps, q = warp % kWarps;
        if (row >= rows) return;  // with kWarps > 1 a CTA is one row
        const int b = row / p.Hq, h = row - b * p.Hq;
        const RowParts r = row_parts(p, b, h);
        const size_t pre_step = (size_t)rows * D, own_step = (size_t)p.Hq * D;
        const float *pre = p.pre_o + (size_t)row * D + lane * kCols;
        const float *own = p.own_o + (p.plan ? ((size_t)p.plan[2 + b] * p.Hq + h) * D : 0) + lane * kCols;
        auto part = [&](int i) { return i < r.n_pre ? pre + i * pre_step : own + (i - r.n_pre) * own_step; };
        Cols<kCols> v[kAhead];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < r.n) v[k] = load_cols<kCols>(part(i0 + k));
        };
        fetch(q * kAhead);
        float top, sum, w0;
        warp_total(r, lane, top, sum, w0);
        float acc[kCols] = {};
        for (int i0 = q * kAhead; i0 < r.n; i0 += kAhead * kWarps) {
            if (i0 > q * kAhead) fetch(i0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k;
                float w = __shfl_sync(0xffffffffu, w0, i & 31);
                if (i < r.n) {
                    if (i >= 32) w = fast_exp2(r.lse(i) - (top == -INFINITY ? 0.f : top));
                    if (w != 0.f)  // an empty partial adds nothing
#pragma unroll
                        for (int c = 0; c < kCols; ++c) acc[c] += w * v[k].v[c];
                }
            }
        }
        if constexpr (kWarps > 1) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc_sh[warp][lane * kCols + c] = acc[c];
            __syncthreads();
            if (warp > 0) return;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                for (int w = 1; w < kWarps; ++w) acc[c] += acc_sh[w][lane * kCols + c];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
        uint32_t packed[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) packed[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
        __nv_bfloat16 *o = p.o + (size_t)row * D + lane * kCols;
        if constexpr (kCols == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(packed[0], packed[1]);
        else *reinterpret_cast<uint32_t *>(o) = packed[0];
        if (lane == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        return;
    }
    // ------------------------------------------------------------- weights
    int i = int(blockIdx.x) - row_ctas;
    const int sub = i % p.subs;
    i /= p.subs;
    const int g = i % p.Hkv, item = i / p.Hkv;
    if (item >= p.plan[0]) return;
    const int *it = p.plan + dec::plan_items_offset(p.B) + 3 * item;
    const int b = it[0], lo = it[1] + sub * kWeightKeys, hi = min(it[2], lo + kWeightKeys);
    if (lo >= hi) return;
    for (int h = warp; h < p.G; h += kFinishThreads / 32) {
        float top, sum, w0;
        warp_total(row_parts(p, b, g * p.G + h), lane, top, sum, w0);
        if (lane == 0) lse_sh[h] = top + log2f(sum);
    }
    __syncthreads();
    const size_t base = (size_t)(b * p.Hkv + g) * p.max_seqlen;
    constexpr int kKeys = 4;  // keys of a thread in flight
    for (int j0 = lo + threadIdx.x; j0 < hi; j0 += kKeys * kFinishThreads) {
        float old[kKeys], w[kKeys] = {};
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const int j = j0 + k * kFinishThreads;
            if (j < hi) old[k] = p.weights[base + j];
        }
        if (p.G % 4 == 0) {
            for (int h = 0; h < p.G; h += 4) {
                float4 x[kKeys];
#pragma unroll
                for (int k = 0; k < kKeys; ++k) {
                    const int j = j0 + k * kFinishThreads;
                    if (j < hi) x[k] = __ldcs(reinterpret_cast<const float4 *>(p.scores + (base + j) * p.G + h));
                }
#pragma unroll
                for (int k = 0; k < kKeys; ++k)
                    if (j0 + k * kFinishThreads < hi)
                        w[k] += (fast_exp2(x[k].x - lse_sh[h]) + fast_exp2(x[k].y - lse_sh[h + 1])) +
                                (fast_exp2(x[k].z - lse_sh[h + 2]) + fast_exp2(x[k].w - lse_sh[h + 3]));
            }
        } else {
            for (int h = 0; h < p.G; ++h)
#pragma unroll
                for (int k = 0; k < kKeys; ++k) {
                    const int j = j0 + k * kFinishThreads;
                    if (j < hi) w[k] += fast_exp2(p.scores[(base + j) * p.G + h] - lse_sh[h]);
                }
        }
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const int j = j0 + k * kFinishThreads;
            if (j < hi) p.weights[base + j] = old[k] + w[k];
        }
    }
}

template <int D>
int launch_prefix(const DecodePrefixLaunch &a, const PrefixOrder &po, float *part_o, float *part_lse,
                  cudaStream_t stream) {
    using C = fwd::Cfg<D>;
    CUtensorMap mq, mk, mv;
    const int G = a.Hq / a.Hkv;
    if (!encode_bf16_3d(&mq, a.q, D, uint64_t(a.Hq), uint64_t(a.B), 64, uint32_t(G), uint32_t(po.rb)) ||
        !encode_bf16_3d(&mk, a.kprefix, D, uint64_t(a.P), uint64_t(a.Hkv), 64, fwd::kBlockN) ||
        !encode_bf16_3d(&mv, a.vprefix, D, uint64_t(a.P), uint64_t(a.Hkv), 64, fwd::kBlockN))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (shared prefix)");
    fwd::PrefixParams p = {};
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.po = po;
    p.B = a.B;
    p.N = a.P;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = G;
    p.d_store = D;
    p.order = kNaiveHeadFirst;  // the segments are fixed by the block index: no work counter
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    auto kernel = fwd::fwd_kernel<D, fwd::kMapPrefix>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncGetAttributes(fwd_kernel, prefix)");
        if (fa.numRegs != fwd::kLaunchRegs || fa.maxThreadsPerBlock < fwd::kThreads)
            return note_cuda_error(cudaErrorInvalidConfiguration,
                                   "fwd_kernel (prefix) register count differs from the setmaxnreg split");
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes + fwd::kTurnBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(fwd_kernel, prefix)");
        if (dev >= 0) attr_set[dev] = true;
    }
    kernel<<<dim3(unsigned(po.grid)), dim3(fwd::kThreads), C::kSmemBytes + fwd::kTurnBytes, stream>>>(mq, mk, mv, p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "fwd_kernel (prefix) launch");
}

template <int D>
int launch_own(const DecodePrefixLaunch &a, const PrefixLayout &l, bool behind_prefix, cudaStream_t stream) {
    constexpr int S = dec::kBaseStages<D>;
    using C = dec::Cfg<D, S>;
    CUtensorMap mk, mv;
    const uint64_t planes = uint64_t(a.B) * a.Hkv;
    if (!encode_bf16_3d(&mk, a.kcache, D, uint64_t(a.max_seqlen), planes, 64, dec::kKeysPerStage) ||
        !encode_bf16_3d(&mv, a.vcache, D, uint64_t(a.max_seqlen), planes, 64, dec::kKeysPerStage))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (own keys)");
    dec::OwnParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.seqlens = a.seqlens;
    p.ws_o = reinterpret_cast<float *>(a.workspace + l.own_o);
    p.ws_lse = reinterpret_cast<float *>(a.workspace + l.own_lse);
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.max_seqlen = a.max_seqlen;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    p.plan_out = reinterpret_cast<int *>(a.workspace + l.plan);
    p.scores = a.weights ? reinterpret_cast<float *>(a.workspace + l.scores) : nullptr;
    p.target = own_target(a.num_sms);
    p.min_chunk = kOwnMinChunk;
    auto kernel = dec::decode_kernel<D, S, true>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(decode_kernel, own keys)");
        if (dev >= 0) attr_set[dev] = true;
    }
    const dim3 grid(unsigned(a.Hkv), unsigned(l.own_items), 1);
    cudaError_t e;
    if (behind_prefix) {
        e = dec::launch_programmatic(kernel, grid, dim3(dec::kThreads), C::kSmemBytes, stream, mk, mv, p);
    } else {
        kernel<<<grid, dim3(dec::kThreads), C::kSmemBytes, stream>>>(mk, mv, p);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? 0 : note_cuda_error(e, "decode_kernel launch (own keys)");
}

// Longest chunk that own_item can choose for these sizes.
long long own_max_chunk(int B, int Hkv, int max_seqlen, int sms) {
    const long long t = own_target(sms);
    long long c = ((long long)B * max_seqlen * Hkv + t - 1) / t;
    c = (c + dec::kChunkGranule - 1) / dec::kChunkGranule * dec::kChunkGranule;
    if (c < kOwnMinChunk) c = kOwnMinChunk;
    return c < max_seqlen ? c : max_seqlen;
}

template <int D>
int launch_all(const DecodePrefixLaunch &a, cudaStream_t stream) {
    PrefixLayout l;
    FinishParams f = {};
    const int G = a.Hq / a.Hkv;
    if (!decode_prefix_layout(a.B, a.Hq, a.Hkv, a.P, a.d, a.max_seqlen, a.weights != nullptr, a.num_sms, &l))
        return ATTN_ERR_ARG;
    float *pre_o = reinterpret_cast<float *>(a.workspace + l.pre_o);
    float *pre_lse = reinterpret_cast<float *>(a.workspace + l.pre_lse);
    // Four warps a row while a warp a row would leave SMs short of two CTAs.
    const long long rows = (long long)a.B * a.Hq;
    const bool wide = rows < 8LL * a.num_sms;
    long long grid = wide ? rows : (rows + kFinishThreads / 32 - 1) / (kFinishThreads / 32);
    if (a.weights) {
        f.subs = int((own_max_chunk(a.B, a.Hkv, a.max_seqlen, a.num_sms) + kWeightKeys - 1) / kWeightKeys);
        grid += (long long)l.own_items * a.Hkv * f.subs;
    }
    if (grid > 0x7fffffffLL) return ATTN_ERR_ARG;  // before anything is launched
    if (a.P > 0) {
        prefix_order(&f.po, a.B, G, a.Hkv, a.P, a.num_sms);
        const int rc = launch_prefix<D>(a, f.po, pre_o, pre_lse, stream);
        if (rc) return rc;
    }
    if (a.max_seqlen > 0) {
        const int rc = launch_own<D>(a, l, a.P > 0, stream);
        if (rc) return rc;
        f.plan = reinterpret_cast<const int *>(a.workspace + l.plan);
    }
    f.own_o = reinterpret_cast<const float *>(a.workspace + l.own_o);
    f.own_lse = reinterpret_cast<const float *>(a.workspace + l.own_lse);
    f.pre_o = pre_o;
    f.pre_lse = pre_lse;
    f.scores = reinterpret_cast<const float *>(a.workspace + l.scores);
    f.o = static_cast<__nv_bfloat16 *>(a.o);
    f.lse = a.lse;
    f.weights = a.weights;
    f.B = a.B;
    f.Hq = a.Hq;
    f.Hkv = a.Hkv;
    f.G = G;
    f.P = a.P;
    f.max_seqlen = a.max_seqlen;
    auto finish = wide ? finish_kernel<D, kFinishThreads / 32> : finish_kernel<D, 1>;
    const cudaError_t e = dec::launch_programmatic(finish, dim3(unsigned(grid)), dim3(kFinishThreads), 0,
                                                   stream, f);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "finish_kernel launch");
}

}  // namespace

bool decode_prefix_layout(int B, int Hq, int Hkv, int P, int d, int max_seqlen, bool weights, int num_sms,
                          PrefixLayout *l) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)B * Hq;
    PrefixOrder po = {};
    if (P > 0 && !prefix_order(&po, B, Hq / Hkv, Hkv, P, num_sms)) return false;
    const long long items = max_seqlen > 0 ? (own_target(num_sms) + Hkv - 1) / Hkv + B : 0;
    if (items > 65535) return false;  // grid.y of the own keys' launch
    l->own_items = int(items);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += up(n);
        return here;
    };
    l->plan = take(items ? (size_t)(2 + 2LL * B + 3 * items) * sizeof(int) : 0);
    l->own_o = take((size_t)items * Hq * d * sizeof(float));
    l->own_lse = take((size_t)items * Hq * sizeof(float));
    l->pre_o = take((size_t)po.slots * rows * d * sizeof(float));
    l->pre_lse = take((size_t)po.slots * rows * sizeof(float));
    l->scores = take(weights ? rows * max_seqlen * sizeof(float) : 0);
    l->bytes = at;
    return true;
}

int decode_prefix_launch(const DecodePrefixLaunch &a, cudaStream_t stream) {
    return a.d == 64 ? launch_all<64>(a, stream) : launch_all<128>(a, stream);
}

cudaError_t decode_prefix_take_status(int *bits) {
    int zero = 0, fwd_bits = 0, dec_bits = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&fwd_bits, g_fwd_status, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&dec_bits, g_decode_status, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_fwd_status, &zero, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_decode_status, &zero, sizeof(int));
    *bits = fwd_bits | dec_bits;
    return e;
}

}  // namespace attn
