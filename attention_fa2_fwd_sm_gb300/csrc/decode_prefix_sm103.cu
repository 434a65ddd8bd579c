// decode_prefix_sm103.cu -- decode for a batch whose sequences share a prefix,
// and decode that accumulates the attention weight of every cached key.
//
// Each sequence b attends the P keys of the prefix (one copy per KV head for
// the whole batch) and the len_b keys of its own cache:
//     s_j = scale <q, k_j>,  L = log sum_j exp(s_j),  o = sum_j exp(s_j - L) v_j,
//     weights[b, g, j] += sum over the group's heads of exp(s_j - L)  (own keys).
// Softmax partials over disjoint sets of keys merge exactly: (o_i, L_i) give
// L = log sum_i exp(L_i) and o = sum_i exp(L_i - L) o_i.  So three kernels, or four:
//
//   1. Prefix: fwd_kernel<D, kMapPrefix> (fwd_kernel.cuh).  For one KV head the
//      B * G query rows are a matrix, and S = Q K^T and P V are matrix products
//      whose keys are read once for the whole batch: tcgen05, 128 rows a tile
//      whatever B * G is, since even a tile of one row outruns HBM.  Shares of
//      key blocks as in prefix_order.cuh.
//   2. Own keys: own_kernel (own_keys_sm103.cu), HBM-bound; with weights it also
//      writes the scores (4 G bytes a key beside 4 d read).
//      It is launched first, on some of the SMs, and the prefix's kernel
//      programmatically behind it, so that both run at once: the one waits for
//      memory, the other for the tensor cores.
//   3. Merge: the partials of every row.
//   4. With weights: the scores become weights now that L is known.
// 128 sequences, 32K shared + 512 .. 1024 own keys, 64 heads, 8 KV heads, d = 128: 137 to
// 142 us, where the prefix alone takes 100 (1370 TFLOP/s) and the own keys alone 72; 32
// with 8K + 256 .. 512: 28 to 37 by the GPU, alone 22 and 18, with weights 43.  32 of 8K to
// 16K own keys, no prefix: 227 us, with weights 281.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_tile.cuh"
#include "fwd_kernel.cuh"
#include "own_keys.cuh"
#include "prefix_order.cuh"

namespace attn {

namespace {

constexpr int kMergeThreads = 128, kWeightThreads = 256;
constexpr int kWeightCtasPerSm = 8;  // (4 to 12: the same within 2 %; 16: 5 % slower)
// Of one CTA.  A step of one sequence of 8K keys, of 8 of 1000, of 64 of 300: with 64
// keys 17.8, 17.2, 27.1 us, with 256 16.4, 15.8, 25.1, with 1024 16.5, 16.4, 27.0.
constexpr int kMinWeightKeys = 256;

struct MergeParams {
    const int2 *own_rows;  // own_keys.cuh; null: no own keys
    const int *seqlens;
    const float *own_o, *own_lse, *pre_o, *pre_lse;
    __nv_bfloat16 *o;
    float *lse, *row_lse;  // natural log, and log2 units for the weights; either may be null
    const int2 *pre_rows;  // null: no prefix
    int B, Hq, Hkv, G;
    PrefixOrder po;
};

struct WeightParams {
    const long long *plan;
    const int *seqlens;
    const float *scores, *row_lse;
    float *weights;
    int B, Hkv, G, max_seqlen;
};

// The partials of row (b, h): those of the prefix, then those of b's own keys.
struct RowParts {
    size_t pre, own;  // row of the first one in each array of partials
    int pre_stride, own_stride, n_pre, n;
    __device__ __forceinline__ size_t row(int i) const {
        return i < n_pre ? pre + (size_t)i * pre_stride : own + (size_t)(i - n_pre) * own_stride;
    }
};

// Where to find the two, from the indices alone.
struct RowPlace {
    int b, j, pre_row, own_row;
    size_t pre;
};

__device__ __forceinline__ RowPlace row_place(const MergeParams &p, int row) {
    RowPlace r;
    r.b = row / p.Hq;
    const int h = row - r.b * p.Hq, g = h / p.G;
    r.j = h - g * p.G;
    r.own_row = r.b * p.Hkv + g;
    r.pre = r.pre_row = 0;
    if (p.pre_rows) {
        const int m = r.b / p.po.rb / 2;
        r.pre_row = prefix_row(p.po, g, m);
        // In lockstep the units of a partial number lie one behind the other.
        r.pre = (size_t)(r.b - (p.po.lockstep ? 0 : 2 * m * p.po.rb)) * p.G + r.j;
    }
    return r;
}

__device__ __forceinline__ RowParts row_parts(const MergeParams &p, const RowPlace &at) {
    RowParts r = {};
    int2 pre = make_int2(0, 0), own = pre;
    if (p.pre_rows) pre = p.pre_rows[at.pre_row];
    if (p.own_rows) {
        own = p.own_rows[at.own_row];  // not written for a sequence without keys
        if (p.seqlens[at.b] <= 0) own = make_int2(0, 0);
    }
    r.pre_stride = p.po.id_rows;
    r.own_stride = p.G;
    r.pre = at.pre + (size_t)pre.x * p.po.id_rows;
    r.own = (size_t)own.x * p.G + at.j;
    r.n_pre = pre.y;
    r.n = pre.y + own.y;
    return r;
}

// Maximum and sum of 2^(lse_i - maximum) over a row's partials, by one warp;
// w0 is 2^(lse_lane - maximum).
template <typename Lse>
__device__ __forceinline__ void warp_total(const RowParts &r, Lse lse, int lane, float &top, float &sum, float &w0) {
    const float l0 = lane < r.n ? lse(lane) : -INFINITY;
    top = l0;
    for (int i = lane + 32; i < r.n; i += 32) top = fmaxf(top, lse(i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float ref = top == -INFINITY ? 0.f : top;
    sum = w0 = fast_exp2(l0 - ref);
    for (int i = lane + 32; i < r.n; i += 32) sum += fast_exp2(lse(i) - ref);
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

// A row (b, h) by kWarps warps of a CTA.  A row's chain is what bounds the merge:
// its counts, then its partials' L, then their outputs.  The outputs do not depend
// on the L's, so the first kAhead of each warp are loaded before L is known, and
// what follows from the indices alone is done before the wait.
template <int D, int kWarps, int kAhead>
__global__ void __launch_bounds__(kWarps > 1 ? kWarps * 32 : kMergeThreads) merge_kernel(const MergeParams p) {
    constexpr int kCols = D / 32;  // columns of a lane
    __shared__ float acc_sh[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = p.B * p.Hq;
    constexpr int kRows = kWarps > 1 ? 1 : kMergeThreads / 32;
    const int row = blockIdx.x * kRows + warp / kWarps, q = warp % kWarps;
    if (row >= rows) return;  // with kWarps > 1 a CTA is one row (no thread of it leaves)
    const RowPlace at = row_place(p, row);
    griddep_wait();
    const RowParts r = row_parts(p, at);
    auto part = [&](int i) { return (i < r.n_pre ? p.pre_o : p.own_o) + r.row(i) * D + lane * kCols; };
    auto lse = [&](int i) { return (i < r.n_pre ? p.pre_lse : p.own_lse)[r.row(i)]; };
    Cols<kCols> v[kAhead];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k < r.n) v[k] = load_cols<kCols>(part(i0 + k));
    };
    fetch(q * kAhead);
    float top, sum, w0;
    warp_total(r, lse, lane, top, sum, w0);
    float acc[kCols] = {};
    for (int i0 = q * kAhead; i0 < r.n; i0 += kAhead * kWarps) {
        if (i0 > q * kAhead) fetch(i0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k;
            float w = __shfl_sync(0xffffffffu, w0, i & 31);
            if (i < r.n) {
                if (i >= 32) w = fast_exp2(lse(i) - (top == -INFINITY ? 0.f : top));
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
        const int used = min(kWarps, (r.n + kAhead - 1) / kAhead);  // warps that had a partial
        for (int w = 1; w < used; ++w)
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[c] += acc_sh[w][lane * kCols + c];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
    uint32_t packed[kCols / 2];
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) packed[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    __nv_bfloat16 *o = p.o + (size_t)row * D + lane * kCols;
    if constexpr (kCols == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t *>(o) = packed[0];
    if (lane == 0) {
        const float L = sum == 0.f ? -INFINITY : top + log2f(sum);
        if (p.lse) p.lse[row] = L * 0.69314718055994531f;
        if (p.row_lse) p.row_lse[row] = L;
    }
}

// What to subtract from a row's scores: a row whose scores are all -inf has no
// softmax, adds nothing, and leaves 2^(-inf - inf) = 0 instead of NaN.
__device__ __forceinline__ float weight_ref(float L) { return L == -INFINITY ? INFINITY : L; }

// The weights of n neighbouring keys of one KV head's row, G = 4 kQuads: a thread
// takes one float4 of a key's G scores (a warp's loads are 512 consecutive bytes)
// and kQuads neighbours add up.
template <int kQuads>
__device__ __forceinline__ void add_weights(const float *scores, const float *lse, float *weights, int n) {
    constexpr int kBatch = 8, kStep = kWeightThreads / kQuads;
    const int quad = threadIdx.x % kQuads, key0 = threadIdx.x / kQuads;
    const float4 *src = reinterpret_cast<const float4 *>(scores) + quad;
    const float L[4] = {weight_ref(lse[4 * quad]), weight_ref(lse[4 * quad + 1]), weight_ref(lse[4 * quad + 2]),
                        weight_ref(lse[4 * quad + 3])};
    for (int j0 = 0; j0 < n; j0 += kBatch * kStep) {
        float4 x[kBatch];
        float old[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int j = j0 + key0 + k * kStep;
            if (j < n) {
                x[k] = __ldcs(src + (size_t)j * kQuads);
                if (quad == 0) old[k] = weights[j];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int j = j0 + key0 + k * kStep;
            float w = 0.f;
            if (j < n)
                w = (fast_exp2(x[k].x - L[0]) + fast_exp2(x[k].y - L[1])) +
                    (fast_exp2(x[k].z - L[2]) + fast_exp2(x[k].w - L[3]));
#pragma unroll
            for (int off = 1; off < kQuads; off <<= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
            if (j < n && quad == 0) weights[j] = old[k] + w;
        }
    }
}

// CTAs with equal shares of the own keys in the numbering of own_keys.cuh.
// Bound by the scores' traffic (4 G bytes a key, most of it from L2).
// kQuads: G / 4 where that is a power of two, else 0.
template <int kQuads>
__global__ void __launch_bounds__(kWeightThreads) weight_kernel(const WeightParams p) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long total = p.plan[1];
    const long long share = max((long long)kMinWeightKeys, own::quotient(total + gridDim.x - 1, gridDim.x));
    const long long lo = blockIdx.x * share;
    if (lo >= total) return;
    // The last sequence that starts at or before lo (of several, the one with keys).
    int b = -1;
    for (int first = 0; first < p.B; first += 256) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = first + 32 * k + lane;
            n += __popc(__ballot_sync(0xffffffffu, i < p.B && p.plan[2 + i] <= lo));
        }
        b += n;
        if (n < 256) break;
    }
    own::Place at;
    const long long rem = lo - p.plan[2 + b];
    at.b = b;
    at.len = own::length_of(p.seqlens, p.max_seqlen, b);
    at.g = int(own::quotient(rem, at.len));
    at.j = int(rem - (long long)at.g * at.len);
    at.left = min(share, total - lo);
    while (true) {
        const int n = at.keys(), row = at.b * p.Hkv + at.g;
        const size_t key = (size_t)row * p.max_seqlen + at.j;
        const float *scores = p.scores + key * p.G, *lse = p.row_lse + (size_t)row * p.G;
        float *weights = p.weights + key;
        if constexpr (kQuads > 0)
            add_weights<kQuads>(scores, lse, weights, n);
        else
            for (int j = threadIdx.x; j < n; j += kWeightThreads) {
                float w = 0.f;
                for (int h = 0; h < p.G; ++h) w += fast_exp2(scores[(size_t)j * p.G + h] - weight_ref(lse[h]));
                weights[j] += w;
            }
        at.left -= n;
        if (at.left == 0) return;
        at.next(p.seqlens, p.max_seqlen, p.Hkv);
    }
}

template <int D>
int launch_prefix(const DecodePrefixLaunch &a, const PrefixLayout &l, const PrefixOrder &po, cudaStream_t stream) {
    using C = fwd::Cfg<D>;
    CUtensorMap mq, mk, mv;
    const int G = a.Hq / a.Hkv;
    if (!encode_bf16_3d(&mq, a.q, D, uint64_t(a.Hq), uint64_t(a.B), 64, uint32_t(G), uint32_t(po.rb)) ||
        !encode_bf16_3d(&mk, a.kprefix, D, uint64_t(a.P), uint64_t(a.Hkv), 64, fwd::kBlockN) ||
        !encode_bf16_3d(&mv, a.vprefix, D, uint64_t(a.P), uint64_t(a.Hkv), 64, fwd::kBlockN))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (shared prefix)");
    fwd::PrefixParams p = {};
    p.part_o = reinterpret_cast<float *>(a.workspace + l.pre_o);
    p.part_lse = reinterpret_cast<float *>(a.workspace + l.pre_lse);
    p.rows = reinterpret_cast<int2 *>(a.workspace + l.pre_rows);
    p.seqlens = a.max_seqlen > 0 ? a.seqlens : nullptr;
    p.max_seqlen = a.max_seqlen;
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
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes + fwd::kPrefixSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(fwd_kernel, prefix)");
        if (dev >= 0) attr_set[dev] = true;
    }
    const dim3 grid(unsigned(prefix_grid(po))), block(fwd::kThreads);
    constexpr size_t smem = C::kSmemBytes + fwd::kPrefixSmemBytes;
    cudaError_t e;
    if (a.max_seqlen > 0) {  // behind the own keys' kernel, beside it on the GPU
        e = dec::launch_programmatic(kernel, grid, block, smem, stream, mq, mk, mv, p);
    } else {
        kernel<<<grid, block, smem, stream>>>(mq, mk, mv, p);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? 0 : note_cuda_error(e, "fwd_kernel (prefix) launch");
}

template <int D>
int launch_all(const DecodePrefixLaunch &a, cudaStream_t stream) {
    PrefixLayout l;
    MergeParams m = {};
    const int G = a.Hq / a.Hkv;
    if (!decode_prefix_layout(a.B, a.Hq, a.Hkv, a.P, a.d, a.max_seqlen, a.weights != nullptr, a.num_sms, &l))
        return ATTN_ERR_ARG;
    if (a.max_seqlen > 0) {
        const int rc = own_launch(a, l, stream);
        if (rc) return rc;
        m.own_rows = reinterpret_cast<const int2 *>(a.workspace + l.own_rows);
        m.seqlens = a.seqlens;
    }
    if (a.P > 0) {
        prefix_order(&m.po, a.B, G, a.Hkv, a.P, a.d, a.max_seqlen, l.own_ctas, a.num_sms);
        const int rc = launch_prefix<D>(a, l, m.po, stream);
        if (rc) return rc;
        m.pre_rows = reinterpret_cast<const int2 *>(a.workspace + l.pre_rows);
    }
    m.own_o = reinterpret_cast<const float *>(a.workspace + l.own_o);
    m.own_lse = reinterpret_cast<const float *>(a.workspace + l.own_lse);
    m.pre_o = reinterpret_cast<const float *>(a.workspace + l.pre_o);
    m.pre_lse = reinterpret_cast<const float *>(a.workspace + l.pre_lse);
    m.o = static_cast<__nv_bfloat16 *>(a.o);
    m.lse = a.lse;
    m.row_lse = a.weights ? reinterpret_cast<float *>(a.workspace + l.row_lse) : nullptr;
    m.B = a.B;
    m.Hq = a.Hq;
    m.Hkv = a.Hkv;
    m.G = G;
    // Warps a row by what the rows leave of an SM's.  Whole calls, in us, by warps a
    // row (1, 2, 4, 16): 8192 rows 88, 91, 95, 141; 2048 rows with some 12 partials
    // 37, 36, 38, 49; 512 rows 18, 17, 16, 19; 64 rows with 57 partials 30, 22, 17, 12.
    const long long rows = (long long)a.B * a.Hq;
    const int warps = rows >= 24LL * a.num_sms ? 1 : rows >= 8LL * a.num_sms ? 2 : rows >= a.num_sms ? 4 : 16;
    auto merge = warps == 1   ? merge_kernel<D, 1, 8>
                 : warps == 2 ? merge_kernel<D, 2, 4>
                 : warps == 4 ? merge_kernel<D, 4, 4>
                              : merge_kernel<D, 16, 4>;
    const int per_cta = warps == 1 ? kMergeThreads / 32 : 1;
    cudaError_t e = dec::launch_programmatic(merge, dim3(unsigned((rows + per_cta - 1) / per_cta)),
                                             dim3(warps == 1 ? kMergeThreads : warps * 32), 0, stream, m);
    if (e != cudaSuccess) return note_cuda_error(e, "merge_kernel launch");
    if (!a.weights) return 0;
    WeightParams w = {};
    w.plan = reinterpret_cast<const long long *>(a.workspace + l.plan);
    w.seqlens = a.seqlens;
    w.scores = reinterpret_cast<const float *>(a.workspace + l.scores);
    w.row_lse = m.row_lse;
    w.weights = a.weights;
    w.B = a.B;
    w.Hkv = a.Hkv;
    w.G = G;
    w.max_seqlen = a.max_seqlen;
    const long long most = ((long long)a.B * a.Hkv * a.max_seqlen + kMinWeightKeys - 1) / kMinWeightKeys;
    const long long ctas = most < kWeightCtasPerSm * a.num_sms ? most : kWeightCtasPerSm * a.num_sms;
    auto weigh = G == 4 ? weight_kernel<1> : G == 8 ? weight_kernel<2> : G == 16 ? weight_kernel<4> : weight_kernel<0>;
    e = dec::launch_programmatic(weigh, dim3(unsigned(ctas)), dim3(kWeightThreads), 0, stream, w);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "weight_kernel launch");
}

}  // namespace

int own_ctas(int B, int G, int Hkv, int P, int d, int max_seqlen, int num_sms) {
    if (max_seqlen <= 0) return 0;
    const long long keys = (long long)B * Hkv * max_seqlen;
    const long long cta = own::kMinShare * own_groups(G), ctas = (keys + cta - 1) / cta;
    const int most = int(ctas < num_sms ? ctas : num_sms);
    return P > 0 ? prefix_own_sms(B, G, Hkv, P, d, max_seqlen, most, num_sms) : most;
}

bool decode_prefix_layout(int B, int Hq, int Hkv, int P, int d, int max_seqlen, bool weights, int num_sms,
                          PrefixLayout *l) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)B * Hq;
    l->own_ctas = own_ctas(B, Hq / Hkv, Hkv, P, d, max_seqlen, num_sms);
    PrefixOrder po = {};
    if (P > 0 && !prefix_order(&po, B, Hq / Hkv, Hkv, P, d, max_seqlen, l->own_ctas, num_sms)) return false;
    const size_t parts = max_seqlen > 0 ? (size_t)l->own_ctas * own_groups(Hq / Hkv) + (size_t)B * Hkv : 0;
    const size_t pre = (size_t)po.ids * po.id_rows;
    if (parts > 0x7fffffff) return false;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += up(n);
        return here;
    };
    l->plan = take(max_seqlen > 0 ? (size_t)(2 + B) * sizeof(long long) : 0);
    l->own_rows = take(max_seqlen > 0 ? (size_t)B * Hkv * sizeof(int2) : 0);
    l->own_o = take(parts * (Hq / Hkv) * d * sizeof(float));
    l->own_lse = take(parts * (Hq / Hkv) * sizeof(float));
    l->pre_rows = take((size_t)po.rows * sizeof(int2));
    l->pre_o = take(pre * d * sizeof(float));
    l->pre_lse = take(pre * sizeof(float));
    l->scores = take(weights ? rows * max_seqlen * sizeof(float) : 0);
    l->row_lse = take(weights ? rows * sizeof(float) : 0);
    l->bytes = at;
    return true;
}

int decode_prefix_launch(const DecodePrefixLaunch &a, cudaStream_t stream) {
    return a.d == 64 ? launch_all<64>(a, stream) : launch_all<128>(a, stream);
}

cudaError_t decode_prefix_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_fwd_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_fwd_status, &zero, sizeof(int));
}

}  // namespace attn
