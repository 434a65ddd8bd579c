// evict_sm103.cu -- eviction from a decode cache by accumulated attention weight.
//
// Every head of every sequence (a row) keeps `keep` of its n cached keys: first
// those whose position is among the latest `recent`, then the heaviest, the
// lowest slot first among equals.  Kept keys in slots below `keep` stay where
// they are; the i-th of the slots below `keep` that lost its key (a hole)
// receives the i-th kept key from the slots at or past `keep` (a filler).
// Attention does not depend on the order of its keys, and this order moves the
// fewest rows: one per evicted key, instead of everything behind it.  No slot is
// both read and written, so rows move in place and in parallel.
//
// select_kernel, a CTA a row: each key becomes a 32-bit rank whose unsigned order
// is the order above (recent keys highest), kept in shared memory; a radix
// select finds the keep-th largest rank in four 8-bit passes; two ballot passes
// over the slots in order number the ties, the holes and the fillers.  The
// histogram has a column per lane, so a warp's 32 increments never meet in one
// bank although most weights share their exponent bits.  Work: 8 bytes a key
// from HBM, then shared memory only.
// move_kernel: 2 * 2 d bytes a row each way, HBM-bound.  Where a cache has at
// most kFusedMoves slots past `keep` (a decode loop that evicts what it appends)
// the selecting CTA moves its rows itself and the second launch falls away.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_kernel.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHistBytes = 256 * 32 * 4;
constexpr int kMaxKeys = 48 * 1024;  // ranks that fit in shared memory; longer rows are read again each pass
constexpr int kFusedMoves = 64;

struct Params {
    EvictLaunch a;
    int *head;     // [rows][2]: keys to move, n
    int *src;      // [rows][slots]: in place the fillers, else the source of every slot
    int *holes;    // [rows][gaps]
    int slots, gaps, in_place;
};

// Larger is kept longer.  NaN ranks below every number; -0 equals +0.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (isnan(w)) return 0;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Row {
    const float *w;
    const int *pos;
    long long after;  // positions past this one are recent
    __device__ __forceinline__ uint32_t rank(int i) const {
        return (long long)(pos ? pos[i] : i) > after ? 0xffffffffu : rank_of(w[i]);
    }
};

// Exclusive prefix of one value per warp, and the total.
__device__ __forceinline__ int warp_offsets(int v, int *sh, int &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    int x = sh[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    total = __shfl_sync(0xffffffffu, x, 31);
    return __shfl_sync(0xffffffffu, x, warp) - v;
}

// One row's K, V, weight and position from slot `from` to slot `to`; unit u of
// 2 * d / 8 is 16 bytes of K, then of V.
__device__ __forceinline__ uint4 load_unit(const EvictLaunch &a, long long row, int from, int u) {
    const int half = a.d / 8;
    const char *base = static_cast<const char *>(u < half ? a.kcache : a.vcache);
    return *reinterpret_cast<const uint4 *>(base + ((row * a.max_seqlen + from) * half + (u < half ? u : u - half)) * 16);
}
__device__ __forceinline__ void store_unit(const EvictLaunch &a, long long row, int to, int u, uint4 v) {
    const int half = a.d / 8;
    char *base = static_cast<char *>(u < half ? a.kout : a.vout);
    *reinterpret_cast<uint4 *>(base + ((row * a.out_seqlen + to) * half + (u < half ? u : u - half)) * 16) = v;
}
__device__ __forceinline__ void move_scalars(const EvictLaunch &a, long long row, int from, int to) {
    const long long i = row * a.max_seqlen + from, o = row * a.out_seqlen + to;
    if (a.weights_out) a.weights_out[o] = a.weights[i];
    if (a.pos_out) a.pos_out[o] = a.cache_pos ? a.cache_pos[i] : from;
}

template <bool kShared, bool kFused>
__global__ void __launch_bounds__(kThreads) select_kernel(const Params p) {
    extern __shared__ uint32_t smem[];
    uint32_t *hist = smem;               // [256][32]
    uint32_t *ranks = smem + 256 * 32;   // [n], when they fit
    __shared__ int part[kWarps];
    __shared__ uint32_t found[2];        // the digit, and how many are above it
    __shared__ int fused_holes[kFused ? kFusedMoves : 1], fused_src[kFused ? kFusedMoves : 1];
    const EvictLaunch &a = p.a;
    const long long row = blockIdx.x;
    const int b = int(row / a.Hkv), t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if constexpr (!kFused) griddep_launch_dependents();
    const int n = min(max(a.seqlens[b], 0), a.max_seqlen);
    const int kept = min(n, a.keep);
    if (t == 0) {
        if (a.seqlens_out && row == (long long)b * a.Hkv) a.seqlens_out[b] = kept;
        if constexpr (!kFused) p.head[2 * row + 1] = n;
    }
    int *src = kFused ? fused_src : p.src + row * p.slots;
    int *holes = kFused ? fused_holes : p.holes + row * p.gaps;
    if (n <= a.keep) {  // nothing to evict
        if constexpr (!kFused) {
            if (t == 0) p.head[2 * row] = 0;
            if (!p.in_place)
                for (int i = t; i < n; i += kThreads) src[i] = i;
        }
        return;
    }
    Row r;
    r.w = a.weights + row * a.max_seqlen;
    r.pos = a.cache_pos ? a.cache_pos + row * a.max_seqlen : nullptr;
    r.after = (long long)(a.cur_pos ? a.cur_pos[b] : n - 1) - a.recent;
    auto rank = [&](int i) { return kShared ? ranks[i] : r.rank(i); };

    // Radix select of the keep-th largest rank: `value` collects its digits,
    // `want` counts down to its place among the ranks that share them.
    uint32_t value = 0;
    int want = a.keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = t; i < 256 * 32; i += kThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i = t; i < n; i += kThreads) {
            uint32_t x;
            if (kShared && shift == 24) ranks[i] = x = r.rank(i);
            else x = rank(i);
            if ((x & mask) == value) atomicAdd(&hist[(x >> shift & 255u) * 32 + lane], 1u);
        }
        __syncthreads();
        // Column sums: warp w owns the 8 digits below 256 - 8 w, highest first.
        int count[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            int c = int(hist[(255 - 8 * warp - k) * 32 + lane]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
            count[k] = c;
            sum += c;
        }
        int total;
        int above = warp_offsets(sum, part, total);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (lane == 0 && above < want && above + count[k] >= want) {
                found[0] = uint32_t(255 - 8 * warp - k);
                found[1] = uint32_t(above);
            }
            above += count[k];
        }
        __syncthreads();
        value |= found[0] << shift;
        want -= int(found[1]);
    }

    // Slots in order, a contiguous range a warp.  Ties keep the first `want`.
    const int range = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;
    const int i0 = min(warp * range, n), i1 = min(i0 + range, n);
    const uint32_t below = (1u << lane) - 1;
    int ties = 0, total;
    for (int i = i0; i < i1; i += 32)
        ties += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && rank(i + lane) == value));
    const int ties0 = warp_offsets(ties, part, total);
    // Pass 0 counts the warp's holes and fillers, pass 1 writes them down.
    int hole = 0, fill = 0, moves = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int tie = ties0;
        for (int i = i0; i < i1; i += 32) {
            const int s = i + lane;
            const uint32_t x = s < i1 ? rank(s) : 0;
            const bool same = s < i1 && x == value;
            const uint32_t same_mask = __ballot_sync(0xffffffffu, same);
            const bool keep = s < i1 && (x > value || (same && tie + __popc(same_mask & below) < want));
            tie += __popc(same_mask);
            const bool is_hole = s < i1 && s < a.keep && !keep, is_fill = keep && s >= a.keep;
            const uint32_t hm = __ballot_sync(0xffffffffu, is_hole), fm = __ballot_sync(0xffffffffu, is_fill);
            if (pass == 1) {
                if (is_hole) holes[hole + __popc(hm & below)] = s;
                if (is_fill) {
                    const int f = fill + __popc(fm & below);
                    // Out of place the fillers wait behind the holes for src to be complete.
                    if (p.in_place) src[f] = s;
                    else holes[p.gaps / 2 + f] = s;
                }
                if (!p.in_place && s < a.keep && !is_hole && s < i1) src[s] = s;
            }
            hole += __popc(hm);
            fill += __popc(fm);
        }
        if (pass == 0) {
            hole = warp_offsets(hole, part, moves);
            fill = warp_offsets(fill, part, total);
        }
    }
    if constexpr (kFused) {
        __syncthreads();
        const int units = a.d / 4;
        for (int i = t; i < moves * units; i += kThreads) {
            const int m = i / units, u = i % units;
            store_unit(a, row, holes[m], u, load_unit(a, row, src[m], u));
            if (u == 0) move_scalars(a, row, src[m], holes[m]);
        }
    } else {
        if (t == 0) p.head[2 * row] = moves;
        if (!p.in_place) {
            __syncthreads();
            for (int i = t; i < moves; i += kThreads) src[holes[i]] = holes[p.gaps / 2 + i];
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;  // cache rows of one CTA's turn
constexpr int kMoveBatch = 4;  // 16-byte units a thread has in flight

// Grid-stride over (row, 32 moved keys).
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Params p, long long turns, int per_row) {
    griddep_wait();
    const EvictLaunch &a = p.a;
    const int units = a.d / 4;
    for (long long turn = blockIdx.x; turn < turns; turn += gridDim.x) {
        const long long row = turn / per_row;
        const int first = int(turn - row * per_row) * kMoveRows;
        const int count = p.in_place ? p.head[2 * row] : min(p.head[2 * row + 1], a.keep);
        const int items = min(kMoveRows, count - first) * units;
        const int *src = p.src + row * p.slots + first, *to = p.holes + row * p.gaps + first;
        for (int i0 = threadIdx.x; i0 < items; i0 += kMoveBatch * kMoveThreads) {
            uint4 v[kMoveBatch];
#pragma unroll
            for (int k = 0; k < kMoveBatch; ++k) {
                const int i = i0 + k * kMoveThreads;
                if (i < items) v[k] = load_unit(a, row, src[i / units], i % units);
            }
#pragma unroll
            for (int k = 0; k < kMoveBatch; ++k) {
                const int i = i0 + k * kMoveThreads;
                if (i < items) {
                    const int m = i / units, u = i % units;
                    const int dst = p.in_place ? to[m] : first + m;
                    store_unit(a, row, dst, u, v[k]);
                    if (u == 0) move_scalars(a, row, src[m], dst);
                }
            }
        }
    }
}

struct Layout {
    size_t head, src, holes, bytes;
    int slots, gaps;
    bool fused;
};

Layout layout(const EvictLaunch &a) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)a.B * a.Hkv;
    const bool in_place = a.kout == a.kcache;
    const int past = a.max_seqlen > a.keep ? a.max_seqlen - a.keep : 0;
    const int most = past < a.keep ? past : a.keep;  // moves of a row
    Layout l = {};
    l.fused = in_place && past <= kFusedMoves;
    if (l.fused) return l;
    l.slots = in_place ? most : (a.keep < a.max_seqlen ? a.keep : a.max_seqlen);
    l.gaps = in_place ? most : 2 * most;
    l.head = 0;
    l.src = up(rows * 2 * sizeof(int));
    l.holes = l.src + up(rows * l.slots * sizeof(int));
    l.bytes = l.holes + up(rows * l.gaps * sizeof(int));
    return l;
}

template <bool kShared, bool kFused>
cudaError_t launch_select(const Params &p, size_t smem, cudaStream_t stream) {
    auto kernel = select_kernel<kShared, kFused>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kHistBytes + (kShared ? kMaxKeys * 4 : 0));
        if (e != cudaSuccess) return e;
        if (dev >= 0) attr_set[dev] = true;
    }
    kernel<<<dim3(unsigned(p.a.B * p.a.Hkv)), dim3(kThreads), smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace evict

size_t evict_workspace_bytes(const EvictLaunch &a) { return evict::layout(a).bytes; }

int evict_launch(const EvictLaunch &a, cudaStream_t stream) {
    using namespace evict;
    const Layout l = layout(a);
    Params p = {};
    p.a = a;
    p.in_place = a.kout == a.kcache;
    p.slots = l.slots;
    p.gaps = l.gaps;
    if (!l.fused) {
        p.head = reinterpret_cast<int *>(a.workspace + l.head);
        p.src = reinterpret_cast<int *>(a.workspace + l.src);
        p.holes = reinterpret_cast<int *>(a.workspace + l.holes);
    }
    const bool shared = a.max_seqlen <= kMaxKeys;
    const size_t smem = kHistBytes + (shared ? (size_t)a.max_seqlen * 4 : 0);
    cudaError_t e = l.fused ? (shared ? launch_select<true, true>(p, smem, stream)
                                      : launch_select<false, true>(p, smem, stream))
                            : (shared ? launch_select<true, false>(p, smem, stream)
                                      : launch_select<false, false>(p, smem, stream));
    if (e != cudaSuccess) return note_cuda_error(e, "select_kernel launch");
    if (l.fused || l.slots == 0) return 0;
    const int per_row = (l.slots + kMoveRows - 1) / kMoveRows;
    const long long turns = (long long)a.B * a.Hkv * per_row;
    const long long grid = turns < 8LL * a.num_sms ? turns : 8LL * a.num_sms;
    e = dec::launch_programmatic(move_kernel, dim3(unsigned(grid)), dim3(kMoveThreads), 0, stream, p, turns, per_row);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "move_kernel launch");
}

}  // namespace attn
