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
// select_kernel, one row a cluster of 1, 2, 4 or 8 CTAs, a contiguous range of
// slots each: every key becomes a 32-bit rank whose unsigned order is the order
// above (recent keys highest), kept in shared memory.  A radix select finds the
// keep-th largest rank by 8-bit digits: the CTAs count digits, exchange their 256
// counts through distributed shared memory and each take the same digit; the
// second pass also gathers the ranks that still qualify, a few per cent, and the
// handful that share 16 bits after it are compared with one another (two more
// passes over the gathered ones where there are more).  Two ballot sweeps over the
// slots in order then number the holes and the fillers.  The histogram has a
// column per lane, so a warp's 32 increments never meet in one bank although most
// weights share their exponent bits.  What bounds it is one SM's instruction rate
// and the exchanges' latency (32 rows of 32K keys that need no moving: 29 us on an
// SM a row, 18.5 on four), hence the cluster where there are fewer rows than SMs.
// Without the direct comparison 22 us; without the gathering 0 to 0.7 us more, 3 on
// 8 rows of 128K.
// Where at most kFewMoves keys go, the smallest are found one after the other
// instead (256 rows of 4K keys, 1, 2, 4, 8 of them: 6.9, 8.9, 13.0, 21.2 us; by the
// radix select 13.7).
// move_kernel: 2 * 2 d bytes a row each way, HBM-bound (32 rows of 8000 keys to a
// new cache: 262 MB, 42 us, 6.2 TB/s).  Where a cache has at most kFusedMoves slots
// past `keep` (a decode loop that evicts what it appends) the selecting CTA or
// cluster moves its rows itself and the second launch falls away (256 rows, 1 key of
// 4K: 5.7 us, 15.8 with two launches; 64 keys of 4K 12.5 and 15.8; 16 of 16K in 64 rows
// 14.7 and 17.8; of 128K in 8 rows 20.4 and 21.8).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_tile.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace evict {

constexpr int kHistBytes = 256 * 32 * 4;
constexpr int kListKeys = 4096;       // ranks that the second pass may gather
constexpr int kMaxKeys = 42 * 1024;  // of one CTA: ranks that fit in shared memory; longer ranges are read again each pass
constexpr int kFinalKeys = 128;        // ranks with the same upper half that are compared directly
constexpr int kFusedMoves = 64;
constexpr int kFewMoves = 4;

struct Params {
    EvictLaunch a;
    int *head;     // [rows][2]: keys to move, n
    int *src;      // [rows][slots]: in place the fillers, else the source of every slot: another slot, or ~i for fillers[i]
    int *holes;    // [rows][gaps]: in place the holes, else the fillers
    int slots, gaps, in_place, cluster;
};

// Larger is kept longer.  NaN ranks below every number; -0 equals +0.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (isnan(w)) return 0;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Key {
    float w;
    int pos;
};
struct Row {
    const float *w;
    const int *pos;
    long long after;  // positions past this one are recent
    __device__ __forceinline__ Key key(int i) const { return {w[i], pos ? pos[i] : i}; }
    __device__ __forceinline__ uint32_t rank(Key k) const { return (long long)k.pos > after ? 0xffffffffu : rank_of(k.w); }
};

// Exclusive prefix of one value per warp, and the total.
template <int kWarps>
__device__ __forceinline__ int warp_offsets(int v, int *sh, int &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    int x = lane < kWarps ? sh[lane] : 0;
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

// Calls f(slot, load(slot)) for the slots of [i0, i1) that this thread visits, `step`
// apart, kBatch loads at a time.  None of them is conditional (past the end they
// repeat the last slot), so that all are on their way together: the first pass over
// 8K keys a CTA takes 3.1 us instead of 4.9.
template <int kBatch, typename Load, typename F>
__device__ __forceinline__ void visit(int i0, int i1, int step, Load load, F f) {
    for (int i = i0; i < i1; i += kBatch * step) {
        decltype(load(0)) x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) x[k] = load(min(i + k * step, i1 - 1));
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (i + k * step < i1) f(i + k * step, x[k]);
    }
}

// Who moves the kept keys: move_kernel, or the CTA or the cluster that selects them.
enum Mover { kLater = 0, kCta = 1, kCluster = 2 };

// A cluster (kCta: a single CTA) selects the kept keys of one row.
template <bool kShared, Mover kMover, int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const Params p) {
    namespace cg = cooperative_groups;
    constexpr bool kFused = kMover != kLater;
    constexpr int kWarps = kThreads / 32;
    extern __shared__ uint32_t smem[];
    uint32_t *hist = smem;               // [256][32]
    uint32_t *list = smem + 256 * 32;    // [kListKeys] gathered ranks
    uint32_t *ranks = list + kListKeys;  // [keys of this CTA], when they fit
    __shared__ int part[kWarps];
    __shared__ int counts[2][256];       // digit counts of this CTA (in turns: the others may still read the last)
    __shared__ int totals[4];            // this CTA's tallies
    __shared__ int theirs[8][4];         // those of the cluster's
    __shared__ int tally[4][32];         // of each warp: kept below and past `keep`, ties below and past
    __shared__ int listed;               // entries of the list
    __shared__ uint32_t found[3];        // the digit, how many are above it, how many have it
    __shared__ uint32_t finals[kFinalKeys], every[kFinalKeys];  // of this CTA; of the cluster
    __shared__ int final_count;
    __shared__ unsigned long long least[kWarps], least_here[2];
    __shared__ int fused_holes[kFused ? kFusedMoves : 1], fused_src[kFused ? kFusedMoves : 1], fused_moves;
    __shared__ int gone_slots[kFewMoves];
    const EvictLaunch &a = p.a;
    const cg::cluster_group cluster = cg::this_cluster();
    const int peers = kMover == kCta ? 1 : p.cluster, peer = kMover == kCta ? 0 : int(cluster.block_rank());
    const long long row = blockIdx.x / peers;
    const int b = int(row / a.Hkv), t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if constexpr (!kFused) griddep_launch_dependents();
    const int listed_keys = a.seqlens[b], newest = a.cur_pos ? a.cur_pos[b] : 0;
    if constexpr (!kFused)  // for the first digit, while the loads are on their way
        for (int i = t; i < 256 * 32; i += kThreads) hist[i] = 0;
    const int n = min(max(listed_keys, 0), a.max_seqlen);
    const int kept = min(n, a.keep);
    if (t == 0 && peer == 0) {
        if (a.seqlens_out && row == (long long)b * a.Hkv) a.seqlens_out[b] = kept;
        if constexpr (!kFused) p.head[2 * row + 1] = n;
    }
    int *src = kFused ? fused_src : p.src + row * p.slots;
    int *holes = kFused ? fused_holes : p.holes + row * p.gaps;
    if constexpr (kMover == kCluster) src = cluster.map_shared_rank(src, 0), holes = cluster.map_shared_rank(holes, 0);
    if (n <= a.keep) {  // nothing to evict
        if constexpr (!kFused) {
            if (t == 0 && peer == 0) p.head[2 * row] = 0;
            if (!p.in_place)
                for (int i = peer * kThreads + t; i < n; i += peers * kThreads) src[i] = i;
        }
        return;
    }
    Row r;
    r.w = a.weights + row * a.max_seqlen;
    r.pos = a.cache_pos ? a.cache_pos + row * a.max_seqlen : nullptr;
    r.after = (long long)(a.cur_pos ? newest : n - 1) - a.recent;
    // This CTA's slots.
    const int chunk = ((n + peers - 1) / peers + 31) / 32 * 32;
    const int lo = min(peer * chunk, n), hi = min(lo + chunk, n);
    auto key = [&](int i) { return r.key(i); };
    auto rank = [&](int i) { return kShared ? ranks[i - lo] : r.rank(r.key(i)); };
    auto cluster_sync = [&]() {
        if (peers > 1) cluster.sync();
        else __syncthreads();
    };
    int moves = 0;

    if (kFused && n - a.keep <= kFewMoves) {
        // A few keys go: find the smallest (rank, slot from the end), then the
        // next one, a pass each.
        if constexpr (kShared)
            visit<8>(lo + t, hi, kThreads, key, [&](int i, Key k) { ranks[i - lo] = r.rank(k); });  // each thread its own
        unsigned long long last = 0;
        for (int e = 0; e < n - a.keep; ++e) {
            unsigned long long low = ~0ull;
            visit<8>(lo + t, hi, kThreads, rank, [&](int i, uint32_t x) {
                const unsigned long long key = (unsigned long long)x << 32 | uint32_t(~i);
                if ((e == 0 || key > last) && key < low) low = key;
            });
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const unsigned long long y = __shfl_xor_sync(0xffffffffu, low, off);
                low = y < low ? y : low;
            }
            if (lane == 0) least[warp] = low;
            __syncthreads();
            low = least[lane % kWarps];
#pragma unroll
            for (int off = kWarps / 2; off > 0; off >>= 1) {
                const unsigned long long y = __shfl_xor_sync(0xffffffffu, low, off);
                low = y < low ? y : low;
            }
            if constexpr (kMover == kCluster) {
                // (In turns: the others may still read the last one.)
                if (t == 0) least_here[e & 1] = low;
                cluster.sync();
                low = lane < peers ? *cluster.map_shared_rank(&least_here[e & 1], lane) : ~0ull;
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) {
                    const unsigned long long y = __shfl_xor_sync(0xffffffffu, low, off);
                    low = y < low ? y : low;
                }
                low = __shfl_sync(0xffffffffu, low, 0);
            }
            last = low;
            if (t == 0) gone_slots[e] = int(~uint32_t(low));
            __syncthreads();
        }
        if constexpr (kMover == kCluster) cluster.barrier_arrive();  // this CTA has read all that it will of the others
        if (t == 0) {
            // Holes: the evicted slots below keep, in order.  Fillers: the slots past it that stay.
            int gone[kFewMoves];
            const int count = n - a.keep;
            unsigned past = 0;
            for (int e = 0; e < count; ++e) {
                const int s = gone_slots[e];
                if (s >= a.keep) {
                    past |= 1u << (s - a.keep);
                    continue;
                }
                int at = moves++;
                for (; at > 0 && gone[at - 1] > s; --at) gone[at] = gone[at - 1];
                gone[at] = s;
            }
            for (int e = 0, f = 0; e < count; ++e)
                if (!(past >> e & 1)) fused_src[f++] = a.keep + e;
            for (int m = 0; m < moves; ++m) fused_holes[m] = gone[m];
            fused_moves = moves;
        }
        __syncthreads();
        moves = fused_moves;
    } else {
        // Radix select of the keep-th largest rank: `value` collects its digits,
        // `want` counts down to its place among the ranks that share them.
        uint32_t value = 0;
        int want = a.keep;
        bool gathered = false;  // the list holds every rank that still qualifies
        if (t == 0) listed = final_count = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (kFused || shift < 24)
                for (int i = t; i < 256 * 32; i += kThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            auto count = [&](uint32_t x) { atomicAdd(&hist[(x >> shift & 255u) * 32 + lane], 1u); };
            if (shift == 24) {
                visit<8>(lo + t, hi, kThreads, key, [&](int i, Key k) {
                    const uint32_t x = r.rank(k);
                    if (kShared) ranks[i - lo] = x;
                    count(x);
                });
            } else if (gathered) {
                visit<4>(t, listed, kThreads, [&](int i) { return list[i]; },
                         [&](int, uint32_t x) { if ((x & mask) == value) count(x); });
            } else if (shift == 16) {
                // Whole warps, eight keys a lane: one reservation in the list for all of them.
                for (int i0 = lo + warp * 32; i0 < hi; i0 += 8 * kThreads) {
                    uint32_t x[8], some[8];
                    int total = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = i0 + k * kThreads + lane < hi ? rank(i0 + k * kThreads + lane) : ~value;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        some[k] = __ballot_sync(0xffffffffu, (x[k] & mask) == value);
                        total += __popc(some[k]);
                    }
                    int at = 0;
                    if (lane == 0 && total > 0) at = atomicAdd(&listed, total);
                    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (some[k] >> lane & 1) {
                            count(x[k]);
                            const int to = at + __popc(some[k] & ((1u << lane) - 1));
                            if (to < kListKeys) list[to] = x[k];
                        }
                        at += __popc(some[k]);
                    }
                }
            } else {
                visit<8>(lo + t, hi, kThreads, rank, [&](int, uint32_t x) { if ((x & mask) == value) count(x); });
            }
            __syncthreads();
            if (shift == 16) gathered = listed <= kListKeys;
            // Column sums of this CTA, then over the cluster: warp w owns kDigits digits from 255 - kDigits w down.
            constexpr int kDigits = 256 / kWarps;
            int *mine = counts[shift >> 3 & 1];
#pragma unroll
            for (int k = 0; k < kDigits; ++k) {
                const int digit = 255 - kDigits * warp - k;
                const int c = __reduce_add_sync(0xffffffffu, int(hist[digit * 32 + lane]));
                if (lane == 0) mine[digit] = c;
            }
            cluster_sync();
            // Lane k of a warp holds its k-th digit, highest first.
            int c = 0;
            if (lane < kDigits) {
                const int digit = 255 - kDigits * warp - lane;
                if (peers > 1) {
                    int theirs[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) theirs[q] = q < peers ? cluster.map_shared_rank(mine, q)[digit] : 0;
#pragma unroll
                    for (int q = 0; q < 8; ++q) c += theirs[q];
                } else {
                    c = mine[digit];
                }
            }
            int total, upto = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            const int above = warp_offsets<kWarps>(__shfl_sync(0xffffffffu, upto, 31), part, total) + upto - c;
            if (lane < kDigits && above < want && above + c >= want) {
                found[0] = uint32_t(255 - kDigits * warp - lane);
                found[1] = uint32_t(above);
                found[2] = uint32_t(c);
            }
            __syncthreads();
            value |= found[0] << shift;
            want -= int(found[1]);
            if (shift == 16 && found[2] <= kFinalKeys) {
                // So few share 16 bits that they are compared with one another: one
                // exchange instead of two.
                const int left = int(found[2]);
                auto pick = [&](int, uint32_t x) {
                    if ((x & 0xffff0000u) == value) finals[atomicAdd(&final_count, 1)] = x;
                };
                if (gathered) visit<4>(t, listed, kThreads, [&](int i) { return list[i]; }, pick);
                else visit<8>(lo + t, hi, kThreads, rank, pick);
                cluster_sync();
                if (t < left) {
                    uint32_t x = 0;
                    if (peers > 1) {
                        int i = t;
                        for (int q = 0; q < peers; ++q) {
                            const int n_q = *cluster.map_shared_rank(&final_count, q);
                            if (i < n_q) {
                                x = cluster.map_shared_rank(finals, q)[i];
                                break;
                            }
                            i -= n_q;
                        }
                    } else {
                        x = finals[t];
                    }
                    every[t] = x;
                }
                __syncthreads();
                if (t < left) {
                    const uint32_t x = every[t];
                    int more = 0, same = 0;
                    for (int i = 0; i < left; ++i) more += every[i] > x, same += every[i] == x;
                    if (more < want && more + same >= want) {  // one value: equal threads write equal numbers
                        found[0] = x;
                        found[1] = uint32_t(more);
                    }
                }
                __syncthreads();
                value = found[0];
                want -= int(found[1]);
                break;
            }
        }

        // Slots in order, a contiguous range a warp.  Of the ranks equal to `value` the first `want` are kept.
        const int range = (hi - lo + kWarps * 32 - 1) / (kWarps * 32) * 32;
        const int i0 = min(lo + warp * range, hi), i1 = min(i0 + range, hi);
        const uint32_t below = (1u << lane) - 1;
        constexpr int kBatch = 4;
        const int mid = min(max(a.keep, i0), i1);  // slots past `keep` from here on
        auto sweep = [&](int from, int to, auto f) {  // f(slot, rank, inside) by whole warps, in order
            for (int i = from; i < to; i += kBatch * 32) {
                uint32_t x[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) x[k] = rank(min(i + k * 32 + lane, to - 1));
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (i + k * 32 < to) f(i + k * 32 + lane, x[k], i + k * 32 + lane < to);
            }
        };
        // First sweep: keys above `value` and ties, below `keep` and past it.
        int up[2] = {0, 0}, tie[2] = {0, 0};
        sweep(i0, mid, [&](int, uint32_t x, bool in) { up[0] += in && x > value, tie[0] += in && x == value; });
        sweep(mid, i1, [&](int, uint32_t x, bool in) { up[1] += in && x > value, tie[1] += in && x == value; });
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            up[k] = __reduce_add_sync(0xffffffffu, up[k]);
            tie[k] = __reduce_add_sync(0xffffffffu, tie[k]);
        }
        // Where this warp's ties, holes and fillers start.  Slots go up with the
        // warp and with the CTA, and within either the ties below `keep` come
        // before those past it, so four counts of every warp and of every CTA
        // say all of it: one exchange.
        if (lane == 0) {
            tally[0][warp] = up[0], tally[1][warp] = up[1];
            tally[2][warp] = tie[0], tally[3][warp] = tie[1];
        }
        __syncthreads();
        int mine[4];  // lane w: the counts of warp w
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[k] = lane < kWarps ? tally[k][lane] : 0;
        auto scan = [&](int v) {  // sum over the lanes up to this one
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += y;
            }
            return v;
        };
        int ties = 0, hole = 0, fill = 0;  // ahead of this CTA, then of this warp
        if (peers > 1) {
            if (warp == 0)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int sum = __reduce_add_sync(0xffffffffu, mine[k]);
                    if (lane == 0) totals[k] = sum;
                }
            cluster.sync();
            if (warp == 0)  // a lane a number; the other warps read the copy
                theirs[lane >> 2][lane & 3] = (lane >> 2) < peers ? cluster.map_shared_rank(totals, lane >> 2)[lane & 3] : 0;
            __syncthreads();
            if constexpr (!kFused) cluster.barrier_arrive();  // this CTA has read all that it will of the others
            int t0 = 0;  // ties ahead of CTA q
            for (int q = 0; q < peers; ++q) {
                if (q < peer) fill += theirs[q][1] + min(theirs[q][3], max(want - t0 - theirs[q][2], 0));
                if (q == peer) ties = t0, hole = moves;
                const int left = max(want - t0, 0), start = min(q * chunk, n);
                moves += max(min(min(start + chunk, n), a.keep) - start, 0) - theirs[q][0] - min(theirs[q][2], left);
                t0 += theirs[q][2] + theirs[q][3];
            }
        }
        {
            const int upto = scan(mine[2] + mine[3]);
            const int left = max(want - ties - (upto - mine[2] - mine[3]), 0);
            const int s0 = min(lo + lane * range, hi);
            const int gaps = lane < kWarps ? max(min(min(s0 + range, hi), a.keep) - s0, 0) - mine[0] - min(mine[2], left) : 0;
            const int fills = mine[1] + min(mine[3], max(left - mine[2], 0));
            const int gaps_upto = scan(gaps), fills_upto = scan(fills);
            if (peers == 1) moves = __shfl_sync(0xffffffffu, gaps_upto, 31);
            ties += __shfl_sync(0xffffffffu, upto - mine[2] - mine[3], warp);
            hole += __shfl_sync(0xffffffffu, gaps_upto - gaps, warp);
            fill += __shfl_sync(0xffffffffu, fills_upto - fills, warp);
        }
        auto stays = [&](uint32_t x, bool in) {
            const uint32_t same = __ballot_sync(0xffffffffu, in && x == value);
            bool yes = in && x > value;
            if (same) {
                yes |= (same >> lane & 1) && ties + __popc(same & below) < want;
                ties += __popc(same);
            }
            return yes;
        };
        sweep(i0, mid, [&](int s, uint32_t x, bool in) {
            const bool gone = !stays(x, in) && in;
            const uint32_t all = __ballot_sync(0xffffffffu, gone);
            const int at = hole + __popc(all & below);
            hole += __popc(all);
            if (!p.in_place && in) src[s] = gone ? ~at : s;
            if (p.in_place && gone) holes[at] = s;
        });
        int *fillers = p.in_place ? src : holes;
        sweep(mid, i1, [&](int s, uint32_t x, bool in) {
            const bool filler = stays(x, in);
            const uint32_t all = __ballot_sync(0xffffffffu, filler);
            if (filler) fillers[fill + __popc(all & below)] = s;
            fill += __popc(all);
        });
        if constexpr (kMover == kCluster) {
            // The first CTA has the lists; every other takes a copy.
            cluster.sync();
            if (peer > 0 && t < moves) fused_src[t] = src[t], fused_holes[t] = holes[t];
            __syncthreads();
            cluster.barrier_arrive();
        }
    }
    if constexpr (kFused) {
        __syncthreads();
        const int units = a.d / 4;
        for (int i = peer * kThreads + t; i < moves * units; i += peers * kThreads) {
            const int m = i / units, u = i % units, from = fused_src[m], to = fused_holes[m];
            store_unit(a, row, to, u, load_unit(a, row, from, u));
            if (u == 0) move_scalars(a, row, from, to);
        }
        if constexpr (kMover == kCluster) cluster.barrier_wait();
    } else {
        if (t == 0 && peer == 0) p.head[2 * row] = moves;
        if (peers > 1) cluster.barrier_wait();  // no CTA leaves while another may read its shared memory
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;  // cache rows of one CTA's turn
constexpr int kMoveBatch = 8;  // 16-byte units a thread has in flight

// `per_row` CTAs a row, each every per_row-th kMoveRows of its moved keys.  kUnits: 16-byte units of a key and its
// value (d / 4) where that divides the CTA, so that a thread keeps one unit and
// steps over keys without a division; 0: any d.
template <int kUnits>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Params p, int per_row) {
    __shared__ int from[kMoveRows], to[kMoveRows];
    griddep_wait();
    const EvictLaunch &a = p.a;
    const int units = kUnits ? kUnits : a.d / 4, half = units / 2;
    const long long row = blockIdx.x / per_row;
    const int count = p.in_place ? p.head[2 * row] : min(p.head[2 * row + 1], a.keep);
    for (int first = int(blockIdx.x % per_row) * kMoveRows; first < count; first += per_row * kMoveRows) {
        const int keys = min(kMoveRows, count - first);
        if (int(threadIdx.x) < keys) {
            const int m = first + threadIdx.x, *list = p.holes + row * p.gaps;
            int s = p.src[row * p.slots + m];
            if (s < 0) s = list[~s];
            from[threadIdx.x] = s;
            to[threadIdx.x] = p.in_place ? list[m] : m;
        }
        __syncthreads();
        if (int(threadIdx.x) < keys) move_scalars(a, row, from[threadIdx.x], to[threadIdx.x]);
        if constexpr (kUnits > 0) {
            constexpr int kStep = kMoveThreads / kUnits;
            const int u = threadIdx.x % kUnits, m0 = threadIdx.x / kUnits;
            const bool key = u < half;
            const char *in = static_cast<const char *>(key ? a.kcache : a.vcache) +
                             row * a.max_seqlen * (half * 16) + (key ? u : u - half) * 16;
            char *out = static_cast<char *>(key ? a.kout : a.vout) + row * a.out_seqlen * (half * 16) +
                        (key ? u : u - half) * 16;
#pragma unroll
            for (int m1 = 0; m1 < kMoveRows; m1 += kMoveBatch * kStep) {
                uint4 v[kMoveBatch];
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k) {
                    const int m = m0 + m1 + k * kStep;
                    if (m < keys) v[k] = __ldcs(reinterpret_cast<const uint4 *>(in + (long long)from[m] * (half * 16)));
                }
#pragma unroll
                for (int k = 0; k < kMoveBatch; ++k) {
                    const int m = m0 + m1 + k * kStep;
                    if (m < keys)
                        *reinterpret_cast<uint4 *>(out + (long long)to[m] * (half * 16)) = v[k];
                }
            }
        } else {
            for (int i = threadIdx.x; i < keys * units; i += kMoveThreads) {
                const int m = i / units, u = i % units;
                store_unit(a, row, to[m], u, load_unit(a, row, from[m], u));
            }
        }
        __syncthreads();  // the lists are free for the next turn
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
    l.gaps = most;
    l.head = 0;
    l.src = up(rows * 2 * sizeof(int));
    l.holes = l.src + up(rows * l.slots * sizeof(int));
    l.bytes = l.holes + up(rows * l.gaps * sizeof(int));
    return l;
}

template <bool kShared, Mover kMover, int kThreads>
cudaError_t launch_select(const Params &p, size_t smem, cudaStream_t stream) {
    auto kernel = select_kernel<kShared, kMover, kThreads>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kHistBytes + (kListKeys + (kShared ? kMaxKeys : 0)) * 4);
        if (e != cudaSuccess) return e;
        if (dev >= 0) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.a.B) * unsigned(p.a.Hkv) * unsigned(p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(p.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
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
    // CTAs a row: while every row's cluster still has its SMs to itself (a cluster
    // lies within one of the 8 parts of the GPU, each of which has half a cluster
    // left over in the mean) and a CTA 2048 keys or more.  In us, with 1, 2, 4 and 8
    // CTAs a row: 8 rows of 16K keys 18.5, 17.1, 15.1, 15.1; 8 of 128K 197, 114, 36, 25; 16
    // of 8K 14.4, 14.4, 13.7, 16.4; 8 of 4K 11.7, and 13.7 with eight (an exchange costs
    // what it saves).  The fused form, 16 keys of 8 rows: of 8K 10.4, 11.8, 11.6, 12.3; of
    // 16K 14.6, 14.3, 12.2, 12.7; of 64K 72, 26.5, 19.0, 16.1; of 128K 136, 77, 27, 20.4.
    // Where the clusters do not all fit: 16 rows of 64K 75, 28.5, 20.7, 31.7 (15 rows 18.0
    // with eight); 38 rows of 64K 75, 28.8, 37.8 with one, two, four (36 rows 22.4).
    const long long rows = (long long)a.B * a.Hkv;
    p.cluster = 1;
    if (a.max_seqlen >= (l.fused ? 16384 : 8192))
        while (p.cluster < 8 && (rows + 4) * p.cluster * 2 <= a.num_sms && a.max_seqlen / (p.cluster * 2) >= 2048) p.cluster *= 2;
    const int keys = ((a.max_seqlen + p.cluster - 1) / p.cluster + 31) / 32 * 32;
    const bool shared = keys <= kMaxKeys;
    const size_t smem = kHistBytes + (kListKeys + (shared ? (size_t)keys : 0)) * 4;
    // Threads: a CTA with few keys spends its time at barriers, which are cheaper with
    // 512 threads (2048 keys of each of 64 CTAs 15.1 us, 16.5 with 1024), one with many
    // on its keys (8K of 128 CTAs 19.2 and 18.5; one key of 64 rows of 8K by the fused
    // form 7.5 and 6.9).  Two of more rows than SMs share an SM with 512 threads, up to
    // some length (256 rows of 8K 21 and 26; one key of 256 rows of 4K 6.9 and 9.6, of 8K
    // 8.9 and 11.6, of 16K 18.6 and 15.8).
    const bool many = keys > (rows > a.num_sms ? 12288 : 4096);
    auto select = [&](auto mover) {
        constexpr Mover m = decltype(mover)::value;
        return !shared ? launch_select<false, m, 1024>(p, smem, stream)
               : many  ? launch_select<true, m, 1024>(p, smem, stream)
                       : launch_select<true, m, 512>(p, smem, stream);
    };
    cudaError_t e = !l.fused        ? select(std::integral_constant<Mover, kLater>())
                    : p.cluster > 1 ? select(std::integral_constant<Mover, kCluster>())
                                    : select(std::integral_constant<Mover, kCta>());
    if (e != cudaSuccess) return note_cuda_error(e, "select_kernel launch");
    if (l.fused || l.slots == 0) return 0;
    // In place the number of moves is known on the device only and may be far from
    // the most: about as many CTAs as the GPU holds.  Whole calls, in us, with 2, 8, 32
    // CTAs an SM and with one for every kMoveRows slots: 128 rows of 32K keys to 16000
    // (8190 of them move) 240, 215, 203, 204; 256 of 8K to 4096 115, 116, 108, 109; one key past
    // 4096 in 256 rows of 8K slots 14.8, 15.4, 18.4, 26.8; 100 past 16000 in 128 of 32K 19.6,
    // 19.5, 22.2, 38.7.  Out of place the most is usual.
    long long per_row = (l.slots + kMoveRows - 1) / kMoveRows;
    const long long most = p.in_place ? (8LL * a.num_sms + rows - 1) / rows : 0x7fffffffLL / rows;
    if (per_row > most) per_row = most;
    auto move = a.d == 128 ? move_kernel<32> : (a.d == 64 ? move_kernel<16> : move_kernel<0>);
    e = dec::launch_programmatic(move, dim3(unsigned(rows * per_row)), dim3(kMoveThreads), 0, stream, p, int(per_row));
    return e == cudaSuccess ? 0 : note_cuda_error(e, "move_kernel launch");
}

}  // namespace attn
