// decode_tree_sm103.cu -- attention of several drafted tokens per sequence over a
// cache in pages (or contiguous): each attends all cached keys and, of the drafted
// keys behind them, those that the tree's mask names.
//
// For KV head g of sequence b the rows are a matrix of G T queries (head of the
// group, token), all against the same keys:
//     s = scale q k^T  (-inf where the mask hides the key),  o = softmax(s) v.
// The keys are read once for all rows.  With R = G T rows a key costs 4 d bytes and
// 4 d R flops: below some 280 rows HBM bounds it, above that the tensor cores.  So
// S = Q K^T and P V are tcgen05 products of 128 rows and 128 keys whatever R is;
// a tile of few rows is idle for the most part, but still faster than HBM.
//
// A CTA an SM, persistent, as in fwd_kernel.cuh: a TMA warp, an issuing warp, and
// two chains of four softmax warps, whose products and exponentials overlap.
//   kRows (R > 128): the chains hold two tiles of rows, and both visit every key
//     block; units of 256 rows, `mt` units a KV head, side by side on mt SMs so
//     that all but one find the keys in L2.
//   kKeys (R <= 128): one tile; the chains take turns with the key blocks (of 64
//     keys), each with two score buffers, so that the products' latency is not in a
//     chain's way; their softmax states are merged in the epilogue, where each of
//     them adds up half of the columns from both accumulators.
// The blocks of all (sequence, KV head) pairs, in that order, are cut into equal
// shares, one a CTA (group of mt): nothing depends on how ragged the lengths are.  A
// pair that lies in one share is written out at once; one that is cut goes through
// partials: share s writes its first segment's to slot 2 s (a pair that began
// before) and its last one's to 2 s + 1 (a pair that goes on), and merge_kernel adds
// up slot 2 s + 1, 2 (s + 1), 2 (s + 2), ...
//
// Pages: a block of 128 keys is 128 / page_size boxes, each from the page that the
// table names; a box on no page is filled with zeros by coordinates past the end.
// Columns past the last key, on no page, or hidden by the mask become -inf before the
// softmax.  A probability of 0 does not hide a V of infinity or NaN from the product,
// so the softmax warps clean the blocks that hold drafted keys before they hand P
// over: rows behind the last key, which may hold anything, become zeros, and so do
// elements of drafted rows that are not finite, which the epilogue then adds to the
// rows that see them.
//
// Precision: scores, maxima, sums, partials in fp32; probabilities are rounded to
// bf16 for the product with V, because the instruction takes both operands in one
// 16-bit type; outputs are rounded once more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_tile.cuh"
#include "sm103_ptx.cuh"

namespace attn {

static __device__ int g_tree_status;

namespace dtree {

// mbar_wait_warp in fewer instructions: the waits are many, and a unit of few blocks
// runs most of the kernel's code once, out of a cold instruction cache.  The clock is
// read every 16th time around.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 1; limit_ns > 0; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (it & 15u) continue;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *abort != 0 || now - t0 > limit_ns)) break;
    }
    if ((threadIdx.x & 31) == 0) {
        *abort = 1;
        atomicOr(&g_tree_status, kStatusTimeout);
    }
    __syncwarp();
    return false;
}

constexpr int kTileM = 128;  // rows of a tile
constexpr int kThreads = 384;
// As in fwd_kernel.cuh: 384 threads x 168 registers at launch are shared out anew.
constexpr int kLaunchRegs = 168, kCtrlRegs = 120, kSoftmaxRegs = 192;
static_assert(128 * kCtrlRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kTmemCols = 512;
constexpr int kTurnStride = 20, kTurnFloats = 32 * kTurnStride;
constexpr int kMaskWords = 8;  // 32-bit words of a row's mask: 256 drafted tokens
constexpr int kMergeWarps = 4;

constexpr int kUnitInts = 12;  // of a unit in the queue

// Keys of a block.  Where the chains take turns, HBM is what they wait for, and small
// blocks hold less of the ring while they are worked on.
constexpr int block_keys(bool keys) { return keys ? 64 : 128; }

template <int D, bool kKeys>
struct Cfg {
    static constexpr int kBlock = block_keys(kKeys);
    static constexpr int kChunks = D / 64, kQChunkBytes = kTileM * 128, kChunkBytes = kBlock * 128;
    static constexpr int kQTiles = kKeys ? 1 : 2;
    static constexpr int kQBytes = kTileM * D * 2, kKVBytes = kBlock * D * 2;
    static constexpr int kStages = (D == 128 ? 1 : 2) * (kKeys ? 10 : 4);
    static constexpr int kOCol = 2 * kTileM;
    static constexpr int kDataBytes = kQTiles * kQBytes + kStages * kKVBytes;
    static constexpr int kTurnOffset = kDataBytes, kStateOffset = kTurnOffset + 8 * kTurnFloats * 4;
    static constexpr int kOddOffset = kStateOffset + (kKeys ? 2 * 2 * kTileM * 8 : 0);
    static constexpr int kBarOffset = kOddOffset + 4 * kMaskWords * 4;
    // barriers
    // (S and P: [chain][buffer])
    static constexpr int kBuffers = kKeys ? 2 : 1;
    static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 8, kOFull = 12, kOEmpty = 14, kStateFull = 16,
                         kDrain = 17, kUFull = 18, kUEmpty = 20, kKVFull = 22, kKVEmpty = 22 + kStages,
                         kNumBars = 22 + 2 * kStages;
    static constexpr int kUnitOffset = (kBarOffset + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kSmemBytes = kUnitOffset + 2 * kUnitInts * 4 + 16 + 1024;  // units, tmem, abort; alignment
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Params {
    const int *seqlens, *draft_lens, *table;
    const unsigned long long *mask;
    const __nv_bfloat16 *v;
    __nv_bfloat16 *o;
    float *lse;                // natural log, or null
    float *part_o, *part_lse;  // [2 shares][rows][D], [2 shares][rows] (log2 units)
    int4 *cuts;                // [shares]: {b, g, partials, drafted tokens} of the pair that goes on behind a share
    int B, Hkv, G, T, rows;
    int num_pages, page_size, shift, cap, max_pages;
    int mt, shares;
    float scale_log2;
    unsigned long long wait_ns;
};

// A piece of work: blocks [j0, j0 + n) of the nb blocks of pair (b, g); n = 0: the end.  holes: some of its entries may be
// no page.
struct Unit {
    int b, g, j0, n, nb, len, tb, keys, holes;
    __device__ __forceinline__ void put(volatile int *e) const {
        e[0] = b, e[1] = g, e[2] = j0, e[3] = n, e[4] = nb, e[5] = len, e[6] = tb, e[7] = keys, e[8] = holes;
    }
    __device__ __forceinline__ void get(const volatile int *e) {
        b = e[0], g = e[1], j0 = e[2], n = e[3], nb = e[4], len = e[5], tb = e[6], keys = e[7], holes = e[8];
    }
};

__device__ __forceinline__ void load_sequence(const Params &p, int b, int &len, int &tb) {
    len = min(max(p.seqlens[b], 0), p.cap);
    tb = p.draft_lens ? min(max(p.draft_lens[b], 0), p.T) : p.T;
}
__device__ __forceinline__ int keys_of(const Params &p, int len, int tb) {
    return tb > 0 ? int(min((long long)len + tb, (long long)p.cap)) : 0;
}
template <int kBlock>
__device__ __forceinline__ int blocks_of(int keys) {
    return (keys + kBlock - 1) / kBlock;
}

// Blocks of all pairs (all lanes of the calling warp).  The host bounds the sum, and all places in it, below 2^31.
template <int kBlock>
__device__ __forceinline__ unsigned all_blocks(const Params &p) {
    unsigned n = 0;
#pragma unroll 4
    for (int b = threadIdx.x & 31; b < p.B; b += 32) {
        int len, tb;
        load_sequence(p, b, len, tb);
        n += blocks_of<kBlock>(keys_of(p, len, tb));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n * p.Hkv;
}

// The pair of block x, and which of its blocks x is (j0); all lanes of the calling warp.  (The lengths are in the L1
// by now.)
template <int kBlock>
__device__ __forceinline__ Unit find_block(const Params &p, unsigned x) {
    const int lane = threadIdx.x & 31;
    Unit u = {};
    unsigned before = 0;
#pragma unroll 1
    for (int first = 0; first < p.B; first += 32) {
        int len = 0, tb = 0, keys = 0;
        if (first + lane < p.B) {
            load_sequence(p, first + lane, len, tb);
            keys = keys_of(p, len, tb);
        }
        const unsigned n = unsigned(blocks_of<kBlock>(keys)) * p.Hkv;
        unsigned upto = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        const unsigned base = before + upto - n;
        const uint32_t hit = __ballot_sync(0xffffffffu, x >= base && x < base + n);
        if (hit) {
            const int src = __ffs(hit) - 1;
            u.b = first + src;
            u.len = __shfl_sync(0xffffffffu, len, src);
            u.tb = __shfl_sync(0xffffffffu, tb, src);
            u.keys = __shfl_sync(0xffffffffu, keys, src);
            u.nb = blocks_of<kBlock>(u.keys);
            const unsigned rem = x - __shfl_sync(0xffffffffu, base, src);
            u.g = int(rem / unsigned(u.nb));
            u.j0 = int(rem - unsigned(u.g) * unsigned(u.nb));
            return u;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return u;
}

// Bits [u, u + 32) of a row's mask; keys before the drafted ones (u < 0) are seen by all.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t (&m)[kMaskWords], int u) {
    const int i = u >> 5;  // rounds down
    uint32_t lo = i < 0 ? ~0u : 0u, hi = i < -1 ? ~0u : 0u;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) {
        if (w == i) lo = m[w];
        if (w == i + 1) hi = m[w];
    }
    return __funnelshift_r(lo, hi, u & 31);
}

// V rows [first, kBlock) of a block in shared memory, by the four warps of a chain (`warp` of them; the swizzle stays
// within a row's 128 bytes of a chunk, which eight lanes take): rows from `end` on become zeros; in the drafted rows
// before it, of which row `first` is number `u0`, elements that are not finite do, and the row's bit in `odd` is set.
template <int kChunks, int kBlock>
__device__ __forceinline__ void clean_rows(uint8_t *v, int warp, int first, int end, int u0, uint32_t *odd) {
    const int lane = threadIdx.x & 31;
    for (int row = first + warp * 4 + (lane >> 3); row < kBlock; row += 16) {
        bool found = false;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            uint4 *at = reinterpret_cast<uint4 *>(v + c * (kBlock * 128) + row * 128 + (lane & 7) * 16);
            if (row >= end) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
            }
            uint4 x = *at;
            uint32_t *w = &x.x;
            bool here = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u, here = true;
                if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0x0000ffffu, here = true;
            }
            if (here) *at = x;
            found |= here;
        }
        const int u = u0 + row - first;
        if (found) atomicOr(odd + (u >> 5), 1u << (u & 31));
    }
}

// Adds to n columns of a stored row the elements of V that are not finite.
template <typename T>
__device__ __noinline__ void add_odd(T *to, const __nv_bfloat16 *v, int n) {
    for (int i = 0; i < n; ++i) {
        const float y = __bfloat162float(v[i]);
        if (!isfinite(y)) to[i] = T(float(to[i]) + y);
    }
}

template <int D, bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Params p) {
    using C = Cfg<D, kKeys>;
    constexpr int kBlock = C::kBlock;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + C::kQTiles * C::kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    volatile int *units = reinterpret_cast<volatile int *>(smem + C::kUnitOffset);  // two entries
    // Drafted V rows of a unit that are not finite everywhere; of four units in turn, since the other chain may still
    // read the last one's, and the next one's has to be empty by then.
    uint32_t *odd_rows = reinterpret_cast<uint32_t *>(smem + C::kOddOffset);
    static_assert(4 * kMaskWords == 32, "one warp clears them");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kUnitOffset + 2 * kUnitInts * 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = blockIdx.x / p.mt, m = blockIdx.x - share * p.mt;
    auto bar = [&](int i) { return smem_u32(bars + i); };
    int *status = &g_tree_status;

    griddep_launch_dependents();  // the merge waits for this grid to end
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(C::kQFull + t), 1);
            mbar_init(bar(C::kQEmpty + t), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(C::kSFull + 2 * t + i), 1);
                mbar_init(bar(C::kPFull + 2 * t + i), 4);
            }
            mbar_init(bar(C::kOFull + t), 1);
            mbar_init(bar(C::kOEmpty + t), kKeys ? 8 : 4);
            mbar_init(bar(C::kUFull + t), 1);
            mbar_init(bar(C::kUEmpty + t), 3 + 8);  // the K, V and MMA warps, the softmax warps
        }
        mbar_init(bar(C::kStateFull), 8);
        mbar_init(bar(C::kDrain), 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(C::kKVFull + s), 1);
            mbar_init(bar(C::kKVEmpty + s), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) odd_rows[lane] = 0;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    // The share [lo, lo + left) of the blocks: warp 3 finds its first unit, warp 2 what lies behind it.
    Unit u = {};
    int left = 0;
    if (warp == 2 || warp == 3) {
        const unsigned total = all_blocks<kBlock>(p), S = (total + p.shares - 1) / p.shares, lo = share * S;
        left = int(lo < total ? min(S, total - lo) : 0);
        if (warp == 3) {
            if (left > 0) u = find_block<kBlock>(p, lo);
        } else if (m == 0) {
            // Where the merge finds the pair that goes on behind this share: from the lengths alone, so that a launch
            // whose waits run out leaves the merge wrong numbers but no wrong addresses.
            int4 cut = make_int4(0, 0, 0, 0);
            if (left > 0) {
                const Unit at = find_block<kBlock>(p, lo + left - 1);
                const int rest = at.nb - at.j0 - 1;
                if (at.j0 < left && rest > 0) cut = make_int4(at.b, at.g, 1 + int((rest + S - 1) / S), at.tb);
            }
            if (lane == 0) p.cuts[share] = cut;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        const bool second = !kKeys && (2 * m + 1) * kTileM < p.rows;  // a second tile
        const uint64_t drain_ns = 1000000000ull;
        volatile int no_abort = 0;
        if (warp == 3) {
            // -------------------------------------------- planner: the units, and Q
            uint32_t q_loads = 0;  // per tile (both are loaded for every unit that has them)
            bool ok = true;
            u.holes = p.table != nullptr;  // (the first unit's entries are looked at block by block)
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                u.n = left > 0 ? min(left, u.nb - u.j0) : 0;
                if (p.table && qi > 0) {
                    // Ahead of the other warps: whether the unit needs looking at all.
                    const int *table = p.table + (size_t)u.b * p.max_pages;
                    const int last = min(u.keys, (u.j0 + u.n) * kBlock) - 1;
                    bool hole = false;
                    for (int i = ((u.j0 * kBlock) >> p.shift) + lane; u.n > 0 && i <= last >> p.shift; i += 32) {
                        const int page = table[i];
                        hole |= page < 0 || page >= p.num_pages;
                    }
                    u.holes = __any_sync(0xffffffffu, hole);
                }
                if (qi >= 2) ok = wait_warp(bar(C::kUEmpty + qs), ((qi >> 1) - 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    u.put(units + kUnitInts * qs);
                    mbar_arrive(bar(C::kUFull + qs));
                }
                __syncwarp();
                if (u.n == 0) break;
                for (int t = 0; t < (second ? 2 : 1); ++t) {
                    if (q_loads > 0) ok = wait_warp(bar(C::kQEmpty + t), (q_loads - 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(C::kQFull + t), C::kQBytes);
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_3d(smem_u32(sQ + t * C::kQBytes + c * C::kQChunkBytes), &tmQ, bar(C::kQFull + t), c * 64,
                                        (2 * m + t) * kTileM, u.b * p.Hkv + u.g);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                ++q_loads;
                left -= u.n;
                if (left <= 0) continue;
                u.j0 = 0;
                if (++u.g == p.Hkv) {
                    u.g = 0;
                    do {
                        load_sequence(p, ++u.b, u.len, u.tb);
                        u.keys = keys_of(p, u.len, u.tb);
                    } while (u.keys == 0);
                    u.nb = blocks_of<kBlock>(u.keys);
                }
            }
            __syncwarp();
            // Copies have to land before the CTA goes (bounded), whatever became of the other warps.
            if (!ok && lane == 0)
                for (int t = 0; t < (second ? 2 : 1); ++t)
                    if (q_loads > 0 && !mbar_wait_bounded(bar(C::kQFull + t), (q_loads - 1) & 1, drain_ns, &no_abort, status))
                        atomicOr(status, kStatusDrainTimeout);
            __syncwarp();
        } else if (warp == 0 || warp == 2) {
            // ------------------------------------- producers: warp 0 K, warp 2 V
            // Blocks alternate in the ring, K at even fills and V at odd ones; neither warp waits for the other's slots.
            const uint32_t kv = warp == 0 ? 0 : 1;
            const CUtensorMap *map = warp == 0 ? &tmK : &tmV;
            uint32_t blocks = 0;  // loaded so far
            bool ok = true;
            const int boxes = p.table && p.page_size < kBlock ? kBlock / p.page_size : 1;
            const int box_bytes = C::kChunkBytes / boxes;
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                u.get(units + kUnitInts * qs);
                __syncwarp();
                mbar_arrive_elect(bar(C::kUEmpty + qs));
                if (u.n == 0) break;
                // Lane i holds entry base + i of the table, and the one 32 behind it.
                const int *table = p.table ? p.table + (size_t)u.b * p.max_pages : nullptr;
                const int used = (u.keys + p.page_size - 1) >> p.shift;
                auto entry = [&](int i) { return table && i < used ? table[i] : -1; };
                int base = (u.j0 * kBlock) >> p.shift;
                int cur = entry(base + lane), nxt = entry(base + 32 + lane);
                for (int j = 0; j < u.n; ++j) {
                    const uint32_t fill = 2 * blocks + kv, slot = fill % C::kStages, round = fill / C::kStages;
                    if (round > 0) ok = wait_warp(bar(C::kKVEmpty + slot), (round - 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    const uint32_t fb = bar(C::kKVFull + slot), to = smem_u32(sKV + slot * C::kKVBytes);
                    if (lane == 0) mbar_arrive_expect_tx(fb, C::kKVBytes);
                    const int key = (u.j0 + j) * kBlock, first = key >> p.shift;
                    if (table && first >= base + 32) {
                        base += 32;
                        cur = nxt;
                        nxt = entry(base + 32 + lane);
                    }
                    for (int i = 0; i < boxes; ++i) {
                        const int page = table ? __shfl_sync(0xffffffffu, cur, (first - base + i) & 31) : u.b;
                        const int row = !table ? key : boxes > 1 ? 0 : key & (p.page_size - 1);
                        const int plane = page >= 0 && page < p.num_pages ? page * p.Hkv + u.g : p.num_pages * p.Hkv;
                        if (lane == 0)
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(to + c * C::kChunkBytes + i * box_bytes, map, fb, c * 64, row, plane);
                    }
                    __syncwarp();
                    ++blocks;
                }
            }
            __syncwarp();
            if (!ok && lane == 0)
                for (uint32_t s = kv; s < C::kStages; s += 2) {
                    if (2 * blocks <= s) continue;  // fills below 2 blocks + kv are out
                    const uint32_t last = (2 * blocks - 2 + kv - s) / C::kStages;  // round of the slot's last fill
                    if (!mbar_wait_bounded(bar(C::kKVFull + s), last & 1, drain_ns, &no_abort, status))
                        atomicOr(status, kStatusDrainTimeout);
                }
            __syncwarp();
            if (warp == 2) {
                // Sequences without a token: zeros, and a log-sum-exp of nothing.
                for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
                    int len, tb;
                    load_sequence(p, b, len, tb);
                    if (tb > 0) continue;
                    const size_t rows = (size_t)p.Hkv * p.rows, units16 = rows * (D / 8);
                    uint4 *o = reinterpret_cast<uint4 *>(p.o + (size_t)b * rows * D);
                    for (size_t i = lane; i < units16; i += 32) o[i] = make_uint4(0, 0, 0, 0);
                    if (p.lse)
                        for (size_t i = lane; i < rows; i += 32) p.lse[(size_t)b * rows + i] = -INFINITY;
                }
                __syncwarp();
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            constexpr uint32_t kIdescQK = idesc_bf16_f32(kTileM, kBlock, 0), kIdescPV = idesc_bf16_f32(kTileM, D, 1);
            uint32_t fills = 0;
            uint32_t q_used = 0;
            uint32_t p_odd = 0, o_odd = 0, used = 0;  // a bit a chain: waits for P, units done, whether there was one
            bool ok = true;
            const int chains = second ? 2 : 1;  // (kRows)
            auto wait_slot = [&](uint32_t f) {
                return wait_warp(bar(C::kKVFull + f % C::kStages), (f / C::kStages) & 1, p.wait_ns, abort_flag);
            };
            const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t dK = smem_desc_sw128(smem_u32(sKV), 16, 1024);
            const uint64_t dV = smem_desc_sw128(smem_u32(sKV), C::kChunkBytes, 1024);
            auto slot_off = [&](uint32_t f) { return uint64_t(f % C::kStages * (C::kKVBytes >> 4)); };
            auto issue_qk = [&](int t, int buf, uint32_t fK) {
                const uint64_t a0 = dQ + uint64_t((kKeys ? 0 : t) * (C::kQBytes >> 4)), b0 = dK + slot_off(fK);
#pragma unroll
                for (int g = 0; g < D / 64; ++g) {
                    uint64_t a[4], b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = a0 + uint64_t((g * C::kQChunkBytes + i * 32) >> 4);
                        b[i] = b0 + uint64_t((g * C::kChunkBytes + i * 32) >> 4);
                    }
                    tc_mma_ss_x4_elect(tmem_base + t * kTileM + buf * kBlock, a, b, kIdescQK, g > 0 ? 1u : 0u);
                }
            };
            auto issue_pv = [&](int t, int buf, uint32_t fV, bool acc) {
                const uint64_t b0 = dV + slot_off(fV);
#pragma unroll
                for (int g = 0; g < kBlock / 64; ++g) {
                    uint32_t a[4];
                    uint64_t b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = g * 4 + i;
                        a[i] = tmem_base + t * kTileM + buf * kBlock + kk * 8;
                        b[i] = b0 + uint64_t((kk * 16 * 128) >> 4);
                    }
                    tc_mma_ts_x4_elect(tmem_base + C::kOCol + t * D, a, b, kIdescPV, (acc || g > 0) ? 1u : 0u);
                }
            };
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                const int n = __shfl_sync(0xffffffffu, int(units[kUnitInts * qs + 3]), 0);
                mbar_arrive_elect(bar(C::kUEmpty + qs));
                if (n == 0) break;
                const uint32_t f0 = fills;  // K_j at f0 + 2 j, V_j behind it
                // The first product of each chain and buffer.
                ok = wait_warp(bar(C::kQFull), q_used & 1, p.wait_ns, abort_flag);
                if (ok && !kKeys && second) ok = wait_warp(bar(C::kQFull + 1), q_used & 1, p.wait_ns, abort_flag);
#pragma unroll 1
                for (int i = 0; i < (kKeys ? 4 : 2); ++i) {
                    const int j = kKeys ? i : 0, t = i & 1, buf = kKeys ? i >> 1 : 0;
                    if (!ok || j >= n || (!kKeys && t >= chains)) break;
                    ok = wait_slot(f0 + 2 * j);
                    if (!ok) break;
                    tc_fence_after();
                    issue_qk(t, buf, f0 + 2 * j);
                    tc_commit_elect(bar(C::kSFull + 2 * t + buf));
                    if (j == n - 1) tc_commit_elect(bar(C::kQEmpty + (kKeys ? 0 : t)));  // Q's last product
                }
                ++q_used;
                for (int j = 0; ok && j < n; ++j) {
                    const uint32_t fV = f0 + 2 * j + 1;
                    bool v_ready = false;
#pragma unroll 1
                    for (int i = 0; i < (kKeys ? 1 : 2); ++i) {
                        const int t = kKeys ? j & 1 : i, buf = kKeys ? j >> 1 & 1 : 0, tb = 2 * t + buf;
                        if (!kKeys && i >= chains) break;
                        ok = wait_warp(bar(C::kPFull + tb), p_odd >> tb & 1, p.wait_ns, abort_flag);
                        if (!ok) break;
                        p_odd ^= 1u << tb;
                        const bool first = kKeys ? j < 2 : j == 0;
                        if (first && (used >> t & 1)) {
                            ok = wait_warp(bar(C::kOEmpty + t), ~(o_odd >> t) & 1, p.wait_ns, abort_flag);
                            if (!ok) break;
                        }
                        if (!v_ready) {
                            ok = wait_slot(fV);
                            if (!ok) break;
                            v_ready = true;
                        }
                        tc_fence_after();
                        issue_pv(t, buf, fV, !first);
                        if (kKeys || t == chains - 1) tc_commit_elect(bar(C::kKVEmpty + fV % C::kStages));
                        const int next = j + (kKeys ? 4 : 1);  // into the buffer that P has been read from
                        if (next < n) {
                            ok = wait_slot(f0 + 2 * next);
                            if (!ok) break;
                            issue_qk(t, buf, f0 + 2 * next);
                            tc_commit_elect(bar(C::kSFull + tb));
                            if (next == n - 1) tc_commit_elect(bar(C::kQEmpty + (kKeys ? 0 : t)));
                        }
                        if (j + (kKeys ? 2 : 1) >= n) {  // the chain's last block
                            tc_commit_elect(bar(C::kOFull + t));
                            o_odd ^= 1u << t;
                            used |= 1u << t;
                        }
                    }
                }
                fills = f0 + 2 * n;
            }
            tc_commit_elect(bar(C::kDrain));
            if (!wait_warp(bar(C::kDrain), 0, drain_ns, &no_abort) && lane == 0)
                atomicOr(status, kStatusDrainTimeout);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------- softmax / epilogue
        const int t = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_off = uint32_t(quarter * 32) << 16;
        const uint32_t tS0 = tmem_base + lane_off + t * kTileM, tO = tmem_base + lane_off + C::kOCol;
        const int row0 = kKeys ? 0 : (2 * m + t) * kTileM, row = row0 + r;
        const int token = row % p.T;
        const bool has_rows = row0 + quarter * 32 < p.rows;  // of this warp; the others only keep step
        const bool has_tile = row0 < p.rows;
        const bool both = kKeys || (2 * m + 1) * kTileM < p.rows;  // whether chain 1 is at work
        const float sl2 = p.scale_log2;
        const int limit = p.rows - row0;  // rows of the tile in use, if below 128
        float *turn = reinterpret_cast<float *>(smem + C::kTurnOffset) + (warp - 4) * kTurnFloats;
        float2 *states = reinterpret_cast<float2 *>(smem + C::kStateOffset);  // [unit parity][chain][row]
        uint32_t s_odd = 0, o_waits = 0, o_waits1 = 0;  // s_odd: a bit a buffer
        uint32_t kv_base = 0;
        bool ok = true;
        for (uint32_t qi = 0; ok; ++qi) {
            const uint32_t qs = qi & 1;
            ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
            if (!ok) break;
            u.get(units + kUnitInts * qs);
            __syncwarp();
            mbar_arrive_elect(bar(C::kUEmpty + qs));
            if (u.n == 0) break;
            const uint32_t f0 = kv_base;
            kv_base += 2 * u.n;
            if (!has_tile) continue;
            const bool live = row < p.rows && token < u.tb;
            // What the row sees of the drafted tokens.
            uint32_t seen[kMaskWords];
#pragma unroll
            for (int w = 0; w < kMaskWords; ++w) seen[w] = 0;
            if ((u.j0 + u.n) * (long long)kBlock > u.len && live) {
                const int words = (p.T + 63) / 64;
                const unsigned long long *mrow = p.mask ? p.mask + ((size_t)u.b * p.T + token) * words : nullptr;
                const int end = u.keys - u.len;  // drafted keys that exist
#pragma unroll
                for (int w = 0; w < kMaskWords / 2; ++w) {
                    const int in = mrow ? end : min(end, token + 1);  // a chain sees what is before it
                    unsigned long long x = !mrow ? ~0ull : w < words ? mrow[w] : 0ull;
                    if (in < 64 * w + 64) x = in <= 64 * w ? 0ull : x & ((1ull << (in - 64 * w)) - 1);
                    seen[2 * w] = uint32_t(x);
                    seen[2 * w + 1] = uint32_t(x >> 32);
                }
            }
            const int *table = u.holes ? p.table + (size_t)u.b * p.max_pages : nullptr;  // null: nothing to look at
            const int boxes = p.page_size < kBlock ? kBlock / p.page_size : 1;  // (with a table only)
            const int used = (u.keys + p.page_size - 1) >> p.shift;
            // Lane i looks at entry i of a block's pages, one block ahead.
            auto page_of = [&](int j) {
                const int i = (((u.j0 + j) * kBlock) >> p.shift) + lane;
                return table && lane < boxes && i < used && j < u.n ? table[i] : -1;
            };
            constexpr int kStep = kKeys ? 2 : 1, kQuads = kBlock / 32;
            const int jt = kKeys ? t : 0;
            int ahead = page_of(jt);
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = jt; j < u.n; j += kStep) {
                uint32_t on_page = ~0u;
                if (table) {
                    on_page = __ballot_sync(0xffffffffu, ahead >= 0 && ahead < p.num_pages);
                    ahead = page_of(j + kStep);
                }
                const int buf = kKeys ? j >> 1 & 1 : 0;
                const uint32_t tS = tS0 + buf * kBlock;
                ok = wait_warp(bar(C::kSFull + 2 * t + buf), s_odd >> buf & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                s_odd ^= 1u << buf;
                // S complete: so are all products before it, and K's slot is free once the last chain to use it says so.
                if (quarter == 0 && (kKeys || t == (both ? 1 : 0)))
                    mbar_arrive_elect(bar(C::kKVEmpty + (f0 + 2 * j) % C::kStages));
                if (has_rows) {
                    tc_fence_after();
                    uint32_t sr[kQuads][32];
#pragma unroll
                    for (int c = 0; c < kQuads; ++c) tmem_ld32(tS + c * 32, sr[c]);
                    tmem_wait_ld();
                    float s[kBlock];
#pragma unroll
                    for (int c = 0; c < kQuads; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(sr[c][i]);
                    const int kv0 = (u.j0 + j) * kBlock;
                    const uint32_t all = boxes >= 32 ? ~0u : (1u << boxes) - 1;
                    if (kv0 + kBlock > u.len || (table && (on_page & all) != all)) {
#pragma unroll
                        for (int c = 0; c < kQuads; ++c) {
                            uint32_t bits = mask_bits(seen, kv0 + 32 * c - u.len);
                            if (table) {
                                const int per = 32 / (p.page_size < 32 ? p.page_size : 32);  // pages in 32 keys: 1 or 2
                                const int at = p.page_size < kBlock ? 32 * c / p.page_size : 0;
                                if (!(on_page >> at & 1)) bits &= per == 2 ? 0xffff0000u : 0u;
                                if (per == 2 && !(on_page >> (at + 1) & 1)) bits &= 0x0000ffffu;
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(bits >> i & 1)) s[c * 32 + i] = -INFINITY;
                        }
                    }
                    auto block_max = [&]() {
                        float mq[kQuads];
#pragma unroll
                        for (int c = 0; c < kQuads; ++c) {
                            float x = fmax3(s[32 * c], s[32 * c + 1], s[32 * c + 2]);
#pragma unroll
                            for (int i = 3; i < 31; i += 2) x = fmax3(x, s[32 * c + i], s[32 * c + i + 1]);
                            mq[c] = fmaxf(x, s[32 * c + 31]);
                        }
                        if constexpr (kQuads == 2) return fmaxf(mq[0], mq[1]);
                        else return fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
                    };
                    auto exp_block = [&](float neg_m) {
                        float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < kQuads; ++c) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float x0, x1;
                                ffma2(x0, x1, s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1], sl2, sl2, neg_m, neg_m);
                                const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                                const int a = (i & 3) * 2;
                                fadd2(ls[a], ls[a + 1], p0, p1);
                                pk[i] = pack_bf16x2(p0, p1);
                            }
                            tmem_st16(tS + c * 16, pk);
                        }
                        return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
                    };
                    // The reference maximum is exact for the first block that shows the row a key, and kept while the
                    // exponentials cannot overflow (their sum below 2^60); see fwd_kernel.cuh.
                    float corr = 1.f, l_blk;
                    bool again = false, twice = false;
                    do {
                        if (m_run == -INFINITY || again) {
                            const float m_new = fmaxf(m_run, block_max() * sl2);
                            if (again && m_new > m_run) corr = fast_exp2(m_run - m_new);
                            m_run = m_new;
                        }
                        l_blk = exp_block(m_run == -INFINITY ? 0.f : -m_run);
                        again = !again && __any_sync(0xffffffffu, !(l_blk < 0x1p60f));
                        if (again) {
                            tmem_wait_st();
                            twice = true;
                        }
                    } while (again);
                    if (twice && j > jt && __any_sync(0xffffffffu, corr != 1.f)) {
                        if constexpr (kKeys) {
                            // S(j) was issued ahead of the chain's last product into O: wait for that (its V slot, which
                            // nobody can have filled and freed again before this block's P).
                            const uint32_t f = f0 + 2 * (j - kStep) + 1;
                            ok = wait_warp(bar(C::kKVEmpty + f % C::kStages), (f / C::kStages) & 1, p.wait_ns, abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t ov[32];
                            tmem_ld32(tO + t * D + c * 32, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * corr);
                            tmem_st32(tO + t * D + c * 32, ov);
                        }
                    }
                    l_run = l_run * corr + l_blk;
                    tmem_wait_st();
                    tc_fence_before();
                }
                if ((u.j0 + j + 1) * kBlock > u.len && (kKeys || t == 0)) {
                    // (the other chain's product of this block is issued behind this one's)
                    const uint32_t fV = f0 + 2 * j + 1, slot = fV % C::kStages;
                    ok = wait_warp(bar(C::kKVFull + slot), (fV / C::kStages) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    const int kv0 = (u.j0 + j) * kBlock, at = max(u.len - kv0, 0);
                    clean_rows<C::kChunks, kBlock>(sKV + slot * C::kKVBytes, quarter, at, u.keys - kv0, kv0 + at - u.len,
                                                   odd_rows + (qi & 3) * kMaskWords);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                mbar_arrive_elect(bar(C::kPFull + 2 * t + buf));
            }
            if (!ok) break;

            // Epilogue: to the outputs where the unit is all of the pair, else to a partial.
            const bool whole = u.n == u.nb;
            const size_t out_row = ((size_t)u.b * p.Hkv + u.g) * p.rows + row0;
            const size_t part_row = (size_t)(2 * share + (u.j0 > 0 ? 0 : 1)) * p.rows + row0;
            const bool has1 = kKeys && u.n > 1;  // whether chain 1 has an accumulator of this unit
            float f[2] = {0.f, 0.f}, L, sum;      // factors of the accumulators; the row's log-sum-exp (log2) and sum
            if constexpr (kKeys) {
                float2 *mine = states + (qi & 1) * 2 * kTileM;
                mine[t * kTileM + r] = make_float2(m_run, l_run);
                __syncwarp();
                mbar_arrive_elect(bar(C::kStateFull));
                ok = wait_warp(bar(C::kStateFull), qi & 1, p.wait_ns, abort_flag);
                if (ok) ok = wait_warp(bar(C::kOFull), o_waits & 1, p.wait_ns, abort_flag);
                if (ok && has1) ok = wait_warp(bar(C::kOFull + 1), o_waits1 & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                ++o_waits;
                if (has1) ++o_waits1;
                const float2 a = mine[r], c = mine[kTileM + r];
                const float top = fmaxf(a.x, c.x), ref = top == -INFINITY ? 0.f : top;
                f[0] = fast_exp2(a.x - ref);
                f[1] = fast_exp2(c.x - ref);
                sum = f[0] * a.y + f[1] * c.y;
                L = top + __log2f(sum);
                f[0] /= sum;
                f[1] /= sum;
            } else {
                ok = wait_warp(bar(C::kOFull + t), o_waits & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                ++o_waits;
                sum = l_run;
                f[0] = 1.f / sum;
                L = m_run + __log2f(sum);
            }
            tc_fence_after();
            const uint32_t *odd = odd_rows + (qi & 3) * kMaskWords;
            const bool any_odd = __any_sync(0xffffffffu, lane < kMaskWords && odd[lane & 7] != 0);
            if (t == 0 && quarter == 0 && lane < kMaskWords) odd_rows[((qi + 2) & 3) * kMaskWords + lane] = 0;
            if (has_rows) {
                const bool any = live && sum != 0.f;  // (NaN stays NaN)
                // A thread holds a row; the warp turns 64 bytes of each of its 32 rows at a time through shared memory, so
                // that four lanes store them.
                const int first = quarter * 32 + (lane >> 2);
                constexpr int kCols = kKeys ? D / 2 : D;  // of this warp
                const int col0 = kKeys ? t * kCols : 0;
#pragma unroll 1
                for (int c = 0; c < kCols / 32; ++c) {
                    const int col = col0 + c * 32;
                    uint32_t ov[32], ow[32];
                    float x[32];
                    tmem_ld32(tO + (kKeys ? 0 : t * D) + col, ov);
                    if (has1) tmem_ld32(tO + D + col, ow);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(ov[i]) * f[0];
                    if (has1)
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] += __uint_as_float(ow[i]) * f[1];
                    if (!any)
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0.f;
                    if (whole) {
                        uint4 pk[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            pk[g] = make_uint4(pack_bf16x2(x[8 * g], x[8 * g + 1]), pack_bf16x2(x[8 * g + 2], x[8 * g + 3]),
                                               pack_bf16x2(x[8 * g + 4], x[8 * g + 5]), pack_bf16x2(x[8 * g + 6], x[8 * g + 7]));
                        __syncwarp();
#pragma unroll
                        for (int g = 0; g < 4; ++g) *reinterpret_cast<uint4 *>(turn + lane * kTurnStride + g * 4) = pk[g];
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (first + 8 * k < limit)
                                *reinterpret_cast<uint4 *>(p.o + (out_row + first + 8 * k) * D + col + (lane & 3) * 8) =
                                    *reinterpret_cast<const uint4 *>(turn + (8 * k + (lane >> 2)) * kTurnStride + (lane & 3) * 4);
                    } else {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            __syncwarp();
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const float *y = x + half * 16 + g * 4;
                                *reinterpret_cast<float4 *>(turn + lane * kTurnStride + g * 4) = make_float4(y[0], y[1], y[2], y[3]);
                            }
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (first + 8 * k < limit)
                                    *reinterpret_cast<float4 *>(p.part_o + (part_row + first + 8 * k) * D + col + half * 16 + (lane & 3) * 4) =
                                        *reinterpret_cast<const float4 *>(turn + (8 * k + (lane >> 2)) * kTurnStride + (lane & 3) * 4);
                        }
                    }
                }
                if (any_odd) {
                    __syncwarp();  // behind the warp's stores
#pragma unroll 1
                    for (int w = 0; w < kMaskWords; ++w)
                        for (uint32_t bits = any ? odd[w] & mask_bits(seen, 32 * w) : 0u; bits; bits &= bits - 1) {
                            const int key = u.len + 32 * w + __ffs(bits) - 1;
                            const int page = p.table ? p.table[(size_t)u.b * p.max_pages + (key >> p.shift)] : u.b;
                            const int in = p.table ? key & (p.page_size - 1) : key;
                            const __nv_bfloat16 *v = p.v + (((size_t)page * p.Hkv + u.g) * p.page_size + in) * D + col0;
                            if (whole) add_odd(p.o + (out_row + r) * D + col0, v, kCols);
                            else add_odd(p.part_o + (part_row + r) * D + col0, v, kCols);
                        }
                }
                if ((!kKeys || t == 0) && r < limit) {
                    if (!whole) p.part_lse[part_row + r] = any ? L : -INFINITY;
                    else if (p.lse) p.lse[out_row + r] = any ? L * 0.69314718055994531f : -INFINITY;
                }
            }
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(bar(C::kOEmpty + (kKeys ? 0 : t)));
            if (has1) mbar_arrive_elect(bar(C::kOEmpty + 1));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// The rows of the pair that goes on behind share blockIdx.x, a warp each: their
// partials (2 x + 1, 2 (x + 1), 2 (x + 2), ...) by the log-sum-exps' weights.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const Params p) {
    constexpr int kCols = D / 32, kAhead = 8;
    griddep_wait();
    const int4 cut = p.cuts[blockIdx.x];
    const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (cut.z == 0 || row >= p.rows) return;
    auto at = [&](int i) { return (size_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.rows + row; };
    auto lse = [&](int i) { return i < cut.z ? p.part_lse[at(i)] : -INFINITY; };
    float top = -INFINITY, sum = 0.f, acc[kCols] = {};
    for (int i = lane; i < cut.z; i += 32) top = fmaxf(top, lse(i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float ref = top == -INFINITY ? 0.f : top;
    for (int i0 = 0; i0 < cut.z; i0 += kAhead) {
        float v[kAhead][kCols], w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            w[k] = lse(i0 + k);
            if (i0 + k < cut.z) {
                const float *x = p.part_o + at(i0 + k) * D + lane * kCols;
#pragma unroll
                for (int c = 0; c < kCols; ++c) v[k][c] = x[c];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            w[k] = fast_exp2(w[k] - ref);
            sum += w[k];
            if (i0 + k < cut.z)
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[c] += w[k] * v[k][c];
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
    const size_t out = ((size_t)cut.x * p.Hkv + cut.y) * p.rows + row;
    uint32_t packed[kCols / 2];
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) packed[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    __nv_bfloat16 *o = p.o + out * D + lane * kCols;
    if constexpr (kCols == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t *>(o) = packed[0];
    if (lane == 0 && p.lse) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

struct Layout {
    int mt, shares;
    size_t cuts, part_o, part_lse, bytes;
};
Layout layout_of(int B, int G, int Hkv, int T, int d, long long cap, int num_sms) {
    Layout l;
    const size_t rows = size_t(G) * T;
    l.mt = int((rows + 2 * kTileM - 1) / (2 * kTileM));
    const int block = block_keys(rows <= kTileM);
    const long long most = (long long)B * Hkv * ((cap + block - 1) / block);
    const int groups = num_sms / l.mt > 0 ? num_sms / l.mt : 1;
    l.shares = int(most < groups ? most : groups);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    l.cuts = 0;
    l.part_o = up(size_t(l.shares) * sizeof(int4));
    l.part_lse = l.part_o + up(2 * size_t(l.shares) * rows * d * sizeof(float));
    l.bytes = l.part_lse + up(2 * size_t(l.shares) * rows * sizeof(float));
    return l;
}

template <int D, bool kKeys>
int launch(const DecodeTreeLaunch &a, const Layout &l, cudaStream_t stream) {
    using C = Cfg<D, kKeys>;
    const int G = a.Hq / a.Hkv;
    CUtensorMap mq, mk, mv;
    const uint32_t box = uint32_t(a.table && a.page_size < C::kBlock ? a.page_size : C::kBlock);
    const uint64_t planes = uint64_t(a.num_pages) * a.Hkv;
    if (!encode_bf16_3d(&mq, a.q, D, uint64_t(G) * a.T, uint64_t(a.B) * a.Hkv, 64, kTileM) ||
        !encode_bf16_3d(&mk, a.kpages, D, uint64_t(a.page_size), planes, 64, box) ||
        !encode_bf16_3d(&mv, a.vpages, D, uint64_t(a.page_size), planes, 64, box))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (drafted tokens)");
    Params p = {};
    p.seqlens = a.seqlens;
    p.draft_lens = a.draft_lens;
    p.table = a.table;
    p.mask = a.mask;
    p.v = static_cast<const __nv_bfloat16 *>(a.vpages);
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.lse = a.lse;
    p.cuts = reinterpret_cast<int4 *>(a.workspace + l.cuts);
    p.part_o = reinterpret_cast<float *>(a.workspace + l.part_o);
    p.part_lse = reinterpret_cast<float *>(a.workspace + l.part_lse);
    p.B = a.B;
    p.Hkv = a.Hkv;
    p.G = G;
    p.T = a.T;
    p.rows = G * a.T;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.shift = a.page_shift;
    p.cap = a.page_size * a.max_pages;
    p.max_pages = a.max_pages;
    p.mt = l.mt;
    p.shares = l.shares;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    auto kernel = tree_kernel<D, kKeys>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncGetAttributes(tree_kernel)");
        if (fa.numRegs != kLaunchRegs || fa.maxThreadsPerBlock < kThreads)
            return note_cuda_error(cudaErrorInvalidConfiguration, "tree_kernel register count differs from the setmaxnreg split");
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(tree_kernel)");
        if (dev >= 0) attr_set[dev] = true;
    }
    kernel<<<dim3(unsigned(l.shares * l.mt)), dim3(kThreads), C::kSmemBytes, stream>>>(mq, mk, mv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return note_cuda_error(e, "tree_kernel launch");
    if (l.shares == 1) return 0;  // nothing is cut
    e = dec::launch_programmatic(merge_kernel<D>, dim3(unsigned(l.shares), unsigned((p.rows + kMergeWarps - 1) / kMergeWarps)),
                                 dim3(kMergeWarps * 32), 0, stream, p);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "merge_kernel (drafted tokens) launch");
}

}  // namespace dtree

size_t decode_tree_workspace_bytes(int B, int G, int Hkv, int T, int d, long long cap, int num_sms) {
    return dtree::layout_of(B, G, Hkv, T, d, cap, num_sms).bytes;
}

int decode_tree_launch(const DecodeTreeLaunch &a, cudaStream_t stream) {
    using namespace dtree;
    const int G = a.Hq / a.Hkv;
    const Layout l = layout_of(a.B, G, a.Hkv, a.T, a.d, (long long)a.page_size * a.max_pages, a.num_sms);
    const bool keys = G * a.T <= kTileM;
    if (a.d == 64) return keys ? launch<64, true>(a, l, stream) : launch<64, false>(a, l, stream);
    return keys ? launch<128, true>(a, l, stream) : launch<128, false>(a, l, stream);
}

cudaError_t decode_tree_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_tree_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_tree_status, &zero, sizeof(int));
}

}  // namespace attn
