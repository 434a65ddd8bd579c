// decode_tree_sm103.cu -- attention of several drafted tokens per sequence over a
// cache in pages (or contiguous): each attends all cached keys and, of the drafted
// keys behind them, those that the tree's mask names.
//
// For KV head g of sequence b the rows are a matrix of G T queries (head of the
// group, token), all against the same keys:
//     s = scale q k^T  (-inf where the mask hides the key),  o = softmax(s) v.
// The keys are read once for all rows.  With R = G T rows a key costs 4 d bytes and
// 4 d R flops: below some 280 rows HBM bounds it, above that the tensor cores.  So
// S = Q K^T and P V are tcgen05 products of 128 rows whatever R is; a tile of few rows
// is idle for the most part, but still faster than HBM.
//
// A CTA an SM, persistent: warps that load, issue MMAs and plan, and two chains of
// four softmax warps, as in fwd_kernel.cuh.
//   pairs_kernel (R <= 128): each chain is a pipeline of its own, with loading and
//     issuing warps, a ring of 64-key blocks, and two score buffers, so that the
//     products' latency is not in its way.  The chains take the two halves of the CTA's
//     share, one from its begin on, one from its end back: when one starts or ends a
//     pair, the other one keeps the memory busy, and the pair that both have a part of
//     comes last in both, so that they add up their states in the CTA.
//   rows_kernel (R > 128): the chains hold two tiles of rows, and both visit every
//     block of 128 keys in the ring; units of 256 rows, `mt` units a KV head, side by
//     side on mt SMs so that all but one find the keys in L2.
// The blocks of all (sequence, KV head) pairs, in that order, are cut into equal
// shares, one a CTA or group of mt CTAs: nothing depends on how ragged the
// lengths are.  A pair that lies in one share is written out at once; one that is cut
// goes through partials: share s writes its first segment's to slot 2 s (a pair
// that began before) and its last one's to 2 s + 1 (a pair that goes on), and
// merge_kernel adds up slot 2 s + 1, 2 (s + 1), 2 (s + 2), ...  Where no pair has many
// blocks, shares end with pairs instead, and there is nothing to merge.
//
// Pages: a block of keys is one box, or several where pages are smaller, each from
// the page that the table names; a box on no page is filled with zeros by coordinates
// past the end.  Columns past the last key, on no page, or hidden by the mask become
// -inf before the softmax.  A probability of 0 does not hide a V of infinity or NaN
// from the product, so the softmax warps clean the blocks that hold drafted keys
// before they hand P over: rows behind the last key, which may hold anything, become
// zeros, and so do elements of drafted rows that are not finite, which the epilogue
// then adds to the rows that see them.
//
// What it measured (kernels alone, d = 128, 64 query and 8 KV heads; the copy rate is 6.75 TB/s):
//   one token, 64 users of 8001 .. 16001 keys: 436 us contiguous (7.1 TB/s), 459 in pages of 16 (6.9);
//   16 tokens, 32 users of up to 8192 keys, pages of 64: 148 us (5.8 TB/s), of which some 15 are the start, the last
//     CTAs' late end (they differ by 6%, as the memory serves some SMs better) and the merge;
//   64 tokens, 16 users of up to 32768 keys: 569 to 582 us, 1570 TFLOP/s (all 512 rows of a pair counted), 0.8 of the rate of a
//     large matrix product: some 3000 clocks a block of 128 keys, of which the products need 2048;
//   8 tokens, 128 users of 512 keys: 61 to 66 us; a pair costs its start and end (4 us) besides its keys.
// One kernel for both, of 128-key blocks with both chains at every block, took 524 us for the first (pages of 128), 167 for
// the second and 655 for the third.
//
// Precision: scores, maxima, sums, partials in fp32; probabilities are rounded to
// bf16 for the product with V, whose instruction takes both operands in one 16-bit type;
// outputs are rounded once more.  Outputs are 0.0023 off (relative, against 64 bits),
// with probabilities in 32 bits they would be 0.0017 off, by their own rounding.
// Probabilities as two bf16 terms would get there, for twice the product with V, and
// twice what the softmax warps pack and store; not taken, nor measured.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

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
constexpr int kMaskWords = 8;  // 32-bit words of a row's mask: 256 drafted tokens
constexpr int kLongUnit = 16;  // blocks; a look at the pages of as many is not felt
constexpr int kUnitInts = 12;  // of a unit in the queue
constexpr int kMergeWarps = 8;
constexpr uint64_t kDrainNs = 1000000000ull;  // for copies and products in flight when a CTA gives up
constexpr int kSmemMax = 227 * 1024;

struct Params {
    const int *seqlens, *draft_lens, *table;
    const unsigned long long *mask;
    const __nv_bfloat16 *v;
    __nv_bfloat16 *o;
    float *lse;                // natural log, or null
    float *part_o, *part_lse;  // [2 shares][rows][D], [2 shares][rows] (log2 units)
    int4 *cuts;                // [shares]: {b, g, partials, 0} of the pair that goes on behind a share
    int B, Hkv, T, rows;
    int num_pages, page_size, shift, cap, max_pages;
    int mt, shares;
    bool whole;          // shares end with pairs
    bool wide;           // outputs and partials are 32-byte aligned
    int q_rows;          // pairs_kernel: rows of Q in shared memory
    float scale_log2;
    unsigned long long wait_ns;
};

// A piece of work: blocks [j0, j0 + n) of the nb blocks of pair (b, g); n = 0: the end.  holes: some of its entries may be
// no page.
// joint: the other chain has the rest of the CTA's part of the pair.
struct Unit {
    int b, g, j0, n, nb, len, tb, keys, holes, joint;
    __device__ __forceinline__ void put(volatile int *e) const {
        e[0] = b, e[1] = g, e[2] = j0, e[3] = n, e[4] = nb, e[5] = len, e[6] = tb, e[7] = keys, e[8] = holes, e[9] = joint;
    }
    __device__ __forceinline__ void get(const volatile int *e) {
        b = e[0], g = e[1], j0 = e[2], n = e[3], nb = e[4], len = e[5], tb = e[6], keys = e[7], holes = e[8], joint = e[9];
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

// A share [lo, lo + left) of the blocks, S in a full one.
struct Share {
    unsigned lo, S;
    int left;
};
template <int kBlock>
__device__ __forceinline__ Share share_of(const Params &p, int share) {
    const unsigned total = all_blocks<kBlock>(p);
    Share s;
    s.S = (total + p.shares - 1) / p.shares;
    s.lo = min(share * s.S, total);
    unsigned end = min(s.lo + s.S, total);
    if (p.whole) {  // on to the pairs' ends
        auto up = [&](unsigned x) {
            if (x == total) return x;
            const Unit u = find_block<kBlock>(p, x);
            return u.j0 > 0 ? x + u.nb - u.j0 : x;
        };
        s.lo = up(s.lo);
        end = up(end);
    }
    s.left = int(end - s.lo);
    return s;
}

// Where the merge finds the pair that goes on behind a share: from the lengths alone, so that a launch whose waits run out
// leaves the merge wrong numbers but no wrong addresses.
template <int kBlock>
__device__ __forceinline__ void write_cut(const Params &p, int share, const Share &s) {
    int4 cut = make_int4(0, 0, 0, 0);
    if (s.left > 0) {
        const Unit at = find_block<kBlock>(p, s.lo + s.left - 1);
        const int rest = at.nb - at.j0 - 1;
        if (at.j0 < s.left && rest > 0) cut = make_int4(at.b, at.g, 1 + int((rest + s.S - 1) / s.S), 0);
    }
    if ((threadIdx.x & 31) == 0) p.cuts[share] = cut;
}

// On to the pair behind; call only while a block is left.
template <int kBlock>
__device__ __forceinline__ void next_pair(const Params &p, Unit &u) {
    u.j0 = 0;
    if (++u.g < p.Hkv) return;
    u.g = 0;
    do {
        load_sequence(p, ++u.b, u.len, u.tb);
        u.keys = keys_of(p, u.len, u.tb);
    } while (u.keys == 0);
    u.nb = blocks_of<kBlock>(u.keys);
}

// Back to the end of the pair before; call only while a block is left there.
template <int kBlock>
__device__ __forceinline__ void previous_pair(const Params &p, Unit &u) {
    if (--u.g < 0) {
        u.g = p.Hkv - 1;
        do {
            load_sequence(p, --u.b, u.len, u.tb);
            u.keys = keys_of(p, u.len, u.tb);
        } while (u.keys == 0);
        u.nb = blocks_of<kBlock>(u.keys);
    }
    u.j0 = u.nb;
}

// Whether an entry of the unit's blocks is no page (all lanes of the calling warp).
template <int kBlock>
__device__ __forceinline__ bool look_for_holes(const Params &p, const Unit &u) {
    const int *table = p.table + (size_t)u.b * p.max_pages;
    const int last = (min(u.keys, (u.j0 + u.n) * kBlock) - 1) >> p.shift;
    bool hole = false;
    for (int i = ((u.j0 * kBlock) >> p.shift) + int(threadIdx.x & 31); u.n > 0 && i <= last; i += 32) {
        const int page = table[i];
        hole |= page < 0 || page >= p.num_pages;
    }
    return __any_sync(0xffffffffu, hole);
}

// Where a unit's blocks lie: lane i holds entry base + i of its row of the table, and the one 32 behind it.
template <int kBlock>
struct Pages {
    const int *table;
    int base, used, cur, nxt;
    __device__ __forceinline__ void start(const Params &p, const Unit &u) {
        table = p.table ? p.table + (size_t)u.b * p.max_pages : nullptr;
        used = (u.keys + p.page_size - 1) >> p.shift;
        base = (u.j0 * kBlock) >> p.shift;
        cur = entry(base);
        nxt = entry(base + 32);
    }
    __device__ __forceinline__ int entry(int first) const {
        const int i = first + int(threadIdx.x & 31);
        return table && i < used ? table[i] : -1;
    }
    // The block that starts at `key`, chunk by chunk to `to`; all lanes of the warp, in the blocks' order.
    template <int kChunks>
    __device__ __forceinline__ void load(const Params &p, const Unit &u, int key, const CUtensorMap *map, uint32_t full,
                                         uint32_t to) {
        constexpr int kChunkBytes = kBlock * 128;
        const int lane = threadIdx.x & 31;
        const int none = p.num_pages * p.Hkv;
        if (!table || p.page_size >= kBlock) {
            int plane = u.b * p.Hkv + u.g, row = key;
            if (table) {
                const int page = take(p, key);
                plane = page >= 0 && page < p.num_pages ? page * p.Hkv + u.g : none;
                row = key & (p.page_size - 1);
            }
            if (lane == 0)
#pragma unroll
                for (int c = 0; c < kChunks; ++c) tma_load_3d(to + c * kChunkBytes, map, full, c * 64, row, plane);
        } else {
            const int boxes = kBlock / p.page_size, bytes = p.page_size * 128;
            take(p, key);
            const int mine = cur >= 0 && cur < p.num_pages ? cur * p.Hkv + u.g : none;
            const int at = ((key >> p.shift) - base) & 31;
#pragma unroll 4
            for (int i = 0; i < boxes; ++i) {
                const int plane = __shfl_sync(0xffffffffu, mine, at + i);
                if (lane == 0)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(to + c * kChunkBytes + i * bytes, map, full, c * 64, 0, plane);
            }
        }
        __syncwarp();
    }

  private:
    __device__ __forceinline__ int take(const Params &p, int key) {
        const int first = key >> p.shift;
        if (first >= base + 32) {
            base += 32;
            cur = nxt;
            nxt = entry(base + 32);
        }
        return __shfl_sync(0xffffffffu, cur, (first - base) & 31);
    }
};

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

// The 64 scores at tS in TMEM that the row does not see become -inf: keys on no page (on_page: a bit a page of the block),
// and of the keys from the drafted ones on (u: the number of the first score's; negative: cached) those from `end` on and
// those without a bit in w.  For pairs_kernel: few of its blocks need it, and the others would carry its code through their
// loop (128 users of 512 keys, 8 tokens 67 us, now 60; 32 users of up to 16384 keys, 16 tokens, d = 64 162, now 156).  In
// rows_kernel, where a block has twice the keys, the mask stays in registers (38 users of 64 keys, 64 tokens 37 us, out of
// line 39), in a loop of its own.
__device__ __noinline__ void hide_scores(uint32_t tS, int u, int end, unsigned long long w0, unsigned long long w1,
                                         unsigned long long w2, unsigned long long w3, uint32_t on_page, int page_size) {
    auto word = [&](int i) {
        const int left = end - 32 * i;
        if (i < 0) return ~0u;
        if (i >= kMaskWords || left <= 0) return 0u;
        const unsigned long long w = i < 2 ? w0 : i < 4 ? w1 : i < 6 ? w2 : w3;
        const uint32_t x = uint32_t(i & 1 ? w >> 32 : w);
        return left < 32 ? x & ((1u << left) - 1) : x;
    };
    uint32_t x[2][32];
    __syncwarp();
    tmem_ld32(tS, x[0]);
    tmem_ld32(tS + 32, x[1]);
    tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 2; ++h, u += 32) {
        uint32_t bits = __funnelshift_r(word(u >> 5), word((u >> 5) + 1), u & 31);
        // Pages of 16: two in 32 keys.
        const int at = page_size < 64 ? 32 * h / page_size : 0;
        if (!(on_page >> at & 1)) bits &= page_size == 16 ? 0xffff0000u : 0u;
        if (page_size == 16 && !(on_page >> (at + 1) & 1)) bits &= 0x0000ffffu;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(bits >> i & 1)) x[h][i] = 0xff800000u;  // -inf
        __syncwarp();
        tmem_st32(tS + 32 * h, x[h]);
    }
    tmem_wait_st();
}

// What a row sees of a unit's drafted tokens, 64 a word; loaded ahead, looked at where the blocks end.
struct Seen {
    unsigned long long w[kMaskWords / 2] = {};
    int b = -1;  // whose they are: the KV heads of a sequence have the same
    __device__ __forceinline__ void load(const Params &p, const Unit &u, int token) {
        if (!p.mask || b == u.b) return;
        b = u.b;
        const int words = (p.T + 63) / 64;
        const unsigned long long *row = p.mask + ((size_t)u.b * p.T + token) * words;
#pragma unroll
        for (int i = 0; i < kMaskWords / 2; ++i)
            if (i < words) w[i] = row[i];
    }
    // The first drafted token that the row does not see, nor any behind it.
    __device__ __forceinline__ int end(const Params &p, const Unit &u, int token, bool live) const {
        const int drafted = u.keys - u.len;
        return !live ? 0 : p.mask ? drafted : min(drafted, token + 1);
    }
    // The scores of the 64 keys from `key` on, at tS.
    __device__ __forceinline__ void hide(const Params &p, const Unit &u, int token, bool live, uint32_t tS, int key,
                                         uint32_t on_page) const {
        const bool all = !p.mask;
        hide_scores(tS, key - u.len, end(p, u, token, live), all ? ~0ull : w[0], all ? ~0ull : w[1], all ? ~0ull : w[2],
                    all ? ~0ull : w[3], on_page, p.page_size);
    }
    // As 32-bit words, without keys that do not exist; without a mask, a chain sees what is before it.
    __device__ __forceinline__ void bits(const Params &p, const Unit &u, int token, bool live, uint32_t (&out)[kMaskWords]) const {
        const int end = this->end(p, u, token, live);
#pragma unroll
        for (int i = 0; i < kMaskWords / 2; ++i) {
            unsigned long long x = p.mask ? w[i] : ~0ull;
            if (end < 64 * i + 64) x = end <= 64 * i ? 0ull : x & ((1ull << (end - 64 * i)) - 1);
            out[2 * i] = uint32_t(x);
            out[2 * i + 1] = uint32_t(x >> 32);
        }
    }
};

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

// One row's scores of a block, at tS in TMEM, become probabilities in their place.
template <int kBlock>
struct Scores {
    static constexpr int kQuads = kBlock / 32;
    float s[kBlock];
    __device__ __forceinline__ void load(uint32_t tS) {
        uint32_t sr[kQuads][32];
#pragma unroll
        for (int c = 0; c < kQuads; ++c) tmem_ld32(tS + c * 32, sr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kQuads; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(sr[c][i]);
    }
    // Keys from `key` on, of which the row sees `seen` from key `len` on; on_page: a bit a page of the block.
    __device__ __forceinline__ void hide(const Params &p, const uint32_t (&seen)[kMaskWords], int key, int len, bool pages,
                                         uint32_t on_page) {
#pragma unroll
        for (int c = 0; c < kQuads; ++c) {
            uint32_t bits = mask_bits(seen, key + 32 * c - len);
            if (pages) {
                const bool halves = p.page_size == 16;  // two pages in 32 keys
                const int at = p.page_size < kBlock ? 32 * c / p.page_size : 0;
                if (!(on_page >> at & 1)) bits &= halves ? 0xffff0000u : 0u;
                if (halves && !(on_page >> (at + 1) & 1)) bits &= 0x0000ffffu;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1)) s[c * 32 + i] = -INFINITY;
        }
    }
    __device__ __forceinline__ float top() const {
        float m[kQuads];
#pragma unroll
        for (int c = 0; c < kQuads; ++c) {
            float x = fmax3(s[32 * c], s[32 * c + 1], s[32 * c + 2]);
#pragma unroll
            for (int i = 3; i < 31; i += 2) x = fmax3(x, s[32 * c + i], s[32 * c + i + 1]);
            m[c] = fmaxf(x, s[32 * c + 31]);
        }
        if constexpr (kQuads == 2) return fmaxf(m[0], m[1]);
        else return fmax3(m[0], m[1], fmaxf(m[2], m[3]));
    }
    // 2^(s scale - m) in bf16 to tS; their sum.
    __device__ __forceinline__ float exponentials(uint32_t tS, float sl2, float neg_m) const {
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
    }
};

// A row's running softmax.  The reference is the maximum of the first block that shows the row a key, and kept until a
// score is more than 2^16 times as heavy: then the row's output is scaled.  Every row decides for itself, so that none
// depends on another.  The decision is by the maximum of every block, before its exponentials.  By their sum, after which
// the few blocks that need it take them again (as in fwd_kernel.cuh), costs no maxima, but the scores have to be kept, and
// the code is twice as long.  In us, by the sum and by the maximum: 128 users of 512 keys, 8 tokens 71, 63; 16 users of up
// to 32768 keys, 64 tokens, d = 64 486, 468; d = 128 591, 593, in pages of 16 594, 602.
constexpr float kSlack = 16.f;  // log2 units
struct State {
    float m, l, corr;
    __device__ __forceinline__ void clear() { m = -INFINITY, l = 0.f; }
    // Log-sum-exp in log2 units; -inf for a row without a key.
    __device__ __forceinline__ float total(bool live) const { return live && l != 0.f ? m + __log2f(l) : -INFINITY; }
    // Adds a block; true (for all lanes) if the reference of a row moved, so that its output has to be scaled by corr.
    // Rows past the last one (`use` false) hold anything.
    template <int kBlock>
    __device__ __forceinline__ bool add(const Scores<kBlock> &s, uint32_t tS, float sl2, bool use) {
        const float top = s.top() * sl2;
        corr = 1.f;
        if (m == -INFINITY) m = top;
        const bool over = use && top > m + kSlack;
        if (over) corr = fast_exp2(m - top), m = top;
        const bool moved = __any_sync(0xffffffffu, over);  // (brings the lanes together for the stores to TMEM, too)
        l = l * corr + s.exponentials(tS, sl2, m == -INFINITY ? 0.f : -m);
        return moved;
    }
};

// (Out of line: its code is not in the loops' way.  16 users of up to 32768 keys, 64 tokens, 588 us, now 580; d = 64 487,
// now 469; 32 users of up to 16384 keys, 16 tokens, d = 64 157, now 152.)
template <int D>
__device__ __noinline__ void scale_output(uint32_t tO, float corr) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_ld32(tO + c * 32, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * corr);
        tmem_st32(tO + c * 32, x);
    }
}

// 32 bytes to global memory: whole sectors, so that lanes that hold a row each need no help from one another to store it;
// in two halves where the tensors are only 16-byte aligned.
__device__ __forceinline__ void store_32(void *to, const uint32_t (&x)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// A warp's 32 rows of a finished unit, rows [row0, row0 + 32) of the pair, a thread each: columns [col0, col0 + kCols) of
// the accumulator at tO in TMEM or, where there are two (kTwo), of both, kOther columns apart, times f (and f2): to the
// outputs where the unit is all of the pair (`whole`), else to row `part` and so on of the partials.  L: the row's
// log-sum-exp in log2 units, -inf if it has none; odd: drafted rows with elements left out.
// (Instructions on TMEM are the whole warp's, here and above: where lanes may have gone apart before one, __syncwarp or a
// vote brings them together.)
template <int kCols, int D, bool kTwo, int kOther>
__device__ __forceinline__ void store_rows(const Params &p, const Unit &u, bool whole, size_t part, int row0, uint32_t tO,
                                           int col0, float f, float f2, float L, int token, bool live, const Seen &mask,
                                           const uint32_t *odd, const uint32_t *odd2) {
    const int lane = threadIdx.x & 31;
    const size_t row = whole ? ((size_t)u.b * p.Hkv + u.g) * p.rows + row0 : part + row0;
    const int rows = p.rows - row0;  // in use, if below 32
    const bool any = L != -INFINITY;  // (NaN stays NaN)
#pragma unroll 1
    for (int col = col0; col < col0 + kCols; col += 32 * (kTwo || kCols < 64 ? 1 : 2)) {
        constexpr int kHalves = kTwo || kCols < 64 ? 1 : 2;
        uint32_t x[2][32];
        __syncwarp();  // lanes without a row, that have stored nothing, and the others
        tmem_ld32(tO + col, x[0]);
        if constexpr (kTwo || kHalves == 2) tmem_ld32(tO + col + (kTwo ? kOther : 32), x[1]);
        tmem_wait_ld();
        auto scaled = [&](int h, int i, float &a, float &b) {
            float c = -0.f, d = -0.f;
            if constexpr (kTwo) ffma2(c, d, __uint_as_float(x[1][i]), __uint_as_float(x[1][i + 1]), f2, f2, -0.f, -0.f);
            ffma2(a, b, __uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1]), f, f, c, d);
        };
        if (lane < rows && whole) {
            __nv_bfloat16 *to = p.o + (row + lane) * D + col;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float a, b;
                        scaled(h, 16 * g + 2 * i, a, b);
                        y[i] = any ? pack_bf16x2(a, b) : 0u;
                    }
                    store_32(to + 32 * h + 16 * g, y, p.wide);
                }
        } else if (lane < rows) {
            float *to = p.part_o + (row + lane) * D + col;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        float a, b;
                        scaled(h, 8 * g + i, a, b);
                        y[i] = any ? __float_as_uint(a) : 0u;
                        y[i + 1] = any ? __float_as_uint(b) : 0u;
                    }
                    store_32(to + 32 * h + 8 * g, y, p.wide);
                }
        }
    }
    if (lane < rows && col0 == 0) {
        if (!whole) p.part_lse[row + lane] = L;
        else if (p.lse) p.lse[row + lane] = L * 0.69314718055994531f;
    }
    const uint32_t here = lane < kMaskWords ? odd[lane] | odd2[lane] : 0u;
    if (__any_sync(0xffffffffu, here != 0)) {
        uint32_t seen[kMaskWords];
        mask.bits(p, u, token, live && any, seen);
#pragma unroll 1
        for (int w = 0; w < kMaskWords; ++w)
            for (uint32_t bits = (odd[w] | odd2[w]) & mask_bits(seen, 32 * w); bits; bits &= bits - 1) {
                const int key = u.len + 32 * w + __ffs(bits) - 1;
                const int page = p.table ? p.table[(size_t)u.b * p.max_pages + (key >> p.shift)] : u.b;
                const int in = p.table ? key & (p.page_size - 1) : key;
                const __nv_bfloat16 *v = p.v + (((size_t)page * p.Hkv + u.g) * p.page_size + in) * D + col0;
                if (whole) add_odd(p.o + (row + lane) * D + col0, v, kCols);
                else add_odd(p.part_o + (row + lane) * D + col0, v, kCols);
            }
        __syncwarp();
    }
}

// Row of the partials that a cut unit of share `share`, whose first block is j0, begins at.
__device__ __forceinline__ size_t part_row(const Params &p, int share, int j0) {
    return (size_t)(2 * share + (j0 > 0 ? 0 : 1)) * p.rows;
}

// A softmax warp's look at the pages of a unit's blocks, one block ahead: lane i at page i of the block.
template <int kBlock>
struct Holes {
    const int *table;  // null: nothing to look at
    int boxes, used, ahead;
    __device__ __forceinline__ void start(const Params &p, const Unit &u) {
        table = u.holes ? p.table + (size_t)u.b * p.max_pages : nullptr;
        boxes = p.page_size < kBlock ? kBlock / p.page_size : 1;
        used = (u.keys + p.page_size - 1) >> p.shift;
        look(p, u, 0);
    }
    __device__ __forceinline__ void look(const Params &p, const Unit &u, int j) {
        const int lane = threadIdx.x & 31, i = (((u.j0 + j) * kBlock) >> p.shift) + lane;
        ahead = table && lane < boxes && i < used && j < u.n ? table[i] : -1;
    }
    // The bits of block j's pages; then looks at the next one.
    __device__ __forceinline__ uint32_t next(const Params &p, const Unit &u, int j) {
        if (!table) return ~0u;
        const uint32_t on = __ballot_sync(0xffffffffu, ahead >= 0 && ahead < p.num_pages);
        look(p, u, j + 1);
        return on | ~((1u << boxes) - 1);
    }
};

// Sequences without a token: zeros, and a log-sum-exp of nothing (one warp of every CTA).
template <int D>
__device__ __forceinline__ void clear_idle(const Params &p) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        int len, tb;
        load_sequence(p, b, len, tb);
        if (tb > 0) continue;
        const size_t rows = (size_t)p.Hkv * p.rows, units16 = rows * (D / 8);
        uint4 *o = reinterpret_cast<uint4 *>(p.o + (size_t)b * rows * D);
#pragma unroll 1
        for (size_t i = lane; i < units16; i += 32) o[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (size_t i = lane; p.lse && i < rows; i += 32) p.lse[(size_t)b * rows + i] = -INFINITY;
    }
    __syncwarp();
}

// MMAs of one block: S (columns of `keys` keys) = Q K^T, four steps of 16 columns a chunk; O += P V, steps of 16 keys.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tS, uint64_t q, uint32_t q_chunk, uint64_t k, uint32_t k_chunk, uint32_t idesc) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
        uint64_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = q + uint64_t((g * q_chunk + i * 32) >> 4);
            b[i] = k + uint64_t((g * k_chunk + i * 32) >> 4);
        }
        tc_mma_ss_x4_elect(tS, a, b, idesc, g > 0 ? 1u : 0u);
    }
}
template <int kBlock>
__device__ __forceinline__ void issue_pv(uint32_t tO, uint32_t tP, uint64_t v, uint32_t idesc, bool acc) {
#pragma unroll
    for (int g = 0; g < kBlock / 64; ++g) {
        uint32_t a[4];
        uint64_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kk = g * 4 + i;
            a[i] = tP + kk * 8;
            b[i] = v + uint64_t((kk * 16 * 128) >> 4);
        }
        tc_mma_ts_x4_elect(tO, a, b, idesc, (acc || g > 0) ? 1u : 0u);
    }
}

// ------------------------------------------------------------------ few rows
// Shared memory: Q and the ring of each chain, then the rest.  Q has p.q_rows rows; the MMAs read on behind them, in what
// is shared memory all the same, and make rows that nobody looks at.
template <int D>
struct PairCfg {
    static constexpr int kBlock = 64, kChunks = D / 64, kChunkBytes = kBlock * 128, kKVBytes = kBlock * D * 2;
    // Blocks of a chain's ring.  64 KB on their way are enough for a chain, and more are not better: 64 users of 8001 .. 16001
    // keys, one token, d = 128, 4 stages 431 us, 5 433, 6 452, 12 451 (7.2 and 6.9 TB/s); d = 64 the same with 4 as with 12.
    // An even number, so that K and V have slots of their own: a loader that waits for a slot has then waited for the
    // round before it too, and no parity is taken for the one of two rounds ago.
    static constexpr int kStages = 4;
    static_assert(kStages >= 4 && kStages % 2 == 0, "see above; the next but one K is issued ahead of V");
    // barriers of a chain (S and P: a buffer each)
    static constexpr int kQFull = 0, kQEmpty = 1, kSFull = 2, kPFull = 4, kOFull = 6, kOEmpty = 7, kUFull = 8, kUEmpty = 10,
                         kDrain = 12, kJoint = 13, kKVFull = 14, kKVEmpty = 14 + kStages, kNumBars = 14 + 2 * kStages;
    // 16 warps: 512 threads x 128 registers at launch are shared out anew.
    static constexpr int kThreads = 512, kCtrlRegs = 88, kSoftmaxRegs = 160;
    static_assert(256 * kCtrlRegs + 256 * kSoftmaxRegs <= 512 * 128, "register split");
    static constexpr int kStateOffset = 2 * 4 * kMaskWords * 4;  // the chains' states of a joint unit, and its parts
    static constexpr int kBarOffset = kStateOffset + 2 * kTileM * 8 + 32, kUnitOffset = (kBarOffset + 2 * kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kFixedBytes = kUnitOffset + 2 * 2 * kUnitInts * 4 + 16;
    static __host__ __device__ int q_bytes(int q_rows) { return q_rows * 128 * kChunks; }
    static __host__ __device__ int chain_bytes(int q_rows) { return q_bytes(q_rows) + kStages * kKVBytes; }
    static int smem_bytes(int q_rows) { return 2 * chain_bytes(q_rows) + kFixedBytes + 1024; }
    static_assert(2 * (kTileM * D * 2 + kStages * kKVBytes) + kFixedBytes + 1024 <= kSmemMax, "shared memory");
};

// A place in a ring, and the parity of the round.
struct Place {
    uint32_t slot = 0, odd = 0;
    __device__ __forceinline__ void next(uint32_t stages) {
        if (++slot == stages) slot = 0, odd ^= 1;
    }
};

template <int D>
__global__ void __launch_bounds__(PairCfg<D>::kThreads, 1)
    pairs_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const Params p) {
    using C = PairCfg<D>;
    constexpr int kBlock = C::kBlock;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Per chain: warps that plan and load Q and K, that load V, that issue MMAs, one to spare; then the softmax warps.  At
    // d = 64 the spare one shares its issue slots with the softmax warp of the first 32 rows, which is all there is of few
    // tokens, instead of the K loader: 64 users, one token, 252 us, now 247; in pages of 16 285, 273; 16 tokens 161 either
    // way.  (At d = 128, where a block has twice the bytes, 32 users with 16 tokens 148.3 us, and 149.)
    enum { kLoadK, kLoadV, kIssue, kSpare, kSoftmax };
    const int t = warp >> 2 & 1, place = warp & 3;
    const int role = warp >= 8 ? kSoftmax : D == 64 && (place == kLoadK || place == kSpare) ? kSpare - place : place;
    const int share = blockIdx.x;
    constexpr uint32_t stages = C::kStages;
    const int q_bytes = C::q_bytes(p.q_rows), chain_bytes = C::chain_bytes(p.q_rows);
    uint8_t *sQ = smem + t * chain_bytes, *ring = sQ + q_bytes, *rest = smem + 2 * chain_bytes;
    uint32_t *all_odd = reinterpret_cast<uint32_t *>(rest);  // [chain][four units in turn]
    uint32_t *odd_rows = all_odd + t * 4 * kMaskWords;
    float2 *states = reinterpret_cast<float2 *>(rest + C::kStateOffset);  // [chain][row]
    volatile int *parts = reinterpret_cast<volatile int *>(states + 2 * kTileM);  // [chain]: first block, blocks, which of the four units in turn
    uint64_t *all_bars = reinterpret_cast<uint64_t *>(rest + C::kBarOffset);
    volatile int *units = reinterpret_cast<volatile int *>(rest + C::kUnitOffset) + t * 2 * kUnitInts;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rest + C::kUnitOffset + 2 * 2 * kUnitInts * 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(all_bars + t * C::kNumBars + i); };

    griddep_launch_dependents();  // the merge waits for this grid to end
    if (threadIdx.x >= 256) {  // a barrier a thread
        const int i = int(threadIdx.x) - 256;
        if (i < 2 * C::kNumBars) {
            const int k = i % C::kNumBars;
            const bool four = k == C::kPFull || k == C::kPFull + 1 || k == C::kOEmpty;
            // (a unit's slot: the V and MMA warps, the softmax warps)
            mbar_init(smem_u32(all_bars + i), four ? 4 : k == C::kUEmpty || k == C::kUEmpty + 1 ? 2 + 4 : k == C::kJoint ? 8 : 1);
        }
        if (i == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    static_assert(2 * C::kNumBars <= 256, "one thread each");
    if (role == kSoftmax && (warp & 3) == 0) odd_rows[lane] = 0;
    static_assert(4 * kMaskWords == 32, "one warp clears them");
    if (role == kIssue && t == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    Unit u = {};
    Pages<kBlock> pages = {};
    int left = 0;
    bool two = false;  // whether both chains have blocks
    if (role == kLoadK) {
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        // Chain 0 takes the share's first half, from its begin on, chain 1 the other one, from its end back.
        const Share s = share_of<kBlock>(p, share);
        const int half = (s.left + 1) / 2;
        left = t == 0 ? half : s.left - half;
        two = s.left > 1;
        if (left > 0) {
            u = find_block<kBlock>(p, t == 0 ? s.lo : s.lo + s.left - 1);
            if (t > 0) ++u.j0;  // (there: the block behind the unit)
            u.n = t == 0 ? min(left, u.nb - u.j0) : min(left, u.j0);
            if (t > 0) u.j0 -= u.n;
            // The halves meet inside a pair.
            u.joint = u.n == left && (t == 0 ? two && u.j0 + u.n < u.nb : u.j0 > 0);
            pages.start(p, u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_all = *tmem_slot, tmem = tmem_all + t * 256;  // scores at [0, 64) and [64, 128), the output behind

    if (role != kSoftmax) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kCtrlRegs));
        volatile int no_abort = 0;
        if (role == kLoadK || role == kLoadV) {
            // ------------------------- loaders: the units, Q and K; V from what the other one says
            // K and V alternate in the ring.
            const bool is_k = role == kLoadK;
            Place at;
            if (!is_k) at.next(stages);
            uint32_t fills = is_k ? 0 : 1, q_loads = 0;  // fills: the number of the next one in the ring
            bool ok = true;
            u.holes = p.table != nullptr;  // (the first unit's entries are looked at block by block)
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                if (is_k) {
                    if (p.table && qi > 0) u.holes = look_for_holes<kBlock>(p, u);
                    if (qi >= 2) ok = wait_warp(bar(C::kUEmpty + qs), ((qi >> 1) - 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    if (lane == 0) {
                        u.put(units + kUnitInts * qs);
                        mbar_arrive(bar(C::kUFull + qs));
                    }
                    __syncwarp();
                } else {
                    ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    u.get(units + kUnitInts * qs);
                    __syncwarp();
                    mbar_arrive_elect(bar(C::kUEmpty + qs));
                    if (u.n > 0) pages.start(p, u);
                }
                if (u.n == 0) break;
#pragma unroll 1
                for (int j = 0; j < u.n; ++j) {
                    if (fills >= stages) ok = wait_warp(bar(C::kKVEmpty + at.slot), at.odd ^ 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    const uint32_t full = bar(C::kKVFull + at.slot);
                    if (lane == 0) mbar_arrive_expect_tx(full, C::kKVBytes);
                    pages.template load<C::kChunks>(p, u, (u.j0 + j) * kBlock, is_k ? &tmK : &tmV, full,
                                                    smem_u32(ring + at.slot * C::kKVBytes));
                    fills += 2;
                    at.next(stages);
                    at.next(stages);
                    if (is_k && j == 0) {
                        if (q_loads > 0) ok = wait_warp(bar(C::kQEmpty), (q_loads - 1) & 1, p.wait_ns, abort_flag);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(C::kQFull), q_bytes);
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_u32(sQ + c * p.q_rows * 128), &tmQ, bar(C::kQFull), c * 64, 0, u.b * p.Hkv + u.g);
                        }
                        __syncwarp();
                        ++q_loads;
                    }
                }
                if (!ok) break;
                if (is_k) {
                    left -= u.n;
                    if (left == 0) {
                        u.n = 0;
                        continue;
                    }
                    if (t == 0) {
                        next_pair<kBlock>(p, u);
                        u.n = min(left, u.nb);
                    } else {
                        previous_pair<kBlock>(p, u);
                        u.n = min(left, u.nb);
                        u.j0 -= u.n;
                    }
                    u.joint = u.n == left && (t == 0 ? two && u.n < u.nb : u.j0 > 0);
                    pages.start(p, u);
                }
            }
            __syncwarp();
            // Copies have to land before the CTA goes (bounded), whatever became of the other warps: this warp's last one
            // into every slot.
            if (!ok && lane == 0) {
                Place back = at;
                for (uint32_t f = fills; f >= 2 && f + stages > fills; f -= 2) {
                    for (int i = 0; i < 2; ++i) {
                        if (back.slot == 0) back.slot = stages, back.odd ^= 1;
                        --back.slot;
                    }
                    if (!mbar_wait_bounded(bar(C::kKVFull + back.slot), back.odd, kDrainNs, &no_abort, &g_tree_status))
                        atomicOr(&g_tree_status, kStatusDrainTimeout);
                }
                if (q_loads > 0 && !mbar_wait_bounded(bar(C::kQFull), (q_loads - 1) & 1, kDrainNs, &no_abort, &g_tree_status))
                    atomicOr(&g_tree_status, kStatusDrainTimeout);
            }
            __syncwarp();
        } else if (role == kSpare) {
            if (t > 0) clear_idle<D>(p);
            else if (!p.whole) write_cut<kBlock>(p, share, share_of<kBlock>(p, share));
        } else {
            // ------------------------------------------------------ MMA issuer
            constexpr uint32_t kIdescQK = idesc_bf16_f32(kTileM, kBlock, 0), kIdescPV = idesc_bf16_f32(kTileM, D, 1);
            const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024), dK = smem_desc_sw128(smem_u32(ring), 16, 1024),
                           dV = smem_desc_sw128(smem_u32(ring), C::kChunkBytes, 1024);
            const uint32_t q_chunk = p.q_rows * 128;
            Place k, v;  // of the next K and V
            v.next(stages);
            uint32_t p_odd = 0, done = 0;  // p_odd: a bit a buffer
            bool ok = true;
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                const int n = __shfl_sync(0xffffffffu, int(units[kUnitInts * qs + 3]), 0);
                mbar_arrive_elect(bar(C::kUEmpty + qs));
                if (n == 0) break;
                ok = wait_warp(bar(C::kQFull), qi & 1, p.wait_ns, abort_flag);
                // S(0), S(1); then P(j) V and S(j + 2) into the buffer that P(j) has been read from.
#pragma unroll 1
                for (int j = -2; ok && j < n; ++j) {
                    const int buf = j & 1;
                    if (j >= 0) {
                        ok = wait_warp(bar(C::kPFull + buf), p_odd >> buf & 1, p.wait_ns, abort_flag);
                        if (ok && j == 0 && done > 0) ok = wait_warp(bar(C::kOEmpty), (done - 1) & 1, p.wait_ns, abort_flag);
                        if (ok) ok = wait_warp(bar(C::kKVFull + v.slot), v.odd, p.wait_ns, abort_flag);
                        if (!ok) break;
                        p_odd ^= 1u << buf;
                        tc_fence_after();
                        issue_pv<kBlock>(tmem + 128, tmem + buf * kBlock, dV + uint64_t(v.slot * (C::kKVBytes >> 4)), kIdescPV, j > 0);
                        tc_commit_elect(bar(C::kKVEmpty + v.slot));
                        v.next(stages);
                        v.next(stages);
                        if (j == n - 1) tc_commit_elect(bar(C::kOFull));
                    }
                    if (j + 2 < n) {
                        ok = wait_warp(bar(C::kKVFull + k.slot), k.odd, p.wait_ns, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue_qk<D>(tmem + buf * kBlock, dQ, q_chunk, dK + uint64_t(k.slot * (C::kKVBytes >> 4)), C::kChunkBytes, kIdescQK);
                        tc_commit_elect(bar(C::kSFull + buf));
                        tc_commit_elect(bar(C::kKVEmpty + k.slot));
                        k.next(stages);
                        k.next(stages);
                        if (j + 2 == n - 1) tc_commit_elect(bar(C::kQEmpty));  // Q's last product
                    }
                }
                ++done;
            }
            tc_commit_elect(bar(C::kDrain));
            if (!wait_warp(bar(C::kDrain), 0, kDrainNs, &no_abort) && lane == 0) atomicOr(&g_tree_status, kStatusDrainTimeout);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // ------------------------------------------------- softmax / epilogue
        const int quarter = warp & 3, row = quarter * 32 + lane, token = row % p.T;
        const uint32_t lanes = uint32_t(quarter * 32) << 16, tS0 = tmem + lanes, tO = tmem + lanes + 128;
        const bool has_rows = quarter * 32 < p.rows;  // of this warp; the others only keep step
        Place at;  // of the next block's K
        Seen mask;
        uint32_t s_odd = 0;
        bool ok = true;
        for (uint32_t qi = 0; ok; ++qi) {
            const uint32_t qs = qi & 1;
            ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
            if (!ok) break;
            u.get(units + kUnitInts * qs);
            __syncwarp();
            mbar_arrive_elect(bar(C::kUEmpty + qs));
            if (u.n == 0) break;
            const bool live = row < p.rows && token < u.tb;
            if ((u.j0 + u.n) * kBlock > u.len || u.joint) mask.load(p, u, token);
            Holes<kBlock> holes;
            holes.start(p, u);
            uint32_t *odd = odd_rows + (qi & 3) * kMaskWords;
            State st;
            st.clear();
            Place last = at;  // of the last block's V
#pragma unroll 1
            for (int j = 0; j < u.n; ++j) {
                const int buf = j & 1, key = (u.j0 + j) * kBlock;
                const uint32_t on_page = holes.next(p, u, j);
                ok = wait_warp(bar(C::kSFull + buf), s_odd >> buf & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                s_odd ^= 1u << buf;
                at.next(stages);
                if (has_rows) {
                    const uint32_t tS = tS0 + buf * kBlock;
                    tc_fence_after();
                    if (key + kBlock > u.len || on_page != ~0u) mask.hide(p, u, token, live, tS, key, on_page);
                    Scores<kBlock> s;
                    s.load(tS);
                    if (st.add(s, tS, p.scale_log2, row < p.rows) && j > 0) {
                        // S(j) was issued ahead of the last product into O: wait for that, by its V slot, which nobody can
                        // have filled and freed again before this block's P.
                        ok = wait_warp(bar(C::kKVEmpty + last.slot), last.odd, p.wait_ns, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        scale_output<D>(tO, st.corr);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                if (key + kBlock > u.len) {
                    ok = wait_warp(bar(C::kKVFull + at.slot), at.odd, p.wait_ns, abort_flag);
                    if (!ok) break;
                    const int first = max(u.len - key, 0);
                    clean_rows<C::kChunks, kBlock>(ring + at.slot * C::kKVBytes, quarter, first, u.keys - key, key + first - u.len, odd);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                last = at;
                at.next(stages);
                __syncwarp();
                mbar_arrive_elect(bar(C::kPFull + buf));
            }
            if (ok) ok = wait_warp(bar(C::kOFull), qi & 1, p.wait_ns, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (u.joint) {
                // The last unit of both chains: each has the other's state and stores half of the columns.
                states[t * kTileM + row] = make_float2(st.m, st.l);
                if (quarter == 0 && lane == 0) parts[3 * t] = u.j0, parts[3 * t + 1] = u.n, parts[3 * t + 2] = int(qi & 3);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_elect(smem_u32(all_bars + C::kJoint));
                ok = wait_warp(smem_u32(all_bars + C::kJoint), 0, p.wait_ns, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const float2 a = states[row], c = states[kTileM + row];
                const float top = fmaxf(a.x, c.x), ref = top == -INFINITY ? 0.f : top;
                const float f = fast_exp2(a.x - ref), f2 = fast_exp2(c.x - ref), sum = f * a.y + f2 * c.y;
                const bool whole = parts[1] + parts[4] == u.nb;
                const uint32_t *other = all_odd + ((1 - t) * 4 + parts[3 * (1 - t) + 2]) * kMaskWords;
                if (has_rows)
                    store_rows<D / 2, D, true, 256>(p, u, whole, part_row(p, share, parts[0]), quarter * 32,
                                                    tmem_all + lanes + 128, t * (D / 2), f / sum, f2 / sum,
                                                    live && sum != 0.f ? top + __log2f(sum) : -INFINITY, token, live, mask, odd, other);
                tc_fence_before();
                break;
            }
            // (the next unit but one has none yet, and this warp's mates are all past the last one)
            if (quarter == 0 && lane < kMaskWords) odd_rows[((qi + 2) & 3) * kMaskWords + lane] = 0;
            if (has_rows)
                store_rows<D, D, false, 0>(p, u, u.n == u.nb, part_row(p, share, u.j0), quarter * 32, tO, 0, 1.f / st.l, 0.f,
                                           st.total(live), token, live, mask, odd, odd);
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(bar(C::kOEmpty));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (role == kIssue && t == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_all, kTmemCols);
    }
}

// ----------------------------------------------------------------- many rows
template <int D>
struct RowsCfg {
    static constexpr int kBlock = 128, kChunks = D / 64, kChunkBytes = 128 * 128;
    static constexpr int kQBytes = kTileM * D * 2, kKVBytes = kBlock * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kOCol = 2 * kTileM;
    static constexpr int kOddOffset = 2 * kQBytes + kStages * kKVBytes;
    static constexpr int kBarOffset = kOddOffset + 4 * kMaskWords * 4;
    static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6, kOFull = 8, kOEmpty = 10, kUFull = 12, kUEmpty = 14,
                         kDrain = 16, kKVFull = 17, kKVEmpty = 17 + kStages, kNumBars = 17 + 2 * kStages;
    static constexpr int kUnitOffset = (kBarOffset + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kSmemBytes = kUnitOffset + 2 * kUnitInts * 4 + 16 + 1024;  // units, tmem, abort; alignment
    static_assert(kSmemBytes <= kSmemMax, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Params p) {
    using C = RowsCfg<D>;
    constexpr int kBlock = C::kBlock;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + 2 * C::kQBytes;
    uint32_t *odd_rows = reinterpret_cast<uint32_t *>(smem + C::kOddOffset);  // of four units in turn
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
    volatile int *units = reinterpret_cast<volatile int *>(smem + C::kUnitOffset);  // two entries
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kUnitOffset + 2 * kUnitInts * 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = blockIdx.x / p.mt, m = blockIdx.x - share * p.mt;
    const bool second = (2 * m + 1) * kTileM < p.rows;  // a second tile
    auto bar = [&](int i) { return smem_u32(bars + i); };

    griddep_launch_dependents();  // the merge waits for this grid to end
    if (threadIdx.x >= 128) {  // a barrier a thread
        const int i = int(threadIdx.x) - 128;
        if (i < C::kNumBars) {
            const bool four = (i >= C::kPFull && i < C::kPFull + 2) || (i >= C::kOEmpty && i < C::kOEmpty + 2);
            // (a unit's slot: the K, V and MMA warps, the softmax warps)
            mbar_init(bar(i), four ? 4 : i >= C::kUEmpty && i < C::kUEmpty + 2 ? 3 + 8 : 1);
        }
        if (i == 0) *abort_flag = 0;
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
    Unit u = {};
    int left = 0;
    if (warp == 3) {
        const Share s = share_of<kBlock>(p, share);
        left = s.left;
        if (left > 0) u = find_block<kBlock>(p, s.lo);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
        volatile int no_abort = 0;
        if (warp == 3) {
            // -------------------------------------------- planner: the units, and Q
            uint32_t q_loads = 0;  // per tile (both are loaded for every unit)
            bool ok = true;
            u.holes = p.table != nullptr;  // (a short first unit's entries are looked at block by block)
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                u.n = left > 0 ? min(left, u.nb - u.j0) : 0;
                if (p.table && (qi > 0 || u.n >= kLongUnit)) u.holes = look_for_holes<kBlock>(p, u);
                if (qi >= 2) ok = wait_warp(bar(C::kUEmpty + qs), ((qi >> 1) - 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    u.put(units + kUnitInts * qs);
                    mbar_arrive(bar(C::kUFull + qs));
                }
                __syncwarp();
                if (u.n == 0) break;
#pragma unroll 1
                for (int t = 0; t < (second ? 2 : 1); ++t) {
                    if (q_loads > 0) ok = wait_warp(bar(C::kQEmpty + t), (q_loads - 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(C::kQFull + t), C::kQBytes);
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_3d(smem_u32(sQ + t * C::kQBytes + c * C::kChunkBytes), &tmQ, bar(C::kQFull + t), c * 64,
                                        (2 * m + t) * kTileM, u.b * p.Hkv + u.g);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                ++q_loads;
                left -= u.n;
                if (left > 0) next_pair<kBlock>(p, u);
            }
            __syncwarp();
            // Copies have to land before the CTA goes (bounded), whatever became of the other warps.
            if (!ok && lane == 0)
                for (int t = 0; t < (second ? 2 : 1); ++t)
                    if (q_loads > 0 && !mbar_wait_bounded(bar(C::kQFull + t), (q_loads - 1) & 1, kDrainNs, &no_abort, &g_tree_status))
                        atomicOr(&g_tree_status, kStatusDrainTimeout);
            __syncwarp();
        } else if (warp != 1) {
            // ------------------------------------- loaders: warp 0 K, warp 2 V
            // Blocks alternate in the ring, K at even fills and V at odd ones; neither warp waits for the other's slots.
            const uint32_t kv = warp == 0 ? 0 : 1;
            if (warp == 2 && m == 0 && !p.whole) write_cut<kBlock>(p, share, share_of<kBlock>(p, share));
            uint32_t blocks = 0;  // loaded so far
            bool ok = true;
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                u.get(units + kUnitInts * qs);
                __syncwarp();
                mbar_arrive_elect(bar(C::kUEmpty + qs));
                if (u.n == 0) break;
                Pages<kBlock> pages;
                pages.start(p, u);
                for (int j = 0; j < u.n; ++j) {
                    const uint32_t fill = 2 * blocks + kv, slot = fill % C::kStages, round = fill / C::kStages;
                    if (round > 0) ok = wait_warp(bar(C::kKVEmpty + slot), (round - 1) & 1, p.wait_ns, abort_flag);
                    if (!ok) break;
                    const uint32_t full = bar(C::kKVFull + slot);
                    if (lane == 0) mbar_arrive_expect_tx(full, C::kKVBytes);
                    pages.template load<C::kChunks>(p, u, (u.j0 + j) * kBlock, kv ? &tmV : &tmK, full,
                                                    smem_u32(sKV + slot * C::kKVBytes));
                    ++blocks;
                }
            }
            __syncwarp();
            if (!ok && lane == 0)
                for (uint32_t s = kv; s < C::kStages; s += 2) {
                    if (2 * blocks <= s) continue;  // fills below 2 blocks + kv are out
                    const uint32_t last = (2 * blocks - 2 + kv - s) / C::kStages;  // round of the slot's last fill
                    if (!mbar_wait_bounded(bar(C::kKVFull + s), last & 1, kDrainNs, &no_abort, &g_tree_status))
                        atomicOr(&g_tree_status, kStatusDrainTimeout);
                }
            __syncwarp();
            if (warp == 2) clear_idle<D>(p);
        } else {
            // ------------------------------------------------------ MMA issuer
            constexpr uint32_t kIdescQK = idesc_bf16_f32(kTileM, kBlock, 0), kIdescPV = idesc_bf16_f32(kTileM, D, 1);
            const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024), dK = smem_desc_sw128(smem_u32(sKV), 16, 1024),
                           dV = smem_desc_sw128(smem_u32(sKV), C::kChunkBytes, 1024);
            const int tiles = second ? 2 : 1;
            uint32_t fills = 0, blocks = 0, done = 0;
            bool ok = true;
            auto slot_off = [&](uint32_t f) { return uint64_t(f % C::kStages * (C::kKVBytes >> 4)); };
            auto wait_slot = [&](uint32_t f) {
                return wait_warp(bar(C::kKVFull + f % C::kStages), (f / C::kStages) & 1, p.wait_ns, abort_flag);
            };
            for (uint32_t qi = 0; ok; ++qi) {
                const uint32_t qs = qi & 1;
                ok = wait_warp(bar(C::kUFull + qs), (qi >> 1) & 1, p.wait_ns, abort_flag);
                if (!ok) break;
                const int n = __shfl_sync(0xffffffffu, int(units[kUnitInts * qs + 3]), 0);
                mbar_arrive_elect(bar(C::kUEmpty + qs));
                if (n == 0) break;
                // S(t, 0); then P(t, j) V and S(t, j + 1), so that the commit that announces S(t, j + 1) says that P(t, j) V
                // is complete too.
                for (int j = -1; ok && j < n; ++j) {
                    const uint32_t fV = fills + 2 * j + 1, fK = fV + 1;
#pragma unroll 1
                    for (int t = 0; t < tiles; ++t) {
                        if (j >= 0) {
                            ok = wait_warp(bar(C::kPFull + t), blocks & 1, p.wait_ns, abort_flag);
                            if (ok && j == 0 && done > 0) ok = wait_warp(bar(C::kOEmpty + t), (done - 1) & 1, p.wait_ns, abort_flag);
                            if (ok && t == 0) ok = wait_slot(fV);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv<kBlock>(tmem + C::kOCol + t * D, tmem + t * kTileM, dV + slot_off(fV), kIdescPV, j > 0);
                            if (t == tiles - 1) tc_commit_elect(bar(C::kKVEmpty + fV % C::kStages));
                        } else {
                            ok = wait_warp(bar(C::kQFull + t), done & 1, p.wait_ns, abort_flag);
                            if (!ok) break;
                        }
                        if (j + 1 < n) {
                            if (t == 0) ok = wait_slot(fK);
                            if (!ok) break;
                            tc_fence_after();
                            issue_qk<D>(tmem + t * kTileM, dQ + uint64_t(t * (C::kQBytes >> 4)), C::kChunkBytes, dK + slot_off(fK),
                                        C::kChunkBytes, kIdescQK);
                            tc_commit_elect(bar(C::kSFull + t));
                            if (j + 1 == n - 1) tc_commit_elect(bar(C::kQEmpty + t));  // Q's last product
                        } else {
                            tc_commit_elect(bar(C::kOFull + t));
                        }
                    }
                    if (j >= 0) ++blocks;
                }
                fills += 2 * n;
                ++done;
            }
            tc_commit_elect(bar(C::kDrain));
            if (!wait_warp(bar(C::kDrain), 0, kDrainNs, &no_abort) && lane == 0) atomicOr(&g_tree_status, kStatusDrainTimeout);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------- softmax / epilogue
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int row0 = (2 * m + t) * kTileM + quarter * 32, row = row0 + lane, token = row % p.T;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t tS = tmem + lanes + t * kTileM, tO = tmem + lanes + C::kOCol + t * D;
        const bool has_rows = row0 < p.rows;  // of this warp; the others only keep step
        const bool frees = quarter == 0 && t == (second ? 1 : 0);  // K's slots: the last chain to see S
        uint32_t blocks = 0, fills = 0;
        Seen mask;
        Holes<kBlock> holes;
        bool ok = true;
        // A unit, and the loads that its blocks need: the next one's before the rows of the last are stored (38 users, 64
        // tokens, 2048 keys 152 us, now 147; 16 users of up to 32768 keys 581, now 573).
        auto fetch = [&](uint32_t qi, Unit &x, Seen &seen, Holes<kBlock> &h) {
            if (!wait_warp(bar(C::kUFull + (qi & 1)), (qi >> 1) & 1, p.wait_ns, abort_flag)) return false;
            x.get(units + kUnitInts * (qi & 1));
            __syncwarp();
            mbar_arrive_elect(bar(C::kUEmpty + (qi & 1)));
            if (x.n == 0 || (t > 0 && !second)) return true;
            if ((x.j0 + x.n) * kBlock > x.len) seen.load(p, x, token);
            h.start(p, x);
            return true;
        };
        ok = fetch(0, u, mask, holes);
        for (uint32_t qi = 0; ok; ++qi) {
            if (u.n == 0) break;
            if (t > 0 && !second) {
                ok = fetch(qi + 1, u, mask, holes);
                continue;
            }
            const bool live = row < p.rows && token < u.tb;
            // A warp whose rows have no token leaves its scores as they are: rows that nobody looks at.  (16 users x 32768
            // keys, 64 tokens, of which 32 are there: 602 -> 566 us.)
            const bool any_live = __any_sync(0xffffffffu, live);
            uint32_t *odd = odd_rows + (qi & 3) * kMaskWords;
            State st;
            st.clear();
            // A block; masked: keys may be drafted, or on no page.
            auto step = [&](int j, auto masked) {
                constexpr bool kMasked = decltype(masked)::value;
                const int key = (u.j0 + j) * kBlock;
                const uint32_t on_page = kMasked ? holes.next(p, u, j) : ~0u;
                ok = wait_warp(bar(C::kSFull + t), blocks & 1, p.wait_ns, abort_flag);
                if (!ok) return;
                if (frees) mbar_arrive_elect(bar(C::kKVEmpty + fills % C::kStages));
                if (any_live) {
                    tc_fence_after();
                    Scores<kBlock> s;
                    s.load(tS);
                    if (kMasked && (key + kBlock > u.len || on_page != ~0u)) {
                        uint32_t seen[kMaskWords];
                        mask.bits(p, u, token, live, seen);
                        s.hide(p, seen, key, u.len, holes.table != nullptr, on_page);
                    }
                    if (st.add(s, tS, p.scale_log2, row < p.rows) && j > 0) scale_output<D>(tO, st.corr);
                    tmem_wait_st();
                    tc_fence_before();
                }
                if (kMasked && key + kBlock > u.len && t == 0) {
                    // (the other tile's product of this block is issued behind this one's)
                    const uint32_t slot = (fills + 1) % C::kStages;
                    ok = wait_warp(bar(C::kKVFull + slot), ((fills + 1) / C::kStages) & 1, p.wait_ns, abort_flag);
                    if (!ok) return;
                    const int first = max(u.len - key, 0);
                    clean_rows<C::kChunks, kBlock>(sKV + slot * C::kKVBytes, quarter, first, u.keys - key, key + first - u.len, odd);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                mbar_arrive_elect(bar(C::kPFull + t));
                ++blocks;
                fills += 2;
            };
            // The blocks of cached keys alone in a loop without the mask's code: 16 users of up to 32768 keys, 64 tokens, 602
            // us, then 591; in pages of 16 607, then 590; 4 users of up to 8192, 256 tokens, 176, then 171.
            const int plain = holes.table ? 0 : min(u.n, max(0, u.len / kBlock - u.j0));
            int j = 0;
            for (; ok && j < plain; ++j) step(j, std::false_type{});
            for (; ok && j < u.n; ++j) step(j, std::true_type{});
            Unit next = {};
            Seen next_mask = mask;
            if (ok) ok = fetch(qi + 1, next, next_mask, holes);
            if (ok) ok = wait_warp(bar(C::kOFull + t), qi & 1, p.wait_ns, abort_flag);
            if (!ok) break;
            tc_fence_after();
            // (the next unit but one has none yet; of the last one's, the other tile is past its products, hence its stores)
            if (t == 0 && quarter == 0 && lane < kMaskWords) odd_rows[((qi + 2) & 3) * kMaskWords + lane] = 0;
            if (has_rows)
                store_rows<D, D, false, 0>(p, u, u.n == u.nb, part_row(p, share, u.j0), row0, tO, 0, 1.f / st.l, 0.f,
                                           st.total(live), token, live, mask, odd, odd);
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(bar(C::kOEmpty + t));
            u = next;
            mask = next_mask;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Rows of the pair that goes on behind share x: their partials (2 x + 1, 2 (x + 1), 2 (x + 2), ...) by the
// log-sum-exps' weights.  A warp takes kRows rows at once, with the loads of all of them in flight; kSplit warps share
// the partials of the same rows.  x is blockIdx.x; or, where pairs are few and rows many, the blockIdx.x-th share that has
// such a pair, so that no blocks only look and leave.  1 user of up to 8192 keys, both kernels, by blockIdx.x and by
// search: 2 tokens (16 rows) 18.9 us, 20.6; 4 tokens 20.6, 20.6; 8 tokens (2432 blocks or 128) 22.6, 20.6; 32 tokens 31.6,
// 26.7.
template <int D, int kSplit>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const Params p) {
    constexpr int kCols = D / 32, kRows = 4, kAhead = 2;
    using Vec = typename std::conditional<kCols == 4, float4, float2>::type;
    __shared__ float acc_sh[kSplit > 1 ? kSplit : 1][kRows][D], sum_sh[kSplit > 1 ? kSplit : 1][kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kSplit;
    const int row0 = (blockIdx.y * (kMergeWarps / kSplit) + warp / kSplit) * kRows;
    griddep_wait();
    int4 cut = make_int4(0, 0, 0, 0);
    int x = blockIdx.x;
    if (kSplit == 1 || gridDim.x == unsigned(p.shares)) {
        cut = p.cuts[x];
    } else {
        __shared__ int4 cut_sh;
        __shared__ int x_sh, counts[kMergeWarps];
        if (threadIdx.x == 0) cut_sh = cut;
        int before = 0;
        for (int first = 0; first < p.shares; first += kMergeWarps * 32) {
            const int i = first + int(threadIdx.x);
            const int4 c = i < p.shares ? p.cuts[i] : make_int4(0, 0, 0, 0);
            const uint32_t vote = __ballot_sync(0xffffffffu, c.z > 0);
            if (first > 0) __syncthreads();
            if (lane == 0) counts[warp] = __popc(vote);
            __syncthreads();
            int rank = before + __popc(vote & ((1u << lane) - 1));
            for (int w = 0; w < kMergeWarps; ++w) {
                rank += w < warp ? counts[w] : 0;
                before += counts[w];
            }
            if (c.z > 0 && rank == x) cut_sh = c, x_sh = i;
        }
        __syncthreads();
        cut = cut_sh;
        x = x_sh;
    }
    if (cut.z == 0 || (kSplit == 1 && row0 >= p.rows)) return;
    const int rows = min(kRows, p.rows - row0);  // (below 1: none, but the warp keeps step)
    auto at = [&](int i, int r) { return (size_t)(2 * (x + i) + (i == 0 ? 1 : 0)) * p.rows + row0 + r; };
    // Lane 8 r + k: row r's partials k, k + 8, ...; the first kHeld of them stay in registers.
    constexpr int kHeld = 5;
    const int r8 = lane >> 3, k8 = lane & 7;
    Vec v[kAhead][kRows];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (i0 + k < cut.z && r < rows) v[k][r] = reinterpret_cast<const Vec *>(p.part_o + at(i0 + k, r) * D)[lane];
    };
    float held[kHeld], top = -INFINITY;
#pragma unroll
    for (int q = 0; q < kHeld; ++q) held[q] = k8 + 8 * q < cut.z && r8 < rows ? p.part_lse[at(k8 + 8 * q, r8)] : -INFINITY;
    fetch(part * kAhead);  // (does not depend on the weights)
#pragma unroll
    for (int q = 0; q < kHeld; ++q) top = fmaxf(top, held[q]);
    for (int i = k8 + 8 * kHeld; i < cut.z; i += 8)
        if (r8 < rows) top = fmaxf(top, p.part_lse[at(i, r8)]);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[kRows][kCols] = {}, sum = 0.f;
    for (int i0 = part * kAhead; i0 < cut.z; i0 += kSplit * kAhead) {
        if (i0 > part * kAhead) fetch(i0);
        // The weight of partial i0 + k is with lane (i0 + k) % 8 of the row's eight.
        const int mine = i0 + ((k8 - i0) & 7);
        float w = -INFINITY;
        if (mine < i0 + kAhead && mine < cut.z) {
            const int q = mine >> 3;
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (q == h) w = held[h];
            if (q >= kHeld && r8 < rows) w = p.part_lse[at(mine, r8)];
        }
        w = fast_exp2(w - ref);
        sum += w;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float f = __shfl_sync(0xffffffffu, w, 8 * r + ((i0 + k) & 7));
                if (f == 0.f || i0 + k >= cut.z) continue;  // an empty partial adds nothing
                const float *x = reinterpret_cast<const float *>(&v[k][r]);
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[r][c] += f * x[c];
            }
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if constexpr (kSplit > 1) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) reinterpret_cast<Vec *>(acc_sh[part][r])[lane] = *reinterpret_cast<Vec *>(acc[r]);
        if (k8 == 0) sum_sh[part][r8] = sum;
        __syncthreads();
        if (part > 0) return;
        for (int w = 1; w < kSplit; ++w) {
            sum += sum_sh[w][r8];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const Vec x = reinterpret_cast<const Vec *>(acc_sh[w][r])[lane];
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[r][c] += reinterpret_cast<const float *>(&x)[c];
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
    const size_t out = ((size_t)cut.x * p.Hkv + cut.y) * p.rows + row0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float f = __shfl_sync(0xffffffffu, inv, 8 * r);
        if (r >= rows) continue;
        uint32_t packed[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) packed[c] = pack_bf16x2(acc[r][2 * c] * f, acc[r][2 * c + 1] * f);
        __nv_bfloat16 *o = p.o + (out + r) * D + lane * kCols;
        if constexpr (kCols == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(packed[0], packed[1]);
        else *reinterpret_cast<uint32_t *>(o) = packed[0];
    }
    if (k8 == 0 && r8 < rows && p.lse) p.lse[out + r8] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

// Shares end with pairs where a pair can have at most this many keys.  In us, d = 128, with shares of equal length and
// with whole pairs, few rows (8 tokens x 8 heads): 1 x 8 pairs of 512 keys 12.5, 14.4 (and a launch less); 8 x 8 of 512
// 16.4, 14.4, of 1024 21.8, 17.4, of 2048 24.6, 24.6; 32 x 8 of 1024 40.9, 34.2, of 2048 59.6, 53.7; 128 x 8 of 256
// 53.7, 44.9.  Many rows: 8 x 8 pairs x 256 rows of 512 keys 22.6, 20.6, of 1024 24.8, 26.7; 32 x 8 x 512 of 1024 88, 85,
// of 2048 134, 137; 8 x 256 of 1024 20.5, 24.7.
long long whole_keys(bool few, long long pairs, int num_sms) {
    if (few) return pairs >= num_sms ? 2048 : 4 * pairs >= num_sms ? 1024 : 512;
    return pairs >= num_sms ? 1024 : 512;
}

struct Layout {
    int mt, shares;
    bool whole;
    size_t cuts, part_o, part_lse, bytes;
};
Layout layout_of(int B, int G, int Hkv, int T, int d, long long cap, int num_sms) {
    Layout l;
    const size_t rows = size_t(G) * T;
    const bool few = rows <= size_t(kTileM);
    l.mt = few ? 1 : int((rows + 2 * kTileM - 1) / (2 * kTileM));
    const int block = few ? 64 : 128;
    const long long most = (long long)B * Hkv * ((cap + block - 1) / block);
    const int groups = num_sms / l.mt > 0 ? num_sms / l.mt : 1;
    l.shares = int(most < groups ? most : groups);
    l.whole = cap <= whole_keys(few, (long long)B * Hkv, num_sms);
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    l.cuts = 0;
    l.part_o = up(size_t(l.shares) * sizeof(int4));
    l.part_lse = l.part_o + up(2 * size_t(l.shares) * rows * d * sizeof(float));
    l.bytes = l.part_lse + up(2 * size_t(l.shares) * rows * sizeof(float));
    return l;
}

template <int D>
int launch(const DecodeTreeLaunch &a, const Layout &l, cudaStream_t stream) {
    const int G = a.Hq / a.Hkv, rows = G * a.T;
    const bool few = rows <= kTileM;
    const int block = few ? PairCfg<D>::kBlock : RowsCfg<D>::kBlock, q_rows = few ? (rows + 7) / 8 * 8 : kTileM;
    CUtensorMap mq, mk, mv;
    const uint32_t box = uint32_t(a.table && a.page_size < block ? a.page_size : block);
    const uint64_t planes = uint64_t(a.num_pages) * a.Hkv;
    if (!encode_bf16_3d(&mq, a.q, D, uint64_t(rows), uint64_t(a.B) * a.Hkv, 64, uint32_t(q_rows)) ||
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
    p.T = a.T;
    p.rows = rows;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.shift = a.page_shift;
    p.cap = a.page_size * a.max_pages;
    p.max_pages = a.max_pages;
    p.mt = l.mt;
    p.shares = l.shares;
    p.whole = l.whole;
    p.wide = ((reinterpret_cast<uintptr_t>(a.o) | reinterpret_cast<uintptr_t>(a.workspace)) & 31u) == 0;
    p.q_rows = q_rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    auto kernel = few ? pairs_kernel<D> : rows_kernel<D>;
    const int threads = few ? PairCfg<D>::kThreads : kThreads;
    const int smem = few ? PairCfg<D>::smem_bytes(q_rows) : RowsCfg<D>::kSmemBytes;
    static bool attr_set[2][kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[few][dev]) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncGetAttributes(drafted tokens)");
        if (fa.numRegs != (few ? 65536 / PairCfg<D>::kThreads : kLaunchRegs) || fa.maxThreadsPerBlock < threads)
            return note_cuda_error(cudaErrorInvalidConfiguration, "register count differs from the setmaxnreg split (drafted tokens)");
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(drafted tokens)");
        if (dev >= 0) attr_set[few][dev] = true;
    }
    kernel<<<dim3(unsigned(l.shares * l.mt)), dim3(unsigned(threads)), smem, stream>>>(mq, mk, mv, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return note_cuda_error(e, "kernel launch (drafted tokens)");
    if (l.shares == 1 || l.whole) return 0;  // nothing is cut
    // Few pairs are cut into many partials each: then all warps of a block take a part of them.
    const bool split = l.shares >= 8LL * a.B * a.Hkv;
    const int per = split ? 4 : 4 * kMergeWarps, groups = (rows + per - 1) / per;
    const bool find = split && groups > 8;  // (see merge_kernel)
    e = dec::launch_programmatic(split ? merge_kernel<D, kMergeWarps> : merge_kernel<D, 1>,
                                 dim3(unsigned(find ? a.B * a.Hkv : l.shares), unsigned(groups)), dim3(kMergeWarps * 32), 0, stream, p);
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
    return a.d == 64 ? launch<64>(a, l, stream) : launch<128>(a, l, stream);
}

cudaError_t decode_tree_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_tree_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_tree_status, &zero, sizeof(int));
}

}  // namespace attn
