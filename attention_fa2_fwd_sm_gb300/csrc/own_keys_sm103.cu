// own_keys_sm103.cu -- decode over the sequences' own cached keys beside a shared
// prefix: one query row per query head, ragged lengths, softmax partials out.
//
// HBM-bound: 4 d bytes a key and KV head, each read once.  What keeps the
// memory busy is that no part of the GPU ever has less to do than another and
// that the rings never run dry, so the kernel is persistent and its shares are
// exact.  An SM holds one CTA of two or three groups: four warps that compute, one
// that issues TMA loads, a ring and barriers of their own.  With T keys in all,
// numbered by (sequence, KV head, key), group c takes keys [c S, (c + 1) S), S =
// ceil(T Hkv / groups) rounded up (find_share), however they fall on the sequences; a
// share is cut into segments at the ends of the sequences' heads, the group's TMA
// warp runs ahead over those ends while its other warps finish a segment, and the
// SM's other groups are not held up by either.  128 sequences of 512 to 1024 keys, 64
// heads, 8 KV heads, d = 128: 72 us with the merge, 5.6 TB/s; 32 of 8K to 16K: 225 us,
// 7.1 TB/s.  (One CTA a chunk, as in the ragged decode: 81 us, and up to 255, where
// 1.26 waves of equal chunks left SMs idle.)  The lengths are on the device; every
// warp finds its place in them by itself, from registers for up to 256 sequences.
//
// Segment partials are numbered c + (row b * Hkv + g): both numbers go up along
// the shares and one of them at every cut, so the numbers are distinct, a row's
// are consecutive, and there are at most groups + B * Hkv of them.
//
// A stage is 64 keys, 16 a warp.  Up to 8 query heads a KV head (kWide false) they
// are the N dimension of m16n8k16 MMAs: S^T = K Q^T and O^T = V^T P^T, keys and
// then columns of V on M, so that no row of an MMA is idle; P^T gets from the one
// layout to the other by movmatrix.  9 to 16 heads are the M dimension as in
// decode_sm103.cu.  Heads on N take half the MMAs and half the accumulator
// registers, which lets three groups share an SM instead of two; a stage takes its
// group about 1600 clocks, mostly latency, and one CTA an SM has to draw HBM's full
// rate from part of the SMs, because the prefix's kernel has the others: 90 GB/s an
// SM with up to 8 heads on N, 52 with them on M.  (On all SMs 72 and 74 us for the 128
// sequences above, 225 and 230 for the 32.)
//
// Probabilities are rounded to bf16 for the product with V, as in the other
// attention kernels: the instruction takes both operands in one 16-bit type, and V
// is bf16.  Each is off by at most 2^-8 of itself, independently of the others, so
// over many keys the outputs' own rounding is the larger: they are 1.0 to 1.4 times as
// far from the 64-bit result as with probabilities in 32 bits.  Everything that adds
// up stays in fp32: scores, maxima, sums (of the unrounded probabilities),
// accumulators, partials and weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_tile.cuh"
#include "own_keys.cuh"
#include "sm103_ptx.cuh"

namespace attn {

static __device__ int g_own_status;

namespace own {

using namespace dec;

// out = in^T for the 8 x 8 matrix of b16 whose row r is in lanes 4r .. 4r + 3.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t in) {
    uint32_t out;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(out) : "r"(in));
    return out;
}

template <int D, bool kWide>
struct Cfg {
    static constexpr int kGroups = kWide ? 2 : 3, kWarps = kGroups * kConsumerWarps;  // consumer warps
    static constexpr int kThreads = (kWarps + kGroups) * 32;
    static constexpr int kStages = (D == 128 ? 6 : 12) / kGroups;  // of a group's ring
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = kKeysPerStage * 128;
    static constexpr int kTileBytes = kKeysPerStage * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kGroups * kStages * kStageBytes;
    // Combine area of a consumer warp: kRows heads of kCols columns, kStride
    // words apart (no bank conflicts on the way in), and (maximum, sum) a head.
    static constexpr int kRows = kWide ? 16 : 8, kCols = kWide ? 32 : 64, kStride = kWide ? 40 : 68;
    static constexpr int kTurnBytes = kWarps * kRows * kStride * 4;
    static constexpr int kStateBytes = kWarps * kRows * 8;
    static constexpr int kSmemBytes = kRingBytes + kTurnBytes + kStateBytes + kGroups * 2 * kStages * 8 + 16 + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct Params {
    const __nv_bfloat16 *q;
    const int *seqlens;
    float *part_o, *part_lse;  // [partial][G][D], [partial][G] (log2 units)
    float *scores;             // [B, Hkv, max_seqlen, G] log2 units, or null
    long long *plan;           // {S, T Hkv, first key of each sequence in the numbering}
    int2 *rows;                // [B * Hkv] first partial and number of partials (rows with keys only)
    int B, Hq, Hkv, G, max_seqlen;
    int narrow;  // fewer than 2^29 keys in the caches
    float scale_log2;
    unsigned long long wait_ns;
};

// The lengths of 256 sequences from `first` on, over the lanes of a warp.
constexpr int kRound = 8;
__device__ __forceinline__ void load_lengths(const Params &p, int first, int (&len)[kRound]) {
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
        const int i = first + 32 * k + int(threadIdx.x & 31);
        len[k] = i < p.B ? length_of(p.seqlens, p.max_seqlen, i) : 0;
    }
}

// Where group `cta` of `ctas` starts (left = 0: it has no share).  All lanes of
// the calling warp; `write`: also write the plan down.  Int: wide enough for the
// number of keys, so that the common case scans and divides in 32 bits.
// `len` holds load_lengths(0), which the caller has had time to wait for.
template <typename Int>
__device__ __forceinline__ Place find_share(const Params &p, int (&len)[kRound], int cta, int ctas, bool write) {
    const int lane = threadIdx.x & 31;
    Int T = 0;
    for (int first = 0; first < p.B; first += 32 * kRound) {
        if (first > 0) load_lengths(p, first, len);
#pragma unroll
        for (int k = 0; k < kRound; ++k) T += len[k];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) T += __shfl_xor_sync(0xffffffffu, T, off);
    T *= Int(p.Hkv);
    Int S = (T + Int(ctas) - 1) / Int(ctas);
    // Whole stages where there are keys enough; few keys are better spread.
    const Int unit = S > 4 * kKeysPerStage ? Int(kKeysPerStage) : Int(kMinShare);
    S = S == 0 ? unit : (S + unit - 1) / unit * unit;
    const Int lo = Int(cta) * S;
    if (write && lane == 0) {
        p.plan[0] = (long long)S;
        p.plan[1] = (long long)T;
    }
    Place at = {0, 0, 0, 0, lo < T ? (long long)min(S, T - lo) : 0};
    Int before = 0;  // keys of the sequences before, over all KV heads
    bool searching = at.left > 0;
    for (int first = 0; first < p.B && (write || searching); first += 32 * kRound) {
        if (p.B > 32 * kRound) load_lengths(p, first, len);
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            if (first + 32 * k >= p.B) break;
            const Int n = Int(len[k]) * Int(p.Hkv);
            Int upto = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const Int y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
            const Int base = before + upto - n;
            if (write && first + 32 * k + lane < p.B) p.plan[2 + first + 32 * k + lane] = (long long)base;
            const uint32_t hit = __ballot_sync(0xffffffffu, searching && lo >= base && lo < base + n);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const Int rem = lo - __shfl_sync(0xffffffffu, base, src);
                at.b = first + 32 * k + src;
                at.len = __shfl_sync(0xffffffffu, len[k], src);
                at.g = int(rem / Int(at.len));
                at.j = int(rem - Int(at.g) * Int(at.len));
                searching = false;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    return at;
}

// Among the four computing warps of a group.
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kConsumerWarps * 32) : "memory");
}

// One segment's running state in a consumer warp: the maxima and (per lane) sums
// of the two heads that this lane's scores belong to, and the output
// accumulators.  kWide: heads gq and gq + 8, acc[c] = O[heads][8 c ..]; else heads
// 2 tq and 2 tq + 1, acc[c] = O^T[16 c ..][heads].
template <int D, bool kWide>
struct State {
    static constexpr int kTiles = kWide ? D / 8 : D / 16;
    float m[2], l[2], acc[kTiles][4];
    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][i] = 0.f;
    }
    // acc[c][i] belongs to head index head(i).
    static __device__ __forceinline__ constexpr int head(int i) { return kWide ? i >> 1 : i & 1; }
    // The maxima move to at least mx; returns the exponents' offsets.
    __device__ __forceinline__ void raise(const float (&mx)[2], float (&offset)[2]) {
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m_new = fmaxf(m[r], mx[r]);
            corr[r] = m_new == -INFINITY ? 1.f : fast_exp2(m[r] - m_new);
            m[r] = m_new;
            offset[r] = m_new == -INFINITY ? 0.f : -m_new;
            l[r] *= corr[r];
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][i] *= corr[head(i)];
        }
    }
};

// Query heads of one KV head as MMA operands.
template <int D, bool kWide>
struct Queries {
    static constexpr int kRegs = kWide ? 4 : 2;
    uint32_t v[D / 16][kRegs];
    __device__ __forceinline__ void load(const Params &p, int row) {
        const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
        const __nv_bfloat16 *q = p.q + ((size_t)row * p.G + gq) * D + tq * 2;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
                // kWide: A operand, registers (head gq, gq + 8) x (columns, columns + 8); else B, columns, columns + 8.
                const int up = kWide ? i & 1 : 0, right = kWide ? i >> 1 : i;
                v[ks][i] = gq + 8 * up < p.G ? *reinterpret_cast<const uint32_t *>(q + 8 * up * D + ks * 16 + 8 * right) : 0u;
            }
    }
};

// 16 keys of a stage, rows key0 .. key0 + 15 of the tiles at kt and vt, of which
// n_valid (1..16) belong to the segment; `scores`: where the first one's go, or null.
template <int D>
__device__ __forceinline__ void add_keys(State<D, true> &st, const Queries<D, true> &q, uint32_t kt, uint32_t vt, int key0,
                                         int n_valid, float sl2, int G, float *scores) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3, sub = lane >> 3, rr = lane & 7;
    float sc[2][4] = {};
    {
        const int key = key0 + ((sub & 2) ? 8 : 0) + rr;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(tile_unit_addr(kt, key, 2 * ks + (sub & 1)), b0, b1, b2, b3);
            mma_bf16_16816(sc[0], q.v[ks], b0, b1);
            mma_bf16_16816(sc[1], q.v[ks], b2, b3);
        }
    }
    // Scores in log2 units, masked past the segment's end.
    float mx[2] = {-INFINITY, -INFINITY}, offset[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int kl = h * 8 + tq * 2 + (e & 1), hq = gq + ((e & 2) ? 8 : 0);
            const bool in = kl < n_valid;
            sc[h][e] = in ? sc[h][e] * sl2 : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], sc[h][e]);
            if (scores && in && hq < G) scores[kl * G + hq] = sc[h][e];
        }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    }
    st.raise(mx, offset);
    uint32_t pa[4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float p0 = fast_exp2(sc[h][2 * r] + offset[r]), p1 = fast_exp2(sc[h][2 * r + 1] + offset[r]);
            st.l[r] += p0 + p1;
            pa[2 * h + r] = pack_bf16x2(p0, p1);
        }
    const int key = key0 + ((sub & 1) ? 8 : 0) + rr;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(tile_unit_addr(vt, key, 2 * c + (sub >> 1)), b0, b1, b2, b3);
        if (n_valid < 16) {
            b0 = mask_pair(b0, 2 * tq, n_valid);
            b1 = mask_pair(b1, 8 + 2 * tq, n_valid);
            b2 = mask_pair(b2, 2 * tq, n_valid);
            b3 = mask_pair(b3, 8 + 2 * tq, n_valid);
        }
        mma_bf16_16816(st.acc[2 * c], pa, b0, b1);
        mma_bf16_16816(st.acc[2 * c + 1], pa, b2, b3);
    }
}

template <int D>
__device__ __forceinline__ void add_keys(State<D, false> &st, const Queries<D, false> &q, uint32_t kt, uint32_t vt, int key0,
                                         int n_valid, float sl2, int G, float *scores) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3, sub = lane >> 3, rr = lane & 7;
    float sa[4] = {}, sb[4] = {};  // two chains of MMAs, over the even and the odd steps
    {
        const int key = key0 + ((sub & 1) ? 8 : 0) + rr;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a[4];
            ldsm_x4(tile_unit_addr(kt, key, 2 * ks + (sub >> 1)), a[0], a[1], a[2], a[3]);
            mma_bf16_16816(ks & 1 ? sb : sa, a, q.v[ks][0], q.v[ks][1]);
        }
    }
    // sa: (key gq, heads 2tq and 2tq + 1), (key gq + 8, the same), in log2 units, masked past the segment's end.
    float mx[2], offset[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) sa[e] = gq + 8 * (e >> 1) < n_valid ? (sa[e] + sb[e]) * sl2 : -INFINITY;
    if (scores) {
        float *to = scores + gq * G + 2 * tq;
#pragma unroll
        for (int k = 0; k < 2; ++k, to += 8 * G)
            if (gq + 8 * k < n_valid) {
                if ((G & 1) == 0) {
                    if (2 * tq < G) *reinterpret_cast<float2 *>(to) = make_float2(sa[2 * k], sa[2 * k + 1]);
                } else {
                    if (2 * tq < G) to[0] = sa[2 * k];
                    if (2 * tq + 1 < G) to[1] = sa[2 * k + 1];
                }
            }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(sa[r], sa[2 + r]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], off));
    }
    st.raise(mx, offset);
    float pr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        pr[e] = fast_exp2(sa[e] + offset[e & 1]);
        st.l[e & 1] += pr[e];
    }
    // P^T (keys x heads) as the B operand.
    const uint32_t b0 = transpose_8x8(pack_bf16x2(pr[0], pr[1])), b1 = transpose_8x8(pack_bf16x2(pr[2], pr[3]));
    const int key = key0 + ((sub & 2) ? 8 : 0) + rr;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint32_t a[4];
        ldsm_x4_t(tile_unit_addr(vt, key, 2 * c + (sub & 1)), a[0], a[1], a[2], a[3]);
        if (n_valid < 16) {
            a[0] = mask_pair(a[0], 2 * tq, n_valid);
            a[1] = mask_pair(a[1], 2 * tq, n_valid);
            a[2] = mask_pair(a[2], 8 + 2 * tq, n_valid);
            a[3] = mask_pair(a[3], 8 + 2 * tq, n_valid);
        }
        mma_bf16_16816(st.acc[c], a, b0, b1);
    }
}

template <int D, bool kWide>
__global__ void __launch_bounds__(Cfg<D, kWide>::kThreads, 1)
    own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16, const Params p) {
    using C = Cfg<D, kWide>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *turns = reinterpret_cast<float *>(smem + C::kRingBytes);                     // [group][warp][kRows][kStride]
    float2 *states = reinterpret_cast<float2 *>(smem + C::kRingBytes + C::kTurnBytes);  // [group][warp][kRows]
    uint64_t *barriers = reinterpret_cast<uint64_t *>(smem + C::kRingBytes + C::kTurnBytes + C::kStateBytes);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(barriers + C::kGroups * 2 * C::kStages);
    int *status = &g_own_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Computing warps first, then a TMA warp for every group.
    const bool loads = warp >= C::kWarps;
    const int group = loads ? warp - C::kWarps : warp / kConsumerWarps, slice = warp % kConsumerWarps;
    const int part0 = blockIdx.x * C::kGroups + group;  // the group's number in the grid
    uint8_t *ring = smem + group * C::kStages * C::kStageBytes;
    uint64_t *bars = barriers + group * 2 * C::kStages;  // full, then empty
    float *turn = turns + group * kConsumerWarps * C::kRows * C::kStride;
    float2 *state = states + group * kConsumerWarps * C::kRows;

    griddep_launch_dependents();  // the prefix's grid, which reads nothing from here, may take the other SMs
    int lengths[kRound];
    load_lengths(p, 0, lengths);
    if (threadIdx.x == 0) {
        for (int g = 0; g < C::kGroups; ++g)
            for (int s = 0; s < C::kStages; ++s) {
                mbar_init(smem_u32(barriers + (2 * g) * C::kStages + s), 1);                   // full
                mbar_init(smem_u32(barriers + (2 * g + 1) * C::kStages + s), kConsumerWarps);  // empty
            }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == C::kWarps * 32) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    const bool write = blockIdx.x == 0 && warp == 0;
    // (groups + 1) shares stay below 2^31 where the caches' keys stay below 2^29.
    Place at = p.narrow ? find_share<unsigned>(p, lengths, part0, gridDim.x * C::kGroups, write)
                        : find_share<long long>(p, lengths, part0, gridDim.x * C::kGroups, write);
    __syncthreads();
    if (at.left == 0) return;  // whole warps; nothing below waits for all of the CTA

    // Share, where a row can go on behind it (a longer one holds every row's rest; the last may be shorter).
    const unsigned share = unsigned(min(at.left, 0x40000000LL));
    int slot = 0, round = 0;  // of the ring's next stage to issue (producer) or use (consumers)
    if (loads) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            bool ok = true;
            while (ok) {
                const int n = at.keys(), plane = at.b * p.Hkv + at.g;
                for (int i = 0; i < n; i += kKeysPerStage) {
                    const int s = slot;
                    ok = round == 0 || mbar_wait_bounded(smem_u32(bars + C::kStages + s), (round - 1) & 1, p.wait_ns,
                                                         abort_flag, status);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(bars + s), kt = smem_u32(ring + s * C::kStageBytes);
                    const int key = at.j + i;
                    if (n - i >= kKeysPerStage) {
                        mbar_arrive_expect_tx(fb, C::kStageBytes);
#pragma unroll
                        for (int c = 0; c < C::kChunks; ++c) {
                            tma_load_3d(kt + c * C::kChunkBytes, &tmK, fb, c * 64, key, plane);
                            tma_load_3d(kt + C::kTileBytes + c * C::kChunkBytes, &tmV, fb, c * 64, key, plane);
                        }
                    } else {
                        // A segment's end: only the groups of 16 keys that a warp will use.
                        const int groups = (n - i + 15) / 16;
                        mbar_arrive_expect_tx(fb, groups * 16 * D * 4);
                        for (int w = 0; w < groups; ++w)
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c) {
                                const uint32_t to = kt + c * C::kChunkBytes + w * 2048;
                                tma_load_3d(to, &tmK16, fb, c * 64, key + 16 * w, plane);
                                tma_load_3d(to + C::kTileBytes, &tmV16, fb, c * 64, key + 16 * w, plane);
                            }
                    }
                    if (++slot == C::kStages) slot = 0, ++round;
                }
                if (!ok) break;
                at.left -= n;
                if (at.left == 0) break;
                at.next(p.seqlens, p.max_seqlen, p.Hkv);
            }
            // Whatever becomes of the other warps, this one leaves only when the
            // last fill of every slot has landed (bounded, by a second at least), so
            // that no copy writes shared memory when the CTA is gone.
            volatile int no_abort = 0;
            const uint64_t limit = p.wait_ns > 1000000000ull ? p.wait_ns : 1000000000ull;
            for (int s = 0; s < C::kStages; ++s) {
                const int last = s < slot ? round : round - 1;  // round of this slot's last fill
                if (last >= 0 && !mbar_wait_bounded(smem_u32(bars + s), last & 1, limit, &no_abort, status))
                    atomicOr(status, kStatusDrainTimeout);
            }
        }
    } else {
        // ------------------------------------------------------------ consumer
        // A warp whose wait ran out does no more work but still meets the others
        // at every barrier of the segments ahead.
        const int gq = lane >> 2, tq = lane & 3;
        bool ok = true;
        Queries<D, kWide> q;
        q.load(p, at.b * p.Hkv + at.g);
        State<D, kWide> st;
        while (true) {
            const int n = at.keys(), row = at.b * p.Hkv + at.g, len = at.len;
            const bool first_of_row = at.j == 0;
            st.clear();
            float *scores = p.scores ? p.scores + ((size_t)row * p.max_seqlen + at.j + slice * 16) * p.G : nullptr;
            for (int i = 0; ok && i < n; i += kKeysPerStage) {
                const int s = slot, phase = round & 1;
                if (++slot == C::kStages) slot = 0, ++round;
                ok = mbar_wait_warp(smem_u32(bars + s), phase, p.wait_ns, abort_flag, status);
                if (!ok) break;
                const int n_valid = min(16, n - i - slice * 16);  // keys of this warp
                if (n_valid > 0) {
                    const uint32_t kt = smem_u32(ring + s * C::kStageBytes);
                    add_keys<D>(st, q, kt, kt + C::kTileBytes, slice * 16, n_valid, p.scale_log2, p.G,
                                scores ? scores + (size_t)i * p.G : nullptr);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(bars + C::kStages + s));
            }

            // On to the next segment: its queries arrive while this one is finished.
            at.left -= n;
            if (at.left > 0) {
                at.next(p.seqlens, p.max_seqlen, p.Hkv);
                q.load(p, at.b * p.Hkv + at.g);
            }

            // The warps' states become the segment's partial, kCols columns at a time.
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = st.l[r];
                if constexpr (kWide) {
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    if (tq == 0) state[slice * C::kRows + gq + 8 * r] = make_float2(st.m[r], l);
                } else {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                    if (gq == 0) state[slice * C::kRows + 2 * tq + r] = make_float2(st.m[r], l);
                }
            }
            group_sync(group);
            // Lane l of every warp: the maximum and sum of head l % kRows over the
            // warps, each of the 32 / kRows lanes of a head over some of them.
            constexpr int kPer = kConsumerWarps * C::kRows / 32;
            float2 theirs[kPer];
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                theirs[k] = state[lane + 32 * k];  // [warp][head] flat
                top = fmaxf(top, theirs[k].x);
            }
#pragma unroll
            for (int off = C::kRows; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int k = 0; k < kPer; ++k) sum += fast_exp2(theirs[k].x - ref) * theirs[k].y;
#pragma unroll
            for (int off = C::kRows; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float over = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) f[r] = fast_exp2(st.m[r] - __shfl_sync(0xffffffffu, ref, kWide ? gq + 8 * r : 2 * tq + r));
            const size_t part = (size_t)part0 + row;
            if (first_of_row && slice == 0 && lane == 0)
                p.rows[row] = make_int2(int(part), 1 + int((unsigned(len - n) + share - 1) / share));
            if (ok && slice == 0 && lane < p.G)
                p.part_lse[part * p.G + lane] = sum == 0.f ? -INFINITY : top + __log2f(sum);
            // A warp stores heads `slice`, `slice` + 4, ...
            constexpr int kStores = C::kRows / kConsumerWarps;
            float inv[kStores];
#pragma unroll
            for (int k = 0; k < kStores; ++k) inv[k] = __shfl_sync(0xffffffffu, over, slice + kConsumerWarps * k);
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += C::kCols) {
                float *mine = turn + slice * C::kRows * C::kStride;
                if constexpr (kWide) {
#pragma unroll
                    for (int u = 0; u < C::kCols / 8; ++u) {
                        const float(&a)[4] = st.acc[c0 / 8 + u];
                        float *to = mine + gq * C::kStride + u * 8 + tq * 2;
                        *reinterpret_cast<float2 *>(to) = make_float2(a[0] * f[0], a[1] * f[0]);
                        *reinterpret_cast<float2 *>(to + 8 * C::kStride) = make_float2(a[2] * f[1], a[3] * f[1]);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < C::kCols / 16; ++u) {
                        const float(&a)[4] = st.acc[c0 / 16 + u];
                        float *to = mine + 2 * tq * C::kStride + u * 16 + gq;
                        to[0] = a[0] * f[0];
                        to[C::kStride] = a[1] * f[1];
                        to[8] = a[2] * f[0];
                        to[C::kStride + 8] = a[3] * f[1];
                    }
                }
                group_sync(group);
#pragma unroll
                for (int k = 0; k < kStores; ++k) {
                    const int h = slice + kConsumerWarps * k;
                    if (h >= p.G) break;
                    float *to = p.part_o + (part * p.G + h) * D + c0;
                    if constexpr (kWide) {
                        float v = 0.f;
#pragma unroll
                        for (int w = 0; w < kConsumerWarps; ++w) v += turn[(w * C::kRows + h) * C::kStride + lane];
                        if (ok) to[lane] = v * inv[k];
                    } else {
                        float2 v = make_float2(0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kConsumerWarps; ++w) {
                            const float2 x = *reinterpret_cast<const float2 *>(turn + (w * C::kRows + h) * C::kStride + 2 * lane);
                            v.x += x.x;
                            v.y += x.y;
                        }
                        if (ok) *reinterpret_cast<float2 *>(to + 2 * lane) = make_float2(v.x * inv[k], v.y * inv[k]);
                    }
                }
                group_sync(group);
            }
            if (at.left == 0) break;
        }
    }
}

template <int D, bool kWide>
int launch(const DecodePrefixLaunch &a, const PrefixLayout &l, cudaStream_t stream) {
    using C = Cfg<D, kWide>;
    CUtensorMap mk, mv, mk16, mv16;
    const uint64_t planes = uint64_t(a.B) * a.Hkv, keys = uint64_t(a.max_seqlen);
    if (!encode_bf16_3d(&mk, a.kcache, D, keys, planes, 64, kKeysPerStage) ||
        !encode_bf16_3d(&mv, a.vcache, D, keys, planes, 64, kKeysPerStage) ||
        !encode_bf16_3d(&mk16, a.kcache, D, keys, planes, 64, 16) ||
        !encode_bf16_3d(&mv16, a.vcache, D, keys, planes, 64, 16))
        return note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (own keys)");
    Params p = {};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.seqlens = a.seqlens;
    p.part_o = reinterpret_cast<float *>(a.workspace + l.own_o);
    p.part_lse = reinterpret_cast<float *>(a.workspace + l.own_lse);
    p.scores = a.weights ? reinterpret_cast<float *>(a.workspace + l.scores) : nullptr;
    p.plan = reinterpret_cast<long long *>(a.workspace + l.plan);
    p.rows = reinterpret_cast<int2 *>(a.workspace + l.own_rows);
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.max_seqlen = a.max_seqlen;
    p.narrow = planes * keys < (1ull << 29);
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.wait_ns = a.wait_ns;
    auto kernel = own_kernel<D, kWide>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(own_kernel)");
        if (dev >= 0) attr_set[dev] = true;
    }
    kernel<<<dim3(unsigned(l.own_ctas)), dim3(C::kThreads), C::kSmemBytes, stream>>>(mk, mv, mk16, mv16, p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "own_kernel launch");
}

}  // namespace own

int own_launch(const DecodePrefixLaunch &a, const PrefixLayout &l, cudaStream_t stream) {
    const bool wide = a.Hq / a.Hkv > 8;
    if (a.d == 64) return wide ? own::launch<64, true>(a, l, stream) : own::launch<64, false>(a, l, stream);
    return wide ? own::launch<128, true>(a, l, stream) : own::launch<128, false>(a, l, stream);
}

cudaError_t own_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_own_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_own_status, &zero, sizeof(int));
}

}  // namespace attn
