// own_keys_sm103.cu -- decode over the sequences' own cached keys beside a shared
// prefix: one query row per query head, ragged lengths, softmax partials out.
//
// HBM-bound: 4 d bytes a key and KV head, each read once.  What keeps the
// memory busy is that no CTA ever has less to do than another and that its ring
// never runs dry, so the kernel is persistent and its share exact: with T keys
// in all, numbered by (sequence, KV head, key), CTA c takes keys [c S, (c + 1) S),
// S = max(kMinShare, ceil(T Hkv / CTAs) rounded up to 64), however they fall on
// the sequences; a share is cut into segments at the ends of the sequences' heads,
// and the TMA warp runs ahead over those ends while the other warps finish a
// segment.  (One CTA a chunk, as in the ragged decode: 81 us on 128 sequences of
// 512 to 1024 keys, 8 KV heads, d = 128, and up to 255 us on 32 of 8K to 16K,
// where 1.26 waves of equal chunks left SMs idle.)  The lengths are on the device;
// every warp finds its place in them by itself, from registers for up to 256
// sequences.
//
// Segment partials are numbered c + (row b * Hkv + g): both numbers go up along
// the shares and one of them at every cut, so the numbers are distinct, a row's
// are consecutive, and there are at most CTAs + B * Hkv of them.
//
// The arithmetic of a stage is the decode kernel's (decode_sm103.cu): four warps
// of 16 keys each, m16n8k16 MMAs with the group's query heads on M, a running
// maximum and sum a warp.  A stage takes four warps about 1400 clocks, mostly
// latency, so two groups of four take turns: one CTA an SM then draws HBM's full
// rate from half of the SMs, and the prefix's kernel has the others.
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

constexpr int kGroups = 2, kWarps = kGroups * kConsumerWarps;  // consumer warps: a group takes every other stage
constexpr int kOwnThreads = (kWarps + 1) * 32;

template <int D>
struct Cfg {
    static constexpr int kStages = D == 128 ? 6 : 12;  // even: a slot always belongs to the same group
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = kKeysPerStage * 128;
    static constexpr int kTileBytes = kKeysPerStage * D * 2;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kRingBytes = kStages * kStageBytes;
    // Combine area: 16 rows of 32 columns (40 words apart: no bank conflicts)
    // and (maximum, sum) per row for each consumer warp.
    static constexpr int kTurnStride = 40;
    static constexpr int kTurnBytes = kWarps * kMaxGroup * kTurnStride * 4;
    static constexpr int kStateBytes = kWarps * kMaxGroup * 8;
    static constexpr int kSmemBytes = kRingBytes + kTurnBytes + kStateBytes + 2 * kStages * 8 + 16 + 1024;
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

// Where CTA `cta` of `ctas` starts (left = 0: it has no share).  All lanes of
// the calling warp; `write`: also write the plan down.  Int: wide enough for the
// number of keys, so that the common case scans and divides in 32 bits.
template <typename Int>
__device__ __forceinline__ Place find_share(const Params &p, int cta, int ctas, bool write) {
    constexpr int kRound = 8;  // groups of 32 sequences whose lengths are loaded together
    const int lane = threadIdx.x & 31;
    int len[kRound];
    auto load = [&](int first) {
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const int i = first + 32 * k + lane;
            len[k] = i < p.B ? length_of(p.seqlens, p.max_seqlen, i) : 0;
        }
    };
    Int T = 0;
    for (int first = 0; first < p.B; first += 32 * kRound) {
        load(first);
#pragma unroll
        for (int k = 0; k < kRound; ++k) T += len[k];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) T += __shfl_xor_sync(0xffffffffu, T, off);
    T *= Int(p.Hkv);
    Int S = ((T + Int(ctas) - 1) / Int(ctas) + kKeysPerStage - 1) / kKeysPerStage * kKeysPerStage;
    if (S < kMinShare) S = kMinShare;
    const Int lo = Int(cta) * S;
    if (write && lane == 0) {
        p.plan[0] = (long long)S;
        p.plan[1] = (long long)T;
    }
    Place at = {0, 0, 0, 0, lo < T ? (long long)min(S, T - lo) : 0};
    Int before = 0;  // keys of the sequences before, over all KV heads
    bool searching = at.left > 0;
    for (int first = 0; first < p.B && (write || searching); first += 32 * kRound) {
        if (p.B > 32 * kRound) load(first);
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

__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 1)
    own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16, const Params p) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *turn = reinterpret_cast<float *>(smem + C::kRingBytes);                          // [warp][16][40]
    float2 *state = reinterpret_cast<float2 *>(smem + C::kRingBytes + C::kTurnBytes);       // [warp][16]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kRingBytes + C::kTurnBytes + C::kStateBytes);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 2 * C::kStages);
    int *status = &g_own_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_launch_dependents();  // the prefix's grid, which reads nothing from here, may take the other SMs
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(bars + s), 1);                            // full
            mbar_init(smem_u32(bars + C::kStages + s), kConsumerWarps);  // empty: the group that used it
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == kWarps * 32) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    const bool write = blockIdx.x == 0 && warp == 0;
    // (CTAs + 1) shares stay below 2^31 where the caches' keys stay below 2^29: a share is at most twice its equal part or kMinShare.
    Place at = p.narrow ? find_share<unsigned>(p, blockIdx.x, gridDim.x, write)
                        : find_share<long long>(p, blockIdx.x, gridDim.x, write);
    __syncthreads();
    if (at.left == 0) return;

    // Share, where a row can go on behind it (a longer one holds every row's rest; the last may be shorter).
    const unsigned share = unsigned(min(at.left, 0x40000000LL));
    long long fills = 0;  // ring fills issued (producer) or used (consumers)
    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            bool ok = true;
            while (ok) {
                const int n = at.keys(), plane = at.b * p.Hkv + at.g;
                for (int i = 0; i < n; i += kKeysPerStage) {
                    const int s = int(fills % C::kStages);
                    const long long round = fills / C::kStages;
                    ok = round == 0 || mbar_wait_bounded(smem_u32(bars + C::kStages + s), (round - 1) & 1, p.wait_ns,
                                                         abort_flag, status);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(bars + s), kt = smem_u32(smem + s * C::kStageBytes);
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
                    ++fills;
                }
                at.left -= n;
                if (at.left == 0) break;
                at.next(p.seqlens, p.max_seqlen, p.Hkv);
            }
        }
    } else {
        // ------------------------------------------------------------ consumer
        // A warp whose wait ran out does no more work but still meets the others
        // at every barrier of the segments ahead.
        const int gq = lane >> 2, tq = lane & 3;
        const float sl2 = p.scale_log2;
        const int group = warp / kConsumerWarps, slice = warp % kConsumerWarps;  // of the stages; of a stage's keys
        bool ok = true;
        // Q fragments (A operand, rows = query heads of the group, k = head dim).
        uint32_t qa[D / 16][4];
        auto load_q = [&](int row) {
            const __nv_bfloat16 *q = p.q + ((size_t)row * p.G + gq) * D + tq * 2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qa[ks][i] = gq + ((i & 1) ? 8 : 0) < p.G
                                    ? *reinterpret_cast<const uint32_t *>(q + ((i & 1) ? 8 * D : 0) + ks * 16 + ((i & 2) ? 8 : 0))
                                    : 0u;
        };
        load_q(at.b * p.Hkv + at.g);
        while (true) {
            const int n = at.keys(), row = at.b * p.Hkv + at.g, len = at.len;
            const bool first_of_row = at.j == 0;
            float m_st[2] = {-INFINITY, -INFINITY}, l_st[2] = {0.f, 0.f};
            float acc[D / 8][4];
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][i] = 0.f;
            for (int i = 0; ok && i < n; i += kKeysPerStage, ++fills) {
                if (int(fills & 1) != group) continue;
                const int s = int(fills % C::kStages);
                ok = mbar_wait_warp(smem_u32(bars + s), (fills / C::kStages) & 1, p.wait_ns, abort_flag, status);
                if (!ok) break;
                const int n_valid = min(16, n - i - slice * 16);  // keys of this warp
                if (n_valid > 0) {
                    const uint32_t kt = smem_u32(smem + s * C::kStageBytes), vt = kt + C::kTileBytes;
                    const int sub = lane >> 3, rr = lane & 7;
                    float sc[2][4] = {};
                    {
                        const int key = slice * 16 + ((sub & 2) ? 8 : 0) + rr;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(tile_unit_addr(kt, key, 2 * ks + (sub & 1)), b0, b1, b2, b3);
                            mma_bf16_16816(sc[0], qa[ks], b0, b1);
                            mma_bf16_16816(sc[1], qa[ks], b2, b3);
                        }
                    }
                    // Scores in log2 units, masked past the segment's end.
                    float x[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int kl = h * 8 + tq * 2 + (e & 1);
                            x[h][e] = kl < n_valid ? sc[h][e] * sl2 : -INFINITY;
                        }
                    if (p.scores) {
                        float *to = p.scores + ((size_t)row * p.max_seqlen + at.j + i + slice * 16) * p.G;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kl = h * 8 + tq * 2 + (e & 1), hq = gq + ((e & 2) ? 8 : 0);
                                if (kl < n_valid && hq < p.G) to[kl * p.G + hq] = x[h][e];
                            }
                    }
                    uint32_t pa[4];
                    float corr[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {  // rows gq (e = 0, 1) and gq + 8 (e = 2, 3)
                        float mx = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float m_new = fmaxf(m_st[r], mx);
                        corr[r] = m_new == -INFINITY ? 1.f : fast_exp2(m_st[r] - m_new);
                        m_st[r] = m_new;
                        const float nm = m_new == -INFINITY ? 0.f : -m_new;
                        const float p00 = fast_exp2(x[0][2 * r] + nm), p01 = fast_exp2(x[0][2 * r + 1] + nm);
                        const float p10 = fast_exp2(x[1][2 * r] + nm), p11 = fast_exp2(x[1][2 * r + 1] + nm);
                        l_st[r] = l_st[r] * corr[r] + (p00 + p01 + p10 + p11);
                        pa[r] = pack_bf16x2(p00, p01);      // keys 2tq..: rounded to bf16 for the product with V
                        pa[2 + r] = pack_bf16x2(p10, p11);  // keys 8 + 2tq..
                    }
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        acc[c][0] *= corr[0];
                        acc[c][1] *= corr[0];
                        acc[c][2] *= corr[1];
                        acc[c][3] *= corr[1];
                    }
                    {
                        const int key = slice * 16 + ((sub & 1) ? 8 : 0) + rr;
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
                            mma_bf16_16816(acc[2 * c], pa, b0, b1);
                            mma_bf16_16816(acc[2 * c + 1], pa, b2, b3);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(bars + C::kStages + s));
            }

            // On to the next segment: its queries arrive while this one is finished.
            at.left -= n;
            if (at.left > 0) {
                at.next(p.seqlens, p.max_seqlen, p.Hkv);
                load_q(at.b * p.Hkv + at.g);
            }

            // The warps' states become the segment's partial, 32 columns at a time.
            const bool high = p.G > 8;  // rows 8..15 are in use
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = l_st[r];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (tq == 0 && (r == 0 || high)) state[warp * kMaxGroup + gq + 8 * r] = make_float2(m_st[r], l);
            }
            consumer_sync();
            float f[2] = {0.f, 0.f};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float top = -INFINITY;
                if (r == 1 && !high) break;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[w * kMaxGroup + gq + 8 * r].x);
                f[r] = fast_exp2(m_st[r] - (top == -INFINITY ? 0.f : top));
            }
            const size_t part = (size_t)blockIdx.x + row;
            if (first_of_row && threadIdx.x == 0)
                p.rows[row] = make_int2(int(part), 1 + int((unsigned(len - n) + share - 1) / share));
            // A thread stores column `col` of rows row0 and row0 + 8: their sums once, ahead of the columns.
            const int col = threadIdx.x & 31, row0 = threadIdx.x >> 5;
            float inv[kMaxGroup / kWarps];
#pragma unroll
            for (int k = 0; k < kMaxGroup / kWarps; ++k) {
                const int h = row0 + kWarps * k;
                if (h >= p.G) break;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[w * kMaxGroup + h].x);
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 st = state[w * kMaxGroup + h];
                    sum += fast_exp2(st.x - ref) * st.y;
                }
                inv[k] = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
                if (ok && col == 0) p.part_lse[part * p.G + h] = sum == 0.f ? -INFINITY : top + __log2f(sum);
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float *mine = turn + (warp * kMaxGroup + gq) * C::kTurnStride + tq * 2;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float(&a)[4] = acc[4 * c + u];
                    *reinterpret_cast<float2 *>(mine + u * 8) = make_float2(a[0] * f[0], a[1] * f[0]);
                    if (high)
                        *reinterpret_cast<float2 *>(mine + 8 * C::kTurnStride + u * 8) =
                            make_float2(a[2] * f[1], a[3] * f[1]);
                }
                consumer_sync();
#pragma unroll
                for (int k = 0; k < kMaxGroup / kWarps; ++k) {
                    const int h = row0 + kWarps * k;
                    if (h >= p.G) break;
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += turn[(w * kMaxGroup + h) * C::kTurnStride + col];
                    if (ok) p.part_o[(part * p.G + h) * D + c * 32 + col] = v * inv[k];
                }
                consumer_sync();
            }
            if (at.left == 0) break;
        }
    }
    __syncthreads();
    if (*abort_flag && warp == kWarps && lane == 0) {
        // A wait ran out.  Before the CTA exits, wait (bounded, with a fixed
        // limit) for the copies of the last fill of every ring slot so that none
        // is still writing shared memory.
        volatile int no_abort = 0;
        for (long long i = fills > C::kStages ? fills - C::kStages : 0; i < fills; ++i)
            if (!mbar_wait_bounded(smem_u32(bars + i % C::kStages), (i / C::kStages) & 1, 1000000000ull, &no_abort,
                                   status))
                atomicOr(status, kStatusDrainTimeout);
    }
}

template <int D>
int launch(const DecodePrefixLaunch &a, const PrefixLayout &l, cudaStream_t stream) {
    using C = Cfg<D>;
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
    auto kernel = own_kernel<D>;
    static bool attr_set[kMaxDevices] = {};
    const int dev = slot_for_device();
    if (dev < 0 || !attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return note_cuda_error(e, "cudaFuncSetAttribute(own_kernel)");
        if (dev >= 0) attr_set[dev] = true;
    }
    kernel<<<dim3(unsigned(l.own_ctas)), dim3(kOwnThreads), C::kSmemBytes, stream>>>(mk, mv, mk16, mv16, p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "own_kernel launch");
}

}  // namespace own

int own_launch(const DecodePrefixLaunch &a, const PrefixLayout &l, cudaStream_t stream) {
    return a.d == 64 ? own::launch<64>(a, l, stream) : own::launch<128>(a, l, stream);
}

cudaError_t own_take_status(int *bits) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_own_status, sizeof(int));
    if (e != cudaSuccess) return e;
    return cudaMemcpyToSymbol(g_own_status, &zero, sizeof(int));
}

}  // namespace attn
