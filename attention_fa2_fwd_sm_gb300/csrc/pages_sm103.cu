// pages_sm103.cu -- the pages of a cache: taken, copied on write, shared by
// forked sequences, freed, and moved together.
//
// A pool holds `num_pages` pages of K and of V in every layer; one table and one
// array of reference counts serve all layers.  The rules (attn.h has them in full)
// are sums over the tables, so that the results do not depend on any order:
//     refs[p] = number of table entries that hold p; p is free where it is 0;
//     the i-th page that is needed (by sequence, then slot) is the i-th free one;
//     compaction: n pages in use; the i-th free page below n takes the i-th used
//     page from n on.
//
// What bounds them: the tables and counts are small (4 bytes a page and an entry),
// so the plans are latency, a handful of dependent passes by one CTA; the copies
// are HBM-bound, 4 d bytes a row and head read and as many written.  A warp copies
// 4 KB at a time with all of its loads in flight.  Compaction of 1 GB in 2 layers:
// 328 us, 6.6 TB/s read and written (a grid of 8 CTAs an SM, of which 4 fit at once).
// A step of 64 beams (fork, then room for one token with copies on write) takes 17.0 us
// in three launches: the fork 2.2, the rest the plan, up to four passes over lengths,
// entries and counts by one CTA, and the copies.  Room for one token where no page is
// shared 10.7 (the copies' launch finds nothing to do); a trim 1.8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "decode_tile.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace pages {

constexpr int kThreads = 256;      // copies and tables
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kLanes = 8;          // of the plan, for one sequence
constexpr int kRound = 16;         // pages a thread looks at together
constexpr int kUnits = 256;        // 16-byte units that a warp copies together (8 a lane)

struct Params {
    int *table, *table_out, *refs;
    const int *seqlens, *new_lens, *parent;
    int *lens_out, *info;
    uint4 *k, *v;
    int B, T, num_pages, page_size, shift, max_pages, layers, Hkv, row_units;
    // workspace: [num_pages] each, [B] each
    int *writers, *latest, *list, *shared, *needs;
    int4 *copies;
};

__device__ __forceinline__ int clamp_len(const Params &p, int n) { return min(max(n, 0), p.max_pages << p.shift); }
__device__ __forceinline__ bool is_page(const Params &p, int e) { return e >= 0 && e < p.num_pages; }
__device__ __forceinline__ int pages_of(const Params &p, int len) { return (len + p.page_size - 1) >> p.shift; }

// The pages of [0, num_pages) that `want` says, counted over the block in order:
// calls got(i, page) for the i-th of them while i < limit; returns how many there
// are up to where it stopped (at least `limit` of them, or all).
template <typename Want, typename Got>
__device__ __forceinline__ int ranked(const Params &p, int first, int end, int limit, int (*counts)[kPlanWarps], Want want,
                                      Got got) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int found = 0;
    for (int at = first; at < end && found < limit; at += kRound * kPlanThreads) {
        uint32_t votes[kRound];
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const int page = at + k * kPlanThreads + int(threadIdx.x);
            votes[k] = __ballot_sync(0xffffffffu, page < end && want(page));
            if (lane == 0) counts[k][warp] = __popc(votes[k]);
        }
        __syncthreads();
        if (warp == 0) {  // running totals of the 16 x 32 counts, 16 a lane
            int mine[kRound], sum = 0;
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
                const int flat = lane * kRound + i;
                mine[i] = sum;
                sum += counts[flat / kPlanWarps][flat % kPlanWarps];
            }
            int upto = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += y;
            }
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
                const int flat = lane * kRound + i;
                counts[flat / kPlanWarps][flat % kPlanWarps] = mine[i] + upto - sum;
            }
            if (lane == 31) counts[kRound][0] = upto;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kRound; ++k)
            if (votes[k] >> lane & 1) {
                const int i = found + counts[k][warp] + __popc(votes[k] & ((1u << lane) - 1));
                if (i < limit) got(i, at + k * kPlanThreads + int(threadIdx.x));
            }
        found += counts[kRound][0];
        __syncthreads();
    }
    return found;
}

// Slots of sequence b that the next rows go to: [lo, hi), the first `live` rows of
// slot lo being in use.
struct Reach {
    int lo, hi, live;
};
__device__ __forceinline__ Reach reach_of(const Params &p, int b) {
    const int len = clamp_len(p, p.seqlens[b]), cap = p.max_pages << p.shift;
    const int want = p.new_lens ? max(p.new_lens[b], 0) : p.T;
    const int end = want < cap - len ? len + want : cap;
    Reach r;
    r.lo = len >> p.shift;
    r.hi = end > len ? pages_of(p, end) : r.lo;
    r.live = len & (p.page_size - 1);
    return r;
}

// One CTA.  A slot of the reach needs a page where its entry is none, or is a page
// that other entries hold too -- unless all that hold it are about to be written to
// (then the last of them, by sequence and slot, keeps it).
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const Params p) {
    __shared__ int counts[kRound + 1][kPlanWarps];
    __shared__ int warp_sums[kPlanWarps], num_shared;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
    constexpr int kTeams = kPlanThreads / kLanes;
    griddep_launch_dependents();
    auto entry = [&](int b, int slot) { return p.table + (size_t)b * p.max_pages + slot; };
    if (threadIdx.x == 0) num_shared = 0;
    // Shared pages in the reach: their writers are counted.
    bool any = false;
    for (int b = team; b < p.B; b += kTeams) {
        const Reach r = reach_of(p, b);
        for (int s = r.lo + sub; s < r.hi; s += kLanes) {
            const int e = *entry(b, s);
            if (is_page(p, e) && p.refs[e] > 1) {
                any = true;
                p.writers[e] = 0;
                p.latest[e] = -1;
            }
        }
    }
    any = __syncthreads_or(any);
    if (any) {
        for (int b = team; b < p.B; b += kTeams) {
            const Reach r = reach_of(p, b);
            for (int s = r.lo + sub; s < r.hi; s += kLanes) {
                const int e = *entry(b, s);
                if (is_page(p, e) && p.refs[e] > 1) {
                    atomicAdd(p.writers + e, 1);
                    atomicMax(p.latest + e, b * p.max_pages + s);
                }
            }
        }
        __syncthreads();
    }
    auto needs = [&](int b, int slot, int e) {
        if (!is_page(p, e)) return true;
        const int refs = __ldcg(p.refs + e);
        return refs > 1 && !(__ldcg(p.writers + e) == refs && __ldcg(p.latest + e) == b * p.max_pages + slot);
    };
    // Pages needed by each sequence, then by all before it.
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTeams) {
        const int b = b0 + team;
        int n = 0;
        if (b < p.B) {
            const Reach r = reach_of(p, b);
            for (int s = r.lo + sub; s < r.hi; s += kLanes) {
                const int e = *entry(b, s);
                n += needs(b, s, e) ? 1 : 0;
                if (is_page(p, e) && p.refs[e] > 1 && __ldcg(p.latest + e) == b * p.max_pages + s) {
                    // One of its writers puts it down (in any order: only its own count is changed by it).
                    const int i = atomicAdd(&num_shared, 1);
                    if (i < p.num_pages) p.shared[i] = e;
                }
            }
        }
        int upto = n;  // over the lanes, hence over the sequences in order
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        if (lane == 31) warp_sums[warp] = upto;
        __syncthreads();
        int base = before, sum = 0;
        for (int w = 0; w < kPlanWarps; ++w) {
            if (w < warp) base += warp_sums[w];
            sum += warp_sums[w];
        }
        if (b < p.B && sub == 0) p.needs[b] = base + upto - n;
        before += sum;
        __syncthreads();
    }
    const int total = before;
    const int found = total == 0 ? 0
                                 : ranked(p, 0, p.num_pages, total, counts, [&](int page) { return p.refs[page] == 0; },
                                          [&](int i, int page) { p.list[i] = page; });
    const bool enough = found >= total;
    if (threadIdx.x == 0) {
        p.info[0] = enough ? total : 0;
        p.info[1] = enough ? 0 : total - found;
    }
    __syncthreads();
    for (int b = team; b < p.B; b += kTeams) {
        const Reach r = reach_of(p, b);
        const uint32_t mates = ((1u << kLanes) - 1) << (lane / kLanes * kLanes);
        int next = enough ? p.needs[b] : 0;
        if (sub == 0) p.copies[b] = make_int4(-1, -1, 0, 0);
        __syncwarp(mates);
        for (int s0 = r.lo; enough && s0 < r.hi; s0 += kLanes) {
            const int s = s0 + sub;
            int *at = entry(b, s);
            const int e = s < r.hi ? *at : 0;
            const bool need = s < r.hi && needs(b, s, e);
            const uint32_t vote = __ballot_sync(mates, need) & mates;
            if (need) {
                const int page = p.list[next + __popc(vote & ((1u << lane) - 1))];
                *at = page;
                if (is_page(p, e) && s == r.lo && r.live > 0) p.copies[b] = make_int4(e, page, r.live, 0);
            }
            next += __popc(vote);
        }
    }
    // The counts change only now: every need above was judged by the old ones.
    __syncthreads();
    if (!enough) return;
    for (int i = threadIdx.x; i < min(num_shared, p.num_pages); i += kPlanThreads) {
        const int e = p.shared[i], refs = p.refs[e], left = refs - __ldcg(p.writers + e);
        p.refs[e] = left > 0 ? left : 1;
    }
    for (int i = threadIdx.x; i < total; i += kPlanThreads) p.refs[p.list[i]] = 1;
}

// Units [0, n) from `from` to `to` by a warp, at most kUnits.
__device__ __forceinline__ void copy_units(const uint4 *from, uint4 *to, int n) {
    const int lane = threadIdx.x & 31;
    uint4 x[kUnits / 32];
#pragma unroll
    for (int i = 0; i < kUnits / 32; ++i)
        if (i * 32 + lane < n) x[i] = __ldcs(from + i * 32 + lane);
#pragma unroll
    for (int i = 0; i < kUnits / 32; ++i)
        if (i * 32 + lane < n) to[i * 32 + lane] = x[i];
}

// Block (b, y): the planes (layer, K or V, head) of sequence b's copy, if it has one.
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const Params p) {
    griddep_wait();
    const int4 c = p.copies[blockIdx.x];
    if (c.x < 0) return;
    const int units = c.z * p.row_units, per = (units + kUnits - 1) / kUnits, planes = p.layers * 2 * p.Hkv;
    const size_t plane_units = (size_t)p.page_size * p.row_units;
    for (int i = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); i < planes * per; i += gridDim.y * (kThreads / 32)) {
        const int plane = i / per, u = (i - plane * per) * kUnits;
        const int h = plane % p.Hkv, kv = plane / p.Hkv & 1, layer = plane / p.Hkv / 2;
        uint4 *base = (kv ? p.v : p.k) + (size_t)layer * p.num_pages * p.Hkv * plane_units + u;
        copy_units(base + ((size_t)c.x * p.Hkv + h) * plane_units, base + ((size_t)c.y * p.Hkv + h) * plane_units,
                   min(kUnits, units - u));
    }
}

// A thread an entry of the new table.
__global__ void __launch_bounds__(kThreads) fork_kernel(const Params p) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b = int(i / p.max_pages), s = int(i - (long long)b * p.max_pages);
    if (b >= p.B) return;
    const int from = p.parent[b];
    const bool has = from >= 0 && from < p.B;
    const int len = has ? clamp_len(p, p.seqlens[from]) : 0;
    if (s == 0) p.lens_out[b] = len;
    const int old = p.table[i];
    if (from == b) {
        p.table_out[i] = old;
        return;
    }
    const int e = has && s < pages_of(p, len) ? p.table[(size_t)from * p.max_pages + s] : -1;
    if (is_page(p, old)) atomicSub(p.refs + old, 1);
    if (is_page(p, e)) atomicAdd(p.refs + e, 1);
    p.table_out[i] = is_page(p, e) ? e : -1;
}

__global__ void __launch_bounds__(kThreads) trim_kernel(const Params p) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b = int(i / p.max_pages), s = int(i - (long long)b * p.max_pages);
    if (b >= p.B) return;
    const int keep = clamp_len(p, p.new_lens[b]);
    if (s == 0 && p.lens_out) p.lens_out[b] = min(clamp_len(p, p.seqlens[b]), keep);
    if (s < pages_of(p, keep)) return;
    const int old = p.table[i];
    if (is_page(p, old)) atomicSub(p.refs + old, 1);
    p.table[i] = -1;
}

// One CTA: n pages in use; holes below n (into `list`) and pages in use from n on
// (into `writers`), paired in order; latest[page] is where a page goes.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const Params p) {
    __shared__ int counts[kRound + 1][kPlanWarps];
    griddep_launch_dependents();
    auto used = [&](int page) { return p.refs[page] > 0; };
    const int n = ranked(p, 0, p.num_pages, 0x7fffffff, counts, used, [](int, int) {});
    const int moves = ranked(p, 0, n, 0x7fffffff, counts, [&](int page) { return !used(page); },
                             [&](int i, int page) { p.list[i] = page; });
    __syncthreads();
    ranked(p, n, p.num_pages, moves, counts, used, [&](int i, int page) {
        p.writers[i] = page;
        p.latest[page] = p.list[i];
    });
    if (threadIdx.x == 0) {
        p.info[0] = n;
        p.info[1] = moves;
        p.needs[0] = n;  // (info is the caller's to change)
        p.needs[1] = moves;
    }
    for (int page = n + threadIdx.x; page < p.num_pages; page += kPlanThreads)
        if (!used(page)) p.latest[page] = page;  // (no entry should hold it)
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += kPlanThreads) {
        const int from = p.writers[i];
        p.refs[p.list[i]] = p.refs[from];
        p.refs[from] = 0;
    }
}

// All CTAs: the moved pages of every layer, 4 KB a warp at a time, their counts, and
// the tables' entries.
__global__ void __launch_bounds__(kThreads) compact_kernel(const Params p) {
    griddep_wait();
    const int n = p.needs[0], moves = p.needs[1];
    const long long thread = (long long)blockIdx.x * kThreads + threadIdx.x, threads = (long long)gridDim.x * kThreads;
    for (long long i = thread; i < (long long)p.B * p.max_pages; i += threads) {
        const int e = p.table[i];
        if (is_page(p, e) && e >= n) p.table[i] = p.latest[e];
    }
    const int units = p.Hkv * p.page_size * p.row_units, per = (units + kUnits - 1) / kUnits;
    const long long all = (long long)moves * p.layers * 2 * per, warps = threads / 32;
    for (long long i = thread / 32; i < all; i += warps) {
        const int u = int(i % per) * kUnits;
        const long long r = i / per;
        const int kv = int(r & 1), layer = int((r >> 1) % p.layers), m = int((r >> 1) / p.layers);
        uint4 *base = (kv ? p.v : p.k) + (size_t)layer * p.num_pages * units + u;
        copy_units(base + (size_t)p.writers[m] * units, base + (size_t)p.list[m] * units, min(kUnits, units - u));
    }
}

size_t layout(int B, int num_pages, char *base, Params *p) {
    const size_t rows = B > 2 ? B : 2;
    size_t at = 0;
    auto take = [&](size_t n) {
        char *here = base + at;
        at += (n + 15) / 16 * 16;
        return here;
    };
    char *parts[6];
    for (int i = 0; i < 4; ++i) parts[i] = take(size_t(num_pages) * 4);
    parts[4] = take(rows * 4);
    parts[5] = take(rows * sizeof(int4));
    if (p) {
        p->writers = reinterpret_cast<int *>(parts[0]);
        p->latest = reinterpret_cast<int *>(parts[1]);
        p->list = reinterpret_cast<int *>(parts[2]);
        p->shared = reinterpret_cast<int *>(parts[3]);
        p->needs = reinterpret_cast<int *>(parts[4]);
        p->copies = reinterpret_cast<int4 *>(parts[5]);
    }
    return at;
}

Params params_of(const PagesLaunch &a) {
    Params p = {};
    p.table = a.table;
    p.table_out = a.table_out;
    p.refs = a.refs;
    p.seqlens = a.seqlens;
    p.new_lens = a.new_lens;
    p.parent = a.parent;
    p.lens_out = a.lens_out;
    p.info = a.info;
    p.k = static_cast<uint4 *>(a.kpages);
    p.v = static_cast<uint4 *>(a.vpages);
    p.B = a.B;
    p.T = a.T;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.max_pages = a.max_pages;
    p.layers = a.layers;
    p.Hkv = a.Hkv;
    p.row_units = a.d / 8;
    if (a.workspace) layout(a.B, a.num_pages, a.workspace, &p);
    return p;
}

int table_blocks(const PagesLaunch &a) { return int(((long long)a.B * a.max_pages + kThreads - 1) / kThreads); }

}  // namespace pages

size_t pages_workspace_bytes(int B, int num_pages) { return pages::layout(B, num_pages, nullptr, nullptr); }

int pages_extend_launch(const PagesLaunch &a, cudaStream_t stream) {
    using namespace pages;
    const Params p = params_of(a);
    extend_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return note_cuda_error(e, "extend_kernel launch");
    // A block of eight warps copies 32 KB at a time.
    const long long warps = (long long)a.layers * 2 * a.Hkv * (((long long)a.page_size * p.row_units + kUnits - 1) / kUnits);
    const long long want = (warps + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid(unsigned(a.B), unsigned(want < 64 ? want : 64));
    e = dec::launch_programmatic(copy_rows_kernel, grid, dim3(kThreads), 0, stream, p);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "copy_rows_kernel launch");
}

int pages_fork_launch(const PagesLaunch &a, cudaStream_t stream) {
    pages::fork_kernel<<<pages::table_blocks(a), pages::kThreads, 0, stream>>>(pages::params_of(a));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "fork_kernel launch");
}

int pages_trim_launch(const PagesLaunch &a, cudaStream_t stream) {
    pages::trim_kernel<<<pages::table_blocks(a), pages::kThreads, 0, stream>>>(pages::params_of(a));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "trim_kernel launch");
}

int pages_compact_launch(const PagesLaunch &a, cudaStream_t stream) {
    using namespace pages;
    const Params p = params_of(a);
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return note_cuda_error(e, "compact_plan_kernel launch");
    e = dec::launch_programmatic(compact_kernel, dim3(unsigned(8 * a.num_sms)), dim3(kThreads), 0, stream, p);
    return e == cudaSuccess ? 0 : note_cuda_error(e, "compact_kernel launch");
}

}  // namespace attn
