// tree_sm103.cu -- trees of drafted tokens: which nodes each node sees, and the
// accepted path's keys and values moved to the front of the drafted rows.
//
// A node sees itself and what its parent sees: anc(t) = {t} + anc(parent(t)); its
// depth is |anc(t)| - 1.  With s steps upwards known for every node, 2 s are one
// look-up away: a(t) |= a(up(t)), up(t) = up(up(t)), log2 T rounds whatever the
// tree's depth.  A block per sequence; latency.
//
// Acceptance: the set bits of the accepted node's mask are its path, in the rows'
// order, and the i-th of them goes to row len + i.  Since the i-th set bit is at
// least i, rows move towards the front only: taken in order, no row is overwritten
// before it has been read, so the move needs no second buffer.  A thread owns 16
// bytes of a head's rows and takes the path in batches, all loads of a batch before
// its stores.  4 d bytes read and written a row and head: launch- or latency-bound
// (few rows 4.3 us, 64 users with 8 layers 10.2, of which HBM needs 7.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "attn_internal.h"

namespace attn {
namespace tree {

constexpr int kMaxNodes = 256, kWords = kMaxNodes / 64;
constexpr int kThreads = 256;
constexpr int kBatch = 8;  // rows whose loads are in flight together

struct MaskParams {
    const int *parents, *seqlens, *draft_lens;
    unsigned long long *mask;
    int *positions;
    int T;
};

__global__ void __launch_bounds__(kMaxNodes) mask_kernel(const MaskParams p) {
    __shared__ unsigned long long seen[kMaxNodes][kWords];
    __shared__ int ups[kMaxNodes];
    const int b = blockIdx.x, t = threadIdx.x, words = (p.T + 63) / 64;
    const int live = p.draft_lens ? min(max(p.draft_lens[b], 0), p.T) : p.T;
    int up = t < live ? p.parents[(size_t)b * p.T + t] : -1;
    if (up >= t) up = -1;  // not before the node: a root
    if (up < 0) up = -1;
    unsigned long long mine[kWords];
#pragma unroll
    for (int w = 0; w < kWords; ++w) seen[t][w] = mine[w] = t < live && t / 64 == w ? 1ull << (t & 63) : 0;
    ups[t] = up;
    for (int step = 1; step < live; step *= 2) {
        __syncthreads();
        int next = -1;
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) mine[w] |= seen[up][w];
            next = ups[up];
        }
        __syncthreads();
        up = next;
#pragma unroll
        for (int w = 0; w < kWords; ++w) seen[t][w] = mine[w];
        ups[t] = up;
    }
    if (t >= p.T) return;
    int depth = -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        depth += __popcll(mine[w]);
        if (w < words) p.mask[((size_t)b * p.T + t) * words + w] = mine[w];
    }
    if (p.positions) p.positions[(size_t)b * p.T + t] = int(unsigned(p.seqlens ? p.seqlens[b] : 0) + unsigned(max(depth, 0)));
}

struct AcceptParams {
    uint4 *k, *v;
    const int *table, *seqlens, *last;
    const unsigned long long *mask;
    int *lens_out;
    int B, T, layers, Hkv, row_units, num_pages, page_size, shift, max_pages, chunks;
};

__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptParams p) {
    // Where a path row comes from and goes to, in units from the first of a plane's head 0; from = -1: it stays.
    __shared__ long long from[kMaxNodes], to[kMaxNodes];
    const int b = blockIdx.x / p.chunks, chunk = blockIdx.x - b * p.chunks;
    const int cap = p.max_pages * p.page_size, words = (p.T + 63) / 64;
    const int len = min(max(p.seqlens[b], 0), cap), last = p.last[b];
    const bool any = last >= 0 && last < p.T;
    const unsigned long long *row = p.mask ? p.mask + ((size_t)b * p.T + max(min(last, p.T - 1), 0)) * words : nullptr;
    const long long head_units = (long long)p.page_size * p.row_units;
    int n = 0;
    if (any && !p.mask) {
        n = last + 1;  // a chain: every row is in its place
    } else if (any) {
        const int t = threadIdx.x;
        int rank = 0;
        bool on = false;
        for (int w = 0; w < words; ++w) {
            unsigned long long bits = row[w];
            if (w == words - 1 && (p.T & 63)) bits &= (1ull << (p.T & 63)) - 1;  // nothing past the last node
            n += __popcll(bits);
            if (w < t / 64) rank += __popcll(bits);
            if (w == t / 64) {
                rank += __popcll(bits & ((1ull << (t & 63)) - 1));
                on = bits >> (t & 63) & 1;
            }
        }
        if (on) {
            auto place = [&](int r) -> long long {
                if (r >= cap || r < 0) return -1;
                const int page = p.table ? p.table[(size_t)b * p.max_pages + (r >> p.shift)] : b;
                if (page < 0 || page >= p.num_pages) return -1;
                return (long long)page * p.Hkv * head_units + (long long)(p.table ? r & (p.page_size - 1) : r) * p.row_units;
            };
            const long long dst = place(len + rank);
            from[rank] = rank == t || dst < 0 ? -1 : place(len + t);
            to[rank] = dst;
        }
    }
    if (chunk == 0 && threadIdx.x == 0 && p.lens_out) p.lens_out[b] = n < cap - len ? len + n : cap;
    __syncthreads();
    if (!p.mask || n == 0) return;
    const int owners = p.layers * 2 * p.Hkv * p.row_units;
    for (int i = chunk * kThreads + threadIdx.x; i < owners; i += p.chunks * kThreads) {
        const int unit = i % p.row_units, plane = i / p.row_units;
        const int h = plane % p.Hkv, kv = plane / p.Hkv & 1, layer = plane / p.Hkv / 2;
        uint4 *base = (kv ? p.v : p.k) + (size_t)layer * p.num_pages * p.Hkv * head_units + h * head_units + unit;
        for (int r = 0; r < n; r += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (r + j < n && from[r + j] >= 0) x[j] = base[from[r + j]];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (r + j < n && from[r + j] >= 0) base[to[r + j]] = x[j];
        }
    }
}

}  // namespace tree

int tree_mask_launch(const TreeLaunch &a, cudaStream_t stream) {
    tree::MaskParams p = {a.parents, a.seqlens, a.draft_lens, a.mask_out, a.positions, a.T};
    tree::mask_kernel<<<a.B, (a.T + 31) / 32 * 32, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "mask_kernel launch");
}

int tree_accept_launch(const TreeLaunch &a, cudaStream_t stream) {
    tree::AcceptParams p = {};
    p.k = static_cast<uint4 *>(a.kpages);
    p.v = static_cast<uint4 *>(a.vpages);
    p.table = a.table;
    p.seqlens = a.seqlens;
    p.last = a.last;
    p.mask = a.mask;
    p.lens_out = a.lens_out;
    p.B = a.B;
    p.T = a.T;
    p.layers = a.layers;
    p.Hkv = a.Hkv;
    p.row_units = a.d / 8;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.shift = a.page_shift;
    p.max_pages = a.max_pages;
    const long long owners = (long long)a.layers * 2 * a.Hkv * p.row_units, most = 0x7fffffffLL / a.B;
    long long chunks = a.mask ? (owners + tree::kThreads - 1) / tree::kThreads : 1;
    p.chunks = int(chunks < most ? chunks : most);
    tree::accept_kernel<<<unsigned(p.chunks * (long long)a.B), tree::kThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "accept_kernel launch");
}

}  // namespace attn
