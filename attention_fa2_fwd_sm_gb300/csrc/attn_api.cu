// attn_api.cu -- the extern "C" boundary of libattn.so: argument validation
// (entirely on the host, before any CUDA call), dispatch to the kernels,
// device status reporting and the host-side view of the scheduler.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "dkdv_order.cuh"
#include "prefix_order.cuh"
#include "tile_order.cuh"

namespace attn {

namespace {

std::atomic<long long> g_wait_ns{10LL * 1000 * 1000 * 1000};  // 10 s

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

int current_num_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    static int cached[kMaxDevices] = {0};
    if (dev >= 0 && dev < kMaxDevices && cached[dev] > 0) return cached[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return -1;
    if (dev >= 0 && dev < kMaxDevices) cached[dev] = n;
    return n;
}

bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxSplits = kDecodeMaxSplits;
constexpr int kDecodeMaxGroup = 16;

}  // namespace

namespace {
thread_local char g_last_error[256] = "";
}

int note_cuda_error(cudaError_t e, const char *where) {
    snprintf(g_last_error, sizeof(g_last_error), "%s: %s (%d)", where, cudaGetErrorString(e), int(e));
    return ATTN_ERR_CUDA;
}

bool encode_bf16_3d(CUtensorMap *map, const void *base, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                    uint32_t box0, uint32_t box1, uint32_t box2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {dim0, dim1, dim2};
    const cuuint64_t strides[2] = {dim0 * 2, dim0 * dim1 * 2};
    const cuuint32_t box[3] = {box0, box1, box2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int fwd_run(const FwdLaunch &a, cudaStream_t stream) {
    // The library's choice: the one-CTA kernel (every head dimension).
    if (a.scheme == kSchemePair) return fwd_pair_launch(a, stream);
    return fwd_launch(a, stream);
}

}  // namespace attn

using namespace attn;

extern "C" {

int attn_version(void) { return 100; }

const char *attn_last_error(void) { return g_last_error; }

const char *attn_strerror(int code) {
    switch (code) {
        case ATTN_OK: return "ok";
        case ATTN_ERR_ARG: return "invalid argument (null/misaligned pointer, bad size, Hq % Hkv, scale)";
        case ATTN_ERR_UNSUPPORTED: return "unsupported head dimension or group size";
        case ATTN_ERR_WORKSPACE: return "workspace missing or too small";
        case ATTN_ERR_CUDA: return "CUDA runtime or driver call failed";
        case ATTN_ERR_TIMEOUT: return "a bounded device wait ran out";
        default: return "unknown status code";
    }
}

long long attn_set_wait_timeout_ns(long long ns) {
    if (ns < 0) ns = 0;
    return g_wait_ns.exchange(ns);
}

long long attn_fwd_units(int B, int Hq, int N) {
    if (B <= 0 || Hq <= 0 || N <= 0) return 0;
    return (long long)B * Hq * unit_blocks(N);
}

int attn_tile_map(int tile_order, int B, int Hq, int Hkv, int N, int causal, long long unit, int *b, int *h,
                  int *m) {
    if (!b || !h || !m || B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (tile_order < kHeadFirst || tile_order > kNaiveHeadFirst) return ATTN_ERR_ARG;
    const long long total = attn_fwd_units(B, Hq, N);
    if (unit < 0 || unit >= total) return ATTN_ERR_ARG;
    const Tile t = unit_to_tile(tile_order, unit, Hq, Hq / Hkv, unit_blocks(N), causal ? 1 : 0);
    *b = t.b;
    *h = t.h;
    *m = t.m;
    return ATTN_OK;
}

int attn_tile_map_die_split(int B, int Hq, int Hkv, int N, int causal, int die, long long k, int *b,
                            int *h, int *m) {
    if (!b || !h || !m || B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (die < 0 || die >= kDies) return ATTN_ERR_ARG;
    const int nb = unit_blocks(N);
    const long long u = die_split_unit(die, k, B, Hkv, Hq / Hkv, nb);
    if (u < 0) return ATTN_ERR_ARG;
    const Tile t = unit_to_tile(kDieSplitHeadFirst, u, Hq, Hq / Hkv, nb, causal ? 1 : 0);  // head-first ids
    *b = t.b;
    *h = t.h;
    *m = t.m;
    return ATTN_OK;
}

int attn_bwd_tile_map(int tile_order, int B, int Hkv, int N, int causal, int num_sms, long long unit, int *b,
                      int *g, int *j) {
    if (!b || !g || !j || B <= 0 || Hkv <= 0 || N <= 0 || num_sms <= 0) return ATTN_ERR_ARG;
    if (tile_order < kHeadFirst || tile_order > kNaiveHeadFirst) return ATTN_ERR_ARG;
    if ((long long)B * Hkv >= (1LL << 31)) return ATTN_ERR_ARG;
    const int nblk = (N + kKeyBlock - 1) / kKeyBlock;
    if (unit < 0 || unit >= (long long)B * Hkv * nblk) return ATTN_ERR_ARG;
    const KvTile t = dkdv_unit_to_tile(tile_order, unit, B, Hkv, nblk,
                                       dkdv_window(tile_order, causal ? 1 : 0, B, Hkv, nblk, num_sms));
    *b = t.b;
    *g = t.g;
    *j = t.j;
    return ATTN_OK;
}

int attn_die_map(int *die_of_sm, int capacity, float *stats) {
    if (capacity < 0 || (capacity > 0 && !die_of_sm)) return ATTN_ERR_ARG;
    return die_map_query(die_of_sm, capacity, stats);
}

// tile_order of the forward entry points: an order in the low byte, at most
// one tile-scheme flag above it.
static int order_of(int tile_order) { return tile_order & 0xff; }
static int scheme_of(int tile_order) {
    const int f = tile_order & ~0xff;
    if (f == 0) return kSchemeAuto;
    if (f == ATTN_FWD_SINGLE_CTA) return kSchemeSingle;
    if (f == ATTN_FWD_CTA_PAIR) return kSchemePair;
    return -1;
}

static int validate_fwd_sizes(int B, int Hq, int Hkv, int N, int d, float scale, int tile_order) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0) return ATTN_ERR_ARG;
    if (Hq % Hkv) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    const int order = order_of(tile_order), scheme = scheme_of(tile_order);
    if (order < kHeadFirst || order > kDieSplitHeadFirst || scheme < 0) return ATTN_ERR_ARG;
    if (d != 56 && d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (scheme == kSchemePair && d != 128) return ATTN_ERR_UNSUPPORTED;
    // tensor-map limits: each dimension < 2^32, strides < 2^40 bytes
    if ((long long)B * Hq >= (1LL << 31) || (long long)N * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    // The persistent forward and backward kernels take work units (at most
    // B * Hq * ceil(N / 128) of them) from 32-bit counters.
    if ((long long)B * Hq * ((N + 127) / 128) >= (1LL << 31)) return ATTN_ERR_ARG;
    return ATTN_OK;
}

static int validate_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                        int Hq, int Hkv, int N, int d, float scale, int tile_order) {
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_ARG;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_ARG;
    return validate_fwd_sizes(B, Hq, Hkv, N, d, scale, tile_order);
}

static FwdLaunch fwd_problem(int B, int Hq, int Hkv, int N, int d, float scale, int causal, int tile_order,
                             int sms) {
    FwdLaunch a;
    a.q = a.k = a.v = nullptr;
    a.o = nullptr;
    a.lse = nullptr;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.N = N;
    a.d = d;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.order = order_of(tile_order);
    a.scheme = scheme_of(tile_order);
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return a;
}

int attn_fwd_ex(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                int Hkv, int N, int d, float scale, int causal, int tile_order,
                attn_stream_t stream) {
    int rc = validate_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, tile_order);
    if (rc != ATTN_OK) return rc;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    FwdLaunch a = fwd_problem(B, Hq, Hkv, N, d, scale, causal, tile_order, sms);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    return fwd_run(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_fwd_host_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int kv_heads_per_chunk) {
    if (validate_fwd_sizes(B, Hq, Hkv, N, d, 1.f, kHeadFirst) != ATTN_OK) return 0;
    if (kv_heads_per_chunk > Hkv) return 0;
    const int gc = kv_heads_per_chunk > 0 ? kv_heads_per_chunk : host_default_chunk(Hq, Hkv, N);
    return 2 * host_chunk_layout(Hq, Hkv, N, d, gc).slot_bytes;
}

int attn_fwd_host(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                  int N, int d, float scale, int causal, int tile_order, int kv_heads_per_chunk,
                  void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (!q || !k || !v || !o) return ATTN_ERR_ARG;
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_ARG;
    int rc = validate_fwd_sizes(B, Hq, Hkv, N, d, scale, tile_order);
    if (rc != ATTN_OK) return rc;
    if (kv_heads_per_chunk > Hkv) return ATTN_ERR_ARG;
    const int gc = kv_heads_per_chunk > 0 ? kv_heads_per_chunk : host_default_chunk(Hq, Hkv, N);
    const size_t need = 2 * host_chunk_layout(Hq, Hkv, N, d, gc).slot_bytes;
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    FwdHostLaunch a;
    a.fwd = fwd_problem(B, Hq, Hkv, N, d, scale, causal, tile_order, sms);
    a.q_host = q;
    a.k_host = k;
    a.v_host = v;
    a.o_host = o;
    a.lse_host = lse;
    a.kv_heads_per_chunk = gc;
    a.workspace = workspace;
    return fwd_host_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_fwd_host_trace(int enable) { return fwd_host_trace(enable); }

long long attn_fwd_host_trace_read(float *ms, long long capacity) {
    if (capacity < 0 || (capacity > 0 && !ms)) return ATTN_ERR_ARG;
    const long long n = fwd_host_trace_read(ms, capacity);
    return n == -1 ? ATTN_ERR_ARG : n;
}

// Split-KV forward: the key range of each head in `splits` pieces of
// `chunk_keys` keys (a multiple of the 128-key block); kv_splits <= 0 picks
// the fewest pieces whose K and V of one KV head fit in 32 MiB.
constexpr int kMaxKvSplits = 64;
static bool splitkv_plan(int N, int d, int kv_splits, int *splits, int *chunk_keys) {
    if (kv_splits > kMaxKvSplits) return false;
    int s = kv_splits;
    if (s <= 0) {
        const long long budget_keys = (32LL << 20) / (4LL * d);  // K + V bf16 of one head per key: 4 d bytes
        s = int((N + budget_keys - 1) / budget_keys);
        if (s < 1) s = 1;
        if (s > kMaxKvSplits) s = kMaxKvSplits;
    }
    long long chunk = (N + s - 1) / s;
    chunk = (chunk + 127) / 128 * 128;
    *chunk_keys = int(chunk);
    *splits = int((N + chunk - 1) / chunk);
    return true;
}

static void splitkv_layout(int B, int Hq, int N, int d, int splits, size_t *o_bytes, size_t *lse_bytes) {
    const size_t rows = (size_t)B * Hq * N;
    *o_bytes = (rows * splits * d * sizeof(float) + 255) / 256 * 256;
    *lse_bytes = rows * splits * sizeof(float);
}

size_t attn_fwd_splitkv_workspace_bytes(int B, int Hq, int N, int d, int kv_splits) {
    if (B <= 0 || Hq <= 0 || N <= 0 || (d != 56 && d != 64 && d != 128)) return 0;
    int splits = 0, chunk = 0;
    if (!splitkv_plan(N, d, kv_splits, &splits, &chunk)) return 0;
    size_t a = 0, b = 0;
    splitkv_layout(B, Hq, N, d, splits, &a, &b);
    return a + b;
}

int attn_fwd_splitkv(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                     int N, int d, float scale, int causal, int kv_splits, void *workspace, size_t workspace_bytes,
                     attn_stream_t stream) {
    int rc = validate_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, kHeadFirst);
    if (rc != ATTN_OK) return rc;
    int splits = 0, chunk = 0;
    if (!splitkv_plan(N, d, kv_splits, &splits, &chunk)) return ATTN_ERR_ARG;
    if ((long long)B * Hq * unit_blocks(N) * splits >= (1LL << 31)) return ATTN_ERR_ARG;
    size_t o_bytes = 0, lse_bytes = 0;
    splitkv_layout(B, Hq, N, d, splits, &o_bytes, &lse_bytes);
    if (!workspace || !aligned16(workspace) || workspace_bytes < o_bytes + lse_bytes) return ATTN_ERR_WORKSPACE;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    FwdSplitLaunch a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.N = N;
    a.d = d;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.splits = splits;
    a.chunk_keys = chunk;
    a.part_o = static_cast<float *>(workspace);
    a.part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + o_bytes);
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return fwd_split_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
             int Hkv, int N, int d, float scale, int causal, attn_stream_t stream) {
    return attn_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, ATTN_ORDER_HEAD_FIRST,
                       stream);
}

size_t attn_bwd_workspace_bytes(int B, int Hq, int N) {
    if (B <= 0 || Hq <= 0 || N <= 0) return 0;
    return (size_t)B * Hq * (size_t)((N + 127) / 128) * 128 * 2 * sizeof(float);
}

size_t attn_bwd_workspace_bytes_ex(int B, int Hq, int Hkv, int N, int d, int causal) {
    if (validate_fwd_sizes(B, Hq, Hkv, N, d, 1.f, kHeadFirst) != ATTN_OK) return 0;
    const size_t base = attn_bwd_workspace_bytes(B, Hq, N);
    const size_t part = bwd_part_bytes(B, Hkv, N, d, bwd_kv_split(B, Hq, Hkv, N, causal));
    return part ? (base + 255) / 256 * 256 + part : base;
}

int attn_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout, const float *lse,
             void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int N, int d, float scale, int causal,
             int tile_order, void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    int rc = validate_fwd(q, k, v, dq, nullptr, B, Hq, Hkv, N, d, scale, kHeadFirst);
    if (rc != ATTN_OK) return rc;
    if (!aligned16(o) || !aligned16(dout) || !aligned16(dk) || !aligned16(dv)) return ATTN_ERR_ARG;
    if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_ARG;
    if (tile_order < kHeadFirst || tile_order > kNaiveHeadFirst) return ATTN_ERR_ARG;
    const size_t need = (size_t)B * Hq * (size_t)((N + 127) / 128) * 128 * 2 * sizeof(float);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    // The dK/dV pass's query-head split, when the workspace also holds its partials.
    const int kv_split = bwd_kv_split(B, Hq, Hkv, N, causal);
    const size_t part_at = (need + 255) / 256 * 256;
    const size_t part_bytes = bwd_part_bytes(B, Hkv, N, d, kv_split);
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    BwdLaunch a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.dout = dout;
    a.lse = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.N = N;
    a.d = d;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.order = tile_order;
    a.workspace = static_cast<float *>(workspace);
    if (part_bytes > 0 && workspace_bytes >= part_at + part_bytes) {
        a.kv_split = kv_split;
        a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + part_at);
    }
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return bwd_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t attn_decode_workspace_bytes(int B, int Hq, int d, int num_splits) {
    if (B <= 0 || Hq <= 0 || d <= 0 || num_splits <= 1) return 0;
    const size_t parts = (size_t)B * Hq * num_splits;
    size_t o_bytes = parts * d * sizeof(float);
    o_bytes = (o_bytes + 255) / 256 * 256;
    return o_bytes + parts * sizeof(float);
}

// Split count: aim at about 5/3 CTAs per SM in all (the decode kernel keeps
// two CTAs resident per SM, and a grid just over one wave leaves a tail wave
// on a few SMs), never below 512 keys per split, at most kMaxSplits.  Chosen
// from a sweep of split counts over batch {1, 8, 32} x keys {8K, 32K, 128K}
// (H_Q = 64, H_KV = 8, d = 128), where it lands within a few percent of the
// best split count in every configuration.
static int splits_for(int B, int Hkv, int max_seqlen, int sms) {
    const long long ctas = (long long)B * Hkv;
    const long long target = (5LL * sms) / 3;
    long long s = (target + ctas / 2) / ctas;  // round to nearest
    const long long by_len = max_seqlen / 512;
    if (s > by_len) s = by_len;
    if (s > kMaxSplits) s = kMaxSplits;
    if (s < 1) s = 1;
    // Long caches: double the splits while each keeps at least 4096 keys and
    // the grid stays within four CTAs per SM (about 1.7 waves of two resident
    // CTAs per SM); the split sweep measured that 1-3% faster.
    while (2 * s <= kMaxSplits && max_seqlen / (2 * s) >= 4096 && ctas * 2 * s <= 4LL * sms) s *= 2;
    return int(s);
}

int attn_decode_num_splits(int B, int Hq, int Hkv, int max_seqlen) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || max_seqlen < 0 || Hq % Hkv) return ATTN_ERR_ARG;
    const int sms = current_num_sms();
    if (sms <= 0) return ATTN_ERR_CUDA;
    return splits_for(B, Hkv, max_seqlen, sms);
}

// Varlen decode: work-list capacity and the chunk rule (see attn.h).
constexpr int kVarlenMinChunk = 512;
static long long varlen_target(int sms) {
    const long long t = (5LL * sms) / 3;
    return t > 0 ? t : 1;
}
static long long varlen_max_items(int B, int Hkv, int sms) {
    const long long t = varlen_target(sms);
    return (t + Hkv - 1) / Hkv + B;
}
static void varlen_layout(int B, int Hq, int d, long long items, size_t *plan_bytes, size_t *o_bytes,
                          size_t *lse_bytes) {
    *plan_bytes = ((size_t)(2 + 2LL * B + 3 * items) * sizeof(int) + 255) / 256 * 256;
    *o_bytes = ((size_t)items * Hq * d * sizeof(float) + 255) / 256 * 256;
    *lse_bytes = (size_t)items * Hq * sizeof(float);
}

size_t attn_decode_varlen_workspace_bytes(int B, int Hq, int Hkv, int d) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv) return 0;
    const int sms = current_num_sms();
    if (sms <= 0) return 0;
    size_t a, b, c;
    varlen_layout(B, Hq, d, varlen_max_items(B, Hkv, sms), &a, &b, &c);
    return a + b + c;
}

int attn_decode_varlen(const void *q, const void *kcache, const void *vcache, const int *seqlens, void *o,
                       int B, int Hq, int Hkv, int d, float scale, int max_seqlen, void *workspace,
                       size_t workspace_bytes, attn_stream_t stream) {
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) || !seqlens ||
        (reinterpret_cast<uintptr_t>(seqlens) & 3u))
        return ATTN_ERR_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || max_seqlen <= 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > kDecodeMaxGroup) return ATTN_ERR_UNSUPPORTED;
    if (B > (1 << 20) || Hkv > 65535 || (long long)max_seqlen * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    // the plan's T * Hkv stays below 2^62; the merge grid has B * Hq blocks
    if ((double)B * (double)max_seqlen * (double)Hkv >= 4.0e18 || (long long)B * Hq > 0x7fffffffLL)
        return ATTN_ERR_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return ATTN_ERR_WORKSPACE;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    const long long items = varlen_max_items(B, Hkv, sms);
    if (items > 65535) return ATTN_ERR_ARG;  // grid.y limit of the decode launch
    size_t plan_bytes, o_bytes, lse_bytes;
    varlen_layout(B, Hq, d, items, &plan_bytes, &o_bytes, &lse_bytes);
    if (workspace_bytes < plan_bytes + o_bytes + lse_bytes) return ATTN_ERR_WORKSPACE;
    DecodeLaunch a;
    a.q = q;
    a.kcache = kcache;
    a.vcache = vcache;
    a.seqlens = seqlens;
    a.o = o;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.max_seqlen = max_seqlen;
    a.num_splits = 0;
    a.scale = scale;
    char *ws = static_cast<char *>(workspace);
    a.plan = reinterpret_cast<int *>(ws);
    a.ws_o = reinterpret_cast<float *>(ws + plan_bytes);
    a.ws_lse = reinterpret_cast<float *>(ws + plan_bytes + o_bytes);
    a.varlen_max_items = int(items);
    a.varlen_target = varlen_target(sms);
    a.varlen_min_chunk = kVarlenMinChunk;
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return decode_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_decode(const void *q, const void *kcache, const void *vcache, const int *seqlens, void *o,
                int B, int Hq, int Hkv, int d, float scale, int num_splits, int max_seqlen,
                void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) || !seqlens ||
        (reinterpret_cast<uintptr_t>(seqlens) & 3u))
        return ATTN_ERR_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || max_seqlen <= 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    if (num_splits > kMaxSplits) return ATTN_ERR_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > kDecodeMaxGroup) return ATTN_ERR_UNSUPPORTED;
    if (B > 65535 || Hkv > 65535 || (long long)max_seqlen * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    if (num_splits <= 0) {
        const int sms = current_num_sms();
        if (sms <= 0) return ATTN_ERR_CUDA;
        num_splits = splits_for(B, Hkv, max_seqlen, sms);
    }
    const size_t need = attn_decode_workspace_bytes(B, Hq, d, num_splits);
    if (need > 0 && (!workspace || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 15u)))
        return ATTN_ERR_WORKSPACE;
    DecodeLaunch a;
    a.q = q;
    a.kcache = kcache;
    a.vcache = vcache;
    a.seqlens = seqlens;
    a.o = o;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.max_seqlen = max_seqlen;
    a.num_splits = num_splits;
    a.scale = scale;
    const size_t parts = (size_t)B * Hq * num_splits;
    size_t o_bytes = (parts * d * sizeof(float) + 255) / 256 * 256;
    a.ws_o = need ? reinterpret_cast<float *>(workspace) : nullptr;
    a.ws_lse = need ? reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + o_bytes) : nullptr;
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = current_num_sms();  // 0 if unknown: the base ring
    return decode_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

static_assert(ATTN_DECODE_NOALLOC_SCRATCH_BYTES == attn::kDecodeNoAllocScratchBytes,
              "header and library disagree on the built-in scratch size");

int attn_decode_noalloc(const void *q, const void *kcache, const void *vcache, const int *seqlens,
                        void *o, int B, int Hq, int Hkv, int d, float scale, int num_splits,
                        int max_seqlen, attn_stream_t stream) {
    // The argument checks of attn_decode, made here first so that a bad call
    // is refused before the one-time scratch set-up touches CUDA.
    if (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(o) || !seqlens ||
        (reinterpret_cast<uintptr_t>(seqlens) & 3u))
        return ATTN_ERR_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || max_seqlen <= 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    if (num_splits > kMaxSplits) return ATTN_ERR_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > kDecodeMaxGroup) return ATTN_ERR_UNSUPPORTED;
    if (B > 65535 || Hkv > 65535 || (long long)max_seqlen * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    const size_t cap = kDecodeNoAllocScratchBytes;
    if (num_splits <= 0) {
        const int sms = current_num_sms();
        if (sms <= 0) return ATTN_ERR_CUDA;
        num_splits = splits_for(B, Hkv, max_seqlen, sms);
        while (num_splits > 1 && attn_decode_workspace_bytes(B, Hq, d, num_splits) > cap) --num_splits;
    } else if (attn_decode_workspace_bytes(B, Hq, d, num_splits) > cap) {
        return ATTN_ERR_WORKSPACE;
    }
    void *scratch = nullptr;
    const cudaError_t se = decode_noalloc_scratch(&scratch);
    if (se != cudaSuccess || !scratch) return note_cuda_error(se, "cudaGetSymbolAddress(scratch)");
    return attn_decode(q, kcache, vcache, seqlens, o, B, Hq, Hkv, d, scale, num_splits, max_seqlen,
                       scratch, cap, stream);
}

// Rotary positions.  The two tables of strides hold (batch, head, token) per
// tensor; a stride of a dimension of extent 1 is never used and set to 0.
static bool rope_strides(const long long *s, bool output, int B, int H, int N, int d, long long *out) {
    const long long extent[3] = {B, H, N};
    const long long packed[3] = {(long long)H * N * d, (long long)N * d, d};
    for (int i = 0; i < 3; ++i) {
        long long v = s ? s[i] : packed[i];
        if (extent[i] == 1) v = 0;
        else if (v % 8 || v < (output ? d : 0) || v >= (1LL << 40)) return false;
        out[i] = v;
    }
    return true;
}

static int rope_tensor(RopeTensor *t, const void *in, void *out, const long long *in_s, const long long *out_s, int B,
                       int H, int N, int d) {
    long long a[3], b[3];
    if (!aligned16(in) || !aligned16(out)) return ATTN_ERR_ARG;
    if (!rope_strides(in_s, false, B, H, N, d, a) || !rope_strides(out_s, true, B, H, N, d, b)) return ATTN_ERR_ARG;
    if (in == out && (a[0] != b[0] || a[1] != b[1] || a[2] != b[2])) return ATTN_ERR_ARG;
    t->in = static_cast<const __nv_bfloat16 *>(in);
    t->out = static_cast<__nv_bfloat16 *>(out);
    t->in_b = a[0], t->in_h = a[1], t->in_n = a[2];
    t->out_b = b[0], t->out_h = b[1], t->out_n = b[2];
    t->heads = H;
    return ATTN_OK;
}

// A bf16 tensor [B, heads, N, d] by its strides, in units of 8 elements (16
// bytes), which base, strides and rows are multiples of; heads = 0: absent.
struct Rows {
    const void *p = nullptr;
    long long s[3] = {}, n[3] = {};
    long long d = 0;
    __int128 span = 0;  // from the first row to the last
    Rows(const void *base, const long long (&strides)[3], int B, int H, int N, int cols) : p(H > 0 ? base : nullptr), d(cols / 8) {
        const int extent[3] = {B, H, N};
        for (int i = 0; i < 3; ++i) {
            s[i] = strides[i] / 8, n[i] = extent[i];
            span += (__int128)s[i] * (n[i] - 1);
        }
    }
    bool same(const Rows &o) const {
        if (p != o.p || d != o.d) return false;
        for (int i = 0; i < 3; ++i)
            if (n[i] != o.n[i] || (n[i] > 1 && s[i] != o.s[i])) return false;
        return true;
    }
};

// One dimension of the distance between an element of one tensor and an
// element of another: it adds s * y, lo <= y <= hi.
struct Reach {
    __int128 s, lo, hi;
};

// Whether the distances at + sum s_i y_i meet (-width, width); the dimensions
// by falling stride, so that after each only the few y_i are left that the
// smaller ones can make up for.  `budget` bounds the search: strides that do
// not nest can leave many, and such tensors pass for apart.
static bool meets(const Reach *dim, int n, __int128 at, __int128 width, int *budget) {
    if (--*budget < 0) return false;
    if (n == 0) return at > -width && at < width;
    __int128 lo = 0, hi = 0;  // what the smaller strides can add
    for (int i = 1; i < n; ++i) lo += dim[i].s * dim[i].lo, hi += dim[i].s * dim[i].hi;
    // -width < at + s y + [lo, hi] < width
    const __int128 s = dim[0].s;
    auto floor_div = [&](__int128 x) { return x >= 0 ? x / s : -((-x + s - 1) / s); };
    __int128 first = floor_div(-width - at - hi) + 1, last = -floor_div(-(width - at - lo)) - 1;
    if (first < dim[0].lo) first = dim[0].lo;
    if (last > dim[0].hi) last = dim[0].hi;
    for (__int128 y = first; y <= last && *budget >= 0; ++y)
        if (meets(dim + 1, n - 1, at + s * y, width, budget)) return true;
    return false;
}

// Whether the two share an element.  Views of one fused projection interleave
// without sharing any, so their address ranges do not tell.
static bool share_elements(const Rows &a, const Rows &b) {
    if (!a.p || !b.p) return false;
    // Rows of the same width meet where they start less than it apart.
    const __int128 apart = ((__int128)reinterpret_cast<uintptr_t>(a.p) - (__int128)reinterpret_cast<uintptr_t>(b.p)) / 16;
    if (apart + a.span <= -a.d || apart - b.span >= a.d) return false;
    Reach dim[6];
    int n = 0;
    auto add = [&](long long s, long long lo, long long hi) {
        if (s == 0 || lo == hi) return;
        for (int i = 0; i < n; ++i)
            if (dim[i].s == s) {
                dim[i].lo += lo, dim[i].hi += hi;
                return;
            }
        int i = n++;
        for (; i > 0 && dim[i - 1].s < s; --i) dim[i] = dim[i - 1];
        dim[i] = {s, lo, hi};
    };
    for (int i = 0; i < 3; ++i) {
        add(a.s[i], 0, a.n[i] - 1);
        add(b.s[i], 1 - b.n[i], 0);
    }
    int budget = 2000;
    return meets(dim, n, apart, a.d, &budget);
}

// Whether two rows of one tensor share an element (a stride that is smaller than
// what the smaller strides span).
static bool shares_with_itself(const Rows &a) {
    if (!a.p) return false;
    Reach dim[3];
    int n = 0;
    for (int k = 0; k < 3; ++k) {
        if (a.n[k] < 2) continue;
        if (a.s[k] < a.d) return true;
        int i = n++;
        for (; i > 0 && dim[i - 1].s < a.s[k]; --i) dim[i] = dim[i - 1];
        dim[i] = {a.s[k], 1 - a.n[k], a.n[k] - 1};
    }
    int budget = 2000;
    for (int i = 0; i < n; ++i) {  // the first dimension in which the two differ
        dim[i].lo = 1;
        if (meets(dim + i, n - i, 0, a.d, &budget)) return true;
    }
    return false;
}

// An array of whole numbers or frequencies that a call reads (or, the new lengths, writes); null or empty: absent.
struct Array {
    const void *p;
    __int128 bytes;
};

static bool arrays_meet(const Array &a, const Array &b) {
    if (!a.p || !b.p) return false;
    const __int128 apart = (__int128)reinterpret_cast<uintptr_t>(a.p) - (__int128)reinterpret_cast<uintptr_t>(b.p);
    return apart < b.bytes && -apart < a.bytes;
}

// Whether a row of the tensor and the array share a byte: rows are whole units, so the array may be taken for the units that
// it touches, [0, len) from its first one.  A row at distance x meets it if -d < x < len; twice that, less the difference of
// the two, is what meets() asks for.
static bool rows_meet(const Rows &a, const Array &b) {
    if (!a.p || !b.p || b.bytes <= 0) return false;
    const __int128 at = (__int128)reinterpret_cast<uintptr_t>(b.p), first = at / 16, len = (at + b.bytes + 15) / 16 - first;
    const __int128 apart = (__int128)reinterpret_cast<uintptr_t>(a.p) / 16 - first;
    if (apart >= len || apart + a.span <= -a.d) return false;
    Reach dim[3];
    int n = 0;
    for (int k = 0; k < 3; ++k) {
        if (a.s[k] == 0 || a.n[k] < 2) continue;
        int i = n++;
        for (; i > 0 && dim[i - 1].s < 2 * (__int128)a.s[k]; --i) dim[i] = dim[i - 1];
        dim[i] = {2 * (__int128)a.s[k], 0, a.n[k] - 1};
    }
    int budget = 2000;
    return meets(dim, n, 2 * apart + a.d - len, a.d + len, &budget);
}

static Rows rows_in(const RopeTensor &t, int B, int N, int d) { return Rows(t.in, {t.in_b, t.in_h, t.in_n}, B, t.heads, N, d); }
static Rows rows_out(const RopeTensor &t, int B, int N, int d) { return Rows(t.out, {t.out_b, t.out_h, t.out_n}, B, t.heads, N, d); }

// The tensors of a rotation, and that no output is laid over what it must not be.
static int rope_tensors(RopeLaunch *a, const void *q, void *q_out, const void *k, void *k_out, int B, int Hq, int Hkv, int N,
                        int d, const long long *strides) {
    int rc = rope_tensor(&a->t[0], q, q_out, strides, strides ? strides + 3 : nullptr, B, Hq, N, d);
    if (rc == ATTN_OK && k)
        rc = rope_tensor(&a->t[1], k, k_out, strides ? strides + 6 : nullptr, strides ? strides + 9 : nullptr, B, Hkv, N, d);
    if (rc != ATTN_OK) return rc;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) {
            const Rows in = rows_in(a->t[i], B, N, d), out = rows_out(a->t[j], B, N, d);
            if (!(i == j && in.same(out)) && share_elements(in, out)) return ATTN_ERR_ARG;
        }
    if (share_elements(rows_out(a->t[0], B, N, d), rows_out(a->t[1], B, N, d))) return ATTN_ERR_ARG;
    if (shares_with_itself(rows_out(a->t[0], B, N, d)) || shares_with_itself(rows_out(a->t[1], B, N, d))) return ATTN_ERR_ARG;
    return ATTN_OK;
}

// The same for an append into caches [entries, Hkv, slots, d].
static int append_tensors(RopeLaunch *a, const void *q, void *q_out, const void *k, const void *v, void *kcache,
                          void *vcache, int B, int Hq, int Hkv, int T, int d, int entries, int slots,
                          const long long *strides) {
    const long long row = (long long)slots * d;
    int rc = rope_tensor(&a->t[0], q, q_out, strides, strides ? strides + 3 : nullptr, B, Hq, T, d);
    // The caches' strides are their own, so they are set apart from the inputs'.
    for (int i = 1; rc == ATTN_OK && i < 3; ++i) {
        rc = rope_tensor(&a->t[i], i == 1 ? k : v, i == 1 ? kcache : vcache, strides ? strides + 3 + 3 * i : nullptr,
                         nullptr, B, Hkv, T, d);
        a->t[i].out_b = Hkv * row;
        a->t[i].out_h = row;
        a->t[i].out_n = d;
    }
    if (rc != ATTN_OK) return rc;
    // The outputs: q_out (which may be q) and all of both caches.
    const Rows rotated = rows_out(a->t[0], B, T, d);
    const Rows caches[2] = {rows_out(a->t[1], entries, slots, d), rows_out(a->t[2], entries, slots, d)};
    for (int i = 0; i < 3; ++i) {
        const Rows in = rows_in(a->t[i], B, T, d);
        if ((i > 0 || !in.same(rotated)) && share_elements(in, rotated)) return ATTN_ERR_ARG;
        for (const Rows &cache : caches)
            if (share_elements(in, cache)) return ATTN_ERR_ARG;
    }
    if (shares_with_itself(rotated) || share_elements(rotated, caches[0]) || share_elements(rotated, caches[1]) || share_elements(caches[0], caches[1]))
        return ATTN_ERR_ARG;
    return ATTN_OK;
}

static bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static int rope_common(const double *inv_freq, int B, int Hq, int N, int d, int rotary_dim, float out_scale,
                       int min_rotary) {
    if (B <= 0 || Hq <= 0 || N <= 0) return ATTN_ERR_ARG;
    if (d <= 0 || d % 8 || d > 512) return ATTN_ERR_UNSUPPORTED;
    if (rotary_dim < min_rotary || rotary_dim > d || rotary_dim % 2) return ATTN_ERR_ARG;
    if (rotary_dim > 0 && (!inv_freq || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))) return ATTN_ERR_ARG;
    if (!std::isfinite(out_scale)) return ATTN_ERR_ARG;
    return ATTN_OK;
}

int attn_rope(const void *q, void *q_out, const void *k, void *k_out, const int *positions, long long position_stride,
              const double *inv_freq, int B, int Hq, int Hkv, int N, int d, int rotary_dim, int interleaved,
              float out_scale, int inverse, const long long *strides, attn_stream_t stream) {
    int rc = rope_common(inv_freq, B, Hq, N, d, rotary_dim, out_scale, 2);
    if (rc != ATTN_OK) return rc;
    if (!aligned4(positions) || position_stride < 0 || (!k != !k_out) || (k && Hkv <= 0)) return ATTN_ERR_ARG;
    RopeLaunch a;
    rc = rope_tensors(&a, q, q_out, k, k_out, B, Hq, Hkv, N, d, strides);
    if (rc != ATTN_OK) return rc;
    a.inv_freq = inv_freq;
    a.pos = positions;
    a.pos_stride = position_stride;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.inverse = inverse ? 1 : 0;
    a.out_scale = out_scale;
    a.num_sms = current_num_sms();
    if (a.num_sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    return rope_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_freqs(double *inv_freq, int rotary_dim, double base, int rule, double factor, double low, double high,
                    double trained_len) {
    if (!inv_freq || rotary_dim < 2 || rotary_dim % 2 || !(base > 1.0) || !std::isfinite(base)) return ATTN_ERR_ARG;
    if (rule < ATTN_ROPE_PLAIN || rule > ATTN_ROPE_BY_PARTS) return ATTN_ERR_ARG;
    if (rule != ATTN_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return ATTN_ERR_ARG;
    if (rule == ATTN_ROPE_BASE) {
        if (rotary_dim < 4) return ATTN_ERR_ARG;
        base *= std::pow(factor, double(rotary_dim) / (rotary_dim - 2));
    }
    if (rule == ATTN_ROPE_BY_PARTS && (!(low < high) || !std::isfinite(high - low) || !(trained_len > 0.0) || !std::isfinite(trained_len)))
        return ATTN_ERR_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (rule == ATTN_ROPE_LINEAR) f /= factor;
        if (rule == ATTN_ROPE_BY_PARTS) {
            double g = (trained_len * f / 6.283185307179586476925 - low) / (high - low);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f *= g + (1.0 - g) / factor;
        }
        inv_freq[i] = f;
    }
    return ATTN_OK;
}

// Whether [a, a + n) and [b, b + m) share a byte.
static bool bytes_overlap(const void *a, size_t n, const void *b, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + m && y < x + n;
}

static bool ints_overlap(const int *a, const int *b, int n) { return a && b && a < b + n && b < a + n; }

int attn_rope_append(const void *q, void *q_out, const void *k, const void *v, void *kcache, void *vcache,
                     const int *seqlens, const int *start_pos, const int *new_lens, int *seqlens_out, int *cache_pos,
                     float *weights, const double *inv_freq, int B, int Hq, int Hkv, int T, int d, int rotary_dim,
                     int interleaved, float out_scale, int max_seqlen, const long long *strides, attn_stream_t stream) {
    int rc = rope_common(inv_freq, B, Hq, T, d, rotary_dim, out_scale, 0);
    if (rc != ATTN_OK) return rc;
    if (Hkv <= 0 || max_seqlen <= 0 || !seqlens) return ATTN_ERR_ARG;
    for (const void *ptr : {(const void *)seqlens, (const void *)start_pos, (const void *)new_lens,
                            (const void *)seqlens_out, (const void *)cache_pos, (const void *)weights})
        if (!aligned4(ptr)) return ATTN_ERR_ARG;
    if (ints_overlap(seqlens_out, seqlens, B) || ints_overlap(seqlens_out, start_pos, B) ||
        ints_overlap(seqlens_out, new_lens, B))
        return ATTN_ERR_ARG;
    if (!aligned16(kcache) || !aligned16(vcache)) return ATTN_ERR_ARG;
    const long long row = (long long)max_seqlen * d;
    if ((double)B * Hkv * (double)row >= 9.0e18) return ATTN_ERR_ARG;
    RopeLaunch a;
    rc = append_tensors(&a, q, q_out, k, v, kcache, vcache, B, Hq, Hkv, T, d, B, max_seqlen, strides);
    if (rc != ATTN_OK) return rc;
    a.inv_freq = inv_freq;
    a.pos = start_pos;
    a.B = B;
    a.N = T;
    a.d = d;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.out_scale = out_scale;
    a.append = true;
    a.lens = seqlens;
    a.new_lens = new_lens;
    a.lens_out = seqlens_out;
    a.cache_pos = cache_pos;
    a.weights = weights;
    a.max_seqlen = max_seqlen;
    a.num_sms = current_num_sms();
    if (a.num_sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    return rope_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

// The caches of the paged calls (see attn.h): whether the sizes fit each other.
static int paged_sizes(const int *page_table, int B, int Hkv, int num_pages, int page_size, int max_pages) {
    if (B <= 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ATTN_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(page_table) & 3u) != 0) return ATTN_ERR_ARG;
    if ((long long)page_size * max_pages > (1LL << 30)) return ATTN_ERR_ARG;
    if ((long long)num_pages * Hkv > 0x7fffffffLL || (long long)B * Hkv > 0x7fffffffLL) return ATTN_ERR_ARG;
    if (page_table) return page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) ? ATTN_ERR_ARG : ATTN_OK;
    return num_pages != B || max_pages != 1 ? ATTN_ERR_ARG : ATTN_OK;
}

// log2 of the page size; one page a sequence: above every row.
static int page_shift_of(const int *page_table, int page_size) {
    int s = 0;
    while (page_table && (1 << s) < page_size) ++s;
    return page_table ? s : 30;
}

static int axes_common(const int *positions, long long axis_stride, long long position_stride, int num_axes,
                       const int *axes) {
    if (!aligned4(positions) || !aligned4(axes)) return ATTN_ERR_ARG;
    if (axis_stride < 0 || position_stride < 0 || num_axes < 1 || num_axes > 4) return ATTN_ERR_ARG;
    return ATTN_OK;
}

// From the first position to the last.
static __int128 positions_bytes(long long axis_stride, long long position_stride, int num_axes, int B, int N) {
    return ((__int128)axis_stride * (num_axes - 1) + (__int128)position_stride * (B - 1) + N) * 4;
}

int attn_rope_axes(const void *q, void *q_out, const void *k, void *k_out, const int *positions, long long axis_stride,
                   long long position_stride, int num_axes, const double *inv_freq, const int *axes, int B, int Hq,
                   int Hkv, int N, int d, int rotary_dim, int interleaved, float out_scale, int inverse,
                   const long long *strides, attn_stream_t stream) {
    int rc = rope_common(inv_freq, B, Hq, N, d, rotary_dim, out_scale, 2);
    if (rc == ATTN_OK) rc = axes_common(positions, axis_stride, position_stride, num_axes, axes);
    if (rc != ATTN_OK) return rc;
    if (!positions || (!k != !k_out) || (k && Hkv <= 0)) return ATTN_ERR_ARG;
    RopeLaunch a;
    rc = rope_tensors(&a, q, q_out, k, k_out, B, Hq, Hkv, N, d, strides);
    if (rc != ATTN_OK) return rc;
    const Array arrays[] = {{positions, positions_bytes(axis_stride, position_stride, num_axes, B, N)},
                            {axes, rotary_dim / 2 * 4}, {inv_freq, rotary_dim / 2 * 8}};
    for (const Array &x : arrays)  // other blocks still read them
        if (rows_meet(rows_out(a.t[0], B, N, d), x) || rows_meet(rows_out(a.t[1], B, N, d), x)) return ATTN_ERR_ARG;
    a.inv_freq = inv_freq;
    a.pos = positions;
    a.pos_stride = position_stride;
    a.axis_stride = axis_stride;
    a.num_axes = num_axes;
    a.axes = axes;
    a.B = B;
    a.N = N;
    a.d = d;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.inverse = inverse ? 1 : 0;
    a.out_scale = out_scale;
    a.num_sms = current_num_sms();
    if (a.num_sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    return rope_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_axes_append(const void *q, void *q_out, const void *k, const void *v, void *kpages, void *vpages,
                          const int *page_table, const int *seqlens, const int *positions, long long axis_stride,
                          long long position_stride, int num_axes, const int *new_lens, int *seqlens_out,
                          const double *inv_freq, const int *axes, int B, int Hq, int Hkv, int T, int d, int rotary_dim,
                          int interleaved, float out_scale, int num_pages, int page_size, int max_pages,
                          const long long *strides, attn_stream_t stream) {
    int rc = rope_common(inv_freq, B, Hq, T, d, rotary_dim, out_scale, 0);
    if (rc == ATTN_OK) rc = axes_common(positions, axis_stride, position_stride, num_axes, axes);
    if (rc == ATTN_OK) rc = paged_sizes(page_table, B, Hkv, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    if (!seqlens || !aligned4(seqlens) || !aligned4(new_lens) || !aligned4(seqlens_out)) return ATTN_ERR_ARG;
    const __int128 lens = (__int128)B * 4;
    const Array written = {seqlens_out, lens};
    const Array arrays[] = {{seqlens, lens}, {new_lens, lens}, {page_table, lens * max_pages},
                            {positions, positions_bytes(axis_stride, position_stride, num_axes, B, T)},
                            {axes, rotary_dim / 2 * 4}, {inv_freq, rotary_dim / 2 * 8}};
    for (const Array &x : arrays)  // other blocks still read them
        if (arrays_meet(x, written)) return ATTN_ERR_ARG;
    if (!aligned16(kpages) || !aligned16(vpages)) return ATTN_ERR_ARG;
    const long long row = (long long)page_size * d;
    if ((double)num_pages * Hkv * (double)row >= 9.0e18) return ATTN_ERR_ARG;
    RopeLaunch a;
    rc = append_tensors(&a, q, q_out, k, v, kpages, vpages, B, Hq, Hkv, T, d, num_pages, page_size, strides);
    if (rc != ATTN_OK) return rc;
    const Rows outs[] = {rows_out(a.t[0], B, T, d), rows_out(a.t[1], num_pages, page_size, d),
                         rows_out(a.t[2], num_pages, page_size, d)};
    for (const Rows &out : outs) {
        if (rows_meet(out, written)) return ATTN_ERR_ARG;
        for (const Array &x : arrays)
            if (rows_meet(out, x)) return ATTN_ERR_ARG;
    }
    for (const RopeTensor &t : a.t)
        if (rows_meet(rows_in(t, B, T, d), written)) return ATTN_ERR_ARG;
    a.inv_freq = inv_freq;
    a.pos = positions;
    a.pos_stride = position_stride;
    a.axis_stride = axis_stride;
    a.num_axes = num_axes;
    a.axes = axes;
    a.table = page_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_shift = page_shift_of(page_table, page_size);
    a.B = B;
    a.N = T;
    a.d = d;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.out_scale = out_scale;
    a.append = true;
    a.lens = seqlens;
    a.new_lens = new_lens;
    a.lens_out = seqlens_out;
    a.max_seqlen = page_size * max_pages;
    a.num_sms = current_num_sms();
    if (a.num_sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    return rope_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

static int decode_prefix_sizes(int B, int Hq, int Hkv, int P, int d, int max_seqlen) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || P < 0 || max_seqlen < 0 || Hq % Hkv) return ATTN_ERR_ARG;
    if (P == 0 && max_seqlen == 0) return ATTN_ERR_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > kDecodeMaxGroup) return ATTN_ERR_UNSUPPORTED;
    if (Hkv > 65535 || (long long)B * Hq > (1 << 30) || max_seqlen > (1 << 30) || P > (1 << 30)) return ATTN_ERR_ARG;
    // tensor-map limits, and the work list's total of keys stays below 2^62
    if ((long long)max_seqlen * d * 2 >= (1LL << 39) || (long long)P * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    if ((double)B * (double)max_seqlen * (double)Hkv >= 4.0e18) return ATTN_ERR_ARG;
    return ATTN_OK;
}

size_t attn_decode_prefix_workspace_bytes(int B, int Hq, int Hkv, int P, int d, int max_seqlen, int with_weights) {
    if (decode_prefix_sizes(B, Hq, Hkv, P, d, max_seqlen) != ATTN_OK) return 0;
    const int sms = current_num_sms();
    PrefixLayout l;
    if (sms <= 0 || !decode_prefix_layout(B, Hq, Hkv, P, d, max_seqlen, with_weights != 0, sms, &l)) return 0;
    return l.bytes;
}

int attn_decode_prefix(const void *q, const void *kprefix, const void *vprefix, const void *kcache, const void *vcache,
                       const int *seqlens, void *o, float *lse, float *weights, int B, int Hq, int Hkv, int P, int d,
                       float scale, int max_seqlen, void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    const int rc = decode_prefix_sizes(B, Hq, Hkv, P, d, max_seqlen);
    if (rc != ATTN_OK) return rc;
    if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(weights)) return ATTN_ERR_ARG;
    if (P > 0 && (!aligned16(kprefix) || !aligned16(vprefix))) return ATTN_ERR_ARG;
    if (max_seqlen > 0 && (!aligned16(kcache) || !aligned16(vcache) || !seqlens || !aligned4(seqlens)))
        return ATTN_ERR_ARG;
    if (weights && max_seqlen == 0) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    if (!workspace || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    PrefixLayout l;
    if (!decode_prefix_layout(B, Hq, Hkv, P, d, max_seqlen, weights != nullptr, sms, &l)) return ATTN_ERR_ARG;
    if (workspace_bytes < l.bytes) return ATTN_ERR_WORKSPACE;
    DecodePrefixLaunch a;
    a.q = q;
    a.kprefix = kprefix;
    a.vprefix = vprefix;
    a.kcache = kcache;
    a.vcache = vcache;
    a.seqlens = seqlens;
    a.o = o;
    a.lse = lse;
    a.weights = weights;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.P = P;
    a.d = d;
    a.max_seqlen = max_seqlen;
    a.scale = scale;
    a.workspace = static_cast<char *>(workspace);
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return decode_prefix_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_decode_prefix_segment(int B, int Hq, int Hkv, int P, int d, int max_seqlen, long long own_keys, int num_sms,
                               int cta, int i, int *out) {
    PrefixOrder o;
    if (!out || P <= 0 || num_sms <= 0 || num_sms > (1 << 20) || i < 0 || own_keys < 0 ||
        decode_prefix_sizes(B, Hq, Hkv, P, d, max_seqlen) != ATTN_OK ||
        !prefix_order(&o, B, Hq / Hkv, Hkv, P, d, max_seqlen, own_ctas(B, Hq / Hkv, Hkv, P, d, max_seqlen, num_sms), num_sms) || cta < 0 ||
        cta >= prefix_grid(o))
        return ATTN_ERR_ARG;
    const PrefixShares s = prefix_shares(o, own_keys * Hkv);
    const int share = prefix_share(o, cta);
    const unsigned hi = prefix_begin(o, s, share + 1);
    const int u = prefix_start(o, prefix_begin(o, s, share), hi, i);
    if (u < 0) return 0;
    const PrefixSegment seg = prefix_segment(o, hi, cta, u);
    const int last = prefix_holder(o, s, unsigned(seg.row + 1) * o.nblk - 1);
    const int v[6] = {seg.g, seg.m, seg.j0, seg.n, share + seg.row, last + seg.row};
    for (int k = 0; k < 6; ++k) out[k] = v[k];
    return 1;
}

size_t attn_cache_evict_workspace_bytes(int B, int Hkv, int max_seqlen, int keep, int in_place) {
    if (B <= 0 || Hkv <= 0 || max_seqlen <= 0 || keep <= 0 || (long long)B * Hkv > 0x7fffffffLL) return 0;
    EvictLaunch a = {};
    a.B = B;
    a.Hkv = Hkv;
    a.max_seqlen = max_seqlen;
    a.keep = keep;
    a.kout = in_place ? nullptr : &a;  // in place: the same address as kcache
    return evict_workspace_bytes(a);
}

int attn_cache_evict(const void *kcache, const void *vcache, const float *weights, const int *cache_pos,
                     const int *seqlens, const int *cur_pos, void *kout, void *vout, float *weights_out, int *pos_out,
                     int *seqlens_out, int B, int Hkv, int d, int max_seqlen, int out_seqlen, int keep, int recent,
                     void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (B <= 0 || Hkv <= 0 || max_seqlen <= 0 || out_seqlen <= 0 || keep <= 0 || keep > out_seqlen || recent < 0 ||
        recent > keep)
        return ATTN_ERR_ARG;
    if (d <= 0 || d % 8 || d > 512) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hkv > 0x7fffffffLL || max_seqlen > (1 << 30)) return ATTN_ERR_ARG;
    const size_t rows = (size_t)B * Hkv;
    if ((double)rows * (max_seqlen > out_seqlen ? max_seqlen : out_seqlen) * d >= 4.0e18) return ATTN_ERR_ARG;
    if (!aligned16(kcache) || !aligned16(vcache) || !aligned16(kout) || !aligned16(vout)) return ATTN_ERR_ARG;
    if (!weights || !seqlens) return ATTN_ERR_ARG;
    for (const void *ptr : {(const void *)weights, (const void *)cache_pos, (const void *)seqlens, (const void *)cur_pos,
                            (const void *)weights_out, (const void *)pos_out, (const void *)seqlens_out})
        if (!aligned4(ptr)) return ATTN_ERR_ARG;
    if (ints_overlap(seqlens_out, seqlens, B) || ints_overlap(seqlens_out, cur_pos, B)) return ATTN_ERR_ARG;
    const bool in_place = kout == kcache;
    if (in_place && (vout != vcache || weights_out != weights || pos_out != cache_pos || out_seqlen != max_seqlen))
        return ATTN_ERR_ARG;
    // An output may overlap no other output and, but for its own in place, no input.
    const size_t in4 = rows * max_seqlen * 4, out4 = rows * out_seqlen * 4;
    const size_t in = rows * max_seqlen * d * 2, out = rows * out_seqlen * d * 2;
    const struct {
        const void *p;
        size_t n;
    } ins[] = {{kcache, in}, {vcache, in}, {weights, in4}, {cache_pos, in4}},
      outs[] = {{kout, out}, {vout, out}, {weights_out, out4}, {pos_out, out4}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if ((!(in_place && i == j) && bytes_overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) ||
                (j < i && bytes_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)))
                return ATTN_ERR_ARG;
    EvictLaunch a;
    a.kcache = kcache;
    a.vcache = vcache;
    a.weights = weights;
    a.cache_pos = cache_pos;
    a.seqlens = seqlens;
    a.cur_pos = cur_pos;
    a.kout = kout;
    a.vout = vout;
    a.weights_out = weights_out;
    a.pos_out = pos_out;
    a.seqlens_out = seqlens_out;
    a.B = B;
    a.Hkv = Hkv;
    a.d = d;
    a.max_seqlen = max_seqlen;
    a.out_seqlen = out_seqlen;
    a.keep = keep;
    a.recent = recent;
    a.workspace = static_cast<char *>(workspace);
    const size_t need = evict_workspace_bytes(a);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
    a.num_sms = current_num_sms();
    if (a.num_sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    return evict_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

// Whether any two of the arrays share a byte (null ones do not).
struct Span {
    const void *p;
    size_t n;
};
static bool any_overlap(const Span *s, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if (bytes_overlap(s[i].p, s[i].n, s[j].p, s[j].n)) return true;
    return false;
}

// Trees of drafted tokens.
static bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
constexpr int kMaxDraft = 256;

int attn_tree_mask(const int *parents, const int *seqlens, const int *draft_lens, long long *mask, int *positions, int B,
                   int T, attn_stream_t stream) {
    if (B <= 0 || T <= 0 || T > kMaxDraft || !parents || !mask || !aligned8(mask)) return ATTN_ERR_ARG;
    if (!aligned4(parents) || !aligned4(seqlens) || !aligned4(draft_lens) || !aligned4(positions)) return ATTN_ERR_ARG;
    const size_t nodes = size_t(B) * T * 4, lens = size_t(B) * 4, bits = size_t(B) * T * ((T + 63) / 64) * 8;
    const struct {
        const void *p;
        size_t n;
    } ins[] = {{parents, nodes}, {seqlens, lens}, {draft_lens, lens}};
    for (const auto &in : ins)
        if (bytes_overlap(mask, bits, in.p, in.n) || bytes_overlap(positions, nodes, in.p, in.n)) return ATTN_ERR_ARG;
    if (bytes_overlap(mask, bits, positions, nodes)) return ATTN_ERR_ARG;
    TreeLaunch a;
    a.parents = parents;
    a.seqlens = seqlens;
    a.draft_lens = draft_lens;
    a.mask_out = reinterpret_cast<unsigned long long *>(mask);
    a.positions = positions;
    a.B = B;
    a.T = T;
    return tree_mask_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

static int decode_tree_sizes(int B, int Hq, int Hkv, int T, int d, int page_size, int max_pages) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || T <= 0 || Hq % Hkv || page_size <= 0 || max_pages <= 0) return ATTN_ERR_ARG;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq / Hkv > kDecodeMaxGroup || T > kMaxDraft) return ATTN_ERR_UNSUPPORTED;
    const long long cap = (long long)page_size * max_pages;
    if (cap > (1 << 30) || (long long)B * Hkv > 0x7fffffffLL) return ATTN_ERR_ARG;
    return (double)B * Hkv * (double)((cap + 63) / 64) < 2147483648.0 ? ATTN_OK : ATTN_ERR_ARG;
}

size_t attn_decode_tree_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int page_size, int max_pages) {
    if (decode_tree_sizes(B, Hq, Hkv, T, d, page_size, max_pages) != ATTN_OK) return 0;
    const int sms = current_num_sms();
    return sms <= 0 ? 0 : decode_tree_workspace_bytes(B, Hq / Hkv, Hkv, T, d, (long long)page_size * max_pages, sms);
}

int attn_decode_tree(const void *q, const void *kpages, const void *vpages, const int *page_table, const int *seqlens,
                     const long long *mask, const int *draft_lens, void *o, float *lse, int B, int Hq, int Hkv, int T,
                     int d, float scale, int num_pages, int page_size, int max_pages, void *workspace,
                     size_t workspace_bytes, attn_stream_t stream) {
    int rc = decode_tree_sizes(B, Hq, Hkv, T, d, page_size, max_pages);
    if (rc == ATTN_OK) rc = paged_sizes(page_table, B, Hkv, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    if (!aligned16(q) || !aligned16(kpages) || !aligned16(vpages) || !aligned16(o) || !seqlens) return ATTN_ERR_ARG;
    if (!aligned4(seqlens) || !aligned4(draft_lens) || !aligned4(lse) || !aligned8(mask)) return ATTN_ERR_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_ARG;
    // tensor-map limits
    if ((long long)page_size * d * 2 >= (1LL << 39) || (long long)(Hq / Hkv) * T * d * 2 >= (1LL << 39)) return ATTN_ERR_ARG;
    if (!workspace || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
    const int sms = current_num_sms();
    if (sms <= 0) return note_cuda_error(cudaErrorNoDevice, "device query");
    const size_t need = decode_tree_workspace_bytes(B, Hq / Hkv, Hkv, T, d, (long long)page_size * max_pages, sms);
    if (workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    // An output may overlap no input, nor the workspace.
    const size_t rows = size_t(B) * Hq * T, cache = size_t(num_pages) * Hkv * page_size * d * 2, lens = size_t(B) * 4;
    const Span outs[] = {{o, rows * d * 2}, {lse, rows * 4}, {workspace, need}};
    const Span ins[] = {{q, rows * d * 2}, {kpages, cache}, {vpages, cache}, {page_table, lens * max_pages}, {seqlens, lens},
                        {draft_lens, lens}, {mask, size_t(B) * T * ((T + 63) / 64) * 8}};
    if (any_overlap(outs, 3)) return ATTN_ERR_ARG;
    for (const Span &x : outs)
        for (const Span &y : ins)
            if (bytes_overlap(x.p, x.n, y.p, y.n)) return ATTN_ERR_ARG;
    DecodeTreeLaunch a;
    a.q = q;
    a.kpages = kpages;
    a.vpages = vpages;
    a.table = page_table;
    a.seqlens = seqlens;
    a.draft_lens = draft_lens;
    a.mask = reinterpret_cast<const unsigned long long *>(mask);
    a.o = o;
    a.lse = lse;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.T = T;
    a.d = d;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.page_shift = page_shift_of(page_table, page_size);
    a.max_pages = max_pages;
    a.scale = scale;
    a.workspace = static_cast<char *>(workspace);
    a.wait_ns = (unsigned long long)g_wait_ns.load();
    a.num_sms = sms;
    return decode_tree_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

// Pools of all layers [layers, num_pages, Hkv, page_size, d].
static int pools(const void *k, const void *v, int layers, int Hkv, int d, int num_pages, int page_size, size_t *bytes) {
    if (layers <= 0 || Hkv <= 0) return ATTN_ERR_ARG;
    if (d <= 0 || d % 8 || d > 512) return ATTN_ERR_UNSUPPORTED;
    if (!aligned16(k) || !aligned16(v)) return ATTN_ERR_ARG;
    if ((double)layers * num_pages * Hkv * ((double)page_size * d) >= 4.0e18) return ATTN_ERR_ARG;
    if ((long long)layers * 2 * Hkv * (d / 8) > 0x3fffffffLL) return ATTN_ERR_ARG;  // counted in 32 bits
    *bytes = (size_t)layers * num_pages * Hkv * page_size * d * 2;
    return bytes_overlap(k, *bytes, v, *bytes) ? ATTN_ERR_ARG : ATTN_OK;
}

int attn_tree_accept(void *kpages, void *vpages, const int *page_table, const int *seqlens, const long long *mask,
                     const int *last, int *seqlens_out, int layers, int B, int Hkv, int T, int d, int num_pages,
                     int page_size, int max_pages, attn_stream_t stream) {
    int rc = paged_sizes(page_table, B, Hkv, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    size_t bytes = 0;
    rc = pools(kpages, vpages, layers, Hkv, d, num_pages, page_size, &bytes);
    if (rc != ATTN_OK) return rc;
    if (T <= 0 || T > kMaxDraft || !seqlens || !last) return ATTN_ERR_ARG;
    if (!aligned4(seqlens) || !aligned4(last) || !aligned4(seqlens_out) || !aligned8(mask)) return ATTN_ERR_ARG;
    const size_t lens = size_t(B) * 4;
    const struct {
        const void *p;
        size_t n;
    } ins[] = {{seqlens, lens}, {last, lens}, {mask, size_t(B) * T * ((T + 63) / 64) * 8}, {page_table, lens * max_pages}};
    for (const auto &in : ins)
        for (void *out : {kpages, vpages, (void *)seqlens_out})
            if (bytes_overlap(out, out == seqlens_out ? lens : bytes, in.p, in.n)) return ATTN_ERR_ARG;
    if (bytes_overlap(seqlens_out, lens, kpages, bytes) || bytes_overlap(seqlens_out, lens, vpages, bytes)) return ATTN_ERR_ARG;
    TreeLaunch a;
    a.kpages = kpages;
    a.vpages = vpages;
    a.table = page_table;
    a.seqlens = seqlens;
    a.mask = reinterpret_cast<const unsigned long long *>(mask);
    a.last = last;
    a.lens_out = seqlens_out;
    a.layers = layers;
    a.B = B;
    a.Hkv = Hkv;
    a.T = T;
    a.d = d;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.page_shift = page_shift_of(page_table, page_size);
    a.max_pages = max_pages;
    return tree_accept_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

// The pages of a cache.
static int tables(const int *page_table, const int *refs, int B, int num_pages, int page_size, int max_pages) {
    if (!page_table || !refs || !aligned4(refs)) return ATTN_ERR_ARG;
    const int rc = paged_sizes(page_table, B, 1, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    return (long long)B * max_pages > (1 << 30) || num_pages > (1 << 30) ? ATTN_ERR_ARG : ATTN_OK;
}

size_t attn_pages_workspace_bytes(int B, int num_pages) {
    return B <= 0 || num_pages <= 0 || B > (1 << 30) || num_pages > (1 << 30) ? 0 : pages_workspace_bytes(B, num_pages);
}

static int pages_moves(PagesLaunch *a, int *page_table, int *refs, void *kpages, void *vpages, int *info, int layers, int B,
                       int Hkv, int d, int num_pages, int page_size, int max_pages, const int *seqlens,
                       const int *new_lens, void *workspace, size_t workspace_bytes) {
    int rc = tables(page_table, refs, B, num_pages, page_size, max_pages);
    if (rc == ATTN_OK) rc = paged_sizes(page_table, B, Hkv, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    size_t bytes = 0;
    rc = pools(kpages, vpages, layers, Hkv, d, num_pages, page_size, &bytes);
    if (rc != ATTN_OK) return rc;
    // A page's 16-byte units, rounded up to a warp's 256, are counted in 32 bits.
    if ((long long)Hkv * page_size * (d / 8) > 0x7fffffffLL - 255) return ATTN_ERR_ARG;
    if (!info || !aligned4(info) || !aligned4(seqlens) || !aligned4(new_lens)) return ATTN_ERR_ARG;
    const size_t need = pages_workspace_bytes(B, num_pages), lens = size_t(B) * 4;
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    const Span arrays[] = {{page_table, lens * max_pages}, {refs, size_t(num_pages) * 4}, {info, 8}, {seqlens, lens},
                           {kpages, bytes}, {vpages, bytes}, {workspace, need}};
    if (any_overlap(arrays, int(sizeof(arrays) / sizeof(Span)))) return ATTN_ERR_ARG;
    for (const Span &s : arrays)  // (the two lengths are only read)
        if (s.p != seqlens && bytes_overlap(new_lens, lens, s.p, s.n)) return ATTN_ERR_ARG;
    a->table = page_table;
    a->refs = refs;
    a->seqlens = seqlens;
    a->new_lens = new_lens;
    a->kpages = kpages;
    a->vpages = vpages;
    a->info = info;
    a->layers = layers;
    a->B = B;
    a->Hkv = Hkv;
    a->d = d;
    a->num_pages = num_pages;
    a->page_size = page_size;
    a->max_pages = max_pages;
    a->workspace = static_cast<char *>(workspace);
    a->num_sms = current_num_sms();
    return a->num_sms <= 0 ? note_cuda_error(cudaErrorNoDevice, "device query") : ATTN_OK;
}

int attn_pages_extend(int *page_table, int *refs, const int *seqlens, const int *new_lens, int T, void *kpages,
                      void *vpages, int *info, int layers, int B, int Hkv, int d, int num_pages, int page_size,
                      int max_pages, void *workspace, size_t workspace_bytes, attn_stream_t stream) {
    if (!seqlens || T < 0) return ATTN_ERR_ARG;
    PagesLaunch a;
    const int rc = pages_moves(&a, page_table, refs, kpages, vpages, info, layers, B, Hkv, d, num_pages, page_size,
                               max_pages, seqlens, new_lens, workspace, workspace_bytes);
    if (rc != ATTN_OK) return rc;
    a.T = T;
    return pages_extend_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_compact(int *page_table, int *refs, void *kpages, void *vpages, int *info, int layers, int B, int Hkv,
                       int d, int num_pages, int page_size, int max_pages, void *workspace, size_t workspace_bytes,
                       attn_stream_t stream) {
    PagesLaunch a;
    const int rc = pages_moves(&a, page_table, refs, kpages, vpages, info, layers, B, Hkv, d, num_pages, page_size,
                               max_pages, nullptr, nullptr, workspace, workspace_bytes);
    if (rc != ATTN_OK) return rc;
    return pages_compact_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_fork(const int *page_table, int *page_table_out, int *refs, const int *seqlens, int *seqlens_out,
                    const int *parent, int B, int num_pages, int page_size, int max_pages, attn_stream_t stream) {
    const int rc = tables(page_table, refs, B, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    if (!page_table_out || !seqlens || !seqlens_out || !parent) return ATTN_ERR_ARG;
    for (const int *ptr : {(const int *)page_table_out, seqlens, (const int *)seqlens_out, parent})
        if (!aligned4(ptr)) return ATTN_ERR_ARG;
    const size_t lens = size_t(B) * 4;
    const Span arrays[] = {{page_table, lens * max_pages}, {page_table_out, lens * max_pages}, {refs, size_t(num_pages) * 4},
                           {seqlens, lens}, {seqlens_out, lens}, {parent, lens}};
    if (any_overlap(arrays, int(sizeof(arrays) / sizeof(Span)))) return ATTN_ERR_ARG;
    PagesLaunch a;
    a.table = const_cast<int *>(page_table);
    a.table_out = page_table_out;
    a.refs = refs;
    a.seqlens = seqlens;
    a.lens_out = seqlens_out;
    a.parent = parent;
    a.B = B;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    return pages_fork_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_trim(int *page_table, int *refs, const int *seqlens, int *seqlens_out, const int *keep_lens, int B,
                    int num_pages, int page_size, int max_pages, attn_stream_t stream) {
    const int rc = tables(page_table, refs, B, num_pages, page_size, max_pages);
    if (rc != ATTN_OK) return rc;
    if (!seqlens || !keep_lens || !aligned4(seqlens) || !aligned4(seqlens_out) || !aligned4(keep_lens)) return ATTN_ERR_ARG;
    const size_t lens = size_t(B) * 4;
    const Span arrays[] = {{page_table, lens * max_pages}, {refs, size_t(num_pages) * 4},
                           {seqlens_out == seqlens ? nullptr : seqlens, lens}, {seqlens_out, lens}};
    if (any_overlap(arrays, int(sizeof(arrays) / sizeof(Span)))) return ATTN_ERR_ARG;
    for (const Span &s : {arrays[0], arrays[1], arrays[3]})
        if (bytes_overlap(keep_lens, lens, s.p, s.n)) return ATTN_ERR_ARG;
    PagesLaunch a;
    a.table = page_table;
    a.refs = refs;
    a.seqlens = seqlens;
    a.lens_out = seqlens_out;
    a.new_lens = keep_lens;
    a.B = B;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.max_pages = max_pages;
    return pages_trim_launch(a, reinterpret_cast<cudaStream_t>(stream));
}

int attn_device_status(attn_stream_t stream) {
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return ATTN_ERR_CUDA;
    int a = 0, b = 0, c = 0, e = 0, f = 0, g = 0, h = 0, i = 0;
    if (fwd_take_status(&a) != cudaSuccess || decode_take_status(&b) != cudaSuccess ||
        bwd_take_status(&c) != cudaSuccess || fwd_pair_take_status(&e) != cudaSuccess ||
        fwd_split_take_status(&f) != cudaSuccess || decode_prefix_take_status(&g) != cudaSuccess ||
        own_take_status(&h) != cudaSuccess || decode_tree_take_status(&i) != cudaSuccess)
        return ATTN_ERR_CUDA;
    return (a | b | c | e | f | g | h | i) ? ATTN_ERR_TIMEOUT : ATTN_OK;
}

}  // extern "C"
