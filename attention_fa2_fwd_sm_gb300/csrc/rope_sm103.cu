// rope_sm103.cu -- rotary positions: of q and k before attention, of their
// gradients after it, and of new tokens on their way into a decode cache.
//
// A token at position p has pair i of its rotated columns turned by the angle
// a = p f_i:
//     (x, y) -> s (x cos a - y sin a,  y cos a + x sin a),
// pairs (x_i, x_{i + r/2}) in the half layout and (x_2i, x_2i+1) in the
// interleaved one; columns from r on are copied.  The rotation is orthogonal,
// so the gradient is the same map with the angle negated.
//
// Angles.  In fp32 the product p f_i is off by up to 2^-24 p f_i radians: 0.06
// at a million.  Instead f_i becomes a 64-bit fixed-point number of turns,
// u = frac(f_i / 2 pi) 2^64, and the phase p u mod 2^64 is one integer product
// that drops whole turns exactly.  Its top 32 bits, as a signed fraction of a
// half turn, go to sincospif: the angle is off by 2^-24 of a half turn at any
// position (u itself by less than one unit, which makes 2^-33 turns of the
// farthest).  The conversion of f_i is integer arithmetic too (a 53-bit mantissa
// times 2^130 / 2 pi, 181 bits, so that u is right up to f_i = 2^54): this GPU has
// few fp64 units, and eight conversions a thread on them would take as long as the
// thread's memory traffic.
//
// What bounds it: every element is read and written once (4 bytes), nothing
// else of size moves, so HBM.  A thread owns one 8-column unit of one token
// (in the half layout its partner unit too), computes that unit's sines once
// and applies them to up to kMaxHeads heads, whose loads it issues together.
// 8192 tokens, 64 + 8 heads, d = 128 (302 MB): 48.4 us, 6.2 TB/s; one head a
// thread 100 us (the sines), 4 or 16 heads 48.5, loads of 2 or 8 heads at a time
// 49.0 and 48.6.  2048 tokens, 32 + 8 heads: 8.9 us in blocks of 128 threads, 10.3
// in blocks of 256, whose last wave is the coarser.
//
// Several axes (kAxes): a token has up to four positions (time, height, width; the
// depth in a tree) and pair i turns by the one that axes[i] names.  The phase of a
// pair is then its own axis's product; nothing else changes, and nothing else is
// read but 4 bytes an axis and token: 8192 tokens of 64 + 8 heads by three axes take
// 50 us (6.0 TB/s of reads and writes; 49 to 50 by one position).  Appending by axes
// also looks the row's page up: a row of a sequence is a row of one of its pages.
// 4 x 2000 tokens, ragged, into pages of 16: 53.5 us, as into a contiguous cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace rope {

constexpr int kThreads = 128;
constexpr int kMaxHeads = 8;   // heads a thread visits with one set of sines
constexpr int kBatch = 4;      // heads whose loads are in flight together
constexpr int kMaxPairs = 256; // rotary_dim <= 512
constexpr int kMaxAxes = 4;

// Item layouts.  Vector items are 8 columns (16 bytes), half: 8 columns and
// the 8 that they pair with; the pair forms take any even rotary_dim, one
// pair an item.
enum Layout : int { kHalfVec = 0, kInterVec = 1, kHalfPair = 2, kInterPair = 3 };

struct Params {
    RopeTensor t[3];      // q, k and (appending) v
    int chunks[3];        // head chunks of each in the grid's y
    int heads_per_chunk;
    const double *inv_freq;
    const int *pos;       // rope: [N] a batch entry, pos_stride apart (null: 0..N-1); append: first position (null: lens)
    long long pos_stride;
    const int *lens, *new_lens;  // append
    int *lens_out, *cache_pos;
    float *weights;
    long long tokens;     // B * N
    int N, r, items, rot_items, max_seqlen;
    float scale, sign;
    // kAxes
    const int *axes;       // [r / 2] (null: all 0)
    const int *table;      // [B, max_pages] (null: sequence b's only page is b)
    long long axis_stride; // between the axes in pos
    int num_axes, max_pages, num_pages, page_shift;
};

// 2^130 / (2 pi), rounded: its upper and its lower 64 bits.
constexpr unsigned long long kTurnsHi = 0xA2F9836E4E441529ull, kTurnsLo = 0xFC2757D1F534DDC1ull;

// frac(f / 2 pi) in units of 2^-64 turns.  f = m 2^(e - 1075) with a 53-bit m,
// so f / 2 pi * 2^64 = (m kTurns 2^-64) 2^(e - 1077).  Frequencies from 2^54 up, and
// infinities and NaN, give 0: no position has a meaningful angle there.
__device__ __forceinline__ unsigned long long turns_of(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int e = int(bits >> 52) & 0x7ff;
    unsigned long long m = bits & 0xfffffffffffffull;
    if (e) m |= 1ull << 52;
    const int shift = 1077 - (e ? e : 1);
    if (shift <= 0 || shift >= 128) return 0;
    // The upper 128 of the product's 192 bits.
    const unsigned long long low = __umul64hi(m, kTurnsLo), lo = m * kTurnsHi + low;
    const unsigned long long hi = __umul64hi(m, kTurnsHi) + (lo < low);
    const unsigned long long u = shift >= 64 ? hi >> (shift - 64) : (lo >> shift) | (hi << (64 - shift));
    return (long long)bits < 0 ? 0ull - u : u;
}

__device__ __forceinline__ void sin_cos(unsigned long long turns, int pos, float sign, float scale, float &c,
                                        float &s) {
    const unsigned long long phase = (unsigned long long)(long long)pos * turns;
    sincospif(float(int(phase >> 32)) * 0x1p-31f, &s, &c);
    c *= scale;
    s *= sign * scale;
}

__device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// (x, y) -> (x c - y s, y c + x s) for the four pairs whose x and y sit in
// matching halves of two registers each.
__device__ __forceinline__ void turn_half(uint4 &x, uint4 &y, const float (&c)[8], const float (&s)[8]) {
    uint32_t *px = &x.x, *py = &y.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack(px[i]), b = unpack(py[i]);
        px[i] = pack_bf16x2(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
        py[i] = pack_bf16x2(b.x * c[2 * i] + a.x * s[2 * i], b.y * c[2 * i + 1] + a.y * s[2 * i + 1]);
    }
}
__device__ __forceinline__ void turn_inter(uint4 &x, const float (&c)[8], const float (&s)[8]) {
    uint32_t *px = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack(px[i]);
        px[i] = pack_bf16x2(a.x * c[i] - a.y * s[i], a.y * c[i] + a.x * s[i]);
    }
}

// Grid: x over (token, item), y over the head chunks of q, then k, then v.
template <int kLayout, bool kAppend, bool kAxes>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
    __shared__ unsigned long long turns[kMaxPairs];
    __shared__ int axis_of[kAxes ? kMaxPairs : 1];
    for (int i = threadIdx.x; i < p.r / 2; i += kThreads) {
        turns[i] = turns_of(p.inv_freq[i]);
        if constexpr (kAxes) axis_of[i] = p.axes ? min(max(p.axes[i], 0), p.num_axes - 1) : 0;
    }
    __syncthreads();

    const long long flat = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long token = flat / p.items;
    const int item = int(flat - token * p.items);
    if (token >= p.tokens) return;
    const int b = int(token / p.N), n = int(token - (long long)b * p.N);

    // This block's tensor and heads.
    int chunk = blockIdx.y, which = 0;
    while (chunk >= p.chunks[which]) chunk -= p.chunks[which++];
    const RopeTensor &t = p.t[which];
    const int h0 = chunk * p.heads_per_chunk, h1 = min(h0 + p.heads_per_chunk, t.heads);

    int pos = 0, more[kMaxAxes - 1] = {};  // on axis 0 and on the others
    long long row = n, entry = b;      // row of the output, and the batch entry or page that it is in
    bool store = true;
    if constexpr (kAxes) {
        if (p.pos) {
            const int *at = p.pos + b * p.pos_stride + n;
            pos = at[0];
#pragma unroll
            for (int a = 1; a < kMaxAxes; ++a)
                if (a < p.num_axes) more[a - 1] = at[a * p.axis_stride];
        }
    }
    auto pos_of = [&](int pair) {
        if constexpr (!kAxes) return pos;
        const int a = axis_of[pair];
        return a == 0 ? pos : a == 1 ? more[0] : a == 2 ? more[1] : more[2];
    };
    if constexpr (kAppend) {
        const int len = min(max(p.lens[b], 0), p.max_seqlen);
        const int added = p.new_lens ? min(max(p.new_lens[b], 0), p.N) : p.N;
        if constexpr (!kAxes) {
            pos = int(unsigned(p.pos ? p.pos[b] : len) + unsigned(n));
        } else if (!p.pos) {
            pos = int(unsigned(len) + unsigned(n));
            more[0] = more[1] = more[2] = pos;
        }
        if (which > 0) {
            row = (long long)len + n;
            store = n < added && row < p.max_seqlen;
            if constexpr (kAxes) {
                if (store && p.table) {
                    const int page = p.table[(long long)b * p.max_pages + (row >> p.page_shift)];
                    store = page >= 0 && page < p.num_pages;
                    entry = page;
                }
                row &= (1LL << p.page_shift) - 1;
            } else if (which == 1 && item == 0 && store) {
                for (int h = h0; h < h1; ++h) {
                    const long long at = ((long long)b * t.heads + h) * p.max_seqlen + row;
                    if (p.cache_pos) p.cache_pos[at] = pos;
                    if (p.weights) p.weights[at] = 0.f;
                }
            }
        } else if (blockIdx.y == 0 && item == 0 && n == 0 && p.lens_out) {
            p.lens_out[b] = int(min((long long)len + added, (long long)p.max_seqlen));
        }
        if (!store) return;
    } else if constexpr (!kAxes) {
        pos = p.pos ? p.pos[b * p.pos_stride + n] : n;
    }
    const bool turn = item < p.rot_items && which < 2;
    const __nv_bfloat16 *src = t.in + b * t.in_b + n * t.in_n;
    __nv_bfloat16 *dst = t.out + entry * t.out_b + row * t.out_n;

    if constexpr (kLayout == kHalfVec || kLayout == kInterVec) {
        constexpr int kFreqs = kLayout == kHalfVec ? 8 : 4;
        float c[8], s[8];
        auto sines = [&]() {  // while the first heads' loads are in flight (2048 tokens, 32 + 8 heads: 9.1 to 10.2 us, now 8.4)
            if (turn)
#pragma unroll
                for (int i = 0; i < kFreqs; ++i) sin_cos(turns[item * kFreqs + i], pos_of(item * kFreqs + i), p.sign, p.scale, c[i], s[i]);
        };
        if (kLayout == kHalfVec && item < p.rot_items) {
            src += item * 8;
            dst += item * 8;
            const int half = p.r / 2;
            for (int h = h0; h < h1; h += kBatch) {
                uint4 x[kBatch], y[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (h + i < h1) {
                        const __nv_bfloat16 *q = src + (h + i) * t.in_h;
                        x[i] = __ldcs(reinterpret_cast<const uint4 *>(q));
                        y[i] = __ldcs(reinterpret_cast<const uint4 *>(q + half));
                    }
                if (h == h0) sines();
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (h + i < h1) {
                        if (turn) turn_half(x[i], y[i], c, s);
                        __nv_bfloat16 *q = dst + (h + i) * t.out_h;
                        *reinterpret_cast<uint4 *>(q) = x[i];
                        *reinterpret_cast<uint4 *>(q + half) = y[i];
                    }
            }
        } else {
            const int col = kLayout == kHalfVec ? p.r + (item - p.rot_items) * 8 : item * 8;
            src += col;
            dst += col;
            for (int h = h0; h < h1; h += kBatch) {
                uint4 x[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (h + i < h1) x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + (h + i) * t.in_h));
                if (h == h0 && kLayout == kInterVec) sines();
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (h + i < h1) {
                        if (kLayout == kInterVec && turn) turn_inter(x[i], c, s);
                        *reinterpret_cast<uint4 *>(dst + (h + i) * t.out_h) = x[i];
                    }
            }
        }
    } else {
        // One pair an item; items past the rotated ones are neighbouring columns.
        const bool split = kLayout == kHalfPair && item < p.rot_items;
        const int cx = split ? item : 2 * item, cy = split ? item + p.r / 2 : 2 * item + 1;
        float c = 1.f, s = 0.f;
        if (turn) sin_cos(turns[item], pos_of(item), p.sign, p.scale, c, s);
        for (int h = h0; h < h1; ++h) {
            const __nv_bfloat16 *q = src + h * t.in_h;
            __nv_bfloat16 x = q[cx], y = q[cy];
            if (turn) {
                const float fx = __bfloat162float(x), fy = __bfloat162float(y);
                x = __float2bfloat16_rn(fx * c - fy * s);
                y = __float2bfloat16_rn(fy * c + fx * s);
            }
            __nv_bfloat16 *w = dst + h * t.out_h;
            w[cx] = x;
            w[cy] = y;
        }
    }
}

template <bool kAppend, bool kAxes>
auto kernel_of(int layout) {
    switch (layout) {
        case kHalfVec: return rope_kernel<kHalfVec, kAppend, kAxes>;
        case kInterVec: return rope_kernel<kInterVec, kAppend, kAxes>;
        case kHalfPair: return rope_kernel<kHalfPair, kAppend, kAxes>;
        default: return rope_kernel<kInterPair, kAppend, kAxes>;
    }
}

}  // namespace rope

int rope_launch(const RopeLaunch &a, cudaStream_t stream) {
    using namespace rope;
    Params p = {};
    const int half = a.rotary_dim / 2;
    const bool vec = a.interleaved ? a.rotary_dim % 8 == 0 : half % 8 == 0;
    const int layout = a.interleaved ? (vec ? kInterVec : kInterPair) : (vec ? kHalfVec : kHalfPair);
    switch (layout) {
        case kHalfVec: p.rot_items = half / 8; p.items = p.rot_items + (a.d - a.rotary_dim) / 8; break;
        case kInterVec: p.rot_items = a.rotary_dim / 8; p.items = a.d / 8; break;
        default: p.rot_items = half; p.items = a.d / 2;
    }
    p.inv_freq = a.inv_freq;
    p.pos = a.pos;
    p.pos_stride = a.pos_stride;
    p.lens = a.lens;
    p.new_lens = a.new_lens;
    p.lens_out = a.lens_out;
    p.cache_pos = a.cache_pos;
    p.weights = a.weights;
    p.tokens = (long long)a.B * a.N;
    p.N = a.N;
    p.r = a.rotary_dim;
    p.max_seqlen = a.max_seqlen;
    p.scale = a.out_scale;
    p.sign = a.inverse ? -1.f : 1.f;
    p.axes = a.axes;
    p.table = a.table;
    p.axis_stride = a.axis_stride;
    p.num_axes = a.num_axes;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.page_shift = a.page_shift;
    const long long gx = (p.tokens * p.items + kThreads - 1) / kThreads;
    // Heads per thread: as many as share the sines while the grid still has two
    // blocks per SM; a short call takes one head a thread.  In us, one head and
    // eight: 64 tokens of 8 + 2 heads 3.4 and 4.1; 128 x 1 token of 64 + 8 heads 4.4
    // and 4.8; 2048 tokens of 32 + 8 heads 16.4 and 8.9.
    int per = kMaxHeads;
    auto grid_y = [&](int c) {
        long long y = 0;
        for (const auto &t : a.t) y += (t.heads + c - 1) / c;
        return y;
    };
    while (per > 1 && gx * grid_y(per) < 2LL * a.num_sms && grid_y(per / 2) <= 65535) per /= 2;
    p.heads_per_chunk = per;
    for (int i = 0; i < 3; ++i) {
        p.t[i] = a.t[i];
        p.chunks[i] = (a.t[i].heads + per - 1) / per;
    }
    const long long gy = grid_y(per);
    if (gx > 0x7fffffffLL || gy > 65535) return ATTN_ERR_ARG;
    void (*kernel)(Params) = a.num_axes > 0 ? (a.append ? kernel_of<true, true>(layout) : kernel_of<false, true>(layout))
                                            : (a.append ? kernel_of<true, false>(layout) : kernel_of<false, false>(layout));
    kernel<<<dim3(unsigned(gx), unsigned(gy)), kThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : note_cuda_error(e, "rope_kernel launch");
}

}  // namespace attn
