// prefix_order.cuh -- how the prefix phase of the shared-prefix decode is cut
// into work: which CTA computes which key blocks for which query rows.  Pure
// arithmetic, the same on the host and inside the kernels.
//
// The B * G query rows that read KV head g are packed into 128-row MMA tiles of
// `rb` whole batch entries each (rb * G <= 128), two tiles a unit, `mt` units a
// head; each has to visit all nblk key blocks of the prefix.  Shares of key
// blocks go to as many CTAs as there are SMs, whatever the head count:
//   lockstep  every group of mt CTAs takes one share of the (head, key block)
//             space, a CTA per unit, so the CTAs that run side by side read the
//             same key blocks at the same time and all but one find them in L2;
//   linear    the share is cut from the (head, unit, key block) space.
// Lockstep unless it would leave more than a tenth of the SMs idle (mt near the
// SM count).  A row below is a head (lockstep) or a unit of a head (linear).
//
// The prefix is bound by the tensor cores, the sequences' own keys by HBM, so
// the two run at the same time on different SMs: the own keys' kernel, ahead on
// the stream, holds `own` SMs (prefix_own_sms), the first `early` shares start at
// once on the others, and the `late` ones wait for its SMs.  So that all end
// together, a late share is shorter by what the own keys take, tau key blocks'
// worth of time, estimated from their number T:
//     early a + late b = total,  b = a - tau  (b = 0 where a <= tau).
// The shares depend on the lengths alone, so results do not depend on timing.
// Where nothing is left for the late ones and it makes no share much longer, every
// row gets a whole number of shares (`aligned` of them): a share that goes on in
// the next row pays for a second start and end (32 x (8K + 256 .. 512) keys 36.8 us,
// 41.5 without).
//
// A CTA's share is one segment per row that it touches; each segment writes one
// partial per query row, numbered share + row (both go up along the shares, one
// of them at every cut): the numbers are distinct, a row's consecutive.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

constexpr int kPrefixTileRows = 128;
constexpr int kPrefixBlock = 128;  // keys

struct PrefixOrder {
    int nblk;      // key blocks of the prefix
    int rb, mt;    // batch entries per tile; units (two tiles) per KV head
    int lockstep;
    int early, late;  // shares
    int unit_rows;    // query rows of a unit, its last tile full
    int id_rows;      // query rows of a partial number
    int ids;          // partial numbers
    int rows;         // rows of the order
    unsigned total;   // key blocks over all of them; below 2^30, as every product below
    unsigned own_cost;  // key blocks' worth of time of one own key and KV head, in 2^-32
};

// Lengths of the early and the late shares; aligned: shares per row, or 0.
struct PrefixShares {
    unsigned a, b, aligned;
};

// One piece of work: key blocks [j0, j0 + n) of unit m of KV head g.
struct PrefixSegment {
    int g, m, j0, n, row;
};

ATTN_HD int prefix_grid(const PrefixOrder &o) { return (o.early + o.late) * (o.lockstep ? o.mt : 1); }
ATTN_HD int prefix_share(const PrefixOrder &o, int cta) { return o.lockstep ? cta / o.mt : cta; }
ATTN_HD int prefix_row(const PrefixOrder &o, int g, int m) { return o.lockstep ? g : g * o.mt + m; }

// T: own keys over all KV heads.
ATTN_HD PrefixShares prefix_shares(const PrefixOrder &o, long long T) {
    const unsigned e = unsigned(o.early), l = unsigned(o.late);
    // (no memory holds 2^38 keys, and own_cost is below 2^26)
    const unsigned long long wide = (unsigned long long)(T < (1LL << 38) ? T : (1LL << 38)) * o.own_cost >> 32;
    const unsigned tau = wide < (1u << 30) ? unsigned(wide) : (1u << 30);
    PrefixShares s;
    s.a = (o.total + e - 1) / e;
    s.b = 0;
    if (l > 0 && s.a > tau) {
        s.a = unsigned((o.total + (unsigned long long)l * tau + e + l - 1) / (e + l));
        s.b = e * s.a >= o.total ? 0 : (o.total - e * s.a + l - 1) / l;
    }
    s.aligned = 0;
    const unsigned rows = unsigned(o.rows), nblk = unsigned(o.nblk);
    if (s.b == 0 && e >= rows) {
        const unsigned a = (nblk + e / rows - 1) / (e / rows);
        if (a <= s.a + s.a / 8) {
            s.a = a;
            s.aligned = (nblk + a - 1) / a;
        }
    }
    return s;
}

// First key block of a share in the order's space; a share may be empty.
ATTN_HD unsigned prefix_begin(const PrefixOrder &o, const PrefixShares &s, int share) {
    const unsigned x = unsigned(share), e = unsigned(o.early);
    if (s.aligned) {
        const unsigned row = x / s.aligned, in = (x - row * s.aligned) * s.a;
        return row < unsigned(o.rows) ? row * unsigned(o.nblk) + in : o.total;
    }
    const unsigned at = x <= e ? x * s.a : e * s.a + (x - e) * s.b;
    return at < o.total ? at : o.total;
}
// The share that holds key block x.
ATTN_HD int prefix_holder(const PrefixOrder &o, const PrefixShares &s, unsigned x) {
    if (s.aligned) return int(x / unsigned(o.nblk) * s.aligned + x % unsigned(o.nblk) / s.a);
    const unsigned early = unsigned(o.early) * s.a;
    return int(x < early ? x / s.a : unsigned(o.early) + (x - early) / s.b);
}

// First key block of the i-th segment of a share [lo, hi), or -1.
ATTN_HD int prefix_start(const PrefixOrder &o, unsigned lo, unsigned hi, int i) {
    const unsigned u = i == 0 ? lo : (lo / unsigned(o.nblk) + i) * unsigned(o.nblk);
    return u < hi ? int(u) : -1;
}

ATTN_HD PrefixSegment prefix_segment(const PrefixOrder &o, unsigned hi, int cta, int u) {
    PrefixSegment s;
    s.row = int(unsigned(u) / unsigned(o.nblk));
    s.m = o.lockstep ? cta % o.mt : s.row % o.mt;
    s.g = o.lockstep ? s.row : s.row / o.mt;
    s.j0 = u - s.row * o.nblk;
    const int left = int(hi - unsigned(u));
    s.n = left < o.nblk - s.j0 ? left : o.nblk - s.j0;
    return s;
}

// Measured rates.  The own keys' kernel draws this many bytes a microsecond on
// `own` SMs (segments of 768 keys; a third more in long ones), up to what HBM gives.
constexpr double kHbmRate = 6.0e6;
inline double prefix_own_rate(int d, int G, int own) {
    const double sm = (d == 128 ? (G > 8 ? 52.0 : 90.0) : (G > 8 ? 38.0 : 75.0)) * 1e3;
    return own * sm < kHbmRate ? own * sm : kHbmRate;
}
// A unit's key block takes this many microseconds, with two tiles and with one;
// twice that beside own keys that take all of HBM's rate.
inline double prefix_block_us(int d, bool two_tiles, double own_rate) {
    const double us = d == 128 ? (two_tiles ? 1.55 : 1.2) : (two_tiles ? 1.37 : 1.0);
    return own_rate < kHbmRate ? us : 2 * us;
}

// SMs for the own keys' kernel beside a prefix, `most` at most: in proportion to
// what the two have to do if the caches are three quarters full, so that in the
// usual case no share has to wait, and leaving whole groups of mt.  128 x (32K
// shared + 512 .. 1024 own) keys: 24 SMs 191 us, 32 153, 40 138, 48 143, 64 147, 104 172
// (with the shares' balance; the two phases one after the other 176); 32 x (8K + 256
// .. 512): 24 SMs 44, 32 37, 40 36.5, 48 34.5, 56 37, 76 45, 36.8 with the choice made
// here; 64 x (8K + 256 .. 512) 69, 56, 49, 46, 46, 56, and 50.7.
inline int prefix_own_sms(int B, int G, int Hkv, int P, int d, int max_seqlen, int most, int num_sms) {
    const int rb = kPrefixTileRows / G, tiles = (B + rb - 1) / rb, mt = (tiles + 1) / 2;
    const double own = 0.75 * B * Hkv * (double)max_seqlen * 4 * d / prefix_own_rate(d, G, 1);
    int left = num_sms;  // SMs that the prefix starts on
    for (int i = 0; i < 2; ++i) {  // at first as if the own keys left bandwidth over
        const double prefix = (double)Hkv * mt * ((P + kPrefixBlock - 1) / kPrefixBlock) *
                              prefix_block_us(d, tiles > 1, prefix_own_rate(d, G, num_sms - left));
        left = int(num_sms * (prefix / (own + prefix)) + 0.5);
    }
    left = mt < num_sms ? (left + mt / 2) / mt * mt : left;
    if (left < (mt < num_sms ? mt : 1)) left = mt < num_sms ? mt : 1;
    int sms = num_sms - left;
    if (sms < 1) sms = 1;
    return sms < most ? sms : most;
}

// `own`: SMs that the own keys' kernel holds (0: none).  False when the problem
// is outside the order's 32-bit counters.
inline bool prefix_order(PrefixOrder *o, int B, int G, int Hkv, int P, int d, int own, int num_sms) {
    o->nblk = (P + kPrefixBlock - 1) / kPrefixBlock;
    o->rb = kPrefixTileRows / G;
    const int tiles = (B + o->rb - 1) / o->rb;
    o->mt = (tiles + 1) / 2;
    const int groups = num_sms / o->mt;
    o->lockstep = 10LL * groups * o->mt >= 9LL * num_sms;
    const int shares = o->lockstep ? groups : num_sms;
    const long long rows = (long long)Hkv * (o->lockstep ? 1 : o->mt), total = rows * o->nblk;
    if (total >= (1LL << 30)) return false;
    o->total = unsigned(total);
    o->rows = int(rows);
    o->early = o->lockstep ? (num_sms - own) / o->mt : num_sms - own;
    if (o->early < 1) o->early = 1;
    if (o->early > total) o->early = int(total);
    o->late = total > o->early && shares > o->early ? shares - o->early : 0;
    o->unit_rows = 2 * o->rb * G;
    o->id_rows = o->unit_rows * (o->lockstep ? o->mt : 1);
    o->ids = o->early + o->late + o->rows;
    const double rate = prefix_own_rate(d, G, own);
    o->own_cost = own > 0 ? unsigned(4.0 * d / rate / prefix_block_us(d, tiles > 1, rate) * 4294967296.0) : 0u;
    return true;
}

}  // namespace attn
