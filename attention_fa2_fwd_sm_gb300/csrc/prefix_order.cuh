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
    // Key blocks' worth of time that the own keys' kernel takes for one key of one KV
    // head, in 2^-32, and that it takes whatever the number of keys.
    unsigned own_key, own_rows;
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

// `keys`: own keys over all KV heads.
ATTN_HD PrefixShares prefix_shares(const PrefixOrder &o, long long keys) {
    const unsigned e = unsigned(o.early), l = unsigned(o.late);
    // (no memory holds 2^38 keys, and own_key is below 2^26)
    unsigned long long wide = (unsigned long long)(keys < (1LL << 38) ? keys : (1LL << 38)) * o.own_key >> 32;
    if (keys > 0) wide += o.own_rows;
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

// Groups of an own keys' CTA, which have a share each.
inline int own_groups(int G) { return G > 8 ? 2 : 3; }

// Measured times of the own keys' kernel beside the prefix's: a group of a CTA
// takes `row` microseconds to start and end a segment and `key` for each of its
// keys, so 3 KV heads of 768 keys at once come to 90 GB/s an SM (d = 128, up to
// 8 heads a KV head), 3 of 12 keys to 7 GB/s.  All of its SMs together draw at
// most what HBM gives.
constexpr double kHbmRate = 6.0e6;  // bytes a microsecond
struct OwnTimes {
    double row, key;
};
inline OwnTimes prefix_own_times(int d, int G) {
    if (d == 128) return G > 8 ? OwnTimes{3.6, 0.0150} : OwnTimes{2.5, 0.0138};
    return G > 8 ? OwnTimes{1.9, 0.0110} : OwnTimes{1.55, 0.00825};
}
// Microseconds that `held` rows with `keys` keys in all keep one SM busy.
inline double prefix_own_us(int d, int G, double held, double keys) {
    const OwnTimes t = prefix_own_times(d, G);
    return (held * t.row + keys * t.key) / own_groups(G);
}
// A unit's key block takes this many microseconds, with two tiles and with one;
// twice that beside own keys that take all of HBM's rate.
inline double prefix_block_us(int d, bool two_tiles, double own_rate) {
    const double us = d == 128 ? (two_tiles ? 1.55 : 1.2) : (two_tiles ? 1.37 : 1.0);
    return own_rate < kHbmRate ? us : 2 * us;
}

// A late share starts when the own keys are done, and the microseconds until its
// first product overlap nothing: without them 16 x (32K + 1K .. 2K) keys give late
// shares of one block (58.5 us, 53.5).
constexpr double kLateStart = 2.0;

// Units in lockstep: whether that leaves at most a tenth of the SMs idle.
ATTN_HD bool prefix_lockstep(int mt, int num_sms) { return 10LL * (num_sms / mt) * mt >= 9LL * num_sms; }

// SMs for the own keys' kernel beside a prefix, `most` at most: in proportion to
// what the two have to do if the caches are three quarters full, and rounded up,
// in lockstep until the prefix starts on whole groups of mt: with too few of them
// the late shares wait for the own keys, with too many they just start sooner.
// In us, by SMs: 128 x (32K shared + 512 .. 1024 own) keys: 24 193, 32 154, 40 (the
// choice) 138, 48 148, 64 150, 104 171, and 176 with one phase behind the other;
// 32 x (8K + 256 .. 512): 24 43, 32 35, 48 34, 64 37, 70 (the choice) 36, 76 42. Short
// own lengths, where a row's start and end are all of its time: 128 x (32K + 8 .. 16)
// 1 SM 958, 4 307, 12 (the choice) 148, 32 118; 32 x (8K + 8 .. 16) 4 84, 41 24.7;
// 1216 x (8K + 32 .. 64) 1 SM 9350, 40 440, 76 (the choice) 354.
inline int prefix_own_sms(int B, int G, int Hkv, int P, int d, int max_seqlen, int most, int num_sms) {
    const int rb = kPrefixTileRows / G, tiles = (B + rb - 1) / rb, mt = (tiles + 1) / 2;
    const double held = (double)B * Hkv, keys = 0.75 * held * max_seqlen;
    const double own = prefix_own_us(d, G, held, keys);
    int left = num_sms;  // SMs that the prefix starts on
    for (int i = 0; i < 2; ++i) {  // at first as if the own keys left bandwidth over
        const double rate = keys * 4 * d * (num_sms - left) / own;
        const double prefix = (double)Hkv * mt * ((P + kPrefixBlock - 1) / kPrefixBlock) * prefix_block_us(d, tiles > 1, rate);
        left = int(num_sms * (prefix / (own + prefix)));
    }
    const int whole = prefix_lockstep(mt, num_sms) ? mt : 1;
    left = left / whole * whole;
    if (left < whole) left = whole;
    int sms = num_sms - left;
    if (sms < 1) sms = 1;
    return sms < most ? sms : most;
}

// `own`: SMs that the own keys' kernel holds (0: none).  False when the problem
// is outside the order's 32-bit counters.
inline bool prefix_order(PrefixOrder *o, int B, int G, int Hkv, int P, int d, int max_seqlen, int own, int num_sms) {
    o->nblk = (P + kPrefixBlock - 1) / kPrefixBlock;
    o->rb = kPrefixTileRows / G;
    const int tiles = (B + o->rb - 1) / o->rb;
    o->mt = (tiles + 1) / 2;
    const int groups = num_sms / o->mt;
    o->lockstep = prefix_lockstep(o->mt, num_sms);
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
    o->own_key = o->own_rows = 0;
    if (own > 0) {
        const double held = (double)B * Hkv, keys = 0.75 * held * max_seqlen;
        const double rate = keys * 4 * d * own / prefix_own_us(d, G, held, keys);
        const double block = prefix_block_us(d, tiles > 1, rate);
        const OwnTimes t = prefix_own_times(d, G);
        const double sms = own_groups(G) * own;
        o->own_key = unsigned((rate < kHbmRate ? t.key / sms : 4.0 * d / kHbmRate) / block * 4294967296.0);
        const double rows = ((rate < kHbmRate ? held * t.row / sms : 0.0) + kLateStart) / block;
        o->own_rows = rows < 1e9 ? unsigned(rows + 0.5) : 1000000000u;
    }
    return true;
}

}  // namespace attn
