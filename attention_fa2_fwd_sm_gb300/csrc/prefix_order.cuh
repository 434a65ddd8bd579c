// prefix_order.cuh -- how the prefix phase of the shared-prefix decode is cut
// into work: which CTA computes which key blocks for which query rows.  Pure
// arithmetic, the same on the host and inside the kernels.
//
// The B * G query rows that read KV head g are packed into 128-row MMA tiles of
// `rb` whole batch entries each (rb * G <= 128), two tiles a unit, `mt` units a
// head; each has to visit all nblk key blocks of the prefix.  Equal shares of
// key blocks go to as many CTAs as there are SMs, whatever the head count:
//   lockstep  every group of mt CTAs takes one share of the (head, key block)
//             space, a CTA per unit, so the CTAs that run side by side read the
//             same key blocks at the same time and all but one find them in L2;
//   linear    the share is cut from the (head, unit, key block) space.
// Lockstep unless it would leave more than a tenth of the SMs idle (mt near the
// SM count).  A CTA's share is one segment per head (or unit) that it touches;
// each segment writes one partial per query row.  A row's partials are numbered
// by CTA: slot 0 is the first CTA that touches it.
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
    int per;       // key blocks of a CTA's share
    int grid, slots;
    unsigned total;  // key blocks over all rows of the order; below 2^31, as every product below
};

// One piece of work: key blocks [j0, j0 + n) of unit m of KV head g.
struct PrefixSegment {
    int g, m, j0, n, slot;
};

ATTN_HD int prefix_row(const PrefixOrder &o, int g, int m) { return o.lockstep ? g : g * o.mt + m; }

// Shares that touch row `row` of the order: the first one and their number.
ATTN_HD int prefix_first(const PrefixOrder &o, int row) { return int(unsigned(row) * unsigned(o.nblk) / unsigned(o.per)); }
ATTN_HD int prefix_parts(const PrefixOrder &o, int row) {
    return int((unsigned(row + 1) * unsigned(o.nblk) - 1) / unsigned(o.per)) - prefix_first(o, row) + 1;
}

// First key block of CTA `cta`'s i-th segment in the order's linear space, or -1.
ATTN_HD int prefix_start(const PrefixOrder &o, int cta, int i) {
    const unsigned lo = unsigned(o.lockstep ? cta / o.mt : cta) * unsigned(o.per);
    const unsigned hi = lo + o.per < o.total ? lo + o.per : o.total;
    const unsigned u = i == 0 ? lo : (lo / unsigned(o.nblk) + i) * unsigned(o.nblk);
    return u < hi ? int(u) : -1;
}

ATTN_HD PrefixSegment prefix_segment(const PrefixOrder &o, int cta, int u) {
    const int share = o.lockstep ? cta / o.mt : cta;
    const int row = int(unsigned(u) / unsigned(o.nblk));
    PrefixSegment s;
    s.m = o.lockstep ? cta % o.mt : row % o.mt;
    s.g = o.lockstep ? row : row / o.mt;
    s.j0 = u - row * o.nblk;
    const unsigned end = unsigned(share + 1) * unsigned(o.per);
    const int left = int((end < o.total ? end : o.total) - unsigned(u));
    s.n = left < o.nblk - s.j0 ? left : o.nblk - s.j0;
    s.slot = share - prefix_first(o, row);
    return s;
}

// False when the problem is outside the order's 32-bit counters.
inline bool prefix_order(PrefixOrder *o, int B, int G, int Hkv, int P, int num_sms) {
    o->nblk = (P + kPrefixBlock - 1) / kPrefixBlock;
    o->rb = kPrefixTileRows / G;
    const int tiles = (B + o->rb - 1) / o->rb;
    o->mt = (tiles + 1) / 2;
    const int groups = num_sms / o->mt;
    o->lockstep = 10LL * groups * o->mt >= 9LL * num_sms;
    const int shares = o->lockstep ? groups : num_sms;
    const long long total = (long long)Hkv * o->nblk * (o->lockstep ? 1 : o->mt);
    if (total >= (1LL << 30)) return false;
    o->total = unsigned(total);
    o->per = int((total + shares - 1) / shares);
    const int used = int((total + o->per - 1) / o->per);
    o->grid = used * (o->lockstep ? o->mt : 1);
    o->slots = 0;
    for (int row = 0; row < Hkv * (o->lockstep ? 1 : o->mt); ++row) {
        const int n = prefix_parts(*o, row);
        if (n > o->slots) o->slots = n;
    }
    return true;
}

}  // namespace attn
