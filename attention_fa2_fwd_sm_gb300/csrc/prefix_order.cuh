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
    long long total;  // key blocks over all rows of the order
};

// One piece of work: key blocks [j0, j0 + n) of unit m of KV head g.
struct PrefixSegment {
    int g, m, j0, n, slot;
};

ATTN_HD int prefix_row(const PrefixOrder &o, int g, int m) { return o.lockstep ? g : g * o.mt + m; }

// Shares that touch row `row` of the order: the first one and their number.
ATTN_HD int prefix_first(const PrefixOrder &o, int row) { return int((long long)row * o.nblk / o.per); }
ATTN_HD int prefix_parts(const PrefixOrder &o, int row) {
    return int((((long long)row + 1) * o.nblk - 1) / o.per) - prefix_first(o, row) + 1;
}

// First key block of CTA `cta`'s i-th segment in the order's linear space, or -1.
ATTN_HD long long prefix_start(const PrefixOrder &o, int cta, int i) {
    const long long lo = (long long)(o.lockstep ? cta / o.mt : cta) * o.per;
    const long long hi = lo + o.per < o.total ? lo + o.per : o.total;
    const long long u = i == 0 ? lo : (lo / o.nblk + i) * o.nblk;
    return u < hi ? u : -1;
}

ATTN_HD PrefixSegment prefix_segment(const PrefixOrder &o, int cta, long long u) {
    const int share = o.lockstep ? cta / o.mt : cta;
    const int row = int(u / o.nblk);
    PrefixSegment s;
    s.m = o.lockstep ? cta % o.mt : row % o.mt;
    s.g = o.lockstep ? row : row / o.mt;
    s.j0 = int(u - (long long)row * o.nblk);
    const long long end = (long long)(share + 1) * o.per;
    const long long left = (end < o.total ? end : o.total) - u;
    s.n = left < o.nblk - s.j0 ? int(left) : o.nblk - s.j0;
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
    o->total = (long long)Hkv * o->nblk * (o->lockstep ? 1 : o->mt);
    if (o->total >= (1LL << 31)) return false;
    o->per = int((o->total + shares - 1) / shares);
    const int used = int((o->total + o->per - 1) / o->per);
    o->grid = used * (o->lockstep ? o->mt : 1);
    o->slots = 0;
    for (int row = 0; row < Hkv * (o->lockstep ? 1 : o->mt); ++row) {
        const int n = prefix_parts(*o, row);
        if (n > o->slots) o->slots = n;
    }
    return true;
}

}  // namespace attn
