// share_rule.cuh -- which tiles a CTA takes (shares.cuh).  Plain arithmetic, for the kernels
// and for a host test.
//
// The tiles of all units, in the order (sequence, head, tile), are dealt out to the CTAs
// in contiguous shares that differ by one tile at most: CTA c of NC takes tiles c W / NC
// to (c + 1) W / NC of W.  Where units are few (eight CTAs each or more), every unit gets
// CTAs of its own instead: no CTA then ends one unit and begins another, or joins two (seven
// sequences of up to 9001 tokens, 21 units: 21 -> 15 us).  One CTA per unit pays for the
// roundings; all tiles over the others, rounded up, are the most that a share has, so no share
// is longer than 8/7 of the mean, rounded up (56 sequences of 131072 tokens and 20 of 29800:
// 290 us with the units' parts rounded down instead, 230 so).
#pragma once

#if defined(__CUDACC__)
#define FATHOM_SHARE_HD __host__ __device__ __forceinline__
#else
#define FATHOM_SHARE_HD inline
#endif

namespace fathom {

// Division of numbers that mostly fit 32 bits.
FATHOM_SHARE_HD long long div_small(long long x, long long y) {
    return (unsigned long long)(x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}

// CTA c's first tile of W, and the CTA that has tile w.
FATHOM_SHARE_HD long long share_start(long long c, long long W, long long NC) { return div_small(c * W, NC); }
FATHOM_SHARE_HD int share_owner(long long w, long long W, long long NC) { return (int)div_small((w + 1) * NC - 1, W); }

// Units with CTAs of their own: whether they have them, the most tiles of a share (all: of one head of every
// sequence, below 2^28), and the CTAs of a unit.
FATHOM_SHARE_HD bool share_own(int units, int ctas) { return units * 8 <= ctas; }
FATHOM_SHARE_HD int share_limit(int all, int heads, int units, int ctas) {
    const unsigned others = ctas - units, sum = (unsigned)all * heads;
    return sum ? (int)((sum + others - 1) / others) : 1;
}
FATHOM_SHARE_HD int share_parts(int tiles, int limit) { return (int)((unsigned)(tiles + limit - 1) / (unsigned)limit); }

// CTA i of a sequence's: head, tiles first .. first + count - 1, and its place j among the unit's `parts`.
struct OwnShare {
    int head, first, count, j;
};
FATHOM_SHARE_HD OwnShare share_of(unsigned i, unsigned parts, unsigned tiles) {   // j tiles below 2^32: 608 2^21
    OwnShare z;
    const unsigned j = i % parts, first = j * tiles / parts;
    z.head = (int)(i / parts);
    z.first = (int)first;
    z.count = (int)((j + 1) * tiles / parts - first);
    z.j = (int)j;
    return z;
}

}  // namespace fathom
