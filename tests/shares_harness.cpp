// Host build of the arithmetic that deals tiles out to CTAs (bit_plane_kv_gb300/csrc/share_rule.cuh),
// exported so that a CPU test can go over whole batches.
#include "share_rule.cuh"

using namespace fathom;

extern "C" int own_rule(int units, int ctas) { return share_own(units, ctas); }

// Units with CTAs of their own: out[5 n ..] = CTA, sequence, head, first tile, tiles; how many.  -1: more CTAs than there are.
extern "C" int own_shares(int seqs, int heads, int ctas, const int *tiles, int *out) {
    int all = 0, cta = 0;
    for (int s = 0; s < seqs; ++s) all += tiles[s];
    const int limit = share_limit(all, heads, seqs * heads, ctas);
    for (int s = 0; s < seqs; ++s) {
        const int parts = share_parts(tiles[s], limit);
        for (int i = 0; i < parts * heads; ++i, ++cta) {
            if (cta >= ctas) return -1;
            const OwnShare z = share_of(i, parts, tiles[s]);
            const int f[] = {cta, s, z.head, z.first, z.count};
            for (int k = 0; k < 5; ++k) out[5 * cta + k] = f[k];
            if (z.j != i % parts) return -1;
        }
    }
    return cta;
}

// Equal shares of W tiles: first tiles of CTAs 0 .. NC, and whether every tile's owner is the CTA that has it.
extern "C" int equal_shares(long long W, int NC, long long *start, const long long *check, int n) {
    for (int c = 0; c <= NC; ++c) start[c] = share_start(c, W, NC);
    for (int i = 0; i < n; ++i) {
        const int c = share_owner(check[i], W, NC);
        if (c < 0 || c >= NC || start[c] > check[i] || start[c + 1] <= check[i]) return 0;
    }
    return 1;
}

extern "C" int tile_owner(long long w, long long W, int NC) { return share_owner(w, W, NC); }
