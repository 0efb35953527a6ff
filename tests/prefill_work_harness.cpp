// Host build of the prompt attention's work arithmetic (bit_plane_kv_gb300/csrc/prefill_work.cuh),
// exported so that a CPU test can go over the shares of an item.
#include "prefill_work.cuh"

// out: nt0, nt1, steps, half, from, k0, lk, off of share `rank` of `split` of the item at token t0
extern "C" void prefill_work(int lq, int lk, int tw, int t0, int flip, int rank, int split, int *out) {
    fathom::Work g = {};
    g.lq = lq;
    g.lk = lk;
    g.off = lk - lq;
    g.t0 = t0;
    g.flip = flip;
    fathom::work_steps(g, tw);
    if (split > 1) fathom::work_share(g, rank, split);
    const int f[] = {g.nt0, g.nt1, g.steps, g.half, g.from, g.k0, g.lk, g.off};
    for (int i = 0; i < 8; ++i) out[i] = f[i];
}

// Cluster barriers that a row warp passes when its wait for work brings `items` items (0: it ran out at once).
extern "C" int prefill_meetings(int items, int meetings) {
    int passed = 0;
    fathom::work_items([&](fathom::Work &) { return items-- > 0; },
                       [&](const fathom::Work &, auto meet) {
                           for (int i = 0; i < meetings; ++i) meet();
                       },
                       [&] { ++passed; }, meetings);
    return passed;
}
