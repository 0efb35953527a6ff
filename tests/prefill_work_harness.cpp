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

// The steps of that share that read value rows which some query does not see: out[4 n ..] = step, r0, r1, r2; how many.
extern "C" int prefill_edges(int lq, int lk, int tw, int t0, int flip, int rank, int split, int *out) {
    fathom::Work g = {};
    g.lq = lq;
    g.lk = lk;
    g.off = lk - lq;
    g.t0 = t0;
    g.flip = flip;
    fathom::work_steps(g, tw);
    if (split > 1) fathom::work_share(g, rank, split);
    int n = 0;
    for (int j = fathom::work_first_edge(g); j < g.steps; ++j, ++n) {
        const fathom::EdgeRows e = fathom::work_edge(g, j);
        const int f[] = {j, e.r0, e.r1, e.r2};
        for (int i = 0; i < 4; ++i) out[4 * n + i] = f[i];
    }
    return n;
}

// Cluster barriers that a warp passes, of `meetings`, when its item took it past `met` of them.
extern "C" int prefill_meetings(int meetings, int met) {
    int passed = 0;
    auto sync = [&] { ++passed; };
    fathom::Meetings cluster{meetings};
    for (int i = 0; i < met; ++i) cluster.meet(sync);
    cluster.rest(sync);
    return passed;
}
