// prefill_work.cuh -- a work item of the prompt attention: which rows, and the steps of 128
// keys that each of its two tiles takes.  Plain arithmetic, for the kernel and for a host test.
#pragma once

#if defined(__CUDACC__)
#define FATHOM_WORK_HD __host__ __device__ __forceinline__
#else
#define FATHOM_WORK_HD inline
#endif

namespace fathom {

constexpr int kRows = 128;          // rows of a tile
constexpr int kKeys = 128;          // keys per step

// A work item: 256 rows of a sequence and what they see.
struct alignas(16) Work {
    int group;      // of gp query heads
    int q0, lq;     // the sequence's first query row, its query tokens
    int k0, lk;     // its first key row, its key tokens
    int off;        // query token t sees keys j <= t + off
    int t0;         // first token; tile w starts at t0 + (w ^ flip) * (128 / gp)
    int nt0, nt1;   // steps of 128 keys of the two tiles
    int steps;      // the larger; -1: no more work
    int from;       // keys of the sequence before k0 (shares of a cluster: those of other CTAs)
    int flip;       // rows for one tile only: whether tile 1 takes them
    int half;       // bit w: tile w's last step has 64 keys or fewer and is worked on as half a step
    int again;      // worked on a second time, values that are not finite counting as 0
};

FATHOM_WORK_HD int work_min(int a, int b) { return a < b ? a : b; }
FATHOM_WORK_HD int work_max(int a, int b) { return a > b ? a : b; }

// Keys that some row of tile w sees; `tw` tokens per tile.
FATHOM_WORK_HD int work_keys(const Work &g, int tw, int w) {
    const int start = g.t0 + (w ^ g.flip) * tw, last = work_min(start + tw, g.lq) - 1;
    return start <= last ? work_max(work_min(g.lk, last + g.off + 1), 0) : 0;
}

// The steps, of an item whose q0 .. t0 and flip are set.
FATHOM_WORK_HD void work_steps(Work &g, int tw) {
    const int keys0 = work_keys(g, tw, 0), keys1 = work_keys(g, tw, 1);
    g.nt0 = (keys0 + kKeys - 1) / kKeys;
    g.nt1 = (keys1 + kKeys - 1) / kKeys;
    g.half = (keys0 > 0 && (keys0 - 1) % kKeys < kKeys / 2 ? 1 : 0) | (keys1 > 0 && (keys1 - 1) % kKeys < kKeys / 2 ? 2 : 0);
    g.steps = work_max(g.nt0, g.nt1);
}

// The share of CTA `rank` of `split` in the steps, its keys counted from the first of them.
FATHOM_WORK_HD void work_share(Work &g, int rank, int split) {
    const int from = g.steps * rank / split, to = g.steps * (rank + 1) / split;
    // a tile's last step is here or it is not; a flag without it would be a step that nobody computes
    if (g.nt0 <= from || g.nt0 > to) g.half &= ~1;
    if (g.nt1 <= from || g.nt1 > to) g.half &= ~2;
    g.nt0 = work_min(work_max(g.nt0 - from, 0), to - from);
    g.nt1 = work_min(work_max(g.nt1 - from, 0), to - from);
    g.steps = work_max(g.nt0, g.nt1);
    g.from = from * kKeys;
    g.k0 += from * kKeys;
    g.lk -= from * kKeys;
    g.off -= from * kKeys;
}

// The item's first key that some query of it does not see.
FATHOM_WORK_HD int work_first_unseen(const Work &g) { return work_max(g.t0 + g.off + 1, 0); }

// The first step that reads value rows which some query of it does not see.
FATHOM_WORK_HD int work_first_edge(const Work &g) { return work_first_unseen(g) / kKeys; }

// Those rows of such a step (j * 128 and on): r0 .. r1 - 1 of the sequence, and r1 .. r2 - 1 behind its end.
struct EdgeRows {
    int r0, r1, r2;
};
FATHOM_WORK_HD EdgeRows work_edge(const Work &g, int j) {
    const bool half0 = j >= g.nt0 || (j + 1 == g.nt0 && (g.half & 1));
    const bool half1 = j >= g.nt1 || (j + 1 == g.nt1 && (g.half & 2));
    EdgeRows e;
    e.r2 = half0 && half1 ? kKeys / 2 : kKeys;
    e.r0 = work_min(work_max(work_first_unseen(g) - j * kKeys, 0), e.r2);
    e.r1 = work_min(work_max(g.lk - j * kKeys, e.r0), e.r2);
    return e;
}

// The cluster barriers that a row warp passes, `left` of them still to come.  A warp whose wait for its
// item ran out passes the rest all the same: the cluster's other warps wait for it there without a limit.
struct Meetings {
    int left;
    template <typename Sync>
    FATHOM_WORK_HD void meet(Sync sync) {
        sync();
        --left;
    }
    template <typename Sync>
    FATHOM_WORK_HD void rest(Sync sync) {
        while (left > 0) meet(sync);
    }
};

}  // namespace fathom
