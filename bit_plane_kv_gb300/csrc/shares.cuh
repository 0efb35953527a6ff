// shares.cuh -- equal shares of work over sequences of unequal lengths, and the join of
// softmax states that several CTAs hold of one unit.
#pragma once

#include "blackwell.cuh"
#include "share_rule.cuh"

namespace fathom {

struct Share {
    long long W, NC, w0;      // all tiles, CTAs that have some, this CTA's first tile
    int seq, head, tile;      // where it begins
    int count;                // its tiles
    int own_first, own_last;  // the unit's CTAs where it has its own, else -1
};
template <int kWarps>
struct ShareSmem {
    long long sum[kWarps], before;
    int part;
};

// This CTA's share.  tiles_of(s): tiles of one head of sequence s.
template <int kWarps, typename Tiles>
__device__ __forceinline__ Share find_share(int seqs, int heads, Tiles tiles_of, ShareSmem<kWarps> &sm) {
    constexpr int kThreads = 32 * kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, grid = gridDim.x;
    Share z{0, 1, 0, 0, 0, 0, 0, -1, -1};
    auto split = [&](long long sum) {
        z.W = sum * heads;
        z.NC = min((long long)grid, max(1LL, z.W));
        if (cta >= z.NC) return;
        z.w0 = share_start(cta, z.W, z.NC);
        z.count = (int)(share_start(cta + 1, z.W, z.NC) - z.w0);
    };
    auto begin = [&](long long first, int tiles) {   // the sequence's first tile, its tiles
        z.head = (int)div_small(z.w0 - first, tiles);
        z.tile = (int)(z.w0 - first - (long long)z.head * tiles);
    };
    auto scan = [&](auto x) {   // inclusive sums over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const auto y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    if (seqs <= 128) {   // every warp for itself, four sequences per lane, one round of loads
        int t[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e] = 4 * lane + e < seqs ? tiles_of(4 * lane + e) : 0;
            sum += t[e];
        }
        int upto = scan(sum);
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        const bool own = share_own(seqs * heads, grid);
        int c[4];   // what is searched: tiles, or CTAs
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = t[e];
        if (own) {
            const int limit = share_limit(all, heads, seqs * heads, grid);
            sum = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[e] = share_parts(t[e], limit);
                sum += c[e];
            }
            upto = scan(sum);
        } else {
            split(all);
        }
        const long long at = own ? cta : z.w0;
        const unsigned hit = __ballot_sync(0xffffffffu, (long long)upto * heads > at);
        const int f = hit ? __ffs(hit) - 1 : 0;
        long long before = (long long)(upto - sum) * heads;
        int s = 4 * lane, mine = c[0], tiles = t[0];
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (s == 4 * lane + e && before + (long long)c[e] * heads <= at) {
                before += (long long)c[e] * heads;
                ++s;
                mine = c[e + 1];
                tiles = t[e + 1];
            }
        z.seq = __shfl_sync(0xffffffffu, s, f);
        before = __shfl_sync(0xffffffffu, before, f);
        mine = __shfl_sync(0xffffffffu, mine, f);
        tiles = __shfl_sync(0xffffffffu, tiles, f);
        if (own) {
            z.count = 0;
            if (!hit) return z;
            const OwnShare o = share_of((unsigned)(at - before), mine, tiles);
            z.head = o.head;
            z.tile = o.first;
            z.count = o.count;
            z.own_first = cta - o.j;
            z.own_last = z.own_first + mine - 1;
        } else if (z.count) {
            begin(before, tiles);
        }
        return z;
    }
    // every thread the sum of a contiguous part; the part that holds w0 is searched by every warp
    const int per = (seqs + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int s = tid * per; s < min((tid + 1) * per, seqs); ++s) mine += tiles_of(s);
    const long long upto = scan(mine);
    if (lane == 31) sm.sum[warp] = upto;
    __syncthreads();
    long long sum = 0, before = upto - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm.sum[w];
        sum += sm.sum[w];
    }
    split(sum);
    if (before * heads <= z.w0 && z.w0 < (before + mine) * heads) { sm.part = tid; sm.before = before; }
    __syncthreads();
    if (!z.count) return z;
    before = sm.before;
    for (int s0 = sm.part * per;; s0 += 32) {
        const long long x = s0 + lane < seqs ? tiles_of(s0 + lane) : 0, end = before + scan(x);
        const unsigned hit = __ballot_sync(0xffffffffu, end * heads > z.w0);
        if (hit || s0 >= seqs) {
            const int f = hit ? __ffs(hit) - 1 : 0;
            z.seq = min(s0 + f, seqs - 1);
            begin(__shfl_sync(0xffffffffu, (end - x) * heads, f), max(1, (int)__shfl_sync(0xffffffffu, x, f)));
            return z;
        }
        before = __shfl_sync(0xffffffffu, end, 31);
    }
}

// ---------------------------------------------------------------- partial states
// A unit that several CTAs hold a share of: each leaves (m, l, o[D]) per head, m its largest
// score before a factor that turns scores into powers of two, o and l relative to it, and
// takes a ticket; the last to arrive joins them, in their order, so
// that the result does not depend on the order of arrival.  Of more than 32 shares,
// groups of 16 are joined first, each by its last share and into its first one's place.
constexpr float kNoScore = -3.402823466e38f;   // where there is none yet: finite, so that a difference is a number
struct Parts {
    float *o, *ml;   // [CTA][2][G][D] and [CTA][2][G][2] = (m, l): a CTA has at most two shares to be joined
    unsigned *ticket, *group_ticket;   // zero between calls: a unit's, by its first CTA; a group's, at its first share's place
};
struct JoinSmem {
    float weight[FATHOM_MAX_G][32], m[FATHOM_MAX_G], l[FATHOM_MAX_G], f[FATHOM_MAX_G];
    int last;
};

// Called by every thread of the CTA after the CTA's state of the unit lies in its place.
// c_first, c_last: the unit's CTAs; before: whether the first of them holds tiles of an
// earlier unit too (its share of this one is then its second); scale [G]: the scores'
// factors, in shared memory.  done(e, o, m, l, scale) gets the joined sums of elements e ..
// e + 3 of the unit's [G][D].
template <int kWarps, int kD, int kHeads, typename Done>
__device__ __forceinline__ void join_parts(const Parts &parts, int G, int c_first, int c_last, bool before, const float *scale,
                                           JoinSmem &jn, Done done) {
    constexpr int kThreads = 32 * kWarps, kGroup = 16;
    constexpr int kVecs = (kHeads * kD / 4 + kThreads - 1) / kThreads;
    constexpr int kBatch = kVecs > 1 ? 8 : 16;   // loads in flight per thread and vector
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto slot_of = [&](int x) { return 2 * x + (x == c_first && before ? 1 : 0); };
    const int shares = c_last - c_first + 1;
    int x_first = c_first;   // what is joined: shares x_first, x_first + every, ...
    int every = 1, n = shares;
    unsigned *ticket = parts.ticket + c_first;   // of all units that it holds a share of, one goes on behind it
    bool final = shares <= 32;
    if (!final) {
        x_first += ((int)blockIdx.x - c_first) / kGroup * kGroup;
        n = min(kGroup, c_last - x_first + 1);
        ticket = parts.group_ticket + slot_of(x_first);
    }
    for (;;) {
        __syncthreads();
        if (tid == 0) {   // the CTA's state before its ticket, the others' after it
            unsigned before_it;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before_it) : "l"(ticket) : "memory");
            jn.last = before_it == (unsigned)(n - 1) ? 1 : 0;
        }
        __syncthreads();
        if (!jn.last) return;
        if (tid == 0) *ticket = 0u;
        if (tid < G) { jn.m[tid] = kNoScore; jn.l[tid] = 0.0f; }
        float4 acc[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int x0 = 0; x0 < n; x0 += 32) {
            const int nx = min(n - x0, 32);
            float4 v[kVecs][kBatch];
            auto fetch = [&](int x) {
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int e = 4 * (tid + k * kThreads);
#pragma unroll
                    for (int y = 0; y < kBatch; ++y)
                        if (e < G * kD && x + y < nx)
                            v[k][y] = __ldcg(reinterpret_cast<const float4 *>(
                                parts.o + (size_t)(slot_of(x_first + (x0 + x + y) * every) * G) * kD + e));
                }
            };
            float2 mls[(kHeads + kWarps - 1) / kWarps];
#pragma unroll
            for (int i = 0; i < (kHeads + kWarps - 1) / kWarps; ++i) {
                const int h = warp + i * kWarps;
                mls[i] = make_float2(kNoScore, 0.0f);
                if (lane < nx && h < G)
                    mls[i] = __ldcg(reinterpret_cast<const float2 *>(
                        parts.ml + ((size_t)slot_of(x_first + (x0 + lane) * every) * G + h) * 2));
            }
            fetch(0);   // under way while the weights are computed
            __syncthreads();
#pragma unroll
            for (int i = 0; i < (kHeads + kWarps - 1) / kWarps; ++i) {
                const int h = warp + i * kWarps;
                if (h >= G) break;
                const float2 ml = mls[i];
                float mx = ml.x;
#pragma unroll
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float old = jn.m[h], mn = fmaxf(old, mx);
                const float wt = exp2_approx((ml.x - mn) * scale[h]);
                float ls = ml.y * wt;   // a NaN stays
#pragma unroll
                for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                jn.weight[h][lane] = wt;
                __syncwarp();
                if (lane == 0) {
                    const float fo = exp2_approx((old - mn) * scale[h]);
                    jn.f[h] = fo;
                    jn.l[h] = jn.l[h] * fo + ls;
                    jn.m[h] = mn;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int e = 4 * (tid + k * kThreads);
                const float fo = e < G * kD ? jn.f[e / kD] : 0.0f;
                acc[k].x *= fo; acc[k].y *= fo; acc[k].z *= fo; acc[k].w *= fo;
            }
#pragma unroll 1
            for (int x = 0; x < nx; x += kBatch) {
                if (x) fetch(x);
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int e = 4 * (tid + k * kThreads);
#pragma unroll
                    for (int y = 0; y < kBatch; ++y)
                        if (e < G * kD && x + y < nx) {
                            const float wt = jn.weight[e / kD][x + y];
                            acc[k].x = fmaf(v[k][y].x, wt, acc[k].x);
                            acc[k].y = fmaf(v[k][y].y, wt, acc[k].y);
                            acc[k].z = fmaf(v[k][y].z, wt, acc[k].z);
                            acc[k].w = fmaf(v[k][y].w, wt, acc[k].w);
                        }
                }
            }
            __syncthreads();   // weights and factors are read before the next 32 replace them
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = 4 * (tid + k * kThreads);
            if (e >= G * kD) continue;
            const int h = e / kD;
            if (final) {
                done(e, acc[k], jn.m[h], jn.l[h], scale[h]);
            } else {
                const size_t to = (size_t)slot_of(x_first);
                *reinterpret_cast<float4 *>(parts.o + to * G * kD + e) = acc[k];
                if (e % kD == 0) *reinterpret_cast<float2 *>(parts.ml + (to * G + h) * 2) = make_float2(jn.m[h], jn.l[h]);
            }
        }
        if (final) return;
        x_first = c_first;
        every = kGroup;
        n = (shares + kGroup - 1) / kGroup;
        ticket = parts.ticket + c_first;
        final = true;
    }
}

}  // namespace fathom
