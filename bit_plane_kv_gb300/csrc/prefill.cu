// prefill.cu -- causal attention of packed prompts (grouped query heads), on the
// fifth generation tensor cores.
//
// One CTA takes 256 query rows of one sequence: the query heads that share a KV
// head are interleaved with the tokens (row = token * Gp + head, Gp the largest
// power of two in the group), so a K or V tile read once serves all of them and
// the causal edge is narrow.  The rows form two tiles of 128, worked on in turn:
// while the tensor cores multiply for one, four warps exponentiate the other's
// scores (thread = row).  Per tile and 128 keys:
//   S = Q K^T           both operands in shared memory, S in tensor memory
//   P = exp2(c S - m)   registers; P back to tensor memory, rounded to the rows' type (both
//                       operands of an instruction have one type; in pieces that would keep
//                       fp32, as the decode attention's, P V would take three times as long)
//   O = O + P V         P from tensor memory, V from shared memory
// with c = log2(e) / sqrt(D) and the running maximum m, sum l of a softmax in one
// pass.  The exponentials of a row are taken against a maximum that may be up to
// 2^8 too small (m is raised, and O and l rescaled, only beyond that): O, 64 KB of
// tensor memory, is touched by the row's own thread in a few tiles only.
// A warp loads Q and a ring of K and V tiles by TMA; one elected lane of another
// issues the matrix instructions; CTAs stay and take over the work of those that have
// not started, so that one item's epilogue runs beside the next one's loads and
// products.  With fewer items than half the SMs, clusters share an item's keys.
//
// Bound: a tile's chain S -> softmax -> P V, S of the next keys (P takes the place of
// S in tensor memory, which S, P and O of two tiles fill, so the next S waits for it):
// about 2700 clocks per 128 keys and two tiles where the products alone take 2050.
// Measured, 32 query heads on 8 KV heads, 128 channels, bf16: one prompt of 16384
// tokens 1330 us (2.2 TFLOP, 1.65 PFLOP/s; 1.90 measured for library products), 12
// prompts of up to 2048 tokens 168 us (1.10 PFLOP/s), 16 tokens against 8192 24 us.
// What the steps gave on the 16k prompt: one thread per row with a full pass for the
// maximum 2029 us; matrix instructions behind an elected lane instead of lane 0
// 1883 -> 1445 us (their issue, not their execution, had been the bound); CTAs that
// take over work 1445 -> 1370 us, and 237 -> 182 us for the packed prompts; whole-line
// stores 173 -> 165 us there (the second look at rows that are not finite, below, took 4 of
// them back).
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "blackwell.cuh"
#include "prefill_work.cuh"

namespace fathom {

namespace {

// Warps 0-3 and 4-7: the two tiles' rows (a warp reaches the 32 lanes of tensor
// memory that its number modulo 4 names); then one warp issues the matrix
// instructions and one the loads.
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kPrefillThreads = 320;
constexpr uint32_t kPanel = 128 * 128;   // bytes of 128 rows x 64 channels

// Tensor memory columns: the two S (and P) tiles, then the two O tiles.
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

constexpr int kAgain = 16;   // places for items to be worked on again; a CTA turns to them when 8 are left

template <int kPanels>   // 64-channel panels of a row: 1 (D <= 64) or 2
struct PrefillSmem {
    static constexpr int kStages = kPanels == 2 ? 4 : 8;
    static constexpr uint32_t kTile = kPanels * kPanel;
    alignas(1024) unsigned char q[2][kTile];
    alignas(1024) unsigned char kv[kStages][kTile];
    alignas(128) unsigned char out[8][32 * 128];   // a warp's rows of O, 64 channels, on their way out
    alignas(16) uint64_t answer[2];   // to the request for another CTA's work
    Work work[4];                     // the item being worked on, the next, and two before
    uint64_t q_full[2], q_empty[2], kv_full[kStages], kv_empty[kStages], s_full[2], p_full[2], o_full[2];
    uint64_t work_full[2], work_empty[2], cleaned[2], answered, drained;
    Work again[kAgain];               // items that have to be worked on again
    int agains;                       // how many
    int noted[4];                     // which of the items in work are among them
    uint32_t odd[2];                  // kSplit: values that a tile's products read were set to 0
    uint32_t tmem;
};

// Set when a bounded wait ran out: the call's results are not valid.
__device__ unsigned g_wait_expired;

struct PrefillArgs {
    int seqs, heads, kv_heads, D, total_q, total_k, gp, lg_gp, groups, tiles;
    int split;  // CTAs that share a work item's keys
    int64_t out_token, out_head, v_token, v_head;
    const int32_t *cu_q, *cu_k;
    const uint16_t *v;   // for values that are put back (below)
    void *out;
    float *lse;
};

// ---------------------------------------------------------------- rows behind a query
// P V runs over whole tiles, so a value row that a query does not see enters its sums
// with the weight 0, and 0 x NaN and 0 x infinity are NaN.  An item with a result that is not
// finite is therefore worked on again, once: what is not finite among the value rows from the first one on that
// some of its queries does not see, a few hundred at most, counts as 0 then (copy_rows), and
// the rows that do see such a value get it back at their end (put_back).  Every other result
// is, bit for bit, the one for zeros in their place, and it takes the same time whatever the number of
// keys before.  With few rows (kSplit) that is done the first time (clean_rows).
// (Tried: the values gone over always, by the warp that issues the products or by one or two
// warps of their own, in shared memory or ahead of time in device memory: packed prompts 4
// to 9 % slower.  The test of the results and the notes of what to do again cost 2 %.)

// acc + 0 x, two values at once: NaN from the first x that is not finite on.
template <int kDtype>
__device__ __forceinline__ uint32_t add_zero_times(uint32_t x, uint32_t acc) {
    if constexpr (kDtype == FATHOM_BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
}
// The two values, 0 in the place of one that is not finite.
template <int kDtype>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x) {
    constexpr uint32_t kTop = kDtype == FATHOM_BF16 ? 0x7f80u : 0x7c00u;   // infinity; a NaN is larger
    return ((x & 0x7fffu) < kTop ? x & 0xffffu : 0u) | ((x >> 16 & 0x7fffu) < kTop ? x & 0xffff0000u : 0u);
}

// Rows r0 .. r1 - 1 of a V tile in shared memory (kPanels panels of 128 bytes per row), by a
// warp: whether there was something that is not finite; it is 0 now.  (Not inlined: that made the
// loop around it, the one that issues the products, 10 % slower.)
template <int kPanels, int kDtype>
__device__ __noinline__ bool clean_rows(unsigned char *tile, int r0, int r1) {
    const int lane = threadIdx.x & 31;
    uint32_t acc[4] = {};
#pragma unroll 4
    for (int e = r0 * 8 + lane; e < r1 * 8; e += 32)
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            const uint4 x = *reinterpret_cast<const uint4 *>(tile + p * kPanel + e * 16);
            acc[0] = add_zero_times<kDtype>(x.x, acc[0]);
            acc[1] = add_zero_times<kDtype>(x.y, acc[1]);
            acc[2] = add_zero_times<kDtype>(x.z, acc[2]);
            acc[3] = add_zero_times<kDtype>(x.w, acc[3]);
        }
    if (!__any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0)) return false;
    for (int e = r0 * 8 + lane; e < r1 * 8; e += 32)
        for (int p = 0; p < kPanels; ++p) {
            uint4 &x = *reinterpret_cast<uint4 *>(tile + p * kPanel + e * 16);
            x = make_uint4(finite_or_zero<kDtype>(x.x), finite_or_zero<kDtype>(x.y), finite_or_zero<kDtype>(x.z),
                           finite_or_zero<kDtype>(x.w));
        }
    fence_async_smem();
    __syncwarp();
    return true;
}

// A V tile, as TMA leaves it, from the rows at `v` by a warp, but rows from `first` on with 0 in the place of what
// is not finite, and 0 from row `end` on.
template <int kPanels, int kDtype>
__device__ __noinline__ void copy_rows(unsigned char *tile, const uint16_t *v, int64_t v_token, int D, int first, int end) {
    constexpr int kPieces = 8 * kPanels;   // of 16 bytes, per row
#pragma unroll 8
    for (int e = threadIdx.x & 31; e < kKeys * kPieces; e += 32) {
        const int r = e / kPieces, c = e % kPieces;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < end && c * 8 < D) x = *reinterpret_cast<const uint4 *>(v + r * v_token + c * 8);
        if (r >= first)
            x = make_uint4(finite_or_zero<kDtype>(x.x), finite_or_zero<kDtype>(x.y), finite_or_zero<kDtype>(x.z),
                           finite_or_zero<kDtype>(x.w));
        *reinterpret_cast<uint4 *>(tile + c / 8 * kPanel + r * 128 + ((c % 8 ^ (r & 7)) << 4)) = x;
    }
    fence_async_smem();
    __syncwarp();
}

template <int kDtype>
__device__ __forceinline__ float wide(uint32_t x) {
    return kDtype == FATHOM_BF16 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((unsigned short)x));
}

// The values that are not finite among the rows that a query sees from the item's first unseen one on, added
// to its result: rows r0 .. r1 - 1 of an item (as of a Work that has all its keys), by a warp, four channels per lane.
template <int kDtype>
__device__ __noinline__ void put_back(const PrefillArgs &a, int group, int q0, int lq, int k0, int lk, int t0, int r0, int r1) {
    const int c = 4 * (threadIdx.x & 31), head0 = group << a.lg_gp;
    __syncwarp();   // the rows of out are there
    if (c < a.D) {
        const uint16_t *v = a.v + (int64_t)k0 * a.v_token + head0 / (a.heads / a.kv_heads) * a.v_head + c;
        float sum[4] = {};   // 0, or not finite
        for (int r = r0, j = max(t0 + lk - lq + 1, 0); r < r1; ++r) {
            const int t = t0 + (r >> a.lg_gp), seen = min(lk, t + lk - lq + 1);
            if (t >= lq) break;
            for (; j < seen; ++j) {
                const uint2 x = *reinterpret_cast<const uint2 *>(v + j * a.v_token);
                const float y[4] = {wide<kDtype>(x.x & 0xffffu), wide<kDtype>(x.x >> 16), wide<kDtype>(x.y & 0xffffu),
                                    wide<kDtype>(x.y >> 16)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(fabsf(y[i]) < CUDART_INF_F)) sum[i] += y[i];
            }
            if (sum[0] == 0.0f && sum[1] == 0.0f && sum[2] == 0.0f && sum[3] == 0.0f) continue;
            uint2 &o = *reinterpret_cast<uint2 *>((uint16_t *)a.out + (int64_t)(q0 + t) * a.out_token +
                                                  (head0 + (r & (a.gp - 1))) * a.out_head + c);
            const uint2 x = o;
            o = make_uint2(pack2<kDtype>(wide<kDtype>(x.x & 0xffffu) + sum[0], wide<kDtype>(x.x >> 16) + sum[1]),
                           pack2<kDtype>(wide<kDtype>(x.y & 0xffffu) + sum[2], wide<kDtype>(x.y >> 16) + sum[3]));
        }
    }
    __syncwarp();
}

__device__ __forceinline__ int clamp_to(int x, int hi) { return min(max(x, 0), hi); }

// kSteps: 16-channel steps of a row (4, 6 or 8; channels from D on are zero in shared
// memory).  A constant, so that no branch stands between the matrix instructions:
// with a runtime count the unrolled and guarded instructions were issued with wrong
// descriptors.
// kSplit: few rows.  The CTAs of a cluster take the same 256 rows and a share of their
// keys each; at the end each row's partial results meet, through distributed shared
// memory, in the CTA that its warp's number names.
template <int kSteps, int kDtype, bool kSplit>
__global__ void __launch_bounds__(kPrefillThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PrefillArgs a) {
    constexpr int kPanels = (kSteps + 3) / 4;
    using Smem = PrefillSmem<kPanels>;
    constexpr int kStages = Smem::kStages;
    constexpr uint32_t kTile = Smem::kTile;
    extern __shared__ unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&sm.kv_full[i]), 1);
            mbar_init(smem_addr(&sm.kv_empty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&sm.q_full[w]), 1);
            mbar_init(smem_addr(&sm.q_empty[w]), 1);
            mbar_init(smem_addr(&sm.s_full[w]), 1);
            mbar_init(smem_addr(&sm.p_full[w]), 4);
            mbar_init(smem_addr(&sm.o_full[w]), 1);
            mbar_init(smem_addr(&sm.cleaned[w]), 1);
            mbar_init(smem_addr(&sm.work_full[w]), 1);
            mbar_init(smem_addr(&sm.work_empty[w]), kLoadWarp);   // every other warp reads it
        }
        for (int i = 0; i < 4; ++i) sm.noted[i] = 0;
        sm.agains = 0;
        mbar_init(smem_addr(&sm.answered), 1);
        mbar_init(smem_addr(&sm.drained), 1);
        mbar_init_fence();
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&sm.tmem), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    bool ok = true;

    // ---- the work item of a blockIdx.x: which sequence and which 256 rows, the last tiles first (they see
    // the most keys); a whole warp
    const int tw = kRows >> a.lg_gp;
    const int rank = kSplit ? (int)(blockIdx.x % a.split) : 0;
    const int first_item = kSplit ? (int)(blockIdx.x / a.split) : (int)blockIdx.x;
    int turns = 0;   // items of one tile so far
    int seen_s0 = 0, seen_before = 0;   // the 32 sequences that held the last item, and the tile pairs before them
    int held_s0 = -1, q0 = 0, lq = 0, k0 = 0, lk = 0;   // the 32 sequences at hand, one per lane
    auto geometry = [&](int item) {
        Work g;
        g.group = item % a.groups;
        const int nth = a.tiles - 1 - item / a.groups;
        int seq = -1, tile = 0;
        auto pairs = [&](int s0) {   // of 256-row pairs of tiles: this lane's sequence's
            if (s0 != held_s0) {
                held_s0 = s0;
                q0 = lq = k0 = lk = 0;
                if (s0 + lane < a.seqs) {
                    q0 = clamp_to(a.cu_q[s0 + lane], a.total_q);
                    lq = max(clamp_to(a.cu_q[s0 + lane + 1], a.total_q) - q0, 0);
                    k0 = clamp_to(a.cu_k[s0 + lane], a.total_k);
                    lk = max(clamp_to(a.cu_k[s0 + lane + 1], a.total_k) - k0, 0);
                }
            }
            return (int)((((long long)lq << a.lg_gp) + 2 * kRows - 1) / (2 * kRows));
        };
        // items come in falling order: the search starts where the last one ended
        while (nth < seen_before && seen_s0 > 0) {
            seen_s0 -= 32;
            seen_before -= __reduce_add_sync(0xffffffffu, pairs(seen_s0));
        }
        for (; seen_s0 < a.seqs; seen_s0 += 32) {
            const int n = pairs(seen_s0);
            int upto = seen_before + n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto - seen_before, o);
                if (lane >= o) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, nth < upto);
            if (hit) {
                const int l = __ffs(hit) - 1;
                seq = l;
                tile = nth - __shfl_sync(0xffffffffu, upto - n, l);
                break;
            }
            seen_before = __shfl_sync(0xffffffffu, upto, 31);
        }
        g.lq = g.nt0 = g.nt1 = g.steps = g.q0 = g.k0 = g.lk = g.off = g.t0 = g.from = g.flip = g.half = g.again = 0;
        if (seq < 0) return g;   // the grid counts up to a tile pair per sequence more than needed
        g.q0 = __shfl_sync(0xffffffffu, q0, seq);
        g.lq = __shfl_sync(0xffffffffu, lq, seq);
        g.k0 = __shfl_sync(0xffffffffu, k0, seq);
        g.lk = __shfl_sync(0xffffffffu, lk, seq);
        g.off = g.lk - g.lq;
        g.t0 = tile << (8 - a.lg_gp);
        // rows for one tile only go to either in turn, so that its epilogue runs beside the other's products
        // (1000 prompts of 16 tokens, 32 heads on 8: 213 -> 133 us)
        g.flip = !kSplit && g.lq - g.t0 <= tw ? turns++ & 1 : 0;
        work_steps(g, tw);
        if constexpr (kSplit) work_share(g, rank, a.split);
        return g;
    };
    // ---- the CTA takes over the work of CTAs that have not started: while the loads of one item run, the
    // load warp asks for the next, works out its geometry and leaves it for the other warps
    int round = 0;   // items published (read) so far
    auto get_work = [&](Work &g) {
        const int slot = round & 1;
        // a tile without keys waits here while the other goes over all of them (2^28 keys: about 3 s)
        ok = ok && warp_wait(smem_addr(&sm.work_full[slot]), (round >> 1) & 1, 5 * kWaitLimitNs);
        // every field from one lane: the compiler then knows that the warp branches as one (without that the
        // loops below ran 9 % slower)
        const int *f = &sm.work[round & 3].group;
        auto field = [&](int i) { return __shfl_sync(0xffffffffu, f[i], 0); };
        g.group = field(0); g.q0 = field(1); g.lq = field(2); g.k0 = field(3); g.lk = field(4);
        g.off = field(5); g.t0 = field(6); g.nt0 = field(7); g.nt1 = field(8); g.steps = field(9);
        g.from = field(10); g.flip = field(11); g.half = field(12);
        if (lane == 0) mbar_arrive(smem_addr(&sm.work_empty[slot]));
        ++round;
        return ok && g.steps >= 0;
    };

    if (warp == kLoadWarp) {
        int st = 0, nq0 = 0, nq1 = 0;   // the ring's next stage; Q tiles loaded so far
        uint32_t turn = 1;              // parity of the stage's last release; true at once in the first turn
        auto publish = [&](const Work &g) {
            const int slot = round & 1;
            ok = ok && warp_wait(smem_addr(&sm.work_empty[slot]), ((round >> 1) & 1) ^ 1);
            if (lane == 0 && ok) {
                sm.work[round & 3] = g;
                mbar_arrive(smem_addr(&sm.work_full[slot]));
            }
            __syncwarp();
            ++round;
        };
        auto loaded = [&](const Work &g) {
            nq0 += g.nt0 > 0;
            nq1 += g.nt1 > 0;
            const int end = st + 2 * g.steps;
            turn ^= (uint32_t)(end / kStages) & 1u;
            st = end % kStages;
        };
        // Until all warps have read an item without rows: they are done with all others then.
        auto all_done = [&] {
            Work none = {};
            publish(none);
            ok = ok && warp_wait(smem_addr(&sm.work_empty[(round - 1) & 1]), ((round - 1) >> 1) & 1, 5 * kWaitLimitNs);
        };
        // The items noted so far, all over again: by the whole warp, and V tiles with rows behind a query not by TMA.
        auto work_again = [&] {
            const int n = __shfl_sync(0xffffffffu, sm.agains, 0);
            for (int i = 0; i < 2 * n && ok; ++i) {
                if (i == n) all_done();
                const Work r = sm.again[i % n];
                if (i >= n) {
                    put_back<kDtype>(a, r.group, r.q0, r.lq, r.k0, r.lk, r.t0, 0, 2 * kRows);
                    continue;
                }
                publish(r);
                const int hq = r.group << a.lg_gp, hk = hq / (a.heads / a.kv_heads);
                auto load = [&](uint32_t bar, unsigned char *to, const void *map, int head, int row) {
                    if (lane == 0) {
                        mbar_expect(bar, kTile);
                        for (int p = 0; p < kPanels; ++p) tma_load_3d(smem_addr(to) + p * kPanel, map, bar, 64 * p, head, row);
                    }
                    __syncwarp();
                };
                for (int w = 0; w < 2 && ok; ++w) {
                    if ((w ? r.nt1 : r.nt0) == 0) continue;
                    if (!(ok = warp_wait(smem_addr(&sm.q_empty[w]), ((w ? nq1 : nq0) & 1) ^ 1))) break;
                    load(smem_addr(&sm.q_full[w]), sm.q[w], &map_q, hq, r.q0 + r.t0 + (w ^ r.flip) * tw);
                }
                int s = st;
                uint32_t t = turn;
                for (int x = 0; x < 2 * r.steps && ok; ++x) {
                    if (!(ok = warp_wait(smem_addr(&sm.kv_empty[s]), t))) break;
                    const int j = x >> 1;
                    if ((x & 1) && j >= work_first_edge(r)) {
                        copy_rows<kPanels, kDtype>(sm.kv[s], a.v + (int64_t)(r.k0 + j * kKeys) * a.v_token + hk * a.v_head,
                                                   a.v_token, a.D, work_first_unseen(r) - j * kKeys, r.lk - j * kKeys);
                        if (lane == 0) mbar_arrive(smem_addr(&sm.kv_full[s]));
                    } else {
                        load(smem_addr(&sm.kv_full[s]), sm.kv[s], (x & 1) ? &map_v : &map_k, hk, r.k0 + j * kKeys);
                    }
                    if (++s == kStages) { s = 0; t ^= 1; }
                }
                ok = __all_sync(0xffffffffu, ok);
                loaded(r);
            }
            __syncwarp();
            if (lane == 0) sm.agains = 0;
            __syncwarp();
        };
        Work g = geometry(first_item);
        int asked = 0;
        for (bool more = true; ok && more;) {
            do {
                publish(g);
                if (!ok) break;
                if (elect_one()) {
                    if (!kSplit) {
                        mbar_expect(smem_addr(&sm.answered), 16);
                        request_cta(smem_addr(sm.answer), smem_addr(&sm.answered));
                    }
                    const int hq = g.group << a.lg_gp, hk = hq / (a.heads / a.kv_heads);
                    for (int w = 0; w < 2 && ok; ++w) {
                        if ((w ? g.nt1 : g.nt0) == 0) continue;
                        if (!(ok = mbar_wait(smem_addr(&sm.q_empty[w]), ((w ? nq1 : nq0) & 1) ^ 1))) break;
                        const uint32_t bar = smem_addr(&sm.q_full[w]);
                        mbar_expect(bar, kTile);
                        for (int p = 0; p < kPanels; ++p)
                            tma_load_3d(smem_addr(sm.q[w]) + p * kPanel, &map_q, bar, 64 * p, hq, g.q0 + g.t0 + (w ^ g.flip) * tw);
                    }
                    int s = st;
                    uint32_t t = turn;
                    for (int i = 0; i < 2 * g.steps && ok; ++i) {   // K_0, V_0, K_1, V_1, ...
                        if (!(ok = mbar_wait(smem_addr(&sm.kv_empty[s]), t))) break;
                        const uint32_t bar = smem_addr(&sm.kv_full[s]);
                        mbar_expect(bar, kTile);
                        for (int p = 0; p < kPanels; ++p)
                            tma_load_3d(smem_addr(sm.kv[s]) + p * kPanel, (i & 1) ? &map_v : &map_k, bar, 64 * p, hk,
                                        g.k0 + (i >> 1) * kKeys);
                        if (++s == kStages) { s = 0; t ^= 1; }
                    }
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok);
                loaded(g);
                int item = -1;
                if (!kSplit && ok) {
                    ok = warp_wait(smem_addr(&sm.answered), asked++ & 1);
                    if (ok) item = granted_cta(sm.answer[0], sm.answer[1]);
                    fence_async_smem();   // the answer is read before the next one is asked for
                    __syncwarp();
                }
                more = item >= 0;
                if (more) g = geometry(item);
            } while (ok && more && (kSplit || __shfl_sync(0xffffffffu, sm.agains, 0) < kAgain - 8));
            if (!kSplit && ok) {
                all_done();
                work_again();
            }
        }
        g.steps = -1;
        publish(g);
        if (!ok) {   // the copies in flight land before the CTA ends
            const unsigned long long t0 = global_ns();
            while (global_ns() - t0 < 10000000ull) {}
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t type = kDtype == FATHOM_BF16 ? 1u : 0u;
        const uint32_t desc_s = mma_desc(type, kRows, kKeys, false), desc_h = mma_desc(type, kRows, kKeys / 2, false);
        const uint32_t desc_o = mma_desc(type, kRows, kSteps * 16, true);
        // descriptors of the first 16 channels (keys) of each operand; the others lie at fixed offsets, and
        // the address field of a descriptor counts 16 bytes
        const uint64_t desc_q = smem_desc(smem_addr(sm.q[0]), 0);
        const uint64_t desc_k = smem_desc(smem_addr(sm.kv[0]), 0), desc_v = smem_desc(smem_addr(sm.kv[0]), kPanel);
        // S of tile w against the K tile of a stage, all of its keys or the first 64
        auto scores = [&](int w, int st, bool half) {
            const uint64_t dq = desc_q + w * (kTile >> 4), dk = desc_k + st * (kTile >> 4);
            if (half) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const uint32_t at = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
                    mma_ss(tmem + kColS + w * 128, dq + at, dk + at, desc_h, k > 0);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const uint32_t at = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
                    mma_ss(tmem + kColS + w * 128, dq + at, dk + at, desc_s, k > 0);
                }
            }
            mma_commit(smem_addr(&sm.s_full[w]));
        };
        auto values = [&](int w, int st, bool first, bool half) {
            const uint64_t dv = desc_v + st * (kTile >> 4);
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k)
                mma_ts(tmem + kColO + w * 128, tmem + kColS + w * 128 + k * 8, dv + ((k * 16 * 128) >> 4), desc_o,
                       k > 0 ? 1u : (uint32_t)!first);
            if (!half) {
#pragma unroll
                for (int k = kKeys / 32; k < kKeys / 16; ++k)
                    mma_ts(tmem + kColO + w * 128, tmem + kColS + w * 128 + k * 8, dv + ((k * 16 * 128) >> 4), desc_o, 1u);
            }
            mma_commit(smem_addr(&sm.o_full[w]));
        };
        const uint32_t full = smem_addr(sm.kv_full), empty = smem_addr(sm.kv_empty);
        const uint32_t q_full = smem_addr(sm.q_full), q_empty = smem_addr(sm.q_empty), p_full = smem_addr(sm.p_full);
        int cur = 0;                                // the ring's stages in turn: K_0, V_0, K_1, V_1, ...
        uint32_t pc = 0, pq0 = 0, pq1 = 0, pp0 = 0, pp1 = 0;   // parities of the next wait on each barrier
        auto products = [&](const Work &g) {   // of an item
            const int tail = g.lk - (g.steps - 1) * kKeys;   // live rows of the last V tile
            [[maybe_unused]] uint32_t odd = 0;
            ok = warp_wait(full + 8 * cur, pc) && (g.nt0 == 0 || warp_wait(q_full, pq0)) &&
                 (g.nt1 == 0 || warp_wait(q_full + 8, pq1));
            if (!ok) return;
            pq0 ^= g.nt0 > 0;
            pq1 ^= g.nt1 > 0;
            if (elect_one()) {
                tc_fence_after();
                if (g.nt0 > 0) scores(0, cur, g.nt0 == 1 && (g.half & 1));
                if (g.nt0 == 1) mma_commit(q_empty);
                if (g.nt1 > 0) scores(1, cur, g.nt1 == 1 && (g.half & 2));
                if (g.nt1 == 1) mma_commit(q_empty + 8);
                mma_commit(empty + 8 * cur);
            }
            __syncwarp();
            for (int j = 0; j < g.steps; ++j) {
                int sv = cur + 1, sk;
                uint32_t pv = pc, pk;
                if (sv == kStages) { sv = 0; pv ^= 1; }
                sk = sv + 1;
                pk = pv;
                if (sk == kStages) { sk = 0; pk ^= 1; }
                cur = sk;   // K_{j+1}, or the next item's K_0
                pc = pk;
                const bool more = j + 1 < g.steps;
                if (!(ok = warp_wait(full + 8 * sv, pv) && (!more || warp_wait(full + 8 * sk, pk)))) break;
                if constexpr (kSplit) {
                    if (j >= work_first_edge(g)) {
                        const EdgeRows e = work_edge(g, j);
                        odd |= clean_rows<kPanels, kDtype>(sm.kv[sv], e.r0, e.r1);
                    }
                }
                if (!more && tail < kKeys) {
                    // rows behind the sequence's end: their weights are 0, and 0 x NaN would not be
                    for (int e = tail * 8 + lane; e < kKeys * 8; e += 32)
                        for (int p = 0; p < kPanels; ++p)
                            *reinterpret_cast<int4 *>(sm.kv[sv] + p * kPanel + e * 16) = make_int4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                if (j < g.nt0) {
                    if (!(ok = warp_wait(p_full, pp0))) break;
                    pp0 ^= 1;
                    tc_fence_after();
                    if (elect_one()) {
                        values(0, sv, j == 0, j + 1 == g.nt0 && (g.half & 1));
                        if (j + 1 < g.nt0) scores(0, sk, j + 2 == g.nt0 && (g.half & 1));
                        if (j + 2 == g.nt0) mma_commit(q_empty);
                        if (kSplit && j + 1 == g.nt0) {
                            sm.odd[0] = odd;
                            mbar_arrive(smem_addr(&sm.cleaned[0]));
                        }
                    }
                    __syncwarp();
                }
                if (j < g.nt1) {
                    if (!(ok = warp_wait(p_full + 8, pp1))) break;
                    pp1 ^= 1;
                    tc_fence_after();
                    if (elect_one()) {
                        values(1, sv, j == 0, j + 1 == g.nt1 && (g.half & 2));
                        mma_commit(empty + 8 * sv);
                        if (j + 1 < g.nt1) scores(1, sk, j + 2 == g.nt1 && (g.half & 2));
                        if (j + 2 == g.nt1) mma_commit(q_empty + 8);
                        if (kSplit && j + 1 == g.nt1) {
                            sm.odd[1] = odd;
                            mbar_arrive(smem_addr(&sm.cleaned[1]));
                        }
                        if (more) mma_commit(empty + 8 * sk);
                    }
                } else if (elect_one()) {
                    mma_commit(empty + 8 * sv);
                    if (more) mma_commit(empty + 8 * sk);
                }
                __syncwarp();
            }
        };
        for (Work g; ok && get_work(g);) {
            if (g.steps == 0) continue;
            products(g);
        }
        __syncwarp();
        if (elect_one()) mma_commit(smem_addr(&sm.drained));
        __syncwarp();
        warp_wait(smem_addr(&sm.drained), 0);   // no matrix instruction outlives the tensor memory
    } else {
        const int w = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + kColS + w * 128, to = tmem + lanes + kColO + w * 128;
        const float c = 1.4426950408889634f / sqrtf((float)a.D);   // log2(e) / sqrt(D)
        // How far (log2) a row's maximum may rise above m before m follows, and the power of two by which all
        // weights are scaled.  A bf16 weight is as exact at any scale, and at most 1 here: O overflows only where
        // the sum of the values themselves does (weights of up to 2^32, with a lag of 32, made an average of values
        // of 2^100 infinite; ordinary scores do not rise by 2^8 above those of the first 64 keys).  fp16 weights are
        // kept larger, at most 2^15, so that fewer fall among the subnormals.
        constexpr float kLag = 8.0f, kShift = kDtype == FATHOM_F16 ? 7.0f : -8.0f;
        uint32_t ps = 0, po = 0;   // parities of the next wait for S, and for the last product into O
        Meetings cluster{kSplit ? 2 : 0};
        // (a plain loop here: with the items' code in a function of its own, tiles without rows held up the other
        // tile: 1000 prompts of 16 tokens 132 -> 191 us)
        for (Work g; get_work(g);) {
            // no rows (anything before this `continue` makes packed prompts 10 % slower)
            if (!kSplit && g.t0 + (w ^ g.flip) * tw >= g.lq) continue;
            const int nt = w ? g.nt1 : g.nt0;
            const int token = g.t0 + (w ^ g.flip) * tw + (row >> a.lg_gp);
            const int at = token < g.lq ? g.q0 + token : -1;   // row of out; -1: behind the sequence
            const int head = (g.group << a.lg_gp) + (row & (a.gp - 1));
            // keys this row sees, and the fewest that a row of this warp sees
            const int seen = min(g.lk, token + g.off + 1);
            const int seen_min = min(g.lk, g.t0 + (w ^ g.flip) * tw + (((warp & 3) * 32) >> a.lg_gp) + g.off + 1);
            float m = -CUDART_INF_F, l = 0.0f;   // m in log2 units; -inf: no finite score yet
            auto step = [&](int j, auto halves) {   // 128 keys, or the first 64 of the last ones
                constexpr int kHalves = decltype(halves)::value;
                if (!(ok = warp_wait(smem_addr(&sm.s_full[w]), ps))) return;
                ps ^= 1;
                tc_fence_after();
                const bool edge = (j + 1) * kKeys > seen_min;
                const int live = seen - j * kKeys;
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                uint32_t s[4][32];   // columns 32 b .. 32 b + 31 of S
                tmem_ld32(ts, s[0]);
                tmem_ld32(ts + 32, s[1]);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {   // 64 keys at a time
                    float top = -CUDART_INF_F, top2 = -CUDART_INF_F;
#pragma unroll
                    for (int b = 2 * h; b < 2 * h + 2; ++b) {
                        tmem_wait_ld(s[b]);
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * b + i >= live) s[b][i] = 0xff800000u;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            top = fmaxf(top, __uint_as_float(s[b][i]));
                            top2 = fmaxf(top2, __uint_as_float(s[b][i + 1]));
                        }
                    }
                    top = fmaxf(top, top2) * c;
                    const bool raise = top > m + kLag;
                    if (__any_sync(0xffffffffu, raise)) {
                        // m rises by a whole power of two, so that what was computed against the old one is
                        // scaled exactly: l, O, and the first half's weights of this tile
                        float f = 1.0f;
                        if (raise) {
                            const float up = m == -CUDART_INF_F ? top : m + ceilf(top - m);
                            f = exp2f(m - up);
                            m = up;
                        }
                        l *= f;
                        sum[0].x *= f; sum[0].y *= f; sum[1].x *= f; sum[1].y *= f;
                        if (h == 1) {
                            tmem_wait_st();
#pragma unroll 1
                            for (int b = 0; b < 2; ++b) {
                                uint32_t o[16];
                                tmem_ld16(ts + 16 * b, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = scale2<kDtype>(o[i], f);
                                tmem_st16(ts + 16 * b, o);
                            }
                        }
                        if (j > 0) {
                            if (!(ok = warp_wait(smem_addr(&sm.o_full[w]), po ^ 1))) return;   // the product before
                            tc_fence_after();
#pragma unroll 1
                            for (int b = 0; b < kSteps; ++b) {
                                uint32_t o[16];
                                tmem_ld16(to + 16 * b, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st16(to + 16 * b, o);
                            }
                        }
                    }
                    const float shift = kShift - (m == -CUDART_INF_F ? 0.0f : m);
                    const float2 cc = make_float2(c, c), mm = make_float2(shift, shift);
#pragma unroll
                    for (int b = 2 * h; b < 2 * h + 2; ++b) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = make_float2(__uint_as_float(s[b][2 * i]), __uint_as_float(s[b][2 * i + 1]));
                            x = fma2(x, cc, mm);
                            x.x = exp2_approx(x.x);
                            x.y = exp2_approx(x.y);
                            sum[i & 1] = add2(sum[i & 1], x);
                            pk[i] = pack2<kDtype>(x.x, x.y);
                        }
                        tmem_st16(ts + 16 * b, pk);
                        if (h == 0 && kHalves == 2) tmem_ld32(ts + 64 + 32 * b, s[2 + b]);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sm.p_full[w]));
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                po ^= 1;
            };
            const int full = nt - (nt > 0 ? g.half >> w & 1 : 0);
            for (int j = 0; j < full && ok; ++j) step(j, std::integral_constant<int, 2>());
            if (full < nt && ok) step(full, std::integral_constant<int, 1>());
            // ---- O / l, rounded once
            ok = ok && (nt == 0 || warp_wait(smem_addr(&sm.o_full[w]), po ^ 1));
            [[maybe_unused]] bool cleaned = false;   // kSplit: values that these rows' products read were set to 0
            if (kSplit && nt > 0) {
                ok = ok && warp_wait(smem_addr(&sm.cleaned[w]), 0);
                cleaned = ok && sm.odd[w];
            }
            if (ok || kSplit) {
                tc_fence_after();
                // kSplit: the other CTAs' (O, m, l, cleaned) of these rows, [share][channel, then those][row of the warp]
                constexpr int kShare = (kSteps * 16 + 3) * 32;
                static_assert(!kSplit || 7 * kShare * 4 <= (int)sizeof(sm.kv), "shares reuse the ring");
                const int per = 8 / (kSplit ? a.split : 1), dst = warp / per;   // warps per CTA, and this one's CTA
                [[maybe_unused]] float *shares = reinterpret_cast<float *>(sm.kv) + warp % per * kShare + lane;   // += per * kShare each
                float own = 1.0f;
                [[maybe_unused]] float other[7];
                if constexpr (kSplit) {
                    cluster.meet(cluster_sync);   // no CTA reads its ring any more
                    if (rank != dst) {
                        const uint32_t to_dst = cluster_addr(smem_addr(shares + (rank < dst ? rank : rank - 1) * per * kShare), dst);
                        if (nt > 0) {
#pragma unroll 1
                            for (int b = 0; b < kSteps / 2; ++b) {
                                uint32_t x[32];
                                tmem_ld32(to + 32 * b, x);
                                tmem_wait_ld(x);
#pragma unroll
                                for (int i = 0; i < 32; ++i) cluster_store(to_dst + (32 * b + i) * 128, __uint_as_float(x[i]));
                            }
                        }
                        cluster_store(to_dst + kSteps * 16 * 128, ok ? m : -CUDART_INF_F);
                        cluster_store(to_dst + (kSteps * 16 + 1) * 128, ok ? l : 0.0f);
                        cluster_store(to_dst + (kSteps * 16 + 2) * 128, cleaned ? 1.0f : 0.0f);
                    }
                    cluster.meet(cluster_sync);   // every share is there
                    if (rank == dst) {
                        float top = m;
#pragma unroll
                        for (int x = 0; x < 7; ++x) {
                            other[x] = x < a.split - 1 ? shares[x * per * kShare + kSteps * 16 * 32] : -CUDART_INF_F;
                            top = fmaxf(top, other[x]);
                        }
                        // a share holds nothing when its l is 0; one whose scores are all NaN has m = -inf too, and
                        // its l, which is NaN, has to stay
                        own = m == -CUDART_INF_F ? 0.0f : exp2f(m - top);
                        l *= own;
#pragma unroll
                        for (int x = 0; x < 7; ++x) {
                            const float part = x < a.split - 1 ? shares[x * per * kShare + (kSteps * 16 + 1) * 32] : 0.0f;
                            other[x] = other[x] == -CUDART_INF_F ? 0.0f : exp2f(other[x] - top);
                            if (part != 0.0f) l += other[x] * part;
                            if (x < a.split - 1) cleaned |= shares[x * per * kShare + (kSteps * 16 + 2) * 32] != 0.0f;
                        }
                        m = top;
                    }
                }
                const bool mine = at >= 0 && ok && (!kSplit || rank == dst);
                // of a row that sees no key 0, of one with a NaN among its scores NaN
                const float inv_other = l == 0.0f ? 0.0f : 1.0f / l, inv = kSplit ? own * inv_other : inv_other;
                const float none = l == l ? 0.0f : l;
                const bool some = kSplit ? own != 0.0f && nt > 0 : seen > 0;   // O holds something for this row
                const int row_at = mine ? at : -1;
                float2 odd = make_float2(0.0f, 0.0f);   // 0 as long as the row is finite
                unsigned char *stage = sm.out[warp];
                // 64 channels at a time through shared memory, so that a store writes four whole lines and
                // not 32 pieces of as many rows
#pragma unroll 1
                for (int b = 0; b < (!kSplit || rank == dst ? kSteps / 2 : 0); ++b) {
                    uint32_t x[32];
                    if (nt > 0) {
                        tmem_ld32(to + 32 * b, x);
                        tmem_wait_ld(x);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float v = some ? __uint_as_float(x[i]) * inv : none;
                        if constexpr (kSplit) {
#pragma unroll
                            for (int y = 0; y < 7; ++y)
                                if (other[y] != 0.0f) v = fmaf(shares[y * per * kShare + (32 * b + i) * 32], other[y] * inv_other, v);
                        }
                        x[i] = __float_as_uint(v);
                    }
#pragma unroll
                    for (int i = 0; i < (kSplit ? 0 : 16); ++i)
                        odd = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                   make_float2(0.0f, 0.0f), odd);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pk[e] = pack2<kDtype>(__uint_as_float(x[8 * i + 2 * e]), __uint_as_float(x[8 * i + 2 * e + 1]));
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + (((4 * (b & 1) + i) ^ (lane & 7)) << 4)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    if ((b & 1) || b + 1 == kSteps / 2) {
                        __syncwarp();
                        const int ch = lane & 7, col = 64 * (b >> 1) + 8 * ch;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int rr = 4 * i + (lane >> 3);
                            const uint4 v = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
                            const int t = __shfl_sync(0xffffffffu, row_at, rr);
                            const int h = (g.group << a.lg_gp) + (((warp & 3) * 32 + rr) & (a.gp - 1));
                            if (t >= 0 && col < a.D)
                                *reinterpret_cast<uint4 *>((uint16_t *)a.out + (int64_t)t * a.out_token + h * a.out_head + col) = v;
                        }
                        __syncwarp();
                    }
                }
                const float lse = l == 0.0f ? -CUDART_INF_F : ((m - kShift) + log2f(l)) * 0.6931471805599453f;
                if (mine && a.lse) a.lse[(int64_t)at * a.heads + head] = lse;
                if constexpr (kSplit) {
                    if (__any_sync(0xffffffffu, cleaned && ok && rank == dst))
                        put_back<kDtype>(a, g.group, g.q0, g.lq, g.k0 - g.from, g.lk + g.from, g.t0, 32 * warp, 32 * warp + 32);
                } else if (__any_sync(0xffffffffu, mine && !(odd.x + odd.y == 0.0f))) {
                    // noted once, by the first warp of the item that comes here
                    const int at = (round - 1) & 3;
                    if (lane == 0 && !sm.work[at].again && atomicExch(&sm.noted[at], round) != round) {
                        Work &r = sm.again[atomicAdd(&sm.agains, 1)];
                        r = sm.work[at];
                        r.again = 1;
                    }
                    __syncwarp();
                }
                tc_fence_before();
            }
        }
        __syncwarp();
        cluster.rest(cluster_sync);
    }
    if (kSplit && warp >= 8) {   // the rows' warps meet twice; so do these
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    if (!ok) atomicExch(&g_wait_expired, 1u);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::mutex mu;
    static EncodeFn fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        fn = (EncodeFn)p;
    }
    return fn;
}

// Rows [tokens][heads][D] as tiles of `box_tokens` x `box_heads` rows x 64 channels;
// channels from D on read as zero.
bool encode_rows(CUtensorMap *map, int dtype, const void *base, int D, int heads, int tokens, int64_t head_stride,
                 int64_t token_stride, int box_heads, int box_tokens) {
    const EncodeFn fn = encode_fn();
    if (!fn) { set_error("prefill_attn: the driver does not offer cuTensorMapEncodeTiled"); return false; }
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)(tokens > 0 ? tokens : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head_stride : D) * 2,
                                   (cuuint64_t)(tokens > 1 ? token_stride : D) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, one[3] = {1, 1, 1};
    const CUresult r = fn(map, dtype == FATHOM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          3, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) { set_error("prefill_attn: cuTensorMapEncodeTiled failed (%d)", (int)r); return false; }
    return true;
}

}  // namespace

static cudaLaunchConfig_t cluster_config(cudaLaunchAttribute *attr, unsigned grid, int cluster, size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kPrefillThreads);
    cfg.dynamicSmemBytes = smem;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)cluster;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of that many CTAs that the current device holds at once (8 CTAs: 15, not 19 as by
// the number of SMs, for a cluster lies within a GPC); asked once per device, as every form
// of the kernel takes a whole SM.
template <typename F>
static int resident_clusters(F *kernel, int cluster, size_t smem) {
    constexpr int kDevices = 16;
    static std::atomic<int> known[kDevices][9];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool keep = dev < kDevices;
    if (keep && (n = known[dev][cluster].load(std::memory_order_relaxed)) != 0) return n - 1;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_config(&attr, (unsigned)cluster, cluster, smem);
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) { cudaGetLastError(); return 0; }
    if (keep) known[dev][cluster].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <typename F, typename... Args>
static cudaError_t launch_cluster(F *kernel, unsigned grid, int cluster, size_t smem, cudaStream_t st,
                                  const Args &...args) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = cluster_config(&attr, grid, cluster, smem);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool wait_expired_prefill() {
    unsigned v = 0;
    const unsigned none = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_expired, sizeof v) != cudaSuccess) return false;
    if (v) cudaMemcpyToSymbol(g_wait_expired, &none, sizeof none);
    return v != 0;
}

int launch_prefill_attn(const fathom_prompts &p, const void *q, const void *k, const void *v, const int32_t *cu_q,
                        const int32_t *cu_k, void *out, float *lse, cudaStream_t st) {
    const int G = p.heads / p.kv_heads;
    PrefillArgs a;
    a.seqs = p.seqs; a.heads = p.heads; a.kv_heads = p.kv_heads; a.D = p.D;
    a.total_q = p.total_q; a.total_k = p.total_k;
    a.lg_gp = 0;
    while (a.lg_gp < 7 && G % (2 << a.lg_gp) == 0) ++a.lg_gp;
    a.gp = 1 << a.lg_gp;
    a.groups = p.heads / a.gp;
    a.out_token = p.out_token; a.out_head = p.out_head;
    a.v_token = p.v_token; a.v_head = p.v_head;
    a.v = (const uint16_t *)v;
    a.cu_q = cu_q; a.cu_k = cu_k; a.out = out; a.lse = lse;
    // pairs of tiles, at most: exact for one sequence
    const long long tiles = ((long long)p.total_q * a.gp + (2LL * kRows - 1) * p.seqs) / (2 * kRows);
    if (tiles * a.groups > 0x7fffffffLL) { set_error("prefill_attn: too many rows for one launch"); return FATHOM_EINVAL; }
    a.tiles = (int)tiles;
    CUtensorMap mq, mk, mv;
    if (p.total_k == 0) k = v = q;   // no key is loaded; the maps only have to be well formed
    if (!encode_rows(&mq, p.dtype, q, p.D, p.heads, p.total_q, p.q_head, p.q_token, a.gp, kRows / a.gp) ||
        !encode_rows(&mk, p.dtype, k, p.D, p.kv_heads, p.total_k, p.k_head, p.k_token, 1, kKeys) ||
        !encode_rows(&mv, p.dtype, v, p.D, p.kv_heads, p.total_k, p.v_head, p.v_token, 1, kKeys))
        return FATHOM_ECUDA;
    // With few work items, clusters of 2, 4 or 8 CTAs share an item's keys, as long as each gets a few
    // steps and all clusters are resident at once
    const long long items = tiles * a.groups;
    const bool few = 2 * items <= device_sm_count() && p.total_k >= 8 * kKeys;
#define FATHOM_PREFILL(SS, DD)                                                                     \
    do {                                                                                           \
        const size_t smem = sizeof(PrefillSmem<(SS + 3) / 4>) + 1024;                              \
        a.split = 1;                                                                               \
        if (few) {                                                                                 \
            ensure_smem(prefill_kernel<SS, DD, true>, smem);                                       \
            while (a.split < 8 && p.total_k >= 4 * kKeys * 2 * a.split &&                          \
                   items <= resident_clusters(prefill_kernel<SS, DD, true>, 2 * a.split, smem))    \
                a.split *= 2;                                                                      \
        }                                                                                          \
        const unsigned grid = (unsigned)(items * a.split);                                         \
        if (a.split > 1) {                                                                         \
            e = launch_cluster(prefill_kernel<SS, DD, true>, grid, a.split, smem, st, mq, mk, mv, a); \
        } else {                                                                                   \
            ensure_smem(prefill_kernel<SS, DD, false>, smem);                                      \
            prefill_kernel<SS, DD, false><<<grid, kPrefillThreads, smem, st>>>(mq, mk, mv, a);     \
        }                                                                                          \
    } while (0)
    cudaError_t e = cudaSuccess;
    const bool bf = p.dtype == FATHOM_BF16;
    if (p.D <= 64) { if (bf) FATHOM_PREFILL(4, FATHOM_BF16); else FATHOM_PREFILL(4, FATHOM_F16); }
    else if (p.D <= 96) { if (bf) FATHOM_PREFILL(6, FATHOM_BF16); else FATHOM_PREFILL(6, FATHOM_F16); }
    else { if (bf) FATHOM_PREFILL(8, FATHOM_BF16); else FATHOM_PREFILL(8, FATHOM_F16); }
#undef FATHOM_PREFILL
    if (e != cudaSuccess) return launch_failed("prefill_kernel", e);
    return launch_status("prefill_kernel");
}

}  // namespace fathom
