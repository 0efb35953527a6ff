// evict.cu -- eviction from a paged KV cache by accumulated attention weight:
// the kept set of every unit, then its rows and mass moved together.
// Measured, 128 channels, bf16, both kernels, to other pages and in place: 256 units of
// 16k tokens cut back to 4096 each 204 and 222 us (1.0 GB moved in rows of 256 bytes, 2 KB
// apart; about 25 us of it choose the kept sets); 8 units of 8192 tokens cut to 2048 14.5
// and 21 us; 8 units of 131072 cut to 16384 68 and 126 us.  In place a chunk of rows is
// loaded, met for and stored before the next one's loads start.  Tried for that: bulk
// copies through shared memory (210 us for the 256 units' move alone; 76 us for the 8 units).
#include "blackwell.cuh"

namespace fathom {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kDigits = 3, kBins = 2048;   // 11, 11 and 10 bits of a key
constexpr int kMaxKeys = 20 * 1024;        // that a CTA keeps in shared memory

// The mass as an unsigned key of the same order; a NaN is the largest.
__device__ __forceinline__ uint32_t mass_key(float x) { return x != x ? 0xffffffffu : order_f32(x); }

// A cluster of `parts` CTAs per unit, each with a contiguous part of its tokens, whose
// keys it keeps in shared memory (as many as fit; the others are read again).  The key
// of the last kept token comes from three histograms of 11, 11 and 10 bits, each over
// the keys that agree with the digits found so far and added up over the cluster; then
// each warp counts a contiguous part's tokens above and at that key, and after the
// counts before its own it writes the kept tokens in ascending order.
__global__ void __launch_bounds__(kSelThreads, 2)
evict_select_kernel(fathom_pages p, int parts, int room, const int32_t *__restrict__ lens,
                    const float *__restrict__ mass, size_t mass_stride, int keep, int n_sink, int n_recent,
                    int32_t *__restrict__ kept, int32_t *__restrict__ lens_out) {
    pdl_enter();
    extern __shared__ uint32_t keys[];   // [room]
    __shared__ alignas(8) unsigned hist[kDigits][kBins], s_total[2];
    __shared__ unsigned s_prefix, s_left, s_sum[kSelWarps];
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    const int u = blockIdx.x / parts, rank = blockIdx.x % parts, s = u / p.kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = min(max(lens[s], 0), p.max_pages * p.page_tokens);
    int32_t *kr = kept + (size_t)u * keep;
    if (u % p.kv_heads == 0 && rank == 0 && tid == 0) lens_out[s] = min(n, keep);
    const int all = rank * kSelThreads + tid, step = parts * kSelThreads;
    if (n <= keep) {
        for (int j = all; j < keep; j += step) kr[j] = j < n ? j : -1;
        return;
    }
    const float *mr = mass + (size_t)u * mass_stride;
    const int lo = n_sink, hi = n - n_recent, want = keep - n_sink - n_recent;
    for (int j = all; j < n_sink; j += step) kr[j] = j;
    for (int j = all; j < n_recent; j += step) kr[keep - n_recent + j] = hi + j;
    if (want == 0) return;
    auto meet = [&] { if (parts > 1) cluster_sync(); else __syncthreads(); };
    // the warp's tokens b0 .. b1 - 1, the CTA's from b on
    const int seg = ((hi - lo) / (kSelWarps * parts) + 32) / 32 * 32;
    const int b = (int)min((long long)lo + (long long)rank * kSelWarps * seg, (long long)hi);
    const int end = (int)min((long long)b + kSelWarps * seg, (long long)hi);
    const int b0 = min(b + warp * seg, end), b1 = min(b0 + seg, end);
    for (int i = tid; i < kDigits * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    unsigned prefix = 0, left = (unsigned)want;
    __syncthreads();
    auto key_at = [&](int i) { return i - b < room ? keys[i - b] : mass_key(mr[i]); };
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), bins = d == 2 ? 1024 : 2048;
        if (d == 0) {
            for (int i = b + tid; i < end; i += 4 * kSelThreads) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = i + e * kSelThreads < end ? mr[i + e * kSelThreads] : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = i + e * kSelThreads;
                    if (at >= end) break;
                    const uint32_t key = mass_key(x[e]);
                    if (at - b < room) keys[at - b] = key;
                    atomicAdd(&hist[0][key >> 21], 1u);
                }
            }
        } else {
            const int above = d == 1 ? 21 : 10;
            for (int i = b + tid; i < end; i += kSelThreads) {
                const uint32_t key = key_at(i);
                if (key >> above == prefix >> above) atomicAdd(&hist[d][(key >> shift) & (bins - 1)], 1u);
            }
        }
        meet();
        // thread t: bins B - 2 t and B - 2 t - 1, the largest first
        unsigned c[2] = {0, 0};
        if (2 * tid < bins) {
            const uint32_t at = smem_addr(&hist[d][bins - 2 - 2 * tid]);
            for (int r = 0; r < parts; ++r) {
                const uint2 x = parts > 1 ? cluster_load2(cluster_addr(at, r))
                                          : *reinterpret_cast<const uint2 *>(&hist[d][bins - 2 - 2 * tid]);
                c[0] += x.y;
                c[1] += x.x;
            }
        }
        unsigned before = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) s_sum[warp] = before;
        __syncthreads();
        unsigned sums = lane < warp ? s_sum[lane] : 0u;   // of the warps before this one
        before += __reduce_add_sync(0xffffffffu, sums) - c[0] - c[1];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (before < left && left <= before + c[e]) {
                s_prefix = prefix | ((unsigned)(bins - 1 - 2 * tid - e) << shift);
                s_left = left - before;
            }
            before += c[e];
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
    }
    const uint32_t T = prefix;
    const int ties = (int)left;   // of the tokens at key T, the first `ties` are kept
    int gt = 0, eq = 0;
    for (int i = b0 + lane; i - lane < b1; i += 32) {
        const uint32_t key = i < b1 ? key_at(i) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i < b1 && key > T));
        eq += __popc(__ballot_sync(0xffffffffu, i < b1 && key == T));
    }
    if (lane == 0) { s_gt[warp] = gt; s_eq[warp] = eq; }
    __syncthreads();
    int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
    int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
    if (parts > 1) {
        if (tid == kSelThreads - 1) { s_total[0] = (unsigned)(gt_before + gt); s_total[1] = (unsigned)(eq_before + eq); }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            const uint2 x = cluster_load2(cluster_addr(smem_addr(s_total), r));
            gt_before += (int)x.x;
            eq_before += (int)x.y;
        }
        cluster_sync();   // no shared memory of another CTA is read any more
    }
    int at = n_sink + gt_before + min(eq_before, ties);
    for (int i = b0 + lane; i - lane < b1; i += 32) {
        const uint32_t key = i < b1 ? key_at(i) : 0u;
        const unsigned below = (1u << lane) - 1u;
        const unsigned be = __ballot_sync(0xffffffffu, i < b1 && key == T);
        const bool keep_it = i < b1 && (key > T || (key == T && eq_before + __popc(be & below) < ties));
        const unsigned bk = __ballot_sync(0xffffffffu, keep_it);
        if (keep_it) kr[at + __popc(bk & below)] = i;
        at += __popc(bk);
        eq_before += __popc(be);
    }
}

// CTA (x, u), the last x: unit u's mass.  The others: its rows, in one of two ways.
//
// To other pages (no destination page is the source page of the same place): the x-th,
// (x + CTAs)-th, ... chunk of rows, K and V together, in any order.
//
// In place: a team of CTAs, a cluster, for each of K and V and each slice of the channels,
// chunk after chunk.  Row j goes to position j and comes from position kept[j] >= j, so a write
// can only hit a source of the same or an earlier row: the team loads a chunk of rows,
// meets at the barrier and then stores the chunk.
constexpr int kMoveThreads = 256, kMoveUnroll = 8;

__global__ void __launch_bounds__(kMoveThreads, 4)
evict_move_kernel(fathom_pages p, int lg, int team, int slices, int4 *kp, int4 *vp, const int32_t *__restrict__ table,
                  const int32_t *__restrict__ lens, int keep, const int32_t *__restrict__ dst_table, int dst_pages,
                  const int32_t *kept, const float *mass, size_t mass_stride, float *mass_out, size_t out_stride) {
    pdl_enter();
    const int u = blockIdx.y, s = u / p.kv_heads, h = u % p.kv_heads, tid = threadIdx.x;
    const int n = min(min(max(lens[s], 0), p.max_pages << lg), keep);
    const int32_t *kr = kept + (size_t)u * keep;
    if (blockIdx.x == gridDim.x - 1) {
        const float *mr = mass + u * mass_stride;
        float *mo = mass_out + u * out_stride;
        for (int j0 = 0; j0 < n; j0 += kMoveThreads * kMoveUnroll) {
            float x[kMoveUnroll];
#pragma unroll
            for (int e = 0; e < kMoveUnroll; ++e) {
                const int j = j0 + e * kMoveThreads + tid;
                if (j < n) x[e] = mr[kr[j]];
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kMoveUnroll; ++e) {
                const int j = j0 + e * kMoveThreads + tid;
                if (j < n) mo[j] = x[e];
            }
        }
        return;
    }
    const int32_t *ta = table + (size_t)s * p.max_pages, *tb = dst_table + (size_t)s * dst_pages;
    const int64_t head = h * p.head_stride;
    const int pieces = p.D / 8;   // 16-byte pieces of a row
    // where row j of the kept ones lies and goes, in pieces; false: nowhere, or it is there already
    auto place = [&](int j, int i, int64_t &src, int64_t &dst) {
        const int a = ta[i >> lg], b = tb[j >> lg];
        if (a < 0 || a >= p.num_pages || b < 0 || b >= p.num_pages) return false;
        src = (a * p.page_stride + head + (i & (p.page_tokens - 1)) * p.token_stride) / 8;
        dst = (b * p.page_stride + head + (j & (p.page_tokens - 1)) * p.token_stride) / 8;
        return src != dst;
    };
    bool same = false;
    for (int q = tid; q < min(p.max_pages, (n + p.page_tokens - 1) >> lg); q += kMoveThreads) same |= ta[q] == tb[q];
    if (!__syncthreads_or(same)) {
        constexpr int kRowsUnroll = kMoveUnroll / 2;
        const int R = kMoveThreads / pieces, r = tid / pieces, c = tid % pieces;   // rows per step
        const int chunk = R * kRowsUnroll;
        if (r >= R) return;
        for (int j0 = blockIdx.x * chunk; j0 < n; j0 += chunk * (gridDim.x - 1)) {
            int4 x[kRowsUnroll], y[kRowsUnroll];
            int64_t to[kRowsUnroll];
            int i[kRowsUnroll];
#pragma unroll
            for (int e = 0; e < kRowsUnroll; ++e) {
                const int j = j0 + e * R + r;
                i[e] = j < n ? kr[j] : -1;
            }
#pragma unroll
            for (int e = 0; e < kRowsUnroll; ++e) {
                int64_t src;
                if (i[e] < 0 || !place(j0 + e * R + r, i[e], src, to[e])) { to[e] = -1; continue; }
                x[e] = kp[src + c];
                y[e] = vp[src + c];
            }
#pragma unroll
            for (int e = 0; e < kRowsUnroll; ++e)
                if (to[e] >= 0) { kp[to[e] + c] = x[e]; vp[to[e] + c] = y[e]; }
        }
        return;
    }
    const int which = blockIdx.x / team;   // slice which / 2 of K (even) or V
    if (which >= 2 * slices) return;
    int4 *rows = (which & 1) ? vp : kp;
    const int per = (pieces + slices - 1) / slices, c0 = (which >> 1) * per, own = min(per, pieces - c0);   // pieces
    const int R = kMoveThreads / own, c = c0 + tid % own;   // rows per step of a CTA
    const int r = tid / own < R ? tid / own + (int)(blockIdx.x % team) * R * kMoveUnroll : n;
    const int chunk = R * kMoveUnroll * team;
    int i[kMoveUnroll];   // kept[j] of the chunk to come
#pragma unroll
    for (int e = 0; e < kMoveUnroll; ++e) i[e] = r + e * R < n ? kr[r + e * R] : -1;
    for (int j0 = r; j0 - r < n; j0 += chunk) {
        int4 x[kMoveUnroll];
        int64_t to[kMoveUnroll];
#pragma unroll
        for (int e = 0; e < kMoveUnroll; ++e) {
            int64_t src;
            if (i[e] < 0 || !place(j0 + e * R, i[e], src, to[e])) { to[e] = -1; continue; }
            x[e] = rows[src + c];
        }
#pragma unroll
        for (int e = 0; e < kMoveUnroll; ++e) {
            const int j = j0 + chunk + e * R;
            i[e] = j < n ? kr[j] : -1;
        }
        if (team > 1) cluster_sync(); else __syncthreads();
#pragma unroll
        for (int e = 0; e < kMoveUnroll; ++e)
            if (to[e] >= 0) rows[to[e] + c] = x[e];
    }
}

}  // namespace

int launch_paged_evict(const fathom_pages &p, void *kp, void *vp, const int32_t *table, const int32_t *lens,
                       const float *mass, size_t mass_stride, int keep, int n_sink, int n_recent,
                       const int32_t *dst_table, int dst_pages, int32_t *kept, int32_t *lens_out, float *mass_out,
                       size_t mass_out_stride, cudaStream_t st) {
    const int units = p.seqs * p.kv_heads;
    int lg = 0;
    while ((1 << lg) < p.page_tokens) ++lg;
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;
    // CTAs per unit: 2, 4 or 8 where a part is longer than 8192 tokens, while all are resident at once
    // (8 units, 64 rows kept, the move included: 32768 tokens by one CTA 40 us, by four 18, by eight 19;
    // 8192 tokens by one 13.5, by eight 17)
    const int cap = p.max_pages * p.page_tokens;
    int parts = 1;
    while (parts < 8 && 2LL * units * parts <= 2LL * sms && cap / parts > 8192) parts *= 2;
    const int part = (cap / (kSelWarps * parts) + 32) / 32 * 32 * kSelWarps;
    const int room = part < kMaxKeys ? part : kMaxKeys;
    const size_t smem = (size_t)room * sizeof(uint32_t);
    ensure_smem(evict_select_kernel, kMaxKeys * sizeof(uint32_t));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * parts));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, parts, room, lens, mass, mass_stride, keep, n_sink,
                                       n_recent, kept, lens_out);
    if (e != cudaSuccess) return launch_failed("evict_select_kernel", e);
    // In place: CTAs of a team (8 would cost 5 us more at the start), then halves of the channels, until they fill
    // the device.  To other pages: CTAs per unit, until two waves of four per SM have work.
    const int chunk = kMoveThreads / (p.D / 8) * (kMoveUnroll / 2), chunks = (keep + chunk - 1) / chunk;
    int team = 1;
    while (team < 4 && 2LL * units * team < 2LL * sms && 2 * team <= chunks) team *= 2;
    const int slices = team == 4 && p.D >= 32 && 2LL * units * team < 2LL * sms ? 2 : 1;
    int ctas = (8 * sms + units - 1) / units;
    ctas = ctas > chunks ? chunks : ctas;
    ctas = ctas < 2 * team * slices ? 2 * team * slices : ctas;
    cfg.gridDim = dim3((unsigned)((ctas / team + 1) * team), (unsigned)units);   // and one for the mass
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    attr[1].val.clusterDim.x = (unsigned)team;
    cfg.numAttrs = team > 1 ? 2 : 1;
    // the row loads in flight need the L1, of which the selection's shared memory would leave little
    raise_func_attr((const void *)evict_move_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                    cudaSharedmemCarveoutMaxL1);
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel, p, lg, team, slices, (int4 *)kp, (int4 *)vp, table, lens, keep, dst_table,
                           dst_pages, (const int32_t *)kept, mass, mass_stride, mass_out, mass_out_stride);
    if (e != cudaSuccess) return launch_failed("evict_move_kernel", e);
    return launch_status("paged_evict");
}

}  // namespace fathom
