// evict.cu -- eviction from a paged KV cache by accumulated attention weight:
// the kept set of every unit, then its rows and mass moved together.
// Measured, 128 channels, bf16: 256 units of up to 16k tokens cut back to 4096 each
// 26 us (the kept sets) + 167 us (the move to other pages: 1.0 GB in rows of 256 bytes,
// 2 KB apart, 6.0 TB/s); 8 units of 8192 tokens cut to 2048 14 + 7 us.  In place the
// move takes 205 and 17 us: it has an order to keep.  Tried for that order: twice the
// loads in flight from a pipelined loop (220 us), bulk copies through shared memory
// (210 us; 76 us for the 8 units).
#include "fathom_internal.cuh"

namespace fathom {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;

// The mass as an unsigned key of the same order; a NaN is the largest.
__device__ __forceinline__ uint32_t mass_key(float x) { return x != x ? 0xffffffffu : order_f32(x); }

// One CTA per unit.  The key of the last kept token comes from four histograms
// of 8 bits (each over the keys that agree with the digits found so far); then
// each warp counts a contiguous part's tokens above and at that key, the counts
// are scanned, and the kept tokens are written in ascending order.
__global__ void __launch_bounds__(kSelThreads, 2)
evict_select_kernel(fathom_pages p, const int32_t *__restrict__ lens, const float *__restrict__ mass,
                    size_t mass_stride, int keep, int n_sink, int n_recent, int32_t *__restrict__ kept,
                    int32_t *__restrict__ lens_out) {
    pdl_enter();
    __shared__ unsigned hist[256];
    __shared__ unsigned s_prefix, s_left;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    const int u = blockIdx.x, s = u / p.kv_heads, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = min(max(lens[s], 0), p.max_pages * p.page_tokens);
    int32_t *kr = kept + (size_t)u * keep;
    if (u % p.kv_heads == 0 && tid == 0) lens_out[s] = min(n, keep);
    if (n <= keep) {
        for (int j = tid; j < keep; j += kSelThreads) kr[j] = j < n ? j : -1;
        return;
    }
    const float *mr = mass + (size_t)u * mass_stride;
    const int lo = n_sink, hi = n - n_recent, want = keep - n_sink - n_recent;
    for (int j = tid; j < n_sink; j += kSelThreads) kr[j] = j;
    for (int j = tid; j < n_recent; j += kSelThreads) kr[keep - n_recent + j] = hi + j;
    if (want == 0) return;
    if (tid == 0) { s_prefix = 0; s_left = (unsigned)want; }
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const unsigned prefix = s_prefix;
        const unsigned mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i = lo + tid; i < hi; i += kSelThreads) {
            const uint32_t key = mass_key(mr[i]);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {   // lane l: bins 255 - 8 l down to 248 - 8 l
            unsigned c[8], sum = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) { c[b] = hist[255 - 8 * lane - b]; sum += c[b]; }
            unsigned before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned x = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += x;
            }
            before -= sum;
            const unsigned left = s_left;
            __syncwarp();
            if (before < left && left <= before + sum) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (before < left && left <= before + c[b]) {
                        s_prefix = prefix | ((unsigned)(255 - 8 * lane - b) << shift);
                        s_left = left - before;
                    }
                    before += c[b];
                }
            }
        }
        __syncthreads();
    }
    const uint32_t T = s_prefix;
    const int ties = (int)s_left;   // of the tokens at key T, the first `ties` are kept
    const int seg = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int b0 = min(lo + warp * seg, hi), b1 = min(b0 + seg, hi);
    int gt = 0, eq = 0;
    for (int i = b0 + lane; i - lane < b1; i += 32) {
        const uint32_t key = i < b1 ? mass_key(mr[i]) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i < b1 && key > T));
        eq += __popc(__ballot_sync(0xffffffffu, i < b1 && key == T));
    }
    if (lane == 0) { s_gt[warp] = gt; s_eq[warp] = eq; }
    __syncthreads();
    int at = n_sink, eq_before = 0;
    for (int w = 0; w < warp; ++w) {
        at += s_gt[w] + min(max(ties - eq_before, 0), s_eq[w]);
        eq_before += s_eq[w];
    }
    for (int i = b0 + lane; i - lane < b1; i += 32) {
        const uint32_t key = i < b1 ? mass_key(mr[i]) : 0u;
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
// In place: channels of slice x / 2 of K (x even) or V, x < 2 slices, chunk after chunk.
// Row j goes to position j and comes from position kept[j] >= j, so a write can only
// hit a source of the same or an earlier row: the CTA loads a chunk of rows, meets at
// the barrier and then stores the chunk.
constexpr int kMoveThreads = 256, kMoveUnroll = 8;

__global__ void __launch_bounds__(kMoveThreads, 4)
evict_move_kernel(fathom_pages p, int lg, int slices, int4 *kp, int4 *vp, const int32_t *__restrict__ table,
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
    if ((int)blockIdx.x >= 2 * slices) return;
    int4 *rows = (blockIdx.x & 1) ? vp : kp;
    const int per = (pieces + slices - 1) / slices;   // pieces of a slice
    const int c0 = (blockIdx.x >> 1) * per, pc = min(per, pieces - c0);
    if (pc <= 0) return;
    const int R = kMoveThreads / pc, r = tid / pc, c = c0 + tid % pc;
    for (int j0 = 0; j0 < n; j0 += R * kMoveUnroll) {
        int4 x[kMoveUnroll];
        int64_t to[kMoveUnroll];
#pragma unroll
        for (int e = 0; e < kMoveUnroll; ++e) {
            const int j = j0 + e * R + r;
            int64_t src;
            if (r >= R || j >= n || !place(j, kr[j], src, to[e])) { to[e] = -1; continue; }
            x[e] = rows[src + c];
        }
        __syncthreads();
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
    cudaError_t e = launch_pdl(evict_select_kernel, dim3(units), dim3(kSelThreads), 0, st, p, lens, mass, mass_stride,
                               keep, n_sink, n_recent, kept, lens_out);
    if (e != cudaSuccess) { set_error("evict_select_kernel: %s", cudaGetErrorString(e)); return FATHOM_ECUDA; }
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;
    int slices = 1;   // of a row, 32 bytes at least, until the CTAs fill the device (in place)
    while (2 * slices <= p.D / 16 && 2LL * units * slices < 2LL * sms) slices *= 2;
    // CTAs per unit: those, or more until two waves of four per SM have work (to other pages)
    const int chunk = kMoveThreads / (p.D / 8) * (kMoveUnroll / 2), chunks = (keep + chunk - 1) / chunk;
    int ctas = (8 * sms + units - 1) / units;
    ctas = ctas > chunks ? chunks : ctas;
    ctas = ctas < 2 * slices ? 2 * slices : ctas;
    e = launch_pdl(evict_move_kernel, dim3(ctas + 1, units), dim3(kMoveThreads), 0, st, p, lg, slices,
                   (int4 *)kp, (int4 *)vp, table, lens, keep, dst_table, dst_pages, (const int32_t *)kept, mass,
                   mass_stride, mass_out, mass_out_stride);
    if (e != cudaSuccess) { set_error("evict_move_kernel: %s", cudaGetErrorString(e)); return FATHOM_ECUDA; }
    return launch_status("paged_evict");
}

}  // namespace fathom
