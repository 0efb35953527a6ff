// paged.cu -- a paged KV cache: append of new rows, and decode attention of one
// new token per sequence.
#include <cuda_bf16.h>

#include <type_traits>

#include "fathom_internal.cuh"

namespace fathom {

namespace {

__host__ __device__ inline int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// ---------------------------------------------------------------- append
// One thread per 16 bytes of a new row, K and V alike: bound by the bytes, each
// read and written once (28 us for 157 MB, launch included: 5.6 TB/s).
__global__ void __launch_bounds__(256)
paged_append_kernel(fathom_pages p, int lg, int4 *__restrict__ kp, int4 *__restrict__ vp,
                    const int32_t *__restrict__ table, const int4 *__restrict__ kn, const int4 *__restrict__ vn,
                    int total, int64_t new_token, int64_t new_head, const int32_t *__restrict__ start,
                    const int32_t *__restrict__ cu_new) {
    const unsigned pieces = p.D / 8, row = pieces * p.kv_heads;
    const unsigned long long e = (unsigned long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= (unsigned long long)total * row) return;
    const int t = (int)(e >> 32 ? e / row : (unsigned)e / row);
    const unsigned r = (unsigned)(e - (unsigned long long)t * row), h = r / pieces, c = r - h * pieces;
    int s = t, i = 0;
    if (cu_new) {
        int lo = 0, hi = p.seqs;   // the last sequence that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu_new[mid] <= t) lo = mid; else hi = mid;
        }
        s = lo;
        i = t - cu_new[s];
        if (i < 0 || t >= cu_new[s + 1]) return;
    }
    const long long pos = (long long)start[s] + i;
    if (pos < 0 || pos >= (long long)p.max_pages << lg) return;
    const int page = table[(size_t)s * p.max_pages + (pos >> lg)];
    if (page < 0 || page >= p.num_pages) return;
    const int64_t dst = (page * p.page_stride + h * p.head_stride + (pos & (p.page_tokens - 1)) * p.token_stride) / 8 + c;
    const int64_t src = (t * new_token + h * new_head) / 8 + c;
    kp[dst] = kn[src];
    vp[dst] = vn[src];
}

// ---------------------------------------------------------------- decode
// One new token per sequence over its cache: o_h = sum_i softmax_i(q_h . k_i / sqrt(D)) v_i.
// Bound by the cache's bytes, each K and V row read once for the G heads of a unit.
//
// The 64-token tiles of all units, in unit order, are dealt out to
// the CTAs in equal contiguous shares, whatever the sequences' lengths; a unit that
// several CTAs share is joined by the last of them to arrive at the unit's ticket.
// In a tile each warp takes its own 16 tokens, in 16-byte asynchronous copies to a
// ring of its own, so that warps wait for their own copies only.
//
// Products run on the tensor cores without rounding the fp32 operands: q and the
// softmax weights are sums of three pieces of the rows' type (8 or 11 bits each), and
// the 16 rows of a matrix operand hold them side by side -- for G <= 4, row 4 i + h is
// piece i of head h; for G <= 8, rows h and 8 + h are the first two pieces and a
// second instruction adds the third -- so a K or V fragment is read from shared
// memory once for all heads and pieces.
//
// Measured, 128 channels, bf16, 4 heads per unit: 32 sequences of up to 32k tokens
// (2.3 GB) 358 us, 6.4 TB/s, the copy rate 6.8; one sequence of 4096 tokens 15 us, of
// which the data take 3 (start and page numbers 2.5 us, the first data 1, two or four
// tiles 2, merge and ticket 2, the join 4: dependent accesses of about a microsecond
// each); 61 sequences of up to 3001 tokens, 64 channels, 8 heads, fp16: 34 us.
// Shares that CTAs take from a counter as they finish, instead of equal ones, gained
// nothing (359 us): CTAs finish a fifth apart, but DRAM is busy until the end.

constexpr int kDecWarps = 4, kDecThreads = 32 * kDecWarps;
// CTAs resident per SM, and stages of their rings
__host__ __device__ constexpr int dec_ctas(int d) { return d == 128 ? 2 : 3; }
constexpr int kMaxDecCtas = 3;   // the larger
__host__ __device__ constexpr int dec_stages(int d) { return d == 128 ? 3 : 4; }

__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __nv_bfloat16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __half) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_pair(uint32_t v, __nv_bfloat16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack_pair(uint32_t v, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
// Two values as three pairs of pieces, x = piece[0] + piece[1] + piece[2] up to 2^-24 |x|.
template <typename T>
__device__ __forceinline__ void split3(float x, float y, uint32_t (&piece)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        piece[i] = pack_pair(x, y, T());
        const float2 r = unpack_pair(piece[i], T());
        x -= r.x;
        y -= r.y;
    }
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct DecArgs {
    fathom_pages p;
    int lg, G, cap, logit_stride;   // logits [units][G][logit_stride], rows of whole 16 bytes
    const float *q;
    const void *kp, *vp;
    const int32_t *table, *lens;
    float *out, *part_o, *part_ml, *lse, *logits;   // shares: [CTA][2][G][D] and [CTA][2][G][2] = (m, l)
    unsigned *ticket, *group_ticket;   // of a unit's shares, by its first CTA; of a group, at its first share's place
};

// Join of a unit's shares, 32 at a time; in the place of DecSmem::o.
struct JoinSmem {
    float weight[FATHOM_MAX_G][32], m[FATHOM_MAX_G], l[FATHOM_MAX_G], f[FATHOM_MAX_G];
};

// 16-token rows of a warp's stage: K, then V; 16-byte piece c of row t lies at piece
// c ^ (t & 7), which keeps ldmatrix free of bank conflicts.
template <int kD>
struct DecSmem {
    static constexpr int kDecStages = dec_stages(kD);
    static constexpr int kTile = 16 * kDecWarps;
    static constexpr int kRowBytes = kD * 2;
    static_assert(sizeof(JoinSmem) <= sizeof(float) * kDecWarps * FATHOM_MAX_G * kD, "the join reuses o");
    alignas(128) unsigned char ring[kDecWarps][kDecStages][2][16 * kRowBytes];
    float o[kDecWarps][FATHOM_MAX_G][kD];
    float m[kDecWarps][FATHOM_MAX_G], l[kDecWarps][FATHOM_MAX_G];
    unsigned live[kDecWarps][kDecStages];   // which of the 16 tokens there are
    long long sum[kDecWarps], before;
    int part, last;
};

// Division of numbers that mostly fit 32 bits, and the first tile of CTA c's share.
__device__ __forceinline__ long long div64(long long x, long long y) {
    return (unsigned long long)(x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}
__device__ __forceinline__ long long share(long long c, long long W, long long NC) { return div64(c * W, NC); }

// Position in the order (sequence, head, tile); `tiles` of the sequence.
struct DecCursor {
    int seq, head, tile, tiles, n;
};

template <typename T, int kD, int kTwo, bool kMass>   // kTwo: G > 4
__global__ void __launch_bounds__(kDecThreads, dec_ctas(kD))
paged_attn_kernel(const DecArgs a) {
    pdl_enter();
    using Smem = DecSmem<kD>;
    constexpr int kTile = Smem::kTile, kRowBytes = Smem::kRowBytes, kDecStages = Smem::kDecStages;
    constexpr int kNT = kD / 8, kKS = kD / 16, kPieces = kD / 8;
    extern __shared__ __align__(128) unsigned char dec_smem[];
    Smem &sm = *reinterpret_cast<Smem *>(dec_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const fathom_pages &p = a.p;
    const int D = p.D, H = p.kv_heads, G = a.G;
    auto length = [&](int s) { return min(max(a.lens[s], 0), a.cap); };
    auto tiles_of = [&](int n) { return (n + kTile - 1) / kTile; };

    // ---- all tiles, this CTA's share of them, and the sequence it starts in
    long long W = 0, first = 0, w0 = 0, w1 = 0, NC = 1;   // first: the sequence's first tile
    const long long cta = blockIdx.x;
    int seq0 = 0;
    auto split = [&](long long sum) {
        W = sum * H;
        // every CTA there is when each gets four tiles or more, else fewer CTAs and longer shares, down to
        // one per SM: a share less to join costs less than a tile more (one 4k sequence: 304 shares of
        // two tiles 15.6 us, 152 of four 11.6 us)
        NC = min((long long)gridDim.x, max(1LL, max(W / 4, min(W, (long long)gridDim.x / dec_ctas(kD)))));
        if (cta < NC) { w0 = share(cta, W, NC); w1 = share(cta + 1, W, NC); }
    };
    // inclusive sums over the lanes; the lane whose tiles hold w0, given the sum before them
    auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    if (p.seqs <= 128) {   // every warp for itself, four sequences per lane, one round of loads
        int t[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e] = 4 * lane + e < p.seqs ? tiles_of(length(4 * lane + e)) : 0;
            sum += t[e];
        }
        const long long upto = scan(sum);
        split(__shfl_sync(0xffffffffu, upto, 31));
        const unsigned hit = __ballot_sync(0xffffffffu, upto * H > w0);
        const int f = hit ? __ffs(hit) - 1 : 0;
        long long before = (upto - sum) * H;
        int s = 4 * lane;
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (s == 4 * lane + e && before + (long long)t[e] * H <= w0) { before += (long long)t[e] * H; ++s; }
        seq0 = __shfl_sync(0xffffffffu, s, f);
        first = __shfl_sync(0xffffffffu, before, f);
    } else {
        // every thread the sum of a contiguous part; the part that holds w0 is searched by every warp
        const int per = (p.seqs + kDecThreads - 1) / kDecThreads;
        long long mine = 0;
        for (int s = tid * per; s < min((tid + 1) * per, p.seqs); ++s) mine += tiles_of(length(s));
        const long long upto = scan(mine);
        if (lane == 31) sm.sum[warp] = upto;
        __syncthreads();
        long long sum = 0, before = upto - mine;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            if (w < warp) before += sm.sum[w];
            sum += sm.sum[w];
        }
        split(sum);
        if (before * H <= w0 && w0 < (before + mine) * H) { sm.part = tid; sm.before = before; }
        __syncthreads();
        if (w0 < w1) {
            before = sm.before;
            for (int s0 = sm.part * per;; s0 += 32) {
                const long long x = s0 + lane < p.seqs ? tiles_of(length(s0 + lane)) : 0, end = before + scan(x);
                const unsigned hit = __ballot_sync(0xffffffffu, end * H > w0);
                if (hit || s0 >= p.seqs) {
                    const int f = hit ? __ffs(hit) - 1 : 0;
                    seq0 = min(s0 + f, p.seqs - 1);
                    first = __shfl_sync(0xffffffffu, (end - x) * H, f);
                    break;
                }
                before = __shfl_sync(0xffffffffu, end, 31);
            }
        }
    }
    // units of empty sequences
    for (int u = blockIdx.x; u < p.seqs * H; u += gridDim.x)
        if (length(u / H) == 0)
            for (int e = tid; e < G * D; e += kDecThreads) a.out[(size_t)u * G * D + e] = 0.0f;
    if (w0 >= w1) return;
    DecCursor at;   // the tile being computed
    at.seq = seq0;
    at.n = length(at.seq);
    at.tiles = tiles_of(at.n);
    at.head = (int)div64(w0 - first, at.tiles);
    at.tile = (int)(w0 - first - (long long)at.head * at.tiles);
    auto advance = [&](DecCursor &x) {   // true when the unit changes; past the last sequence it stays there
        if (x.seq >= p.seqs || ++x.tile < x.tiles) return false;
        x.tile = 0;
        if (++x.head == H) {
            x.head = 0;
            do {
                if (++x.seq >= p.seqs) { x.n = 0; x.tiles = 1; break; }
                x.n = length(x.seq);
                x.tiles = tiles_of(x.n);
            } while (x.tiles == 0);
        }
        return true;
    };

    // ---- loads: lane t < 16 looks up the page of token t, ahead of its tile's copies
    const char *kb = (const char *)a.kp, *vb = (const char *)a.vp;
    auto lookup = [&](const DecCursor &x) {
        const int i = x.tile * kTile + warp * 16 + (lane & 15);
        int page = -1;
        if (x.seq < p.seqs && i < x.n) {
            page = __ldg(a.table + (size_t)x.seq * p.max_pages + (i >> a.lg));
            if (page >= p.num_pages) page = -1;
        }
        return page;
    };
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp]);
    constexpr uint32_t kHalf = 16 * kRowBytes;
    const int col = lane % kPieces, row0 = lane / kPieces;   // this lane's 16-byte piece, its first row
    constexpr int kRowsPer = 32 / kPieces;
    const int64_t step = 2 * kRowsPer * p.token_stride;
    auto issue = [&](int st, const DecCursor &x, int pid) {   // the copies of a tile whose pages are known
        const unsigned ok = __ballot_sync(0xffffffffu, pid >= 0) & 0xffffu;
        if (lane == 0) sm.live[warp][st] = ok;
        const int64_t at_head = x.head * p.head_stride;
        const int slot0 = (x.tile * kTile + warp * 16) & (p.page_tokens - 1);
        uint32_t dst = ring + st * 2 * kHalf + row0 * kRowBytes;
        if (p.page_tokens >= 16) {   // the 16 tokens lie in one page, the live ones first
            const int page = __shfl_sync(0xffffffffu, pid, 0), n = col * 8 < D ? __popc(ok) : 0;
            int64_t off = page >= 0 ? 2 * (page * p.page_stride + at_head + (slot0 + row0) * p.token_stride) + col * 16 : 0;
#pragma unroll
            for (int i = 0; i < 16 / kRowsPer; ++i) {
                const int t = row0 + i * kRowsPer, bytes = t < n ? 16 : 0;
                const uint32_t to = dst + i * kRowsPer * kRowBytes + ((col ^ (t & 7)) << 4);
                const char *ks = t < n ? kb + off : kb, *vs = t < n ? vb + off : vb;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(ks), "r"(bytes) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + kHalf), "l"(vs), "r"(bytes) : "memory");
                off += step;
            }
            return;
        }
#pragma unroll 1
        for (int i = 0; i < 16 / kRowsPer; ++i) {
            const int t = row0 + i * kRowsPer;
            const int page = __shfl_sync(0xffffffffu, pid, t);
            const int slot = (slot0 + t) & (p.page_tokens - 1);
            const bool live = page >= 0 && col * 8 < D;
            const int64_t off = live ? 2 * (page * p.page_stride + at_head + slot * p.token_stride) + col * 16 : 0;
            const uint32_t to = dst + i * kRowsPer * kRowBytes + ((col ^ (t & 7)) << 4);
            const int bytes = live ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(kb + off), "r"(bytes) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + kHalf), "l"(vb + off), "r"(bytes) : "memory");
        }
    };
    const int count = (int)(w1 - w0);
    DecCursor ld = at;
    int pid;
    {   // the first stages: every page looked up before the first copy
        DecCursor cs[kDecStages - 1];
        int ids[kDecStages - 1];
#pragma unroll
        for (int st = 0; st < kDecStages - 1; ++st) {
            cs[st] = ld;
            ids[st] = lookup(ld);
            advance(ld);
        }
        pid = lookup(ld);
#pragma unroll
        for (int st = 0; st < kDecStages - 1; ++st) {
            if (st < count) issue(st, cs[st], ids[st]);
            cp_async_commit();
        }
    }

    const int head = kTwo ? r : (r & 3);   // this lane's head in score and output fragments
    const float to_log2 = 1.4426950408889634f / sqrtf((float)D);
    uint32_t qa[kKS][4], qb[kTwo ? kKS : 1][2];
    float unscale = 1.0f, m = -CUDART_INF_F, l = 0.0f, o[kNT][4];
    // fp16 weights are kept 2^12 larger, so that their pieces stay clear of the subnormals
    constexpr float kUp = sizeof(T) == 2 && std::is_same<T, __half>::value ? 12.0f : 0.0f;
    bool fresh = true;
    long long unit_w0 = w0 - at.tile;   // index of the unit's first tile

    for (int i = 0; i < count; ++i) {
        if (fresh) {   // a new unit: its queries in pieces, empty sums
            fresh = false;
            const float *qr = a.q + ((size_t)(at.seq * H + at.head) * G + head) * D;
            float2 x[kKS][2];
            float big = 0.0f;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = ks * 16 + 2 * c + 8 * e;
                    x[ks][e] = head < G && k < D ? make_float2(__ldg(qr + k), __ldg(qr + k + 1)) : make_float2(0.0f, 0.0f);
                    x[ks][e].x *= to_log2;
                    x[ks][e].y *= to_log2;
                    big = fmaxf(big, fmaxf(fabsf(x[ks][e].x), fabsf(x[ks][e].y)));
                }
            unscale = 1.0f;
            if (std::is_same<T, __half>::value) {   // a power of two that brings the largest to about 2^12
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                if (big > 0.0f && big < CUDART_INF_F) {
                    const int e = min(max(ilogbf(big) - 12, -126), 126);
                    unscale = ldexpf(1.0f, e);
                    const float up = ldexpf(1.0f, -e);
#pragma unroll
                    for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                        for (int f = 0; f < 2; ++f) { x[ks][f].x *= up; x[ks][f].y *= up; }
                }
            }
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t pc[3];
                    split3<T>(x[ks][e].x, x[ks][e].y, pc);
                    if (kTwo) {
                        qa[ks][2 * e] = pc[0];
                        qa[ks][2 * e + 1] = pc[1];
                        qb[kTwo ? ks : 0][e] = pc[2];
                    } else {
                        qa[ks][2 * e] = r < 4 ? pc[0] : pc[1];
                        qa[ks][2 * e + 1] = r < 4 ? pc[2] : 0u;
                    }
                }
            m = -CUDART_INF_F;
            l = 0.0f;
#pragma unroll
            for (int j = 0; j < kNT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        }
        const int st = i % kDecStages;
        {   // the copies two tiles ahead, into the stage that was read last
            if (i + kDecStages - 1 < count) {
                issue((i + kDecStages - 1) % kDecStages, ld, pid);
                advance(ld);
                pid = lookup(ld);
            }
            cp_async_commit();
            cp_async_wait<kDecStages - 1>();
            __syncwarp();
        }
        {
            const uint32_t kt = ring + st * 2 * kHalf, vt = kt + kHalf;
            const unsigned ok = sm.live[warp][st];
            // scores of 16 tokens: columns 2 c, 2 c + 1 of two 8-token products
            float s[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                // matrices: tokens 0-7 and 8-15 of channels 0-7 and 8-15 of this step
                const int t = (lane & 7) + ((lane >> 4) << 3), pc = 2 * ks + ((lane >> 3) & 1);
                uint32_t kf[4];
                ldmatrix4(kf, kt + t * kRowBytes + ((pc ^ (t & 7)) << 4));
                mma16816(s[0], qa[ks], kf[0], kf[1], T());
                mma16816(s[1], qa[ks], kf[2], kf[3], T());
                if (kTwo) {
                    const uint32_t third[4] = {qb[kTwo ? ks : 0][0], 0u, qb[kTwo ? ks : 0][1], 0u};
                    mma16816(s[0], third, kf[0], kf[1], T());
                    mma16816(s[1], third, kf[2], kf[3], T());
                }
            }
            float x[2][2], top = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[j][e] + s[j][2 + e];
                    if (!kTwo) v += __shfl_xor_sync(0xffffffffu, v, 16);
                    v *= unscale;
                    x[j][e] = (ok >> (8 * j + 2 * c + e)) & 1u ? v : -CUDART_INF_F;
                    top = fmaxf(top, x[j][e]);
                }
            if (kMass) {
                const int i0 = at.tile * kTile + warp * 16 + 2 * c;
                float *lr = a.logits + ((size_t)(at.seq * H + at.head) * G + head) * a.logit_stride;
                if (head < G && (kTwo || r < 4)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (i0 + 8 * j < at.n) *reinterpret_cast<float2 *>(lr + i0 + 8 * j) = make_float2(x[j][0], x[j][1]);
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (__any_sync(0xffffffffu, top > m)) {
                const float mn = fmaxf(m, top);
                const float f = m == -CUDART_INF_F ? 0.0f : exp2_fast(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] *= f;
            }
            const float shift = kUp - (m == -CUDART_INF_F ? 0.0f : m);
            uint32_t pa[4], pb[4] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p0 = exp2_fast(x[j][0] + shift), p1 = exp2_fast(x[j][1] + shift);
                l += p0 + p1;
                uint32_t pc[3];
                split3<T>(p0, p1, pc);
                if (kTwo) {
                    pa[2 * j] = pc[0];
                    pa[2 * j + 1] = pc[1];
                    pb[2 * j] = pc[2];
                } else {
                    pa[2 * j] = r < 4 ? pc[0] : pc[1];
                    pa[2 * j + 1] = r < 4 ? pc[2] : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < kNT; j += 2) {
                // matrices: tokens 0-7 and 8-15 of channels 8 j .. 8 j + 7 and of the next eight
                const int t = lane & 15, pc = j + (lane >> 4);
                uint32_t vf[4];
                ldmatrix4_trans(vf, vt + t * kRowBytes + ((pc ^ (t & 7)) << 4));
                mma16816(o[j], pa, vf[0], vf[1], T());
                mma16816(o[j + 1], pa, vf[2], vf[3], T());
                if (kTwo) {
                    mma16816(o[j], pb, vf[0], vf[1], T());
                    mma16816(o[j + 1], pb, vf[2], vf[3], T());
                }
            }
        }
        __syncwarp();   // the stage is read before its next copies start

        // ---- end of the unit, or of this CTA's share of it
        const int unit = at.seq * H + at.head, tiles = at.tiles;
        const bool turn = advance(at);
        if (!turn && i + 1 < count) continue;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const bool owner = head < G && (kTwo || r < 4);
        if (owner && c == 0) { sm.m[warp][head] = m; sm.l[warp][head] = l; }
        __syncthreads();
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, owner ? sm.m[w][head] : -CUDART_INF_F);
        const float f = m == -CUDART_INF_F ? 0.0f : exp2_fast(m - M);
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = o[j][e] + o[j][2 + e];
                if (!kTwo) v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (owner) sm.o[warp][head][8 * j + 2 * c + e] = v * f;
            }
        __syncthreads();
        // the CTA's state of each head: (m, l, o), to `out` when the unit is all here
        const long long c_first = div64((unit_w0 + 1) * NC - 1, W), c_last = div64((unit_w0 + tiles) * NC - 1, W);
        const bool whole = c_first == c_last;
        const size_t slot = 2 * cta + (w0 < unit_w0 ? 1 : 0);
        constexpr int kAll = (kTwo ? FATHOM_MAX_G : 4) * kD / 4;   // four channels at a time
        constexpr int kVecs = (kAll + kDecThreads - 1) / kDecThreads;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = 4 * (tid + k * kDecThreads);
            if (e < G * D) {
                const int h = e / D, d = e - h * D;   // D is a multiple of 8: the four lie in one head
                float Mh = -CUDART_INF_F, L = 0.0f;
#pragma unroll
                for (int w = 0; w < kDecWarps; ++w) Mh = fmaxf(Mh, sm.m[w][h]);
                float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kDecWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][h][d]);
                    O.x += v.x; O.y += v.y; O.z += v.z; O.w += v.w;
                    L += sm.l[w][h] * (sm.m[w][h] == -CUDART_INF_F ? 0.0f : exp2_fast(sm.m[w][h] - Mh));   // a NaN stays
                }
                if (whole) {
                    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                    float *ou = a.out + (size_t)unit * G * D + e;
                    ou[0] = O.x * inv; ou[1] = O.y * inv; ou[2] = O.z * inv; ou[3] = O.w * inv;
                    if (kMass && d == 0) a.lse[(size_t)unit * G + h] = L == 0.0f ? 0.0f : Mh + log2f(L) - kUp;
                } else {
                    *reinterpret_cast<float4 *>(a.part_o + slot * G * D + e) = O;
                    if (d == 0) *reinterpret_cast<float2 *>(a.part_ml + (slot * G + h) * 2) = make_float2(Mh, L);
                }
            }
        }
        if (!whole) {
            // The last share to arrive joins them, in their order.  Of more than 32 shares, groups of
            // kGroup are joined first, each by its last share and into its first one's place, so that no
            // CTA reads hundreds (one unit of 131072 tokens, 8 heads, 304 shares: 121 -> 33 us)
            constexpr int kGroup = 16;
            const int before = share(c_first, W, NC) < unit_w0;   // only the first share can be a CTA's second
            auto slot_of = [&](long long x) { return (size_t)(2 * x + (x == c_first ? before : 0)); };
            const int shares = (int)(c_last - c_first) + 1;
            long long x_first = c_first;   // what is joined: shares x_first, x_first + every, ...
            int every = 1, n = shares;
            unsigned *ticket = a.ticket + c_first;   // of all units that it holds a share of, one goes on behind it
            bool final = shares <= 32;
            if (!final) {
                x_first += (cta - c_first) / kGroup * kGroup;
                n = (int)min((long long)kGroup, c_last - x_first + 1);
                ticket = a.group_ticket + slot_of(x_first);
            }
            for (;;) {
                __syncthreads();
                if (tid == 0) {
                    __threadfence();   // the CTA's state before its ticket
                    sm.last = atomicAdd(ticket, 1u) == (unsigned)(n - 1) ? 1 : 0;
                    __threadfence();
                }
                __syncthreads();
                if (!sm.last) break;
                if (tid == 0) *ticket = 0u;
                JoinSmem &jn = *reinterpret_cast<JoinSmem *>(sm.o);
                if (tid < G) { jn.m[tid] = -CUDART_INF_F; jn.l[tid] = 0.0f; }
                constexpr int kBatch = kD == 64 ? 8 : (kTwo ? 6 : 16);
                float4 acc[kVecs];
#pragma unroll
                for (int k = 0; k < kVecs; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int x0 = 0; x0 < n; x0 += 32) {
                    const int nx = min(n - x0, 32);
                    float4 v[kVecs][kBatch];
                    auto fetch = [&](int x) {   // shares x0 + x and on, kBatch loads in flight per vector
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int e = 4 * (tid + k * kDecThreads);
#pragma unroll
                            for (int y = 0; y < kBatch; ++y)
                                if (e < G * D && x + y < nx)
                                    v[k][y] = __ldcg(reinterpret_cast<const float4 *>(
                                        a.part_o + slot_of(x_first + (x0 + x + y) * every) * G * D + e));
                        }
                    };
                    constexpr int kHeads = kTwo ? 2 : 1;   // of a warp
                    float2 mls[kHeads];
#pragma unroll
                    for (int i = 0; i < kHeads; ++i) {
                        const int h = warp + i * kDecWarps;
                        mls[i] = make_float2(-CUDART_INF_F, 0.0f);
                        if (lane < nx && h < G)
                            mls[i] = __ldcg(reinterpret_cast<const float2 *>(
                                a.part_ml + (slot_of(x_first + (x0 + lane) * every) * G + h) * 2));
                    }
                    fetch(0);   // under way while the weights are computed
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < kHeads; ++i) {
                        const int h = warp + i * kDecWarps;
                        if (h >= G) break;
                        const float2 ml = mls[i];
                        float mx = ml.x;
#pragma unroll
                        for (int o2 = 16; o2; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
                        const float old = jn.m[h], mn = fmaxf(old, mx);
                        const float wt = ml.x == -CUDART_INF_F ? 0.0f : exp2_fast(ml.x - mn);
                        float ls = ml.y * wt;
#pragma unroll
                        for (int o2 = 16; o2; o2 >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o2);
                        jn.weight[h][lane] = wt;
                        __syncwarp();
                        if (lane == 0) {
                            const float fo = old == -CUDART_INF_F ? 0.0f : exp2_fast(old - mn);
                            jn.f[h] = fo;
                            jn.l[h] = jn.l[h] * fo + ls;
                            jn.m[h] = mn;
                        }
                    }
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < kVecs; ++k) {
                        const int e = 4 * (tid + k * kDecThreads);
                        const float fo = e < G * D ? jn.f[e / D] : 0.0f;
                        acc[k].x *= fo; acc[k].y *= fo; acc[k].z *= fo; acc[k].w *= fo;
                    }
#pragma unroll 1
                    for (int x = 0; x < nx; x += kBatch) {
                        if (x) fetch(x);
#pragma unroll
                        for (int k = 0; k < kVecs; ++k) {
                            const int e = 4 * (tid + k * kDecThreads);
#pragma unroll
                            for (int y = 0; y < kBatch; ++y)
                                if (e < G * D && x + y < nx) {
                                    const float wt = jn.weight[e / D][x + y];
                                    acc[k].x = fmaf(v[k][y].x, wt, acc[k].x);
                                    acc[k].y = fmaf(v[k][y].y, wt, acc[k].y);
                                    acc[k].z = fmaf(v[k][y].z, wt, acc[k].z);
                                    acc[k].w = fmaf(v[k][y].w, wt, acc[k].w);
                                }
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int e = 4 * (tid + k * kDecThreads);
                    if (e >= G * D) continue;
                    const int h = e / D;
                    const float L = jn.l[h];
                    if (final) {
                        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                        float *ou = a.out + (size_t)unit * G * D + e;
                        ou[0] = acc[k].x * inv; ou[1] = acc[k].y * inv; ou[2] = acc[k].z * inv; ou[3] = acc[k].w * inv;
                        if (kMass && e % D == 0) a.lse[(size_t)unit * G + h] = L == 0.0f ? 0.0f : jn.m[h] + log2f(L) - kUp;
                    } else {
                        const size_t to = slot_of(x_first);
                        *reinterpret_cast<float4 *>(a.part_o + to * G * D + e) = acc[k];
                        if (e % D == 0) *reinterpret_cast<float2 *>(a.part_ml + (to * G + h) * 2) = make_float2(jn.m[h], L);
                    }
                }
                if (final) break;
                x_first = c_first;
                every = kGroup;
                n = (shares + kGroup - 1) / kGroup;
                ticket = a.ticket + c_first;
                final = true;
            }
        }
        fresh = true;
        unit_w0 += tiles;
        __syncthreads();   // the merge buffers are free again
    }
    cp_async_wait<0>();
}

// mass[i] += sum_h 2^(logit_h(i) - lse_h), from the logits that the attention left; four
// tokens per thread.
__global__ void __launch_bounds__(256)
paged_mass_kernel(fathom_pages p, int cap, int stride, int G, const int32_t *__restrict__ lens,
                  const float *__restrict__ logits, const float *__restrict__ lse, float *__restrict__ mass,
                  size_t mass_stride) {
    pdl_enter();
    const int u = blockIdx.y, n = min(max(lens[u / p.kv_heads], 0), cap);
    float *mr = mass + u * mass_stride;
    const bool vec = (((uintptr_t)mr) & 15) == 0;
    for (int i = 4 * (blockIdx.x * 256 + threadIdx.x); i < n; i += 4 * 256 * gridDim.x) {
        float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int g = 0; g < G; ++g) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(logits + ((size_t)u * G + g) * stride + i));
            const float z = __ldcg(lse + (size_t)u * G + g);
            w.x += exp2_fast(x.x - z); w.y += exp2_fast(x.y - z); w.z += exp2_fast(x.z - z); w.w += exp2_fast(x.w - z);
        }
        if (vec && i + 3 < n) {
            float4 v = *reinterpret_cast<float4 *>(mr + i);
            v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
            *reinterpret_cast<float4 *>(mr + i) = v;
        } else {
            const float v[4] = {w.x, w.y, w.z, w.w};
            for (int e = 0; e < 4; ++e)
                if (i + e < n) mr[i + e] += v[e];
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T, int kD, int kTwo, bool kMass>
cudaError_t launch_dec(const DecArgs &a, int ctas, cudaStream_t st) {
    const size_t smem = sizeof(DecSmem<kD>);
    static_assert(dec_ctas(kD) * (sizeof(DecSmem<kD>) + 1024) <= 228 * 1024, "resident CTAs");
    ensure_smem(paged_attn_kernel<T, kD, kTwo, kMass>, smem);
    return launch_pdl(paged_attn_kernel<T, kD, kTwo, kMass>, dim3(ctas), dim3(kDecThreads), smem, st, a);
}
template <typename T, int kD>
cudaError_t launch_dec_form(const DecArgs &a, int ctas, cudaStream_t st) {
    if (a.G > 4) return a.logits ? launch_dec<T, kD, 1, true>(a, ctas, st) : launch_dec<T, kD, 1, false>(a, ctas, st);
    return a.logits ? launch_dec<T, kD, 0, true>(a, ctas, st) : launch_dec<T, kD, 0, false>(a, ctas, st);
}

}  // namespace

int launch_paged_append(const fathom_pages &p, void *kp, void *vp, const int32_t *table, const void *kn,
                        const void *vn, int total, int64_t new_token, int64_t new_head, const int32_t *start,
                        const int32_t *cu_new, cudaStream_t st) {
    const long long items = (long long)total * p.kv_heads * (p.D / 8);
    if ((items + 255) / 256 > 0x7fffffffLL) { set_error("paged_append: too many rows for one launch"); return FATHOM_EINVAL; }
    paged_append_kernel<<<(unsigned)((items + 255) / 256), 256, 0, st>>>(
        p, log2_of(p.page_tokens), (int4 *)kp, (int4 *)vp, table, (const int4 *)kn, (const int4 *)vn, total, new_token,
        new_head, start, cu_new);
    return launch_status("paged_append_kernel");
}

PagedWorkspace paged_workspace_layout(const fathom_pages &p, int G, bool mass) {
    PagedWorkspace w;
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;
    const size_t units = (size_t)p.seqs * p.kv_heads, rows = units * G;
    w.ctas = dec_ctas(p.D <= 64 ? 64 : 128) * sms;   // resident at once
    // Tickets, which are zero between calls, take the same bytes whatever the call's sizes: a buffer made for the
    // largest of several calls serves them all.  (A ticket per unit, with the data behind the last one, put a
    // smaller call's partial results into a larger one's tickets.)
    w.ticket_off = 0;
    w.lse_off = align256(3 * (size_t)kMaxDecCtas * sms * sizeof(uint32_t));
    w.part_off = align256(w.lse_off + (mass ? rows * sizeof(float) : 0));
    w.ml_off = align256(w.part_off + (size_t)w.ctas * 2 * G * p.D * sizeof(float));
    w.logit_off = align256(w.ml_off + (size_t)w.ctas * 2 * G * 2 * sizeof(float));
    w.total = align256(w.logit_off + (mass ? rows * (((size_t)p.max_pages * p.page_tokens + 3) / 4 * 4) * sizeof(float) : 0));
    return w;
}

int launch_paged_attn(const fathom_pages &p, int G, const float *q, const void *kp, const void *vp,
                      const int32_t *table, const int32_t *lens, float *out, float *mass, size_t mass_stride,
                      void *ws, cudaStream_t st) {
    const PagedWorkspace w = paged_workspace_layout(p, G, mass != nullptr);
    DecArgs a;
    a.p = p;
    a.lg = log2_of(p.page_tokens);
    a.G = G;
    a.cap = p.max_pages * p.page_tokens;
    a.logit_stride = (a.cap + 3) / 4 * 4;
    a.q = q; a.kp = kp; a.vp = vp; a.table = table; a.lens = lens; a.out = out;
    a.ticket = (unsigned *)((char *)ws + w.ticket_off);
    a.group_ticket = a.ticket + (w.lse_off - w.ticket_off) / sizeof(unsigned) / 3;
    a.part_o = (float *)((char *)ws + w.part_off);
    a.part_ml = (float *)((char *)ws + w.ml_off);
    a.lse = mass ? (float *)((char *)ws + w.lse_off) : nullptr;
    a.logits = mass ? (float *)((char *)ws + w.logit_off) : nullptr;
    cudaError_t e;
    if (p.dtype == FATHOM_BF16)
        e = p.D <= 64 ? launch_dec_form<__nv_bfloat16, 64>(a, w.ctas, st) : launch_dec_form<__nv_bfloat16, 128>(a, w.ctas, st);
    else
        e = p.D <= 64 ? launch_dec_form<__half, 64>(a, w.ctas, st) : launch_dec_form<__half, 128>(a, w.ctas, st);
    if (e != cudaSuccess) return launch_failed("paged_attn_kernel", e);
    if (mass) {
        const int units = p.seqs * p.kv_heads, want = (a.cap + 1023) / 1024, most = (w.ctas * 8 + units - 1) / units;
        e = launch_pdl(paged_mass_kernel, dim3(want < most ? want : most, units), dim3(256), 0, st, p, a.cap, a.logit_stride, G,
                       lens, (const float *)a.logits, (const float *)a.lse, mass, mass_stride);
        if (e != cudaSuccess) return launch_failed("paged_mass_kernel", e);
    }
    return launch_status("paged_attn");
}

}  // namespace fathom
