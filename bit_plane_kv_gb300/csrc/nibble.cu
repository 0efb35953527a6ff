// nibble.cu -- decode attention of one new token per sequence over a paged cache held in
// 4 bits: o_h = sum_i softmax_i(q_h . k_i / sqrt(D)) v_i with k, v = (c - 7.5) a / 8.
#include "nibble.cuh"
#include "shares.cuh"

namespace fathom {

namespace {

// Bound by the cache's bytes, 9 D / 8 per token and KV head, as long as a block of 16 tokens
// costs fewer instructions than the SM issues while its 18 D bytes arrive (392 for D = 128).
//
// Equal shares of tiles of 128 or 256 tokens per CTA (shares.cuh); in a tile each warp takes
// two or four blocks of 16 tokens, in 16-byte asynchronous copies to a ring of its own, so
// that warps wait for their own copies only.
//
// Products run on the tensor cores, the fp32 operands in two pieces, hi + lo: a 16 x 8
// operand holds a head's values in two columns, so four heads fill one instruction.
// A query's pieces are whole numbers of 12 bits (to 2^-22 of its group's largest channel, as
// long as that is not below 2^-23 of the row's), so that the sums over a group of 32 channels
// are exact whatever the tensor cores cut off; a weight's are fp16 (22 bits, and down to
// 2^-38 of the largest).
//
// Codes become fp16 in one operation: four bits left in the low bits of a 16-bit half are
// the subnormal c 2^-24, and a whole byte is (c + 16 c') 2^-24 with its neighbour c'.  Bytes
// take one operation less to lay out than single codes, so the operands hold c and c + 16 c',
// and what that adds is taken out at the other end: for K from the query, q c + q' c' =
// (q - q' / 16) c + (q' / 16) (c + 16 c'), for V from the result.  For K that is the operand
// itself, with - 7.5 sum(q) added to a group's sum.  Sums over V run over all tokens, where
// an offset would cancel away what is left of the sum, so V is centred, (c - 7.5) 2^-9 and
// (c' + c / 16 - 7.5 17 / 16) 2^-9, one multiply-add per two values, exactly; and they move
// to shared memory every kFlush blocks, because the tensor cores cut a sum off at its last
// bit each time, always towards zero.
//
// K's scales multiply a group's partial sums (32 channels), V's the softmax weights:
// (hi + lo) a in three fp16 operations for two tokens, the rounding error of hi a going to
// the second piece; the weights are kept 2^13, the scales 2^k larger (k by the largest scale
// so far), so that these errors stay clear of the subnormals: off by 2^-22, or by 2^-35 of
// the largest weight and scale.  That is little beside the sum as long as all scales of the
// unit that the warp has seen lie within 2^9 of each other (2^-24.5 of it per token at most).
// Once they do not, a small group or a light token of large values would cost the others
// their bits: from there on products are taken in fp32, each block's brought to 2^13 .. 2^14
// by their largest of a head and group, and added to the sums in shared memory (32 x 32k
// tokens 128 -> 207 us, 8 heads per unit 196 -> 384).  The scores' layout (tokens by
// heads) becomes the weights' operand (heads by tokens) by one 8 x 8 transposition in
// registers per 8 tokens and group.
//
// Measured, 128 channels, 4 heads per unit: 32 sequences of up to 32k tokens, 8 KV heads,
// 649 MB, 128 us, 5.1 TB/s (8 heads per unit 196 us; 64 channels 77); one of 131072 tokens
// 40 us, one of 4096 10.4.  300 instructions per block: 63 % of the issue slots, 47 % of the
// logic pipe, and in the rest dependent instructions of 16 warps.

constexpr int kWarps = 4, kThreads = 32 * kWarps;
// Blocks of a step, the more the less a step's bookkeeping costs (32 sequences of up to 32k tokens, 64 channels: two
// 82 us, four 75; sequences of 100 tokens 53 and 57, their few blocks being fewer warps' work).
__host__ __device__ constexpr int nib_blocks(int d) { return d <= 64 ? 4 : 2; }
// CTAs resident per SM (their registers), and the stages of a warp's ring that then fit beside the sums.
__host__ __device__ constexpr int nib_ctas(int nb) { return nb == 1 ? 4 : 3; }
__host__ __device__ constexpr int nib_stages(int d, int nb) {
    const int left = 228 * 1024 / nib_ctas(nb) - 4608 - kWarps * 4 * nb * (d + 8) * 4 - nb * d / 32 * 544, n = left / (kWarps * nib_blocks(d) * nib_block_bytes(d));
    return n > 6 ? 6 : n;
}
constexpr int kMaxCtas = 4;   // the larger

struct NibArgs {
    fathom_nibble_pages p;
    int lg, G, cap;
    const float *q;
    const unsigned char *kv;
    const int32_t *table, *lens;
    float *out, *lse;
    Parts parts;
};

struct Todo {   // a unit to be joined: its CTAs, whether the first has a share of an earlier one, its scores' factors
    int unit, first, last;
    bool before;
    float unscale[FATHOM_MAX_G], beyond[FATHOM_MAX_G];
};
template <int kD, int kNB>
struct NibSmem {
    alignas(128) unsigned char ring[kWarps][nib_stages(kD, kNB)][nib_blocks(kD)][nib_block_bytes(kD)];
    float o[kWarps][4 * kNB][kD + 8];   // rows 8 words apart: four heads' stores meet in no bank
    float m[kWarps][FATHOM_MAX_G], l[kWarps][FATHOM_MAX_G], unscale[FATHOM_MAX_G], beyond[FATHOM_MAX_G];
    Share z;
    Todo todo[2];
    int next_seq[kWarps], next_head[kWarps];   // where a warp's copies have got to
    uint4 pieces[kNB][kD / 32][32];   // a unit's queries as the products take them
    float sums[kNB][kD / 32][8];
    ShareSmem<kWarps> share;
    JoinSmem join;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// One or two groups' codes of 16 tokens: registers 2 g, 2 g + 1 hold tokens 0-7 and 8-15.
template <bool kTrans, bool kPair>
__device__ __forceinline__ void load_codes(uint32_t (&r)[4], uint32_t addr) {
    if (kPair) {
        if (kTrans)
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
        else
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    } else {
        if (kTrans)
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
        else
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
    }
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 halves(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t fma_h2(uint32_t x, uint32_t y, uint32_t z) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}
__device__ __forceinline__ uint32_t fms_h2(uint32_t x, uint32_t y, uint32_t z) {   // x y - z
    uint32_t r;
    asm("{\n.reg .b32 n;\nneg.f16x2 n, %3;\nfma.rn.f16x2 %0, %1, %2, n;\n}\n" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t max_h2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t half_pair(float x) { return pack_half2(x, x); }

// Both halves x < y.
__device__ __forceinline__ bool h2_less(uint32_t x, uint32_t y) {
    return __hblt2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
}
constexpr uint32_t kTop = 0x44004400u, kLow = 0x1fff1fffu;   // 4, and what is next below 2^-7, as pairs

constexpr float kQueryPiece = 1.0f / 4096;   // what the second piece counts
constexpr float kUp = 13.0f;                 // weights are 2^13 larger
constexpr int kFlush = 16;   // blocks
// Four codes of each half of x: the first and third, and both bytes.
struct Codes {
    uint32_t c0, b0, c1, b1;
};
__device__ __forceinline__ Codes split_codes(uint32_t x) {
    Codes r;
    r.c0 = x & 0x000f000fu;
    r.b0 = x & 0x00ff00ffu;
    r.b1 = __byte_perm(x, 0, 0x4341);
    r.c1 = r.b1 & 0x000f000fu;
    return r;
}
// c: (c - 7.5) 2^-9, times 2^15 minus 7.5 2^-9; c + 16 c': (c' + c / 16 - 7.5 17 / 16) 2^-9, times 2^11
__device__ __forceinline__ Codes centred(const Codes &x) {
    return Codes{fma_h2(x.c0, 0x78007800u, 0xa380a380u), fma_h2(x.b0, 0x68006800u, 0xa3f8a3f8u),
                 fma_h2(x.c1, 0x78007800u, 0xa380a380u), fma_h2(x.b1, 0x68006800u, 0xa3f8a3f8u)};
}

// Two products' sums u and v times down, added to four channels of a head that count f times (add false: set).
__device__ __forceinline__ void add_sums(float *at, const float (&u)[4], const float (&v)[4], float down, float f, bool add) {
    float4 *to = reinterpret_cast<float4 *>(at);
    float4 x = make_float4(u[0] + u[1], u[2] + u[3], v[0] + v[1], v[2] + v[3]);
    x = make_float4(x.x * down, fmaf(x.x, -0.0625f, x.y) * down, x.z * down, fmaf(x.z, -0.0625f, x.w) * down);
    if (add) {
        const float4 y = *to;
        x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
    }
    *to = x;
}

// floor(log2(x)) of a normal x > 0 (-127 of a smaller one), and 2^e for -126 <= e <= 127.
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Scales of tokens r and r + 8, group by group.
template <int kGroups>
__device__ __forceinline__ void load_scales(uint32_t (&s)[kGroups], const unsigned char *at, int r) {
    if constexpr (kGroups == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at + 16 * r);
        s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
    } else if constexpr (kGroups == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(at + 8 * r);
        s[0] = v.x; s[1] = v.y;
    } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) s[g] = *reinterpret_cast<const uint32_t *>(at + 4 * (kGroups * r + g));
    }
}

// Elements e .. e + 3 of a unit's result from its joined sums: 2^9 of the codes, a / 8.
template <int kD>
struct Finish {
    float *out, *lse;      // of the unit
    const float *beyond;   // what its heads' scores count beyond unscale
    __device__ __forceinline__ void operator()(int e, float4 o, float m, float l, float unscale) const {
        const float inv = l > 0.0f ? 64.0f / l : 0.0f, ln2 = 0.6931471805599453f;
        *reinterpret_cast<float4 *>(out + e) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (lse && e % kD == 0)   // in natural units from the start: scores up to fp32's largest
            lse[e / kD] = l == 0.0f ? -CUDART_INF_F : fmaf(m * (unscale * ln2), beyond[e / kD], (log2f(l) - kUp) * ln2);
    }
};

template <int kD, int kNB>   // kNB: four heads each
__global__ void __launch_bounds__(kThreads, nib_ctas(kNB))
nibble_attn_kernel(const NibArgs a) {
    pdl_enter();
    using Smem = NibSmem<kD, kNB>;
    constexpr int kBlocks = nib_blocks(kD), kStep = kBlocks * kNibTokens, kTile = kStep * kWarps;
    constexpr int kStages = nib_stages(kD, kNB), kGroups = kD / 32, kBlock = nib_block_bytes(kD);
    extern __shared__ __align__(128) unsigned char nib_smem[];
    Smem &sm = *reinterpret_cast<Smem *>(nib_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int H = a.p.kv_heads, G = a.G;
    auto length = [&](int s) { return min(max(__ldg(a.lens + s), 0), a.cap); };
    auto tiles_of = [&](int n) { return (n + kTile - 1) / kTile; };

    int seq, head, tok, n;   // of the step being computed: its unit, its first token, the sequence's tokens
    int count;
    {
        const Share z = find_share<kWarps>(a.p.seqs, H, [&](int s) { return tiles_of(length(s)); }, sm.share);
#pragma unroll 4
        for (int u = blockIdx.x; u < a.p.seqs * H; u += gridDim.x)   // units of empty sequences
            if (length(u / H) == 0) {
                for (int e = tid; e < G * kD; e += kThreads) a.out[(size_t)u * G * kD + e] = 0.0f;
                if (a.lse && tid < G) a.lse[(size_t)u * G + tid] = -CUDART_INF_F;
            }
        if (!z.count) return;
        count = z.count;
        seq = z.seq;
        head = z.head;
        n = length(seq);
        tok = z.tile * kTile + warp * kStep;
        if (tid == 0) sm.z = z;   // read again at the units' ends
    }
    // a unit's queries on their way to this SM
    auto fetch_queries = [&](int unit) {
        if (warp == 0 && 32 * lane < G * kD) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + (size_t)unit * G * kD + 32 * lane));
    };
    fetch_queries(seq * H + head);
    // the next unit with tokens (none: seq = seqs)
    auto next_unit = [&](int &s, int &h, int &len) {
        if (++h < H) return;
        h = 0;
        do len = ++s < a.p.seqs ? length(s) : 1; while (len == 0);
    };

    // ---- copies: the pages of a warp's blocks are looked up one step ahead (-1: none)
    int ld_tok = tok, ld_n = n, page[kBlocks];
    const int32_t *ld_row;          // the sequence's row of the page table
    const unsigned char *ld_kv;     // the head's part of page 0
    {
        ld_row = a.table + (size_t)seq * a.p.max_pages;
        ld_kv = a.kv + head * a.p.head_stride;
        if (lane == 0) { sm.next_seq[warp] = seq; sm.next_head[warp] = head; }
        __syncwarp();
    }
    auto lookup = [&](int t) {
        if (t >= ld_n) return -1;
        const int x = __ldg(ld_row + (t >> a.lg));
        return x >= a.p.num_pages ? -1 : x;
    };
    auto look_ahead = [&]() {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int t = ld_tok + b * kNibTokens;
            page[b] = b && (t & (a.p.page_tokens - 1)) ? (t < ld_n ? page[b - 1] : -1) : lookup(t);   // often one page
        }
    };
    auto ld_advance = [&]() {
        ld_tok += kTile;
        if (ld_tok - warp * kStep < ld_n) return;
        int s = sm.next_seq[warp], h = sm.next_head[warp];
        next_unit(s, h, ld_n);
        __syncwarp();
        if (lane == 0) { sm.next_seq[warp] = s; sm.next_head[warp] = h; }
        __syncwarp();
        ld_tok = warp * kStep;
        if (s >= a.p.seqs) { ld_n = 0; return; }   // no page from here on
        ld_row = a.table + (size_t)s * a.p.max_pages;
        ld_kv = a.kv + h * a.p.head_stride;
        fetch_queries(s * H + h);
    };
    const uint32_t ring = smem_addr(sm.ring[warp]) + 16 * lane;
    constexpr unsigned kAll = (1u << kBlocks) - 1;
    unsigned filled = 0;   // which blocks of the stages are there, a bit each
    auto issue = [&](int st) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            if (page[b] < 0) continue;
            filled |= 1u << (kBlocks * st + b);
            const int slot = (ld_tok + b * kNibTokens) & (a.p.page_tokens - 1);
            const unsigned char *src = ld_kv + page[b] * a.p.page_stride + (int64_t)(slot / kNibTokens) * kBlock + 16 * lane;
            const uint32_t dst = ring + (kBlocks * st + b) * kBlock;
#pragma unroll
            for (int k = 0; k < (kBlock + 511) / 512; ++k)
                if (512 * (k + 1) <= kBlock || 16 * lane < kBlock - 512 * k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * k), "l"(src + 512 * k) : "memory");
        }
    };
    look_ahead();
#pragma unroll 1
    for (int st = 0; st < kStages - 1; ++st) {
        if (st < count) {
            issue(st);
            ld_advance();
            look_ahead();
        }
        cp_async_commit();
    }

    const float to_log2 = 1.4426950408889634f / sqrtf((float)kD);
    uint32_t qb[kNB][kGroups][2][2];   // q's pieces: columns 2 h + piece, see the products below
    float bias[kNB][kGroups], unscale[kNB];   // - 7.5 sum(q) of a group
    // of head c + 4 nb, before unscale: the largest score, the one that sums in shared memory refer to; and the
    // weights' sum of this lane's tokens.  Differences of scores are taken before they are scaled: large ones keep
    // their last bits
    float m[kNB], kept[kNB], l[kNB], o[kNB][2 * kGroups][4];
    uint32_t grow = 0, least = 0;      // 2^k, and V's smallest scale so far, as pairs
    bool wide = false;                 // scales too far apart for one 2^k
    bool in_smem = false;
    int steps = 0;                     // since the sums moved
    auto flush = [&]() {               // sums in shared memory: without 2^k
        const float down = 1.0f / halves(grow).x;
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
            const float f = exp2_approx((kept[nb] - m[nb]) * unscale[nb]);
            kept[nb] = m[nb];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float(&u)[4] = o[nb][2 * g], (&v)[4] = o[nb][2 * g + 1];
                add_sums(&sm.o[warp][4 * nb + c][32 * g + 4 * r], u, v, down, f, in_smem);
                u[0] = u[1] = u[2] = u[3] = v[0] = v[1] = v[2] = v[3] = 0.0f;
            }
        }
        in_smem = true;
        steps = 0;
    };
    int st = 0, joins = 0;

#pragma unroll 1
    for (int i = 0; i < count;) {
        {   // a new unit: its queries in pieces, empty sums
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb) {
                const int mine = 4 * nb + (r >> 1);
                const float *qr = a.q + ((size_t)(seq * H + head) * G + mine) * kD + 8 * c;
                float x[kGroups][8], big = 0.0f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 v = mine < G ? __ldg(reinterpret_cast<const float4 *>(qr + 32 * g) + e)
                                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        x[g][4 * e] = v.x; x[g][4 * e + 1] = v.y; x[g][4 * e + 2] = v.z; x[g][4 * e + 3] = v.w;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(x[g][e]));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // a power of two that brings the largest to 2^10 .. 2^11, with room for a 16th of its neighbour
                const int up = big > 0.0f && big < CUDART_INF_F ? min(9 - exponent(0.53125f * big), 126) : 0;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    if ((nb * kGroups + g) % kWarps != warp) continue;   // the warps share the work
                    float piece[8], sum = 0.0f, part = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) part = fmaxf(part, fabsf(x[g][e]));
                    part = fmaxf(part, __shfl_xor_sync(0xffffffffu, part, 1));
                    part = fmaxf(part, __shfl_xor_sync(0xffffffffu, part, 2));
                    // a group of smaller channels counts 2^-more, from 2^4 down to where fp16 still holds its 16ths
                    const int more = part > 0.0f && part < CUDART_INF_F ? min(max(9 - exponent(0.53125f * part) - up, 0), min(24, 127 - up)) : 0;
                    const float scale = power(up + more), count = power(4 - more);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = e & 1 ? x[g][e] * scale : fmaf(x[g][e + 1] * scale, -0.0625f, x[g][e] * scale), hi = rintf(y);
                        piece[e] = r & 1 ? rintf((y - hi) * 4096.0f) : hi;
                        sum = fmaf(piece[e], e & 1 ? 1.0625f : 1.0f, sum);   // q' counts in c + 16 c' too
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    if (c == 0) sm.sums[nb][g][r] = sum * count;
#pragma unroll
                    for (int e = 0; e < 8; ++e) piece[e] *= e & 1 ? 0.0625f * count : count;
                    // channels 8 c + 2 k and 4 on, and their neighbours, k = 0, 1
                    sm.pieces[nb][g][lane] = make_uint4(pack_half2(piece[0], piece[4]), pack_half2(piece[1], piece[5]),
                                                        pack_half2(piece[2], piece[6]), pack_half2(piece[3], piece[7]));
                }
                // a / 8 of the scales, 2^-24 of the codes, 2^4 of the pieces.  Up to 2^126, the rest in the log-sum-exp alone: scores that
                // differ at all are further apart than any weight shows
                unscale[nb] = __shfl_sync(0xffffffffu, to_log2 * power(min(17 - up, 126)), 8 * c);
                if (warp == 0 && !(lane & 7)) sm.beyond[4 * nb + (lane >> 3)] = power(max(17 - up, 126) - 126);
                m[nb] = kept[nb] = kNoScore;
                l[nb] = 0.0f;
#pragma unroll
                for (int j = 0; j < 2 * kGroups; ++j) o[nb][j][0] = o[nb][j][1] = o[nb][j][2] = o[nb][j][3] = 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const uint4 v = sm.pieces[nb][g][lane];
                    qb[nb][g][0][0] = v.x; qb[nb][g][0][1] = v.y; qb[nb][g][1][0] = v.z; qb[nb][g][1][1] = v.w;
                    bias[nb][g] = fmaf(sm.sums[nb][g][2 * c + 1], kQueryPiece, sm.sums[nb][g][2 * c]) * (-7.5f / 16777216.0f);
                }
            grow = 0x74007400u;    // 2^14
            least = 0x7bff7bffu;   // fp16's largest
            wide = false;
            in_smem = false;
            steps = 0;
        }
        const int first_tile = tok / kTile, last = min(count, i + tiles_of(n) - first_tile);
#pragma unroll 1
        for (; i < last; ++i, tok += kTile) {
            // the copies kStages - 1 steps ahead, into the stage that was read last
            if (i + kStages - 1 < count) {
                issue(st == 0 ? kStages - 1 : st - 1);
                ld_advance();
                look_ahead();
            }
            cp_async_commit();
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const unsigned there = filled >> (kBlocks * st) & kAll;
            if (there) {
                filled ^= there << (kBlocks * st);
                const unsigned char *blk = sm.ring[warp][st][0];
                const uint32_t codes = ring + kBlocks * st * kBlock;
                // ---- scores of tokens r and r + 8 of each block: columns 2 c, 2 c + 1 are the two pieces of head c
                float s[kBlocks][kNB][2];
                uint32_t vs[kBlocks][kGroups];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint32_t sc[kGroups];
                    load_scales<kGroups>(sc, blk + b * kBlock + nib_scales(kD), r);
                    load_scales<kGroups>(vs[b], blk + b * kBlock + nib_half(kD) + nib_scales(kD), r);
#pragma unroll
                    for (int g0 = 0; g0 < kGroups; g0 += 2) {
                        uint32_t x[4];
                        if (g0 + 1 < kGroups) load_codes<false, true>(x, codes + b * kBlock + g0 * 256);
                        else load_codes<false, false>(x, codes + b * kBlock + g0 * 256);
#pragma unroll
                        for (int g = g0; g < g0 + 2 && g < kGroups; ++g) {
                            const Codes u = split_codes(x[2 * (g - g0)]), v = split_codes(x[2 * (g - g0) + 1]);
                            const float2 f = halves(sc[g]);
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb) {
                                const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                float t[4];
                                mma_f16(t, u.c0, v.c0, u.b0, v.b0, qb[nb][g][0][0], qb[nb][g][0][1], none);
                                mma_f16(t, u.c1, v.c1, u.b1, v.b1, qb[nb][g][1][0], qb[nb][g][1][1], t);
                                t[0] = fmaf(t[1], kQueryPiece, t[0] + bias[nb][g]);
                                t[2] = fmaf(t[3], kQueryPiece, t[2] + bias[nb][g]);
                                s[b][nb][0] = g ? fmaf(f.x, t[0], s[b][nb][0]) : f.x * t[0];
                                s[b][nb][1] = g ? fmaf(f.y, t[2], s[b][nb][1]) : f.y * t[2];
                            }
                        }
                    }
                }
                const bool tail = there != kAll || tok + kStep > n;
                if (tail) {   // tokens that are not there: no weight, whatever their places hold
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        const int left = there >> b & 1u ? n - tok - b * kNibTokens : 0;
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) {
                            if (r >= left) s[b][nb][0] = -CUDART_INF_F;
                            if (r + 8 >= left) s[b][nb][1] = -CUDART_INF_F;
                        }
                        const uint32_t keep = (r < left ? 0xffffu : 0u) | (r + 8 < left ? 0xffff0000u : 0u);
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) {
                            vs[b][g] &= keep;
                            least = __vminu2(vs[b][g] | ~keep, least);
                        }
                    }
                }
                uint32_t most = 0u;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        most = max_h2(most, vs[b][g]);
                        if (!tail && (g & 1)) least = __vimin3_u16x2(vs[b][g], vs[b][g - 1], least);
                        if (!tail && g + 1 == kGroups && !(g & 1)) least = __vminu2(vs[b][g], least);
                    }
                float tops[kNB];
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) {
                    tops[nb] = fmaxf(s[0][nb][0], s[0][nb][1]);
#pragma unroll
                    for (int b = 1; b < kBlocks; ++b) tops[nb] = fmaxf(tops[nb], fmaxf(s[b][nb][0], s[b][nb][1]));
                }
                bool raise = !wide && !(h2_less(mul_h2(most, grow), kTop) && h2_less(kLow, mul_h2(least, grow)));
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb) raise |= tops[nb] > m[nb];
                if (__any_sync(0xffffffffu, raise)) {
                    const float2 mh = halves(most);
                    float top_scale = fmaxf(mh.x, mh.y), ratio = 1.0f;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top_scale = fmaxf(top_scale, __shfl_xor_sync(0xffffffffu, top_scale, d));
                    if (!wide) {
                        const float2 lh = halves(__vminu2(least, __byte_perm(least, 0, 0x1032)));
                        const float low = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(lh.x)));
                        float now = halves(grow).x;
                        if (top_scale * now >= 4.0f) {   // k brings the largest scale to 1 .. 2, and holds until 4
                            const float old = now;
                            now = power(top_scale < CUDART_INF_F ? min(max(-exponent(top_scale), -14), 14) : -14);
                            ratio = now / old;
                            grow = half_pair(now);
                        }
                        wide = !(low * now >= 1.0f / 128);   // k stays from here on
                    }
#pragma unroll
                    for (int nb = 0; nb < kNB; ++nb) {
                        float top = tops[nb];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        top = fmaxf(top, m[nb]);
                        float f = exp2_approx((m[nb] - top) * unscale[nb]);   // of no score yet: 0, and its sums 0 or NaN
                        m[nb] = top;
                        l[nb] *= f;
                        f *= ratio;
#pragma unroll
                        for (int j = 0; j < 2 * kGroups; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nb][j][e] *= f;
                    }
                }
                // ---- weights times V: channels 4 r + (0, 1) and 4 r + (2, 3) of a group are two products' rows
                if (!wide) {
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        uint32_t hi[kNB], lo[kNB];   // weights of tokens r (low half) and r + 8
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) {
                            const float w0 = exp2_approx(fmaf(s[b][nb][0] - m[nb], unscale[nb], kUp));
                            const float w1 = exp2_approx(fmaf(s[b][nb][1] - m[nb], unscale[nb], kUp));
                            l[nb] += w0 + w1;
                            hi[nb] = pack_half2(w0, w1);
                            const float2 h = halves(hi[nb]);
                            lo[nb] = pack_half2(w0 - h.x, w1 - h.y);
                        }
#pragma unroll
                        for (int g0 = 0; g0 < kGroups; g0 += 2) {
                            uint32_t x[4];
                            if (g0 + 1 < kGroups) load_codes<true, true>(x, codes + b * kBlock + nib_half(kD) + g0 * 256);
                            else load_codes<true, false>(x, codes + b * kBlock + nib_half(kD) + g0 * 256);
#pragma unroll
                            for (int g = g0; g < g0 + 2 && g < kGroups; ++g) {
                                const uint32_t f = mul_h2(vs[b][g], grow);
                                uint32_t p[kNB][2];
#pragma unroll
                                for (int nb = 0; nb < kNB; ++nb) {
                                    const uint32_t h = mul_h2(hi[nb], f);
                                    const uint32_t e = fma_h2(lo[nb], f, fms_h2(hi[nb], f, h));
                                    p[nb][0] = transpose8(__byte_perm(h, e, 0x5410));
                                    p[nb][1] = transpose8(__byte_perm(h, e, 0x7632));
                                }
                                const Codes u = centred(split_codes(x[2 * (g - g0)])), v = centred(split_codes(x[2 * (g - g0) + 1]));
#pragma unroll
                                for (int nb = 0; nb < kNB; ++nb) {
                                    mma_f16(o[nb][2 * g], u.c0, u.b0, v.c0, v.b0, p[nb][0], p[nb][1], o[nb][2 * g]);
                                    mma_f16(o[nb][2 * g + 1], u.c1, u.b1, v.c1, v.b1, p[nb][0], p[nb][1], o[nb][2 * g + 1]);
                                }
                            }
                        }
                    }
                }
                if (wide || ++steps == kFlush / kBlocks) flush();
                if (wide) {   // block by block to the sums in shared memory
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        const unsigned char *half = blk + b * kBlock + nib_half(kD);
                        float w[kNB][2];
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                w[nb][i] = exp2_approx(fmaf(s[b][nb][i] - m[nb], unscale[nb], kUp));
                                l[nb] += w[nb][i];
                            }
#pragma unroll 1
                        for (int g = 0; g < kGroups; ++g) {
                            uint32_t x[4];
                            load_codes<true, false>(x, codes + b * kBlock + nib_half(kD) + g * 256);
                            const Codes u = centred(split_codes(x[0])), v = centred(split_codes(x[1]));
                            const float2 f = halves(*reinterpret_cast<const uint32_t *>(half + nib_scales(kD) + 4 * (kGroups * r + g)));
#pragma unroll
                            for (int nb = 0; nb < kNB; ++nb) {
                                const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                float p0 = s[b][nb][0] == -CUDART_INF_F ? 0.0f : w[nb][0] * f.x;   // not there: any scale
                                float p1 = s[b][nb][1] == -CUDART_INF_F ? 0.0f : w[nb][1] * f.y, top = fmaxf(p0, p1);
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                                const int up = min(13 - exponent(top), 110);
                                p0 *= power(up);
                                p1 *= power(up);
                                const uint32_t h = pack_half2(p0, p1);
                                const float2 back = halves(h);
                                const uint32_t e = pack_half2(p0 - back.x, p1 - back.y);
                                const uint32_t q0 = transpose8(__byte_perm(h, e, 0x5410)), q1 = transpose8(__byte_perm(h, e, 0x7632));
                                float t[4], z[4];
                                mma_f16(t, u.c0, u.b0, v.c0, v.b0, q0, q1, none);
                                mma_f16(z, u.c1, u.b1, v.c1, v.b1, q0, q1, none);
                                add_sums(&sm.o[warp][4 * nb + c][32 * g + 4 * r], t, z, power(-up), 1.0f, true);
                            }
                        }
                    }
                }
                __syncwarp();   // the stage is read before its next copy starts
            }
            st = st + 1 == kStages ? 0 : st + 1;
        }

        // ---- end of the unit, or of this CTA's share of it
        const int unit = seq * H + head, tiles = tiles_of(n);
#pragma unroll
        for (int nb = 0; nb < kNB; ++nb) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nb] += __shfl_xor_sync(0xffffffffu, l[nb], d);
            if (r == 0) {
                sm.m[warp][4 * nb + c] = m[nb];
                sm.l[warp][4 * nb + c] = l[nb];
                if (warp == 0) sm.unscale[4 * nb + c] = unscale[nb];
            }
        }
        flush();
        __syncthreads();
        // the CTA's state of each head: (m, l, o), to `out` when the unit is all here
        int c_first = sm.z.own_first, c_last = sm.z.own_last;
        bool second = false, before = false;   // this CTA's share, and the first CTA's, is its second
        if (c_first < 0) {
            const long long W = sm.z.W, NC = sm.z.NC, unit_w0 = sm.z.w0 + i - tok / kTile;   // index of the unit's first tile
            c_first = share_owner(unit_w0, W, NC);
            c_last = share_owner(unit_w0 + tiles - 1, W, NC);
            second = sm.z.w0 < unit_w0;
            before = share_start(c_first, W, NC) < unit_w0;
        }
        const bool whole = c_first == c_last;
        const Finish<kD> finish{a.out + (size_t)unit * G * kD, a.lse ? a.lse + (size_t)unit * G : nullptr, sm.beyond};
        const size_t slot = 2 * (size_t)blockIdx.x + (second ? 1 : 0);
        for (int e = 4 * tid; e < G * kD; e += 4 * kThreads) {
            const int h = e / kD, d = e % kD;
            float M = kNoScore, L = 0.0f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm.m[v][h]);
            float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float f = exp2_approx((sm.m[v][h] - M) * sm.unscale[h]);
                const float4 x = *reinterpret_cast<const float4 *>(&sm.o[v][h][d]);
                O.x = fmaf(x.x, f, O.x); O.y = fmaf(x.y, f, O.y); O.z = fmaf(x.z, f, O.z); O.w = fmaf(x.w, f, O.w);
                L = fmaf(sm.l[v][h], f, L);
            }
            if (whole) {
                finish(e, O, M, L, sm.unscale[h]);
            } else {
                *reinterpret_cast<float4 *>(a.parts.o + slot * G * kD + e) = O;
                if (d == 0) *reinterpret_cast<float2 *>(a.parts.ml + (slot * G + h) * 2) = make_float2(M, L);
            }
        }
        if (!whole) {
            if (tid == 0) {
                sm.todo[joins].unit = unit;
                sm.todo[joins].first = c_first;
                sm.todo[joins].last = c_last;
                sm.todo[joins].before = before;
            }
            if (tid < G) {
                sm.todo[joins].unscale[tid] = sm.unscale[tid];
                sm.todo[joins].beyond[tid] = sm.beyond[tid];
            }
            ++joins;
        }
        next_unit(seq, head, n);
        tok = warp * kStep;
        __syncthreads();   // the merge buffers are free again
    }
    cp_async_wait<0>();
    // the first unit and the last one may have other CTAs' shares; joined here, where the loop's registers are free
#pragma unroll 1
    for (int k = 0; k < joins; ++k) {
        const Todo &t = sm.todo[k];
        const Finish<kD> finish{a.out + (size_t)t.unit * G * kD, a.lse ? a.lse + (size_t)t.unit * G : nullptr, t.beyond};
        join_parts<kWarps, kD, 4 * kNB>(a.parts, G, t.first, t.last, t.before, t.unscale, sm.join, finish);
        __syncthreads();
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int kD, int kNB>
cudaError_t launch(const NibArgs &a, int sms, cudaStream_t st) {
    using Smem = NibSmem<kD, kNB>;
    static_assert(nib_ctas(kNB) * (sizeof(Smem) + 1024) <= 228 * 1024, "resident CTAs");
    ensure_smem(nibble_attn_kernel<kD, kNB>, sizeof(Smem));
    return launch_pdl(nibble_attn_kernel<kD, kNB>, dim3(nib_ctas(kNB) * sms), dim3(kThreads), sizeof(Smem), st, a);
}
template <int kD>
cudaError_t launch_heads(const NibArgs &a, int sms, cudaStream_t st) {
    return a.G > 4 ? launch<kD, 2>(a, sms, st) : launch<kD, 1>(a, sms, st);
}

}  // namespace

NibbleWorkspace nibble_workspace_layout(const fathom_nibble_pages &p, int G) {
    NibbleWorkspace w;
    w.sms = device_sm_count();
    if (w.sms <= 0) w.sms = 152;
    const size_t ctas = (size_t)kMaxCtas * w.sms;
    // Tickets first, as many whatever the call, so that one buffer serves calls of different sizes:
    // one for each CTA's unit that goes on behind it, two for groups of shares that begin at it.
    w.part_off = align256(3 * ctas * sizeof(uint32_t));
    w.ml_off = align256(w.part_off + ctas * 2 * G * p.D * sizeof(float));
    w.total = align256(w.ml_off + ctas * 2 * G * 2 * sizeof(float));
    return w;
}

int launch_nibble_attn(const fathom_nibble_pages &p, int G, const float *q, const void *kv, const int32_t *table,
                       const int32_t *lens, float *out, float *lse, void *ws, cudaStream_t st) {
    const NibbleWorkspace w = nibble_workspace_layout(p, G);
    NibArgs a;
    a.p = p;
    a.lg = 0;
    while ((1 << a.lg) < p.page_tokens) ++a.lg;
    a.G = G;
    a.cap = p.max_pages * p.page_tokens;
    a.q = q; a.kv = (const unsigned char *)kv; a.table = table; a.lens = lens; a.out = out; a.lse = lse;
    a.parts.ticket = (unsigned *)ws;
    a.parts.group_ticket = a.parts.ticket + kMaxCtas * w.sms;
    a.parts.o = (float *)((char *)ws + w.part_off);
    a.parts.ml = (float *)((char *)ws + w.ml_off);
    cudaError_t e;
    if (p.D == 128) e = launch_heads<128>(a, w.sms, st);
    else if (p.D == 96) e = launch_heads<96>(a, w.sms, st);
    else if (p.D == 64) e = launch_heads<64>(a, w.sms, st);
    else e = launch_heads<32>(a, w.sms, st);
    if (e != cudaSuccess) return launch_failed("nibble_attn_kernel", e);
    return launch_status("nibble_attn");
}

}  // namespace fathom
