// rope.cu -- new rows into a paged cache of 16-bit rows or of 4-bit codes, the position
// rotation applied on the way (to the step's queries too), and rows of a 4-bit cache read
// back.
#include <cuda_bf16.h>

#include <type_traits>

#include "nibble.cuh"

namespace fathom {

namespace {

// One thread has 8 channels of a token and goes over some of the token's rows (the heads of
// K, of the queries, of V), so that the rotation's cos and sin, the page and the place are
// found once.  Bound by the bytes, each row read and written once: prompts of 19k tokens, 8
// KV heads and 32 query heads of 128 channels, 473 MB, 75 us, 6.3 TB/s.  In 4 bits the
// coding's instructions and the bytes take about as long: the same rows 85 us.
//
// A pair (x, y) turns by (x cos - y sin, y cos + x sin), a product and a fused multiply-add
// in fp32, off by 2^-24 of |x cos| + |y sin| and of the result.
//
// In 4 bits, 32 channels of a token share a = fp16(max |x|) and are coded as
// clip(floor(x / (a / 8)), -8, 7) + 8 of the exact x.  Values are exact: a quotient that is
// never too large gives the code or the one below it, and one fused multiply-add tells
// which.  Rotated keys are coded from fp32 like the queries, with a bound on what that is
// off by; where a border between two codes, or between two scales, is nearer than the
// bound (one group of 2000), the group is worked out again exactly, and the result is
// rounded to odd (cut off to 24 bits, the last bit set where something was cut), after
// which comparisons with the borders, numbers of 14 bits, and the rounding to fp16 are
// those of the unrounded key.
//
// Rows that turn whole, in halves, have both partners in one thread.  Other rotations take a
// chunk of 8 channels per thread, partners in the other half loaded again: the prompts above
// with 64 of 128 channels rotated 98 us into 16 bits and 150 into 4, in neighbouring pairs
// 118 and 138.

constexpr int kThreads = 128;
constexpr int kBatch = 2;       // rows loaded together
constexpr int kCtas = 6;        // per SM: 24 warps' loads in flight (the prompts above: 5 CTAs 77 us, in 4 bits and back 108 instead of 103)
constexpr int kReadBatch = 4;   // when read back

struct AppendArgs {
    fathom_pages p;              // one of the two caches
    fathom_nibble_pages n;
    void *kp, *vp;               // vp: 16-bit rows only
    const int32_t *table;
    const void *kn, *vn;
    int64_t new_token, new_head;
    const int32_t *start, *cu;
    int total, lg, heads, rows, per_slice;   // rows of a token: K, queries, V
    // rotation
    const float *rope;           // [rope_rows][rot]: cos, then sin; NULL: none
    int rope_rows, rot, pairs, vec;
    const int32_t *positions;
    const void *q;
    void *q_out;
    int q_heads, q_f32;
    int64_t q_token, q_head, out_token, out_head;
};

__device__ __forceinline__ float2 to_floats(uint32_t v, __nv_bfloat16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 to_floats(uint32_t v, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t to_pair(float lo, float hi, __nv_bfloat16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t to_pair(float lo, float hi, __half) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = to_floats(w[i], T());
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(to_pair(x[0], x[1], T()), to_pair(x[2], x[3], T()), to_pair(x[4], x[5], T()), to_pair(x[6], x[7], T()));
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// x c + y s rounded to odd: cut off to 24 bits, the last bit set where something was cut.  r is
// the sum rounded in some way, and what that leaves out makes its size more or less.
__device__ __forceinline__ float to_odd(float r, bool more, bool less) {
    uint32_t u = __float_as_uint(r);
    if ((more || less) && !(u & 1u)) u += more ? 1u : 0xffffffffu;
    return __uint_as_float(u);
}
// Any numbers.  In 64 bits the products are exact (35 bits, none too small or too large), and so is
// the sum with what it leaves out.
__device__ __noinline__ float turn_far(float x, float y, float c, float s) {
    const double p = (double)x * c, q = (double)y * s, h = p + q, b = h - p, e = (p - (h - b)) + (q - b);
    const float r = __double2float_rz(h);
    if (!(fabs(h) < CUDART_INF)) return r;                     // infinities and NaN
    const double d = h - r, rest = d != 0.0 ? d : e;           // |e| is less than h's last bit, d a multiple of it
    return to_odd(r, rest != 0.0 && (rest > 0.0) == (h > 0.0), rest != 0.0 && (rest > 0.0) != (h > 0.0));
}
__device__ __forceinline__ float add_exact(float a, float b, float &left) {
    const float h = a + b, z = h - a;
    left = (a - (h - z)) + (b - z);
    return h;
}
// In 32 bits where the products' errors are numbers too and what their sums leave out cannot change
// the sign of the rest (64 bits for all: one decode step of 61 sessions with its read-back 7.5 -> 16.8 us).
__device__ __forceinline__ float turn_odd(float x, float y, float c, float s) {
    const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
    float t, w2, e2, d;
    const float h = add_exact(p, q, t), w = add_exact(fmaf(x, c, -p), fmaf(y, s, -q), w2);
    const float e = add_exact(t, w, e2), r = add_exact(h, e, d), tail = fabsf(w2) + fabsf(e2);
    auto whole = [](float x, float c, float p) { return (fabsf(p) >= 0x1p-100f && fabsf(p) < 0x1p126f) || x == 0.0f || c == 0.0f; };
    if (!(whole(x, c, p) && whole(y, s, q) && (tail == 0.0f || fabsf(d) > 2.0f * tail))) return turn_far(x, y, c, s);
    return to_odd(r, d != 0.0f && (d > 0.0f) == (r > 0.0f), d != 0.0f && (d > 0.0f) != (r > 0.0f));
}

// The sequence of packed token t and its place in it (false: behind the last one).  Whole
// warps: `first` is the least t of the warp.
__device__ __forceinline__ bool find_token(const int32_t *cu, int seqs, int first, int t, int &s, int &i) {
    s = t;
    i = 0;
    if (!cu) return true;
    int lo = 0, hi = seqs;   // the last sequence that starts at or before `first`: 32 borders at a time
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + (threadIdx.x & 31) * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= first);
        if (below) lo += (31 - __clz(below)) * step;
        hi = min(lo + step, hi);
    }
    s = lo;
    int next = __ldg(cu + s + 1);
    if (t >= next) {         // later tokens of the warp: most often the next sequences
        for (int k = 0; k < 4 && t >= next && s + 1 < seqs; ++k) next = __ldg(cu + ++s + 1);
        if (t >= next) {
            for (lo = s, hi = seqs; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
            }
            s = lo;
            next = __ldg(cu + s + 1);
        }
    }
    i = t - __ldg(cu + s);
    return i >= 0 && t < next;
}

// What a thread's 8 channels, from c0 on, need of the table's row at a position.
struct Turn {
    float cs[8], sn[8];   // sn with the sign of the partner's product
    unsigned live;        // which channels turn
    int from;             // first partner channel of a vector of partners; -1: neighbours; -2: one by one
};
__device__ __forceinline__ int partner_of(int c, int half) { return c < half ? c + half : c - half; }
__device__ __forceinline__ Turn load_turn(const float *row, int c0, int rot, bool pairs, bool vec) {
    Turn t;
    const int half = rot / 2;
    t.live = c0 + 8 <= rot ? 0xffu : c0 < rot ? (1u << (rot - c0)) - 1u : 0u;
    t.from = pairs ? -1 : vec ? partner_of(c0, half) : -2;
    if (vec && t.live) {
        const float4 *c = reinterpret_cast<const float4 *>(row + (pairs ? c0 / 2 : c0 < half ? c0 : c0 - half));
        const float4 *s = c + half / 4;
        const float4 a = __ldg(c), b = __ldg(s);
        if (pairs) {
            const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t.cs[e] = ca[e / 2];
                t.sn[e] = e & 1 ? sa[e / 2] : -sa[e / 2];
            }
        } else {
            const float4 a2 = __ldg(c + 1), b2 = __ldg(s + 1);
            const float g = c0 < half ? -1.0f : 1.0f;
            t.cs[0] = a.x; t.cs[1] = a.y; t.cs[2] = a.z; t.cs[3] = a.w;
            t.cs[4] = a2.x; t.cs[5] = a2.y; t.cs[6] = a2.z; t.cs[7] = a2.w;
            t.sn[0] = g * b.x; t.sn[1] = g * b.y; t.sn[2] = g * b.z; t.sn[3] = g * b.w;
            t.sn[4] = g * b2.x; t.sn[5] = g * b2.y; t.sn[6] = g * b2.z; t.sn[7] = g * b2.w;
        }
        return t;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        t.cs[e] = 1.0f;
        t.sn[e] = 0.0f;
        if (c >= rot) continue;
        const int i = pairs ? c / 2 : (c < half ? c : c - half);
        const bool first = pairs ? !(c & 1) : c < half;
        t.cs[e] = __ldg(row + i);
        t.sn[e] = first ? -__ldg(row + half + i) : __ldg(row + half + i);
    }
    return t;
}

// The partners of a row's 8 channels, 0 for those that do not turn.
template <typename T>
__device__ __forceinline__ uint4 load_partners(const T *row, const uint4 &own, int c0, int rot, const Turn &z) {
    if (z.from >= 0) return __ldg(reinterpret_cast<const uint4 *>(row + z.from));
    uint32_t w[4];
    if (z.from == -1) {
        const uint32_t o[4] = {own.x, own.y, own.z, own.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = z.live >> (2 * i) & 1u ? __byte_perm(o[i], 0, 0x1032) : 0u;
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = z.live >> (2 * i) & 1u ? __ldg(p + partner_of(c0 + 2 * i, rot / 2)) : 0u;
            const uint32_t hi = z.live >> (2 * i + 1) & 1u ? __ldg(p + partner_of(c0 + 2 * i + 1, rot / 2)) : 0u;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A group's scale and the codes of a thread's 8 channels, the lanes of `quad` together.
struct Coded {
    uint32_t word;
    __half a;
};
constexpr float kMagic = 8388624.0f;   // 2^23 + 16: a sum with it, rounded down, ends in 16 + floor
// Eight such sums are the digits of a word; what they share is taken off at the end.
__device__ __forceinline__ uint32_t add_digit(uint32_t word, float sum, int e) { return word + (__float_as_uint(sum) << (4 * e)); }
__device__ __forceinline__ uint32_t digits_done(uint32_t word) {
    constexpr uint32_t kBits = 0x4b000008u;   // the bits of 2^23 + 8
    constexpr uint32_t kAll = kBits + (kBits << 4) + (kBits << 8) + (kBits << 12) + (kBits << 16) + (kBits << 20) + (kBits << 24) + (kBits << 28);
    return word - kAll;
}
__device__ __forceinline__ float over_quad(float x, unsigned quad) {
    x = max_nan(x, __shfl_xor_sync(quad, x, 1));
    return max_nan(x, __shfl_xor_sync(quad, x, 2));
}

// Any values: NaN makes the scale NaN, what is larger than fp16 holds counts as its largest.
__device__ __noinline__ Coded code_any(const float (&y)[8], unsigned quad) {
    float big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = max_nan(big, fabsf(y[e]));
    big = over_quad(big, quad);
    Coded r;
    r.a = big == big ? __float2half_rn(fminf(big, 65504.0f)) : __ushort_as_half((unsigned short)0x7fff);
    r.word = 0x88888888u;
    const float a = __half2float(r.a);
    if (a > 0.0f) {
        const float step = a * 0.125f, inv = 1.0f / step;
        r.word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f = floorf(fminf(fmaxf(y[e] * inv, -9.0f), 8.0f));
            if (f * step > y[e]) f -= 1.0f;                     // (f + 1) step has 14 bits
            else if ((f + 1.0f) * step <= y[e]) f += 1.0f;
            r.word |= (uint32_t)((int)fminf(fmaxf(f, -8.0f), 7.0f) + 8) << (4 * e);
        }
    }
    return r;
}
// Larger or smaller ones than these take the general way.
__device__ __forceinline__ bool ordinary(float big) { return big > 1.0f / 4096 && big < 32768.0f; }

__device__ __forceinline__ Coded code_exact(const float (&y)[8], unsigned quad) {
    float big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = max_nan(big, fabsf(y[e]));
    big = over_quad(big, quad);
    if (!ordinary(big)) return code_any(y, quad);
    Coded r;
    r.a = __float2half_rn(big);
    // two reciprocals around the true one: the lesser product is at most the quotient, and above it less 2^-19
    const float step = __half2float(r.a) * 0.125f, inv = 1.0f / step, under = inv * (1.0f - 0x1p-22f), over = inv * (1.0f + 0x1p-22f);
    const float lowest = -8.0f * step, highest = 7.5f * step;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = fminf(fmaxf(y[e], lowest), highest);
        float t = __fadd_rd(fminf(x * under, x * over), kMagic);
        const float next = t - (kMagic - 1.0f);              // the code above
        if (fmaf(-next, step, x) >= 0.0f) t += 1.0f;
        word = add_digit(word, t, e);
    }
    r.word = digits_done(word);
    return r;
}

// Rotated keys in fp32, off by at most `off`: codes as long as no border is that near, else near is set.
__device__ __forceinline__ Coded code_fast(const float (&y)[8], float big, float off, unsigned quad, bool &near) {
    big = over_quad(big, quad);
    const float all = over_quad(off, quad);
    Coded r;
    r.a = __float2half_rn(big);
    near |= !(ordinary(big) && all < big) ||
            __half_as_ushort(__float2half_rn(big - 2.0f * all)) != __half_as_ushort(__float2half_rn(big + 2.0f * all));
    const float inv = 8.0f / __half2float(r.a);
    uint32_t word = 0;
    float far = 0.0f;                                    // the largest distance from the middle between two borders
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = fminf(fmaxf(y[e] * inv, -7.5f), 7.5f);
        const float t = __fadd_rd(v, kMagic);
        far = fmaxf(far, fabsf(v - (t - kMagic) - 0.5f));
        word = add_digit(word, t, e);
    }
    near |= far > 0.5f - (off * inv + 0x1p-19f);
    r.word = digits_done(word);
    return r;
}
// x, their partners and what turns them, for a chunk of 8 channels.
__device__ __forceinline__ Coded code_turned(const float (&x)[8], const float (&p)[8], const Turn &z, unsigned quad) {
    float y[8], big = 0.0f, part = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = __fmul_rn(p[e], z.sn[e]);
        y[e] = fmaf(x[e], z.cs[e], q);
        big = max_nan(big, fabsf(y[e]));
        part = max_nan(part, fabsf(q));
    }
    bool near = false;
    const Coded r = code_fast(y, big, 0x1.02p-24f * (part + big), quad, near);
    if (!(__ballot_sync(quad, near) & quad)) return r;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = z.live >> e & 1u ? turn_odd(x[e], p[e], z.cs[e], z.sn[e]) : x[e];
    return code_any(y, quad);
}

enum Rows { kKeys, kQueries, kValues };

// A thread's part of rows lo .. hi - 1 of one kind, `src` the token's first one, head_stride apart.
template <typename T, bool kNibble, Rows kKind>
__device__ __forceinline__ void move_rows(const AppendArgs &a, const T *src, int64_t stride, int lo, int hi, int t, int c0, int page,
                                          int slot, const Turn &z, unsigned quad) {
    const bool turns = kKind != kValues && z.live, rotated = a.rope != nullptr;
#pragma unroll 1
    for (int r0 = lo; r0 < hi; r0 += kBatch) {
        uint4 own[kBatch], other[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (r0 + b < hi) {
                const T *row = src + (r0 + b) * stride;
                own[b] = __ldg(reinterpret_cast<const uint4 *>(row + c0));
                other[b] = make_uint4(0, 0, 0, 0);
                if (turns) other[b] = load_partners<T>(row, own[b], c0, a.rot, z);
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int head = r0 + b;
            if (head >= hi) break;
            float x[8], p[8];
            if constexpr (kNibble && kKind != kQueries) {
                unsigned char *blk = (unsigned char *)a.kp + nib_block(a.n, page, head, slot) + (kKind == kValues ? nib_half(a.n.D) : 0);
                const int g = c0 / 32, sub = c0 / 8 & 3, in = slot & (kNibTokens - 1);
                unpack8<T>(own[b], x);
                Coded c;
                if (kKind == kKeys && rotated) {   // also the channels of a group that stay: its four lanes go together
                    unpack8<T>(other[b], p);
                    c = code_turned(x, p, z, quad);
                } else {
                    c = code_exact(x, quad);
                }
                *reinterpret_cast<uint32_t *>(blk + nib_code(g, in) + 4 * sub) = c.word;
                if (sub == 0) *reinterpret_cast<__half *>(blk + nib_scales(a.n.D) + nib_scale(a.n.D, g, in)) = c.a;
                continue;
            }
            uint4 out = own[b];
            float y[8];
            if (turns || (kKind == kQueries && a.q_f32)) {
                unpack8<T>(own[b], x);
                if (turns) {
                    unpack8<T>(other[b], p);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], z.cs[e], __fmul_rn(p[e], z.sn[e]));
                    if (z.live != 0xffu) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (!(z.live >> e & 1u)) y[e] = x[e];
                    }
                    out = pack8<T>(y);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[e];
                }
            }
            if (kKind == kQueries) {
                const int64_t to = t * a.out_token + head * a.out_head + c0;
                if (a.q_f32) {
                    float4 *q = reinterpret_cast<float4 *>((float *)a.q_out + to);
                    q[0] = make_float4(y[0], y[1], y[2], y[3]);
                    q[1] = make_float4(y[4], y[5], y[6], y[7]);
                } else {
                    *reinterpret_cast<uint4 *>((T *)a.q_out + to) = out;
                }
            } else {
                T *rows = (T *)(kKind == kValues ? a.vp : a.kp);
                *reinterpret_cast<uint4 *>(rows + page * a.p.page_stride + head * a.p.head_stride + slot * a.p.token_stride + c0) = out;
            }
        }
    }
}

// The same where all channels turn in halves: a thread has 8 channels of the first half and their partners.
template <typename T, bool kNibble, Rows kKind>
__device__ __forceinline__ void move_halves(const AppendArgs &a, const T *src, int64_t stride, int lo, int hi, int t, int c0, int page,
                                            int slot, const float (&cs)[8], const float (&sn)[8], unsigned quad) {
    const int D = kNibble ? a.n.D : a.p.D, c1 = c0 + D / 2;
#pragma unroll 1
    for (int r0 = lo; r0 < hi; r0 += kBatch) {
        uint4 first[kBatch], second[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (r0 + b < hi) {
                const T *row = src + (r0 + b) * stride;
                first[b] = __ldg(reinterpret_cast<const uint4 *>(row + c0));
                second[b] = __ldg(reinterpret_cast<const uint4 *>(row + c1));
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int head = r0 + b;
            if (head >= hi) break;
            float x0[8], x1[8], y0[8], y1[8], big0 = 0.0f, big1 = 0.0f, part0 = 0.0f, part1 = 0.0f;
            if (kNibble || kKind != kValues) {
                unpack8<T>(first[b], x0);
                unpack8<T>(second[b], x1);
            }
            if (kKind != kValues) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p0 = __fmul_rn(x1[e], -sn[e]), p1 = __fmul_rn(x0[e], sn[e]);
                    y0[e] = fmaf(x0[e], cs[e], p0);
                    y1[e] = fmaf(x1[e], cs[e], p1);
                    if (kNibble && kKind == kKeys) {
                        big0 = max_nan(big0, fabsf(y0[e]));
                        big1 = max_nan(big1, fabsf(y1[e]));
                        part0 = max_nan(part0, fabsf(p0));
                        part1 = max_nan(part1, fabsf(p1));
                    }
                }
            }
            if constexpr (kNibble && kKind != kQueries) {
                Coded a0, a1;
                if (kKind == kKeys) {
                    bool near = false;
                    a0 = code_fast(y0, big0, 0x1.02p-24f * (part0 + big0), quad, near);
                    a1 = code_fast(y1, big1, 0x1.02p-24f * (part1 + big1), quad, near);
                    if (__ballot_sync(quad, near) & quad) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y0[e] = turn_odd(x0[e], x1[e], cs[e], -sn[e]);
                            y1[e] = turn_odd(x1[e], x0[e], cs[e], sn[e]);
                        }
                        a0 = code_any(y0, quad);
                        a1 = code_any(y1, quad);
                    }
                } else {
                    a0 = code_exact(x0, quad);
                    a1 = code_exact(x1, quad);
                }
                unsigned char *blk = (unsigned char *)a.kp + nib_block(a.n, page, head, slot) + (kKind == kValues ? nib_half(D) : 0);
                const int g0 = c0 / 32, g1 = c1 / 32, sub = c0 / 8 & 3, in = slot & (kNibTokens - 1);
                *reinterpret_cast<uint32_t *>(blk + nib_code(g0, in) + 4 * sub) = a0.word;
                *reinterpret_cast<uint32_t *>(blk + nib_code(g1, in) + 4 * sub) = a1.word;
                if (sub < 2)
                    *reinterpret_cast<__half *>(blk + nib_scales(D) + nib_scale(D, sub ? g1 : g0, in)) = sub ? a1.a : a0.a;
                continue;
            }
            if (kKind == kQueries && a.q_f32) {
                float *q = (float *)a.q_out + t * a.out_token + head * a.out_head;
                *reinterpret_cast<float4 *>(q + c0) = make_float4(y0[0], y0[1], y0[2], y0[3]);
                *reinterpret_cast<float4 *>(q + c0 + 4) = make_float4(y0[4], y0[5], y0[6], y0[7]);
                *reinterpret_cast<float4 *>(q + c1) = make_float4(y1[0], y1[1], y1[2], y1[3]);
                *reinterpret_cast<float4 *>(q + c1 + 4) = make_float4(y1[4], y1[5], y1[6], y1[7]);
                continue;
            }
            T *to = kKind == kQueries ? (T *)a.q_out + t * a.out_token + head * a.out_head
                                      : (T *)(kKind == kValues ? a.vp : a.kp) + page * a.p.page_stride + head * a.p.head_stride + slot * a.p.token_stride;
            *reinterpret_cast<uint4 *>(to + c0) = kKind == kValues ? first[b] : pack8<T>(y0);
            *reinterpret_cast<uint4 *>(to + c1) = kKind == kValues ? second[b] : pack8<T>(y1);
        }
    }
}

// kHalves: two chunks of 8 channels per thread, as above, else one.  The four lanes of a
// group of 32 channels are neighbours.
template <typename T, bool kNibble, bool kHalves>
__global__ void __launch_bounds__(kThreads, kCtas)
append_kernel(const AppendArgs a) {
    pdl_enter();
    const int D = kNibble ? a.n.D : a.p.D, H = a.heads, pieces = kHalves ? D / 16 : D / 8;
    const int per = kThreads / pieces, tl = threadIdx.x / pieces, piece = threadIdx.x - tl * pieces;
    const long long tt = (long long)blockIdx.x * per + tl;
    const int t = (int)min(tt, (long long)a.total), c0 = 8 * piece;
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    int s, i;
    const bool in = find_token(a.cu, kNibble ? a.n.seqs : a.p.seqs, __shfl_sync(0xffffffffu, t, 0), t, s, i);
    if (tl >= per || tt >= a.total || !in) return;
    const long long pos = (long long)a.start[s] + i;
    const int max_pages = kNibble ? a.n.max_pages : a.p.max_pages, num_pages = kNibble ? a.n.num_pages : a.p.num_pages;
    Turn z = {};
    if (a.rope) {
        const long long at = a.positions ? (long long)a.positions[t] : pos;
        if (at < 0 || at >= a.rope_rows) return;
        z = load_turn(a.rope + at * a.rot, c0, a.rot, a.pairs, a.vec);
        if (kHalves) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z.sn[e] = -z.sn[e];   // of the second half
        }
    }
    int page = -1;
    if (pos >= 0 && pos < (long long)max_pages << a.lg) page = a.table[(size_t)s * max_pages + (pos >> a.lg)];
    if (page >= num_pages) page = -1;
    const int slot = (int)(pos & ((1 << a.lg) - 1));
    // rows: 0 .. H - 1 keys, then the queries, then the values
    const int Q = a.q_heads, r0 = blockIdx.y * a.per_slice, r1 = min(a.rows, r0 + a.per_slice);
    const T *k = (const T *)a.kn + t * a.new_token, *q = (const T *)a.q + t * a.q_token, *v = (const T *)a.vn + t * a.new_token;
    const int q0 = max(r0 - H, 0), q1 = min(r1 - H, Q), v0 = max(r0 - H - Q, 0), v1 = min(r1 - H - Q, H);
    if constexpr (kHalves) {
        if (page >= 0) move_halves<T, kNibble, kKeys>(a, k, a.new_head, r0, min(r1, H), t, c0, page, slot, z.cs, z.sn, quad);
        move_halves<T, kNibble, kQueries>(a, q, a.q_head, q0, q1, t, c0, page, slot, z.cs, z.sn, quad);
        if (page >= 0) move_halves<T, kNibble, kValues>(a, v, a.new_head, v0, v1, t, c0, page, slot, z.cs, z.sn, quad);
    } else {
        if (page >= 0) move_rows<T, kNibble, kKeys>(a, k, a.new_head, r0, min(r1, H), t, c0, page, slot, z, quad);
        move_rows<T, kNibble, kQueries>(a, q, a.q_head, q0, q1, t, c0, page, slot, z, quad);
        if (page >= 0) move_rows<T, kNibble, kValues>(a, v, a.new_head, v0, v1, t, c0, page, slot, z, quad);
    }
}

// ---------------------------------------------------------------- read back
struct ReadArgs {
    fathom_nibble_pages n;
    const unsigned char *kv;
    const int32_t *table, *start, *cu;
    int total, lg, per_slice;
    void *k_out, *v_out;
    int64_t out_token, out_head;
};

// 8 channels' codes as they are used.  The codes become (c - 7.5) / 8 in fp16 (in the low
// bits of a half c is the subnormal c 2^-24, four bits up 16 c 2^-24), times a exactly in fp32.
template <typename T>
__device__ __forceinline__ void store_values(T *out, uint32_t word, __half a) {
    uint32_t v[4];   // channels (0, 4), (1, 5), (2, 6), (3, 7)
    const uint32_t up = word >> 8;
    const uint32_t low[4] = {word & 0x000f000fu, word & 0x00f000f0u, up & 0x000f000fu, up & 0x00f000f0u};
#pragma unroll
    for (int i = 0; i < 4; ++i)   // times 2^15 or 2^11, minus 7.5 2^-9
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(low[i]), "r"(i & 1 ? 0x68006800u : 0x78007800u), "r"(0xa380a380u));
    const float scale = __half2float(a) * 64.0f;
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
        x[i] = f.x * scale;
        x[i + 4] = f.y * scale;
    }
    if constexpr (std::is_same<T, float>::value) {
        reinterpret_cast<float4 *>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(out) = pack8<T>(x);
    }
}

// A thread has 8 channels of a token, or (kTwo: whole groups in each half of a row) those and
// the 8 that lie half a row on, and goes over some of its rows.
template <typename T, bool kTwo>
__global__ void __launch_bounds__(kThreads)
nibble_read_kernel(const ReadArgs a) {
    pdl_enter();
    const int D = a.n.D, H = a.n.kv_heads, pieces = kTwo ? D / 16 : D / 8;
    const int per = kThreads / pieces, tl = threadIdx.x / pieces, piece = threadIdx.x - tl * pieces;
    const long long tt = (long long)blockIdx.x * per + tl;
    const int t = (int)min(tt, (long long)a.total);
    int s, i;
    const bool inside = find_token(a.cu, a.n.seqs, __shfl_sync(0xffffffffu, t, 0), t, s, i);
    if (tl >= per || tt >= a.total || !inside) return;
    const long long pos = (long long)a.start[s] + i;
    if (pos < 0 || pos >= (long long)a.n.max_pages << a.lg) return;
    const int page = a.table[(size_t)s * a.n.max_pages + (pos >> a.lg)];
    if (page < 0 || page >= a.n.num_pages) return;
    const int slot = (int)(pos & (a.n.page_tokens - 1)), in = slot & (kNibTokens - 1);
    const int g = piece >> 2, more = D / 64;   // its group, and the other one's distance
    const unsigned char *blk = a.kv + nib_block(a.n, page, 0, slot) + nib_code(g, in) + 4 * (piece & 3);
    const int scale_at = nib_scales(D) + nib_scale(D, g, in) - nib_code(g, in) - 4 * (piece & 3);   // from there
    const int64_t to = t * a.out_token + 8 * piece;
    const int r1 = min(2 * H, ((int)blockIdx.y + 1) * a.per_slice);
#pragma unroll 1
    for (int r0 = blockIdx.y * a.per_slice; r0 < r1; r0 += kReadBatch) {
        uint32_t word[kReadBatch][2];
        __half scale[kReadBatch][2];
#pragma unroll
        for (int b = 0; b < kReadBatch; ++b) {   // rows: the heads of K, then of V
            const int row = r0 + b;
            if (row >= r1) break;
            const unsigned char *part = blk + (row < H ? row * a.n.head_stride : (row - H) * a.n.head_stride + nib_half(D));
#pragma unroll
            for (int k = 0; k < (kTwo ? 2 : 1); ++k) {
                word[b][k] = __ldg(reinterpret_cast<const uint32_t *>(part + k * nib_code(more, 0)));
                scale[b][k] = __ldg(reinterpret_cast<const __half *>(part + scale_at + 4 * k * more));
            }
        }
#pragma unroll
        for (int b = 0; b < kReadBatch; ++b) {
            const int row = r0 + b;
            if (row >= r1) break;
            T *out = row < H ? (T *)a.k_out + to + row * a.out_head : (T *)a.v_out + to + (row - H) * a.out_head;
            store_values<T>(out, word[b][0], scale[b][0]);
            if (kTwo) store_values<T>(out + D / 2, word[b][1], scale[b][1]);
        }
    }
}

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// Rows that a CTA goes over: as many as leave 16 CTAs per SM, at most 16 (one decode step
// spreads over the SMs, prompts read the table's rows once for several heads).
int rows_per_slice(long long ctas, int rows) {
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;
    const long long n = ctas * rows / (16LL * sms);
    return (int)(n < 1 ? 1 : n > 16 ? 16 : n);
}

template <typename T, bool kNibble>
cudaError_t launch_form(const AppendArgs &a, bool halves, dim3 grid, cudaStream_t st) {
    return halves ? launch_pdl(append_kernel<T, kNibble, true>, grid, dim3(kThreads), 0, st, a)
                  : launch_pdl(append_kernel<T, kNibble, false>, grid, dim3(kThreads), 0, st, a);
}

int launch_append(AppendArgs &a, bool nibble, int dtype, const char *what, cudaStream_t st) {
    const int D = nibble ? a.n.D : a.p.D;
    // whole rows that turn in halves: both partners in one thread; in 4 bits each half has whole groups
    const bool halves = a.rope && !a.pairs && a.rot == D && D % (nibble ? 64 : 16) == 0;
    const int per = kThreads / (halves ? D / 16 : D / 8);
    const long long ctas = ((long long)a.total + per - 1) / per;
    a.per_slice = rows_per_slice(ctas, a.rows);
    const int slices = (a.rows + a.per_slice - 1) / a.per_slice;
    if (ctas > 0x7fffffffLL || slices > 65535) { set_error("%s: too many rows for one launch", what); return FATHOM_EINVAL; }
    const dim3 grid((unsigned)ctas, slices);
    const cudaError_t e = nibble ? (dtype == FATHOM_BF16 ? launch_form<__nv_bfloat16, true>(a, halves, grid, st) : launch_form<__half, true>(a, halves, grid, st))
                                 : (dtype == FATHOM_BF16 ? launch_form<__nv_bfloat16, false>(a, halves, grid, st) : launch_form<__half, false>(a, halves, grid, st));
    if (e != cudaSuccess) return launch_failed(what, e);
    return launch_status(what);
}

template <typename T>
cudaError_t launch_read(const ReadArgs &a, bool two, dim3 grid, cudaStream_t st) {
    return two ? launch_pdl(nibble_read_kernel<T, true>, grid, dim3(kThreads), 0, st, a)
               : launch_pdl(nibble_read_kernel<T, false>, grid, dim3(kThreads), 0, st, a);
}

AppendArgs append_args(const int32_t *table, const void *kn, const void *vn, int total, int64_t new_token, int64_t new_head,
                       const int32_t *start, const int32_t *cu, const fathom_rope *rope) {
    AppendArgs a = {};
    a.table = table;
    a.kn = kn; a.vn = vn;
    a.new_token = new_token; a.new_head = new_head;
    a.start = start; a.cu = cu;
    a.total = total;
    if (rope) {
        a.rope = rope->table;
        a.rope_rows = rope->rows;
        a.rot = rope->rot;
        a.pairs = rope->interleaved != 0;
        a.vec = rope->rot % (a.pairs ? 8 : 16) == 0;   // 8 channels' numbers, and halves' partners, side by side
        a.positions = rope->positions;
        if (rope->q) {
            a.q = rope->q; a.q_out = rope->q_out;
            a.q_heads = rope->q_heads;
            a.q_f32 = rope->q_dtype == FATHOM_F32;
            a.q_token = rope->q_token; a.q_head = rope->q_head;
            a.out_token = rope->out_token; a.out_head = rope->out_head;
        }
    }
    return a;
}

}  // namespace

int launch_paged_append_rope(const fathom_pages &p, void *kp, void *vp, const int32_t *table, const void *kn, const void *vn,
                             int total, int64_t new_token, int64_t new_head, const int32_t *start, const int32_t *cu,
                             const fathom_rope &rope, cudaStream_t st) {
    AppendArgs a = append_args(table, kn, vn, total, new_token, new_head, start, cu, &rope);
    a.p = p;
    a.kp = kp; a.vp = vp;
    a.lg = log2_of(p.page_tokens);
    a.heads = p.kv_heads;
    a.rows = 2 * p.kv_heads + a.q_heads;
    return launch_append(a, false, p.dtype, "paged_append_rope", st);
}

int launch_nibble_append(const fathom_nibble_pages &p, void *kv, const int32_t *table, int dtype, const void *kn, const void *vn,
                         int total, int64_t new_token, int64_t new_head, const int32_t *start, const int32_t *cu,
                         const fathom_rope *rope, cudaStream_t st) {
    AppendArgs a = append_args(table, kn, vn, total, new_token, new_head, start, cu, rope);
    a.n = p;
    a.kp = kv;
    a.lg = log2_of(p.page_tokens);
    a.heads = p.kv_heads;
    a.rows = 2 * p.kv_heads + a.q_heads;
    return launch_append(a, true, dtype, "nibble_append", st);
}

int launch_nibble_read(const fathom_nibble_pages &p, const void *kv, const int32_t *table, const int32_t *start,
                       const int32_t *cu, int total, void *k_out, void *v_out, int dtype, int64_t out_token,
                       int64_t out_head, cudaStream_t st) {
    ReadArgs a;
    a.n = p;
    a.kv = (const unsigned char *)kv;
    a.table = table; a.start = start; a.cu = cu;
    a.total = total;
    a.lg = log2_of(p.page_tokens);
    a.k_out = k_out; a.v_out = v_out;
    a.out_token = out_token; a.out_head = out_head;
    const bool two = p.D % 64 == 0;
    const int per = kThreads / (two ? p.D / 16 : p.D / 8);
    const long long ctas = ((long long)total + per - 1) / per;
    a.per_slice = rows_per_slice(ctas, 2 * p.kv_heads);
    const int slices = (2 * p.kv_heads + a.per_slice - 1) / a.per_slice;
    if (ctas > 0x7fffffffLL || slices > 65535) { set_error("nibble_read: too many rows for one launch"); return FATHOM_EINVAL; }
    const dim3 grid((unsigned)ctas, slices);
    const cudaError_t e = dtype == FATHOM_F32    ? launch_read<float>(a, two, grid, st)
                          : dtype == FATHOM_BF16 ? launch_read<__nv_bfloat16>(a, two, grid, st)
                                                 : launch_read<__half>(a, two, grid, st);
    if (e != cudaSuccess) return launch_failed("nibble_read", e);
    return launch_status("nibble_read");
}

}  // namespace fathom
