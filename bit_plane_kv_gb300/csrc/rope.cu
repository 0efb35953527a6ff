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
// found once.  Bound by the bytes: each row read and written once.
//
// A pair (x, y) turns by (x cos - y sin, y cos + x sin).  The products and their sum are
// taken with the rounding errors that two fused multiply-adds give exactly, so a result is
// off by 2^-23 of itself, also where the two products nearly cancel.
//
// In 4 bits, 32 channels of a token share a = fp16(max |x|) and are coded as
// clip(floor(x / (a / 8)), -8, 7) + 8.  Borders between codes are numbers of 14 bits and
// the roundings to fp16 look at 12, so a rotated key is first rounded to odd in fp32 (cut
// off, the last bit set where something was cut): every comparison and rounding after that
// is that of the unrounded key, and codes do not depend on how the rotation was computed.

constexpr int kThreads = 128;
constexpr int kBatch = 4;   // rows loaded together

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

// x c + y s, off by 2^-23 of the result: both products' errors and the sum's are exact.
__device__ __forceinline__ float turn(float x, float y, float c, float s) {
    const float p = __fmul_rn(x, c), r = fmaf(y, s, p);
    return fabsf(r) < CUDART_INF_F ? r + fmaf(x, c, -p) : r;   // the error of an infinity is NaN
}
// x c + y s rounded to odd: cut off to 24 bits, the last bit set where something was cut.
__device__ __forceinline__ float turn_odd(float x, float y, float c, float s) {
    const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
    const float h = p + q, b = h - p;
    const float e = (p - (h - b)) + (q - b) + (fmaf(x, c, -p) + fmaf(y, s, -q));   // what h leaves out
    const float r = h + e, d = e - (r - h);                                        // |e| < |h|
    if (!(fabsf(r) < CUDART_INF_F)) return fabsf(h) < CUDART_INF_F ? r : h;        // the errors of an infinity are NaN
    uint32_t u = __float_as_uint(r);
    if (d != 0.0f && !(u & 1u)) u += (d > 0.0f) == (r > 0.0f) ? 1u : 0xffffffffu;
    return __uint_as_float(u);
}

// The sequence of packed token t and its place in it (false: behind the last one).
__device__ __forceinline__ bool find_token(const int32_t *cu, int seqs, int t, int &s, int &i) {
    s = t;
    i = 0;
    if (!cu) return true;
    int lo = 0, hi = seqs;   // the last sequence that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    s = lo;
    i = t - cu[s];
    return i >= 0 && t < cu[s + 1];
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
    if (!t.live) return t;
    if (vec && !pairs) {
        const int i = c0 < half ? c0 : c0 - half;
        const float sign = c0 < half ? -1.0f : 1.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + i) + e), b = __ldg(reinterpret_cast<const float4 *>(row + half + i) + e);
            t.cs[4 * e] = a.x; t.cs[4 * e + 1] = a.y; t.cs[4 * e + 2] = a.z; t.cs[4 * e + 3] = a.w;
            t.sn[4 * e] = sign * b.x; t.sn[4 * e + 1] = sign * b.y; t.sn[4 * e + 2] = sign * b.z; t.sn[4 * e + 3] = sign * b.w;
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

// kNibble: threads in the order (group, token, 8 channels), so that a group's codes of
// consecutive tokens are written side by side; else (token, 8 channels).
template <typename T, bool kNibble>
__global__ void __launch_bounds__(kThreads)
append_kernel(const AppendArgs a) {
    pdl_enter();
    const int D = kNibble ? a.n.D : a.p.D, H = a.heads, pieces = D / 8;
    const int lane = threadIdx.x & 31;
    int piece, tl, per;
    if (kNibble) {
        const int groups = D / 32;
        per = kThreads / 4 / groups & ~7;   // tokens of a CTA: 8, 8, 16 or 32
        const int g = threadIdx.x / (4 * per);
        tl = threadIdx.x / 4 % per;
        piece = 4 * g + (threadIdx.x & 3);
        if (g >= groups) return;
    } else {
        per = kThreads / pieces;
        tl = threadIdx.x / pieces;
        piece = threadIdx.x - tl * pieces;
        if (tl >= per) return;
    }
    const long long tt = (long long)blockIdx.x * per + tl;
    if (tt >= a.total) return;
    const int t = (int)tt, c0 = 8 * piece;
    const unsigned quad = 0xfu << (lane & ~3);   // the lanes of a group of channels (4 bits)
    int s, i;
    if (!find_token(a.cu, kNibble ? a.n.seqs : a.p.seqs, t, s, i)) return;
    const long long pos = (long long)a.start[s] + i;
    const int max_pages = kNibble ? a.n.max_pages : a.p.max_pages, num_pages = kNibble ? a.n.num_pages : a.p.num_pages;
    Turn z;
    z.live = 0;
    z.from = -1;
    if (a.rope) {
        const long long at = a.positions ? (long long)a.positions[t] : pos;
        if (at < 0 || at >= a.rope_rows) return;
        z = load_turn(a.rope + at * a.rot, c0, a.rot, a.pairs, a.vec);
    }
    int page = -1;
    if (pos >= 0 && pos < (long long)max_pages << a.lg) page = a.table[(size_t)s * max_pages + (pos >> a.lg)];
    if (page >= num_pages) page = -1;
    const int slot = (int)(pos & ((1 << a.lg) - 1));
    const int r1 = min(a.rows, ((int)blockIdx.y + 1) * a.per_slice);
    for (int r0 = blockIdx.y * a.per_slice; r0 < r1; r0 += kBatch) {
        uint4 own[kBatch], other[kBatch];
        const T *src[kBatch];
        // rows: 0 .. H - 1 keys, then the queries, then the values
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = r0 + b;
            if (row >= r1) continue;
            const bool q = row >= H && row < H + a.q_heads;
            if (!q && page < 0) continue;
            if (q) src[b] = (const T *)a.q + t * a.q_token + (row - H) * a.q_head;
            else if (row < H) src[b] = (const T *)a.kn + t * a.new_token + row * a.new_head;
            else src[b] = (const T *)a.vn + t * a.new_token + (row - H - a.q_heads) * a.new_head;
            own[b] = __ldg(reinterpret_cast<const uint4 *>(src[b] + c0));
            if (z.live && z.from >= 0 && row < H + a.q_heads) other[b] = __ldg(reinterpret_cast<const uint4 *>(src[b] + z.from));
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = r0 + b;
            if (row >= r1) continue;
            const bool q = row >= H && row < H + a.q_heads, v = row >= H + a.q_heads;
            if (!q && page < 0) continue;
            float x[8], y[8];
            unpack8<T>(own[b], x);
            if (!v && z.live) {
                if (z.from >= 0) {
                    unpack8<T>(other[b], y);
                } else if (z.from == -1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = z.live >> e & 1u ? (float)src[b][partner_of(c0 + e, a.rot / 2)] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!(z.live >> e & 1u)) y[e] = x[e];
                    else y[e] = kNibble && !q ? turn_odd(x[e], y[e], z.cs[e], z.sn[e]) : turn(x[e], y[e], z.cs[e], z.sn[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e];
            }
            if (q) {
                const int64_t to = t * a.out_token + (row - H) * a.out_head + c0;
                if (a.q_f32) {
                    float4 *out = reinterpret_cast<float4 *>((float *)a.q_out + to);
                    out[0] = make_float4(y[0], y[1], y[2], y[3]);
                    out[1] = make_float4(y[4], y[5], y[6], y[7]);
                } else {
                    *reinterpret_cast<uint4 *>((T *)a.q_out + to) = z.live ? pack8<T>(y) : own[b];
                }
                continue;
            }
            const int head = v ? row - H - a.q_heads : row;
            if constexpr (!kNibble) {
                const int64_t to = page * a.p.page_stride + head * a.p.head_stride + slot * a.p.token_stride + c0;
                *reinterpret_cast<uint4 *>((T *)(v ? a.vp : a.kp) + to) = v || !z.live ? own[b] : pack8<T>(y);
            } else {
                // NaN anywhere in the group makes its scale NaN; larger values than fp16 holds count as its largest
                float big = 0.0f;
                bool nan = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    big = fmaxf(big, fabsf(y[e]));
                    nan |= y[e] != y[e];
                }
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    big = fmaxf(big, __shfl_xor_sync(quad, big, d));
                    nan |= __shfl_xor_sync(quad, (int)nan, d) != 0;
                }
                const __half ah = nan ? __ushort_as_half((unsigned short)0x7fff) : __float2half_rn(fminf(big, 65504.0f));
                const float a16 = __half2float(ah), step = a16 * 0.125f, inv = a16 > 0.0f ? 1.0f / step : 0.0f;
                uint32_t word = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // floor of the exact quotient, clipped: the product by 1 / step is within one of it, and
                    // (f + 1) step has 14 bits
                    float f = floorf(fminf(fmaxf(y[e] * inv, -9.0f), 8.0f));
                    if (f * step > y[e]) f -= 1.0f;
                    else if ((f + 1.0f) * step <= y[e]) f += 1.0f;
                    f = fminf(fmaxf(f, -8.0f), 7.0f);
                    word |= (uint32_t)(a16 > 0.0f ? (int)f + 8 : 8) << (4 * e);
                }
                unsigned char *blk = (unsigned char *)a.kp + nib_block(a.n, page, head, slot) + (v ? nib_half(D) : 0);
                const int g = piece >> 2, in = slot & (kNibTokens - 1);
                *reinterpret_cast<uint32_t *>(blk + nib_code(g, in) + 4 * (piece & 3)) = word;
                if ((piece & 3) == 0) *reinterpret_cast<__half *>(blk + nib_scales(D) + nib_scale(D, g, in)) = ah;
            }
        }
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

// The threads of append_kernel, the other way round: 4 bytes of codes, 8 channels.
template <typename T>
__global__ void __launch_bounds__(kThreads)
nibble_read_kernel(const ReadArgs a) {
    pdl_enter();
    const int D = a.n.D, H = a.n.kv_heads, groups = D / 32;
    const int per = kThreads / 4 / groups & ~7, g = threadIdx.x / (4 * per), tl = threadIdx.x / 4 % per, sub = threadIdx.x & 3;
    const long long tt = (long long)blockIdx.x * per + tl;
    if (g >= groups || tt >= a.total) return;
    const int t = (int)tt;
    int s, i;
    if (!find_token(a.cu, a.n.seqs, t, s, i)) return;
    const long long pos = (long long)a.start[s] + i;
    if (pos < 0 || pos >= (long long)a.n.max_pages << a.lg) return;
    const int page = a.table[(size_t)s * a.n.max_pages + (pos >> a.lg)];
    if (page < 0 || page >= a.n.num_pages) return;
    const int slot = (int)(pos & (a.n.page_tokens - 1)), in = slot & (kNibTokens - 1);
    const unsigned char *blk = a.kv + nib_block(a.n, page, 0, slot);
    const int r1 = min(2 * H, ((int)blockIdx.y + 1) * a.per_slice);
    for (int r0 = blockIdx.y * a.per_slice; r0 < r1; r0 += kBatch) {
        uint32_t word[kBatch];
        __half scale[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {   // rows: the heads of K, then of V
            const int row = r0 + b;
            if (row >= r1) continue;
            const unsigned char *part = blk + (row < H ? row : row - H) * a.n.head_stride + (row < H ? 0 : nib_half(D));
            word[b] = *reinterpret_cast<const uint32_t *>(part + nib_code(g, in) + 4 * sub);
            scale[b] = *reinterpret_cast<const __half *>(part + nib_scales(D) + nib_scale(D, g, in));
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = r0 + b;
            if (row >= r1) continue;
            const float step = __half2float(scale[b]) * 0.125f;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = ((float)(word[b] >> (4 * e) & 15u) - 7.5f) * step;   // exact
            T *out = (T *)(row < H ? a.k_out : a.v_out) + t * a.out_token + (row < H ? row : row - H) * a.out_head + 32 * g + 8 * sub;
            if constexpr (std::is_same<T, float>::value) {
                reinterpret_cast<float4 *>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4 *>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
                *reinterpret_cast<uint4 *>(out) = pack8<T>(x);
            }
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

int launch_append(AppendArgs &a, bool nibble, int dtype, const char *what, cudaStream_t st) {
    const int D = nibble ? a.n.D : a.p.D;
    const int per = nibble ? kThreads / 4 / (D / 32) & ~7 : kThreads / (D / 8);
    const long long ctas = ((long long)a.total + per - 1) / per;
    a.per_slice = rows_per_slice(ctas, a.rows);
    const int slices = (a.rows + a.per_slice - 1) / a.per_slice;
    if (ctas > 0x7fffffffLL || slices > 65535) { set_error("%s: too many rows for one launch", what); return FATHOM_EINVAL; }
    const dim3 grid((unsigned)ctas, slices), block(kThreads);
    cudaError_t e;
    if (nibble)
        e = dtype == FATHOM_BF16 ? launch_pdl(append_kernel<__nv_bfloat16, true>, grid, block, 0, st, a)
                                 : launch_pdl(append_kernel<__half, true>, grid, block, 0, st, a);
    else
        e = dtype == FATHOM_BF16 ? launch_pdl(append_kernel<__nv_bfloat16, false>, grid, block, 0, st, a)
                                 : launch_pdl(append_kernel<__half, false>, grid, block, 0, st, a);
    if (e != cudaSuccess) return launch_failed(what, e);
    return launch_status(what);
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
        a.vec = !a.pairs && rope->rot % 16 == 0;   // 8 channels have 8 partners side by side
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
    const int per = kThreads / 4 / (p.D / 32) & ~7;
    const long long ctas = ((long long)total + per - 1) / per;
    a.per_slice = rows_per_slice(ctas, 2 * p.kv_heads);
    const int slices = (2 * p.kv_heads + a.per_slice - 1) / a.per_slice;
    if (ctas > 0x7fffffffLL || slices > 65535) { set_error("nibble_read: too many rows for one launch"); return FATHOM_EINVAL; }
    const dim3 grid((unsigned)ctas, slices), block(kThreads);
    const cudaError_t e = dtype == FATHOM_F32    ? launch_pdl(nibble_read_kernel<float>, grid, block, 0, st, a)
                          : dtype == FATHOM_BF16 ? launch_pdl(nibble_read_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                                                 : launch_pdl(nibble_read_kernel<__half>, grid, block, 0, st, a);
    if (e != cudaSuccess) return launch_failed("nibble_read", e);
    return launch_status("nibble_read");
}

}  // namespace fathom
