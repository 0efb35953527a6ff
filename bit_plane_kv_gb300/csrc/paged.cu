// paged.cu -- a paged KV cache: append of new rows, and decode attention of one
// new token per sequence.
#include <cuda_bf16.h>

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
// read and written once.
__global__ void __launch_bounds__(256)
paged_append_kernel(fathom_pages p, int lg, int4 *__restrict__ kp, int4 *__restrict__ vp,
                    const int32_t *__restrict__ table, const int4 *__restrict__ kn, const int4 *__restrict__ vn,
                    int total, int64_t new_token, int64_t new_head, const int32_t *__restrict__ start,
                    const int32_t *__restrict__ cu_new) {
    const int pieces = p.D / 8, row = pieces * p.kv_heads;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= (long long)total * row) return;
    const int t = (int)(e / row), r = (int)(e % row), h = r / pieces, c = r % pieces;
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
__device__ __forceinline__ float row_value(const __nv_bfloat16 *x) { return __bfloat162float(*x); }
__device__ __forceinline__ float row_value(const __half *x) { return __half2float(*x); }

// One CTA per (unit, query head): warp w takes tokens w, w + 8, ..., lane l
// channels l + 32 c; the warps' running states are merged at the end.
template <typename T>
__global__ void __launch_bounds__(256)
paged_attn_kernel(fathom_pages p, int lg, int G, const float *__restrict__ q, const T *__restrict__ kp,
                  const T *__restrict__ vp, const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
                  float *__restrict__ out, float *__restrict__ logits, float *__restrict__ norm) {
    __shared__ float sm[8], sl[8], so[8][FATHOM_MAX_D];
    const int u = blockIdx.x / G, g = blockIdx.x % G, s = u / p.kv_heads, h = u % p.kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = min(max(lens[s], 0), p.max_pages << lg);
    const float scale = 1.0f / sqrtf((float)p.D);
    const size_t row = (size_t)u * G + g;
    float qv[4], o[4] = {0, 0, 0, 0}, m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) qv[c] = lane + 32 * c < p.D ? q[row * p.D + lane + 32 * c] : 0.0f;
    for (int i = warp; i < n; i += 8) {
        const int page = table[(size_t)s * p.max_pages + (i >> lg)];
        const bool ok = page >= 0 && page < p.num_pages;
        float x = 0.0f;
        const int64_t at = ok ? page * p.page_stride + h * p.head_stride + (i & (p.page_tokens - 1)) * p.token_stride : 0;
        if (ok)
            for (int c = 0; c < 4; ++c)
                if (lane + 32 * c < p.D) x = fmaf(qv[c], row_value(kp + at + lane + 32 * c), x);
#pragma unroll
        for (int e = 16; e; e >>= 1) x += __shfl_xor_sync(0xffffffffu, x, e);
        x = ok ? x * scale : -CUDART_INF_F;
        if (logits && lane == 0) logits[row * (p.max_pages << lg) + i] = x;
        const float mn = fmaxf(m, x);
        const float f = m == -CUDART_INF_F ? 0.0f : expf(m - mn), w = mn == -CUDART_INF_F ? 0.0f : expf(x - mn);
        l = l * f + w;
        for (int c = 0; c < 4; ++c) o[c] = o[c] * f + (ok && lane + 32 * c < p.D ? w * row_value(vp + at + lane + 32 * c) : 0.0f);
        m = mn;
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    for (int c = 0; c < 4; ++c) so[warp][lane + 32 * c] = o[c];
    __syncthreads();
    float M = -CUDART_INF_F, L = 0.0f, O = 0.0f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < 8; ++w) {
        const float f = sm[w] == -CUDART_INF_F ? 0.0f : expf(sm[w] - M);
        L += f * sl[w];
        if (threadIdx.x < FATHOM_MAX_D) O += f * so[w][threadIdx.x];
    }
    if (threadIdx.x < p.D) out[row * p.D + threadIdx.x] = L > 0.0f ? O / L : 0.0f;
    if (norm && threadIdx.x == 0) norm[row] = L > 0.0f ? M + logf(L) : 0.0f;
}

__global__ void __launch_bounds__(256)
paged_mass_kernel(fathom_pages p, int lg, int G, const int32_t *__restrict__ lens, const float *__restrict__ logits,
                  const float *__restrict__ norm, float *__restrict__ mass, size_t mass_stride) {
    const int u = blockIdx.y, cap = p.max_pages << lg, n = min(max(lens[u / p.kv_heads], 0), cap);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        float w = 0.0f;
        for (int g = 0; g < G; ++g) w += expf(logits[((size_t)u * G + g) * cap + i] - norm[(size_t)u * G + g]);
        mass[u * mass_stride + i] += w;
    }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T>
void launch_attn(const fathom_pages &p, int G, const float *q, const void *kp, const void *vp, const int32_t *table,
                 const int32_t *lens, float *out, float *logits, float *norm, cudaStream_t st) {
    paged_attn_kernel<T><<<p.seqs * p.kv_heads * G, 256, 0, st>>>(p, log2_of(p.page_tokens), G, q, (const T *)kp,
                                                                  (const T *)vp, table, lens, out, logits, norm);
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
    const size_t rows = (size_t)p.seqs * p.kv_heads * G;
    w.ctas = 0;
    w.ticket_off = 0;
    w.lse_off = align256((size_t)p.seqs * p.kv_heads * sizeof(uint32_t));
    w.part_off = align256(w.lse_off + rows * sizeof(float));
    w.logit_off = w.part_off;
    w.total = align256(w.logit_off + (mass ? rows * ((size_t)p.max_pages * p.page_tokens) * sizeof(float) : 0));
    return w;
}

int launch_paged_attn(const fathom_pages &p, int G, const float *q, const void *kp, const void *vp,
                      const int32_t *table, const int32_t *lens, float *out, float *mass, size_t mass_stride,
                      void *ws, cudaStream_t st) {
    const PagedWorkspace w = paged_workspace_layout(p, G, mass != nullptr);
    float *logits = mass ? (float *)((char *)ws + w.logit_off) : nullptr;
    float *norm = mass ? (float *)((char *)ws + w.lse_off) : nullptr;
    if (p.dtype == FATHOM_BF16) launch_attn<__nv_bfloat16>(p, G, q, kp, vp, table, lens, out, logits, norm, st);
    else launch_attn<__half>(p, G, q, kp, vp, table, lens, out, logits, norm, st);
    int rc = launch_status("paged_attn_kernel");
    if (rc || !mass) return rc;
    const int cap = p.max_pages * p.page_tokens;
    const dim3 grid(cap / 256 / 4 + 1, p.seqs * p.kv_heads);
    paged_mass_kernel<<<grid, 256, 0, st>>>(p, log2_of(p.page_tokens), G, lens, logits, norm, mass, mass_stride);
    return launch_status("paged_mass_kernel");
}

}  // namespace fathom
