// prefill.cu -- causal attention of packed prompts (grouped query heads).
#include <cuda_bf16.h>

#include "fathom_internal.cuh"

namespace fathom {

namespace {

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half *o) { *o = __float2half_rn(x); }

// One warp per (query token, head): lane l holds channels l + 32 c; running
// maximum, sum and weighted values over the keys one at a time.
template <typename T>
__global__ void __launch_bounds__(256)
prefill_row_kernel(fathom_prompts p, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                   const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, T *__restrict__ out,
                   float *__restrict__ lse) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.total_q * p.heads) return;
    const int t = (int)(row / p.heads), h = (int)(row % p.heads);
    int lo = 0, hi = p.seqs;   // the last sequence that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const int q0 = cu_q[lo], q1 = min(cu_q[lo + 1], p.total_q);
    if (t < q0 || t >= q1) return;
    const int k0 = max(cu_k[lo], 0), k1 = min(cu_k[lo + 1], p.total_k);
    const int seen = min(k1 - k0, t - q0 + 1 + (k1 - k0) - (q1 - q0));
    const int hk = h / (p.heads / p.kv_heads);
    const float scale = 1.0f / sqrtf((float)p.D);
    float qv[4], o[4] = {0, 0, 0, 0}, m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = lane + 32 * c;
        qv[c] = j < p.D ? to_float(q[t * p.q_token + h * p.q_head + j]) : 0.0f;
    }
    for (int i = 0; i < seen; ++i) {
        const T *kr = k + (k0 + i) * p.k_token + hk * p.k_head, *vr = v + (k0 + i) * p.v_token + hk * p.v_head;
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = lane + 32 * c;
            if (j < p.D) s = fmaf(qv[c], to_float(kr[j]), s);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= scale;
        const float mn = fmaxf(m, s);
        const float f = m == -CUDART_INF_F ? 0.0f : expf(m - mn), w = mn == -CUDART_INF_F ? 0.0f : expf(s - mn);
        l = l * f + w;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = lane + 32 * c;
            if (j < p.D) o[c] = o[c] * f + w * to_float(vr[j]);
        }
        m = mn;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int j = lane + 32 * c;
        if (j < p.D) from_float(l > 0.0f ? o[c] / l : 0.0f, out + t * p.out_token + h * p.out_head + j);
    }
    if (lse && lane == 0) lse[(size_t)t * p.heads + h] = l > 0.0f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace

int launch_prefill_attn(const fathom_prompts &p, const void *q, const void *k, const void *v, const int32_t *cu_q,
                        const int32_t *cu_k, void *out, float *lse, cudaStream_t st) {
    const long long rows = (long long)p.total_q * p.heads;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (p.dtype == FATHOM_BF16)
        prefill_row_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p, (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)k,
                                                                (const __nv_bfloat16 *)v, cu_q, cu_k,
                                                                (__nv_bfloat16 *)out, lse);
    else
        prefill_row_kernel<__half><<<grid, 256, 0, st>>>(p, (const __half *)q, (const __half *)k, (const __half *)v,
                                                         cu_q, cu_k, (__half *)out, lse);
    return launch_status("prefill_row_kernel");
}

}  // namespace fathom
