// latent_attn.cu -- attention of each sequence's new tokens over the paged
// latent cache (kda_latent_attn), the plain version: one block a (token, head).
#include "kernels.h"
#include "paged.cuh"

namespace kda {
namespace {

constexpr int NT = 128;

__global__ void __launch_bounds__(NT)
latent_attn_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ cache,
                   const int32_t *__restrict__ table, const int32_t *__restrict__ kv_lens,
                   const int32_t *__restrict__ cu, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse,
                   int tokens, int H, int dk, int dv, int N, int per_seq, int num_pages, int page_size,
                   int max_pages, long long page_stride, float scale, bool full, int *err)
{
    __shared__ float qs[576], p[NT], red[4];
    __shared__ int seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    const int t = (int)(row / H);
    if (warp == 0) {
        const int n = paged::sequence_of(cu, N, per_seq, tokens, t);
        if (lane == 0) seq = n;
    }
    __syncthreads();
    if (seq >= N) return;
    const int b = paged::token_offset(cu, seq, per_seq, tokens), e = paged::token_offset(cu, seq + 1, per_seq, tokens);
    if (t < b) return;
    const int kv = kv_lens[seq];
    bool bad = kv < 0 || kv > (long long)max_pages * page_size;
    if (!bad)
        for (int i = tid; i * page_size < kv; i += NT) {
            const int pg = table[(long long)seq * max_pages + i];
            bad |= pg < 0 || pg >= num_pages;
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_device_error(err, paged::kErrBadPage);
        return;
    }
    const int see = full ? kv : min(kv, max(0, kv - (e - b) + (t - b) + 1));
    for (int c = tid; c < dk; c += NT) qs[c] = to_f(q[row * dk + c]) * scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < see; j0 += NT) {
        const int j = j0 + tid;
        float x = -INFINITY;
        if (j < see) {
            const __nv_bfloat16 *k = cache + table[(long long)seq * max_pages + j / page_size] * page_stride +
                                     (long long)(j % page_size) * dk;
            x = 0.f;
            for (int c = 0; c < dk; ++c) x = fmaf(qs[c], to_f(k[c]), x);
        }
        float mx = x;
        for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        mx = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float f = expf(m - mx);
        m = mx;
        p[tid] = expf(x - m);
        __syncthreads();
        l *= f;
        for (int i = 0; i < 4; ++i) o[i] *= f;
        for (int i = 0; i < min(NT, see - j0); ++i) {
            const int jj = j0 + i;
            const __nv_bfloat16 *k = cache + table[(long long)seq * max_pages + jj / page_size] * page_stride +
                                     (long long)(jj % page_size) * dk;
            l += p[i];
            for (int c = 0; c < dv / NT; ++c) o[c] = fmaf(p[i], to_f(k[tid + c * NT]), o[c]);
        }
        __syncthreads();
    }
    for (int c = 0; c < dv / NT; ++c)
        out[row * dv + tid + c * NT] = from_f<__nv_bfloat16>(l > 0.f ? o[c] / l : 0.f);
    if (lse && tid == 0) lse[row] = m + logf(l);
}

}  // namespace

cudaError_t launch_latent_attn(const void *q, const void *cache, const PagedPlan &p, void *out, float *lse,
                               int dk, int dv, float scale, bool full, int *err, cudaStream_t st)
{
    latent_attn_kernel<<<p.T * p.H, NT, 0, st>>>(
        (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)cache, p.page_table, p.kv_lens, p.cu_seqlens,
        (__nv_bfloat16 *)out, lse, p.T, p.H, dk, dv, p.N, p.cu_seqlens ? 1 : p.T / p.N, p.num_pages, p.page_size,
        p.max_pages, p.page_stride, scale, full, err);
    return cudaGetLastError();
}

}  // namespace kda
