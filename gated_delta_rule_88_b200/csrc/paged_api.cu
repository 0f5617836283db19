// paged_api.cu -- the C ABI of the paged latent cache's operators
// (include/kda.h): argument validation, workspace, launch.
#include "api_internal.h"

using kda::aligned16;
using kda::aligned4;
using kda::cuda_fail;
using kda::fail;

// The checks that kda_latent_attn and kda_latent_append share.
static kda_status check_plan(const char *fn, const kda::PagedPlan &p, int dk, kda_dtype dtype) {
    if (!p.page_table || !p.kv_lens) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (!aligned4(p.page_table) || !aligned4(p.kv_lens) || !aligned4(p.cu_seqlens))
        return fail(KDA_ERR_INVALID_ARG, "%s: page_table, kv_lens and cu_seqlens must be 4-byte aligned", fn);
    if (p.T < 0 || p.H <= 0 || dk <= 0 || p.N <= 0 || p.num_pages <= 0 || p.max_pages <= 0)
        return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes T=%d H=%d dk=%d num_seqs=%d num_pages=%d max_pages=%d", fn,
                    p.T, p.H, dk, p.N, p.num_pages, p.max_pages);
    if (p.N > 65535) return fail(KDA_ERR_INVALID_ARG, "%s: num_seqs=%d exceeds 65535", fn, p.N);
    if (p.H > 65535) return fail(KDA_ERR_INVALID_ARG, "%s: H=%d exceeds 65535", fn, p.H);
    if (!p.cu_seqlens && p.T % p.N)
        return fail(KDA_ERR_INVALID_ARG, "%s: without cu_seqlens T must be a multiple of num_seqs (%d, %d)", fn, p.T,
                    p.N);
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (p.page_size != 16 && p.page_size != 32 && p.page_size != 64 && p.page_size != 128)
        return fail(KDA_ERR_UNSUPPORTED, "%s: page_size=%d (supported: 16, 32, 64, 128)", fn, p.page_size);
    if ((long long)p.max_pages * p.page_size > 0x7fffff00LL)
        return fail(KDA_ERR_INVALID_ARG, "%s: max_pages * page_size exceeds 2^31 - 256", fn);
    if (p.page_stride < (long long)p.page_size * dk || p.page_stride % 8 || p.page_stride > (1LL << 38))
        return fail(KDA_ERR_INVALID_ARG, "%s: page_stride=%lld (a multiple of 8, at least page_size * dk)", fn,
                    p.page_stride);
    if ((long long)p.T * p.H > 0x7fffff00LL || (long long)p.T * p.H * dk > (1LL << 40))
        return fail(KDA_ERR_INVALID_ARG, "%s: problem too large (T=%d H=%d)", fn, p.T, p.H);
    return KDA_OK;
}

static bool finite_f(float x) { return x == x && x <= 3.4028234e38f && x >= -3.4028234e38f; }

// kda_latent_attn; give_up: its waits do so at once.
static kda_status latent_attn(const char *fn, bool give_up, const void *q, const void *cache, const int32_t *page_table,
                              const int32_t *kv_lens, const int32_t *cu_seqlens, void *out, float *lse, int T, int H,
                              int dk, int dv, int num_seqs, int num_pages, int page_size, int max_pages,
                              long long page_stride, float scale, unsigned flags, kda_dtype dtype, void *stream) {
    kda::t_msg[0] = 0;
    if (!q || !cache || !out) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (page_stride == 0) page_stride = (long long)page_size * dk;
    const kda::PagedPlan p{page_table, kv_lens, cu_seqlens, T, H, num_seqs, num_pages, page_size, max_pages, page_stride};
    kda_status s = check_plan(fn, p, dk, dtype);
    if (s != KDA_OK) return s;
    if (flags & ~(unsigned)KDA_ATTN_FULL) return fail(KDA_ERR_INVALID_ARG, "%s: unknown flag bits 0x%x", fn, flags);
    if (!finite_f(scale * 1.4426951f)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out))
        return fail(KDA_ERR_INVALID_ARG, "%s: q, cache and out must be 16-byte aligned", fn);
    if (!aligned4(lse)) return fail(KDA_ERR_INVALID_ARG, "%s: lse must be 4-byte aligned", fn);
    if (dtype != KDA_BF16 || (dv != 256 && dv != 512) || (dk != dv && dk != dv + 64))
        return fail(KDA_ERR_UNSUPPORTED, "%s: dtype=%d dk=%d dv=%d (supported: bf16, dv in {256, 512}, dk - dv in {0, 64})",
                    fn, (int)dtype, dk, dv);
    if (T == 0) return KDA_OK;
    cudaStream_t st = (cudaStream_t)stream;
    cudaMemPool_t mp;
    int sms = 148;
    cudaError_t e = kda::get_pool(&mp, &sms);
    if (e != cudaSuccess) return cuda_fail(e, "kda_latent_attn memory pool");
    void *ws = nullptr;
    const size_t bytes = kda::latent_attn_workspace(p, dv, sms);
    if (bytes && (e = cudaMallocFromPoolAsync(&ws, bytes, mp, st)) != cudaSuccess)
        return cuda_fail(e, "kda_latent_attn workspace allocation");
    e = kda::launch_latent_attn(q, cache, p, out, lse, dk, dv, scale, (flags & KDA_ATTN_FULL) != 0, give_up,
                                ws, sms, kda::error_word(), st);
    cudaError_t e2 = ws ? cudaFreeAsync(ws, st) : cudaSuccess;
    if (e != cudaSuccess) return cuda_fail(e, "kda_latent_attn launch");
    if (e2 != cudaSuccess) return cuda_fail(e2, "kda_latent_attn workspace release");
    return KDA_OK;
}

extern "C" {

kda_status kda_latent_attn(const void *q, const void *cache, const int32_t *page_table, const int32_t *kv_lens,
                           const int32_t *cu_seqlens, void *out, float *lse, int T, int H, int dk, int dv,
                           int num_seqs, int num_pages, int page_size, int max_pages, long long page_stride,
                           float scale, unsigned flags, kda_dtype dtype, void *stream) {
    return latent_attn("kda_latent_attn", false, q, cache, page_table, kv_lens, cu_seqlens, out, lse, T, H,
                       dk, dv, num_seqs, num_pages, page_size, max_pages, page_stride, scale, flags, dtype, stream);
}

kda_status kda_selftest_latent_attn(const void *q, const void *cache, const int32_t *page_table, const int32_t *kv_lens,
                                    const int32_t *cu_seqlens, void *out, float *lse, int T, int H, int dk, int dv,
                                    int num_seqs, int num_pages, int page_size, int max_pages, long long page_stride,
                                    float scale, unsigned flags, kda_dtype dtype, void *stream) {
    kda::t_msg[0] = 0;
    const char *fn = "kda_selftest_latent_attn";
    if (dk != 576 || dv != 512) return fail(KDA_ERR_UNSUPPORTED, "%s: dk=%d dv=%d (supported: 576, 512)", fn, dk, dv);
    return latent_attn(fn, true, q, cache, page_table, kv_lens, cu_seqlens, out, lse, T, H, dk, dv, num_seqs, num_pages,
                       page_size, max_pages, page_stride, scale, flags, dtype, stream);
}

kda_status kda_latent_append(const void *kv, void *cache, const int32_t *page_table, const int32_t *kv_lens,
                             const int32_t *cu_seqlens, const void *q_pe, void *q, const float *freqs, int T, int H,
                             int dk, int rot, int num_seqs, int num_pages, int page_size, int max_pages,
                             long long page_stride, long long kv_stride, long long q_pe_ts, long long q_pe_hs,
                             unsigned flags, float scale, kda_dtype dtype, void *stream) {
    kda::t_msg[0] = 0;
    const char *fn = "kda_latent_append";
    if (!kv || !cache) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (page_stride == 0) page_stride = (long long)page_size * dk;
    const kda::PagedPlan p{page_table, kv_lens, cu_seqlens, T, H, num_seqs, num_pages, page_size, max_pages, page_stride};
    kda_status s = check_plan(fn, p, dk, dtype);
    if (s != KDA_OK) return s;
    if (flags & ~(unsigned)KDA_ROPE_INTERLEAVED)
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown flag bits 0x%x", fn, flags);
    if (!finite_f(scale)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (!q_pe != !q) return fail(KDA_ERR_INVALID_ARG, "%s: q_pe and q come together", fn);
    if (rot < 0 || rot > dk || rot % 16 || rot > 1024 || (rot == 0 && (q_pe || freqs)))
        return fail(KDA_ERR_INVALID_ARG, "%s: rot=%d (a multiple of 16 up to min(dk, 1024); 0 only without q_pe and freqs)",
                    fn, rot);
    if (q_pe_hs == 0) q_pe_hs = rot;
    if (q_pe_ts == 0) q_pe_ts = (long long)H * q_pe_hs;
    if (kv_stride == 0) kv_stride = dk;
    const long long lim = 1LL << 38;
    if (dk % 8 || kv_stride % 8 || kv_stride < dk || kv_stride > lim ||
        (q_pe && (q_pe_hs % 8 || q_pe_ts % 8 || q_pe_hs < rot || q_pe_ts < rot || q_pe_hs > lim || q_pe_ts > lim)))
        return fail(KDA_ERR_INVALID_ARG, "%s: dk and the strides must be multiples of 8 that hold a row (dk=%d kv_stride=%lld "
                    "q_pe_ts=%lld q_pe_hs=%lld)", fn, dk, kv_stride, q_pe_ts, q_pe_hs);
    if (!aligned16(kv) || !aligned16(cache) || !aligned16(q_pe) || !aligned16(q))
        return fail(KDA_ERR_INVALID_ARG, "%s: kv, cache, q_pe and q must be 16-byte aligned", fn);
    if (!aligned4(freqs)) return fail(KDA_ERR_INVALID_ARG, "%s: freqs must be 4-byte aligned", fn);
    if (T == 0) return KDA_OK;
    cudaError_t e = kda::launch_latent_append(kv, cache, p, q_pe, q, freqs, dk, rot, kv_stride, q_pe_ts, q_pe_hs,
                                              (flags & KDA_ROPE_INTERLEAVED) != 0, scale, dtype == KDA_BF16,
                                              kda::error_word(), (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kda_latent_append launch");
    return KDA_OK;
}

kda_status kda_rope(const void *x, const int32_t *positions, const float *freqs, void *out, long long T, int H, int d,
                    int rot, int offset, long long x_stride, long long out_stride, unsigned flags, float scale,
                    kda_dtype dtype, void *stream) {
    kda::t_msg[0] = 0;
    const char *fn = "kda_rope";
    if (!x || !positions || !freqs || !out) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (T < 0 || H <= 0 || d <= 0 || T > 0x7fffffffLL || d > 65536 || (long long)H * d > (1LL << 30))
        return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes T=%lld H=%d d=%d", fn, T, H, d);
    if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (flags & ~(unsigned)(KDA_ROPE_INTERLEAVED | KDA_ROPE_INVERSE))
        return fail(KDA_ERR_INVALID_ARG, "%s: unknown flag bits 0x%x", fn, flags);
    if (!finite_f(scale)) return fail(KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (x_stride == 0) x_stride = (long long)H * d;
    if (out_stride == 0) out_stride = (long long)H * d;
    const long long lim = 1LL << 38;
    if (rot <= 0 || rot % 16 || rot > 1024 || offset < 0 || offset % 8 || d % 8 || offset > d - rot)
        return fail(KDA_ERR_INVALID_ARG, "%s: d=%d rot=%d offset=%d (rot a multiple of 16 up to 1024, d and offset of 8, "
                    "offset + rot <= d)", fn, d, rot, offset);
    if (x_stride % 8 || out_stride % 8 || x_stride < (long long)H * d || out_stride < (long long)H * d ||
        x_stride > lim || out_stride > lim)
        return fail(KDA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 of at least H * d (%lld, %lld)", fn, x_stride,
                    out_stride);
    if (x == out && x_stride != out_stride)
        return fail(KDA_ERR_INVALID_ARG, "%s: in place, the strides must be equal", fn);
    if (!aligned16(x) || !aligned16(out)) return fail(KDA_ERR_INVALID_ARG, "%s: x and out must be 16-byte aligned", fn);
    if (!aligned4(positions) || !aligned4(freqs))
        return fail(KDA_ERR_INVALID_ARG, "%s: positions and freqs must be 4-byte aligned", fn);
    if (T == 0) return KDA_OK;
    cudaError_t e = kda::launch_rope(x, positions, freqs, out, T, H, d, rot, offset, x_stride, out_stride,
                                     (flags & KDA_ROPE_INTERLEAVED) != 0, (flags & KDA_ROPE_INVERSE) != 0, scale,
                                     dtype == KDA_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kda_rope launch");
    return KDA_OK;
}

static kda_status check_pool(const char *fn, const void *pool, int planes, int num_pages, long long page_bytes) {
    if (!pool) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (planes <= 0 || planes > 65535 || num_pages <= 0 || page_bytes <= 0 || page_bytes % 16 || page_bytes > (1LL << 34))
        return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes planes=%d num_pages=%d page_bytes=%lld (planes <= 65535, page_bytes "
                    "a multiple of 16)", fn, planes, num_pages, page_bytes);
    if (!aligned16(pool)) return fail(KDA_ERR_INVALID_ARG, "%s: the pool must be 16-byte aligned", fn);
    return KDA_OK;
}

kda_status kda_pages_copy(void *pool, const int32_t *src, const int32_t *dst, int count, int planes, int num_pages,
                          long long page_bytes, void *stream) {
    kda::t_msg[0] = 0;
    const char *fn = "kda_pages_copy";
    kda_status s = check_pool(fn, pool, planes, num_pages, page_bytes);
    if (s != KDA_OK) return s;
    if (count < 0 || count > 4096) return fail(KDA_ERR_INVALID_ARG, "%s: count=%d out of [0, 4096]", fn, count);
    if (count == 0) return KDA_OK;
    if (!src || !dst) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (!aligned4(src) || !aligned4(dst)) return fail(KDA_ERR_INVALID_ARG, "%s: src and dst must be 4-byte aligned", fn);
    cudaMemPool_t mp;
    int sms = 148;
    cudaError_t e = kda::get_pool(&mp, &sms);
    if (e != cudaSuccess) return cuda_fail(e, "kda_pages_copy device");
    e = kda::launch_pages_copy(pool, src, dst, count, planes, num_pages, page_bytes, sms, kda::error_word(),
                               (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kda_pages_copy launch");
    return KDA_OK;
}

kda_status kda_pages_compact(void *pool, const int32_t *pages, int32_t *new_pages, long long count, int planes,
                             int num_pages, long long page_bytes, void *stream) {
    kda::t_msg[0] = 0;
    const char *fn = "kda_pages_compact";
    kda_status s = check_pool(fn, pool, planes, num_pages, page_bytes);
    if (s != KDA_OK) return s;
    if (num_pages > 524288) return fail(KDA_ERR_INVALID_ARG, "%s: num_pages=%d exceeds 524288", fn, num_pages);
    if (count < 0 || count > (1LL << 31)) return fail(KDA_ERR_INVALID_ARG, "%s: count=%lld out of [0, 2^31]", fn, count);
    if (count == 0) return KDA_OK;                        // nothing is live: nothing moves
    if (!pages || !new_pages) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer argument", fn);
    if (!aligned4(pages) || !aligned4(new_pages))
        return fail(KDA_ERR_INVALID_ARG, "%s: pages and new_pages must be 4-byte aligned", fn);
    cudaStream_t st = (cudaStream_t)stream;
    cudaMemPool_t mp;
    int sms = 148;
    cudaError_t e = kda::get_pool(&mp, &sms);
    if (e != cudaSuccess) return cuda_fail(e, "kda_pages_compact memory pool");
    void *scratch = nullptr;
    e = cudaMallocFromPoolAsync(&scratch, kda::pages_compact_scratch_bytes(num_pages), mp, st);
    if (e != cudaSuccess) return cuda_fail(e, "kda_pages_compact scratch allocation");
    e = kda::launch_pages_compact(pool, pages, new_pages, count, planes, num_pages, page_bytes, (int *)scratch, sms,
                                  kda::error_word(), st);
    cudaError_t e2 = cudaFreeAsync(scratch, st);
    if (e != cudaSuccess) return cuda_fail(e, "kda_pages_compact launch");
    if (e2 != cudaSuccess) return cuda_fail(e2, "kda_pages_compact scratch release");
    return KDA_OK;
}

}  // extern "C"
