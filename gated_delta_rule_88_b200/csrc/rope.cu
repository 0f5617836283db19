// rope.cu -- rotary positions (kda_rope) and the write of new tokens into the
// paged latent cache with them (kda_latent_append).
//
// Pair i of a rotated block of `rot` channels turns by a = position * freqs[i]:
//     (x, y) -> s (x cos a - y sin a, x sin a + y cos a).
// Positions reach 2^31, so a is formed in turns in fp64 (one product with
// freqs[i] / 2 pi), reduced by its nearest whole number and only then handed to
// sincospif in fp32: the angle is off by at most 2^-24 * pi whatever the
// position.  Both kernels are memory-bound (each element read once and written
// once): a block first forms the cosines and sines of its tokens in shared
// memory, once for all heads, then streams 16-byte pieces.
#include "kernels.h"
#include "paged.cuh"

namespace kda {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float2 turn(double position, float freq, float scale, bool inverse) {
    const double turns = position * ((double)freq * 0.15915494309189533577);    // 1 / (2 pi)
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    return make_float2(c * scale, (inverse ? -s : s) * scale);
}

// 16 bytes as values and back
template <typename T> struct Piece;
template <> struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&v)[4]) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[8]) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                   pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
};

// Item j (0 <= j < rot / (2 Piece::N)) of a rotated block: two 16-byte pieces,
// either neighbours (interleaved) or half a block apart.
template <typename T>
__device__ __forceinline__ void rotate_item(const T *x, T *y, const float2 *cs, int j, int rot,
                                            bool interleaved) {
    constexpr int P = Piece<T>::N;
    float a[P], b[P], u[P], v[P];
    const int ia = interleaved ? 2 * P * j : P * j;
    const int ib = interleaved ? ia + P : ia + rot / 2;
    Piece<T>::load(x + ia, a);
    Piece<T>::load(x + ib, b);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            const float2 c = cs[P * j + i], d = cs[P * j + P / 2 + i];
            u[2 * i] = a[2 * i] * c.x - a[2 * i + 1] * c.y;
            u[2 * i + 1] = a[2 * i] * c.y + a[2 * i + 1] * c.x;
            v[2 * i] = b[2 * i] * d.x - b[2 * i + 1] * d.y;
            v[2 * i + 1] = b[2 * i] * d.y + b[2 * i + 1] * d.x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 c = cs[P * j + i];
            u[i] = a[i] * c.x - b[i] * c.y;
            v[i] = a[i] * c.y + b[i] * c.x;
        }
    }
    Piece<T>::store(y + ia, u);
    Piece<T>::store(y + ib, v);
}

template <typename T>
__device__ __forceinline__ void copy_piece(const T *x, T *y) {
    *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<const uint4 *>(x);
}

template <typename T>
__global__ void __launch_bounds__(NT)
rope_kernel(const T *x, const int32_t *__restrict__ positions, const float *__restrict__ freqs, T *out,
            long long tokens, int H, int d, int rot, int offset, long long xs, long long os, int tpb,
            bool interleaved, bool inverse, float scale)
{
    extern __shared__ float2 cs[];                       // [tpb][rot / 2]
    constexpr int P = Piece<T>::N;
    const long long t0 = (long long)blockIdx.x * tpb;
    const int nt = (int)min((long long)tpb, tokens - t0);
    const int half = rot / 2;
    for (int e = threadIdx.x; e < nt * half; e += NT)
        cs[e] = turn(positions[t0 + e / half], freqs[e % half], scale, inverse);
    __syncthreads();
    // items of a head: the rotated pairs of pieces, then (out of place) the other pieces
    const int nrot = rot / (2 * P);
    const int per = nrot + (x == out ? 0 : (d - rot) / P);
    const int all = nt * H * per;
    for (int e = threadIdx.x; e < all; e += NT) {
        const int th = e / per, j = e - th * per;
        const int t = th / H, h = th - t * H;
        const T *xr = x + (t0 + t) * xs + (long long)h * d;
        T *yr = out + (t0 + t) * os + (long long)h * d;
        if (j < nrot) {
            rotate_item<T>(xr + offset, yr + offset, cs + t * half, j, rot, interleaved);
        } else {
            const int c = (j - nrot) * P;
            const int at = c < offset ? c : c + rot;
            copy_piece<T>(xr + at, yr + at);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(NT)
latent_append_kernel(const T *__restrict__ kv, T *__restrict__ cache, const int32_t *__restrict__ table,
                     const int32_t *__restrict__ kv_lens, const int32_t *__restrict__ cu,
                     const T *__restrict__ q_pe, T *__restrict__ q, const float *__restrict__ freqs,
                     int tokens, int H, int dk, int rot, int N, int per_seq, int num_pages, int page_size,
                     int max_pages, long long page_stride, long long kvs, long long qts, long long qhs,
                     bool interleaved, float scale, int *err)
{
    // one token a block: its place, its cosines and sines, then its pieces
    extern __shared__ float2 cs[];                       // [rot / 2]
    __shared__ int place[2];                             // page (-1: skip), row in it
    __shared__ int where;                                // position
    constexpr int P = Piece<T>::N;
    const int t = blockIdx.x;
    if (threadIdx.x < 32) {
        const int n = paged::sequence_of(cu, N, per_seq, tokens, t);
        if (threadIdx.x == 0) {
            int page = -1, pos = 0;
            if (n < N) {
                // a token behind the last sequence is no error: it is padding
                const int b = paged::token_offset(cu, n, per_seq, tokens);
                const int e = paged::token_offset(cu, n + 1, per_seq, tokens);
                const long long at = (long long)kv_lens[n] - (e - b) + (t - b);
                if (t < b) page = -2;                    // before the first sequence: padding as well
                else if (at >= 0 && at < (long long)max_pages * page_size) {
                    pos = (int)at;
                    page = table[(long long)n * max_pages + pos / page_size];
                }
                if (page != -2 && (page < 0 || page >= num_pages)) {
                    page = -1;
                    set_device_error(err, paged::kErrBadPage);
                }
            }
            place[0] = page;
            place[1] = pos % page_size;
            where = pos;
        }
    }
    __syncthreads();
    if (place[0] < 0) return;
    const int half = rot / 2;
    if (freqs) {
        for (int i = threadIdx.x; i < half; i += NT) cs[i] = turn(where, freqs[i], scale, false);
        __syncthreads();
    }
    const T *src = kv + t * kvs;
    T *row = cache + (long long)place[0] * page_stride + (long long)place[1] * dk;
    const int turned = freqs ? rot : 0;
    const int nrot = turned / (2 * P), ncopy = (dk - turned) / P;
    // a head of q: its rotary part turned, or copied without positions
    const int nq = q ? (freqs ? rot / (2 * P) : rot / P) : 0;
    const int all = nrot + ncopy + nq * H;
    for (int e = threadIdx.x; e < all; e += NT) {
        if (e < ncopy) {
            copy_piece<T>(src + e * P, row + e * P);
        } else if (e < ncopy + nrot) {
            rotate_item<T>(src + dk - rot, row + dk - rot, cs, e - ncopy, rot, interleaved);
        } else {
            const int h = (e - ncopy - nrot) / nq, j = (e - ncopy - nrot) - h * nq;
            const T *x = q_pe + t * qts + h * qhs;
            T *y = q + ((long long)t * H + h) * dk + dk - rot;
            if (freqs) rotate_item<T>(x, y, cs, j, rot, interleaved);
            else copy_piece<T>(x + j * P, y + j * P);
        }
    }
}

template <typename T>
cudaError_t rope_t(const void *x, const int32_t *positions, const float *freqs, void *out, long long tokens,
                   int H, int d, int rot, int offset, long long xs, long long os, bool interleaved,
                   bool inverse, float scale, cudaStream_t st)
{
    // tokens of a block: enough pieces for four rounds of its threads
    const int pieces = H * (d / Piece<T>::N);
    int tpb = 4 * NT / (pieces > 0 ? pieces : 1);
    tpb = tpb < 1 ? 1 : tpb > 16 ? 16 : tpb;
    const long long blocks = (tokens + tpb - 1) / tpb;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    rope_kernel<T><<<(unsigned)blocks, NT, sizeof(float2) * tpb * (rot / 2), st>>>(
        (const T *)x, positions, freqs, (T *)out, tokens, H, d, rot, offset, xs, os, tpb, interleaved, inverse,
        scale);
    return cudaGetLastError();
}

template <typename T>
cudaError_t append_t(const void *kv, void *cache, const PagedPlan &p, const void *q_pe, void *q, const float *freqs,
                     int dk, int rot, long long kvs, long long qts, long long qhs, bool interleaved, float scale,
                     int *err, cudaStream_t st)
{
    latent_append_kernel<T><<<p.T, NT, sizeof(float2) * (rot / 2), st>>>(
        (const T *)kv, (T *)cache, p.page_table, p.kv_lens, p.cu_seqlens, (const T *)q_pe, (T *)q, freqs, p.T, p.H, dk,
        rot, p.N, p.cu_seqlens ? 1 : p.T / p.N, p.num_pages, p.page_size, p.max_pages, p.page_stride, kvs, qts, qhs,
        interleaved, scale, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const void *x, const int32_t *positions, const float *freqs, void *out,
                        long long tokens, int H, int d, int rot, int offset, long long x_stride,
                        long long out_stride, bool interleaved, bool inverse, float scale, bool bf16,
                        cudaStream_t st)
{
    return bf16 ? rope_t<__nv_bfloat16>(x, positions, freqs, out, tokens, H, d, rot, offset, x_stride,
                                        out_stride, interleaved, inverse, scale, st)
                : rope_t<float>(x, positions, freqs, out, tokens, H, d, rot, offset, x_stride, out_stride,
                                interleaved, inverse, scale, st);
}

cudaError_t launch_latent_append(const void *kv, void *cache, const PagedPlan &p, const void *q_pe, void *q,
                                 const float *freqs, int dk, int rot, long long kv_stride, long long q_pe_ts,
                                 long long q_pe_hs, bool interleaved, float scale, bool bf16, int *err,
                                 cudaStream_t st)
{
    return bf16 ? append_t<__nv_bfloat16>(kv, cache, p, q_pe, q, freqs, dk, rot, kv_stride, q_pe_ts, q_pe_hs,
                                          interleaved, scale, err, st)
                : append_t<float>(kv, cache, p, q_pe, q, freqs, dk, rot, kv_stride, q_pe_ts, q_pe_hs, interleaved,
                                  scale, err, st);
}

}  // namespace kda
