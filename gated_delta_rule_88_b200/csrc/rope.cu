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
    static __device__ __forceinline__ void open(const uint4 &x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(const uint4 &x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
};

// An item is two 16-byte pieces: the two that hold P pairs of a rotated block
// (neighbours if interleaved, else half a block apart), or two to be copied.
template <typename T>
struct Item {
    const T *x0, *x1;            // x1 null: no second piece
    T *y0, *y1;
    const float2 *cs;            // of the item's pairs; null: copied
    // item j of a rotated block of `rot` channels
    __device__ __forceinline__ void turned(const T *x, T *y, const float2 *table, int j, int rot, bool interleaved) {
        constexpr int P = Piece<T>::N;
        const int ia = interleaved ? 2 * P * j : P * j, ib = interleaved ? ia + P : ia + rot / 2;
        x0 = x + ia; x1 = x + ib; y0 = y + ia; y1 = y + ib;
        cs = table + P * j;
    }
    // channels [c, c + P) and [d, d + P) (none if d < 0)
    __device__ __forceinline__ void copied(const T *x, T *y, int c, int d) {
        x0 = x + c; y0 = y + c;
        x1 = d < 0 ? nullptr : x + d; y1 = y + d;
        cs = nullptr;
    }
    __device__ __forceinline__ void run(bool interleaved) {
        constexpr int P = Piece<T>::N;
        uint4 a = *reinterpret_cast<const uint4 *>(x0), b = make_uint4(0, 0, 0, 0);
        if (x1) b = *reinterpret_cast<const uint4 *>(x1);
        if (cs) {
            float u[P], v[P], p[P], q[P];
            Piece<T>::open(a, u);
            Piece<T>::open(b, v);
            if (interleaved) {
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                    const float2 c = cs[i], d = cs[P / 2 + i];
                    p[2 * i] = u[2 * i] * c.x - u[2 * i + 1] * c.y;
                    p[2 * i + 1] = u[2 * i] * c.y + u[2 * i + 1] * c.x;
                    q[2 * i] = v[2 * i] * d.x - v[2 * i + 1] * d.y;
                    q[2 * i + 1] = v[2 * i] * d.y + v[2 * i + 1] * d.x;
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 c = cs[i];
                    p[i] = u[i] * c.x - v[i] * c.y;
                    q[i] = u[i] * c.y + v[i] * c.x;
                }
            }
            a = Piece<T>::pack(p);
            b = Piece<T>::pack(q);
        }
        *reinterpret_cast<uint4 *>(y0) = a;
        if (x1) *reinterpret_cast<uint4 *>(y1) = b;
    }
};

// e / n with inv = 1.f / n: (e + 1/2) / n lies 1 / (2 n) or more from every whole
// number, and the product is off by at most 2^-23 of it, so it is exact while
// (e / n) n < 2^22, i.e. e < 2^22.
__device__ __forceinline__ int quotient(int e, float inv) { return (int)(((float)e + 0.5f) * inv); }

// Blocks an SM and rounds of a block's threads over its items, for 8192 tokens of
// 32 heads of 192 channels: six blocks and eight rounds 36.8 us; four rounds 42.6;
// two or four items of a thread in flight in fewer blocks 37.2 to 46.7.
constexpr int BLOCKS = 6, ROUNDS = 8;

template <typename T>
__global__ void __launch_bounds__(NT, BLOCKS)
rope_kernel(const T *x, const int32_t *__restrict__ positions, const float *__restrict__ freqs, T *out,
            long long tokens, int H, int d, int rot, int offset, long long xs, long long os, int tpb,
            int heads, bool interleaved, bool inverse, float scale)
{
    // tpb tokens, and `heads` of their heads (blockIdx.y-th share)
    extern __shared__ float2 cs[];                       // [tpb][rot / 2]
    constexpr int P = Piece<T>::N;
    const long long t0 = (long long)blockIdx.x * tpb;
    const int nt = (int)min((long long)tpb, tokens - t0);
    const int h0 = blockIdx.y * heads, nh = min(heads, H - h0);
    const int half = rot / 2;
    for (int e = threadIdx.x; e < nt * half; e += NT)
        cs[e] = turn(positions[t0 + e / half], freqs[e % half], scale, inverse);
    __syncthreads();
    // items of a head: the rotated ones, then (out of place) the other pieces two by two
    const int nrot = rot / (2 * P), rest = (d - rot) / P;
    const int per = nrot + (x == out ? 0 : (rest + 1) / 2);
    const int all = nt * nh * per;
    const float inv_per = 1.f / per, inv_nh = 1.f / nh;
    for (int e = threadIdx.x; e < all; e += NT) {
        const int th = quotient(e, inv_per), j = e - th * per;
        const int t = quotient(th, inv_nh), h = h0 + th - t * nh;
        const T *xr = x + (t0 + t) * xs + (long long)h * d;
        T *yr = out + (t0 + t) * os + (long long)h * d;
        Item<T> it;
        if (j < nrot) {
            it.turned(xr + offset, yr + offset, cs + t * half, j, rot, interleaved);
        } else {
            const int c = 2 * (j - nrot) * P, c2 = c + P;
            it.copied(xr, yr, c < offset ? c : c + rot, c2 >= rest * P ? -1 : c2 < offset ? c2 : c2 + rot);
        }
        it.run(interleaved);
    }
}

constexpr int TPB = 8;          // tokens of an append block at most: one a warp

template <typename T>
__global__ void __launch_bounds__(NT, 8)
latent_append_kernel(const T *__restrict__ kv, T *__restrict__ cache, const int32_t *__restrict__ table,
                     const int32_t *__restrict__ kv_lens, const int32_t *__restrict__ cu,
                     const T *__restrict__ q_pe, T *__restrict__ q, const float *__restrict__ freqs,
                     int tokens, int H, int dk, int rot, int N, int per_seq, int num_pages, int page_size,
                     int max_pages, long long page_stride, long long kvs, long long qts, long long qhs,
                     int tpb, bool interleaved, float scale, int *err)
{
    extern __shared__ float2 cs[];                       // [tpb][rot / 2]
    __shared__ long long place[TPB];                     // offset of the token's cache row, -1: skip
    __shared__ int where[TPB];                           // its position
    constexpr int P = Piece<T>::N;
    const int t0 = blockIdx.x * tpb, nt = min(tpb, tokens - t0);
    const int warp = threadIdx.x >> 5;
    if (warp < nt) {
        const int t = t0 + warp;
        const int n = paged::sequence_of(cu, N, per_seq, tokens, t);
        if ((threadIdx.x & 31) == 0) {
            long long row = -1;
            int pos = 0;
            const int b = n < N ? paged::token_offset(cu, n, per_seq, tokens) : tokens;
            if (t >= b) {                                // (else it belongs to no sequence: padding)
                const int e = paged::token_offset(cu, n + 1, per_seq, tokens);
                const long long at = (long long)kv_lens[n] - (e - b) + (t - b);
                int page = -1;
                if (at >= 0 && at < (long long)max_pages * page_size) {
                    pos = (int)at;
                    page = table[(long long)n * max_pages + pos / page_size];
                }
                if (page >= 0 && page < num_pages) row = page * page_stride + (long long)(pos % page_size) * dk;
                else set_device_error(err, paged::kErrBadPage);
            }
            place[warp] = row;
            where[warp] = pos;
        }
    }
    __syncthreads();
    const int half = rot / 2;
    if (freqs) {
        for (int e = threadIdx.x; e < nt * half; e += NT) cs[e] = turn(where[e / half], freqs[e % half], scale, false);
        __syncthreads();
    }
    // items of a token: its latent (turned at the end, the rest copied), then each head of q
    const int turned = freqs ? rot : 0;
    const int nrot = turned / (2 * P), rest = (dk - turned) / P, nkv = nrot + (rest + 1) / 2;
    const int nq = q ? rot / (2 * P) : 0;
    const int per = nkv + nq * H;
    const int all = nt * per;
    const float inv_per = 1.f / per, inv_nq = nq ? 1.f / nq : 0.f;
    for (int e = threadIdx.x; e < all; e += NT) {
        const int t = tpb == 1 ? 0 : quotient(e, inv_per), j = e - t * per;
        if (place[t] < 0) continue;
        const float2 *c = cs + t * half;
        Item<T> it;
        if (j < nkv) {
            const T *src = kv + (t0 + t) * kvs;
            T *row = cache + place[t];
            if (j < nrot) it.turned(src + dk - rot, row + dk - rot, c, j, rot, interleaved);
            else it.copied(src, row, 2 * (j - nrot) * P, 2 * (j - nrot) + 1 < rest ? (2 * (j - nrot) + 1) * P : -1);
        } else {
            const int h = quotient(j - nkv, inv_nq), i = j - nkv - h * nq;
            const T *src = q_pe + (t0 + t) * qts + h * qhs;
            T *row = q + ((long long)(t0 + t) * H + h) * dk + dk - rot;
            if (freqs) it.turned(src, row, c, i, rot, interleaved);
            else it.copied(src, row, 2 * i * P, (2 * i + 1) * P);
        }
        it.run(interleaved);
    }
}

template <typename T>
cudaError_t rope_t(const void *x, const int32_t *positions, const float *freqs, void *out, long long tokens,
                   int H, int d, int rot, int offset, long long xs, long long os, bool interleaved,
                   bool inverse, float scale, cudaStream_t st)
{
    // a block: ROUNDS items a thread, from several tokens or from a share of one token's heads
    constexpr int P = Piece<T>::N;
    const int per = x == out ? rot / (2 * P) : (d / P + 1) / 2;
    const int want = ROUNDS * NT;
    int heads = want / per;
    heads = heads < 1 ? 1 : heads > H ? H : heads;
    int shares = (H + heads - 1) / heads;
    heads = (H + shares - 1) / shares;
    shares = (H + heads - 1) / heads;
    int tpb = want / (heads * per);
    tpb = shares > 1 || tpb < 1 ? 1 : tpb > 16 ? 16 : tpb;
    // few tokens: no more than a round a block
    while (tpb > 1 && tokens / tpb < 512) tpb >>= 1;
    const long long blocks = (tokens + tpb - 1) / tpb;
    if (blocks > 0x7fffffffLL || shares > 65535) return cudaErrorInvalidValue;
    rope_kernel<T><<<dim3((unsigned)blocks, shares), NT, sizeof(float2) * tpb * (rot / 2), st>>>(
        (const T *)x, positions, freqs, (T *)out, tokens, H, d, rot, offset, xs, os, tpb, heads, interleaved, inverse,
        scale);
    return cudaGetLastError();
}

template <typename T>
cudaError_t append_t(const void *kv, void *cache, const PagedPlan &p, const void *q_pe, void *q, const float *freqs,
                     int dk, int rot, long long kvs, long long qts, long long qhs, bool interleaved, float scale,
                     int *err, cudaStream_t st)
{
    // tokens of a block: up to eight (a warp each for their places), while 512 blocks and more are left;
    // heads so many that quotient() would not be exact get one
    int tpb = (long long)p.H * dk > (1 << 18) ? 1 : TPB;
    while (tpb > 1 && p.T / tpb < 512) tpb >>= 1;
    latent_append_kernel<T><<<(p.T + tpb - 1) / tpb, NT, sizeof(float2) * tpb * (rot / 2), st>>>(
        (const T *)kv, (T *)cache, p.page_table, p.kv_lens, p.cu_seqlens, (const T *)q_pe, (T *)q, freqs, p.T, p.H, dk,
        rot, p.N, p.cu_seqlens ? 1 : p.T / p.N, p.num_pages, p.page_size, p.max_pages, p.page_stride, kvs, qts, qhs,
        tpb, interleaved, scale, err);
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
