// rope.cu -- rotary positions (kda_rope) and the write of new tokens into the
// paged latent cache with them (kda_latent_append).
//
// Pair i of a rotated block of `rot` channels turns by a = position * freqs[i]:
//     (x, y) -> s (x cos a - y sin a, x sin a + y cos a).
// Positions reach 2^31, so a is formed in turns as a sum of two fp64 numbers
// (each product with its rounding error, 1 / 2 pi to 107 bits), reduced by its
// nearest whole number and only then handed to sincospif in fp32: that rounding
// is what is left, and the angle off by at most 2^-25 * pi and a little whatever
// position and frequency (by 2^-24 * 1.7 pi at positions of 2^31 and frequency 1 in
// one fp64 product, and in proportion to the frequency beyond).  Both kernels are memory-bound (each element read once and written
// once): a block first forms the cosines and sines of its tokens in shared
// memory, once for all heads, then streams 16-byte pieces.
// Measured (B200): 8192 tokens of 32 heads, 64 of 192 channels turned, bf16: 33.3 us
// (201 MB, 92% of the measured copy rate); 7167 new tokens of a prompt with 32 heads'
// positional parts, 23 us (75 MB, 49%: rows of 128 bytes, 384 and 1152 apart, and a
// look-up of four dependent loads before them).
#include "kernels.h"
#include "paged.cuh"

namespace kda {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float2 turn(double position, float freq, float scale, bool inverse) {
    constexpr double C = 0.15915494309189533577, C2 = -9.839338337591243e-18;      // 1 / (2 pi) = C + C2
    const double f = freq, hi = __dmul_rn(f, C), lo = __fma_rn(f, C2, __fma_rn(f, C, -hi));
    const double t = __dmul_rn(position, hi), tl = __fma_rn(position, lo, __fma_rn(position, hi, -t));
    const double x = (t - rint(t)) + tl;
    float s, c;
    sincospif((float)(2.0 * (x - rint(x))), &s, &c);
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

// The threads of a group (`self` of `size`) walk over rows of `per` items each,
// row by row: the next item of a thread is found without a division.
struct Step {
    int row, at, drow, dat, per;
    __device__ __forceinline__ Step(int self, int size, int per_) : per(per_) {
        row = self / per; at = self - row * per;
        drow = size / per; dat = size - drow * per;
    }
    __device__ __forceinline__ void next() {
        row += drow; at += dat;
        if (at >= per) { at -= per; ++row; }
    }
};

// `rows` rotated blocks, xs / ys elements apart.  An item is the two 16-byte
// pieces that hold P pairs: neighbours if interleaved, else half a block apart.
template <typename T>
__device__ __forceinline__ void turn_rows(const T *x, long long xs, T *y, long long ys, int rows, int rot,
                                          const float2 *cs, bool interleaved, int self, int size)
{
    constexpr int P = Piece<T>::N;
    for (Step e(self, size, rot / (2 * P)); e.row < rows; e.next()) {
        const int ia = interleaved ? 2 * P * e.at : P * e.at, ib = interleaved ? ia + P : ia + rot / 2;
        const T *xr = x + e.row * xs;
        T *yr = y + e.row * ys;
        const uint4 a = *reinterpret_cast<const uint4 *>(xr + ia), b = *reinterpret_cast<const uint4 *>(xr + ib);
        float2 c[P];
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 two = *reinterpret_cast<const float4 *>(cs + P * e.at + i);
            c[i] = make_float2(two.x, two.y);
            c[i + 1] = make_float2(two.z, two.w);
        }
        float u[P], v[P], p[P], q[P];
        Piece<T>::open(a, u);
        Piece<T>::open(b, v);
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                const float2 f = c[i], g = c[P / 2 + i];
                p[2 * i] = u[2 * i] * f.x - u[2 * i + 1] * f.y;
                p[2 * i + 1] = u[2 * i] * f.y + u[2 * i + 1] * f.x;
                q[2 * i] = v[2 * i] * g.x - v[2 * i + 1] * g.y;
                q[2 * i + 1] = v[2 * i] * g.y + v[2 * i + 1] * g.x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                p[i] = u[i] * c[i].x - v[i] * c[i].y;
                q[i] = u[i] * c[i].y + v[i] * c[i].x;
            }
        }
        *reinterpret_cast<uint4 *>(yr + ia) = Piece<T>::pack(p);
        *reinterpret_cast<uint4 *>(yr + ib) = Piece<T>::pack(q);
    }
}

// `rows` rows of d channels without the `gap` channels from `offset` on, copied;
// COPIES pieces of a thread are in flight at a time.
constexpr int COPIES = 4;

template <typename T>
__device__ __forceinline__ void copy_rows(const T *x, long long xs, T *y, long long ys, int rows, int d, int offset,
                                          int gap, int self, int size)
{
    constexpr int P = Piece<T>::N;
    if (d == gap) return;
    Step e(self, size, (d - gap) / P);
    while (e.row < rows) {
        uint4 v[COPIES];
        T *to[COPIES];
#pragma unroll
        for (int k = 0; k < COPIES; ++k) {
            to[k] = nullptr;
            if (e.row < rows) {
                const int c = e.at * P, at = c < offset ? c : c + gap;
                v[k] = *reinterpret_cast<const uint4 *>(x + e.row * xs + at);
                to[k] = y + e.row * ys + at;
                e.next();
            }
        }
#pragma unroll
        for (int k = 0; k < COPIES; ++k)
            if (to[k]) *reinterpret_cast<uint4 *>(to[k]) = v[k];
    }
}

// Blocks an SM (a limit on registers) and 16-byte pieces of a thread, for 8192 tokens
// of 32 heads of 192 channels: 6 and 8 33.4 us (6.0 TB/s, 92% of the measured copy
// rate); 5 or 4 blocks 34.9 and 37.0 us, 8 blocks 41.3; 16 pieces 35.5, 32 42.4, 4
// pieces 40.4.
constexpr int BLOCKS = 6, ROUNDS = 8;

template <typename T>
__global__ void __launch_bounds__(NT, BLOCKS)
rope_kernel(const T *x, const int32_t *__restrict__ positions, const float *__restrict__ freqs, T *out,
            long long tokens, int H, int d, int rot, int offset, long long xs, long long os, int tpb,
            int heads, bool interleaved, bool inverse, float scale)
{
    // tpb tokens, each by NT / tpb threads, and `heads` of their heads (the blockIdx.y-th share)
    extern __shared__ __align__(16) float2 cs[];         // [tpb][rot / 2]
    const long long t0 = (long long)blockIdx.x * tpb;
    const int nt = (int)min((long long)tpb, tokens - t0);
    const int h0 = blockIdx.y * heads, nh = min(heads, H - h0);
    const int half = rot / 2;
    for (int e = threadIdx.x; e < nt * half; e += NT)
        cs[e] = turn(positions[t0 + e / half], freqs[e % half], scale, inverse);
    const int size = NT / tpb, t = threadIdx.x / size, self = threadIdx.x - t * size;
    const T *xr = x + (t0 + t) * xs + (long long)h0 * d;
    T *yr = out + (t0 + t) * os + (long long)h0 * d;
    if (x != out && t < nt) copy_rows<T>(xr, d, yr, d, nh, d, offset, rot, self, size);
    __syncthreads();
    if (t < nt) turn_rows<T>(xr + offset, d, yr + offset, d, nh, rot, cs + t * half, interleaved, self, size);
}

// Tokens of an append block at most: 7167 tokens with 32 heads take 23.0 us with 4,
// 23.9 with 8, 27.7 with 2 and 40.0 with 1 (a block first looks up where its tokens
// go, four loads one after the other).
constexpr int TPB = 4;

template <typename T>
__global__ void __launch_bounds__(NT, BLOCKS)
latent_append_kernel(const T *__restrict__ kv, T *__restrict__ cache, const int32_t *__restrict__ table,
                     const int32_t *__restrict__ kv_lens, const int32_t *__restrict__ cu,
                     const T *q_pe, T *q, const float *__restrict__ freqs,
                     int tokens, int H, int dk, int rot, int N, int per_seq, int num_pages, int page_size,
                     int max_pages, long long page_stride, long long kvs, long long qts, long long qhs,
                     int tpb, bool interleaved, float scale, int *err)
{
    // tpb tokens, each by 8 / tpb warps.  q_pe may be the channels of q that it is written to: each
    // piece is read and written by one thread.
    extern __shared__ __align__(16) float2 cs[];         // [tpb][rot / 2]
    __shared__ long long place[TPB];                     // offset of the token's cache row, -1: skip
    __shared__ int where[TPB];                           // its position
    const int size = NT / tpb, mine = threadIdx.x / size, self = threadIdx.x - mine * size;
    const int t = blockIdx.x * tpb + mine;
    if (self < 32) {
        const int n = t < tokens ? paged::sequence_of(cu, N, per_seq, tokens, t) : N;
        if (self == 0) {
            long long row = -1;
            int pos = 0;
            const int b = n < N ? paged::token_offset(cu, n, per_seq, tokens) : tokens;
            if (t < tokens && t >= b) {                  // (else it belongs to no sequence: padding)
                const int e = paged::token_offset(cu, n + 1, per_seq, tokens);
                const int len = kv_lens[n];
                const long long at = (long long)len - (e - b) + (t - b);
                int page = -1;
                // (of a sequence of impossible length nothing is written; at < len whenever the offsets do not decrease)
                if (at >= 0 && at < len && len <= (long long)max_pages * page_size) {
                    pos = (int)at;
                    page = table[(long long)n * max_pages + pos / page_size];
                }
                if (page >= 0 && page < num_pages) row = page * page_stride + (long long)(pos % page_size) * dk;
                else set_device_error(err, paged::kErrBadPage);
            }
            place[mine] = row;
            where[mine] = pos;
        }
    }
    __syncthreads();
    const int half = rot / 2;
    if (freqs)
        for (int i = self; i < half; i += size) cs[mine * half + i] = turn(where[mine], freqs[i], scale, false);
    const long long row = place[mine];
    const T *src = kv + t * kvs;
    const int turned = freqs ? rot : 0;
    if (row >= 0) copy_rows<T>(src, 0, cache + row, 0, 1, dk - turned, dk, 0, self, size);
    __syncthreads();
    if (row < 0) return;
    const float2 *c = cs + mine * half;
    if (freqs) turn_rows<T>(src + dk - rot, 0, cache + row + dk - rot, 0, 1, rot, c, interleaved, self, size);
    if (q) {
        const T *x = q_pe + t * qts;
        T *y = q + (long long)t * H * dk + dk - rot;
        if (freqs) turn_rows<T>(x, qhs, y, dk, H, rot, c, interleaved, self, size);
        else copy_rows<T>(x, qhs, y, dk, H, rot, rot, 0, self, size);
    }
}

template <typename T>
cudaError_t rope_t(const void *x, const int32_t *positions, const float *freqs, void *out, long long tokens,
                   int H, int d, int rot, int offset, long long xs, long long os, bool interleaved,
                   bool inverse, float scale, cudaStream_t st)
{
    // a block: about ROUNDS 16-byte pieces a thread, of up to eight tokens or of a share of one token's heads
    const int per = (x == out ? rot : d) / Piece<T>::N;
    int heads = ROUNDS * NT / per;
    heads = heads < 1 ? 1 : heads > H ? H : heads;
    int shares = (H + heads - 1) / heads;
    heads = (H + shares - 1) / shares;
    shares = (H + heads - 1) / heads;
    int tpb = 1;
    while (shares == 1 && tpb < 8 && 2LL * tpb * H * per <= ROUNDS * NT && tokens / (2 * tpb) >= 512) tpb *= 2;
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
    // fewer tokens a block while there are not 512 blocks
    int tpb = TPB;
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
