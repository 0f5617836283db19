// pages.cu -- pages of a pool copied, exchanged, cleared and compacted
// (kda_pages_copy, kda_pages_compact).
//
// Both only move bytes: one read and one write of each moved page bound them.
// Measured (B200): 8 states of 2 MB forked into 28 slots and 4 slots cleared, 16.4 us
// (12.8 at the measured copy rate, every source read and every destination written
// once); three pages of 72 KB 2.6 us; 498 of 1200 live pages of 72 KB in 7 planes
// moved, 94 us (78), of which 82 move the pages (95% of the copy rate) and the rest
// is the plan, one block that the moves wait for.
//
// kda_pages_copy takes any list of moves, also overlapping ones ("as before
// the call").  Byte ranges of a page are independent of each other, so a CTA
// takes one range of the page and carries it through ALL moves: it reads the
// range of every source into shared memory, and writes only after the last
// read has landed.  No scratch memory, no ordering between CTAs, no analysis of
// the list.
#include "kernels.h"
#include "paged.cuh"

namespace kda {
namespace {

constexpr int NT = 256;

// The kernels' limits on shared memory are set to what the largest calls take, never to what
// this one does: the limit belongs to the function, and a call on another thread may set it
// between this one's setting and its launch.
constexpr size_t COPY_SMEM = 4096 * 32 + 4096 * 8 + 8192 * 8;      // 4096 moves, 32 bytes each
constexpr size_t PLAN_SMEM = 524288 / 32 * 8;                      // 524,288 pages

// Shared memory of a CTA: the moves' data, (source, destination) of each move
// that counts, and a hash table {destination, last move to it} of `slots` entries
// (a power of two >= 2 count).  piece = 16 << lsh bytes.
__global__ void __launch_bounds__(NT)
pages_copy_kernel(unsigned char *pool, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  int count, int num_pages, long long page_bytes, int lsh, int slots, int *err)
{
    extern __shared__ __align__(16) unsigned char sm[];
    int2 *move = reinterpret_cast<int2 *>(sm + ((size_t)count << (lsh + 4)));
    int *key = reinterpret_cast<int *>(move + count);
    int *last = key + slots;
    const long long at = (long long)blockIdx.x << (lsh + 4);
    const int lanes = (int)min(1LL << lsh, (page_bytes - at) / 16);          // 16-byte lanes of the range
    unsigned char *base = pool + (long long)blockIdx.y * num_pages * page_bytes + at;
    bool bad = false;
    for (int i = threadIdx.x; i < count; i += NT) {
        const int s = src[i], d = dst[i];
        const bool ok = d >= 0 && d < num_pages && s >= -1 && s < num_pages;
        bad |= !ok;
        move[i] = make_int2(s, ok ? d : -1);
    }
    for (int i = threadIdx.x; i < slots; i += NT) { key[i] = -1; last[i] = -1; }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) set_device_error(err, kErrBadSlot);
    __syncthreads();
    for (int e = threadIdx.x; e < count << lsh; e += NT) {
        const int i = e >> lsh, l = e & ((1 << lsh) - 1);
        const int2 m = move[i];
        if (m.y < 0 || l >= lanes) continue;
        unsigned char *to = sm + (size_t)e * 16;
        if (m.x >= 0) cp_async16(to, base + (long long)m.x * page_bytes + 16 * l);
        else *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
    }
    cp_async_commit();
    // while the copies land: the last move to each destination is the one that counts
    auto slot_of = [&](int d) { return (int)(((unsigned)d * 2654435761u) & (unsigned)(slots - 1)); };
    for (int i = threadIdx.x; i < count; i += NT) {
        const int d = move[i].y;
        if (d < 0) continue;
        int s = slot_of(d);
        // at most count < slots keys: an own or empty entry is found within `slots` probes
        for (int tries = 0; tries < slots; ++tries) {
            const int was = atomicCAS(&key[s], -1, d);
            if (was == -1 || was == d) break;
            s = (s + 1) & (slots - 1);
        }
        atomicMax(&last[s], i);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += NT) {
        const int d = move[i].y;
        if (d < 0) continue;
        int s = slot_of(d);
        for (int tries = 0; tries < slots && key[s] != d; ++tries) s = (s + 1) & (slots - 1);
        if (last[s] != i) move[i].y = -1;
    }
    cp_async_wait<0>();
    __syncthreads();
    for (int e = threadIdx.x; e < count << lsh; e += NT) {
        const int i = e >> lsh, l = e & ((1 << lsh) - 1);
        const int d = move[i].y;
        if (d < 0 || l >= lanes) continue;
        *reinterpret_cast<uint4 *>(base + (long long)d * page_bytes + 16 * l) =
            *reinterpret_cast<const uint4 *>(sm + (size_t)e * 16);
    }
}

// ---------------------------------------------------------------- compaction
// Plan, one CTA: a bitmap of the live pages, its prefix counts, the free
// indexes below n and the live ones from n on (as many of each), the renaming.
// scratch: moves, then [moves] destinations and, num_pages / 2 + 1 further on, sources.
constexpr int PLAN_NT = 1024;

__global__ void __launch_bounds__(PLAN_NT)
compact_plan_kernel(const int32_t *pages, int32_t *new_pages, long long count, int num_pages, int *scratch,
                    int *err)
{
    extern __shared__ uint32_t bits[];
    paged::let_next_start();
    const int words = (num_pages + 31) / 32;
    int *before = reinterpret_cast<int *>(bits + words);          // live pages before each word
    __shared__ int part[PLAN_NT / 32];
    const int tid = threadIdx.x;
    int *to = scratch + 64, *from = to + num_pages / 2 + 1;
    for (int w = tid; w < words; w += PLAN_NT) bits[w] = 0;
    __syncthreads();
    bool bad = false;
    for (long long i = tid; i < count; i += PLAN_NT) {
        const int p = pages[i];
        if (p >= num_pages) bad = true;
        else if (p >= 0) atomicOr(&bits[p >> 5], 1u << (p & 31));
    }
    if (bad) set_device_error(err, kErrBadSlot);
    __syncthreads();
    const int per = (words + PLAN_NT - 1) / PLAN_NT;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    int sum = 0;
    for (int w = w0; w < w1; ++w) sum += __popc(bits[w]);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if ((tid & 31) >= o) incl += x;
    }
    if ((tid & 31) == 31) part[tid >> 5] = incl;
    __syncthreads();
    int run = incl - sum, n = 0;
#pragma unroll
    for (int w = 0; w < PLAN_NT / 32; ++w) {
        if (w < tid >> 5) run += part[w];
        n += part[w];
    }
    for (int w = w0; w < w1; ++w) { before[w] = run; run += __popc(bits[w]); }
    __syncthreads();
    auto live_before = [&](int p) {
        return before[p >> 5] + __popc(bits[p >> 5] & ((1u << (p & 31)) - 1u));
    };
    // n <= num_pages; n == num_pages: nothing moves
    const int stay = n < num_pages ? live_before(n) : n;
    for (int p = tid; p < num_pages; p += PLAN_NT) {
        const bool live = (bits[p >> 5] >> (p & 31)) & 1u;
        if (p < n && !live) to[p - live_before(p)] = p;
        else if (p >= n && live) from[live_before(p) - stay] = p;
    }
    if (tid == 0) scratch[0] = n - stay;
    __syncthreads();
    for (long long i = tid; i < count; i += PLAN_NT) {
        const int p = pages[i];
        new_pages[i] = p < n || p >= num_pages ? p : to[live_before(p) - stay];
    }
}

// The moves of the plan: sources (>= n) and destinations (< n) are disjoint.
// Persistent blocks over (plane, move, 16 KB part of the page).
constexpr int PART = NT * 64;

__global__ void __launch_bounds__(NT)
compact_move_kernel(unsigned char *pool, const int *scratch, int planes, int num_pages,
                    long long page_bytes, int parts)
{
    paged::wait_for_previous();
    const int moves = scratch[0];
    const int *to = scratch + 64, *from = to + num_pages / 2 + 1;
    const long long tasks = (long long)planes * moves * parts;
    for (long long k = blockIdx.x; k < tasks; k += gridDim.x) {
        const int part = (int)(k % parts);
        const long long pm = k / parts;
        const int m = (int)(pm % moves), plane = (int)(pm / moves);
        const unsigned char *s = pool + ((long long)plane * num_pages + from[m]) * page_bytes;
        unsigned char *d = pool + ((long long)plane * num_pages + to[m]) * page_bytes;
        const long long a = (long long)part * PART + threadIdx.x * 16;
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (a + j * NT * 16 < page_bytes) x[j] = *reinterpret_cast<const uint4 *>(s + a + j * NT * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (a + j * NT * 16 < page_bytes) *reinterpret_cast<uint4 *>(d + a + j * NT * 16) = x[j];
    }
}

}  // namespace

size_t pages_compact_scratch_bytes(int num_pages) { return 256 + sizeof(int) * 2 * ((size_t)num_pages / 2 + 1); }

cudaError_t launch_pages_copy(void *pool, const int32_t *src, const int32_t *dst, int count, int planes,
                              int num_pages, long long page_bytes, int sms, int *err, cudaStream_t st)
{
    int slots = 32;
    while (slots < 2 * count) slots <<= 1;
    // The range of a CTA: a power of two, 32 KB for all moves together (six CTAs an
    // SM: 32 moves of 2 MB 16.4 us; 64 KB 19.3, 16 KB 16.9), but at least 32 bytes of
    // a page (a DRAM sector); small moves are spread over the SMs in ranges of down to
    // 256 bytes.
    int lsh = 1;
    while (lsh < 12 && ((long long)count << (lsh + 5)) <= 32 * 1024) ++lsh;
    while (lsh > 4 && ((page_bytes * planes) >> (lsh + 4)) < 4 * sms) --lsh;
    while (lsh > 0 && (16LL << (lsh - 1)) >= page_bytes) --lsh;
    const long long ranges = (page_bytes + (16 << lsh) - 1) >> (lsh + 4);
    if (ranges > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = ((size_t)count << (lsh + 4)) + 8 * (size_t)count + 8 * (size_t)slots;
    if (smem > COPY_SMEM) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(pages_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)COPY_SMEM);
    if (e != cudaSuccess) return e;
    pages_copy_kernel<<<dim3((unsigned)ranges, planes), NT, smem, st>>>((unsigned char *)pool, src, dst, count,
                                                                        num_pages, page_bytes, lsh, slots, err);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(void *pool, const int32_t *pages, int32_t *new_pages, long long count,
                                 int planes, int num_pages, long long page_bytes, int *scratch, int sms, int *err,
                                 cudaStream_t st)
{
    const size_t smem = 8 * (size_t)((num_pages + 31) / 32);
    if (smem > PLAN_SMEM) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(compact_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PLAN_SMEM);
    if (e != cudaSuccess) return e;
    compact_plan_kernel<<<1, PLAN_NT, smem, st>>>(pages, new_pages, count, num_pages, scratch, err);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long parts = (page_bytes + PART - 1) / PART;
    if (parts > 0x7fffffffLL) return cudaErrorInvalidValue;
    return paged::launch_after(compact_move_kernel, dim3(8 * sms), dim3(NT), 0, st, (unsigned char *)pool, scratch, planes,
                               num_pages, page_bytes, (int)parts);
}

}  // namespace kda
