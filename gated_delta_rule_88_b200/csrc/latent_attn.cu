// latent_attn.cu -- attention of each sequence's new tokens over the paged
// latent cache (kda_latent_attn) on tcgen05, keys on the rows of the tiles.
//
// All heads of a token attend to the same vectors, so a sequence's (token,
// head) rows are one matrix Q [L * H, dk] against one matrix C [kv, dk] whose
// first dv columns are also the values.  Per tile of 64 keys and tile of R
// rows (R = 32 or 64):
//     S^T = C_tile Q^T              (M = 64 keys, N = R rows, K = dk)
//     P^T = 2^(S^T s - m)           running maximum m per row (column of S^T)
//     O^T += C_tile[:, :dv]^T P^T   (dv / 128 products, M = 128 channels, N = R, K = 64)
// The transposed form wastes nothing when there are few rows (one token of 32
// heads is N = 32), keeps O^T in dv / 128 * R TMEM columns (a 128-row
// tile of O would need all 512), and reads C from shared memory once for both
// products: K-major as keys, MN-major as values, from the same 128-byte-swizzled
// TMA boxes.
//
// Work split: the (row tile, key tile) pairs of all sequences, counted on the
// device from kv_lens and cu_seqlens, are cut into one equal range per SM.  A row
// tile that ends inside one range is finished there; its pieces in several
// ranges go as (O, m, l) in fp32 to a workspace and latent_combine_kernel joins
// them in a fixed order, so results do not depend on timing.  Where that costs no
// more, row tiles stay whole.
//
// Roles: four softmax warps per 32 rows (a thread has one key of S^T and 16 rows),
// a TMA warp, and one warp each to issue the two products, so that S^T of the
// next tile runs while the softmax of this one does.  Every wait is bounded and
// watches an abort flag; a wait that runs out sets the device error word and the
// block drains and returns.
//
// What bounds it (B200, bf16, dv 512, dk 576).  A product of M x N x 16 costs the
// tensor pipe (32 M + 32 N) / 128 cycles, the time to read its operands from shared
// memory, and its issue 36; a tile of 64 keys is 73.7 KB.
//   R = 32 (one token of up to 32 heads): HBM.  64 sequences up to 8192 keys x 32
//     heads: 73 us against 47.6 at the measured copy rate; a block's steady state is
//     3.3 to 3.4 thousand cycles a tile (5.7 TB/s over all SMs), before it 3 us until
//     the first load and 2 us in which the first tiles arrive together, after it 2 us
//     for the last row tile and 5 for the second kernel.  2.5 tiles are in flight; 16 KB
//     more did not help, nor did prefetching into L2 (it takes the loads' place in the
//     queue).
//   R = 64: the round of a stage through the block.  Q takes 74 KB, two tiles the
//     rest: the second product ends, its stages are loaded anew (2.6 thousand cycles,
//     1.6 of them the TMA unit's 62 + 1.84 per 128 bytes for each box), S^T, softmax
//     (1.0), again the second product: 3.5 thousand a tile, where the products alone
//     take 1.9.  4 sequences of up to 500 tokens behind up to 8192 keys: 757 us in
//     pages of 64 (685 TFLOP/s, 41% of the measured dense rate), 861 in pages of 16, whose
//     boxes are a quarter as long.
//   128-key tiles (one in flight) took 95 us and 1.19 ms; one warp for both products
//     115 us and 1.45 ms.
#include "kernels.h"
#include "paged.cuh"
#include "prep_common.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int KT = 64;                        // keys of a tile
// The reference m of a row's exponentials is the maximum of its first tile, and
// is raised only when a later logit lies above it by more than TH powers of two: P up to
// 2^TH keeps its relative precision in bf16, and O up to 2^TH kv_len max |c| in fp32 as long
// as that is finite, hence the header's bound on kv_len times a value, 2^110.  (60
// overflowed from values of 2^67 on.  The times are the same for logits of a standard
// deviation of up to 7.5 powers of two; at 25 and 100 the 4 chunks take 872 and 884 us, with
// 60 861 and 876, and 64 sequences 77.8 and 79.8 with either.)
constexpr float TH = 16.f;
// What a row tile costs besides its key tiles, in key tiles: 32 sequences x 4 tokens
// up to 8000 keys take 101 us with 0, 93.7 with 1, 88 with 2, 84.6 with 4, 87.8 with 8;
// 64 sequences x 1 token 77.7, 76.6, 73, 72 and 75.
constexpr int OV = 4;
// What splitting costs a block, in key tiles (pieces written and joined): at 64
// sequences x 4 tokens of 512 keys (8 tiles) 41.2 us split and 30.9 whole, at one
// sequence of 300 keys 13.9 split and 19.3 whole.  Over 108 shapes (1 to 200 sequences
// of 128 to 4096 keys; 32 heads, 128, and 32 with 4 tokens) 8 comes within 3% and
// 0.2 us of the better of both in 105, 6 in 107, 10 in 99; 6 and 8 have the same
// geometric mean, 10 lies 1.4% above.
constexpr int SPLIT_COST = 8;
// Up to this many key tiles a sequence nothing is split, and the second kernel is not
// even launched: one sequence of 128 keys 10.8 us instead of 11.8 (of 300 keys 16.8
// instead of 13.5).
constexpr int WHOLE_TILES = 4;

__host__ __device__ constexpr uint32_t idesc(int M, int N, bool mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((mn ? 1u : 0u) << 15) | ((mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

constexpr int SMEM = 227 * 1024;

template <int R, int DV, bool PE>
struct Lay {
    static constexpr int MT = DV / 128;                       // stages (128 channels) of a key tile
    static constexpr int NQ = DV / 64 + (PE ? 1 : 0);         // 64-channel pieces of Q
    static constexpr int CG = R / 32;                         // groups of 32 rows, four softmax warps each
    static constexpr int SW = 4 * CG;
    static constexpr int NT = 32 * (SW + 3);
    static constexpr uint32_t HALF = KT * 128;                // 64 keys x 64 channels
    static constexpr uint32_t STAGE = 2 * HALF;
    static constexpr uint32_t QP = R * 128;                   // one piece of Q
    static constexpr uint32_t X_OFF = NQ * QP;                // the positional piece of the keys, two buffers
    static constexpr uint32_t P_OFF = X_OFF + (PE ? 2 * HALF : 0);
    static constexpr uint32_t ST_OFF = P_OFF + KT * R * 2;
    static constexpr uint32_t SMALL = 3 * 1024;               // barriers and small tables
    static constexpr int NS = (SMEM - (int)SMALL - (int)ST_OFF) / (int)STAGE;
    static constexpr uint32_t MISC = ST_OFF + NS * STAGE;
    // TMEM: two S^T tiles (lanes +0 and +16 of the same columns), then O^T
    static constexpr uint32_t O_COL = R;
    static constexpr uint32_t USED = O_COL + MT * R;
    static constexpr uint32_t COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
    // P^T: MN-major, rows of R values swizzled to their width
    static constexpr uint32_t BW = R * 2;
    static constexpr uint32_t B_SBO = 8 * BW;
    static constexpr uint32_t B_LAYOUT = R == 64 ? 2 : 4;
    static constexpr int B_SWZ = R == 64 ? 7 : 3;
    static __device__ __forceinline__ uint32_t p_off(int k, int chunk) {
        return (k >> 3) * B_SBO + (k & 7) * BW + ((chunk ^ ((((k & 7) * BW) >> 7) & B_SWZ)) << 4);
    }
};

// The small tables behind the stages.
struct Small {
    // full[i] is barrier i, ...; s_free and p_full take an arrival of every softmax warp, the others one
    uint64_t full[12], empty[12], x_full[2], x_empty[2], q_full, q_empty, s_full[2], o_full, drain[2], s_free[2], p_full;
    static constexpr int ONE = 35, ALL = 38;
    long long scan[12];
    int scan_rt[12], scan_max[12];
    int start[6];                // sequence, its first token, new tokens, keys; row tile; unit in it
    uint32_t tmem;
    int abort_flag;
    float red[8][32];            // a warp's result per row of its group
    float mine[8][32];           // a warp's own copy of a value per row of its group
};
static_assert(sizeof(Small) <= 3 * 1024, "small tables");

struct Args {
    const int32_t *table, *lens, *cu;
    __nv_bfloat16 *out;
    float *lse;
    float *ws_o, *ws_ml;         // [2 * blocks][R][DV], [2 * blocks][R][2]
    int4 *meta;                  // [2 * blocks]: a split row tile: first row, rows, first block, pieces
    int T, H, N, per, num_pages, page_size, max_pages;
    float sl2;                   // scale * log2 e
    bool full, split;            // split: there is a workspace, row tiles may be split
    int *err;
};

// ---------------------------------------------------------------- schedule
// A sequence's rows and keys.  A row tile costs its key tiles (at least one:
// rows that see nothing are written, too) and OV units more, which come first.
template <int R>
struct Seq {
    int first, L, kv, H;         // first token, new tokens, keys (0 tokens if the length is bad)
    bool full, bad;
    __device__ __forceinline__ void set(const Args &a, int first_, int L_, int kv_) {
        H = a.H; full = a.full || L_ == 1; first = first_; L = L_; kv = kv_;
    }
    __device__ __forceinline__ void load(const Args &a, int n) {
        const int b = paged::token_offset(a.cu, n, a.per, a.T), e = paged::token_offset(a.cu, n + 1, a.per, a.T);
        const int k = a.lens[n];
        bad = k < 0 || (long long)k > (long long)a.max_pages * a.page_size;
        set(a, b, bad ? 0 : max(0, e - b), bad ? 0 : k);
    }
    __device__ __forceinline__ int rows() const { return L * H; }        // T * H < 2^31
    __device__ __forceinline__ int row_tiles() const { return (rows() - 1 + R) / R; }
    // keys that row r sees
    __device__ __forceinline__ int sees(int r) const {
        return full ? kv : min(kv, max(0, kv - L + r / H + 1));
    }
    __device__ __forceinline__ int keys_of(int i) const { return sees(min(rows(), (i + 1) * R) - 1); }
    __device__ __forceinline__ int tiles_of(int i) const { return max(1, (keys_of(i) + KT - 1) / KT); }
    // row tiles i < upto(k) have at most k key tiles
    __device__ __forceinline__ int upto(int k) const {
        if (full) return KT * (long long)k >= kv ? row_tiles() : 0;
        const long long tokens = (long long)KT * k - kv + L;             // tokens that see <= KT k keys
        if (tokens >= L) return row_tiles();
        return tokens <= 0 ? 0 : (int)((unsigned long long)(tokens * H) / R);
    }
    __device__ __forceinline__ long long units() const {
        const int nt = row_tiles();
        if (nt <= 0) return 0;
        if (nt == 1) return tiles_of(0) + OV;
        long long u = (long long)nt * OV;
        int k = tiles_of(0), done = 0;
        while (done < nt) {
            const int c = min(nt, max(done, upto(k)));
            u += (long long)k * (c - done);
            done = c;
            ++k;
        }
        return u;
    }
    // row tile i of unit u, and the unit's place in it
    __device__ __forceinline__ void find(long long u, int &i, int &at) const {
        const int nt = row_tiles();
        if (nt == 1) { i = 0; at = (int)u; return; }
        int k = tiles_of(0), done = 0;
        while (done < nt) {
            const int c = min(nt, max(done, upto(k)));
            const long long here = (long long)(k + OV) * (c - done);
            if (u < here) {
                // (a block's share of a sequence's units fits 31 bits wherever there are that many blocks)
                const long long q = here <= 0x7fffffff ? (unsigned)u / (unsigned)(k + OV) : u / (k + OV);
                i = done + (int)q;
                at = (int)(u - q * (k + OV));
                return;
            }
            u -= here;
            done = c;
            ++k;
        }
        i = nt - 1;
        at = 0;
    }
};

// The segments of a block's range: a row tile of a sequence and key tiles
// [j0, j1) of its `tiles`.  Every role walks them by itself.
template <int R>
struct Walk {
    Seq<R> s;
    int n, i, j0, j1, tiles, at;                // at: the unit of the row tile that the range goes on with
    long long left;                             // units of the range from there on, or row tiles if whole
    bool whole;                                 // row tiles are not split
    __device__ __forceinline__ void start(const Args &a, const Small &sm, long long left_, bool whole_) {
        left = left_;
        whole = whole_;
        j0 = j1 = 0;
        if (left <= 0) return;
        n = sm.start[0]; i = sm.start[4]; at = sm.start[5];
        s.set(a, sm.start[1], sm.start[2], sm.start[3]);
        settle();
    }
    __device__ __forceinline__ void settle() {
        tiles = s.tiles_of(i);
        if (whole) { j0 = 0; j1 = tiles; return; }
        const int take = (int)min((long long)(tiles + OV - at), left);
        j0 = max(0, at - OV);
        j1 = max(0, at + take - OV);
        if (j1 == j0) left = 0;                 // the range ends before the first key tile
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const Args &a) {
        left -= whole ? 1 : min((long long)(tiles + OV - at), left);
        if (left <= 0) return;
        at = 0;
        ++i;
        while (i >= s.row_tiles()) {
            if (++n >= a.N) { left = 0; return; }
            s.load(a, n);
            i = 0;
        }
        settle();
    }
};

// Polls of a wait before it gives up: half a second or more, none in the self-test.
// (A constant: as an argument of the kernel it cost 3 us of 76 at 64 sequences to
// 8192 keys and 1.2 of 16.4 at one sequence of 300.)
template <bool GIVE_UP> constexpr uint32_t LIMIT = GIVE_UP ? 0 : 1u << 24;

template <uint32_t POLLS>
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_test_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < POLLS; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (i > 64) __nanosleep(32);
    }
    return false;
}

// The same for a warp with a barrier per lane (null: none), all of them polled
// at once: a poll costs a few hundred cycles, however many barriers it asks.
__device__ __forceinline__ bool polled(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, bar == nullptr || mbar_test_wait(bar, parity));
}
template <uint32_t POLLS>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (polled(bar, parity)) return true;
    return __all_sync(0xffffffffu, bar == nullptr || wait_on<POLLS>(bar, parity, abort_flag));
}

// One lane of the warp, chosen by the hardware.  The products are issued by
// whole warps under this, with operands that come from lane 0 (uniform_of): the
// compiler then keeps descriptors in uniform registers, as the instruction wants
// them: 36 cycles an issue, 48 from a loop that lane 0 runs alone.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(p));
    return p != 0;
}
template <typename T> __device__ __forceinline__ T uniform_of(T x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
        "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// A 64-row accumulator (16 lanes of each sub-partition): thread l of the warp gets
// row l % 16 of the sub-partition, 16 columns from taddr (l < 16) or the next 16.
__device__ __forceinline__ void tmem_ld_half(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], 16;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Combines v[c] over the 16 lanes of the half warp, per column c, by halving (15
// shuffles instead of 4 * 16): lane l gets the result of column l of the two
// halves' 32.
template <bool MAX>
__device__ __forceinline__ float across_lanes(float (&v)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
            const float other = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = MAX ? fmaxf(keep, other) : keep + other;
        }
    }
    return v[0];
}

template <int R, int DV, bool PE, bool GIVE_UP>
__global__ void __launch_bounds__(Lay<R, DV, PE>::NT, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c, const Args a)
{
    using L = Lay<R, DV, PE>;
    constexpr uint32_t POLLS = LIMIT<GIVE_UP>;
    extern __shared__ __align__(1024) unsigned char sm[];
    Small &z = *reinterpret_cast<Small *>(sm + L::MISC);
    volatile int *abort_flag = &z.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023) {                  // the swizzled tiles need it; the same for every block
        if (tid == 0) set_device_error(a.err, kErrWaitTimeout);
        if (tid < 2 && a.split) a.meta[2 * blockIdx.x + tid].w = 0;
        return;
    }

    // ---- this block's range of the (row tile, key tile) units
    if (warp == 1) {
        for (int i = lane; i < Small::ALL; i += 32) mbar_init(&z.full[0] + i, i < Small::ONE ? 1 : L::SW);
        if (lane == 0) z.abort_flag = 0;
        fence_mbar_init();
    } else if (warp == 2) {
        tmem_alloc(&z.tmem, L::COLS);
        tmem_relinquish();
    }
    const int per = a.N <= L::NT ? 1 : (a.N + L::NT - 1) / L::NT;
    const int n0 = min(a.N, tid * per), n1 = min(a.N, n0 + per);
    long long mysum = 0;                        // units
    int mytiles = 0, mymax = 0;                 // row tiles, and the most key tiles of one
    Seq<R> s0;                                  // the thread's first sequence
    for (int n = n0; n < n1; ++n) {
        Seq<R> s;
        s.load(a, n);
        if (s.bad && blockIdx.x == 0) set_device_error(a.err, paged::kErrBadPage);
        if (n == n0) s0 = s;
        mysum += s.units();
        const int nt = s.row_tiles();
        mytiles += nt;
        if (nt > 0) mymax = max(mymax, s.tiles_of(nt - 1));
    }
    long long incl = mysum;
    int incl_rt = mytiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        const int y = __shfl_up_sync(0xffffffffu, incl_rt, o);
        if (lane >= o) { incl += x; incl_rt += y; }
    }
    mymax = __reduce_max_sync(0xffffffffu, mymax);
    if (lane == 31) { z.scan[warp] = incl; z.scan_rt[warp] = incl_rt; z.scan_max[warp] = mymax; }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = z.tmem;
    long long before = incl - mysum, total = 0;
    int before_rt = incl_rt - mytiles, total_rt = 0;
#pragma unroll
    for (int w = 0; w < L::NT / 32; ++w) {
        const long long x = z.scan[w];
        const int y = z.scan_rt[w];
        if (w < warp) { before += x; before_rt += y; }
        total += x;
        total_rt += y;
        mymax = max(mymax, z.scan_max[w]);
    }
    // Row tiles stay whole where that costs no more: the fullest block's key tiles against an
    // equal share of all and SPLIT_COST for writing the pieces and joining them.
    const long long rounds = (total_rt + (int)gridDim.x - 1) / (int)gridDim.x;
    const bool whole = !a.split || (rounds * (mymax + OV) - SPLIT_COST) * gridDim.x <= total;
    if (whole) { total = total_rt; before = before_rt; mysum = mytiles; }
    // as many ranges as blocks, but none empty: the pieces of a row tile lie in consecutive blocks
    const int G = total < (long long)gridDim.x ? max(1, (int)total) : (int)gridDim.x;
    const int b = blockIdx.x;
    long long u0 = 0, u1 = 0;                   // total * b / G, total * (b + 1) / G
    if (b < G && total > 0) {
        if (total <= 0x7fffffff) {
            // r b and r (b + 1) are below 2^24: their quotients by rounding down (e + 1/2) / G
            const float inv = 1.f / (float)G;
            unsigned q = __umulhi((unsigned)total, 0xffffffffu / (unsigned)gridDim.x);
            if (G != (int)gridDim.x) q = 1;                              // total == G
            unsigned r = (unsigned)total - q * G;
            while (r >= (unsigned)G) { r -= G; ++q; }
            u0 = (long long)q * b + (unsigned)(((float)(r * b) + 0.5f) * inv);
            u1 = (long long)q * (b + 1) + (unsigned)(((float)(r * (b + 1)) + 0.5f) * inv);
        } else {
            u0 = total * b / G;
            u1 = total * (b + 1) / G;
        }
    }
    if (u0 < u1 && u0 >= before && u0 < before + mysum) {
        long long u = u0 - before;
        Seq<R> s = s0;
        int n = n0;
        for (long long here; n + 1 < n1 && u >= (here = whole ? s.row_tiles() : s.units()); s.load(a, ++n)) u -= here;
        int i = (int)u, at = 0;
        if (!whole) s.find(u, i, at);
        z.start[0] = n; z.start[1] = s.first; z.start[2] = s.L; z.start[3] = s.kv; z.start[4] = i; z.start[5] = at;
    }
    __syncthreads();
    Walk<R> w;
    w.start(a, z, u1 - u0, whole);

    if (warp == L::SW) {
        // ---------------- TMA: Q of each segment, then its key tiles ----------------
        int st = 0, st_use = 0, tiles = 0, segs = 0;          // stage, its uses; key tiles and segments so far
        bool ok = true;
        const int rows_box = min(a.page_size, KT);            // rows of a box
        const int lrb = 31 - __clz(rows_box), lps = 31 - __clz(a.page_size);
        auto boxes_of = [&](int j, int end) { return (max(0, min(KT, end - j * KT)) + rows_box - 1) >> lrb; };
        // Each lane has one box of the tile: stage m, half of its channels, rows of box `box` (and
        // lanes 0 .. 3 one of the positional piece), and fetches it as soon as its stage is free.
        const int m = lane >> 3, box = (lane >> 1) & 3, half = lane & 1;
        auto page_of = [&](int j, int boxes, int bx) {
            return bx < boxes ? a.table[(long long)w.n * a.max_pages + ((j * KT + bx * rows_box) >> lps)] : 0;
        };
        for (; w.more() && ok; w.next(a)) {
            const int end = w.s.keys_of(w.i);
            int boxes = boxes_of(w.j0, end);
            int page = page_of(w.j0, boxes, box), page_x = PE && lane < 4 ? page_of(w.j0, boxes, lane) : 0;
            ok = segs == 0 || wait_on<POLLS>(&z.q_empty, (segs - 1) & 1, abort_flag);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (lane == 0) {
                const int row = w.s.first * a.H + w.i * R;
                mbar_arrive_expect_tx(&z.q_full, L::NQ * L::QP);
                for (int p = 0; p < L::NQ; ++p) tma_2d(sm + p * L::QP, &tm_q, 64 * p, row, &z.q_full);
            }
            ++segs;
            for (int j = w.j0; j < w.j1; ++j) {
                const uint32_t bytes = (uint32_t)boxes * rows_box * 128;
                int s = st + m, use = st_use;
                if (s >= L::NS) { s -= L::NS; ++use; }
                bool todo = m < L::MT && (box < boxes || (lane & 7) == 0);
                if (PE) {
                    // (a positional piece is free long before the stages are)
                    uint64_t *eb = tiles < 2 ? nullptr : &z.x_empty[tiles & 1], *fb = &z.x_full[tiles & 1];
                    if (!(ok = warp_wait<POLLS>(eb, ((tiles >> 1) - 1) & 1, abort_flag))) break;
                    if (lane == 0) mbar_arrive_expect_tx(fb, bytes);
                    if (lane < boxes && lane < 4)
                        prep::tma_load_3d(sm + L::X_OFF + (tiles & 1) * L::HALF + lane * rows_box * 128, &tm_c, DV,
                                          (j * KT + lane * rows_box) & (a.page_size - 1), page_x, fb);
                    __syncwarp();
                }
                uint64_t *fb = &z.full[s], *eb = &z.empty[s];
                const uint32_t parity = (use - 1) & 1;
                unsigned char *dst = sm + L::ST_OFF + s * L::STAGE + half * L::HALF + box * rows_box * 128;
                const int x = 128 * m + 64 * half, y = (j * KT + box * rows_box) & (a.page_size - 1);
                for (uint32_t tries = 1; __any_sync(0xffffffffu, todo); ++tries) {
                    if (todo && (use == 0 || mbar_test_wait(eb, parity))) {
                        if ((lane & 7) == 0) mbar_arrive_expect_tx(fb, 2 * bytes);
                        if (box < boxes) prep::tma_load_3d(dst, &tm_c, x, y, page, fb);
                        todo = false;
                    }
                    if ((tries & 63) == 0) {
                        ok = tries < POLLS && !*abort_flag;
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        __nanosleep(32);
                    }
                }
                if (!ok) break;
                st += L::MT;
                if (st >= L::NS) { st -= L::NS; ++st_use; }
                ++tiles;
                if (j + 1 < w.j1) {
                    boxes = boxes_of(j + 1, end);
                    page = page_of(j + 1, boxes, box);
                    if (PE && lane < 4) page_x = page_of(j + 1, boxes, lane);
                }
            }
        }
        if (!ok && lane == 0) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; }
    } else if (warp == L::SW + 1) {
        // ---------------- S^T = C Q^T ----------------
        constexpr uint32_t ID = idesc(64, R, false);
        const uint32_t base = smem_u32(sm);
        const DescParts q_d = smem_desc_parts(base, 16, 1024, 2);
        const DescParts k_d = smem_desc_parts(base + L::ST_OFF, 16, 1024, 2);            // keys, K-major
        const DescParts x_d = smem_desc_parts(base + L::X_OFF, 16, 1024, 2);
        int st = 0, st_use = 0, tiles = 0, segs = 0;
        bool ok = true;
        for (; w.more() && ok; w.next(a)) {
            for (int j = w.j0; j < w.j1 && ok; ++j) {
                const int b2 = uniform_of(tiles & 1);
                const uint32_t d = uniform_of(tmem) + ((uint32_t)(16 * b2) << 16);
                // everything that the tile waits for, asked at once: its stages, its
                // positional piece, a free S^T, Q
                uint64_t *bar = nullptr;
                uint32_t parity = 0;
                if (lane < L::MT) {
                    const int s = st + lane;
                    bar = &z.full[s < L::NS ? s : s - L::NS];
                    parity = (st_use + (s < L::NS ? 0 : 1)) & 1;
                } else if (PE && lane == L::MT) {
                    bar = &z.x_full[b2];
                    parity = (tiles >> 1) & 1;
                } else if (lane == L::MT + 1 && tiles >= 2) {
                    bar = &z.s_free[b2];
                    parity = ((tiles >> 1) - 1) & 1;
                } else if (lane == L::MT + 2 && j == w.j0) {
                    bar = &z.q_full;
                    parity = segs & 1;
                }
                const bool all = polled(bar, parity);
                // else one by one: S^T starts with what has landed
                if (!all) ok = warp_wait<POLLS>(lane < L::MT ? nullptr : bar, parity, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (PE) {
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16_p(d, x_d.lo + ((b2 * L::HALF + kk * 32) >> 4), x_d.hi,
                                        q_d.lo + (((L::NQ - 1) * L::QP + kk * 32) >> 4), q_d.hi, ID, kk > 0);
                        umma_commit(&z.x_empty[b2]);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int m = 0; m < L::MT; ++m) {
                    const uint32_t k_lo = k_d.lo + (uniform_of(st) * L::STAGE >> 4), q_lo = q_d.lo + (2 * m * L::QP >> 4);
                    if (ok && !all) ok = __all_sync(0xffffffffu, wait_on<POLLS>(&z.full[st], st_use & 1, abort_flag));
                    if (ok && elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16_p(d, k_lo + (((kk >> 2) * L::HALF + (kk & 3) * 32) >> 4), k_d.hi,
                                        q_lo + (((kk >> 2) * L::QP + (kk & 3) * 32) >> 4), q_d.hi, ID, PE || m > 0 || kk > 0);
                    }
                    __syncwarp();
                    if (++st == L::NS) { st = 0; ++st_use; }
                }
                if (!ok) break;
                if (elect_one()) {
                    umma_commit(&z.s_full[b2]);
                    if (j + 1 == w.j1) umma_commit(&z.q_empty);
                }
                __syncwarp();
                ++tiles;
            }
            ++segs;
        }
        // never free TMEM or shared memory under a running MMA (the elected lane is the same each time)
        if (elect_one()) {
            if (!ok) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; }
            umma_commit(&z.drain[0]);
            mbar_wait(&z.drain[0], 0, 1u << 20);
        }
    } else if (warp == L::SW + 2) {
        // ---------------- O^T += C^T P^T ----------------
        constexpr uint32_t ID = idesc(128, R, true);
        const uint32_t base = smem_u32(sm);
        const DescParts v_d = smem_desc_parts(base + L::ST_OFF, L::HALF, 1024, 2);       // values, MN-major
        const DescParts p_d = smem_desc_parts(base + L::P_OFF, L::B_SBO, L::B_SBO, L::B_LAYOUT);
        constexpr uint32_t PK = (2 * L::B_SBO) >> 4;
        int st = 0, tiles = 0;
        bool ok = true;
        for (; w.more() && ok; w.next(a))
            for (int j = w.j0; j < w.j1; ++j) {
                if (!(ok = __all_sync(0xffffffffu, wait_on<POLLS>(&z.p_full, tiles & 1, abort_flag)))) break;
                tc_fence_after();
                const uint32_t o = uniform_of(tmem) + L::O_COL, more = uniform_of((int)(j > w.j0));
#pragma unroll
                for (int m = 0; m < L::MT; ++m) {
                    const int s = uniform_of(st);
                    const uint32_t v_lo = v_d.lo + (s * L::STAGE >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            umma_bf16_p(o + m * R, v_lo + ((kk * 2048) >> 4), v_d.hi, p_d.lo + kk * PK, p_d.hi, ID, kk > 0 ? 1 : more);
                        umma_commit(&z.empty[s]);
                        if (m + 1 == L::MT) umma_commit(&z.o_full);
                    }
                    __syncwarp();
                    if (++st == L::NS) st = 0;
                }
                ++tiles;
            }
        if (elect_one()) {
            if (!ok) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; }
            umma_commit(&z.drain[1]);
            mbar_wait(&z.drain[1], 0, 1u << 20);
        }
    } else {
        // ---------------- softmax and output: key r of the tile, rows 16 half .. + 15 of the
        // warp's group of 32; the statistics of the group's row `lane` in each of its warps ----------------
        const int cg = warp >> 2, qd = warp & 3;
        const int t = 32 * qd + lane, half = lane >> 4, r = 16 * qd + (lane & 15);
        const uint32_t lanes = tmem + ((uint32_t)(32 * qd) << 16) + 32 * cg;
        float *mine = z.mine[warp];
        const float *mine_c = mine + 16 * half;
        float (*red)[32] = z.red + 4 * cg;
        int tiles = 0;
        bool ok = true;
        int4 meta[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
        long long at0 = u0;                                              // units of the range before the segment
        for (; w.more() && ok;) {
            const int rows = min(R, w.s.rows() - w.i * R) - 32 * cg;     // of this group
            const int end = w.s.keys_of(w.i);
            const int sees = lane < rows ? w.s.sees(w.i * R + 32 * cg + lane) : 0;
            const int least = __reduce_min_sync(0xffffffffu, lane < rows ? sees : 0x7fffffff);
            // the segment's pages (one of a split tile's pieces with a bad page spoils all of it)
            bool bad = false;
            // (counted in pages: the keys of the next pages may lie past 2^31)
            const int lps = 31 - __clz(a.page_size), stop = (min(w.j1 * KT, end) + a.page_size - 1) >> lps;
            for (int p = (w.j0 * KT >> lps) + t; p < stop; p += 128) {
                const int pg = a.table[(long long)w.n * a.max_pages + p];
                bad |= pg < 0 || pg >= a.num_pages;
            }
            float m_run = -INFINITY, l[16];
            constexpr float NONE = -1e30f;           // stands for no reference: whatever a row sees lies above it by more than TH
            __syncwarp();
            mine[lane] = NONE;
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 16; ++c) l[c] = 0.f;
            // Before the block's first tile the loop runs once on whatever TMEM holds, while Q and the
            // tile are on their way: the pass brings the instructions in and leaves nothing else
            // behind (the first softmax takes 1.4 instead of 3.4 thousand cycles).
            for (int j = w.j0 - (tiles == 0 ? 1 : 0); j < w.j1; ++j) {
                const bool dry = j < w.j0;
                // S^T of this tile is there; O^T, P^T and the maxima of the previous one are done with
                uint64_t *bar = dry ? nullptr : lane == 0 ? &z.s_full[tiles & 1] : lane == 1 && tiles > 0 ? &z.o_full : nullptr;
                ok = ok && warp_wait<POLLS>(bar, lane == 0 ? (tiles >> 1) & 1 : (tiles - 1) & 1, abort_flag);
                tc_fence_after();
                float x[16], y[16];
                tmem_ld_half(lanes + ((uint32_t)(16 * (tiles & 1)) << 16), x);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !dry) mbar_arrive(&z.s_free[tiles & 1]);
                const int key = j * KT + r;
                if (j * KT + KT > least) {
                    // some row does not see the whole tile
                    __syncwarp();
                    mine[lane] = __int_as_float(sees);
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = key < __float_as_int(mine_c[c]) ? x[c] * a.sl2 : -INFINITY;
                    __syncwarp();
                    mine[lane] = m_run == -INFINITY ? NONE : m_run;
                    __syncwarp();
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] *= a.sl2;
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    y[c] = x[c] - mine_c[c];
                    top = fmaxf(top, y[c]);
                }
                const bool high = named_bar_or(1 + cg, 128, !ok || top > TH);
                if (high) {
                    // a row without a reference yet, or one that has outgrown it: the tile's maxima
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = x[c];
                    red[qd][lane] = across_lanes<true>(y, lane);
                    if (named_bar_or(1 + cg, 128, !ok)) { ok = false; break; }
                    const float mt = fmaxf(fmaxf(red[0][lane], red[1][lane]), fmaxf(red[2][lane], red[3][lane]));
                    const bool raise = mt > m_run + TH || (m_run == -INFINITY && mt > -INFINITY);
                    const float f = raise ? exp2f(m_run - mt) : 1.f;
                    if (raise) m_run = mt;
                    if (j > w.j0) {
                        mine[lane] = f;
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 16; ++c) l[c] *= mine_c[c];
                        for (int m = 0; m < L::MT; ++m) {
                            float o[32];
                            tmem_ld32(lanes + L::O_COL + m * R, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] *= mine[c];
                            tmem_st32(lanes + L::O_COL + m * R, o);
                        }
                        tmem_wait_st();
                        __syncwarp();
                    }
                    mine[lane] = m_run == -INFINITY ? NONE : m_run;
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 16; ++c) y[c] = x[c] - mine_c[c];
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = prep::ex2_approx(y[c]);
                // P in bf16, the type of C beside it in the product; the sums l are of the unrounded ones.  Against 64
                // bits the output is off by 2.1e-3 (norm), where a form in 32 bits rounded once has 1.7e-3.
                unsigned char *P = sm + L::P_OFF;
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    *reinterpret_cast<uint4 *>(P + L::p_off(r, 4 * cg + 2 * half + g)) =
                        make_uint4(pack_bf16(x[8 * g], x[8 * g + 1]), pack_bf16(x[8 * g + 2], x[8 * g + 3]),
                                   pack_bf16(x[8 * g + 4], x[8 * g + 5]), pack_bf16(x[8 * g + 6], x[8 * g + 7]));
#pragma unroll
                for (int c = 0; c < 16; ++c) l[c] += x[c];
                if (key >= end && !dry) {
                    // rows that hold no key of this row tile may hold anything: 0 * NaN is not 0
                    const int s0 = (int)((long long)tiles * L::MT % L::NS);
                    for (int m = cg; m < L::MT; m += L::CG) {
                        const int s = s0 + m < L::NS ? s0 + m : s0 + m - L::NS;
                        unsigned char *v = sm + L::ST_OFF + s * L::STAGE + half * L::HALF + r * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(v + 16 * e) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (dry) {
                    m_run = -INFINITY;
                    mine[lane] = NONE;
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 16; ++c) l[c] = 0.f;
                    continue;
                }
                if (lane == 0) mbar_arrive(&z.p_full);
                ++tiles;
            }
            if (!ok) break;
            ok = wait_on<POLLS>(&z.o_full, (tiles - 1) & 1, abort_flag);
            tc_fence_after();
            red[qd][lane] = across_lanes<false>(l, lane);
            if (named_bar_or(1 + cg, 128, !ok)) { ok = false; break; }
            const float sum = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
            bad = named_bar_or(1 + cg, 128, bad);
            if (bad && tid == 0) set_device_error(a.err, paged::kErrBadPage);
            const long long row0 = (long long)w.s.first * a.H + (long long)w.i * R;
            if (w.j0 == 0 && w.j1 == w.tiles) {
                // the whole row tile was here
                // (the sum of a row that sees a key is at least 1, or NaN, which is to show; 0: none)
                mine[lane] = sum == 0.f ? 0.f : 1.f / sum;
                if (a.lse && qd == 0 && lane < rows && !bad)
                    a.lse[row0 + 32 * cg + lane] = sum == 0.f ? -INFINITY : (m_run + log2f(sum)) * 0.693147180559945f;
                __syncwarp();
                // (the test inside, at each store, spills what the loop over key tiles needs: 4 chunks
                // of up to 500 tokens in pages of 64 took 801 us instead of 762)
                if (!bad)
                    for (int m = 0; m < L::MT; ++m) {
                        float o[32];
                        tmem_ld32(lanes + L::O_COL + m * R, o);
                        tmem_wait_ld();
                        __nv_bfloat16 *dst = a.out + (row0 + 32 * cg) * DV + 128 * m + t;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c < rows) dst[(size_t)c * DV] = __float2bfloat16_rn(o[c] * mine[c]);
                    }
            } else {
                // a piece: slot 0 if it continues the row tile, slot 1 if it begins it
                const size_t at = (size_t)(2 * b + (w.j0 == 0 ? 1 : 0)) * R + 32 * cg;
                if (qd == 0) *reinterpret_cast<float2 *>(a.ws_ml + (at + lane) * 2) = make_float2(m_run, bad ? -1.f : sum);
                for (int m = 0; m < L::MT; ++m) {
                    float o[32];
                    tmem_ld32(lanes + L::O_COL + m * R, o);
                    tmem_wait_ld();
                    float *dst = a.ws_o + at * DV + 128 * m + t;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c < rows) dst[(size_t)c * DV] = o[c];
                }
                if (tid == 0) {
                    // the blocks of its first and last key tile; unit u is in block (u G + G - 1) / total
                    const long long first = at0 - w.at + OV, last = first + w.tiles - 1;
                    auto block_of = [&](long long u) { return (int)((u * G + G - 1) / total); };
                    const int b0 = w.j0 == 0 ? b : block_of(first);
                    meta[w.j0 == 0 ? 1 : 0] = make_int4((int)row0, min(R, w.s.rows() - w.i * R), b0, block_of(last) - b0 + 1);
                }
            }
            tc_fence_before();
            __syncwarp();
            at0 += w.tiles + OV - w.at;                                  // (of no use after the last segment)
            w.next(a);
        }
        if (!ok) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; meta[0].w = meta[1].w = 0; }
        // (earlier, the second kernel's blocks would wait beside the running ones: 76 us instead of 73)
        paged::let_next_start();
        if (tid == 0 && a.split) { a.meta[2 * b] = meta[0]; a.meta[2 * b + 1] = meta[1]; }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, L::COLS);
    if (*abort_flag && warp == L::SW && lane == 0) {
        // Some role gave up: never leave with copies in flight into this block's shared memory, whether the
        // TMA warp gave up too or had issued its last tile before.  A barrier without copies, or of a tile
        // that was not issued as a whole, takes all the polls (20 ms).
        auto landed = [](uint64_t *bar) {
            for (int k = 0; k < 2; ++k)
                for (uint32_t i = 0; i < (1u << 18) && !mbar_test_wait(bar, k); ++i) __nanosleep(32);
        };
        for (int s = 0; s < L::NS; ++s) landed(&z.full[s]);
        for (int x = 0; PE && x < 2; ++x) landed(&z.x_full[x]);
        landed(&z.q_full);
    }
}

// Joins the pieces of the row tiles that were split: with M = max m_k,
//     out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,   lse from M and the sum.
// The rows of a split tile are shared out over the blocks whose ranges it lies
// in (block x has up to two such tiles: one that it continues, one that it
// begins).  With few pieces a warp takes a row; with many the block's warps share
// a row's pieces and add their parts up in order, and gridDim.y its channels.
constexpr int CW = 8;                          // warps
constexpr int CY = 4;                          // gridDim.y
constexpr int FEW = 8;                         // pieces that one warp takes

// acc += f y
__device__ __forceinline__ void add_scaled(float4 &acc, float f, const float4 &y) {
    acc.x = fmaf(f, y.x, acc.x); acc.y = fmaf(f, y.y, acc.y);
    acc.z = fmaf(f, y.z, acc.z); acc.w = fmaf(f, y.w, acc.w);
}

template <int R, int DV>
__global__ void __launch_bounds__(32 * CW)
latent_combine_kernel(const float *ws_o, const float *ws_ml, const int4 *meta, __nv_bfloat16 *out, float *lse)
{
    constexpr int V = DV / 128;                // float4's of a row for each lane
    __shared__ float4 part[CW][32];
    __shared__ float part_l[CW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    paged::wait_for_previous();
    for (int e = 0; e < 2; ++e) {
        const int4 mt = meta[2 * blockIdx.x + e];
        if (mt.w == 0) continue;
        const int pieces = min(mt.w, (int)gridDim.x - mt.z), k0 = blockIdx.x - mt.z;
        const bool few = pieces <= FEW;
        auto at = [&](int k, int r) { return (size_t)(k == 0 ? 2 * mt.z + 1 : 2 * (mt.z + k)) * R + r; };
        // rows k0, k0 + pieces, ...: shared out over the warps of all y, or every y has its channels of each
        const int step = pieces * (few ? CY * CW : 1);
        for (int r = k0 + (few ? pieces * (blockIdx.y * CW + warp) : 0); r < mt.y; r += step) {
            auto values = [&](int k) { return reinterpret_cast<const float4 *>(ws_o + at(k, r) * DV) + lane; };
            auto ml = [&](int k) { return *reinterpret_cast<const float2 *>(ws_ml + at(k, r) * 2); };
            float4 first[2][V];                 // the first two pieces (there are two) are asked for before the maxima
            if (few)
#pragma unroll
                for (int v = 0; v < V; ++v) { first[0][v] = values(0)[32 * v]; first[1][v] = values(1)[32 * v]; }
            float M = -INFINITY;
            bool bad = false;
            for (int k = lane; k < pieces; k += 32) {
                const float2 x = ml(k);
                M = fmaxf(M, x.x);
                bad |= x.y < 0.f;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            if (__any_sync(0xffffffffu, bad)) continue;                  // (the same in all warps)
            const float ref = M == -INFINITY ? 0.f : M;
            const size_t row = (size_t)mt.x + r;
            float l = 0.f;
            if (few) {
                float4 acc[V];
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < pieces; ++k) {
                    const float2 x = ml(k);
                    const float f = exp2f(x.x - ref);
#pragma unroll
                    for (int v = 0; v < V; ++v) add_scaled(acc[v], f, k == 0 ? first[0][v] : k == 1 ? first[1][v] : values(k)[32 * v]);
                    l = fmaf(f, x.y, l);
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    reinterpret_cast<uint2 *>(out + row * DV)[32 * v + lane] =
                        make_uint2(pack_bf16(acc[v].x * inv, acc[v].y * inv), pack_bf16(acc[v].z * inv, acc[v].w * inv));
            } else {
                if (blockIdx.y >= V) break;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = warp; k < pieces; k += CW) {
                    const float2 x = ml(k);
                    const float f = exp2f(x.x - ref);
                    add_scaled(acc, f, values(k)[32 * blockIdx.y]);
                    l = fmaf(f, x.y, l);
                }
                __syncthreads();
                part[warp][lane] = acc;
                if (lane == 0) part_l[warp] = l;
                __syncthreads();
                if (warp != 0) continue;
                for (int k = 1; k < CW; ++k) {
                    add_scaled(acc, 1.f, part[k][lane]);
                    l += part_l[k];
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                reinterpret_cast<uint2 *>(out + row * DV)[32 * blockIdx.y + lane] =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            }
            if (lane == 0 && lse && (few || blockIdx.y == 0))
                lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.693147180559945f;
        }
    }
}

cudaError_t make_maps(CUtensorMap *q, CUtensorMap *c, const void *qp, const void *cp, const PagedPlan &p, int dk, int R) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = prep::tensor_map_encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t one[3] = {1, 1, 1};
    const cuuint64_t qd[2] = {(cuuint64_t)dk, (cuuint64_t)p.T * p.H}, qs[1] = {(cuuint64_t)dk * 2};
    const cuuint32_t qb[2] = {64, (cuuint32_t)R};
    if (fn(q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(qp), qd, qs, qb, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const cuuint64_t cd[3] = {(cuuint64_t)dk, (cuuint64_t)p.page_size, (cuuint64_t)p.num_pages};
    const cuuint64_t cs[2] = {(cuuint64_t)dk * 2, (cuuint64_t)p.page_stride * 2};
    const cuuint32_t cb[3] = {64, (cuuint32_t)(p.page_size < KT ? p.page_size : KT), 1};
    if (fn(c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(cp), cd, cs, cb, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

template <int R, int DV, bool PE, bool GIVE_UP = false>
cudaError_t launch_t(const void *q, const void *cache, const PagedPlan &p, void *out, float *lse, float scale, bool full,
                     void *ws, int sms, int *err, cudaStream_t st)
{
    using L = Lay<R, DV, PE>;
    static_assert(L::NS >= L::MT && L::NS <= 12, "a key tile must fit the ring");
    CUtensorMap mq, mc;
    cudaError_t e = make_maps(&mq, &mc, q, cache, p, DV + (PE ? 64 : 0), R);
    if (e != cudaSuccess) return e;
    Args a;
    a.table = p.page_table; a.lens = p.kv_lens; a.cu = p.cu_seqlens;
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.ws_o = (float *)ws;
    a.ws_ml = ws ? a.ws_o + (size_t)2 * sms * R * DV : nullptr;
    a.meta = ws ? (int4 *)(a.ws_ml + (size_t)2 * sms * R * 2) : nullptr;
    a.T = p.T; a.H = p.H; a.N = p.N; a.per = p.cu_seqlens ? 1 : p.T / p.N;
    a.num_pages = p.num_pages; a.page_size = p.page_size; a.max_pages = p.max_pages;
    a.sl2 = scale * 1.44269504088896f;
    a.full = full;
    a.split = ws != nullptr;
    a.err = err;
    const size_t smem = L::MISC + L::SMALL;
    e = cudaFuncSetAttribute(latent_attn_kernel<R, DV, PE, GIVE_UP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    latent_attn_kernel<R, DV, PE, GIVE_UP><<<sms, L::NT, smem, st>>>(mq, mc, a);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.split) return e;
    return paged::launch_after(latent_combine_kernel<R, DV>, dim3(sms, CY), dim3(32 * CW), 0, st, a.ws_o, a.ws_ml, a.meta,
                               a.out, lse);
}

// rows of a tile: 32 when a sequence has no more than that on average (one token of 32 heads), else 64
int rows_of_tile(const PagedPlan &p) { return (long long)p.T * p.H <= 32LL * p.N ? 32 : 64; }

}  // namespace

size_t latent_attn_workspace(const PagedPlan &p, int dv, int sms) {
    if ((long long)p.max_pages * p.page_size <= WHOLE_TILES * KT) return 0;
    const size_t R = rows_of_tile(p);
    return 2 * (size_t)sms * (R * (dv + 2) * sizeof(float) + sizeof(int4));
}

cudaError_t launch_latent_attn(const void *q, const void *cache, const PagedPlan &p, void *out, float *lse,
                               int dk, int dv, float scale, bool full, bool give_up, void *ws, int sms, int *err,
                               cudaStream_t st)
{
    const bool pe = dk != dv;
#define KDA_LA(R, ...) launch_t<R, __VA_ARGS__>(q, cache, p, out, lse, scale, full, ws, sms, err, st)
    if (give_up) {
        if (dv != 512 || !pe) return cudaErrorNotSupported;
        return rows_of_tile(p) == 32 ? KDA_LA(32, 512, true, true) : KDA_LA(64, 512, true, true);
    }
    if (rows_of_tile(p) == 32)
        return dv == 512 ? (pe ? KDA_LA(32, 512, true) : KDA_LA(32, 512, false))
                         : (pe ? KDA_LA(32, 256, true) : KDA_LA(32, 256, false));
    return dv == 512 ? (pe ? KDA_LA(64, 512, true) : KDA_LA(64, 512, false))
                     : (pe ? KDA_LA(64, 256, true) : KDA_LA(64, 256, false));
#undef KDA_LA
}

}  // namespace kda
