// latent_attn.cu -- attention of each sequence's new tokens over the paged
// latent cache (kda_latent_attn) on tcgen05, keys on the rows of the tiles.
//
// All heads of a token attend to the same vectors, so a sequence's (token,
// head) rows are one matrix Q [L * H, dk] against one matrix C [kv, dk] whose
// first dv columns are also the values.  Per tile of 128 keys and tile of R
// rows (R = 32 or 64):
//     S^T = C_tile Q^T           (M = 128 keys, N = R rows, K = dk)
//     P^T = 2^(S^T s - m)        running maximum m per row (column of S^T)
//     O^T += C_tile[:, :dv]^T P^T   (dv / 128 products, M = 128 channels, N = R, K = 128)
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
// them in a fixed order, so results do not depend on timing.
//
// Roles: 4 * R / 32 softmax warps (thread = key row of S^T, 32 columns), one TMA
// warp, one MMA warp.  Every wait is bounded and watches an abort flag; a wait
// that runs out sets the device error word and the block drains and returns.
#include "kernels.h"
#include "paged.cuh"
#include "prep_common.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int KT = 128;                       // keys of a tile
constexpr float TH = 8.f;                     // growth of a maximum (log2) that is let pass

__host__ __device__ constexpr uint32_t idesc(int M, int N, bool mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((mn ? 1u : 0u) << 15) | ((mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int R, int DV, bool PE>
struct Lay {
    static constexpr int MT = DV / 128;                       // stages (128 channels) of a key tile
    static constexpr int NQ = DV / 64 + (PE ? 1 : 0);         // 64-channel pieces of Q
    static constexpr int SW = 4 * (R / 32);                   // softmax warps
    static constexpr int NT = 32 * (SW + 2);
    static constexpr uint32_t STAGE = 32768;                  // 128 keys x 128 channels
    static constexpr uint32_t PBYTES = KT * R * 2;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t QP = R * 128;                   // one piece of Q
    // the positional piece of the keys; at R = 64 P^T takes its place once S^T is done
    static constexpr bool ALIAS = PE && R == 64;
    static constexpr uint32_t X_OFF = Q_OFF + NQ * QP;
    static constexpr uint32_t P_OFF = X_OFF + (PE && !ALIAS ? 16384 : 0);
    static constexpr uint32_t ST_OFF = P_OFF + (ALIAS ? 16384 : PBYTES);
    static constexpr int NS = (227 * 1024 - 1024 - 4096 - (int)ST_OFF) / (int)STAGE;
    static constexpr uint32_t MISC = ST_OFF + NS * STAGE;     // barriers and small tables
    static constexpr uint32_t BYTES = MISC + 4096;
    // TMEM: two S^T buffers, then O^T
    static constexpr uint32_t O_COL = 2 * R;
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

struct Args {
    const int32_t *table, *lens, *cu;
    __nv_bfloat16 *out;
    float *lse;
    float *ws_o, *ws_ml;         // [2 * blocks][R][DV], [2 * blocks][R][2]
    int4 *meta;                  // [blocks]: first row, rows, further pieces
    int T, H, N, per, num_pages, page_size, max_pages;
    float sl2;                   // scale * log2 e
    bool full;
    int *err;
};

// ---------------------------------------------------------------- schedule
// A sequence's rows and keys.  tiles_of(i): key tiles of row tile i (at least
// one: rows that see nothing are written, too).
template <int R>
struct Seq {
    int first, L, kv, H;         // first token, new tokens, keys (0 tokens if the length is bad)
    bool full, bad;
    __device__ __forceinline__ void load(const Args &a, int n) {
        H = a.H;
        full = a.full;
        const int b = paged::token_offset(a.cu, n, a.per, a.T), e = paged::token_offset(a.cu, n + 1, a.per, a.T);
        kv = a.lens[n];
        first = b;
        L = max(0, e - b);
        bad = kv < 0 || (long long)kv > (long long)a.max_pages * a.page_size;
        if (bad) { L = 0; kv = 0; }
    }
    __device__ __forceinline__ int rows() const { return L * H; }        // T * H < 2^31
    __device__ __forceinline__ int row_tiles() const { return (rows() - 1 + R) / R; }
    // keys that row r sees
    __device__ __forceinline__ int sees(int r) const {
        return full ? kv : min(kv, max(0, kv - L + r / H + 1));
    }
    __device__ __forceinline__ int keys_of(int i) const { return sees(min(rows(), (i + 1) * R) - 1); }
    __device__ __forceinline__ int tiles_of(int i) const { return max(1, (keys_of(i) + KT - 1) / KT); }
    // row tiles i < C(k) have at most k key tiles
    __device__ __forceinline__ int upto(int k) const {
        const long long tokens = (long long)KT * k - kv + L;             // tokens that see <= 128 k keys
        if (full) return KT * (long long)k >= kv ? row_tiles() : 0;
        if (tokens >= L) return row_tiles();
        return tokens <= 0 ? 0 : (int)(tokens * H / R);
    }
    __device__ __forceinline__ long long units() const {
        const int nt = row_tiles();
        if (nt <= 0) return 0;
        long long u = 0;
        int k = tiles_of(0), done = 0;
        while (done < nt) {
            const int c = min(nt, max(done, upto(k)));
            u += (long long)k * (c - done);
            done = c;
            ++k;
        }
        return u;
    }
    // row tile and key tile of unit u
    __device__ __forceinline__ void find(long long u, int &i, int &j) const {
        const int nt = row_tiles();
        int k = tiles_of(0), done = 0;
        while (done < nt) {
            const int c = min(nt, max(done, upto(k)));
            const long long here = (long long)k * (c - done);
            if (u < here) {
                i = done + (int)(u / k);
                j = (int)(u % k);
                return;
            }
            u -= here;
            done = c;
            ++k;
        }
        i = nt - 1;
        j = 0;
    }
};

// The segments of a block's range: a row tile of a sequence and key tiles
// [j0, j1) of its `tiles`.  Every role walks them by itself.
template <int R>
struct Walk {
    Seq<R> s;
    int n, i, j0, j1, tiles;
    long long left;
    __device__ __forceinline__ void start(const Args &a, int n_, int i_, int j_, long long left_) {
        n = n_; i = i_; j0 = j_; left = left_;
        if (left > 0) { s.load(a, n); bound(); }
    }
    __device__ __forceinline__ void bound() {
        tiles = s.tiles_of(i);
        j1 = (int)min((long long)tiles, j0 + left);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const Args &a) {
        left -= j1 - j0;
        if (left <= 0) return;
        j0 = 0;
        ++i;
        while (i >= s.row_tiles()) {
            if (++n >= a.N) { left = 0; return; }
            s.load(a, n);
            i = 0;
        }
        bound();
    }
};

__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_test_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < (1u << 24); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (i > 64) __nanosleep(32);
    }
    return false;
}

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

// Combines v[c] of the warp's 32 lanes, per column c: lane c ends up with the
// result of column c.  Halving: 31 shuffles instead of 5 * 32.
template <bool MAX>
__device__ __forceinline__ float across_lanes(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
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

template <int R, int DV, bool PE>
__global__ void __launch_bounds__(Lay<R, DV, PE>::NT, 1)
latent_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c, const Args a)
{
    using L = Lay<R, DV, PE>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::MISC);
    uint64_t *empty = full + L::NS;
    uint64_t *x_full = empty + L::NS, *x_empty = x_full + 1, *q_full = x_full + 2, *q_empty = x_full + 3;
    uint64_t *s_full = x_full + 4;                            // [2]
    uint64_t *p_full = x_full + 6, *o_full = x_full + 7, *drain = x_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_full + 9);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    long long *scan = reinterpret_cast<long long *>(x_full + 10);         // [16] warp sums, then the start
    int *start = reinterpret_cast<int *>(scan + 16);                       // sequence, row tile, key tile
    float *red = reinterpret_cast<float *>(start + 4);                     // [SW][32]
    float *mine = red + L::SW * 32;                                        // [SW][2][32]: a warp's maxima and factors
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < L::NS; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        mbar_init(x_full, 1); mbar_init(x_empty, 1); mbar_init(q_full, 1); mbar_init(q_empty, 1);
        mbar_init(&s_full[0], 1); mbar_init(&s_full[1], 1);
        mbar_init(p_full, L::SW); mbar_init(o_full, 1); mbar_init(drain, 1);
        *abort_flag = 0;
        start[0] = 0; start[1] = 0; start[2] = 0;
        fence_mbar_init();
    }
    if (warp == 0) { tmem_alloc(tmem_slot, L::COLS); tmem_relinquish(); }

    // ---- this block's range of the (row tile, key tile) units
    const int per = (a.N + L::NT - 1) / L::NT;
    const int n0 = min(a.N, tid * per), n1 = min(a.N, n0 + per);
    long long mysum = 0;
    for (int n = n0; n < n1; ++n) {
        Seq<R> s;
        s.load(a, n);
        if (s.bad && blockIdx.x == 0) set_device_error(a.err, paged::kErrBadPage);
        mysum += s.units();
    }
    long long incl = mysum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    long long before = incl - mysum, total = 0;
    for (int w = 0; w < L::NT / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    // as many ranges as blocks, but none empty: the pieces of a row tile lie in consecutive blocks
    const long long G = max(1LL, min((long long)gridDim.x, total));
    const bool works = blockIdx.x < G && total > 0;
    const long long u0 = works ? total * blockIdx.x / G : 0, u1 = works ? total * (blockIdx.x + 1) / G : 0;
    if (u0 < u1 && u0 >= before && u0 < before + mysum) {
        long long u = u0 - before;
        for (int n = n0; n < n1; ++n) {
            Seq<R> s;
            s.load(a, n);
            const long long here = s.units();
            if (u < here) {
                int i, j;
                s.find(u, i, j);
                start[0] = n; start[1] = i; start[2] = j;
                break;
            }
            u -= here;
        }
    }
    __syncthreads();
    Walk<R> w;
    w.start(a, start[0], start[1], start[2], u1 - u0);

    if (warp == L::SW) {
        // ---------------- TMA: Q of each segment, then its key tiles ----------------
        int st = 0, st_use = 0, tiles = 0, segs = 0;          // stage, its uses, X uses, Q uses
        bool ok = true;
        const int lps = 31 - __clz(a.page_size);
        for (; w.more() && ok; w.next(a)) {
            const int end = w.s.keys_of(w.i);
            if (lane == 0) ok = segs == 0 || wait_on(q_empty, (segs - 1) & 1, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                const int row = w.s.first * a.H + w.i * R;
                mbar_arrive_expect_tx(q_full, L::NQ * L::QP);
                for (int p = 0; p < L::NQ; ++p) tma_2d(sm + L::Q_OFF + p * L::QP, &tm_q, 64 * p, row, q_full);
            }
            ++segs;
            for (int j = w.j0; j < w.j1 && ok; ++j) {
                const int pages = (max(0, min(KT, end - j * KT)) + a.page_size - 1) >> lps;
                int page = 0;
                if (lane < pages) page = a.table[(long long)w.n * a.max_pages + ((j * KT) >> lps) + lane];
                // boxes of 64 channels x one page's rows
                for (int m = 0; m <= L::MT && ok; ++m) {
                    const bool x = m == L::MT;
                    if (x && !PE) break;
                    uint64_t *fb = x ? x_full : &full[st];
                    if (lane == 0) ok = x ? tiles == 0 || wait_on(x_empty, (tiles - 1) & 1, abort_flag)
                                          : st_use == 0 || wait_on(&empty[st], (st_use - 1) & 1, abort_flag);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)pages * a.page_size * 128 * (x ? 1 : 2));
                    __syncwarp();
                    unsigned char *dst = sm + (x ? L::X_OFF : L::ST_OFF + st * L::STAGE) + lane * a.page_size * 128;
                    if (lane < pages) {
                        prep::tma_load_3d(dst, &tm_c, 128 * m, 0, page, fb);
                        if (!x) prep::tma_load_3d(dst + 16384, &tm_c, 128 * m + 64, 0, page, fb);
                    }
                    if (!x && ++st == L::NS) { st = 0; ++st_use; }
                }
                ++tiles;
            }
        }
        if (!ok && lane == 0) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; }
        // never leave with copies in flight into this block's shared memory
        __syncwarp();
        if (lane == 0 && !ok) {
            for (int s = 0; s < L::NS; ++s) {
                const int uses = st_use + (s < st ? 1 : 0);
                if (uses > 0) mbar_wait(&full[s], (uses - 1) & 1, 1u << 20);
            }
            if (PE && tiles > 0) mbar_wait(x_full, (tiles - 1) & 1, 1u << 20);
            if (segs > 0) mbar_wait(q_full, (segs - 1) & 1, 1u << 20);
        }
    } else if (warp == L::SW + 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            constexpr uint32_t ID_S = idesc(128, R, false), ID_O = idesc(128, R, true);
            const uint32_t base = smem_u32(sm);
            const DescParts q_d = smem_desc_parts(base + L::Q_OFF, 16, 1024, 2);
            const DescParts k_d = smem_desc_parts(base + L::ST_OFF, 16, 1024, 2);        // keys, K-major
            const DescParts x_d = smem_desc_parts(base + L::X_OFF, 16, 1024, 2);
            const DescParts v_d = smem_desc_parts(base + L::ST_OFF, 16384, 1024, 2);     // values, MN-major
            const DescParts p_d = smem_desc_parts(base + L::P_OFF, L::B_SBO, L::B_SBO, L::B_LAYOUT);
            constexpr uint32_t PK = (2 * L::B_SBO) >> 4;
            int st = 0, st_use = 0, tiles = 0, segs = 0;
            bool ok = true, any = false;
            for (; w.more() && ok; w.next(a)) {
                ok = wait_on(q_full, segs & 1, abort_flag);
                ++segs;
                for (int j = w.j0; j < w.j1 && ok; ++j) {
                    const uint32_t d = tmem + (tiles & 1) * R;
                    int s = st, use = st_use;
                    for (int m = 0; m < L::MT && ok; ++m) {
                        if (!(ok = wait_on(&full[s], use & 1, abort_flag))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16_p(d, k_d.lo + ((s * L::STAGE + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4), k_d.hi,
                                        q_d.lo + (((2 * m + (kk >> 2)) * L::QP + (kk & 3) * 32) >> 4), q_d.hi, ID_S, m > 0 || kk > 0);
                        any = true;
                        if (++s == L::NS) { s = 0; ++use; }
                    }
                    if (PE && ok && (ok = wait_on(x_full, tiles & 1, abort_flag))) {
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16_p(d, x_d.lo + ((kk * 32) >> 4), x_d.hi, q_d.lo + (((L::NQ - 1) * L::QP + kk * 32) >> 4),
                                        q_d.hi, ID_S, 1);
                        if (!L::ALIAS) umma_commit(x_empty);
                    }
                    if (!ok) break;
                    umma_commit(&s_full[tiles & 1]);
                    if (j + 1 == w.j1) umma_commit(q_empty);
                    if (!(ok = wait_on(p_full, tiles & 1, abort_flag))) break;
                    tc_fence_after();
                    for (int m = 0; m < L::MT; ++m) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_bf16_p(tmem + L::O_COL + m * R, v_d.lo + ((st * L::STAGE + kk * 2048) >> 4), v_d.hi,
                                        p_d.lo + kk * PK, p_d.hi, ID_O, j > w.j0 || kk > 0);
                        umma_commit(&empty[st]);
                        if (++st == L::NS) { st = 0; ++st_use; }
                    }
                    if (PE && L::ALIAS) umma_commit(x_empty);
                    if (j + 1 == w.j1) umma_commit(o_full);
                    ++tiles;
                }
            }
            if (!ok) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; }
            // never free TMEM or shared memory under a running MMA
            if (any) {
                umma_commit(drain);
                mbar_wait(drain, 0, 1u << 20);
            }
        }
    } else {
        // ---------------- softmax and output: thread = key t of the tile (TMEM lane),
        // rows 32 cg .. 32 cg + 31 of the row tile ----------------
        const int t = 32 * (warp & 3) + lane, cg = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 32 * cg;
        float *my_m = mine + warp * 64, *my_f = my_m + 32;
        float *my_red = red + cg * 128;
        int tiles = 0, segs = 0;
        bool ok = true;
        int4 meta = make_int4(0, 0, 0, 0);
        for (; w.more() && ok; w.next(a)) {
            const int rows = min(R, w.s.rows() - w.i * R);               // of this row tile
            const int end = w.s.keys_of(w.i);
            const int row = 32 * cg + lane;                              // this lane's row, for the statistics
            const int sees = row < rows ? w.s.sees(w.i * R + row) : 0;
            const int least = __reduce_min_sync(0xffffffffu, row < rows ? sees : 0x7fffffff);
            // the sequence's pages, all of them: every block that has a piece of it comes to the same answer
            bool bad = false;
            for (int p = t; p * a.page_size < w.s.kv; p += 128) {
                const int pg = a.table[(long long)w.n * a.max_pages + p];
                bad |= pg < 0 || pg >= a.num_pages;
            }
            float m_run = -INFINITY, l[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) l[c] = 0.f;
            for (int j = w.j0; j < w.j1; ++j) {
                ok = wait_on(&s_full[tiles & 1], (tiles >> 1) & 1, abort_flag);
                tc_fence_after();
                float x[32], y[32];
                tmem_ld32(lanes + (tiles & 1) * R, x);
                tmem_wait_ld();
                const int key = j * KT + t;
                if (j * KT + KT > least) {
                    // some row of this group does not see the whole tile
                    my_m[lane] = __int_as_float(sees);
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] = key < __float_as_int(my_m[c]) ? x[c] * a.sl2 : -INFINITY;
                    __syncwarp();
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] *= a.sl2;
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) y[c] = x[c];
                my_red[(warp & 3) * 32 + lane] = across_lanes<true>(y, lane);
                if (named_bar_or(1 + cg, 128, !ok)) { ok = false; break; }
                const float mt = fmaxf(fmaxf(my_red[lane], my_red[32 + lane]), fmaxf(my_red[64 + lane], my_red[96 + lane]));
                // the reference is raised only when the maximum has outgrown it by 2^TH
                const bool raise = mt > m_run + TH || (m_run == -INFINITY && mt > -INFINITY);
                const float m_new = raise ? mt : m_run;
                my_m[lane] = m_new == -INFINITY ? 0.f : m_new;
                my_f[lane] = raise ? exp2f(m_run - m_new) : 1.f;
                m_run = m_new;
                const bool any = __any_sync(0xffffffffu, raise) && j > w.j0;
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = prep::ex2_approx(x[c] - my_m[c]);
                if (any) {
                    // the product of the previous tile is complete: S^T of this one was issued after it
#pragma unroll
                    for (int c = 0; c < 32; ++c) l[c] *= my_f[c];
                    for (int m = 0; m < L::MT; ++m) {
                        tmem_ld32(lanes + L::O_COL + m * R, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c) y[c] *= my_f[c];
                        tmem_st32(lanes + L::O_COL + m * R, y);
                    }
                    tmem_wait_st();
                }
                unsigned char *P = sm + L::P_OFF;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<uint4 *>(P + L::p_off(t, 4 * cg + g)) =
                        make_uint4(pack_bf16(x[8 * g], x[8 * g + 1]), pack_bf16(x[8 * g + 2], x[8 * g + 3]),
                                   pack_bf16(x[8 * g + 4], x[8 * g + 5]), pack_bf16(x[8 * g + 6], x[8 * g + 7]));
#pragma unroll
                for (int c = 0; c < 32; ++c) l[c] += x[c];
                if (key >= end && cg == 0) {
                    // rows that hold no key of this row tile may hold anything: 0 * NaN is not 0
                    int s = (int)((long long)tiles * L::MT % L::NS);
                    for (int m = 0; m < L::MT; ++m) {
                        unsigned char *v = sm + L::ST_OFF + s * L::STAGE + t * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            *reinterpret_cast<uint4 *>(v + 16 * e) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(v + 16384 + 16 * e) = make_uint4(0, 0, 0, 0);
                        }
                        if (++s == L::NS) s = 0;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                ++tiles;
            }
            if (!ok) break;
            ok = wait_on(o_full, segs & 1, abort_flag);
            ++segs;
            tc_fence_after();
            my_red[(warp & 3) * 32 + lane] = across_lanes<false>(l, lane);
            if (named_bar_or(1 + cg, 128, !ok)) { ok = false; break; }
            const float sum = (my_red[lane] + my_red[32 + lane]) + (my_red[64 + lane] + my_red[96 + lane]);
            bad = named_bar_or(1 + cg, 128, bad);
            if (bad && tid == 0) set_device_error(a.err, paged::kErrBadPage);
            const long long row0 = (long long)w.s.first * a.H + (long long)w.i * R;
            if (w.j0 == 0 && w.j1 == w.tiles) {
                // the whole row tile was here
                my_m[lane] = sum > 0.f ? 1.f / sum : 0.f;
                __syncwarp();
                if (!bad) {
                    if (a.lse && (warp & 3) == 0 && row < rows)
                        a.lse[row0 + row] = sum > 0.f ? (m_run + log2f(sum)) * 0.693147180559945f : -INFINITY;
                    for (int m = 0; m < L::MT; ++m) {
                        float o[32];
                        tmem_ld32(lanes + L::O_COL + m * R, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * cg + c < rows)
                                a.out[(row0 + 32 * cg + c) * DV + 128 * m + t] = __float2bfloat16_rn(o[c] * my_m[c]);
                    }
                }
            } else {
                // a piece: slot 0 if it continues the row tile, slot 1 if it begins it
                const int slot = 2 * blockIdx.x + (w.j0 == 0 ? 1 : 0);
                if ((warp & 3) == 0) {
                    float *ml = a.ws_ml + ((size_t)slot * R + row) * 2;
                    ml[0] = m_run;
                    ml[1] = bad ? -1.f : sum;
                }
                for (int m = 0; m < L::MT; ++m) {
                    float o[32];
                    tmem_ld32(lanes + L::O_COL + m * R, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        a.ws_o[((size_t)slot * R + 32 * cg + c) * DV + 128 * m + t] = o[c];
                }
                if (w.j0 == 0) {
                    // its last unit lies in block b: u0(b) <= last < u0(b + 1)
                    const long long last = u1 - 1 + (w.tiles - w.j1);
                    long long b = ((last + 1) * G + total - 1) / total - 1;
                    meta = make_int4((int)row0, rows, (int)(b - blockIdx.x), 0);
                }
            }
            tc_fence_before();
            __syncwarp();
        }
        if (!ok) { set_device_error(a.err, kErrWaitTimeout); *abort_flag = 1; meta.z = 0; }
        if (tid == 0) a.meta[blockIdx.x] = meta;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, L::COLS);
}

// Joins the pieces of a row tile that begins in block x's range and goes on in
// the next ones: out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.  One row
// a block; the pieces are shared out over four groups of threads.
template <int R, int DV>
__global__ void __launch_bounds__(DV)
latent_combine_kernel(const float *__restrict__ ws_o, const float *__restrict__ ws_ml, const int4 *__restrict__ meta,
                      __nv_bfloat16 *__restrict__ out, float *__restrict__ lse)
{
    const int b = blockIdx.x, r = blockIdx.y;
    const int4 mt = meta[b];
    if (mt.z == 0 || r >= mt.y) return;
    const int pieces = mt.z + 1;
    auto slot = [&](int k) { return k == 0 ? 2 * b + 1 : 2 * (b + k); };
    __shared__ float4 part[4][DV / 4];
    __shared__ float red[DV / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float M = -INFINITY;
    bool bad = false;
    for (int k = tid; k < pieces; k += DV) {
        const float2 x = *reinterpret_cast<const float2 *>(ws_ml + ((size_t)slot(k) * R + r) * 2);
        M = fmaxf(M, x.x);
        bad |= x.y < 0.f;
    }
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[warp] = M;
    if (__syncthreads_or(bad)) return;
    for (int i = 0; i < DV / 32; ++i) M = fmaxf(M, red[i]);
    const float ref = M == -INFINITY ? 0.f : M;
    const int g = tid / (DV / 4), c = tid % (DV / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int k = g; k < pieces; k += 4) {
        const size_t at = (size_t)slot(k) * R + r;
        const float2 x = *reinterpret_cast<const float2 *>(ws_ml + at * 2);
        const float f = exp2f(x.x - ref);
        const float4 o = *reinterpret_cast<const float4 *>(ws_o + at * DV + 4 * c);
        acc.x = fmaf(f, o.x, acc.x); acc.y = fmaf(f, o.y, acc.y);
        acc.z = fmaf(f, o.z, acc.z); acc.w = fmaf(f, o.w, acc.w);
        l = fmaf(f, x.y, l);
    }
    part[g][c] = acc;
    __syncthreads();                    // (red was read above: every thread is past it)
    if (c == 0) red[g] = l;
    __syncthreads();
    if (g == 0) {
        l = (red[0] + red[1]) + (red[2] + red[3]);
        float4 s = part[0][c];
        for (int k = 1; k < 4; ++k) {
            s.x += part[k][c].x; s.y += part[k][c].y; s.z += part[k][c].z; s.w += part[k][c].w;
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t row = (size_t)mt.x + r;
        *reinterpret_cast<uint2 *>(out + row * DV + 4 * c) =
            make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
        if (c == 0 && lse) lse[row] = l > 0.f ? (M + log2f(l)) * 0.693147180559945f : -INFINITY;
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
    const cuuint32_t cb[3] = {64, (cuuint32_t)p.page_size, 1};
    if (fn(c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(cp), cd, cs, cb, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

template <int R, int DV, bool PE>
cudaError_t launch_t(const void *q, const void *cache, const PagedPlan &p, void *out, float *lse, float scale, bool full,
                     void *ws, int sms, int *err, cudaStream_t st)
{
    using L = Lay<R, DV, PE>;
    static_assert(L::NS >= L::MT, "a key tile must fit the ring");
    static_assert((2 * L::NS + 20) * 8 + 128 + 16 + (L::SW * 32 + L::SW * 64) * 4 + 64 <= 4096, "small tables");
    CUtensorMap mq, mc;
    cudaError_t e = make_maps(&mq, &mc, q, cache, p, DV + (PE ? 64 : 0), R);
    if (e != cudaSuccess) return e;
    Args a;
    a.table = p.page_table; a.lens = p.kv_lens; a.cu = p.cu_seqlens;
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.ws_o = (float *)ws;
    a.ws_ml = a.ws_o + (size_t)2 * sms * R * DV;
    a.meta = (int4 *)(a.ws_ml + (size_t)2 * sms * R * 2);
    a.T = p.T; a.H = p.H; a.N = p.N; a.per = p.cu_seqlens ? 1 : p.T / p.N;
    a.num_pages = p.num_pages; a.page_size = p.page_size; a.max_pages = p.max_pages;
    a.sl2 = scale * 1.44269504088896f;
    a.full = full;
    a.err = err;
    const size_t smem = L::BYTES + 1024;
    e = cudaFuncSetAttribute(latent_attn_kernel<R, DV, PE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    latent_attn_kernel<R, DV, PE><<<sms, L::NT, smem, st>>>(mq, mc, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    latent_combine_kernel<R, DV><<<dim3(sms, R), DV, 0, st>>>(a.ws_o, a.ws_ml, a.meta, a.out, lse);
    return cudaGetLastError();
}

// rows of a tile: 32 when a sequence has no more than that on average (one token of 32 heads), else 64
int rows_of_tile(const PagedPlan &p) { return (long long)p.T * p.H <= 32LL * p.N ? 32 : 64; }

}  // namespace

size_t latent_attn_workspace(const PagedPlan &p, int dv, int sms) {
    const size_t R = rows_of_tile(p);
    return 2 * (size_t)sms * R * (dv + 2) * sizeof(float) + sms * sizeof(int4);
}

cudaError_t launch_latent_attn(const void *q, const void *cache, const PagedPlan &p, void *out, float *lse,
                               int dk, int dv, float scale, bool full, void *ws, int sms, int *err, cudaStream_t st)
{
    const bool pe = dk != dv;
#define KDA_LA(R, DV, PE) launch_t<R, DV, PE>(q, cache, p, out, lse, scale, full, ws, sms, err, st)
    if (rows_of_tile(p) == 32)
        return dv == 512 ? (pe ? KDA_LA(32, 512, true) : KDA_LA(32, 512, false))
                         : (pe ? KDA_LA(32, 256, true) : KDA_LA(32, 256, false));
    return dv == 512 ? (pe ? KDA_LA(64, 512, true) : KDA_LA(64, 512, false))
                     : (pe ? KDA_LA(64, 256, true) : KDA_LA(64, 256, false));
#undef KDA_LA
}

}  // namespace kda
