// Tree attention over the 4-bit paged cache for many query rows, on the tcgen05 tensor cores.
//
// The same operator as tree_attn.cu, for items of more rows (nodes x query heads of a K/V
// head) than its warps can serve at the speed of the cache: then the two products bound it,
// 4 rows D operations a position, and next to them the exponentials and the conversion of the
// codes. One CTA an SM; its warps have one part each and meet at mbarriers only:
//
//   convert  (4 warps for K, 4 for V) a position a thread: codes to 16-bit elements in shared
//            memory, exact, laid out for the tensor core (128-byte swizzle; K contiguous along
//            D, and V as it is, read transposed). All become halves; two tiles of each in a
//            ring, the rows of the next on their way by asynchronous copies. Q, and the K of the
//            tree's nodes, are brought to halves by a power of two for each row, exact for what
//            is within 2^-31 of the row's largest element (bfloat16 for all of K cost twice the
//            conversion);
//   multiply (2 threads, one for each softmax group) S = Q K^T and O += P V, sums in tensor
//            memory: S and O twice, up to all 512 columns; P overwrites the half of S it came
//            from. One thread for both groups could not issue as fast as the products end;
//   softmax  (2 groups of 4 warps) S to P, a row a thread, no exchange between threads, the
//            running maximum and sum in registers. A maximum is followed only once it rises by
//            2^8 (then O is rescaled in place), which is rare; P has the row's largest at 2^7 or
//            more, so that a half keeps what is 2^-31 of it (kHeadroom).
//
// A softmax group takes 64 positions at a time, out of two S in turn: while it works on one, the
// tensor core finishes the products with the P before and makes the next scores (with one S of
// 128 columns the group waited about as long as it worked). Items of more than 128 rows give
// each group 128 rows of its own and all positions; items of up to 128 rows give both groups all
// rows and half of each tile's positions (SPLIT), and the two results are joined at the end:
// tensor memory is read by lanes, and both groups own the same lanes.
// The tree's own nodes are the last tile of an item: V stays as it is and P is multiplied in its
// type; for bfloat16 as a sum of two terms, since eight bits are too few. Every wait gives up
// after two seconds; the request's status then says so, and its results are NaN.
//
// Bound: at D = 128 the scores of 64 positions read 6 KB of operands for 32 clocks of products,
// so shared memory allows 80% of the products' rate; the multiplying warps and softmax take
// about 1900 clocks for 64 positions of 256 rows where that needs 1280. 32 64-node trees over up
// to 8192 positions (32 query heads, 8 K/V heads): 186 us, 0.89 PFLOP/s (47% of the measured
// cuBLAS rate); one over 100000 positions: 107 us.

#include "tc_device.cuh"
#include "tree_attn.cuh"

namespace specv {
namespace {

constexpr int kConvert = 256;     // converting threads: K's, then V's
constexpr int kSoftmax = 256;     // threads of the two softmax groups
constexpr int kThreads = kSoftmax + kConvert + 128;   // the last warpgroup: two warps multiply
constexpr int kMmaWarp = (kSoftmax + kConvert) / 32;
// The tree's tile and an item's rest, in context tiles. With 4, 8 and 16: the trees above 195, 187
// and 195 us, with D = 64 147, 151 and 159; 32-node trees (SPLIT) 129, 123 and 127, with D = 64 88,
// 87 and 90; 128 64-node trees over up to 500 positions 183, 174 and 172.
constexpr int kTreeCost = 8;

template <int D, bool SPLIT>
struct Tc {
    static constexpr int kRows = SPLIT ? 128 : 256;              // of an item
    static constexpr int kOperand = 128 * D * 2;                 // a 128 x D operand of 16 bits
    static constexpr int kK = kRows / 128 * kOperand;            // Q first, then K and V rings
    static constexpr int kV = kK + 2 * kOperand;
    // Rows of codes and scales as they come, a thread its own: D / 2 and D / 16 bytes, the
    // pitch free of bank conflicts. As many tiles of them as fit.
    static constexpr int kPitch = D / 2 + 16;
    static constexpr int kRaws = kOperand * (kRows / 128 + 4) > 192 * 1024 - 1 ? 1 : 2;
    static constexpr int kRaw = kV + 2 * kOperand;               // [K, V][kRaws][128][kPitch]
    static constexpr int kSmall = kRaw + 2 * kRaws * 128 * kPitch;   // barriers and words
    static constexpr int kBytes = kSmall + 6144 + 1024;          // and room to align by 1024
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static constexpr int kColumns = 512;                         // 2 (128 + D), a power of two
};

struct Words {
    uint64_t q_full, q_free, k_full[2], k_free[2], v_full[2], v_free[2], drain[2];
    uint64_t s_full[2][2], p_full[2][2], o_full[2];              // of a softmax group; buffers
    uint64_t o_last[2];                                          // once a part
    // Positions of a K/V tile that are attended. A tile's words are written again for the
    // fourth after it, once the scores of the second after it are done: those were issued
    // after its P was waited for.
    unsigned seen[4][4];
    unsigned long long odd[4];    // tree nodes with NaN or infinities in V; part by part likewise
    uint32_t tmem;
    int gave_up;
    int state[2];                 // SPLIT: 0 no tile, 1 O in the cache's units, 2 in V's
    float top[2][128], sum[2][128];
    // 1 / the power of two of each row of Q and of each node's K; a part's are written again for
    // the second after it, once the scores of the one between are done
    float q_down[2][256], k_down[2][64];
};
static_assert(sizeof(Words) <= 6144, "room for the words");

// Byte of 16-byte chunk `j` of row r of an operand of D elements a row.
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
    return (uint32_t)(j >> 3) * (128 * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

template <int D>
struct Row4 {                     // a position's codes and block scales of one head
    uint4 w[D / 32];
    uint32_t sf[D / 64];
};

template <int n>
__device__ __forceinline__ void cp_async(uint32_t smem, const void *gmem) {
    if constexpr (n == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem), "l"(gmem), "n"(n)
                     : "memory");
}

// Starts the copy of a row to `to`. (Registers as the landing place cost more: a wait for an
// older load there was a wait for these too.)
template <int D>
__device__ __forceinline__ void start_row(const void *codes, const void *scales, uint32_t row,
                                          uint32_t to) {
    const char *c = reinterpret_cast<const char *>(codes) + (int64_t)row * (D / 2);
    const char *s = reinterpret_cast<const char *>(scales) + (int64_t)row * (D / 16);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) cp_async<16>(to + i * 16, c + i * 16);
    cp_async<D / 16>(to + D / 2, s);
}

template <int D>
__device__ __forceinline__ void take_row(const char *from, bool ok, Row4<D> &r) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.w[i] = *reinterpret_cast<const uint4 *>(from + i * 16);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint32_t sf = *reinterpret_cast<const uint32_t *>(from + D / 2 + i * 4);
        r.sf[i] = ok ? sf : 0u;      // zeros for a position that is not there
    }
    __syncwarp();                    // the row has been read: its place can be filled again
}

// The row's elements, as halves, into row t of an operand.
template <int D>
__device__ __forceinline__ void convert_row(const Row4<D> &r, char *to, int t) {
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {               // 32 elements: two blocks
        const uint32_t two = e4m3x2_to_f16x2((r.sf[q / 2] >> (q % 2 * 16)) & 0xffffu);
        const uint32_t f[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
        const uint32_t w[4] = {r.w[q].x, r.w[q].y, r.w[q].z, r.w[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            e2m1x8_to_f16x2(w[i], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = hmul2(h[e], f[i / 2]);
            *reinterpret_cast<uint4 *>(to + chunk_at(t, q * 4 + i)) =
                make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
}

// Eight 16-bit elements of a row, whatever their alignment.
__device__ __forceinline__ uint4 load8(const unsigned short *p, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// T: 1 bf16, 2 f16.
template <int T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (T == 1) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <int T>
__device__ __forceinline__ bool odd16(uint32_t x) {
    constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
    return (x & ex) == ex;
}
template <int T>
__device__ __forceinline__ float value16(uint32_t x) {
    return T == 1 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((unsigned short)x));
}

// Eight elements of type T as halves times `up`, and their largest finite magnitude.
template <int T>
__device__ __forceinline__ float largest8(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = fabsf(value16<T>((w[e / 2] >> (e % 2 * 16)) & 0xffffu));
        if (a < INFINITY) big = fmaxf(big, a);
    }
    return big;
}
template <int T>
__device__ __forceinline__ uint4 halves8(const uint4 &x, float up) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = pack2<2>(value16<T>(w[e] & 0xffffu) * up, value16<T>(w[e] >> 16) * up);
    return make_uint4(h[0], h[1], h[2], h[3]);
}
// The power of two that brings `big` into [2^14, 2^15), 2^126 at most (a row of zeros, or of
// almost nothing), and its reciprocal.
__device__ __forceinline__ float scale_up(float big, float &down) {
    const uint32_t e = max(__float_as_uint(big) >> 23, 15u);   // exponent fields add up to 268
    down = __uint_as_float((e - 14u) << 23);
    return __uint_as_float((268u - e) << 23);
}

// The reference of a row comes from a rounded product f s, within 2^-24 of it, which f s - top in
// one rounding brings to light: as 2^-4 at most up to scores of 2^20, beyond as more than a half
// holds. There the products are rounded alike first (RowTile::apart).
constexpr float kApart = 1048576.f;

constexpr int kHalf = 64 * 128;   // bytes from the first 64 rows of an operand to the others

// Jobs of softmax group m in a part of n tiles, the tree's at `tree` (at or past n: not in it).
__device__ __forceinline__ int group_jobs(bool split, int m, int n, int tree) {
    const int contexts = min(n, tree);
    return split ? contexts + (tree < n && m == 0) : 2 * contexts + (tree < n);
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void *to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// A wait of a whole warp: all of it goes on or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up));
}

// S to P of 64 positions, the thread's row: to halves, or (kTree) of 64 nodes to type T.
template <int T, bool kTree>
struct RowTile {
    static constexpr int kChunks = 2;
    uint32_t s[kChunks][32];

    // The scores (kTree: times down[node]), -inf where `see` has no bit; returns their largest.
    __device__ __forceinline__ float load(uint32_t s_tm, const unsigned (&see)[2],
                                          const float *down) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) tmem_ld32(s_tm + q * 32, s[q]);
        tmem_wait_ld(s[0]);
#pragma unroll
        for (int q = 1; q < kChunks; ++q) tmem_loaded(s[q]);
        if (kTree) {
#pragma unroll
            for (int q = 0; q < kChunks; ++q)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    s[q][e] = __float_as_uint(__uint_as_float(s[q][e]) * down[q * 32 + e]);
        }
        if (kTree || (see[0] & see[1]) != 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < kChunks; ++q)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!((see[q] >> e) & 1)) s[q][e] = 0xff800000u;
        }
        float big[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < kChunks; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                big[e / 2 & 3] = fmaxf(fmaxf(big[e / 2 & 3], __uint_as_float(s[q][e])),
                                       __uint_as_float(s[q][e + 1]));
        return fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
    }
    // The scores times f, which becomes 1.
    __device__ __forceinline__ void apart(float &f) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
                s[q][e] = __float_as_uint(__fmul_rn(__uint_as_float(s[q][e]), f));
        f = 1.f;
    }
    // P = 2^(f s - top) over the scores in tensor memory; returns the row's sum.
    __device__ __forceinline__ float store(uint32_t s_tm, float f, float top) {
        const uint64_t f2 = pack_f32x2(f, f), t2 = pack_f32x2(-top, -top);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
            uint32_t lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float a, b;
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[q][e]),
                                                  __uint_as_float(s[q][e + 1])), f2, t2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum[e / 2 & 1] = add_f32x2(sum[e / 2 & 1], pack_f32x2(a, b));
                const uint32_t h = pack2<kTree ? T : 2>(a, b);
                s[q][e / 2] = h;
                if (kTree && T == 1) lo[e / 2] = pack2<1>(a - bf_lo(h), b - bf_hi(h));
            }
            tmem_st16(s_tm + q * 16, s[q]);
            // what bfloat16 leaves, behind the 32 columns of P
            if (kTree && T == 1) tmem_st16(s_tm + 32 + q * 16, lo);
        }
        float a, b;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), a, b);
        return a + b;
    }
};

template <int T, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_tc_kernel(TreeAttnParams P, int row_tiles, int vec) {
    using C_ = Tc<D, SPLIT>;
    constexpr int RT = C_::kRows, KS = D / 16;
    constexpr int kType = T == 1 ? 1 : 0;                        // of the descriptors
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Words &W = *reinterpret_cast<Words *>(smem + C_::kSmall);
    const uint32_t base = smem_addr(smem);
    const spec_fp4_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        bar_init(&W.q_full, kConvert);
        bar_init(&W.q_free, 2);
        for (int i = 0; i < 2; ++i) {
            bar_init(&W.k_full[i], kConvert / 2);
            bar_init(&W.v_full[i], kConvert / 2);
            bar_init(&W.k_free[i], 2);
            bar_init(&W.v_free[i], 2);
            bar_init(&W.drain[i], 1);
            bar_init(&W.o_full[i], 1);
            bar_init(&W.o_last[i], 1);
            for (int j = 0; j < 2; ++j) {
                bar_init(&W.s_full[i][j], 1);
                bar_init(&W.p_full[i][j], 128);
            }
        }
#ifdef SPEC_DEBUG
        W.gave_up = P.lose;
#else
        W.gave_up = 0;
#endif
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&W.tmem, C_::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = W.tmem;
    volatile int *gave_up = &W.gave_up;
    // tensor memory of softmax group m: two S of 64 columns (and P over each) at 128 m, O behind
    // both groups'
    auto s_at = [&](int m) { return tmem + 128 * m; };
    auto o_at = [&](int m) { return tmem + 256 + D * m; };
    uint32_t done = 0, parts = 0;     // tiles and parts before this one: the phases count them
    AttnPart A;

    // Launched with 96 registers a thread, 20 warps: 8 x 128 + 8 x 88 + 4 x 48 = 20 x 96.
    if (tid >= kSoftmax + kConvert) {
        fewer_registers<48>();
        // ---- multiply: for softmax group m. A job is 64 positions (or nodes): two of a tile,
        // one (the group's) if SPLIT, and one of the tree's tile, which SPLIT leaves to group 0.
        // The whole warp runs the loop and waits, one thread of it issues: what the products
        // are given is then the same in all of the warp, as their uniform operands want it.
        const int m = warp - kMmaWarp;
        if (m < 2) {
            AttnWalk walk(P, C.H * row_tiles, kTreeCost, P.columns);
            const bool lead = elect_one();
            const uint32_t o = o_at(m);
            uint32_t jobs = 0;           // of this group before this part
            bool ok = true;
            while (ok && walk.next(P, A)) {
                const int n = A.stop - A.tile, tree = A.nt - 1 - A.tile;
                const int count = group_jobs(SPLIT, m, n, tree);
                auto scores = [&](int j) {
                    const int i = SPLIT ? j : j >> 1, half = SPLIT ? m : j & 1;
                    const uint32_t c = done + i, buf = (jobs + j) & 1;
                    if (SPLIT || half == 0) {     // a tile's second half came with its first
                        ok = ok && warp_wait(&W.k_full[c & 1], (c >> 1) & 1, gave_up);
                    }
                    if (!ok) return;              // no products of what did not come
                    const uint64_t a = smem_desc(base + (SPLIT ? 0 : m * C_::kOperand), 16, 1024);
                    const uint64_t k = smem_desc(
                        base + C_::kK + (c & 1) * C_::kOperand + half * kHalf, 16, 1024);
                    const uint32_t s = s_at(m) + buf * 64;
                    if (lead) {
#pragma unroll
                        for (int d = 0; d < KS; ++d) {
                            const int off = (d >> 2) * (128 * 128) + (d & 3) * 32;
                            mma_ss(s, desc_plus(a, off), desc_plus(k, off),
                                   mma_desc(0, 64, false), d > 0);
                        }
                        mma_commit(&W.s_full[m][buf]);
                        if (SPLIT || half == 1 || i == tree) mma_commit(&W.k_free[c & 1]);
                        if (j == count - 1) mma_commit(&W.q_free);
                    }
                    __syncwarp();
                };
                ok = ok && warp_wait(&W.q_full, parts & 1, gave_up);
                tc_fence_after();
                if (count > 0) scores(0);
                if (count > 1) scores(1);
                if (count == 0 && ok && lead) bar_arrive(&W.q_free);
                __syncwarp();
                for (int j = 0; ok && j < count; ++j) {
                    const int i = SPLIT ? j : j >> 1, half = SPLIT ? m : j & 1;
                    const uint32_t c = done + i, buf = (jobs + j) & 1;
                    if (SPLIT || half == 0) ok = warp_wait(&W.v_full[c & 1], (c >> 1) & 1, gave_up);
                    ok = ok && warp_wait(&W.p_full[m][buf], ((jobs + j) >> 1) & 1, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = smem_desc(
                        base + C_::kV + (c & 1) * C_::kOperand + half * kHalf, 128 * 128, 1024);
                    const uint32_t p = s_at(m) + buf * 64;
                    if (lead) {
                        if (i == tree) {
                            // bfloat16: the two terms of P, 32 columns each
#pragma unroll
                            for (int s = 0; s < (T == 1 ? 8 : 4); ++s)
                                mma_ts(o, p + s * 8, desc_plus(v, (s & 3) * 2048),
                                       mma_desc(kType, D, true), j > 0 || s > 0);
                        } else {
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                mma_ts(o, p + s * 8, desc_plus(v, s * 2048), mma_desc(0, D, true),
                                       j > 0 || s > 0);
                        }
                        mma_commit(&W.o_full[m]);
                        if (j == count - 1) mma_commit(&W.o_last[m]);
                        if (SPLIT || half == 1 || i == tree) mma_commit(&W.v_free[c & 1]);
                    }
                    __syncwarp();
                    if (j + 2 < count) scores(j + 2);
                }
                if (SPLIT && m == 1 && tree < n && ok) {
                    // the tree's tile passes this group by. It is there, so its places' earlier
                    // phases are over, and this arrival counts for the right one.
                    const uint32_t c = done + tree;
                    ok = warp_wait(&W.k_full[c & 1], (c >> 1) & 1, gave_up) &&
                         warp_wait(&W.v_full[c & 1], (c >> 1) & 1, gave_up);
                    if (ok && lead) {
                        bar_arrive(&W.k_free[c & 1]);
                        bar_arrive(&W.v_free[c & 1]);
                    }
                    __syncwarp();
                }
                jobs += count;
                done += n;
                ++parts;
            }
            if (!ok) {
                // products in flight end before tensor memory is freed
                if (lead) mma_commit(&W.drain[m]);
                for (int i = 0; i < (1 << 20) && !bar_try(&W.drain[m], 0); ++i) {
                }
            }
            __syncwarp();
        }
    } else if (tid >= kSoftmax) {
        fewer_registers<88>();
        // ---- convert: K or V, a position a thread ----
        const bool of_v = tid >= kSoftmax + kConvert / 2;
        const int t = (tid - kSoftmax) % (kConvert / 2), R = P.N * P.G;
        const void *codes = of_v ? C.v : C.k, *scales = of_v ? C.v_sf : C.k_sf;
        const unsigned short *nodes = reinterpret_cast<const unsigned short *>(of_v ? P.v : P.k);
        const int64_t node_stride = of_v ? P.v_stride : P.k_stride;
        uint64_t *full = of_v ? W.v_full : W.k_full, *free = of_v ? W.v_free : W.k_free;
        char *ring = smem + (of_v ? C_::kV : C_::kK);
        constexpr int kRaws = C_::kRaws;
        char *mine = smem + C_::kRaw + ((of_v ? kRaws : 0) * 128 + t) * C_::kPitch;
        const uint32_t mine_s = smem_addr(mine);
        AttnWalk walk(P, C.H * row_tiles, kTreeCost, P.columns);
        bool go = true;               // no wait has given up
        while (walk.next(P, A)) {
            const int b = A.b, ctx = A.ctx, n = A.stop - A.tile, tree = A.nt - 1 - A.tile;
            const int head = A.item / row_tiles, row0 = (A.item - head * row_tiles) * RT;
            const int rows = min(RT, R - row0), contexts = min(n, tree);
            if (P.status && tid == kSoftmax && A.tile == 0 && __ldg(P.ctx_len + b) != ctx)
                atomicMax(P.status + b, SPEC_REQ_BAD_SLOT);    // a lost result (below) outweighs it
            const int32_t *table = C.block_table + (int64_t)b * C.max_blocks;
            // the block of this thread's position in the i-th tile (of some position past them)
            auto page = [&](int i) -> int {
                const uint32_t p = (uint32_t)((A.tile + i) * kTile + t);
                return __ldg(table + min(p / (uint32_t)C.block_size, (uint32_t)C.max_blocks - 1u));
            };
            // the rows of the next kRaws tiles are in flight; bit i % 2 of `there`: tile i's is
            unsigned there = 0;
            auto start = [&](int i, int blk) {
                const int p = (A.tile + i) * kTile + t;
                const bool in = i < contexts && p < ctx, ok = in && blk >= 0 && blk < C.num_blocks;
                if (in && !ok && P.status) atomicMax(P.status + b, SPEC_REQ_BAD_SLOT);
                there = (there & ~(1u << (i & 1))) | (ok ? 1u << (i & 1) : 0u);
                if (i < contexts)
                    start_row<D>(codes, scales,
                                 ok ? fp4_row(C, blk, p % (uint32_t)C.block_size, head) : 0u,
                                 mine_s + i % kRaws * 128 * C_::kPitch);
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            const int page0 = page(0), page1 = page(1);
            int next = kRaws == 1 ? page1 : page(2);
            start(0, page0);
            if (kRaws == 2) start(1, page1);
            go = go && warp_wait(&W.q_free, (parts & 1) ^ 1, gave_up);
            if (go) {
                // Q, the D / 8 chunks of a row side by side: all of it copied to its place, and
                // there made halves
                constexpr int kMine = RT * (D / 8) / kConvert;
#pragma unroll 4
                for (int u = 0; u < kMine; ++u) {
                    const int i = u * kConvert + tid - kSoftmax;
                    const int r = i / (D / 8), j = i - r * (D / 8);
                    const uint32_t to = (r >> 7) * C_::kOperand + chunk_at(r & 127, j);
                    const int rr = row0 + min(r, rows - 1), node = rr / P.G;
                    const unsigned short *from =
                        reinterpret_cast<const unsigned short *>(P.q) +
                        ((int64_t)b * P.N + node) * P.q_stride +
                        (int64_t)(head * P.G + rr - node * P.G) * D + j * 8;
                    if (r >= rows)
                        *reinterpret_cast<uint4 *>(smem + to) = make_uint4(0, 0, 0, 0);
                    else if (vec)
                        cp_async<16>(base + to, from);
                    else
                        *reinterpret_cast<uint4 *>(smem + to) = load8(from, false);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
                for (int u = 0; u < kMine; ++u) {
                    const int i = u * kConvert + tid - kSoftmax;
                    const int r = i / (D / 8), j = i - r * (D / 8);
                    uint4 *at = reinterpret_cast<uint4 *>(smem + (r >> 7) * C_::kOperand +
                                                          chunk_at(r & 127, j));
                    const uint4 x = *at;
                    float big = largest8<T>(x), down;
#pragma unroll
                    for (int o = D / 16; o > 0; o >>= 1)
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    const float up = scale_up(big, down);
                    *at = halves8<T>(x, up);
                    if (j == 0) W.q_down[parts & 1][r] = down;
                }
            }
            if (of_v) {
                if (t == 0) W.odd[parts & 3] = 0ull;
                named_sync(2, kConvert / 2);
            }
            fence_async_smem();
            if (go) bar_arrive(&W.q_full);
            for (int i = 0; i < contexts; ++i) {
                const uint32_t c = done + i;
                const int st = c & 1;
                asm volatile("cp.async.wait_group %0;" ::"n"(kRaws - 1) : "memory");
                const bool ok = there >> (i & 1) & 1;
                const unsigned seen = __ballot_sync(0xffffffffu, ok);
                Row4<D> row;
                take_row<D>(mine + i % kRaws * 128 * C_::kPitch, ok, row);
                const int cur = next;
                next = page(i + kRaws + 1);
                start(i + kRaws, cur);
                go = go && warp_wait(&free[st], ((c >> 1) & 1) ^ 1, gave_up);
                if (go) {
                    if (!of_v && lane == 0) W.seen[c & 3][t >> 5] = seen;
                    convert_row<D>(row, ring + st * C_::kOperand, t);
                    fence_async_smem();
                    bar_arrive(&full[st]);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (tree < n) {
                // the nodes' own rows, zeros up to 64; two threads a row, half of it each
                const uint32_t c = done + tree;
                const int st = c & 1;
                char *to = ring + st * C_::kOperand;
                const int r = t >> 1, j0 = (t & 1) * (D / 16);
                const unsigned short *from =
                    nodes + ((int64_t)b * P.N + min(r, P.N - 1)) * node_stride + head * D + j0 * 8;
                uint4 y[D / 16];
                float down = 1.f;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    y[j] = r < P.N ? load8(from + j * 8, vec) : make_uint4(0, 0, 0, 0);
                if (of_v) {
                    // NaN and infinities are left out of the products
                    bool odd = false;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t *w = reinterpret_cast<uint32_t *>(&y[j]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (odd16<T>(w[e])) {
                                w[e] &= 0xffff0000u;
                                odd = true;
                            }
                            if (odd16<T>(w[e] >> 16)) {
                                w[e] &= 0xffffu;
                                odd = true;
                            }
                        }
                    }
                    if (odd) atomicOr(&W.odd[parts & 3], 1ull << r);
                } else {
                    float big = 0.f;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) big = fmaxf(big, largest8<T>(y[j]));
                    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                    const float up = scale_up(big, down);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) y[j] = halves8<T>(y[j], up);
                }
                go = go && warp_wait(&free[st], ((c >> 1) & 1) ^ 1, gave_up);
                if (go) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        *reinterpret_cast<uint4 *>(to + chunk_at(r, j0 + j)) = y[j];
                    if (!of_v && (t & 1) == 0) W.k_down[parts & 1][r] = down;
                    fence_async_smem();
                    bar_arrive(&full[st]);
                }
            }
            done += n;
            ++parts;
        }
    } else {
        more_registers<128>();
        // ---- softmax: this thread's row. A wait that gives up is followed by none, but the
        // groups' barriers are kept.
        const int m = warp >> 2, R = P.N * P.G;
        const int r = (SPLIT ? 0 : m * 128) + (warp & 3) * 32 + lane;    // of the item
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_tm = o_at(m) + lanes;
        const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
        const float unit = P.scale * kLog2e;
        const float cache_unit = unit * (C.k_scale ? __ldg(C.k_scale) : 1.f);
        AttnWalk walk(P, C.H * row_tiles, kTreeCost, P.columns);
        uint32_t jobs = 0, results = 0;   // of this group so far; parts with any
        bool go = true;
        while (walk.next(P, A)) {
            const int b = A.b, n = A.stop - A.tile, tree = A.nt - 1 - A.tile;
            const int head = A.item / row_tiles, row0 = (A.item - head * row_tiles) * RT;
            const int rows = min(RT, R - row0);
            const bool live = r < rows;
            // top: the row's reference; limit: what raises it, or calls for apart(); down: 1 / Q's power of two
            float top = kNoMax, limit = -INFINITY, sum = 0.f, down = 1.f;
            const unsigned long long mask =
                live ? __ldg(P.mask + (int64_t)b * P.N + (row0 + r) / P.G) &
                           (P.N < 64 ? (1ull << P.N) - 1ull : ~0ull)
                     : 0ull;
            int mine = 0;             // jobs of this group in this part, so far
            // follows the largest score x of a tile; rescales O where it stands
            auto follow = [&](float x, bool units, auto &tile, float &f) {
                const bool raise = __any_sync(0xffffffffu, x > limit);
                if (!raise && !units) return;
                float a = 1.f;
                if (raise) {
                    const float to = attn_reference(top, x);
                    a = ex2(top - to);
                    top = to;
                    sum *= a;
                    limit = attn_limit(top);
                    if (fabsf(top) > kApart) {
                        limit = -INFINITY;      // and so for each tile to come
                        tile.apart(f);
                    }
                }
                if (units) a *= v_scale;
                if (mine == 0) return;
                // the scores at hand were made after the product two before this one's
                go = go && warp_wait(&W.o_full[m], (jobs - 1) & 1, gave_up);
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {      // S stays in registers meanwhile
                    uint32_t o[16];
                    tmem_ld16(o_tm + q * 16, o);
                    tmem_wait_ld16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                    tmem_st16(o_tm + q * 16, o);
                }
            };
            const int count = group_jobs(SPLIT, m, n, tree);
            for (int j = 0; j < count; ++j) {
                const int i = SPLIT ? j : j >> 1, half = SPLIT ? m : j & 1;
                const uint32_t buf = jobs & 1, s_tm = s_at(m) + buf * 64 + lanes;
                go = go && warp_wait(&W.s_full[m][buf], (jobs >> 1) & 1, gave_up);
                if (!go) break;
                tc_fence_after();
                if (mine == 0) down = W.q_down[parts & 1][r];
                unsigned see[2];
                float f = attn_factor((i == tree ? unit : cache_unit) * down);
                if (i == tree) {
                    see[0] = (unsigned)mask;
                    see[1] = (unsigned)(mask >> 32);
                    RowTile<T, true> tile;
                    const float x = fmaxf(kNoMax, tile.load(s_tm, see, W.k_down[parts & 1]) * f);
                    follow(x, true, tile, f);      // O leaves the cache's units
                    sum += tile.store(s_tm, f, top);
                } else {
                    see[0] = W.seen[(done + i) & 3][half * 2];
                    see[1] = W.seen[(done + i) & 3][half * 2 + 1];
                    RowTile<T, false> tile;
                    const float x = fmaxf(kNoMax, tile.load(s_tm, see, nullptr) * f);
                    follow(x, false, tile, f);
                    sum += tile.store(s_tm, f, top);
                }
                tmem_wait_st();
                tc_fence_before();
                bar_arrive(&W.p_full[m][buf]);
                ++jobs;
                ++mine;
            }
            // The result: O is done after the group's last product. Its own barrier tells that:
            // two products may be under way here, and o_full tells only two phases apart.
            if (mine > 0) go = go && warp_wait(&W.o_last[m], results++ & 1, gave_up);
            tc_fence_after();
            if (!go) {      // lost: a sum of NaN makes the rows of this part NaN, and the item's
                sum = NAN;
                if (P.status && lane == 0) atomicMax(P.status + b, SPEC_REQ_INTERNAL);
            }
            const bool whole = A.tile == 0 && A.stop == A.nt;
            // the group's O is in V's units once the tree's tile was among its tiles
            const bool in_v = tree < n && (!SPLIT || m == 0);
            float f[2] = {in_v ? 1.f : v_scale, 0.f};     // of this group's O; of the other's
            bool has[2] = {mine > 0, false};
            if (SPLIT) {
                const int row = (warp & 3) * 32 + lane;
                W.top[m][row] = top;
                W.sum[m][row] = sum;
                if (row == 0) W.state[m] = mine == 0 ? 0 : in_v ? 2 : 1;
                tc_fence_before();
                named_sync(1, kSoftmax);
                tc_fence_after();
                const float other = W.top[m ^ 1][row], most = fmaxf(top, other);
                const int state = W.state[m ^ 1];
                has[1] = state != 0;
                f[0] *= ex2(top - most);
                f[1] = ex2(other - most) * (state == 2 ? 1.f : v_scale);
                sum = sum * ex2(top - most) + W.sum[m ^ 1][row] * ex2(other - most);
                top = most;
            }
            const float norm = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            f[0] *= norm;
            f[1] *= norm;
            const int64_t to = live ? attn_row(P, b, head, row0 + r) : 0;
            float *part = attn_slot(P, blockIdx.x, A.tile == 0, RT, D);
            const bool out32 = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
            const unsigned long long odd = tree < n ? W.odd[parts & 3] & mask : 0ull;
            // SPLIT: the groups take half of the columns each, of both Os
            const uint32_t other_tm = o_at(m ^ 1) + lanes;
            for (int q = SPLIT ? m * (D / 64) : 0; q < (SPLIT ? (m + 1) * (D / 64) : D / 32); ++q) {
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = sum == sum ? 0.f : NAN;
#pragma unroll
                for (int g = 0; g < (SPLIT ? 2 : 1); ++g) {
                    if (!has[g]) continue;      // the same for the whole group
                    uint32_t o[32];
                    tmem_ld32((g ? other_tm : o_tm) + q * 32, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(o[e]), f[g], v[e]);
                }
                if (!live) continue;
                // NaN and infinities of nodes that this row sees
                for (unsigned long long left = odd; left; left &= left - 1) {
                    const int j = __ffsll(left) - 1;
                    const int node = (row0 + r) / P.G;
                    const unsigned short *qp =
                        reinterpret_cast<const unsigned short *>(P.q) +
                        ((int64_t)b * P.N + node) * P.q_stride +
                        (int64_t)(head * P.G + row0 + r - node * P.G) * D;
                    const unsigned short *kp = reinterpret_cast<const unsigned short *>(P.k) +
                                               ((int64_t)b * P.N + j) * P.k_stride + head * D;
                    const unsigned short *vp = reinterpret_cast<const unsigned short *>(P.v) +
                                               ((int64_t)b * P.N + j) * P.v_stride + head * D;
                    float dot = 0.f;
#pragma unroll 1
                    for (int d = 0; d < D; ++d)
                        dot = fmaf(value16<T>(__ldg(qp + d)), value16<T>(__ldg(kp + d)), dot);
                    const float w = ex2(dot * unit - top);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t y = __ldg(vp + q * 32 + e);
                        if (odd16<T>(y)) v[e] += w * value16<T>(y);
                    }
                }
                if (whole && out32) {
                    unsigned short *p = reinterpret_cast<unsigned short *>(P.out) + to * D + q * 32;
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = pack2<T>(v[e + 2 * k], v[e + 2 * k + 1]);
                        store32(p + e, w);
                    }
                } else if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        store_out4<T>(P.out, to * D + q * 32 + e,
                                      make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[e + k]);
                        store32(part + (int64_t)r * D + q * 32 + e, w);
                    }
                }
            }
            if (live && (!SPLIT || m == 0)) {
                if (whole) {
                    if (P.lse) P.lse[to] = attn_lse(top, sum);
                } else {
                    part[RT * D + r] = top;
                    part[RT * (D + 1) + r] = sum;
                }
            }
            tc_fence_before();
            if (SPLIT) named_sync(1, kSoftmax);    // both Os have been read
            done += n;
            ++parts;
        }
        if (tid == 0) attn_note(P, walk.r, A, parts > 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, C_::kColumns);
}

template <int T, int D, bool SPLIT>
cudaError_t launch(const TreeAttnParams &p, int grid, cudaStream_t st) {
    using C_ = Tc<D, SPLIT>;
    const cudaError_t e = cudaFuncSetAttribute(tree_attn_tc_kernel<T, D, SPLIT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C_::kBytes);
    if (e != cudaSuccess) return e;
    const int row_tiles = (p.N * p.G + C_::kRows - 1) / C_::kRows;
    auto vec16 = [](const void *q, int64_t stride) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride % 8 == 0;
    };
    const int vec = vec16(p.q, p.q_stride) && vec16(p.k, p.k_stride) && vec16(p.v, p.v_stride);
    tree_attn_tc_kernel<T, D, SPLIT><<<grid, kThreads, C_::kBytes, st>>>(p, row_tiles, vec);
    return cudaGetLastError();
}

}  // namespace

int tree_attn_tc_cost() { return kTreeCost; }
int tree_attn_tc_rows(int R) { return R > 128 ? 256 : 128; }

cudaError_t launch_tree_attn_tc(const TreeAttnParams &p, int grid, cudaStream_t st) {
    const bool split = tree_attn_tc_rows(p.N * p.G) == 128;
    if (p.cache.D == 64) {
        if (p.dtype == 1)
            return split ? launch<1, 64, true>(p, grid, st) : launch<1, 64, false>(p, grid, st);
        return split ? launch<2, 64, true>(p, grid, st) : launch<2, 64, false>(p, grid, st);
    }
    if (p.dtype == 1)
        return split ? launch<1, 128, true>(p, grid, st) : launch<1, 128, false>(p, grid, st);
    return split ? launch<2, 128, true>(p, grid, st) : launch<2, 128, false>(p, grid, st);
}

}  // namespace specv
