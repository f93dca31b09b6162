// Tree attention over the 4-bit paged cache for many query rows, on the tcgen05 tensor cores.
//
// The same operator as tree_attn.cu, for items of more rows (nodes x query heads of a K/V
// head) than its warps can serve at the speed of the cache: then the two products bound it,
// 4 rows D operations a position, and next to them the exponentials and the conversion of the
// codes. One CTA an SM takes NT tiles of 128 rows of an item against tiles of 128 positions:
//
//   convert  (4 warps) a position each: codes to 16-bit elements in shared memory, exact, laid
//            out for the tensor core (128-byte swizzle; K contiguous along D, and V as it is,
//            read transposed). K becomes the type of Q, V halves; two tiles of each in a ring;
//   multiply (1 thread) S = Q K^T and O += P V, sums in tensor memory (all 512 columns for two
//            row tiles of D = 128: S and O of each); P overwrites the half of S it came from;
//   softmax  (4 warps a row tile, a row a thread, no exchange between threads) S to P with the
//            running maximum and sum in registers. A maximum is followed only once it rises by
//            2^8 (then O is rescaled in place), which is rare. S is read twice, for the maximum
//            and for P, since it does not fit in a thread's registers.
// With two row tiles the tensor core works on one while the other is in softmax. The tree's own
// nodes are the last tile of an item: their rows are copied instead of converted and P is
// multiplied in their type; for bfloat16 as a sum of two terms, since eight bits are too few.
// Every wait gives up after two seconds; the request's status then says so.

#include "tc_device.cuh"
#include "tree_attn.cuh"

namespace specv {
namespace {

constexpr float kRescale = 8.f;
constexpr int kConvert = 128;     // converting threads

template <int D, int NT>
struct Tc {
    static constexpr int kThreads = NT * 128 + kConvert + 32;
    static constexpr int kOperand = 128 * D * 2;                 // a 128 x D operand of 16 bits
    static constexpr int kK = NT * kOperand;                     // Q first, then K and V rings
    static constexpr int kV = kK + 2 * kOperand;
    static constexpr int kSmall = kV + 2 * kOperand;             // barriers and words
    static constexpr int kBytes = kSmall + 512 + 1024;           // and room to align by 1024
    static constexpr int kColumns = NT * (128 + D) > 256 ? 512 : 256;
};

struct Words {
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], drain;
    // positions of a K/V tile that are attended; a tile's words are written again only after
    // the scores of the tile three before, whose P the multiplying thread has waited for
    unsigned seen[4][4];
    unsigned long long odd;       // tree nodes with NaN or infinities in V
    uint32_t tmem;
    int gave_up, flag;
};

// Byte of 16-byte chunk `j` of row r of an operand of D elements a row.
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
    return (uint32_t)(j >> 3) * (128 * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

// A pair of halves that hold e2m1 values, times a block scale, as bfloat16 (exact): the bits of
// a normal half shifted into a bfloat16's place are the value times 2^-112, which the factor
// (scale * 2^112) restores. Zero stays zero; 0.5 is the smallest other magnitude.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h, uint32_t factor) {
    const uint32_t t = ((h >> 3) & 0x0fff0fffu) | (h & 0x80008000u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t), "r"(factor));
    return r;
}

template <int D>
struct Row4 {                     // a position's codes and block scales of one head
    uint4 w[D / 32];
    uint32_t sf[D / 64];
};

template <int D>
__device__ __forceinline__ void load_row(const void *codes, const void *scales, uint32_t row,
                                         bool ok, Row4<D> &r) {
    const uint4 *c = reinterpret_cast<const uint4 *>(codes) + (int64_t)row * (D / 32);
    const uint32_t *s = reinterpret_cast<const uint32_t *>(scales) + (int64_t)row * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.w[i] = ok ? __ldg(c + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.sf[i] = ok ? __ldg(s + i) : 0u;
}

// The row's elements into row t of an operand; BF: as bfloat16, else as halves.
template <int D, bool BF>
__device__ __forceinline__ void convert_row(const Row4<D> &r, char *to, int t) {
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {               // 32 elements: two blocks
        const uint32_t two = e4m3x2_to_f16x2((r.sf[q / 2] >> (q % 2 * 16)) & 0xffffu);
        uint32_t f[2];
        if constexpr (BF) {
            const float2 s = __half22float2(*reinterpret_cast<const __half2 *>(&two));
            const __nv_bfloat162 a = __float2bfloat162_rn(s.x * 0x1p112f);
            const __nv_bfloat162 b = __float2bfloat162_rn(s.y * 0x1p112f);
            f[0] = *reinterpret_cast<const uint32_t *>(&a);
            f[1] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            f[0] = __byte_perm(two, two, 0x1010);
            f[1] = __byte_perm(two, two, 0x3232);
        }
        const uint32_t w[4] = {r.w[q].x, r.w[q].y, r.w[q].z, r.w[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            e2m1x8_to_f16x2(w[i], h);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = BF ? scaled_bf16x2(h[e], f[i / 2]) : hmul2(h[e], f[i / 2]);
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

// A wait of a whole warp: all of it goes on or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up));
}

template <int T, int D, int NT>
__global__ void __launch_bounds__(Tc<D, NT>::kThreads, 1)
    tree_attn_tc_kernel(TreeAttnParams P, int row_tiles, int vec) {
    using C_ = Tc<D, NT>;
    constexpr int RT = NT * 128, KS = D / 16;
    constexpr int kType = T == 1 ? 1 : 0;                        // of the descriptors
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Words &W = *reinterpret_cast<Words *>(smem + C_::kSmall);
    const uint32_t base = smem_addr(smem);
    const spec_fp4_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = P.N * P.G;
    constexpr int kMmaWarp = NT * 4 + kConvert / 32;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&W.k_full[i], kConvert);
            bar_init(&W.v_full[i], kConvert);
            bar_init(&W.k_free[i], 1);
            bar_init(&W.v_free[i], 1);
            bar_init(&W.s_full[i], 1);
            bar_init(&W.p_full[i], 128);
            bar_init(&W.o_full[i], 1);
        }
        bar_init(&W.drain, 1);
        W.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&W.tmem, C_::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = W.tmem;
    volatile int *gave_up = &W.gave_up;
    // tensor memory of row tile m: S (and P over it) at 128 m, O behind all of S
    auto s_at = [&](int m) { return tmem + 128 * m; };
    auto o_at = [&](int m) { return tmem + 128 * NT + D * m; };
    const float k_scale = C.k_scale ? __ldg(C.k_scale) : 1.f;
    const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
    const float unit = P.scale * kLog2e;

    const AttnRange range = attn_range(P, C.H * row_tiles);
    int b = range.b, item = range.item, tile = range.tile;
    uint32_t done = 0;            // tiles before this item: the barriers' phases count them

    for (int64_t at = range.begin; at < range.end;) {
        const int ctx = attn_ctx(P, b), nt = (ctx + kTile - 1) / kTile + 1;
        const int head = item / row_tiles, row0 = (item - head * row_tiles) * RT;
        const int rows = min(RT, R - row0);
        const int64_t first = at - tile;
        const int stop = (int)min((int64_t)nt, tile + (range.end - at));
        const int n = stop - tile;                    // tiles of this part
        const int tree = nt - 1 - tile;               // the tree's place among them, or >= n
        if (P.status && tid == 0 && tile == 0 && __ldg(P.ctx_len + b) != ctx)
            P.status[b] = SPEC_REQ_BAD_SLOT;

        // Q into shared memory
        for (int i = tid; i < RT * (D / 8); i += C_::kThreads) {
            const int r = i / (D / 8), j = i - r * (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int rr = row0 + r, node = rr / P.G;
                v = load8(reinterpret_cast<const unsigned short *>(P.q) +
                              ((int64_t)b * P.N + node) * P.q_stride +
                              (int64_t)(head * P.G + rr - node * P.G) * D + j * 8,
                          vec);
            }
            *reinterpret_cast<uint4 *>(smem + (r >> 7) * C_::kOperand + chunk_at(r & 127, j)) = v;
        }
        fence_async_smem();
        if (tid == 0) W.odd = 0ull;
        __syncthreads();

        if (warp >= NT * 4 && warp < kMmaWarp) {
            // ---- convert ----
            const int t = tid - NT * 128;
            const int32_t *table = C.block_table + (int64_t)b * C.max_blocks;
            auto page = [&](int i) -> int {
                const int p = (tile + i) * kTile + t;
                return i < n && i < tree && p < ctx
                           ? __ldg(table + (uint32_t)p / (uint32_t)C.block_size)
                           : -1;
            };
            Row4<D> kr, vr;
            bool ok = false;
            auto fetch = [&](int i, int blk) {
                const int p = (tile + i) * kTile + t;
                ok = blk >= 0 && blk < C.num_blocks;
                const uint32_t row =
                    ok ? fp4_row(C, blk, p % (uint32_t)C.block_size, head) : 0u;
                if (i < n && i < tree && p < ctx && !ok && P.status)
                    P.status[b] = SPEC_REQ_BAD_SLOT;
                load_row<D>(C.k, C.k_sf, row, ok, kr);
                load_row<D>(C.v, C.v_sf, row, ok, vr);
            };
            int next = page(1);
            fetch(0, page(0));
            for (int i = 0; i < n; ++i) {
                const uint32_t c = done + i;
                const int st = c & 1;
                const uint32_t parity = ((c >> 1) & 1) ^ 1;
                char *ks = smem + C_::kK + st * C_::kOperand;
                char *vs = smem + C_::kV + st * C_::kOperand;
                if (i == tree) {
                    // the nodes' own rows, zeros up to 64; two threads a row
                    const int r = t >> 1;
                    if (!warp_wait(&W.k_free[st], parity, gave_up) ||
                        !warp_wait(&W.v_free[st], parity, gave_up))
                        break;
                    const int64_t row = (int64_t)b * P.N + min(r, P.N - 1);
                    const unsigned short *k =
                        reinterpret_cast<const unsigned short *>(P.k) + row * P.k_stride + head * D;
                    const unsigned short *v =
                        reinterpret_cast<const unsigned short *>(P.v) + row * P.v_stride + head * D;
                    for (int j = t & 1; j < D / 8; j += 2) {
                        uint4 a = make_uint4(0, 0, 0, 0), x = a;
                        if (r < P.N) {
                            a = load8(k + j * 8, vec);
                            x = load8(v + j * 8, vec);
                            uint32_t *w = reinterpret_cast<uint32_t *>(&x);
                            bool odd = false;
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
                            if (odd) atomicOr(&W.odd, 1ull << r);
                        }
                        *reinterpret_cast<uint4 *>(ks + chunk_at(r, j)) = a;
                        *reinterpret_cast<uint4 *>(vs + chunk_at(r, j)) = x;
                    }
                    fence_async_smem();
                    bar_arrive(&W.k_full[st]);
                    bar_arrive(&W.v_full[st]);
                    break;        // it is the last
                }
                const unsigned seen = __ballot_sync(0xffffffffu, ok);
                if (!warp_wait(&W.k_free[st], parity, gave_up)) break;
                if (lane == 0) W.seen[c & 3][t >> 5] = seen;
                convert_row<D, T == 1>(kr, ks, t);
                fence_async_smem();
                bar_arrive(&W.k_full[st]);
                if (!warp_wait(&W.v_free[st], parity, gave_up)) break;
                convert_row<D, false>(vr, vs, t);
                fence_async_smem();
                bar_arrive(&W.v_full[st]);
                const int cur = next;
                next = page(i + 2);
                fetch(i + 1, cur);
            }
        } else if (warp == kMmaWarp) {
            // ---- multiply ----
            if (lane == 0) {
                auto scores = [&](int m, int i) {
                    const uint32_t c = done + i;
                    const uint32_t a = base + m * C_::kOperand;
                    const uint32_t k = base + C_::kK + (c & 1) * C_::kOperand;
                    const uint32_t d = i == tree ? mma_desc(kType, 64, false)
                                                 : mma_desc(kType, 128, false);
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        const uint32_t off = (s >> 2) * (128 * 128) + (s & 3) * 32;
                        mma_ss(s_at(m), smem_desc(a + off, 16, 1024), smem_desc(k + off, 16, 1024),
                               d, s > 0);
                    }
                    mma_commit(&W.s_full[m]);
                };
                bool ok = bar_wait(&W.k_full[done & 1], (done >> 1) & 1, gave_up);
                tc_fence_after();
                if (ok) {
                    for (int m = 0; m < NT; ++m) scores(m, 0);
                    mma_commit(&W.k_free[done & 1]);
                }
                for (int i = 0; ok && i < n; ++i) {
                    const uint32_t c = done + i;
                    const uint32_t v = base + C_::kV + (c & 1) * C_::kOperand;
                    for (int m = 0; m < NT; ++m) {
                        if (m == 0) ok = bar_wait(&W.v_full[c & 1], (c >> 1) & 1, gave_up);
                        ok = ok && bar_wait(&W.p_full[m], c & 1, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        if (i == tree) {
                            // 64 nodes; bfloat16: the two terms of P, 64 columns apart
                            for (int part = 0; part < (T == 1 ? 2 : 1); ++part)
#pragma unroll
                                for (int s = 0; s < 4; ++s)
                                    mma_ts(o_at(m), s_at(m) + part * 64 + s * 8,
                                           smem_desc(v + s * 2048, 128 * 128, 1024),
                                           mma_desc(kType, D, true), i > 0 || part > 0 || s > 0);
                        } else {
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                mma_ts(o_at(m), s_at(m) + s * 8,
                                       smem_desc(v + s * 2048, 128 * 128, 1024),
                                       mma_desc(0, D, true), i > 0 || s > 0);
                        }
                        mma_commit(&W.o_full[m]);
                        if (m == NT - 1) mma_commit(&W.v_free[c & 1]);
                        if (i + 1 < n) {
                            const uint32_t d = c + 1;
                            if (m == 0) ok = bar_wait(&W.k_full[d & 1], (d >> 1) & 1, gave_up);
                            if (!ok) break;
                            tc_fence_after();
                            scores(m, i + 1);
                            if (m == NT - 1) mma_commit(&W.k_free[d & 1]);
                        }
                    }
                }
            }
        } else if (warp < NT * 4) {
            // ---- softmax: this thread's row ----
            const int m = warp >> 2, r = m * 128 + (warp & 3) * 32 + lane;
            const bool live = r < rows;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_tm = s_at(m) + lanes, o_tm = o_at(m) + lanes;
            float top = kNoMax, sum = 0.f;
            const unsigned long long mask =
                live ? __ldg(P.mask + (int64_t)b * P.N + (row0 + r) / P.G) &
                           (P.N < 64 ? (1ull << P.N) - 1ull : ~0ull)
                     : 0ull;
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                const uint32_t c = done + i;
                ok = warp_wait(&W.s_full[m], c & 1, gave_up);
                if (!ok) break;
                tc_fence_after();
                const bool is_tree = i == tree;
                unsigned see[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    see[q] = is_tree ? (q < 2 ? (unsigned)(mask >> (q * 32)) : 0u) : W.seen[c & 3][q];
                const bool all = (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu;
                const float f = is_tree ? unit : unit * k_scale;
                const int chunks = is_tree ? 2 : 4;
                auto scores = [&](int q, uint32_t (&s)[32]) {   // of 32 positions; -inf: not seen
                    tmem_ld32(s_tm + q * 32, s);
                    tmem_wait_ld(s);
                    if (!all) {
                        const unsigned w = q == 0 ? see[0] : q == 1 ? see[1] : q == 2 ? see[2] : see[3];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((w >> e) & 1)) s[e] = 0xff800000u;
                    }
                };
                float big = -INFINITY;
                for (int q = 0; q < chunks; ++q) {
                    uint32_t s[32];
                    scores(q, s);
#pragma unroll
                    for (int e = 0; e < 32; ++e) big = fmaxf(big, __uint_as_float(s[e]));
                }
                const float x = fmaxf(kNoMax, big * f);
                const bool raise = __any_sync(0xffffffffu, x > top + kRescale);
                const bool units = is_tree && i > 0;      // O leaves the cache's units
                if (raise || units) {
                    float a = 1.f;
                    if (raise) {
                        const float to = fmaxf(top, x);
                        a = ex2(top - to);
                        top = to;
                        sum *= a;
                    }
                    if (units) a *= v_scale;
                    if (i > 0) {
                        ok = warp_wait(&W.o_full[m], (c - 1) & 1, gave_up);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t o[32];
                            tmem_ld32(o_tm + q * 32, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tmem_st32(o_tm + q * 32, o);
                        }
                    }
                }
                // P over the scores that have been read: chunk q's 16 columns lie in chunk q / 2
                for (int q = 0; q < chunks; ++q) {
                    uint32_t s[32], p[16];
                    scores(q, s);
                    float l = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float p0 = ex2(fmaf(__uint_as_float(s[e]), f, -top));
                        const float p1 = ex2(fmaf(__uint_as_float(s[e + 1]), f, -top));
                        l += p0 + p1;
                        s[e] = __float_as_uint(p0);
                        s[e + 1] = __float_as_uint(p1);
                    }
                    sum += l;
                    if (!is_tree) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            p[e] = pack2<2>(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                        tmem_st16(s_tm + q * 16, p);
                    } else {
                        // the nodes' P in their type; what bfloat16 leaves in a second term,
                        // behind the 64 columns of scores
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            p[e] = pack2<T>(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                            if (T == 1)
                                s[e] = pack2<1>(__uint_as_float(s[2 * e]) - bf_lo(p[e]),
                                                __uint_as_float(s[2 * e + 1]) - bf_hi(p[e]));
                        }
                        tmem_st16(s_tm + q * 16, p);
                        if (T == 1) tmem_st16(s_tm + 64 + q * 16, s);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                bar_arrive(&W.p_full[m]);
            }
            // the result: O is done after the last tile's product
            ok = ok && warp_wait(&W.o_full[m], (done + n - 1) & 1, gave_up);
            tc_fence_after();
            const bool whole = tile == 0 && stop == nt;
            const float in_cache = tree < n ? 1.f : v_scale;
            const float norm = in_cache * (whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f);
            const int64_t to = live ? attn_row(P, b, head, row0 + r) : 0;
            float *part = attn_slot(P, blockIdx.x, tile == 0, RT, D);
            const unsigned long long odd = tree < n ? W.odd & mask : 0ull;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(o_tm + q * 32, o);
                tmem_wait_ld(o);
                if (!live || !ok) continue;
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * norm;
                // NaN and infinities of nodes that this row sees
                for (unsigned long long left = odd; left; left &= left - 1) {
                    const int j = __ffsll(left) - 1;
                    const unsigned short *qp =
                        reinterpret_cast<const unsigned short *>(P.q) +
                        ((int64_t)b * P.N + (row0 + r) / P.G) * P.q_stride +
                        (int64_t)(head * P.G + (row0 + r) % P.G) * D;
                    const unsigned short *kp = reinterpret_cast<const unsigned short *>(P.k) +
                                               ((int64_t)b * P.N + j) * P.k_stride + head * D;
                    const unsigned short *vp = reinterpret_cast<const unsigned short *>(P.v) +
                                               ((int64_t)b * P.N + j) * P.v_stride + head * D;
                    float dot = 0.f;
                    for (int d = 0; d < D; ++d)
                        dot = fmaf(value16<T>(__ldg(qp + d)), value16<T>(__ldg(kp + d)), dot);
                    const float w = ex2(dot * unit - top);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t y = __ldg(vp + q * 32 + e);
                        if (odd16<T>(y)) v[e] += w * value16<T>(y);
                    }
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        store_out4<T>(P.out, to * D + q * 32 + e,
                                      make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(part + (int64_t)r * D + q * 32 + e) =
                            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
            }
            if (live && ok) {
                if (whole) {
                    if (P.lse) P.lse[to] = attn_lse(top, sum);
                } else {
                    part[RT * D + r] = top;
                    part[RT * (D + 1) + r] = sum;
                }
            }
            tc_fence_before();
        }
        __syncthreads();
        if (*gave_up) {
            if (P.status && tid == 0) P.status[b] = SPEC_REQ_INTERNAL;
            break;
        }
        if (!(tile == 0 && stop == nt))
            attn_join<T, D>(P, range, first, nt, b, head, row0, rows, RT, &W.flag);
        __syncthreads();      // Q and the words are free for the next item
        done += n;
        at += stop - tile;
        tile = 0;
        if (++item == C.H * row_tiles) {
            item = 0;
            ++b;
        }
    }
    // every product has been waited for, unless a wait gave up: then those in flight are, for
    // as long as they can take
    if (warp == kMmaWarp && lane == 0 && *gave_up) {
        mma_commit(&W.drain);
        for (int i = 0; i < (1 << 20) && !bar_try(&W.drain, 0); ++i) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, C_::kColumns);
}

template <int T, int D, int NT>
cudaError_t launch(const TreeAttnParams &p, int grid, cudaStream_t st) {
    using C_ = Tc<D, NT>;
    const cudaError_t e = cudaFuncSetAttribute(tree_attn_tc_kernel<T, D, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C_::kBytes);
    if (e != cudaSuccess) return e;
    const int row_tiles = (p.N * p.G + NT * 128 - 1) / (NT * 128);
    auto vec16 = [](const void *q, int64_t stride) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride % 8 == 0;
    };
    const int vec = vec16(p.q, p.q_stride) && vec16(p.k, p.k_stride) && vec16(p.v, p.v_stride);
    tree_attn_tc_kernel<T, D, NT><<<grid, C_::kThreads, C_::kBytes, st>>>(p, row_tiles, vec);
    return cudaGetLastError();
}

}  // namespace

// Row tiles of 128 that a CTA takes at a time.
int tree_attn_tc_tiles(int R) { return R > 128 ? 2 : 1; }

cudaError_t launch_tree_attn_tc(const TreeAttnParams &p, int grid, cudaStream_t st) {
    const bool two = tree_attn_tc_tiles(p.N * p.G) == 2;
    if (p.cache.D == 64) {
        if (p.dtype == 1) return two ? launch<1, 64, 2>(p, grid, st) : launch<1, 64, 1>(p, grid, st);
        return two ? launch<2, 64, 2>(p, grid, st) : launch<2, 64, 1>(p, grid, st);
    }
    if (p.dtype == 1) return two ? launch<1, 128, 2>(p, grid, st) : launch<1, 128, 1>(p, grid, st);
    return two ? launch<2, 128, 2>(p, grid, st) : launch<2, 128, 1>(p, grid, st);
}

}  // namespace specv
