// Tree attention over the 4-bit paged cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(x_ij - m_i),  x_ij = log2(e) scale q_i.k_j,
// over the context positions and the nodes that node i may see; m_i is a running maximum.
// The rows of an item are the N nodes times the G query heads that share one K/V head, so K and
// V are read once for all of them: 0.5625 bytes an element. With few rows DRAM should bound it;
// what stands in the way is the conversion of the codes, about 2.5 instructions for two
// elements, and the products.
//
// A code times its block scale has at most six significant bits and lies in [2^-10, 2688], so
// it is exact as a half; the tensor scales are applied to the scores and to the result. Q is
// brought to halves by a power of two for each row (exact for what is within 2^-32 of the row's
// largest element) and p is rounded to a half with the row's largest near 1. The products are
// m16n8k16 of halves with float32 sums.
//
// A CTA is four warps; each takes 32 of a tile's 128 positions and keeps its own maxima, sums
// and output in registers, so that the main loop has no barrier. Codes and scales come through
// a ring in shared memory by asynchronous copies. Both products contract over
// an index whose order is free: the head's elements for K, the positions for V. So lane (g, c)
// takes the elements [c D/4, (c+1) D/4) of position g as its share of the K operand, one wide
// load, and the elements [g D/8, (g+1) D/8) of its four positions for V, whose pairs of
// positions are put together by a byte permute. The positions of a group of eight are taken in
// the order 0 1 3 2 4 5 7 6, which with the swizzle of 16-byte units makes both loads free of
// bank conflicts.

#include "tree_attn.cuh"

namespace specv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Tiles in the ring: the one at work and those in flight (two warps' worth of D = 256 take the
// shared memory of three of D = 128).
constexpr int stages(int D) { return D == 256 ? 2 : 3; }
constexpr int kTreeCost = 1;      // the tree's tile and an item's rest, in context tiles
constexpr float kRescale = 8.f;   // a maximum is followed once it rises by 2^8

template <int D>
struct Ring {
    static constexpr int kStages = stages(D);
    static constexpr int kCodes = 32 * D / 2;             // bytes of K (and of V) codes
    static constexpr int kScales = 32 * D / 16;
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kScales, kSeen = kVs + kScales;
    static constexpr int kBytes = kSeen + 16;
};

// Shared memory of a CTA, in bytes from its start.
template <int T, int D, int MT>
struct Smem {
    static constexpr int kRows = 16 * MT;
    static constexpr int kRing = kWarps * stages(D) * Ring<D>::kBytes;
    static constexpr int kTreeStride = D + 8;                              // elements
    static constexpr int kTree = 2 * kMaxN * kTreeStride * 2;              // in the ring's place
    static constexpr int kJoin = kRows * D * 4;                            // likewise
    static constexpr int kFirst = kRing > kTree ? kRing : kTree;
    static constexpr int kQ = kFirst > kJoin ? kFirst : kJoin;
    static constexpr int kQt = kQ + kRows * D * 2;                         // Q in its own type
    static constexpr int kFac = kQt + (T == 1 ? kRows * D * 2 : 0);
    static constexpr int kM = kFac + kRows * 4;
    static constexpr int kL = kM + kWarps * kRows * 4;
    static constexpr int kOdd = kL + kWarps * kRows * 4;
    static constexpr int kBytes = kOdd + 16;
};

// 16-byte unit u of position t's codes lies at unit swizzle(t, u).
template <int D>
__device__ __forceinline__ int swizzle(int t, int u) {
    if (D == 128) return u ^ ((t >> 1) & 3);
    if (D == 256) return u ^ (t & 7);
    return u;
}

template <int T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (T == 2)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
    return __byte_perm(a, b, s);
}

// Copies of `n` bytes (8 or 16) to shared memory; zeros when !ok.
template <int n>
__device__ __forceinline__ void cp_async(uint32_t smem, const void *gmem, bool ok) {
    const int size = ok ? n : 0;
    if constexpr (n == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem),
                     "r"(size)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem), "l"(gmem),
                     "r"(size), "n"(n)
                     : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int n>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float half_bits(uint32_t h) {
    return __half2float(__ushort_as_half((unsigned short)h));
}

// The state of an item in one warp: rows g and g + 8 of each of its MT groups of 16.
template <int D, int MT>
struct Acc {
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];   // l: this lane's share of the row sums

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
            m[i][0] = m[i][1] = kNoMax;
            l[i][0] = l[i][1] = 0.f;
        }
    }
    // Takes new row maxima in: rescales when one has risen far enough (for the whole warp).
    __device__ __forceinline__ void raise(float (&x)[MT][2]) {
        bool up = false;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                x[i][r] = fmaxf(x[i][r], __shfl_xor_sync(0xffffffffu, x[i][r], 1));
                x[i][r] = fmaxf(x[i][r], __shfl_xor_sync(0xffffffffu, x[i][r], 2));
                up |= x[i][r] > m[i][r] + kRescale;
            }
        if (!__any_sync(0xffffffffu, up)) return;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float a[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float to = fmaxf(m[i][r], x[i][r]);
                a[r] = ex2(m[i][r] - to);
                m[i][r] = to;
                l[i][r] *= a[r];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] *= a[e >> 1];
        }
    }
};

// T: 1 bf16, 2 f16; MT: groups of 16 query rows of an item.
template <int T, int D, int MT>
__global__ void __launch_bounds__(kThreads, MT == 2 || D == 256 ? 2 : 3)
    tree_attn_kernel(TreeAttnParams P, int row_tiles) {
    using S = Smem<T, D, MT>;
    using Rg = Ring<D>;
    constexpr int RT = S::kRows, KS = D / 16, kStages = Rg::kStages;
    extern __shared__ __align__(128) char smem[];
    const spec_fp4_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int pg = g ^ ((g >> 1) & 1);                 // position of the g-th column of eight
    const int pt0 = 2 * c + (c & 1), pt1 = 2 * c + 1 - (c & 1);   // ... of columns 2c, 2c + 1
    const int R = P.N * P.G;
    float *s_fac = reinterpret_cast<float *>(smem + S::kFac);
    float *s_m = reinterpret_cast<float *>(smem + S::kM);
    float *s_l = reinterpret_cast<float *>(smem + S::kL);
    unsigned long long *s_odd = reinterpret_cast<unsigned long long *>(smem + S::kOdd);
    char *ring = smem + warp * kStages * Rg::kBytes;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const float k_scale = C.k_scale ? __ldg(C.k_scale) : 1.f;
    const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
    const float unit = P.scale * kLog2e;

    AttnWalk walk(P, C.H * row_tiles, kTreeCost);
    AttnPart A;
    bool any = false;
    Acc<D, MT> acc;

    while (walk.next(P, A)) {
        const int b = A.b, ctx = A.ctx, tile = A.tile;
        const int head = A.item / row_tiles, row0 = (A.item - head * row_tiles) * RT;
        const int rows = min(RT, R - row0);
        const int n = min(A.stop, A.nt - 1) - tile;    // context tiles of this CTA's part
        if (P.status && tid == 0 && tile == 0 && __ldg(P.ctx_len + b) != ctx)
            P.status[b] = SPEC_REQ_BAD_SLOT;
        const int32_t *table = C.block_table + (int64_t)b * C.max_blocks;

        // The block of this lane's position in the part's i-th tile; -1 past the context.
        auto page = [&](int i) -> int {
            const int p = (tile + i) * kTile + warp * 32 + lane;
            return i < n && p < ctx ? __ldg(table + (uint32_t)p / (uint32_t)C.block_size) : -1;
        };
        // Starts the copies of the i-th tile into its ring place.
        auto issue = [&](int i, int blk) {
            if (i < n) {
                const uint32_t st = ring_s + (uint32_t)(i % kStages) * Rg::kBytes;
                const int p = (tile + i) * kTile + warp * 32 + lane;
                const bool ok = blk >= 0 && blk < C.num_blocks;
                const uint32_t row =
                    ok ? fp4_row(C, blk, p % (uint32_t)C.block_size, head) : 0u;
                if (p < ctx && !ok && P.status) P.status[b] = SPEC_REQ_BAD_SLOT;
                const unsigned seen = __ballot_sync(0xffffffffu, ok);
                if (lane == 0)
                    *reinterpret_cast<unsigned *>(ring + (i % kStages) * Rg::kBytes + Rg::kSeen) =
                        seen;
                constexpr int U = D / 32;              // 16-byte units of a position's codes
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int t = (q * 32 + lane) / U, u = lane % U;
                    const uint32_t r = __shfl_sync(0xffffffffu, row, t);
                    const bool o = (seen >> t) & 1;
                    const int64_t src = (int64_t)r * (D / 2) + u * 16;
                    const uint32_t dst = st + t * (D / 2) + swizzle<D>(t, u) * 16;
                    cp_async<16>(dst, reinterpret_cast<const char *>(C.k) + src, o);
                    cp_async<16>(dst + Rg::kV, reinterpret_cast<const char *>(C.v) + src, o);
                }
                const int64_t src = (int64_t)row * (D / 16);
                cp_async<D / 16>(st + Rg::kKs + lane * (D / 16),
                                 reinterpret_cast<const char *>(C.k_sf) + src, ok);
                cp_async<D / 16>(st + Rg::kVs + lane * (D / 16),
                                 reinterpret_cast<const char *>(C.v_sf) + src, ok);
            }
            cp_async_commit();
        };

        int next = page(0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int cur = next;
            next = page(i + 1);
            issue(i, cur);
        }

        // Q, in the order of the products' operands: row r of 16, element d belongs to lane
        // (r % 8, d / (D/4)), step (d % (D/4)) / 4.
        for (int r = warp; r < RT; r += kWarps) {
            constexpr int E = D / 32;                  // elements of a lane, neighbours
            const bool live = r < rows;
            const int rr = live ? row0 + r : 0, node = rr / P.G;
            const unsigned short *q =
                reinterpret_cast<const unsigned short *>(P.q) +
                ((int64_t)b * P.N + node) * P.q_stride +
                (int64_t)(head * P.G + rr - node * P.G) * D + lane * E;
            unsigned short raw[E];
            float x[E], big = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                raw[e] = live ? __ldg(q + e) : (unsigned short)0;
                x[e] = T == 1 ? __uint_as_float((uint32_t)raw[e] << 16) : half_bits(raw[e]);
                const float a = fabsf(x[e]);
                if (a < INFINITY) big = fmaxf(big, a);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
            // 2^k brings the largest into [2^14, 2^15); a row of zeros is left alone
            const int ex = big > 0.f ? ilogbf(big) : 14;
            const float up = ldexpf(1.f, max(-126, min(127, 14 - ex)));
            const int step0 = (lane * E % (D / 4)) / 4, cc = lane * E / (D / 4);
            char *q16 = smem + S::kQ, *qt = smem + S::kQt;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const int in = lane * E % (D / 4) + e;   // element within the lane's quarter
                const int reg = ((in & 2) ? 2 : 0) + ((r & 8) ? 1 : 0);
                const int off = (((r / 16) * KS + (E >= 4 ? step0 + e / 4 : in / 4)) * 32 +
                                 (r % 8) * 4 + cc) * 16 + reg * 4;
                *reinterpret_cast<uint32_t *>(q16 + off) = f16x2(x[e] * up, x[e + 1] * up);
                if (T == 1)
                    *reinterpret_cast<uint32_t *>(qt + off) =
                        (uint32_t)raw[e] | (uint32_t)raw[e + 1] << 16;
            }
            if (lane == 0) s_fac[r] = unit / up;
        }
        __syncthreads();

        float fac[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) fac[i][r] = s_fac[i * 16 + g + r * 8];
        constexpr bool kQRegs = MT == 1 && D <= 128;
        uint32_t qf[kQRegs ? KS : 1][4];
        auto q_frag = [&](const char *base, int i, int kk, uint32_t (&a)[4]) {
            const uint4 v = *reinterpret_cast<const uint4 *>(base + ((i * KS + kk) * 32 + lane) * 16);
            a[0] = v.x;
            a[1] = v.y;
            a[2] = v.z;
            a[3] = v.w;
        };
        if (kQRegs) {
#pragma unroll
            for (int kk = 0; kk < (kQRegs ? KS : 1); ++kk) q_frag(smem + S::kQ, 0, kk, qf[kk]);
        }
        acc.clear();

        for (int i = 0; i < n; ++i) {
            cp_async_wait<kStages - 2>();
            __syncwarp();     // everyone's copies are in, and the place refilled next is free
            {
                const int cur = next;
                next = page(i + kStages);
                issue(i + kStages - 1, cur);
            }
            const char *st = ring + (i % kStages) * Rg::kBytes;
            const unsigned seen = *reinterpret_cast<const unsigned *>(st + Rg::kSeen);
            float s[MT][4][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][j][e] = 0.f;
            // scores: the elements of eight codes (a word) at a time, for all 32 positions
            constexpr int KW = D / 32;                 // words of a lane's share of a position
            uint32_t kw[4][KW], ks[4][KW / 2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 8 * j + pg;
                if constexpr (D == 64) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(st + t * 32 + c * 8);
                    kw[j][0] = v.x;
                    kw[j][1] = v.y;
                    ks[j][0] = e4m3x2_to_f16x2(
                        *reinterpret_cast<const uint8_t *>(st + Rg::kKs + t * 4 + c));
                } else {
#pragma unroll
                    for (int q = 0; q < KW / 4; ++q) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            st + t * (D / 2) + swizzle<D>(t, c * (KW / 4) + q) * 16);
                        kw[j][q * 4] = v.x;
                        kw[j][q * 4 + 1] = v.y;
                        kw[j][q * 4 + 2] = v.z;
                        kw[j][q * 4 + 3] = v.w;
                    }
#pragma unroll
                    for (int q = 0; q < KW / 4; ++q) {
                        const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(
                            st + Rg::kKs + t * (D / 16) + c * (D / 64) + q * 2));
                        ks[j][2 * q] = two;
                        ks[j][2 * q + 1] = prmt(two, two, 0x3232);
                    }
                }
#pragma unroll
                for (int q = 0; q < KW / 2; q += D == 64 ? 1 : 2)
                    ks[j][q] = prmt(ks[j][q], ks[j][q], 0x1010);
            }
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t a[MT][2][4];
                if (!kQRegs) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int q = 0; q < 2; ++q) q_frag(smem + S::kQ, mt, 2 * w + q, a[mt][q]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t r[4];
                    e2m1x8_to_f16x2(kw[j][w], r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = hmul2(r[e], ks[j][w / 2]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (kQRegs) {
                            mma<2>(s[mt][j], qf[2 * w], r[0], r[1]);
                            mma<2>(s[mt][j], qf[2 * w + 1], r[2], r[3]);
                        } else {
                            mma<2>(s[mt][j], a[mt][0], r[0], r[1]);
                            mma<2>(s[mt][j], a[mt][1], r[2], r[3]);
                        }
                    }
                }
            }
            float top[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                top[mt][0] = top[mt][1] = kNoMax;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[mt][j][e] * (fac[mt][e >> 1] * k_scale);
                        if (seen != 0xffffffffu && !((seen >> (8 * j + ((e & 1) ? pt1 : pt0))) & 1))
                            x = -INFINITY;
                        s[mt][j][e] = x;
                        top[mt][e >> 1] = fmaxf(top[mt][e >> 1], x);
                    }
            }
            acc.raise(top);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = ex2(s[mt][j][e] - acc.m[mt][e >> 1]);
                        s[mt][j][e] = p;
                        acc.l[mt][e >> 1] += p;
                    }
            // values: two groups of 16 positions
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    a[mt][0] = f16x2(s[mt][2 * h][0], s[mt][2 * h][1]);
                    a[mt][1] = f16x2(s[mt][2 * h][2], s[mt][2 * h][3]);
                    a[mt][2] = f16x2(s[mt][2 * h + 1][0], s[mt][2 * h + 1][1]);
                    a[mt][3] = f16x2(s[mt][2 * h + 1][2], s[mt][2 * h + 1][3]);
                }
                const int ts[4] = {16 * h + pt0, 16 * h + pt1, 16 * h + 8 + pt0, 16 * h + 8 + pt1};
                constexpr int VW = D / 64;             // words of a lane's share of a position
                constexpr int VG = D == 256 ? 2 : 1;   // block scales of that share
                uint32_t vw[4][VW], sab[VG], scd[VG];
                uint32_t sc[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const char *v = st + Rg::kV + ts[q] * (D / 2);
                    const char *f = st + Rg::kVs + ts[q] * (D / 16);
                    if constexpr (D == 64) {
                        vw[q][0] = *reinterpret_cast<const uint32_t *>(v + g * 4);
                        sc[q] = *reinterpret_cast<const uint8_t *>(f + g / 2);
                    } else if constexpr (D == 128) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(
                            v + swizzle<D>(ts[q], g >> 1) * 16 + (g & 1) * 8);
                        vw[q][0] = w.x;
                        vw[q][1] = w.y;
                        sc[q] = *reinterpret_cast<const uint8_t *>(f + g);
                    } else {
                        const uint4 w =
                            *reinterpret_cast<const uint4 *>(v + swizzle<D>(ts[q], g) * 16);
                        vw[q][0] = w.x;
                        vw[q][1] = w.y;
                        vw[q][2] = w.z;
                        vw[q][3] = w.w;
                        sc[q] = *reinterpret_cast<const uint16_t *>(f + g * 2);
                    }
                }
                if constexpr (VG == 1) {
                    sab[0] = e4m3x2_to_f16x2(sc[0] | sc[1] << 8);
                    scd[0] = e4m3x2_to_f16x2(sc[2] | sc[3] << 8);
                } else {
                    sab[0] = e4m3x2_to_f16x2((sc[0] & 0xff) | (sc[1] & 0xff) << 8);
                    scd[0] = e4m3x2_to_f16x2((sc[2] & 0xff) | (sc[3] & 0xff) << 8);
                    sab[1] = e4m3x2_to_f16x2(sc[0] >> 8 | (sc[1] >> 8) << 8);
                    scd[1] = e4m3x2_to_f16x2(sc[2] >> 8 | (sc[3] >> 8) << 8);
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    uint32_t va[4], vb[4], vc[4], vd[4];
                    e2m1x8_to_f16x2(vw[0][w], va);
                    e2m1x8_to_f16x2(vw[1][w], vb);
                    e2m1x8_to_f16x2(vw[2][w], vc);
                    e2m1x8_to_f16x2(vw[3][w], vd);
                    const uint32_t f0 = sab[w / 2], f1 = scd[w / 2];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t sel = e ? 0x7632 : 0x5410;
                            const uint32_t b0 = hmul2(prmt(va[y], vb[y], sel), f0);
                            const uint32_t b1 = hmul2(prmt(vc[y], vd[y], sel), f1);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma<2>(acc.o[mt][8 * w + 2 * y + e], a[mt], b0, b1);
                        }
                }
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.o[mt][j][e] *= v_scale;
        __syncthreads();      // the ring is free

        if (A.stop == A.nt) {
            // The tree's own nodes: their rows in shared memory, 16 nodes a warp.
            unsigned short *tk = reinterpret_cast<unsigned short *>(smem);
            unsigned short *tv = tk + kMaxN * S::kTreeStride;
            if (tid == 0) *s_odd = 0ull;
            __syncthreads();
            const int keys = min(kMaxN, (P.N + 15) / 16 * 16);
            for (int i = tid; i < keys * (D / 2); i += kThreads) {
                const int t = i / (D / 2), d = (i - t * (D / 2)) * 2;
                uint32_t kv[2] = {0, 0};
                if (t < P.N) {
                    const int64_t row = (int64_t)b * P.N + t;
                    const unsigned short *k = reinterpret_cast<const unsigned short *>(P.k) +
                                              row * P.k_stride + head * D + d;
                    const unsigned short *v = reinterpret_cast<const unsigned short *>(P.v) +
                                              row * P.v_stride + head * D + d;
                    kv[0] = (uint32_t)__ldg(k) | (uint32_t)__ldg(k + 1) << 16;
                    kv[1] = (uint32_t)__ldg(v) | (uint32_t)__ldg(v + 1) << 16;
                    // NaN and infinities in V are left out of the products
                    constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
                    if ((kv[1] & ex) == ex || (kv[1] >> 16 & ex) == ex)
                        atomicOr(s_odd, 1ull << t);
                }
                *reinterpret_cast<uint32_t *>(tk + t * S::kTreeStride + d) = kv[0];
                *reinterpret_cast<uint32_t *>(tv + t * S::kTreeStride + d) = kv[1];
            }
            __syncthreads();
            const int key0 = warp * 16;
            if (key0 < P.N) {
                const unsigned odd = (unsigned)(*s_odd >> key0) & 0xffffu;
                unsigned bits[MT][2];
                float s[MT][2][4], top[MT][2];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int rr = mt * 16 + g + r * 8;
                        bits[mt][r] =
                            rr < rows ? (unsigned)(__ldg(P.mask + (int64_t)b * P.N +
                                                         (row0 + rr) / P.G) >> key0) &
                                            (P.N - key0 >= 16 ? 0xffffu : (1u << (P.N - key0)) - 1u)
                                      : 0u;
                        top[mt][r] = kNoMax;
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][r][e] = 0.f;
                    }
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint32_t a[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        q_frag(smem + (T == 1 ? S::kQt : S::kQ), mt, kk, a[mt]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint2 kv = *reinterpret_cast<const uint2 *>(
                            tk + (key0 + 8 * j + g) * S::kTreeStride + c * (D / 4) + 4 * kk);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma<T>(s[mt][j], a[mt], kv.x, kv.y);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f = T == 1 ? unit : fac[mt][e >> 1];
                            const bool on = (bits[mt][e >> 1] >> (8 * j + 2 * c + (e & 1))) & 1;
                            s[mt][j][e] = on ? s[mt][j][e] * f : -INFINITY;
                            top[mt][e >> 1] = fmaxf(top[mt][e >> 1], s[mt][j][e]);
                        }
                acc.raise(top);
                uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = ex2(s[mt][j][e] - acc.m[mt][e >> 1]);
                            s[mt][j][e] = p;
                            acc.l[mt][e >> 1] += p;
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float p0 = s[mt][j][2 * r], p1 = s[mt][j][2 * r + 1];
                            if (T == 2) {
                                hi[mt][2 * j + r] = f16x2(p0, p1);
                            } else {
                                // eight bits are too few for p: a second product has the rest
                                const uint32_t w = bf16x2(p0, p1);
                                hi[mt][2 * j + r] = w;
                                lo[mt][2 * j + r] = bf16x2(p0 - bf_lo(w), p1 - bf_hi(w));
                            }
                        }
                    }
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const unsigned short *v = tv + g * (D / 8) + j;
                    uint32_t w[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int t = 2 * c + 8 * q;
                        uint32_t x = v[(key0 + t) * S::kTreeStride];
                        uint32_t y = v[(key0 + t + 1) * S::kTreeStride];
                        if (odd) {
                            constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
                            if ((x & ex) == ex) x = 0;
                            if ((y & ex) == ex) y = 0;
                        }
                        w[q] = x | y << 16;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma<T>(acc.o[mt][j], hi[mt], w[0], w[1]);
                        if (T == 1) mma<T>(acc.o[mt][j], lo[mt], w[0], w[1]);
                    }
                }
                // nodes with NaN or infinities in V: only for the rows that see them
                if (odd) {
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        if (!((odd >> t) & 1)) continue;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float p = __shfl_sync(
                                    0xffffffffu, s[mt][t >> 3][2 * r + (t & 1)],
                                    (lane & ~3) | ((t >> 1) & 3));
                                if (!((bits[mt][r] >> t) & 1)) continue;
#pragma unroll
                                for (int j = 0; j < D / 8; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const uint32_t x =
                                            tv[(key0 + t) * S::kTreeStride + (2 * c + e) * (D / 8) + j];
                                        constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
                                        if ((x & ex) == ex)
                                            acc.o[mt][j][2 * r + e] +=
                                                p * (T == 1 ? __uint_as_float(x << 16) : half_bits(x));
                                    }
                            }
                    }
                }
            }
            __syncthreads();
        }

        // The four warps' states become one.
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = acc.l[mt][r];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (c == 0) {
                    s_m[warp * RT + mt * 16 + g + 8 * r] = acc.m[mt][r];
                    s_l[warp * RT + mt * 16 + g + 8 * r] = l;
                }
            }
        __syncthreads();
        float4 *join = reinterpret_cast<float4 *>(smem);   // [D/16][RT][4]: row r, quarter c
        float f[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int rr = mt * 16 + g + 8 * r;
                float m = s_m[rr];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_m[w * RT + rr]);
                f[mt][r] = exp2f(acc.m[mt][r] - m);
            }
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int q = 0; q < D / 16; ++q) {
                            // columns 2c + e of all the products: elements (2c + e) D/8 + j
                            const int e = q / (D / 32), j = (q % (D / 32)) * 4;
                            float4 v = make_float4(
                                acc.o[mt][j][2 * r + e] * f[mt][r], acc.o[mt][j + 1][2 * r + e] * f[mt][r],
                                acc.o[mt][j + 2][2 * r + e] * f[mt][r], acc.o[mt][j + 3][2 * r + e] * f[mt][r]);
                            float4 &to = join[(q * RT + mt * 16 + g + 8 * r) * 4 + c];
                            if (w > 0) {
                                const float4 o = to;
                                v.x += o.x;
                                v.y += o.y;
                                v.z += o.z;
                                v.w += o.w;
                            }
                            to = v;
                        }
            }
            __syncthreads();
        }
        const bool whole = tile == 0 && A.stop == A.nt;
        float *part = attn_slot(P, blockIdx.x, tile == 0, RT, D);
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d4 = i - r * (D / 4), cc = d4 / (D / 16), q = d4 % (D / 16);
            const float4 v = join[(q * RT + r) * 4 + cc];
            float m = s_m[r], l = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_m[w * RT + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) l += s_l[w * RT + r] * exp2f(s_m[w * RT + r] - m);
            if (whole) {
                const float n1 = l == 0.f ? 0.f : 1.f / l;
                const int64_t to = attn_row(P, b, head, row0 + r);
                store_out4<T>(P.out, to * D + d4 * 4,
                              make_float4(v.x * n1, v.y * n1, v.z * n1, v.w * n1));
                if (P.lse && d4 == 0) P.lse[to] = attn_lse(m, l);
            } else {
                reinterpret_cast<float4 *>(part + r * D)[d4] = v;
                if (d4 == 0) {
                    part[RT * D + r] = m;
                    part[RT * (D + 1) + r] = l;
                }
            }
        }
        __syncthreads();      // shared memory is free for the next item
        any = true;
    }
    if (tid == 0) attn_note(P, walk.r, A, any);
}

// The parts of cut items into the result: a CTA has 256 float4s of an item's rows, a thread one
// of each part, eight parts' loads in flight together.
constexpr int kJoinThreads = 256;
template <int T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(TreeAttnParams P, int rows_tile) {
    grid_dep_wait();
    const int c0 = blockIdx.y;
    const int4 note = P.notes[c0];
    if (note.x < 0) return;
    const int b = note.x, c1 = note.z, row_tiles = (P.N * P.G + rows_tile - 1) / rows_tile;
    const int head = note.y / row_tiles, row0 = (note.y - head * row_tiles) * rows_tile;
    const int rows = min(rows_tile, P.N * P.G - row0);
    const int i = blockIdx.x * kJoinThreads + threadIdx.x, r = i / (D / 4), d4 = i - r * (D / 4);
    if (r >= rows) return;
    float m = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; c += 8) {
        float4 v[8];
        float pm[8], pl[8], top = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            pm[u] = kNoMax;
            if (c + u > c1) continue;
            const float *part = attn_slot(P, c + u, c + u == c0, rows_tile, D);
            v[u] = __ldcg(reinterpret_cast<const float4 *>(part) + i);
            pm[u] = __ldcg(part + rows_tile * D + r);
            pl[u] = __ldcg(part + rows_tile * (D + 1) + r);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) top = fmaxf(top, pm[u]);
        const float a = ex2(m - top);
        m = top;
        l *= a;
        o.x *= a;
        o.y *= a;
        o.z *= a;
        o.w *= a;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (c + u > c1) continue;
            const float w = ex2(pm[u] - top);
            o.x = fmaf(v[u].x, w, o.x);
            o.y = fmaf(v[u].y, w, o.y);
            o.z = fmaf(v[u].z, w, o.z);
            o.w = fmaf(v[u].w, w, o.w);
            l = fmaf(pl[u], w, l);
        }
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = attn_row(P, b, head, row0 + r);
    store_out4<T>(P.out, at * D + d4 * 4, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
    if (P.lse && d4 == 0) P.lse[at] = attn_lse(m, l);
}

// How a call is run: by this file's warps (groups of 16 rows of an item, CTAs an SM holds), or,
// with more rows than two groups, on the tcgen05 tensor cores.
struct Plan {
    bool tc;
    int groups, rows, grid;   // rows of an item
};
Plan plan(int R, int D, int sms) {
    Plan p;
    p.tc = R > 32 && D <= 128;
    p.groups = R > 16 && D <= 128 ? 2 : 1;
    p.rows = p.tc ? tree_attn_tc_rows(R) : 16 * p.groups;
    p.grid = sms * (p.tc ? 1 : p.groups == 2 || D == 256 ? 2 : 3);
    return p;
}

template <int T, int D, int MT>
cudaError_t launch(const TreeAttnParams &p, int grid, cudaStream_t st) {
    const int smem = Smem<T, D, MT>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<T, D, MT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int row_tiles = (p.N * p.G + 16 * MT - 1) / (16 * MT);
    tree_attn_kernel<T, D, MT><<<grid, kThreads, smem, st>>>(p, row_tiles);
    return cudaGetLastError();
}

template <int T>
cudaError_t launch_type(const TreeAttnParams &p, const Plan &n, cudaStream_t st) {
    const int D = p.cache.D;
    if (D == 256) return launch<T, 256, 1>(p, n.grid, st);
    if (n.groups == 2)
        return D == 64 ? launch<T, 64, 2>(p, n.grid, st) : launch<T, 128, 2>(p, n.grid, st);
    return D == 64 ? launch<T, 64, 1>(p, n.grid, st) : launch<T, 128, 1>(p, n.grid, st);
}

}  // namespace

namespace {

int64_t notes_bytes(const Plan &n) { return ((int64_t)n.grid * sizeof(int4) + 255) / 256 * 256; }

template <int T, int D>
cudaError_t launch_join(const TreeAttnParams &p, const Plan &n, cudaStream_t st) {
    const dim3 grid((n.rows * (D / 4) + kJoinThreads - 1) / kJoinThreads, n.grid);
    return launch_dependent(join_kernel<T, D>, grid, dim3(kJoinThreads), 0, st, p, n.rows);
}

}  // namespace

int64_t tree_attn_workspace(int R, int D, int sms) {
    const Plan n = plan(R, D, sms);
    const int64_t bytes = (int64_t)n.grid * 2 * n.rows * (D + 2) * (int64_t)sizeof(float);
    return notes_bytes(n) + (bytes + 255) / 256 * 256;
}

cudaError_t launch_tree_attn(const TreeAttnParams &given, cudaStream_t st) {
    if (given.B <= 0) return cudaSuccess;
    TreeAttnParams p = given;
    const int D = p.cache.D;
    const Plan n = plan(p.N * p.G, D, p.sms);
    p.notes = static_cast<int4 *>(p.workspace);
    p.ws = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + notes_bytes(n));
    const cudaError_t e = n.tc             ? launch_tree_attn_tc(p, n.grid, st)
                          : p.dtype == 1 ? launch_type<1>(p, n, st)
                                         : launch_type<2>(p, n, st);
    if (e != cudaSuccess) return e;
    if (p.dtype == 1)
        return D == 64    ? launch_join<1, 64>(p, n, st)
               : D == 128 ? launch_join<1, 128>(p, n, st)
                          : launch_join<1, 256>(p, n, st);
    return D == 64    ? launch_join<2, 64>(p, n, st)
           : D == 128 ? launch_join<2, 128>(p, n, st)
                      : launch_join<2, 256>(p, n, st);
}

}  // namespace specv
