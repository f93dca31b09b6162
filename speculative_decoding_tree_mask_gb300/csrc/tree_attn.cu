// Tree attention over the 4-bit paged cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(x_ij - m_i),  x_ij = log2(e) scale q_i.k_j,
// over the context positions and the nodes that node i may see; m_i follows the row's maximum.
// The rows of an item are the N nodes times the G query heads that share one K/V head, so K and
// V are read once for all of them: 0.5625 bytes an element. With few rows DRAM should bound it;
// what stands in the way is the number of instructions, and the products (the warps' matrix unit
// does 1024 multiplications a clock and SM). One token over 262000 positions of 8 K/V heads x 128:
// 70 us, 4.3 TB/s (63% of the measured copy), 62% of the issue slots and 57% of the integer pipe
// taken. It issues 5.6 instructions for two elements: 2.6 on the integer pipe (conversions, bytes
// put in place, comparisons), the scale's multiplication, 1.0 more on the FMA pipe (addresses and
// float32), 0.45 loads and copies, 0.25 products, 0.3 others. 64 chains of six, 24 rows an item:
// 207 us where the bytes need 79 and the products about 100; the output of 24 rows leaves registers
// for eight warps an SM only, and it issues 7.0 for two elements.
//
// A code times its block scale has at most six significant bits and lies in [2^-10, 2688], so
// it is exact as a half; the tensor scales are applied to the scores and to the result. Q is
// brought to halves by a power of two for each row (bfloat16: exact for what is within 2^-31 of the
// row's largest element) and p is rounded to a half with the row's largest at 2^7 or more (kHeadroom:
// what is 2^-31 of it still counts). The products are
// m16n8k16 of halves with float32 sums, transposed: S^T = K Q^T and O^T = V^T P^T, so that rows
// come in groups of eight (with Q as the 16-row operand, one token of up to eight heads paid
// for 16 rows, and 24 rows for 32).
//
// A CTA is four warps; each takes 32 of a tile's 128 positions and keeps its own maxima, sums
// and output in registers, so that the main loop has no barrier. Codes and scales come through
// a ring in shared memory by asynchronous copies. Both products contract over an index whose
// order is free: the head's elements for K, the positions for V. So lane (g, c) takes the
// elements [c D/4, (c+1) D/4) of the positions g and g + 8 as its share of the K operand, wide
// loads, and the elements [g D/8, (g+1) D/8) of its four positions for V, whose pairs of
// positions are put together by a byte permute; P^T is S^T through movmatrix. The positions of
// a group of eight are taken in the order 0 1 3 2 4 5 7 6, which with the swizzle of 16-byte
// units makes both loads free of bank conflicts. A row's maximum is followed only once it has
// risen by 2^8, so that the lanes need not agree on it for every tile.

#include "tree_attn.cuh"

namespace specv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// The tree's tile and an item's rest, in context tiles. With 2, 4 and 8: the chains above 211, 207
// and 204 us; 64 chains over up to 2000 positions, D = 64, 48, 43 and 40; 128 single tokens over up
// to 1000, 38, 41 and 41; over up to 100, 19 each.
constexpr int kTreeCost = 4;

// CTAs an SM holds, by the registers of the output (D x 8 RG floats a warp) and the ring. One
// more each spills: 24 rows of D = 128 took 378 us with three CTAs, 207 with two.
constexpr int ctas_per_sm(int D, int RG) {
    return D * RG <= 64 ? 5 : D * RG <= 128 ? 4 : D * RG <= 256 ? 3 : 2;
}
// Tiles in the ring: the one at work and those in flight.
constexpr int stages(int D, int RG) { return D == 256 || (D == 128 && RG == 1) ? 2 : 3; }

template <int D, int RG>
struct Ring {
    static constexpr int kStages = stages(D, RG);
    static constexpr int kCodes = 32 * D / 2;             // bytes of K (and of V) codes
    static constexpr int kScales = 32 * D / 16;
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = kKs + kScales, kSeen = kVs + kScales;
    static constexpr int kBytes = kSeen + 16;
};

// Shared memory of a CTA, in bytes from its start.
template <int T, int D, int RG>
struct Smem {
    static constexpr int kRows = 8 * RG;
    static constexpr int kRing = kWarps * stages(D, RG) * Ring<D, RG>::kBytes;
    static constexpr int kTreeStride = D + 8;                              // elements
    static constexpr int kTree = 2 * kMaxN * kTreeStride * 2;              // in the ring's place
    static constexpr int kJoin = D / 4 * (kRows + 1) * 16;                 // likewise
    static constexpr int kFirst = kRing > kTree ? kRing : kTree;
    static constexpr int kQ = kFirst > kJoin ? kFirst : kJoin;
    static constexpr int kQt = kQ + kRows * D * 2;                         // Q in its own type
    static constexpr int kFac = kQt + (T == 1 ? kRows * D * 2 : 0);
    static constexpr int kM = kFac + 2 * kRows * 4;   // factors of the context's, the tree's scores
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

// An 8 x 8 matrix of 16-bit elements, transposed: lane (g, c) has elements 2c, 2c + 1 of row g.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// The state of an item in one warp. Lane (g, c) has rows 2c and 2c + 1 of each of RG groups of
// eight; of these the elements [g D/8, (g+1) D/8): o[i][j][2 h + e] is element g D/8 + 2 j + h of
// row 8 i + 2 c + e.
template <int D, int RG>
struct Acc {
    float o[RG][D / 16][4];
    float m[RG][2], l[RG][2];   // m: the reference, the same in all lanes of a row; l: this lane's

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < RG; ++i) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
            m[i][0] = m[i][1] = kNoMax;
            l[i][0] = l[i][1] = 0.f;
        }
    }
    // Takes this lane's largest scores in: when one in the warp has passed its row's reference
    // far enough, all rows follow theirs.
    __device__ __forceinline__ void raise(float (&x)[RG][2]) {
        bool up = false;
#pragma unroll
        for (int i = 0; i < RG; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) up |= x[i][e] > attn_limit(m[i][e]);
        if (!__any_sync(0xffffffffu, up)) return;
#pragma unroll
        for (int i = 0; i < RG; ++i) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float to = x[i][e];
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) to = fmaxf(to, __shfl_xor_sync(~0u, to, s));
                to = attn_reference(m[i][e], to);
                a[e] = ex2(m[i][e] - to);
                m[i][e] = to;
                l[i][e] *= a[e];
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] *= a[e & 1];
        }
    }
};

// T: 1 bf16, 2 f16; RG: groups of 8 query rows of an item.
template <int T, int D, int RG>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, RG))
    tree_attn_kernel(TreeAttnParams P, int row_tiles) {
    using S = Smem<T, D, RG>;
    using Rg = Ring<D, RG>;
    constexpr int RT = S::kRows, KS = D / 16, kStages = Rg::kStages;
    extern __shared__ __align__(128) char smem[];
    const spec_fp4_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int pg = g ^ ((g >> 1) & 1);                 // position of the g-th of eight
    const int pt0 = 2 * c + (c & 1), pt1 = 2 * c + 1 - (c & 1);   // ... of 2c and 2c + 1
    const int R = P.N * P.G;
    float *s_fac = reinterpret_cast<float *>(smem + S::kFac);
    float *s_m = reinterpret_cast<float *>(smem + S::kM);
    float *s_l = reinterpret_cast<float *>(smem + S::kL);
    unsigned long long *s_odd = reinterpret_cast<unsigned long long *>(smem + S::kOdd);
    char *ring = smem + warp * kStages * Rg::kBytes;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
    const float unit = P.scale * kLog2e;
    const float cache_unit = unit * (C.k_scale ? __ldg(C.k_scale) : 1.f);

    AttnWalk walk(P, C.H * row_tiles, kTreeCost, P.columns);
    AttnPart A;
    bool any = false;
    Acc<D, RG> acc;

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

        // Q, in the order of the products' operands: element d of row r belongs to lane
        // (r % 8, d / (D/4)); two steps of 16 elements make one 16-byte word of a lane.
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
            // 2^k brings the largest into [2^14, 2^15), at most 2^126
            const uint32_t ex = max(__float_as_uint(big) >> 23, 15u);
            const float up = __uint_as_float((268u - ex) << 23);
            const int cc = lane * E / (D / 4);
            char *q16 = smem + S::kQ, *qt = smem + S::kQt;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const int in = lane * E % (D / 4) + e;   // element within the lane's quarter
                const int kk = in / 4;                   // step; its words are elements 0 1, 2 3
                const int off = (((r / 8) * (KS / 2) + kk / 2) * 32 + (r % 8) * 4 + cc) * 16 +
                                (kk & 1) * 8 + (in & 2) * 2;
                *reinterpret_cast<uint32_t *>(q16 + off) = f16x2(x[e] * up, x[e + 1] * up);
                if (T == 1)
                    *reinterpret_cast<uint32_t *>(qt + off) =
                        (uint32_t)raw[e] | (uint32_t)raw[e + 1] << 16;
            }
            if (lane == 0) {
                const float down = __uint_as_float((ex - 14u) << 23);
                s_fac[r] = attn_factor(cache_unit * down);
                s_fac[RT + r] = attn_factor(T == 1 ? unit : unit * down);   // bf16: Q as it is
            }
        }
        __syncthreads();

        float fac[RG][2];
#pragma unroll
        for (int i = 0; i < RG; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) fac[i][e] = s_fac[i * 8 + 2 * c + e];
        // two steps of Q for group i
        auto q_frag = [&](const char *base, int i, int kk2) -> uint4 {
            return *reinterpret_cast<const uint4 *>(base + ((i * (KS / 2) + kk2) * 32 + lane) * 16);
        };
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
            // two groups of 16 positions, 8 j + pg of which are this lane's for K
            float s[2][RG][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[h][r][e] = 0.f;
            // scores: the elements of eight codes (a word) at a time
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
                uint4 qv[RG];
#pragma unroll
                for (int r = 0; r < RG; ++r) qv[r] = q_frag(smem + S::kQ, r, w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[4], y[4];
                    e2m1x8_to_f16x2(kw[2 * h][w], x);
                    e2m1x8_to_f16x2(kw[2 * h + 1][w], y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = hmul2(x[e], ks[2 * h][w / 2]);
                        y[e] = hmul2(y[e], ks[2 * h + 1][w / 2]);
                    }
                    const uint32_t a0[4] = {x[0], y[0], x[1], y[1]}, a1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        mma<2>(s[h][r], a0, qv[r].x, qv[r].y);
                        mma<2>(s[h][r], a1, qv[r].z, qv[r].w);
                    }
                }
            }
            float top[RG][2];
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                top[r][0] = top[r][1] = kNoMax;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // rounded here, not with the difference from m: p may not pass 2^15
                        float x = __fmul_rn(s[h][r][e], fac[r][e & 1]);
                        if (seen != 0xffffffffu &&
                            !((seen >> (16 * h + 8 * (e >> 1) + pg)) & 1))
                            x = -INFINITY;
                        s[h][r][e] = x;
                        top[r][e & 1] = fmaxf(top[r][e & 1], x);
                    }
            }
            acc.raise(top);
#pragma unroll
            for (int r = 0; r < RG; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = ex2(s[h][r][e] - acc.m[r][e & 1]);
                        s[h][r][e] = p;
                        acc.l[r][e & 1] += p;
                    }
            // values
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p0[RG], p1[RG];
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    p0[r] = transpose8(f16x2(s[h][r][0], s[h][r][1]));
                    p1[r] = transpose8(f16x2(s[h][r][2], s[h][r][3]));
                }
                const int t0 = 16 * h;
                const int ts[4] = {t0 + pt0, t0 + pt1, t0 + 8 + pt0, t0 + 8 + pt1};
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
                    for (int y = 0; y < 4; ++y) {
                        // elements 8 w + 2 y and the next, of positions 2c, 2c + 1 and + 8
                        const uint32_t a[4] = {hmul2(prmt(va[y], vb[y], 0x5410), f0),
                                               hmul2(prmt(va[y], vb[y], 0x7632), f0),
                                               hmul2(prmt(vc[y], vd[y], 0x5410), f1),
                                               hmul2(prmt(vc[y], vd[y], 0x7632), f1)};
#pragma unroll
                        for (int r = 0; r < RG; ++r)
                            mma<2>(acc.o[r][4 * w + y], a, p0[r], p1[r]);
                    }
                }
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.o[r][j][e] *= v_scale;
        __syncthreads();      // the ring is free

        if (A.stop == A.nt) {
            // The tree's own nodes: their rows in shared memory, 16 nodes a warp.
            unsigned short *tk = reinterpret_cast<unsigned short *>(smem);
            unsigned short *tv = tk + kMaxN * S::kTreeStride;
            if (tid == 0) *s_odd = 0ull;
            __syncthreads();
            const int keys = min(kMaxN, (P.N + 15) / 16 * 16);
#pragma unroll 4
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
                unsigned bits[RG][2];
                float s[RG][4], top[RG][2];
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = r * 8 + 2 * c + e;
                        bits[r][e] =
                            rr < rows ? (unsigned)(__ldg(P.mask + (int64_t)b * P.N +
                                                         (row0 + rr) / P.G) >> key0) &
                                            (P.N - key0 >= 16 ? 0xffffu : (1u << (P.N - key0)) - 1u)
                                      : 0u;
                        top[r][e] = kNoMax;
                        s[r][e] = s[r][e + 2] = 0.f;
                    }
#pragma unroll
                for (int kk2 = 0; kk2 < KS / 2; ++kk2) {
                    uint4 qv[RG];
#pragma unroll
                    for (int r = 0; r < RG; ++r)
                        qv[r] = q_frag(smem + (T == 1 ? S::kQt : S::kQ), r, kk2);
                    // elements 8 kk2 .. + 7 of this lane's quarter, of nodes g and g + 8
                    uint2 x[2], y[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned short *k = tk + (key0 + g) * S::kTreeStride + c * (D / 4) +
                                                  8 * kk2 + 4 * e;
                        x[e] = *reinterpret_cast<const uint2 *>(k);
                        y[e] = *reinterpret_cast<const uint2 *>(k + 8 * S::kTreeStride);
                    }
                    const uint32_t a0[4] = {x[0].x, y[0].x, x[0].y, y[0].y};
                    const uint32_t a1[4] = {x[1].x, y[1].x, x[1].y, y[1].y};
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        mma<T>(s[r], a0, qv[r].x, qv[r].y);
                        mma<T>(s[r], a1, qv[r].z, qv[r].w);
                    }
                }
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = s_fac[RT + r * 8 + 2 * c + (e & 1)];
                        const bool on = (bits[r][e & 1] >> (g + 8 * (e >> 1))) & 1;
                        s[r][e] = on ? __fmul_rn(s[r][e], f) : -INFINITY;
                        top[r][e & 1] = fmaxf(top[r][e & 1], s[r][e]);
                    }
                acc.raise(top);
                uint32_t hi[RG][2], lo[RG][2];
#pragma unroll
                for (int r = 0; r < RG; ++r) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = ex2(s[r][e] - acc.m[r][e & 1]);
                        s[r][e] = p;
                        acc.l[r][e & 1] += p;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float x = s[r][2 * q], y = s[r][2 * q + 1];
                        if (T == 2) {
                            hi[r][q] = transpose8(f16x2(x, y));
                        } else {
                            // eight bits are too few for p: a second product has the rest
                            const uint32_t w = bf16x2(x, y);
                            hi[r][q] = transpose8(w);
                            lo[r][q] = transpose8(bf16x2(x - bf_lo(w), y - bf_hi(w)));
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t a[4];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        // elements 2 j, 2 j + 1 of nodes 2c + 8 q and the next
                        const unsigned short *v = tv + (key0 + 2 * c + 8 * q) * S::kTreeStride +
                                                  g * (D / 8) + 2 * j;
                        uint32_t x = *reinterpret_cast<const uint32_t *>(v);
                        uint32_t y = *reinterpret_cast<const uint32_t *>(v + S::kTreeStride);
                        if (odd) {
                            constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
                            if ((x & ex) == ex) x &= 0xffff0000u;
                            if ((x >> 16 & ex) == ex) x &= 0xffffu;
                            if ((y & ex) == ex) y &= 0xffff0000u;
                            if ((y >> 16 & ex) == ex) y &= 0xffffu;
                        }
                        a[2 * q] = prmt(x, y, 0x5410);
                        a[2 * q + 1] = prmt(x, y, 0x7632);
                    }
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        mma<T>(acc.o[r][j], a, hi[r][0], hi[r][1]);
                        if (T == 1) mma<T>(acc.o[r][j], a, lo[r][0], lo[r][1]);
                    }
                }
                // nodes with NaN or infinities in V: only for the rows that see them
                if (odd) {
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        if (!((odd >> t) & 1)) continue;
#pragma unroll
                        for (int r = 0; r < RG; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float p = __shfl_sync(0xffffffffu, s[r][2 * (t >> 3) + e],
                                                            (t & 7) * 4 + c);
                                if (!((bits[r][e] >> t) & 1)) continue;
#pragma unroll
                                for (int j = 0; j < D / 8; ++j) {
                                    const uint32_t x =
                                        tv[(key0 + t) * S::kTreeStride + g * (D / 8) + j];
                                    constexpr uint32_t ex = T == 1 ? 0x7f80u : 0x7c00u;
                                    if ((x & ex) == ex)
                                        acc.o[r][j / 2][2 * (j & 1) + e] +=
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
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = acc.l[r][e];
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
                if (g == 0) {
                    s_m[warp * RT + r * 8 + 2 * c + e] = acc.m[r][e];
                    s_l[warp * RT + r * 8 + 2 * c + e] = l;
                }
            }
        __syncthreads();
        // [D/32 of a lane][g][row]: four elements of a row each; the pitch avoids bank conflicts
        float4 *join = reinterpret_cast<float4 *>(smem);
        float f[RG][2];
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = r * 8 + 2 * c + e;
                float m = s_m[rr];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_m[w * RT + rr]);
                f[r][e] = exp2f(acc.m[r][e] - m);
            }
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) {
                            float4 v = make_float4(acc.o[r][2 * q][e] * f[r][e],
                                                   acc.o[r][2 * q][2 + e] * f[r][e],
                                                   acc.o[r][2 * q + 1][e] * f[r][e],
                                                   acc.o[r][2 * q + 1][2 + e] * f[r][e]);
                            float4 &to = join[(q * 8 + g) * (RT + 1) + r * 8 + 2 * c + e];
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
            const int r = i / (D / 4), d4 = i - r * (D / 4), gg = d4 / (D / 32), q = d4 % (D / 32);
            const float4 v = join[(q * 8 + gg) * (RT + 1) + r];
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

// The parts of cut items into the result. A thread has a float4 of a row and, of the parts,
// every PG-th, eight of them in flight together; the PG threads of a float4 meet in shared
// memory. PG is 1 for items of few parts and many rows.
constexpr int kJoinThreads = 256;
template <int T, int D, int PG>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(TreeAttnParams P, int rows_tile) {
    constexpr int F = D / 4, kPer = kJoinThreads / (F * PG);       // rows of a CTA
    __shared__ float4 s_o[PG > 1 ? kJoinThreads : 1];
    __shared__ float2 s_ml[PG > 1 ? kJoinThreads : 1];
    grid_dep_wait();
    const int c0 = blockIdx.y;
    const int4 note = P.notes[c0];
    if (note.x < 0) return;
    const int b = note.x, c1 = note.z, step = P.columns;
    const int row_tiles = (P.N * P.G + rows_tile - 1) / rows_tile;
    const int head = note.y / row_tiles, row0 = (note.y - head * row_tiles) * rows_tile;
    const int rows = min(rows_tile, P.N * P.G - row0);
    const int d4 = threadIdx.x % F, group = threadIdx.x / F % PG;
    const int r = blockIdx.x * kPer + threadIdx.x / (F * PG);
    if (PG == 1 && r >= rows) return;
    float m = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + group * step; c <= c1 && r < rows; c += 8 * PG * step) {
        float4 v[8];
        float pm[8], pl[8], top = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            pm[u] = kNoMax;
            const int k = c + u * PG * step;
            if (k > c1) continue;
            const float *part = attn_slot(P, k, k == c0, rows_tile, D);
            v[u] = __ldcg(reinterpret_cast<const float4 *>(part + r * D) + d4);
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
            if (c + u * PG * step > c1) continue;
            const float w = ex2(pm[u] - top);
            o.x = fmaf(v[u].x, w, o.x);
            o.y = fmaf(v[u].y, w, o.y);
            o.z = fmaf(v[u].z, w, o.z);
            o.w = fmaf(v[u].w, w, o.w);
            l = fmaf(pl[u], w, l);
        }
    }
    if (PG > 1) {
        s_o[threadIdx.x] = o;
        s_ml[threadIdx.x] = make_float2(m, l);
        __syncthreads();
        if (group != 0 || r >= rows) return;
        float top = m;
#pragma unroll
        for (int u = 1; u < PG; ++u) top = fmaxf(top, s_ml[threadIdx.x + u * F].x);
        const float a = ex2(m - top);
        o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
        l *= a;
        m = top;
#pragma unroll
        for (int u = 1; u < PG; ++u) {
            const float2 ml = s_ml[threadIdx.x + u * F];
            const float4 v = s_o[threadIdx.x + u * F];
            const float w = ex2(ml.x - top);
            o.x = fmaf(v.x, w, o.x);
            o.y = fmaf(v.y, w, o.y);
            o.z = fmaf(v.z, w, o.z);
            o.w = fmaf(v.w, w, o.w);
            l = fmaf(ml.y, w, l);
        }
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = attn_row(P, b, head, row0 + r);
    store_out4<T>(P.out, at * D + d4 * 4, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
    if (P.lse && d4 == 0) P.lse[at] = attn_lse(m, l);
}

// How a call is run: by this file's warps (groups of 8 rows of an item), or, with more rows
// than four groups, on the tcgen05 tensor cores. 16 requests of up to 16000 positions, 8 heads,
// here against there: 20 rows 79 us and 104, 32 rows 105 and 104, 36 rows (which would read the
// cache twice here) 174 and 105; at D = 64 54 and 76, 68 and 77, 112 and 77; up to 500 positions 18
// and 23, 23 and 22, 30 and 23. D = 256 has no tcgen05 form: its Q, K and V tiles do not fit in
// shared memory together.
struct Plan {
    bool tc;
    int groups, rows, grid;   // rows of an item
};
Plan plan(int R, int D, int sms) {
    Plan p;
    p.tc = R > 32 && D <= 128;
    const int most = D == 256 ? 2 : 4;
    p.groups = (R + 7) / 8 < most ? (R + 7) / 8 : most;
    p.rows = p.tc ? tree_attn_tc_rows(R) : 8 * p.groups;
    p.grid = sms * (p.tc ? 1 : ctas_per_sm(D, p.groups));
    return p;
}

template <int T, int D, int RG>
cudaError_t launch(const TreeAttnParams &p, int grid, cudaStream_t st) {
    const int smem = Smem<T, D, RG>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<T, D, RG>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int row_tiles = (p.N * p.G + 8 * RG - 1) / (8 * RG);
    tree_attn_kernel<T, D, RG><<<grid, kThreads, smem, st>>>(p, row_tiles);
    return cudaGetLastError();
}

template <int T, int D>
cudaError_t launch_groups(const TreeAttnParams &p, const Plan &n, cudaStream_t st) {
    if (n.groups == 1) return launch<T, D, 1>(p, n.grid, st);
    if (n.groups == 2) return launch<T, D, 2>(p, n.grid, st);
    if constexpr (D <= 128) {
        if (n.groups == 3) return launch<T, D, 3>(p, n.grid, st);
        return launch<T, D, 4>(p, n.grid, st);
    }
    return cudaErrorInvalidValue;
}

template <int T>
cudaError_t launch_type(const TreeAttnParams &p, const Plan &n, cudaStream_t st) {
    if (p.cache.D == 64) return launch_groups<T, 64>(p, n, st);
    if (p.cache.D == 128) return launch_groups<T, 128>(p, n, st);
    return launch_groups<T, 256>(p, n, st);
}

}  // namespace

namespace {

int64_t notes_bytes(const Plan &n) { return ((int64_t)n.grid * sizeof(int4) + 255) / 256 * 256; }

// Columns of CTAs (see tree_attn.cuh): one for each item of a request, unless that leaves more
// than one CTA in sixteen without work. Against one column: the 64 chains 207 us and 260, one token
// 70 and 72, 32 64-node trees 187 and 197, 7 heads 61 and 79. (What the limit gives away: 90 heads of
// 608 CTAs leave one in nine idle, and take 220 us in one column, 157 in 90, in the NHD layout; 144
// and 140 in HND.)
int columns(const TreeAttnParams &p, const Plan &n) {
    const int64_t items = (int64_t)p.cache.H * ((p.N * p.G + n.rows - 1) / n.rows);
    return items <= n.grid && n.grid % items * 16 <= n.grid ? (int)items : 1;
}

template <int T, int D>
cudaError_t launch_join(const TreeAttnParams &p, const Plan &n, cudaStream_t st) {
    constexpr int F = D / 4, PG = D == 256 ? 4 : 8;
    // all CTAs' work in items of about this many parts: over eight, the parts are shared out (one
    // token over 262000 positions 70 us, 78 if not; a chain of 6 over 50000, D = 64, 25 and 26; 16
    // tokens over 8000, which are not, 30, 33 if so; 4 chains of 6 over 8000, nine parts an item,
    // lose by it: 28 us, 23 if not)
    const int R = p.N * p.G, rows = R < n.rows ? R : n.rows;
    const int64_t items = (int64_t)p.B * p.cache.H * ((R + n.rows - 1) / n.rows);
    const int per = kJoinThreads / F;
    if (n.grid > 8 * items && rows <= 32)
        return launch_dependent(join_kernel<T, D, PG>, dim3((rows * PG + per - 1) / per, n.grid),
                                dim3(kJoinThreads), 0, st, p, n.rows);
    return launch_dependent(join_kernel<T, D, 1>, dim3((rows + per - 1) / per, n.grid),
                            dim3(kJoinThreads), 0, st, p, n.rows);
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
    Plan n = plan(p.N * p.G, D, p.sms);
    // no more CTAs than there can be units of work
    const int64_t units = (int64_t)p.B * p.cache.H * ((p.N * p.G + n.rows - 1) / n.rows) *
                          ((p.cache.max_blocks * (int64_t)p.cache.block_size + kTile - 1) / kTile +
                           (n.tc ? tree_attn_tc_cost() : kTreeCost));
    if (units < n.grid) n.grid = (int)units;
    p.columns = columns(p, n);
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
