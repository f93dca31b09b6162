// Attention of new tokens over the paged cache, few query rows a K/V head (decoding, short chains).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(x_ij - m_i),  x_ij = log2(e) scale q_i.k_j,
// over the positions j that row i sees; m_i follows the row's maximum. The rows of an item are the
// tokens times the G query heads that share one K/V head, so K and V are read once for up to 16 MT
// rows, and DRAM bounds it: 4 D bytes a position (2 D over an 8-bit cache) against 4 D operations a
// row.
//
// A CTA is four warps; each takes 32 of a tile's 128 positions, 16 or all 32 at a time, and keeps its
// own references, sums and output in registers: the main loop has no barrier. Each warp has a ring of
// its own in shared memory that asynchronous copies fill, 8 KB of K and V a place (16 positions at
// D = 128, 32 of half that size), so that an SM keeps about 128 KB in flight. (64 tokens over up to 8192
// positions at D = 64: 132 us, 140 with 16 positions at a time; over e4m3 at D = 128: 284 against 320 us for
// 128 tokens.) Products are m16n8k16 with the queries as the 16 rows: with 8 rows an item half of that
// work is lost, but it is a tenth of what the time of the bytes allows. Block-table entries are fetched
// a step before their copies.
//
// One token of 128 requests over up to 8192 positions (32 query and 8 K/V heads x 128, bfloat16): 384 to
// 394 us, 6.8 to 7.0 TB/s (the measured copy: 6.8). Over 500000 positions in e4m3, 64 query heads: 200 us,
// 5.1 TB/s: there the conversions count, issued in 49% of the cycles by eight warps an SM with the
// integer pipe at 49% and DRAM at 66%.
//
// 8-bit caches: codes become halves on the way from shared memory to the products' operands. Both
// products contract over (or produce) an index whose order is free, so lane (g, c) takes the
// elements [c D/4, (c+1) D/4) of its positions as its share of K, and the columns [g D/8, (g+1) D/8)
// of V, wide loads both. Positions in places of eight 16-byte units are XORed so that all loads
// are free of bank conflicts (two-way for 8-bit V at D = 64).
//
// What a row does not see: scores are replaced, never multiplied. A position that no row of the
// item sees is not read at all (zeros stand in its place); where some rows see it, V is looked
// through for NaN and infinities, and a step that has any is added up without the matrix unit.

#pragma once

#include "paged_attn.cuh"

namespace specv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// What an item costs besides its keys, in positions (64 chains of six over up to 8192 positions took
// 259 us with 64 and 256, 269 with 1024; 32 tokens over 1000 39.5, 37.4 and 37.5).
constexpr int kFixed = 256;

template <int KIND, int DP, int MT>
struct Few {
    static constexpr int kRows = 16 * MT;
    static constexpr int kEsz = KIND ? 1 : 2;
    static constexpr int kRow = DP * kEsz;                    // bytes of a position in its place
    static constexpr int kStep = kRow <= 128 ? 32 : 16;       // positions of a place
    static constexpr int kStage = 2 * kStep * kRow;           // K, then V
    static constexpr int kCtas = paged_few_ctas(KIND != 0, DP);
    static constexpr int kStages = kRow == 64 ? 4 : 3;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kPitch = DP + 8;                     // floats of a row being joined
    static constexpr int kJoin = kRows * kPitch * 4;          // in the ring's place
    static constexpr int kQ = kRing > kJoin ? kRing : kJoin;
    static constexpr int kFac = kQ + kRows * DP * 2;
    static constexpr int kM = kFac + kRows * 4;
    static constexpr int kL = kM + kWarps * kRows * 4;
    static constexpr int kSeen = kL + kWarps * kRows * 4;
    static constexpr int kBytes = kSeen + kWarps * kStages * 4;
    static_assert(kBytes * kCtas <= 227 * 1024 - kCtas * 1024, "shared memory of an SM");
};

// The place of 16-byte unit u of position t.
template <int KIND, int DP>
__device__ __forceinline__ int swizzle(int t, int u) {
    if (KIND == 0 || DP == 128) return u ^ (t & 7);
    if (DP == 64) return u ^ ((t >> 1) & 3);
    return u ^ ((u >> 3) << 1) ^ ((t ^ (t >> 1)) & 1) ^ (((t >> 2) & 1) << 2);
}

template <int I>      // 1 bf16, 2 f16
__device__ __forceinline__ void mma(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (I == 2)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldmatrix(uint32_t at) {
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(at)
                 : "memory");
    return r;
}
__device__ __forceinline__ uint4 ldmatrix_t(uint32_t at) {
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(at)
                 : "memory");
    return r;
}
// T: the rows' type; KIND: 0 a cache of that type, 1 e4m3, 2 e5m2; DP: D, up to the next of 64, 128
// and 256; MT: groups of 16 query rows of an item.
template <int T, int KIND, int DP, int MT>
__global__ void __launch_bounds__(kThreads, Few<KIND, DP, MT>::kCtas)
    paged_few_kernel(PagedAttnParams P) {
    using S = Few<KIND, DP, MT>;
    constexpr int I = KIND ? 2 : T;                 // the operands' type
    constexpr int RT = S::kRows, KS = DP / 16, NT = DP / 8, kStages = S::kStages;
    constexpr int NP = S::kStep, HT = NP / 8;       // positions of a step, eights of them
    constexpr unsigned kAll = 0xffffffffu >> (32 - NP);
    constexpr int U = S::kRow / 16;                 // 16-byte units of a position
    extern __shared__ __align__(128) char smem[];
    const spec_kv_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    float *s_fac = reinterpret_cast<float *>(smem + S::kFac);
    float *s_m = reinterpret_cast<float *>(smem + S::kM);
    float *s_l = reinterpret_cast<float *>(smem + S::kL);
    unsigned *s_seen = reinterpret_cast<unsigned *>(smem + S::kSeen) + warp * kStages;
    char *ring = smem + warp * kStages * S::kStage;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
    const float unit = P.scale * kLog2e * (C.k_scale ? __ldg(C.k_scale) : 1.f);
    const int units = C.D * S::kEsz / 16;           // of a position in the cache

    paged_status(P, kThreads);
    // a tile of positions is the least work worth a CTA
    PagedWalk<RT> walk(P, kFixed, (int64_t)P.G * kPosTile);
    PagedPart A;
    bool any = false;

    while (walk.next(P, A)) {
        const int steps = 32 / NP * (A.stop - A.tile);
        auto first = [&](int s) {
            const int i = A.tile + s * NP / 32;
            return (i < A.skip ? i : A.base + i) * kPosTile + warp * 32 + s % (32 / NP) * NP;
        };
        // The block of this lane's position in step s: -1 if no row sees it, -2 if it is not there.
        auto page = [&](int s) -> int {
            const int p = s < steps ? first(s) + lane % NP : A.hi;
            if (p >= A.hi || (p < A.lo && p >= P.sinks)) return -1;
            const int block = paged_page(P, A.b, p);
            return block >= 0 && block < C.num_blocks ? block : -2;
        };
        // Starts the copies of step s into its place.
        auto issue = [&](int s, int block) {
            if (s < steps) {
                const int p = first(s) + lane % NP;
                const uint32_t off = p - P.by_page((uint32_t)p) * C.block_size;
                const uint32_t in = (C.layout == SPEC_KV_NHD ? off * C.H + A.head
                                                             : A.head * C.block_size + off) * units;
                if (block == -2 && P.status) atomicMax(P.status + A.b, SPEC_REQ_BAD_SLOT);
                const unsigned seen = __ballot_sync(0xffffffffu, block >= 0) & kAll;
                if (lane == 0) s_seen[s % kStages] = seen;
                const uint32_t to = ring_s + (uint32_t)(s % kStages) * S::kStage;
#pragma unroll
                for (int q = 0; q < U * NP / 32; ++q) {
                    const int t = (q * 32 + lane) / U, u = lane % U;
                    const int blk = __shfl_sync(0xffffffffu, block, t);
                    const uint32_t from = __shfl_sync(0xffffffffu, in, t) + u;
                    const bool ok = blk >= 0 && u < units;
                    const int64_t k = ok ? blk * C.k_block_stride * S::kEsz + (int64_t)from * 16 : 0;
                    const int64_t v = ok ? blk * C.v_block_stride * S::kEsz + (int64_t)from * 16 : 0;
                    const uint32_t dst = to + t * S::kRow + swizzle<KIND, DP>(t, u) * 16;
                    copy16(dst, static_cast<const char *>(C.k) + k, ok);
                    copy16(dst + NP * S::kRow, static_cast<const char *>(C.v) + v, ok);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int next = page(0);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            const int cur = next;
            next = page(s + 1);
            issue(s, cur);
        }

        // Q in the order of the products' operands, a 16-byte word of a lane for each step.
        const int row0 = A.r * RT;
        for (int r = warp; r < RT; r += kWarps) {
            constexpr int E = DP / 64;                   // pairs of elements of a lane
            const bool live = r < A.rows;
            const unsigned short *q = paged_query(P, A.req.first, A.head, row0 + (live ? r : 0));
            float x[E][2], big = 0.f, down = 1.f, up = 1.f;
            uint32_t raw[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = (e * 32 + lane) * 2;
                const bool in = live && d < C.D;
                raw[e] = in ? (uint32_t)__ldg(q + d) | (uint32_t)__ldg(q + d + 1) << 16 : 0u;
                x[e][0] = value16<T>(raw[e] & 0xffffu);
                x[e][1] = value16<T>(raw[e] >> 16);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float a = fabsf(x[e][h]);
                    if (a < INFINITY) big = fmaxf(big, a);
                }
            }
            if (T == 1 && I == 2) {
                // 2^k brings the row's largest into [2^14, 2^15), at most 2^126
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
                const uint32_t ex = max(__float_as_uint(big) >> 23, 15u);
                up = __uint_as_float((268u - ex) << 23);
                down = __uint_as_float((ex - 14u) << 23);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = (e * 32 + lane) * 2;
                int kk, cc, hi8;
                if (KIND == 0) {
                    kk = d >> 4;
                    cc = (d & 7) >> 1;
                    hi8 = (d >> 3) & 1;
                } else {
                    cc = d / (DP / 4);
                    kk = d % (DP / 4) / 4;
                    hi8 = (d >> 1) & 1;
                }
                const int word = (((r >> 4) * KS + kk) * 32 + (r & 7) * 4 + cc) * 4 +
                                 ((r >> 3) & 1) + 2 * hi8;
                reinterpret_cast<uint32_t *>(smem + S::kQ)[word] =
                    T == 1 && I == 2 ? pack2<2>(x[e][0] * up, x[e][1] * up) : raw[e];
            }
            if (lane == 0) s_fac[r] = paged_factor(unit * down);
        }
        __syncthreads();

        float fac[MT][2], m[MT][2], l[MT][2], o[MT][NT][4];
        uint32_t at[MT][2];                        // ends of this lane's rows g and g + 8
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = i * 16 + e * 8 + g;
                fac[i][e] = s_fac[r];
                m[i][e] = kPagedNoMax;
                l[i][e] = 0.f;
                at[i][e] = r < A.rows ? paged_end(P, A.req.pos, row0 + r) : 0u;
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;

        for (int s = 0; s < steps; ++s) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();     // everyone's copies are in, and the place refilled next is free
            const int cur = next;
            next = page(s + kStages);
            issue(s + kStages - 1, cur);
            const char *st = ring + (s % kStages) * S::kStage;
            const uint32_t st_s = ring_s + (s % kStages) * S::kStage;
            const unsigned seen = s_seen[s % kStages];
            const int j0 = first(s);
            if (seen == 0u) continue;
            // all positions are there and every row sees them
            const bool plain = seen == kAll && all_see(P, A.e0, A.e1, j0, NP);
            float x[MT][HT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < HT; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][h][e] = 0.f;
            const uint4 *qf = reinterpret_cast<const uint4 *>(smem + S::kQ) + lane;
            if constexpr (KIND == 0) {
                const int t = (lane & 7) + ((lane >> 4) << 3), u0 = (lane >> 3) & 1;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint4 k[HT / 2];
#pragma unroll
                    for (int h = 0; h < HT / 2; ++h)
                        k[h] = ldmatrix(st_s + (t + 16 * h) * S::kRow +
                                        swizzle<KIND, DP>(t, 2 * kk + u0) * 16);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint4 a = qf[(i * KS + kk) * 32];
#pragma unroll
                        for (int h = 0; h < HT / 2; ++h) {
                            mma<I>(x[i][2 * h], a, k[h].x, k[h].y);
                            mma<I>(x[i][2 * h + 1], a, k[h].z, k[h].w);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < DP / 64; ++q) {          // 16 bytes of a position: four steps
                    uint32_t w[HT][4];
#pragma unroll
                    for (int h = 0; h < HT; ++h) {
                        const int t = g + 8 * h;
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            st + t * S::kRow + swizzle<KIND, DP>(t, c * (DP / 64) + q) * 16);
                        w[h][0] = v.x;
                        w[h][1] = v.y;
                        w[h][2] = v.z;
                        w[h][3] = v.w;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const uint4 a = qf[(i * KS + q * 4 + k) * 32];
#pragma unroll
                            for (int h = 0; h < HT; ++h)
                                mma<I>(x[i][h], a, halves2<KIND>(w[h][k]), halves2<KIND>(w[h][k] >> 16));
                        }
                }
            }
            // this lane's scores: rows g (e 0, 1) and g + 8, positions 8 h + 2 c + (e & 1)
            unsigned bits[MT][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    bits[i][e] = plain ? kAll
                                       : seen & paged_bits(j0, at[i][e], A.hi, P.window, P.sinks);
            bool up = false;
            float top[MT][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    top[i][e2] = kPagedNoMax;
#pragma unroll
                    for (int h = 0; h < HT; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &y = x[i][h][2 * e2 + e];
                            // rounded here, not with the difference from m: p may not pass 2^15
                            y = __fmul_rn(y, fac[i][e2]);
                            if (!plain && !((bits[i][e2] >> (8 * h + 2 * c + e)) & 1)) y = -INFINITY;
                            top[i][e2] = fmaxf(top[i][e2], y);
                        }
                    up |= top[i][e2] > paged_limit(m[i][e2]);
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float to = top[i][e];
                        to = fmaxf(to, __shfl_xor_sync(~0u, to, 1));
                        to = fmaxf(to, __shfl_xor_sync(~0u, to, 2));
                        to = paged_reference(m[i][e], to);
                        a[e] = ex2(m[i][e] - to);
                        m[i][e] = to;
                        l[i][e] *= a[e];
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][j][e] *= a[e >> 1];
                }
            }
            uint4 p[MT][HT / 2];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int h = 0; h < HT; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[i][h][e] = ex2(x[i][h][e] - m[i][e >> 1]);
                        l[i][e >> 1] += x[i][h][e];
                    }
#pragma unroll
                for (int h = 0; h < HT / 2; ++h) {
                    const float (&y)[4] = x[i][2 * h], (&z)[4] = x[i][2 * h + 1];
                    p[i][h] = make_uint4(pack2<I>(y[0], y[1]), pack2<I>(y[2], y[3]),
                                         pack2<I>(z[0], z[1]), pack2<I>(z[2], z[3]));
                }
            }
            const char *vs = st + NP * S::kRow;
            bool odd = false;
            if (!plain) {
                const uint4 *w = reinterpret_cast<const uint4 *>(vs);
                for (int i = lane; i < NP * U; i += 32) {
                    const uint4 v = w[i];
                    odd |= odd_word<I, KIND>(v.x) | odd_word<I, KIND>(v.y) | odd_word<I, KIND>(v.z) |
                           odd_word<I, KIND>(v.w);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (odd) {
                // Element by element, and only for the rows that see the position; p is rounded as
                // for the products.
#pragma unroll 1
                for (int t = 0; t < NP; ++t)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e2 = 0; e2 < 2; ++e2) {
                            const int from = (lane & ~3) | ((t & 7) >> 1);
                            const uint4 &pp = p[i][HT == 4 && t >= 16 ? HT / 2 - 1 : 0];
                            const uint32_t w0 = __shfl_sync(0xffffffffu, e2 ? pp.y : pp.x, from);
                            const uint32_t w1 = __shfl_sync(0xffffffffu, e2 ? pp.w : pp.z, from);
                            const float pt = value16<I>(((t >> 3 & 1 ? w1 : w0) >> ((t & 1) * 16)) & 0xffffu);
                            if (!((bits[i][e2] >> t) & 1)) continue;
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int d = KIND ? (2 * c + e) * (DP / 8) + j : 8 * j + 2 * c + e;
                                    const int by = d * S::kEsz;
                                    const char *a = vs + t * S::kRow +
                                                    swizzle<KIND, DP>(t, by >> 4) * 16 + (by & 15);
                                    const float v =
                                        KIND ? value16<2>(halves2<KIND>(*reinterpret_cast<const uint8_t *>(a)) &
                                                          0xffffu)
                                             : value16<I>(*reinterpret_cast<const uint16_t *>(a));
                                    float &y = o[i][j][2 * e2 + e];
                                    y = fabsf(v) < INFINITY ? fmaf(pt, v, y) : y + v;
                                }
                        }
            } else if constexpr (KIND == 0) {
                const int t = lane & 15, u0 = lane >> 4;
#pragma unroll
                for (int h = 0; h < HT / 2; ++h)
#pragma unroll
                    for (int j = 0; j < NT; j += 2) {
                        const uint4 v = ldmatrix_t(st_s + (NP + 16 * h + t) * S::kRow +
                                                   swizzle<KIND, DP>(t, j + u0) * 16);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            mma<I>(o[i][j], p[i][h], v.x, v.y);
                            mma<I>(o[i][j + 1], p[i][h], v.z, v.w);
                        }
                    }
            } else {
                // columns g D/8 + j of positions 2c, 2c + 1 and 2c + 8, 2c + 9
#pragma unroll
                for (int h = 0; h < HT / 2; ++h) {
                    const int t0 = 16 * h + 2 * c, ts[4] = {t0, t0 + 1, t0 + 8, t0 + 9};
                    uint32_t w[4][DP / 32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const char *row = vs + ts[q] * S::kRow;
                        if constexpr (DP == 64) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(
                                row + swizzle<KIND, DP>(ts[q], g >> 1) * 16 + (g & 1) * 8);
                            w[q][0] = v.x;
                            w[q][1] = v.y;
                        } else {
#pragma unroll
                            for (int k = 0; k < DP / 128; ++k) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(
                                    row + swizzle<KIND, DP>(ts[q], g * (DP / 128) + k) * 16);
                                w[q][4 * k] = v.x;
                                w[q][4 * k + 1] = v.y;
                                w[q][4 * k + 2] = v.z;
                                w[q][4 * k + 3] = v.w;
                            }
                        }
                }
#pragma unroll
                for (int k = 0; k < DP / 32; ++k)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        // bytes 2y, 2y + 1 of both positions, put together position by position
                        const uint32_t sel = y ? 0x7362 : 0x5140;
                        const uint32_t a = __byte_perm(w[0][k], w[1][k], sel);
                        const uint32_t b = __byte_perm(w[2][k], w[3][k], sel);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            mma<I>(o[i][4 * k + 2 * y], p[i][h], halves2<KIND>(a), halves2<KIND>(b));
                            mma<I>(o[i][4 * k + 2 * y + 1], p[i][h], halves2<KIND>(a >> 16),
                                   halves2<KIND>(b >> 16));
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // The four warps' states become one.
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 1);
                l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 2);
                if (c == 0) {
                    s_m[warp * RT + i * 16 + e * 8 + g] = m[i][e];
                    s_l[warp * RT + i * 16 + e * 8 + g] = l[i][e];
                }
            }
        __syncthreads();      // the ring is free, too
        float *join = reinterpret_cast<float *>(smem);
        float f[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = i * 16 + e * 8 + g;
                float most_m = s_m[r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) most_m = fmaxf(most_m, s_m[w * RT + r]);
                f[i][e] = exp2f(m[i][e] - most_m) * v_scale;
            }
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = i * 16 + (e >> 1) * 8 + g;
                            const int d = KIND ? (2 * c + (e & 1)) * (DP / 8) + j
                                               : 8 * j + 2 * c + (e & 1);
                            float &to = join[r * S::kPitch + d];
                            const float y = o[i][j][e] * f[i][e >> 1];
                            to = w > 0 ? to + y : y;
                        }
            }
            __syncthreads();
        }
        const bool whole = A.whole();
        const int q4 = C.D / 4;
        float *part = paged_slot(P, blockIdx.x, A.begins, RT, DP);
        for (int i = tid; i < A.rows * q4; i += kThreads) {
            const int r = i / q4, d4 = i - r * q4;
            const float4 v = *reinterpret_cast<const float4 *>(join + r * S::kPitch + d4 * 4);
            float top = s_m[r], sum = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w * RT + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_l[w * RT + r] * exp2f(s_m[w * RT + r] - top);
            if (whole) {
                const float n1 = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t to = paged_row(P, A.req.first, A.head, row0 + r);
                paged_store4<T>(P.out, to * C.D + d4 * 4,
                                make_float4(v.x * n1, v.y * n1, v.z * n1, v.w * n1));
                if (P.lse && d4 == 0) P.lse[to] = paged_lse(top, sum);
            } else {
                reinterpret_cast<float4 *>(part + r * DP)[d4] = v;
                if (d4 == 0) {
                    part[RT * DP + r] = top;
                    part[RT * (DP + 1) + r] = sum;
                }
            }
        }
        __syncthreads();      // shared memory is free for the next item
        any = true;
    }
    if (tid == 0) paged_note(P, walk.range, A, RT, any);
}

template <int T, int KIND, int DP, int MT>
cudaError_t launch(const PagedAttnParams &p, int grid, cudaStream_t st) {
    const int smem = Few<KIND, DP, MT>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(paged_few_kernel<T, KIND, DP, MT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    paged_few_kernel<T, KIND, DP, MT><<<grid, kThreads, smem, st>>>(p);
    return cudaGetLastError();
}
template <int T, int KIND>
cudaError_t launch_size(const PagedAttnParams &p, int mt, int grid, cudaStream_t st) {
    const int DP = paged_padded(p.cache.D);
    if (DP == 64)
        return mt == 1 ? launch<T, KIND, 64, 1>(p, grid, st) : launch<T, KIND, 64, 2>(p, grid, st);
    if (DP == 128)
        return mt == 1 ? launch<T, KIND, 128, 1>(p, grid, st)
                         : launch<T, KIND, 128, 2>(p, grid, st);
    return launch<T, KIND, 256, 1>(p, grid, st);
}
}  // namespace

template <int T>
cudaError_t launch_paged_few_type(const PagedAttnParams &p, int mt, int grid, cudaStream_t st) {
    if (p.cache.kind == SPEC_CACHE_SAME) return launch_size<T, 0>(p, mt, grid, st);
    if (p.cache.kind == SPEC_CACHE_FP8_E4M3) return launch_size<T, 1>(p, mt, grid, st);
    return launch_size<T, 2>(p, mt, grid, st);
}


}  // namespace specv
