// Attention of new tokens over the paged cache for many query rows (prompts, chunks of them, mixed
// batches), on the tcgen05 tensor cores.
//
// The same operator as paged_few.cuh for items of up to 256 rows; the two products bound it, 4 D
// operations a row and position. One CTA an SM; its warps have one part each and meet at mbarriers
// only:
//
//   load     (4 warps for K, 4 for V) tiles of 128 positions by asynchronous copies to a ring of
//            five places that K and V share, laid out for the tensor core (128-byte swizzle; K
//            contiguous along D, and V as it is, read transposed). Any page size, stride and layout
//            is a matter of their addresses. 8-bit codes pass through registers and become halves;
//   queries  (2 warps) an item's rows, when the last products of the item before are done;
//   multiply (2 warps, a thread of each issues for one softmax group) S = Q K^T for 128 rows and a
//            whole tile, then O += P V in two halves of 64 positions, the first of which runs while
//            softmax works on the second half. Sums are in tensor memory: S and O twice, all 512
//            columns at D = 128; P overwrites the S it came from;
//   softmax  (2 groups of 4 warps) S to P, a row a thread, no exchange between threads, reference
//            and sum in registers. O is rescaled in place when a reference rises, which is rare.
//
// With S of 64 columns a product reads 6 KB of shared memory for 32 clocks of work and gets 48 clocks
// of its bandwidth; with 128 columns 8 KB for 64 clocks, which is even. One group's softmax runs
// beside the other's products.
//
// Items of up to 128 rows (a decoding request in a mixed batch) leave the second group idle, and
// warps without a live row touch nothing: a tile then takes less time than its bytes do.
//
// What a row does not see: scores are replaced, never multiplied. A position that no row of the
// item sees is not read (zeros stand in its place). In tiles that some rows see in part, V is looked
// through; NaN and infinities are taken out of the products and added, at the end, to the rows that
// see them.
#pragma once

#include "paged_attn.cuh"
#include "tc_device.cuh"

namespace specv {
namespace {

constexpr int kLoad = 256;        // loading threads: K's, then V's
constexpr int kSoftmax = 256;     // threads of the two softmax groups
constexpr int kThreads = kSoftmax + kLoad + 128;   // the last: two warps multiply, two fetch queries
constexpr int kMmaWarp = (kSoftmax + kLoad) / 32;
constexpr int kQuery = 64;        // threads that fetch queries
constexpr int kRing = 5;
// What an item costs besides its keys, in positions.
constexpr int kTcFixed = 256;

template <int DP>
struct Tc {
    static constexpr int kOperand = 128 * DP * 2;                // a 128 x DP operand of 16 bits
    static constexpr int kTiles = 2 * kOperand;                  // Q first, then the ring
    static constexpr int kSmall = kTiles + kRing * kOperand;     // barriers and words
    static constexpr int kBytes = kSmall + 2048 + 1024;          // and room to align by 1024
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static constexpr int kColumns = 512;                         // 2 (128 + DP), a power of two
};

struct Words {
    uint64_t q_full, q_free, full[kRing], free[kRing], drain[2];
    uint64_t s_full[2], p_full[2][2], o_full[2];                 // of a softmax group; halves
    uint64_t o_last[2];                                          // once a part
    // Positions of a tile that are there. K's loader writes a tile's words again for the fourth
    // after it, whose place was that of a V whose products are done.
    unsigned seen[4][4];
    // A part's V has NaN or infinities that not every row sees. Of eight parts: V's loader clears
    // the word of the fourth part to come, where its own other warps are three tiles ahead at most
    // and softmax three behind.
    int odd[8];
    uint32_t tmem;
    int gave_up;
    // 1 / the power of two of each row of Q: a float's upper half. Of two parts: a part of one tile
    // may be read while the next one's queries come.
    unsigned short q_down[2][256];
};
static_assert(sizeof(Words) <= 2048, "room for the words");

// Byte of 16-byte chunk `j` of row r of an operand of D elements a row.
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
    return (uint32_t)(j >> 3) * (128 * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

// A wait of a whole warp: all of it goes on or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up));
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void *to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Whether every row of the item sees all of positions j0 .. j0 + n - 1, as far as they are there.
__device__ __forceinline__ bool all_see(const PagedAttnParams &P, const PagedPart &A, int j0, int n) {
    return j0 + n - 1 <= A.p0 &&
           (P.window == 0 || j0 > A.p1 - P.window || j0 + n - 1 < P.sinks);
}

// The reference of a row comes from a rounded product f s, within 2^-24 of it, which f s - top in
// one rounding brings to light: as 2^-4 at most up to scores of 2^20, beyond as more than a half
// holds. There the products are rounded alike first (Scores::apart).
constexpr float kApart = 1048576.f;

// S to P of 64 positions, the thread's row.
template <int I>
struct Scores {
    uint32_t s[2][32];

    // The scores, -inf where `see` has no bit; returns their largest.
    __device__ __forceinline__ float load(uint32_t s_tm, const unsigned (&see)[2]) {
        tmem_ld32(s_tm, s[0]);
        tmem_ld32(s_tm + 32, s[1]);
        tmem_wait_ld(s[0]);
        tmem_loaded(s[1]);
        if ((see[0] & see[1]) != 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!((see[q] >> e) & 1)) s[q][e] = 0xff800000u;
        }
        float big[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                big[e / 2 & 3] = fmaxf(fmaxf(big[e / 2 & 3], __uint_as_float(s[q][e])),
                                       __uint_as_float(s[q][e + 1]));
        return fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
    }
    // The scores times f, which becomes 1.
    __device__ __forceinline__ void apart(float &f) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
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
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float a, b;
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[q][e]),
                                                  __uint_as_float(s[q][e + 1])), f2, t2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum[e / 2 & 1] = add_f32x2(sum[e / 2 & 1], pack_f32x2(a, b));
                s[q][e / 2] = pack2<I>(a, b);
            }
            tmem_st16(s_tm + q * 16, s[q]);
        }
        float a, b;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), a, b);
        return a + b;
    }
};

// A loading warp's 32 positions of a tile: where they are in the cache.
struct Place {
    int block;                    // -1: no row sees it, -2: it is not there
    uint32_t unit;                // 16-byte units from the block's begin
};

template <int T, int KIND, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(PagedAttnParams P, FastDiv by_page, int vec) {
    using C_ = Tc<DP>;
    constexpr int I = KIND ? 2 : T;                              // the operands' type
    constexpr int kType = I == 1 ? 1 : 0;                        // of the descriptors
    constexpr int RT = kPagedTcRows, KS = DP / 16, kEsz = KIND ? 1 : 2;
    constexpr bool kScaleQ = T == 1 && I == 2;
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Words &W = *reinterpret_cast<Words *>(smem + C_::kSmall);
    const uint32_t base = smem_addr(smem);
    const spec_kv_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        bar_init(&W.q_full, kQuery);
        bar_init(&W.q_free, 2);
        for (int i = 0; i < kRing; ++i) {
            bar_init(&W.full[i], kLoad / 2);
            bar_init(&W.free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&W.drain[i], 1);
            bar_init(&W.s_full[i], 1);
            bar_init(&W.o_full[i], 1);
            bar_init(&W.o_last[i], 1);
            for (int j = 0; j < 2; ++j) bar_init(&W.p_full[i][j], 128);
        }
        for (int i = 0; i < 8; ++i) W.odd[i] = 0;
#ifdef SPEC_DEBUG
        W.gave_up = P.lose;
#else
        W.gave_up = 0;
#endif
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&W.tmem, C_::kColumns);
    paged_status(P, kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = W.tmem;
    volatile int *gave_up = &W.gave_up;
    // tensor memory of softmax group m: S (and P over it) at 128 m, O behind both groups'
    auto s_at = [&](int m) { return tmem + 128 * m; };
    auto o_at = [&](int m) { return tmem + 256 + DP * m; };
    // tiles of K and V take the ring's places in turn: K of tile c is the 2c-th, V the next
    auto slot = [](uint32_t x) { return x % kRing; };
    auto phase = [](uint32_t x) { return (x / kRing) & 1; };
    uint32_t done = 0, parts = 0;     // tiles before this part; parts with any: the phases count them
    PagedPart A;

    // Launched with 96 registers a thread, 20 warps: 8 x 136 + 8 x 72 + 4 x 64 = 20 x 96.
    if (tid >= kSoftmax + kLoad) {
        fewer_registers<64>();
        PagedWalk<RT> walk(P, kTcFixed, (int64_t)P.G * kPosTile);
        const int m = warp - kMmaWarp;
        if (m < 2) {
            // ---- multiply, for softmax group m. The whole warp runs the loop and waits, one
            // thread of it issues: what the products are given is then the same in all of the warp.
            const bool lead = elect_one();
            const uint32_t o = o_at(m), s = s_at(m);
            uint32_t mine = 0;           // tiles of this group before this one
            bool ok = true;
            while (ok && walk.next(P, A)) {
                const int n = A.stop - A.tile;
                if (n == 0) continue;
                ok = warp_wait(&W.q_full, parts & 1, gave_up);
                tc_fence_after();
                if (m == 1 && A.rows <= 128) {
                    // no rows for this group. The tiles are there, so their places' earlier phases
                    // are over, and these arrivals count for the right ones.
                    for (int i = 0; ok && i < 2 * n; ++i) {
                        const uint32_t x = 2 * done + i;
                        ok = warp_wait(&W.full[slot(x)], phase(x), gave_up);
                        if (ok && lead) bar_arrive(&W.free[slot(x)]);
                        __syncwarp();
                    }
                    if (ok && lead) bar_arrive(&W.q_free);
                    __syncwarp();
                    done += n;
                    ++parts;
                    continue;
                }
                auto scores = [&](int i) {
                    const uint32_t x = 2 * (done + i);
                    ok = ok && warp_wait(&W.full[slot(x)], phase(x), gave_up);
                    if (!ok) return;              // no products of what did not come
                    const uint64_t a = smem_desc(base + m * C_::kOperand, 16, 1024);
                    const uint64_t k = smem_desc(base + C_::kTiles + slot(x) * C_::kOperand, 16, 1024);
                    if (lead) {
#pragma unroll
                        for (int d = 0; d < KS; ++d) {
                            const int off = (d >> 2) * (128 * 128) + (d & 3) * 32;
                            mma_ss(s, desc_plus(a, off), desc_plus(k, off),
                                   mma_desc(kType, 128, false), d > 0);
                        }
                        mma_commit(&W.s_full[m]);
                        mma_commit(&W.free[slot(x)]);
                        if (i == n - 1) mma_commit(&W.q_free);
                    }
                    __syncwarp();
                };
                scores(0);
                for (int i = 0; ok && i < n; ++i) {
                    const uint32_t x = 2 * (done + i) + 1;
                    ok = warp_wait(&W.full[slot(x)], phase(x), gave_up);
                    const uint64_t v = smem_desc(base + C_::kTiles + slot(x) * C_::kOperand,
                                                 128 * 128, 1024);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && warp_wait(&W.p_full[m][h], mine & 1, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        if (lead) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ts(o, s + h * 64 + k * 8, desc_plus(v, (h * 4 + k) * 2048),
                                       mma_desc(kType, DP, true), i > 0 || h > 0 || k > 0);
                            mma_commit(&W.o_full[m]);
                            if (h == 1) {
                                if (i == n - 1) mma_commit(&W.o_last[m]);
                                mma_commit(&W.free[slot(x)]);
                            }
                        }
                        __syncwarp();
                    }
                    ++mine;
                    if (ok && i + 1 < n) scores(i + 1);
                }
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
        } else {
            // ---- queries: the D / 8 chunks of a row side by side, rows past the item's zeros ----
            const int t = tid - (kSoftmax + kLoad + 64);
            bool go = true;
            while (walk.next(P, A)) {
                if (A.stop == A.tile) continue;
                go = go && warp_wait(&W.q_free, (parts & 1) ^ 1, gave_up);
                if (go) {
                    const int64_t row0 = (int64_t)A.r * RT;
                    const int chunks = C.D / 8;
                    constexpr int J = DP / 8;
                    for (int i = t; i < RT * J; i += kQuery) {
                        const int r = i / J, j = i - r * J;
                        const uint32_t to = (r >> 7) * C_::kOperand + chunk_at(r & 127, j);
                        const bool in = r < A.rows && j < chunks;
                        const int64_t k = row0 + (in ? r : 0), n = k / P.G;
                        const unsigned short *from =
                            reinterpret_cast<const unsigned short *>(P.q) +
                            (A.req.first + n) * P.q_stride +
                            ((int64_t)A.head * P.G + (k - n * P.G)) * C.D + (in ? j * 8 : 0);
                        if (vec) {
                            copy16(base + to, from, in);
                        } else {
                            uint32_t w[4] = {0, 0, 0, 0};
                            if (in) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = (uint32_t)__ldg(from + 2 * e) |
                                           (uint32_t)__ldg(from + 2 * e + 1) << 16;
                            }
                            *reinterpret_cast<uint4 *>(smem + to) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if (kScaleQ) {
                        // each thread the chunks it brought, a row's beside each other in its warp
                        for (int i = t; i < RT * J; i += kQuery) {
                            const int r = i / J, j = i - r * J;
                            uint4 *at = reinterpret_cast<uint4 *>(
                                smem + (r >> 7) * C_::kOperand + chunk_at(r & 127, j));
                            uint32_t w[4] = {at->x, at->y, at->z, at->w};
                            float big = 0.f;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float a = fabsf(value16<T>((w[e / 2] >> (e % 2 * 16)) & 0xffffu));
                                if (a < INFINITY) big = fmaxf(big, a);
                            }
#pragma unroll
                            for (int o = J / 2; o > 0; o >>= 1)
                                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                            // into [2^14, 2^15), by 2^126 at most
                            const uint32_t ex = max(__float_as_uint(big) >> 23, 15u);
                            const float up = __uint_as_float((268u - ex) << 23);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2<2>(value16<T>(w[e] & 0xffffu) * up,
                                                value16<T>(w[e] >> 16) * up);
                            *at = make_uint4(w[0], w[1], w[2], w[3]);
                            if (j == 0)
                                W.q_down[parts & 1][r] = (unsigned short)((ex - 14u) << 7);
                        }
                    }
                    fence_async_smem();
                    bar_arrive(&W.q_full);
                }
                ++parts;
            }
        }
    } else if (tid >= kSoftmax) {
        fewer_registers<72>();
        // ---- load: K or V, 32 positions a warp ----
        PagedWalk<RT> walk(P, kTcFixed, (int64_t)P.G * kPosTile);
        const bool of_v = tid >= kSoftmax + kLoad / 2;
        const int w4 = (tid - kSoftmax) % (kLoad / 2) / 32;
        const char *cache = static_cast<const char *>(of_v ? C.v : C.k);
        const int64_t stride = (of_v ? C.v_block_stride : C.k_block_stride) * kEsz;
        const int units = C.D * kEsz / 16;                       // of a position in the cache
        constexpr int U = DP * kEsz / 16;                        // ... in the operand's width
        bool go = true;               // no wait has given up
        while (walk.next(P, A)) {
            const int n = A.stop - A.tile;
            if (n == 0) continue;
            auto page = [&](int i) -> int {
                const int p = i < n ? A.position(A.tile + i) + w4 * 32 + lane : A.hi;
                if (p >= A.hi || (p < A.lo && p >= P.sinks)) return -1;
                const int block = paged_page(P, by_page, A.b, p);
                return block >= 0 && block < C.num_blocks ? block : -2;
            };
            auto unit = [&](int i) -> uint32_t {
                const int p = A.position(A.tile + i) + w4 * 32 + lane;
                const uint32_t off = p - by_page((uint32_t)p) * C.block_size;
                return (C.layout == SPEC_KV_NHD ? off * C.H + A.head : A.head * C.block_size + off) *
                       units;
            };
            // where chunk u of the warp's position t is
            auto source = [&](int block, uint32_t in, int t, int u, bool &ok) -> const char * {
                const int blk = __shfl_sync(0xffffffffu, block, t);
                const uint32_t from = __shfl_sync(0xffffffffu, in, t) + u;
                ok = blk >= 0 && u < units;
                return cache + (ok ? blk * stride + (int64_t)from * 16 : 0);
            };
            // Tile i has come to its place: what the rows see in part is looked through.
            auto arrived = [&](int i) {
                const uint32_t x = 2 * (done + i) + of_v;
                if (of_v && !all_see(P, A, A.position(A.tile + i), kPosTile)) {
                    char *to = smem + C_::kTiles + slot(x) * C_::kOperand;
                    bool odd = false;
                    constexpr int J = DP / 8;
#pragma unroll 4
                    for (int q = lane; q < 32 * J; q += 32) {
                        uint4 *at = reinterpret_cast<uint4 *>(to + chunk_at(w4 * 32 + q / J, q % J));
                        const uint4 y = *at;
                        if (!(odd_word<I, 0>(y.x) | odd_word<I, 0>(y.y) | odd_word<I, 0>(y.z) |
                              odd_word<I, 0>(y.w)))
                            continue;
                        odd = true;
                        uint32_t w[4] = {y.x, y.y, y.z, y.w};
                        constexpr uint32_t ex = I == 1 ? 0x7f80u : 0x7c00u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((w[e] & ex) == ex) w[e] &= 0xffff0000u;
                            if ((w[e] >> 16 & ex) == ex) w[e] &= 0xffffu;
                        }
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (odd) W.odd[parts & 7] = 1;
                }
                fence_async_smem();
                bar_arrive(&W.full[slot(x)]);
            };
            auto note = [&](int i, int block) {      // K's warps: which positions are there
                if (block == -2 && P.status) atomicMax(P.status + A.b, SPEC_REQ_BAD_SLOT);
                const unsigned seen = __ballot_sync(0xffffffffu, block >= 0);
                if (!of_v && lane == 0) W.seen[(done + i) & 3][w4] = seen;
            };
            if (of_v && lane == 0 && w4 == 0) W.odd[(parts + 4) & 7] = 0;
            if constexpr (KIND == 0) {
                int next = page(0);
                for (int i = 0; i <= n; ++i) {
                    const int block = next;
                    next = page(i + 1);
                    if (i < n) {
                        const uint32_t x = 2 * (done + i) + of_v;
                        go = go && warp_wait(&W.free[slot(x)], phase(x) ^ 1, gave_up);
                        if (go) {
                            note(i, block);
                            const uint32_t to = base + C_::kTiles + slot(x) * C_::kOperand;
                            const uint32_t in = unit(i);
#pragma unroll
                            for (int q = 0; q < U; ++q) {
                                const int t = (q * 32 + lane) / U, u = lane % U;
                                bool ok;
                                const char *from = source(block, in, t, u, ok);
                                copy16(to + chunk_at(w4 * 32 + t, u), from, ok);
                            }
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (i > 0) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        __syncwarp();     // the warp's copies, all lanes'
                        if (go) arrived(i - 1);
                    }
                }
            } else {
                // a tile's codes wait in registers for its place
                constexpr int Q = U;                          // chunks of a thread
                uint4 y[Q];
                int block = page(0), next = page(1);
                auto fetch = [&](int i, int blk) {
                    const uint32_t in = unit(i);
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        bool ok;
                        const char *from = source(blk, in, (q * 32 + lane) / U, lane % U, ok);
                        y[q] = ok ? __ldg(reinterpret_cast<const uint4 *>(from)) : make_uint4(0, 0, 0, 0);
                    }
                };
                fetch(0, block);
                for (int i = 0; i < n; ++i) {
                    const uint32_t x = 2 * (done + i) + of_v;
                    go = go && warp_wait(&W.free[slot(x)], phase(x) ^ 1, gave_up);
                    if (go) {
                        note(i, block);
                        char *to = smem + C_::kTiles + slot(x) * C_::kOperand;
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            const int t = (q * 32 + lane) / U, u = lane % U;
                            const uint32_t w[4] = {y[q].x, y[q].y, y[q].z, y[q].w};
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                *reinterpret_cast<uint4 *>(to + chunk_at(w4 * 32 + t, 2 * u + h)) =
                                    make_uint4(halves2<KIND>(w[2 * h]), halves2<KIND>(w[2 * h] >> 16),
                                               halves2<KIND>(w[2 * h + 1]),
                                               halves2<KIND>(w[2 * h + 1] >> 16));
                        }
                        __syncwarp();
                        arrived(i);
                    }
                    block = next;
                    next = page(i + 2);
                    if (i + 1 < n) fetch(i + 1, block);
                }
            }
            done += n;
            ++parts;
        }
    } else {
        more_registers<136>();
        // ---- softmax: this thread's row. A wait that gives up is followed by none.
        PagedWalk<RT> walk(P, kTcFixed, (int64_t)P.G * kPosTile);
        const int m = warp >> 2;
        const int r = m * 128 + (warp & 3) * 32 + lane;          // of the item
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_tm = o_at(m) + lanes, s_tm = s_at(m) + lanes;
        const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
        const float unit = P.scale * kLog2e * (C.k_scale ? __ldg(C.k_scale) : 1.f);
        uint32_t mine = 0, results = 0;   // tiles of this group so far; parts
        bool go = true, any = false;
        while (walk.next(P, A)) {
            any = true;
            const int n = A.stop - A.tile;
            const int64_t row0 = (int64_t)A.r * RT;
            const bool live = r < A.rows, work = n > 0 && m * 128 < A.rows;
            const bool warp_live = m * 128 + (warp & 3) * 32 < A.rows;
            const int64_t token = (row0 + min(r, A.rows - 1)) / P.G;
            const int64_t most = (int64_t)C.max_blocks * C.block_size;
            const int at = (int)min(max(A.req.pos + token, (int64_t)-1), most);
            // top: the row's reference; limit: what raises it, or calls for apart()
            float top = kPagedNoMax, limit = -INFINITY, sum = 0.f, factor = 0.f;
            for (int i = 0; work && i < n; ++i, ++mine) {
                go = go && warp_wait(&W.s_full[m], mine & 1, gave_up);
                if (!go) break;
                tc_fence_after();
                if (i == 0)
                    factor = paged_factor(
                        kScaleQ ? unit * __uint_as_float((uint32_t)W.q_down[parts & 1][r] << 16) : unit);
                const int j0 = A.position(A.tile + i);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (warp_live) {
                        unsigned see[2] = {W.seen[(done + i) & 3][2 * h],
                                           W.seen[(done + i) & 3][2 * h + 1]};
                        if (!all_see(P, A, j0 + 64 * h, 64)) {
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                see[q] &= paged_bits(j0 + 64 * h + 32 * q, at, A.hi, P.window, P.sinks);
                        }
                        Scores<I> tile;
                        float f = factor;
                        const float x = fmaxf(kPagedNoMax, tile.load(s_tm + 64 * h, see) * f);
                        if (__any_sync(0xffffffffu, x > limit)) {
                            const float to = paged_reference(top, x), a = ex2(top - to);
                            top = to;
                            sum *= a;
                            limit = paged_limit(top);
                            if (fabsf(top) > kApart) {
                                limit = -INFINITY;      // and so for each tile to come
                                tile.apart(f);
                            }
                            // O so far: the product of the first half may be under way; the
                            // scores at hand were made after those before
                            if (i > 0 || h > 0) {
                                if (h > 0) go = go && warp_wait(&W.o_full[m], 0, gave_up);
                                tc_fence_after();
#pragma unroll 1
                                for (int q = 0; q < DP / 16; ++q) {   // S stays in registers meanwhile
                                    uint32_t o[16];
                                    tmem_ld16(o_tm + q * 16, o);
                                    tmem_wait_ld16(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                    tmem_st16(o_tm + q * 16, o);
                                }
                            }
                        }
                        sum += tile.store(s_tm + 64 * h, f, top);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    bar_arrive(&W.p_full[m][h]);
                }
            }
            // The result: O is done after the group's last product.
            if (work) go = go && warp_wait(&W.o_last[m], results++ & 1, gave_up);
            tc_fence_after();
            if (!go) {      // lost: a sum of NaN makes the rows of this part NaN, and the item's
                sum = NAN;
                if (P.status && lane == 0) atomicMax(P.status + A.b, SPEC_REQ_INTERNAL);
            }
            const bool whole = A.whole();
            const float norm = (whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f) * v_scale;
            const int64_t to = live ? paged_row(P, A.req, A.head, row0 + r) : 0;
            float *part = paged_slot(P, blockIdx.x, A.begins, RT, DP);
            const bool out32 = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
            const bool odd = n > 0 && *(volatile int *)&W.odd[parts & 7] != 0;
            for (int q = 0; warp_live && q < DP / 32; ++q) {
                float v[32];
                __syncwarp();
                if (work && go) {
                    uint32_t o[32];
                    tmem_ld32(o_tm + q * 32, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * norm;
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = sum == sum ? 0.f : NAN;
                }
                if (!live) continue;
                if (odd) {      // NaN and infinities of positions that this row sees
                    for (int i = A.tile; i < A.stop; ++i) {
                        const int j0 = A.position(i);
                        if (all_see(P, A, j0, kPosTile)) continue;
#pragma unroll 1
                        for (int j = j0; j < j0 + kPosTile; ++j) {
                            if (!(paged_bits(j, at, A.hi, P.window, P.sinks) & 1)) continue;
                            const int block = paged_page(P, by_page, A.b, j);
                            if (block < 0 || block >= C.num_blocks) continue;
                            const uint32_t off = j - by_page((uint32_t)j) * C.block_size;
                            const int64_t e0 =
                                block * C.v_block_stride +
                                (int64_t)(C.layout == SPEC_KV_NHD ? off * C.H + A.head
                                                                  : A.head * C.block_size + off) * C.D;
#pragma unroll 1
                            for (int d = q * 32; d < min(q * 32 + 32, C.D); ++d) {
                                const float y =
                                    KIND ? value16<2>(halves2<KIND>(__ldg(static_cast<const uint8_t *>(C.v) +
                                                                         e0 + d)) & 0xffffu)
                                         : value16<I>(__ldg(static_cast<const unsigned short *>(C.v) + e0 + d));
                                if (fabsf(y) < INFINITY) continue;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (e == d - q * 32) v[e] += y;
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (q * 32 + h * 16 >= C.D) break;
                    if (whole && out32) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[k] = pack2<T>(v[h * 16 + 2 * k], v[h * 16 + 2 * k + 1]);
                        store32(reinterpret_cast<unsigned short *>(P.out) + to * C.D + q * 32 + h * 16, w);
                    } else if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            paged_store4<T>(P.out, to * C.D + q * 32 + h * 16 + e,
                                            make_float4(v[h * 16 + e], v[h * 16 + e + 1],
                                                        v[h * 16 + e + 2], v[h * 16 + e + 3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[h * 16 + e + k]);
                            store32(part + (int64_t)r * DP + q * 32 + h * 16 + e, w);
                        }
                    }
                }
            }
            if (live) {
                if (whole) {
                    if (P.lse) P.lse[to] = paged_lse(top, sum);
                } else {
                    part[RT * DP + r] = top;
                    part[RT * (DP + 1) + r] = sum;
                }
            }
            tc_fence_before();
            done += n;
            parts += n > 0;
        }
        if (tid == 0) paged_note(P, walk.range, A, any);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, C_::kColumns);
}

template <int T, int KIND, int DP>
cudaError_t launch(const PagedAttnParams &p, int grid, cudaStream_t st) {
    using C_ = Tc<DP>;
    const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<T, KIND, DP>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C_::kBytes);
    if (e != cudaSuccess) return e;
    const int vec = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.q_stride % 8 == 0;
    paged_tc_kernel<T, KIND, DP><<<grid, kThreads, C_::kBytes, st>>>(
        p, FastDiv((uint32_t)p.cache.block_size), vec);
    return cudaGetLastError();
}

}  // namespace

template <int T>
cudaError_t launch_paged_tc_type(const PagedAttnParams &p, int grid, cudaStream_t st) {
    const bool narrow = p.cache.D <= 64;
    if (p.cache.kind == SPEC_CACHE_SAME)
        return narrow ? launch<T, 0, 64>(p, grid, st) : launch<T, 0, 128>(p, grid, st);
    if (p.cache.kind == SPEC_CACHE_FP8_E4M3)
        return narrow ? launch<T, 1, 64>(p, grid, st) : launch<T, 1, 128>(p, grid, st);
    return narrow ? launch<T, 2, 64>(p, grid, st) : launch<T, 2, 128>(p, grid, st);
}

}  // namespace specv
