// Attention of new tokens over the paged cache for many query rows (prompts, chunks of them, mixed
// batches), on the tcgen05 tensor cores.
//
// The same operator as paged_few.cuh for items of up to 256 rows; the two products bound it, 4 D
// operations a row and position. One CTA an SM; its warps have one part each and meet at mbarriers
// only:
//
//   load     (4 warps for K, 4 for V) tiles of 128 positions to a ring of five places that K and V
//            share, laid out for the tensor core (128-byte swizzle; K contiguous along D, and V as it
//            is, read transposed): by TMA, a box of a page's rows at a time, where the warp's 32
//            positions are all wanted, else by asynchronous copies, whose addresses take any page
//            size. 8-bit codes pass through registers and become halves. An item's queries come
//            after its first tile, as soon as the scores of the item before are done;
//   multiply (2 warps, a thread of each issues for one softmax group) S = Q K^T for 128 rows and 64
//            positions, two of them in turn, and O += P V. Sums are in tensor memory: two S and an O
//            a group, all 512 columns at D = 128; P overwrites the S it came from;
//   softmax  (2 groups of 4 warps) S to P, a row a thread, no exchange between threads, reference
//            and sum in registers. The row's largest score is not looked for: a tile's sum tells
//            when one has passed the reference by too much. Then, which is rare, and for an item's
//            first tile, the scores are read again, the reference raised and O rescaled in place;
//   deal     (1 warp) the CTA's parts, one after another, as words in shared memory: up to four
//            ahead, so that the others neither compute them nor hold them in registers.
//
// While softmax works on one S, the tensor core multiplies with the P before and makes the next
// scores: with one S of 128 columns a group it had to wait for softmax, and softmax for it (2048 tokens
// after 60000: 1.96 ms against 1.54 at the time, and no less when the two groups took turns). The price
// is that a product of 64 columns reads 6 KB of shared memory for 32 clocks of work and gets 48: a
// tile's reads and writes take 2560 clocks, its products 2048. What is left is latency, that of a job of
// 64 positions from S to P and the meetings at its ends: issue slots are taken in 49% of the cycles, the
// tensor pipe is active in 51%, and no other pipe in more than 33%.
//
// 32 query and 8 K/V heads x 128: two prompts of 8192 and 5845 tokens 666 us, 1.25 PFLOP/s (63% of the
// measured cuBLAS rate) one call after another, where the power limit holds the SMs at 1.96 to 1.99 GHz;
// 636 us at 2.07 GHz, calls that stand alone. Over an e4m3 cache 976 us (the codes' way through
// registers); 2048 tokens after 60000 1.54 ms, 1.33 PFLOP/s; a window of 4096 with sinks 230 us, 1.0
// PFLOP/s (items of 35 tiles, two of them seen in part); D = 64 592 us, 0.70 PFLOP/s (softmax costs as
// much as at 128); D = 256, two of 4096 with 16 and 4 heads, 224 us, 0.93 PFLOP/s. Short prompts are far
// from that, since an item's queries, first scores and result overlap with no other item's: 32 of up to
// 512 tokens 125 us, 0.24 PFLOP/s, 128 of up to 100 103 us.
//
// Items of up to 128 rows (a decoding request in a mixed batch) leave the second group idle, and
// warps without a live row touch nothing: a tile then takes less time than its bytes do.
//
// What a row does not see: scores are replaced, never multiplied. A position that no row of the
// item sees is not read (zeros stand in its place). In tiles that some rows see in part, V is looked
// through; NaN and infinities are taken out of the products and added, at the end, to the rows that
// see them.
#pragma once

#include <cuda.h>

#include "paged_attn.cuh"
#include "tc_device.cuh"

namespace specv {
namespace {

constexpr int kLoad = 256;        // loading threads: K's, then V's
constexpr int kSoftmax = 256;     // threads of the two softmax groups
constexpr int kThreads = kSoftmax + kLoad + 128;   // the last warpgroup: two warps multiply
constexpr int kMmaWarp = (kSoftmax + kLoad) / 32;
constexpr int kRing = 5;
// What an item costs besides its keys, in positions, so that CTAs of many short items and of few long
// ones end together. Two prompts of 8192 and 5845 tokens took, with 256, 384, 448, 512:
//   D = 128, 16 bits    671, 637, 642, 646 us   (five of 3300 after 1000: 398, 384, 383, 385)
//   D = 128, 8 bits    1126, 987, 935, 918 us   (eight of 2000: 332, 309, 295, 300)
//   D = 64, 16 bits     598, 609, 607, 611 us   (192: 608)
//   D = 64, 8 bits      685, 646, 648, 654 us   (320: 644; eight of 2000: 201, 181, 177, 177; 32 of 512:
//                                                130, 124, 123, 121)
//   D = 256, two of 4096, 16 bits 230, 234, 237, 240 us; 8 bits 428, 441, 445 us.
template <int KIND, int DP>
constexpr int kTcFixed = DP == 256 ? 256 : KIND ? 448 : DP == 128 ? 384 : 256;

// D above 128: one softmax group and tiles of 64 positions, so that queries, ring and sums take the
// same room.
template <int DP>
struct Tc {
    static constexpr int kGroups = DP == 256 ? 1 : 2;            // of 128 rows
    static constexpr int kPos = DP == 256 ? 64 : 128;            // positions of a tile
    static constexpr int kQuery = 128 * DP * 2;                  // a group's queries, 16-bit elements
    static constexpr int kOperand = kPos * DP * 2;               // a tile of K or V
    static constexpr int kTiles = kGroups * kQuery;              // Q first, then the ring
    static constexpr int kSmall = kTiles + kRing * kOperand;     // barriers and words
    static constexpr int kBytes = kSmall + 2048 + 1024;          // and room to align by 1024
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static constexpr int kColumns = 512;                         // groups x (128 + DP), a power of two
    static constexpr int kReaders = 8 + 5 * kGroups;             // warps that read a part
};

// A part as the warps read it (see PagedPart); b -1: there are no more.
struct PartWords {
    int b, r, head, first, pos, rows;
    uint32_t e0, e1;
    int lo, hi, skip, base, tile, stop, begins, ends;

    template <int PT>
    __device__ __forceinline__ int position(int i) const {
        return (i < skip ? i : base + i) * PT;
    }
};
constexpr int kDealt = 4;
constexpr int kOdd = 16;

struct Words {
    PartWords part[kDealt];
    uint64_t part_full[kDealt], part_free[kDealt];
    uint64_t q_full, q_free, full[kRing], free[kRing], drain[2];
    uint64_t s_full[2][2], p_full[2][2], o_full[2];              // of a softmax group; its two S
    uint64_t o_last[2];                                          // once a part
    // Positions of a tile that are there. K's loader writes a tile's words again for the fourth
    // after it, whose place was that of a V whose products are done.
    alignas(16) unsigned seen[4][4];
    // A part's V has NaN or infinities that not every row sees. V's first loading warp clears the word
    // of the eighth part to come. When it comes to part k, the place of part k - 1's V was given back by
    // K of two tiles earlier, of part k - 3 at the earliest; those products follow part k - 4's, whose
    // word softmax may be about to read. V's other warps are three tiles ahead at most.
    int odd[kOdd];
    uint32_t tmem;
    int gave_up;
    // 1 / the power of two of each row of Q: a float's upper half. Of two parts: a part of one tile
    // may be read while the next one's queries come.
    unsigned short q_down[2][256];
};
static_assert(sizeof(Words) <= 2048, "room for the words");

// Byte of 16-byte chunk `j` of row r of an operand of R rows.
template <int R>
__device__ __forceinline__ uint32_t chunk_at(int r, int j) {
    return (uint32_t)(j >> 3) * (R * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4);
}

// A wait of a whole warp: all of it goes on or none. And an arrival for what all its lanes have done.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gave_up));
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(bar);
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void *to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The reference of a row comes from a rounded product f s, within 2^-24 of it, which f s - top in
// one rounding brings to light: as 2^-4 at most up to scores of 2^20, beyond as more than a half
// holds. There the products are rounded alike first.
constexpr float kApart = 1048576.f;

constexpr int kHalf = 64 * 128;   // bytes from the first 64 rows of an operand to the others

// What the sum of 64 probabilities may come to without its largest being looked for.
constexpr float kMost = 32768.f;

// 32 scores of a row to probabilities 2^(f s - top), packed; returns their sum.
template <int I>
__device__ __forceinline__ uint64_t probabilities(uint32_t (&s)[32], float f, float top, uint64_t sum) {
    const uint64_t f2 = pack_f32x2(f, f), t2 = pack_f32x2(-top, -top);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float a, b;
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f2, t2), a,
                     b);
        a = ex2(a);
        b = ex2(b);
        sum = add_f32x2(sum, pack_f32x2(a, b));
        s[e / 2] = pack2<I>(a, b);
    }
    return sum;
}
__device__ __forceinline__ float largest32(const uint32_t (&s)[32]) {
    float big[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 2)
        big[e / 2 & 1] =
            fmaxf(fmaxf(big[e / 2 & 1], __uint_as_float(s[e])), __uint_as_float(s[e + 1]));
    return fmaxf(big[0], big[1]);
}

// TMA: a box of a tensor to shared memory; `bar` counts its bytes.
__device__ __forceinline__ void tma_box3(uint32_t to, const CUtensorMap *map, int x, int c1, int c2,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(to),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t to, const CUtensorMap *map, int x, int c1, int c2,
                                        int block, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5}], [%6];" ::"r"(to),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(block), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, int bytes) {      // and arrives
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}

// Tensor maps of the cache and the queries (16-bit caches), and their boxes' rows: positions of a
// page, tokens (0: no map).
struct Maps {
    CUtensorMap k, v, q;
    int page_rows, tokens;
};

template <int T, int KIND, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(PagedAttnParams P, int vec, const __grid_constant__ Maps maps) {
    using C_ = Tc<DP>;
    constexpr int I = KIND ? 2 : T;                              // the operands' type
    constexpr int kType = I == 1 ? 1 : 0;                        // of the descriptors
    constexpr int NG = C_::kGroups, RT = 128 * NG, PT = C_::kPos, KS = DP / 16, kEsz = KIND ? 1 : 2;
    constexpr int HALVES = PT / 64;                              // jobs of a tile
    static_assert(RT == paged_tc_rows(DP), "rows of an item");
    constexpr bool kScaleQ = T == 1 && I == 2;
    const int box = KIND ? 0 : maps.page_rows;
    extern __shared__ char raw[];
    char *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Words &W = *reinterpret_cast<Words *>(smem + C_::kSmall);
    const uint32_t base = smem_addr(smem);
    const spec_kv_cache &C = P.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        bar_init(&W.q_full, KIND == 0 && maps.tokens > 0 ? 1 : kLoad / 32);
        bar_init(&W.q_free, NG);
        for (int i = 0; i < kRing; ++i) {
            bar_init(&W.full[i], kLoad / 64);
            bar_init(&W.free[i], NG);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&W.drain[i], 1);
            bar_init(&W.o_full[i], 1);
            bar_init(&W.o_last[i], 1);
            for (int j = 0; j < 2; ++j) {
                bar_init(&W.s_full[i][j], 1);
                bar_init(&W.p_full[i][j], 4);
            }
        }
        for (int i = 0; i < kDealt; ++i) {
            bar_init(&W.part_full[i], 1);
            bar_init(&W.part_free[i], C_::kReaders);
        }
        for (int i = 0; i < kOdd; ++i) W.odd[i] = 0;
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
    // tensor memory of softmax group m: two S of 64 columns (and P over each) at 128 m, O behind both
    // groups'
    auto s_at = [&](int m) { return tmem + 128 * m; };
    auto o_at = [&](int m) { return tmem + 128 * NG + DP * m; };
    // tiles of K and V take the ring's places in turn: K of tile c is the 2c-th, V the next
    auto slot = [](uint32_t x) { return x % kRing; };
    auto phase = [](uint32_t x) { return (x / kRing) & 1; };
    uint32_t done = 0, parts = 0;     // tiles before this part; parts with any: the phases count them
    // the words of the x-th part dealt, once they are there, and when this warp has read them
    auto dealt = [&](uint32_t x) { return warp_wait(&W.part_full[x % kDealt], x / kDealt & 1, gave_up); };
    auto read = [&](uint32_t x) { warp_arrive(&W.part_free[x % kDealt]); };

    // Launched with 96 registers a thread, 20 warps: 8 x 128 + 8 x 88 + 4 x 48 = 20 x 96.
    if (tid >= kSoftmax + kLoad) {
        fewer_registers<48>();
        const int m = warp - kMmaWarp;
        if (m == 2) {
            // ---- deal ----
            PagedWalk<RT, PT> walk(P, kTcFixed<KIND, DP>, (int64_t)P.G * kPosTile);
            PagedPart A;
            bool any = false, go = true;
            for (uint32_t x = 0;; ++x) {
                const bool more = walk.next(P, A);
                go = go && warp_wait(&W.part_free[x % kDealt], (x / kDealt & 1) ^ 1, gave_up);
                if (go && lane == 0) {
                    PartWords &w = W.part[x % kDealt];
                    w = PartWords{more ? A.b : -1, A.r, A.head, A.req.first, A.req.pos, A.rows, A.e0,
                                  A.e1, A.lo, A.hi, A.skip, A.base, A.tile, A.stop, A.begins, A.ends};
                    bar_arrive(&W.part_full[x % kDealt]);
                }
                __syncwarp();
                if (!more) break;
                any = true;
            }
            if (lane == 0) paged_note(P, walk.range, A, RT, any);
        } else if (m < NG) {
            // ---- multiply, for softmax group m. The whole warp runs the loop and waits, one
            // thread of it issues: what the products are given is then the same in all of the warp.
            const bool lead = elect_one();
            const uint32_t o = o_at(m), s = s_at(m);
            uint32_t jobs = 0;           // of this group before this part; a job is 64 positions
            bool ok = true;
            for (uint32_t part = 0;; ++part) {
                ok = ok && dealt(part);
                if (!ok) break;
                const PartWords &A = W.part[part % kDealt];
                const int n = A.stop - A.tile, rows = A.rows, b = A.b;
                read(part);
                if (b < 0) break;
                if (n == 0) continue;
                ok = warp_wait(&W.q_full, parts & 1, gave_up);
                tc_fence_after();
                if (m == 1 && rows <= 128) {
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
                // Places of K of tile i and V of tile i, and the words that follow from them: this warp's
                // own instructions are what a job waits for longest, so they are kept few.
                uint32_t kx = 2 * done, vx = kx + 1;
                const uint64_t q_desc = smem_desc(base + m * C_::kQuery, 16, 1024);
                const uint64_t k0 = smem_desc(base + C_::kTiles, 16, 1024);
                const uint64_t v0 = smem_desc(base + C_::kTiles, PT * 128, 1024);
                uint32_t ks = slot(kx), vs = slot(vx);
                // S of half `half` of the next tile of K
                auto scores = [&](int half, uint32_t buf, bool last) {
                    if (half == 0)                // a tile's second half came with its first
                        ok = ok && warp_wait(&W.full[ks], phase(kx), gave_up);
                    if (!ok) return;              // no products of what did not come
                    if (lead) {
                        const uint64_t k = desc_plus(k0 + ks * (C_::kOperand >> 4), half * kHalf);
#pragma unroll
                        for (int d = 0; d < KS; ++d) {
                            const int in = (d & 3) * 32;
                            mma_ss(s + buf * 64, desc_plus(q_desc, (d >> 2) * (128 * 128) + in),
                                   desc_plus(k, (d >> 2) * (PT * 128) + in),
                                   mma_desc(kType, 64, false), d > 0);
                        }
                        mma_commit(&W.s_full[m][buf]);
                        if (half == HALVES - 1) mma_commit(&W.free[ks]);
                        if (last && half == HALVES - 1) mma_commit(&W.q_free);
                    }
                    __syncwarp();
                    if (half == HALVES - 1) {
                        kx += 2;
                        ks = ks + 2 >= kRing ? ks + 2 - kRing : ks + 2;
                    }
                };
                // O of half `half` of the next tile of V; job: of the part
                auto values = [&](int half, uint32_t buf, int job) {
                    if (half == 0) ok = warp_wait(&W.full[vs], phase(vx), gave_up);
                    ok = ok && warp_wait(&W.p_full[m][buf], (jobs + job) >> 1 & 1, gave_up);
                    if (!ok) return;
                    tc_fence_after();
                    if (lead) {
                        const uint64_t v = desc_plus(v0 + vs * (C_::kOperand >> 4), half * kHalf);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ts(o, s + buf * 64 + k * 8, desc_plus(v, k * 2048),
                                   mma_desc(kType, DP, true), job > 0 || k > 0);
                        mma_commit(&W.o_full[m]);
                        if (job == HALVES * n - 1) mma_commit(&W.o_last[m]);
                        if (half == HALVES - 1) mma_commit(&W.free[vs]);
                    }
                    __syncwarp();
                    if (half == HALVES - 1) {
                        vx += 2;
                        vs = vs + 2 >= kRing ? vs + 2 - kRing : vs + 2;
                    }
                };
                const int count = HALVES * n;
                if constexpr (HALVES == 2) {      // jobs are even here: a half has its S
                    scores(0, 0, n == 1);
                    scores(1, 1, n == 1);
                    for (int i = 0; ok && i < n; ++i) {
                        values(0, 0, 2 * i);
                        if (ok && i + 1 < n) scores(0, 0, i + 2 == n);
                        if (ok) values(1, 1, 2 * i + 1);
                        if (ok && i + 1 < n) scores(1, 1, i + 2 == n);
                    }
                } else {
                    scores(0, jobs & 1, n == 1);
                    if (n > 1) scores(0, (jobs + 1) & 1, n == 2);
                    for (int i = 0; ok && i < n; ++i) {
                        values(0, (jobs + i) & 1, i);
                        if (ok && i + 2 < n) scores(0, (jobs + i) & 1, i + 3 == n);
                    }
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
        // ---- load: K or V, PW positions a warp ----
        constexpr int PW = PT / 4;
        constexpr unsigned kMine = 0xffffffffu >> (32 - PW);
        const bool of_v = tid >= kSoftmax + kLoad / 2;
        const int w4 = (tid - kSoftmax) % (kLoad / 2) / 32;
        const char *cache = static_cast<const char *>(of_v ? C.v : C.k);
        const int64_t stride = (of_v ? C.v_block_stride : C.k_block_stride) * kEsz;
        const int units = C.D * kEsz / 16;                       // of a position in the cache
        constexpr int U = DP * kEsz / 16;                        // ... in the operand's width
        bool go = true;               // no wait has given up
        for (uint32_t part = 0;; ++part) {
            go = go && dealt(part);
            if (!go) break;
            const PartWords &A = W.part[part % kDealt];      // until read(part)
            const int n = A.stop - A.tile;
            if (A.b < 0) break;
            if (n == 0) {
                read(part);
                continue;
            }
            auto page = [&](int i) -> int {
                const int p = i < n && lane < PW ? A.position<PT>(A.tile + i) + w4 * PW + lane : A.hi;
                if (p >= A.hi || (p < A.lo && p >= P.sinks)) return -1;
                const int block = paged_page(P, A.b, p);
                return block >= 0 && block < C.num_blocks ? block : -2;
            };
            auto unit = [&](int i) -> uint32_t {
                const int p = A.position<PT>(A.tile + i) + w4 * PW + lane;
                const uint32_t off = p - P.by_page((uint32_t)p) * C.block_size;
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
                if (of_v && !all_see(P, A.e0, A.e1, A.position<PT>(A.tile + i), PT)) {
                    char *to = smem + C_::kTiles + slot(x) * C_::kOperand;
                    bool odd = false;
                    constexpr int J = DP / 8;
#pragma unroll 4
                    for (int q = lane; q < PW * J; q += 32) {
                        uint4 *at = reinterpret_cast<uint4 *>(to + chunk_at<PT>(w4 * PW + q / J, q % J));
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
                    if (odd) W.odd[parts % kOdd] = 1;
                }
                fence_async_smem();
                warp_arrive(&W.full[slot(x)]);
            };
            auto note = [&](int i, int block) {      // K's warps: which positions are there
                if (block == -2 && P.status) atomicMax(P.status + A.b, SPEC_REQ_BAD_SLOT);
                const unsigned seen = __ballot_sync(0xffffffffu, block >= 0);
                if (!of_v && lane == 0) {
                    if (PW == 32) W.seen[(done + i) & 3][w4] = seen;
                    else reinterpret_cast<unsigned short *>(W.seen[(done + i) & 3])[w4] = (unsigned short)seen;
                }
            };
            // The item's rows, the D / 8 chunks of a row side by side, rows past the item's zeros:
            // issued by all loading threads, and (with the first tile) waited for.
            auto queries = [&] {
                constexpr int J = DP / 8;
                const int row0 = A.r * RT, chunks = C.D / 8, t = tid - kSoftmax;
                if (KIND == 0 && maps.tokens > 0) {
                    // by TMA: boxes of 128 rows and 64 columns. Rows past the item's may be another
                    // request's or no request's: their results go nowhere, and nothing depends on them.
                    if (of_v || w4 != 0) return;
                    go = go && warp_wait(&W.q_free, (parts & 1) ^ 1, gave_up);
                    const int halves = NG > 1 && A.rows > 128 ? 2 : 1, token = A.first + (int)P.by_group((uint32_t)row0);
                    if (go && lane == 0) bar_expect(&W.q_full, halves * C_::kQuery);
                    __syncwarp();
                    const int m = lane / (DP / 64), q = lane % (DP / 64);
                    if (go && m < halves)
                        tma_box3(base + m * C_::kQuery + q * (128 * 128), &maps.q, q * 64,
                                 A.head * P.G, token + m * maps.tokens, &W.q_full);
                    return;
                }
                go = go && warp_wait(&W.q_free, (parts & 1) ^ 1, gave_up);
                if (go) {
#pragma unroll 4
                    for (int i = t; i < RT * J; i += kLoad) {
                        const int r = i / J, j = i - r * J;
                        const uint32_t to = (r >> 7) * C_::kQuery + chunk_at<128>(r & 127, j);
                        const bool in = r < A.rows && j < chunks;
                        const unsigned short *from =
                            paged_query(P, A.first, A.head, row0 + (in ? r : 0)) + (in ? j * 8 : 0);
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
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (kScaleQ && go) {
                    // each thread the chunks it brought, a row's beside each other in its warp
#pragma unroll 4
                    for (int i = t; i < RT * J; i += kLoad) {
                        const int r = i / J, j = i - r * J;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + (r >> 7) * C_::kQuery +
                                                              chunk_at<128>(r & 127, j));
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
                            w[e] = pack2<2>(value16<T>(w[e] & 0xffffu) * up, value16<T>(w[e] >> 16) * up);
                        *at = make_uint4(w[0], w[1], w[2], w[3]);
                        if (j == 0) W.q_down[parts & 1][r] = (unsigned short)((ex - 14u) << 7);
                    }
                }
                fence_async_smem();
                if (go) warp_arrive(&W.q_full);
            };
            if (of_v && lane == 0 && w4 == 0) W.odd[(parts + kOdd / 2) % kOdd] = 0;
            if constexpr (KIND == 0) {
                int next = page(0), pending = -1;     // a tile whose copies are waited for later
                auto settle = [&](bool behind) {
                    if (pending < 0) return;
                    if (behind) asm volatile("cp.async.wait_group 1;" ::: "memory");
                    else asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();     // the warp's copies, all lanes'
                    if (go) arrived(pending);
                    pending = -1;
                };
                for (int i = 0; i < n; ++i) {
                    const int block = next;
                    next = page(i + 1);
                    const uint32_t x = 2 * (done + i) + of_v;
                    go = go && warp_wait(&W.free[slot(x)], phase(x) ^ 1, gave_up);
                    const int j0 = A.position<PT>(A.tile + i);
                    const uint32_t place = C_::kTiles + slot(x) * C_::kOperand + w4 * (PW * 128);
                    const unsigned wanted = __ballot_sync(0xffffffffu, block >= 0);
                    // Of K what is not wanted may be anything; of V it has to be zeros, and what some
                    // rows alone see is looked through.
                    if (go && box > 0 &&
                        (!of_v || (wanted == kMine && all_see(P, A.e0, A.e1, j0, PT)))) {
                        // `box` rows of a page a time (they divide PW and the page), 64 columns
                        note(i, block);
                        const int g = lane / (DP / 64), q = lane % (DP / 64), t = g * box;
                        const unsigned some = t < PW ? wanted >> t & (0xffffffffu >> (32 - box)) : 0u;
                        const int blk = __shfl_sync(0xffffffffu, block,
                                                    some ? t + __ffs(some) - 1 : 0);
                        const unsigned mine = __ballot_sync(0xffffffffu, some != 0u);
                        if (lane == 0) {
                            if (mine) bar_expect(&W.full[slot(x)], __popc(mine) * box * 128);
                            else bar_arrive(&W.full[slot(x)]);
                        }
                        __syncwarp();
                        if (some) {
                            const uint32_t p = (uint32_t)(j0 + w4 * PW + t);
                            const int off = (int)(p - P.by_page(p) * C.block_size);
                            const bool nhd = C.layout == SPEC_KV_NHD;
                            tma_box(base + place + q * (PT * 128) + t * 128, of_v ? &maps.v : &maps.k,
                                    q * 64, nhd ? A.head : off, nhd ? off : A.head, blk,
                                    &W.full[slot(x)]);
                        }
                        settle(false);
                    } else {
                        if (go) {
                            note(i, block);
                            const uint32_t in = unit(i);
#pragma unroll 4
                            for (int q = 0; q < U * PW / 32; ++q) {
                                const int t = (q * 32 + lane) / U, u = lane % U;
                                bool ok;
                                const char *from = source(block, in, t, u, ok);
                                copy16(base + place + chunk_at<PT>(t, u), from, ok);
                            }
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        settle(true);
                        pending = i;
                    }
                    if (i == 0) {
                        queries();
                        settle(false);
                    }
                }
                settle(false);
            } else {
                // a tile's codes wait in registers for its place
                constexpr int Q = U * PW / 32;                // chunks of a thread
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
                                *reinterpret_cast<uint4 *>(to + chunk_at<PT>(w4 * PW + t, 2 * u + h)) =
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
                    if (i == 0) queries();
                }
            }
            read(part);
            done += n;
            ++parts;
        }
        if (!go) {      // copies in flight come to shared memory before it is given back
            const uint64_t t0 = now_ns();
            for (int i = 0; i < (1 << 20) && now_ns() - t0 < 1000000ull; ++i) {
            }
        }
    } else {
        more_registers<128>();
        // ---- softmax: this thread's row. A wait that gives up is followed by none.
        const int m = warp >> 2;
        const int r = m * 128 + (warp & 3) * 32 + lane;          // of the item
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_tm = o_at(m) + lanes;
        const float v_scale = C.v_scale ? __ldg(C.v_scale) : 1.f;
        const float unit = P.scale * kLog2e * (C.k_scale ? __ldg(C.k_scale) : 1.f);
        uint32_t jobs = 0, results = 0;   // of this group so far (64 positions each); parts
        bool go = true;
        uint32_t part_at = 0;
        for (; m < NG; ++part_at) {
            go = go && dealt(part_at);
            if (!go) break;
            const PartWords &A = W.part[part_at % kDealt];   // until read(part_at)
            const int n = A.stop - A.tile, tile0 = A.tile, skip = A.skip, base_tile = A.base;
            if (A.b < 0) break;
            const int row0 = A.r * RT;
            const bool live = r < A.rows, work = n > 0 && m * 128 < A.rows;
            const bool warp_live = m * 128 + (warp & 3) * 32 < A.rows;
            const uint32_t at = paged_end(P, A.pos, row0 + min(r, A.rows - 1));
            float top = kPagedNoMax, sum = 0.f, factor = 0.f;    // top: the row's reference
            bool apart = false;       // a row of the warp has scores beyond kApart
            // Lanes past the item's rows hold queries of the rows behind it (see queries()), which may
            // be anything: they have no vote in what the warp does.
            auto far_apart = [&] {
                return __any_sync(0xffffffffu, live && fabsf(top) > kApart && top != kPagedNoMax) != 0;
            };
            // every row sees all of a job that is not past the first row's end and begins in the last
            // row's window, or is the sinks'
            const uint32_t e0 = A.e0, from = P.window > 0 ? A.e1 - min(A.e1, (uint32_t)P.window) : 0u;
            const int hi = A.hi;
            for (int j = 0; work && j < HALVES * n; ++j, ++jobs) {
                const int i = j / HALVES, h = j % HALVES;
                const uint32_t buf = jobs & 1, s_tm = s_at(m) + lanes + buf * 64;
                const int ti = tile0 + i, j0 = (ti < skip ? ti : base_tile + ti) * PT + 64 * h;
                const bool inside =
                    (uint32_t)(j0 + 64) <= e0 && ((uint32_t)j0 >= from || j0 + 64 <= P.sinks);
                go = go && warp_wait(&W.s_full[m][buf], jobs >> 1 & 1, gave_up);
                if (!go) break;
                tc_fence_after();
                if (j == 0)
                    factor = paged_factor(
                        kScaleQ ? unit * __uint_as_float((uint32_t)W.q_down[parts & 1][r] << 16) : unit);
                if (!warp_live) {
                    tc_fence_before();
                    warp_arrive(&W.p_full[m][buf]);
                    continue;
                }
                const uint2 there = *reinterpret_cast<const uint2 *>(&W.seen[(done + i) & 3][2 * h]);
                const bool plain = inside && (there.x & there.y) == 0xffffffffu;
                auto mask = [&](int q, uint32_t (&y)[32]) {
                    const unsigned see = (q ? there.y : there.x) &
                                         paged_bits(j0 + 32 * q, at, hi, P.window, P.sinks);
                    if (__all_sync(0xffffffffu, see == 0xffffffffu)) return;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((see >> e) & 1)) y[e] = 0xff800000u;
                };
                float job_sum = 0.f;
                bool fine = false;
                // P by the reference at hand, kept if no score was too far above it.
                if (!apart) {
                    uint32_t x[2][32];
                    tmem_ld32(s_tm, x[0]);
                    tmem_ld32(s_tm + 32, x[1]);
                    tmem_wait_ld(x[0]);
                    tmem_loaded(x[1]);
                    if (!plain) {
                        mask(0, x[0]);
                        mask(1, x[1]);
                    }
                    if (j == 0) {
                        const float big = fmaxf(largest32(x[0]), largest32(x[1]));
                        top = paged_reference(kPagedNoMax, fmaxf(kPagedNoMax, big * factor));
                        apart = far_apart();
                    }
                    uint64_t sums[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) sums[q] = probabilities<I>(x[q], factor, top, 0ull);
                    float a, b;
                    unpack_f32x2(add_f32x2(sums[0], sums[1]), a, b);
                    job_sum = a + b;
                    fine = __all_sync(0xffffffffu, !live || job_sum <= kMost) && !apart;
                    if (fine) {
                        tmem_st16(s_tm, x[0]);
                        tmem_st16(s_tm + 16, x[1]);
                    }
                }
                if (!fine) {
                    // The scores again: their largest raises the references of all the warp's rows; P
                    // of 32 positions takes the place of 16 that have been read.
                    float x = kPagedNoMax;
                    auto scores = [&](int q, uint32_t (&y)[32]) {
                        tmem_ld32(s_tm + q * 32, y);
                        tmem_wait_ld(y);
                        mask(q, y);
                    };
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        uint32_t y[32];
                        scores(q, y);
                        x = fmaxf(x, largest32(y) * factor);
                    }
                    const float to = paged_reference(top, x), a = ex2(top - to);
                    top = to;
                    sum *= a;
                    apart = apart || far_apart();
                    if (j > 0) {
                        // the scores at hand were made after the product two before this one's
                        go = go && warp_wait(&W.o_full[m], (jobs - 1) & 1, gave_up);
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < DP / 16; ++q) {
                            uint32_t o[16];
                            tmem_ld16(o_tm + q * 16, o);
                            tmem_wait_ld16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tmem_st16(o_tm + q * 16, o);
                        }
                    }
                    uint64_t sums = 0ull;
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        uint32_t y[32];
                        scores(q, y);
                        if (apart) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                y[e] = __float_as_uint(__fmul_rn(__uint_as_float(y[e]), factor));
                        }
                        sums = probabilities<I>(y, apart ? 1.f : factor, top, sums);
                        tmem_st16(s_tm + q * 16, y);
                    }
                    float b;
                    unpack_f32x2(sums, job_sum, b);
                    job_sum += b;
                }
                sum += job_sum;
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&W.p_full[m][buf]);
            }
            // The result: O is done after the group's last product.
            if (work) go = go && warp_wait(&W.o_last[m], results++ & 1, gave_up);
            tc_fence_after();
            if (!go) {      // lost: a sum of NaN makes the rows of this part NaN, and the item's
                sum = NAN;
                if (P.status && lane == 0) atomicMax(P.status + A.b, SPEC_REQ_INTERNAL);
            }
            const bool whole = A.begins && A.ends;
            const float norm = (whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f) * v_scale;
            const int64_t to = live ? paged_row(P, A.first, A.head, row0 + r) : 0;
            float *part = paged_slot(P, blockIdx.x, A.begins, RT, DP);
            const bool out32 = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
            const bool odd = n > 0 && *(volatile int *)&W.odd[parts % kOdd] != 0;
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
            if (odd && live) {      // NaN and infinities of positions that this row sees
                for (int i = tile0; i < A.stop; ++i) {
                    const int j0 = A.position<PT>(i);
                    if (all_see(P, A.e0, A.e1, j0, PT)) continue;
#pragma unroll 1
                    for (int j = j0; j < j0 + PT; ++j) {
                        if (!(paged_bits(j, at, hi, P.window, P.sinks) & 1)) continue;
                        const int block = paged_page(P, A.b, j);
                        if (block < 0 || block >= C.num_blocks) continue;
                        const uint32_t off = j - P.by_page((uint32_t)j) * C.block_size;
                        const int64_t e0 = block * C.v_block_stride +
                                           (int64_t)(C.layout == SPEC_KV_NHD ? off * C.H + A.head
                                                                             : A.head * C.block_size + off) *
                                               C.D;
#pragma unroll 1
                        for (int d = 0; d < C.D; ++d) {
                            const float y =
                                KIND ? value16<2>(halves2<KIND>(__ldg(static_cast<const uint8_t *>(C.v) +
                                                                     e0 + d)) & 0xffffu)
                                     : value16<I>(__ldg(static_cast<const unsigned short *>(C.v) + e0 + d));
                            if (fabsf(y) < INFINITY) continue;
                            if (whole) {
                                unsigned short *o = static_cast<unsigned short *>(P.out) + to * C.D + d;
                                *o = (unsigned short)pack2<T>(value16<T>(*o) + y, 0.f);
                            } else {
                                part[(int64_t)r * DP + d] += y;
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            read(part_at);
            done += n;
            parts += n > 0;
        }
        if (m < NG && !go) {      // the parts that did not come are lost, too
            PagedWalk<RT, PT> walk(P, kTcFixed<KIND, DP>, (int64_t)P.G * kPosTile);
            PagedPart A;
            for (uint32_t x = 0; walk.next(P, A); ++x) {
                if (x < part_at) continue;
                if (P.status && lane == 0) atomicMax(P.status + A.b, SPEC_REQ_INTERNAL);
                if (r >= A.rows) continue;
                const int64_t to = paged_row(P, A.req.first, A.head, A.r * RT + r);
                float *part = paged_slot(P, blockIdx.x, A.begins, RT, DP);
                for (int e = 0; e < C.D; e += 4) {
                    const float4 v = make_float4(NAN, NAN, NAN, NAN);
                    if (A.whole()) paged_store4<T>(P.out, to * C.D + e, v);
                    else *reinterpret_cast<float4 *>(part + (int64_t)r * DP + e) = v;
                }
                if (A.whole()) {
                    if (P.lse) P.lse[to] = NAN;
                } else {
                    part[RT * DP + r] = kPagedNoMax;
                    part[RT * (DP + 1) + r] = NAN;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, C_::kColumns);
}

// A tensor map of 16-bit elements with 128-byte swizzle: boxes of 64 x box[1] x ...; false if it
// cannot be had.
bool make_map(CUtensorMap &map, int dtype, const void *at, int rank, const cuuint64_t *dims,
              const cuuint64_t *strides, const cuuint32_t *box) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                               cudaEnableDefault, &found);
        if (e != cudaSuccess) cudaGetLastError();
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f)
                                                                         : nullptr;
    }();
    if (!encode) return false;
    for (int i = 0; i + 1 < rank; ++i)
        if (strides[i] >= cuuint64_t(1) << 40) return false;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(&map, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                           : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  (cuuint32_t)rank, const_cast<void *>(at), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

Maps make_maps(const PagedAttnParams &p, int most) {      // most: positions of a loading warp
    Maps m = {};
    const spec_kv_cache &c = p.cache;
    if (c.D < 64) return m;
    const cuuint64_t d = (cuuint64_t)c.D, h = (cuuint64_t)c.H, n = (cuuint64_t)c.block_size;
    // Pages of a multiple of eight positions: boxes of the largest power of two that divides both
    // them and a loading warp's (their places in shared memory begin where the swizzle's pattern does).
    if (n % 8 == 0) {
        const bool nhd = c.layout == SPEC_KV_NHD;
        const cuuint32_t rows = n % 32 == 0 && most == 32 ? 32 : n % 16 == 0 ? 16 : 8;
        const cuuint64_t dims[4] = {d, nhd ? h : n, nhd ? n : h, (cuuint64_t)c.num_blocks};
        const cuuint32_t box[4] = {64, nhd ? 1 : rows, nhd ? rows : 1, 1};
        cuuint64_t strides[3] = {d * 2, (nhd ? h : n) * d * 2, (cuuint64_t)c.k_block_stride * 2};
        bool ok = make_map(m.k, p.dtype, c.k, 4, dims, strides, box);
        strides[2] = (cuuint64_t)c.v_block_stride * 2;
        ok = ok && make_map(m.v, p.dtype, c.v, 4, dims, strides, box);
        if (ok) m.page_rows = (int)rows;
    }
    // Queries whose groups of heads divide 128 rows: boxes of whole tokens.
    if (128 % p.G == 0 && reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.q_stride % 8 == 0) {
        const cuuint64_t dims[3] = {d, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
        const cuuint64_t strides[2] = {d * 2, (cuuint64_t)p.q_stride * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(128 / p.G)};
        if (make_map(m.q, p.dtype, p.q, 3, dims, strides, box)) m.tokens = 128 / p.G;
    }
    return m;
}

template <int T, int KIND, int DP>
cudaError_t launch(const PagedAttnParams &p, int grid, cudaStream_t st) {
    using C_ = Tc<DP>;
    const cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<T, KIND, DP>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C_::kBytes);
    if (e != cudaSuccess) return e;
    const int vec = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.q_stride % 8 == 0;
    paged_tc_kernel<T, KIND, DP><<<grid, kThreads, C_::kBytes, st>>>(p, vec,
                                                                   KIND ? Maps{} : make_maps(p, C_::kPos / 4));
    return cudaGetLastError();
}

template <int T, int KIND>
cudaError_t launch_size(const PagedAttnParams &p, int grid, cudaStream_t st) {
    const int DP = paged_padded(p.cache.D);
    return DP == 64    ? launch<T, KIND, 64>(p, grid, st)
           : DP == 128 ? launch<T, KIND, 128>(p, grid, st)
                       : launch<T, KIND, 256>(p, grid, st);
}

}  // namespace

template <int T>
cudaError_t launch_paged_tc_type(const PagedAttnParams &p, int grid, cudaStream_t st) {
    if (p.cache.kind == SPEC_CACHE_SAME) return launch_size<T, 0>(p, grid, st);
    if (p.cache.kind == SPEC_CACHE_FP8_E4M3) return launch_size<T, 1>(p, grid, st);
    return launch_size<T, 2>(p, grid, st);
}

}  // namespace specv
