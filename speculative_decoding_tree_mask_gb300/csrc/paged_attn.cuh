// What the paged-attention kernels share: how the work is dealt to the CTAs, what a row sees, and
// how the parts of an item are joined. Internal.
//
// The work of a call is a list of items (request, tile of its query rows, K/V head), in that order;
// the rows of a request and a head are its tokens times the G query heads that share the head. An
// item's keys are a list of tiles of kTile positions: the window's, before them the sinks' where the
// window has left them. An item weighs about what it reads, in closed form, so that the weight of a
// request's first r row tiles needs no sum over them:
//   w(r) = G fixed + min(G seq_pos + (r + 1) rows, what a window can span),
// and the total weight, in the items' order, is cut into equal ranges, one for each CTA of a single
// wave, whatever the requests' sizes (which only the device knows). A cut inside an item falls
// between two of its tiles, the same one for both CTAs. (Short items left whole cost more than their
// joining: 256 of up to 8 tiles took 50 us in one CTA each, 37 cut.) Whole items are finished in place;
// the parts of a cut item go to the workspace (row sums and references and the unnormalised rows,
// float32), and a second kernel joins them in their order.
#pragma once

#include "rope_device.cuh"
#include "spec_device.cuh"
#include "spec_internal.h"

namespace specv {

constexpr int kPosTile = 128;       // positions of a tile, where a kernel has no other

// A request as the kernels use it.
struct PagedReq {
    int first, n;                   // its rows
    int pos;                        // position of the first
};
// 0, or what is wrong with request b's numbers.
__device__ __forceinline__ int paged_req(const PagedAttnParams &P, int b, PagedReq &q) {
    int first = b * P.N, end = first + P.N;
    if (P.row_start) {
        first = __ldg(P.row_start + b);
        end = __ldg(P.row_start + b + 1);
    }
    q.first = first;
    q.pos = __ldg(P.seq_pos + b);
    if (first < 0 || end < first || end > P.T || end - first > P.max_new) {
        q.n = 0;
        return SPEC_REQ_BAD_RANGE;
    }
    q.n = end - first;
    if (q.n * P.G <= P.rows_over || q.n * P.G > P.rows_most) {      // another launch's
        q.n = 0;
        return 0;
    }
    const int most = P.cache.max_blocks * P.cache.block_size;   // fits: checked on the host
    return q.n > 0 && (q.pos < 0 || (int64_t)q.pos + q.n > most) ? SPEC_REQ_BAD_SLOT : 0;
}

// Where row i of a request that begins at `pos` ends: the positions up to its token's, that included,
// 0 if it stands before them all. pos may be any int32, so this goes past 2^31 (and not past 2^32),
// and past the table: a window ends with its row's own position, whether the table has that or not.
__device__ __forceinline__ uint32_t paged_end(const PagedAttnParams &P, int pos, int i) {
    const int64_t p = (int64_t)pos + P.by_group((uint32_t)i);
    return (uint32_t)max(p + 1, (int64_t)0);
}

// Weights (see above). RT: rows of a tile, a power of two.
template <int RT>
struct PagedWeights {
    int64_t fixed, grow, cap;       // G fixed; G seq_pos; G times what a window can span

    __device__ __forceinline__ PagedWeights(const PagedAttnParams &P, int pos, int fixed_positions) {
        const int most = P.cache.max_blocks * P.cache.block_size;
        fixed = (int64_t)P.G * fixed_positions;
        grow = (int64_t)P.G * min(max(pos, 0), most);
        cap = P.window > 0 ? (int64_t)P.G * ((int64_t)P.window + min(P.sinks, most)) + RT
                           : (int64_t)1 << 60;
    }
    __device__ __forceinline__ int64_t of(int64_t r) const {
        return fixed + min(grow + (r + 1) * RT, cap);
    }
    // of the tiles before r
    __device__ __forceinline__ int64_t before(int64_t r) const {
        const int64_t k = min(max((cap - grow) / RT, (int64_t)0), r);   // those below the cap
        const int64_t rest = r - k;
        return r * fixed + k * grow + k * (k + 1) / 2 * RT + (rest > 0 ? rest * cap : 0);
    }
};

// A CTA's range of the total weight.
struct PagedRange {
    int64_t total, begin, end;
    int ctas;                       // CTAs that have a range
};

// A CTA's part of an item.
struct PagedPart {
    int b, r, head;                 // request, row tile, K/V head
    PagedReq req;
    int rows;                       // of the tile
    uint32_t e0, e1;                // ends (see paged_end) of its first and last row
    int lo, hi;                     // positions that any row sees: [lo, hi), and those below sinks
    int skip, base;                 // tile i stands at position PT * (i < skip ? i : base + i)
    int tile, stop, nt;             // tiles of this part, of the item
    bool begins, ends;              // the part has the item's begin, its end
    int64_t at, w;                  // where the item begins, its weight

    __device__ __forceinline__ bool whole() const { return begins && ends; }
};

__device__ __forceinline__ int paged_owner(const PagedRange &r, int64_t x) {   // of weight unit x
    return (int)(((x + 1) * r.ctas - 1) / r.total);
}

// Steps through a CTA's parts, in order. Every warp runs it for itself (all 32 lanes).
template <int RT, int PT = kPosTile>
struct PagedWalk {
    PagedRange range;
    int64_t at;                     // where the item at hand begins
    int b, r, head, fixed;          // request, row tile, K/V head at hand
    PagedReq req;

    __device__ __forceinline__ int tiles(const PagedAttnParams &P, const PagedReq &q) const {
        return (q.n * P.G + RT - 1) / RT;           // fits: checked on the host
    }

    // `least`: the least weight that is a CTA's.
    __device__ __forceinline__ PagedWalk(const PagedAttnParams &P, int fixed_positions, int64_t least)
        : fixed(fixed_positions) {
        const unsigned full = 0xffffffffu;
        const int lane = threadIdx.x & 31, per = (P.B + 31) / 32;
        const int b0 = min(P.B, lane * per), b1 = min(P.B, b0 + per);
        auto weigh = [&](int i) -> int64_t {
            PagedReq q;
            paged_req(P, i, q);
            return PagedWeights<RT>(P, q.pos, fixed).before(tiles(P, q)) * P.cache.H;
        };
        int64_t mine = 0;
#pragma unroll 4
        for (int i = b0; i < b1; ++i) mine += weigh(i);
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(full, sum, o);
            if (lane >= o) sum += v;
        }
        range.total = __shfl_sync(full, sum, 31);
        range.ctas = (int)min((int64_t)gridDim.x, max((range.total + least - 1) / least, (int64_t)1));
        range.begin = range.end = at = 0;
        b = head = 0;
        r = 0;
        req = PagedReq{0, 0, 0};
        if (range.total == 0 || (int)blockIdx.x >= range.ctas) return;
        // (total * cta would pass 64 bits only far beyond what can be computed)
        range.begin = range.total / range.ctas * blockIdx.x +
                      range.total % range.ctas * blockIdx.x / range.ctas;
        range.end = range.total / range.ctas * (blockIdx.x + 1) +
                    range.total % range.ctas * (blockIdx.x + 1) / range.ctas;
        const bool here = sum - mine <= range.begin && range.begin < sum;
        if (here) {
            int64_t left = range.begin - (sum - mine);
            int i = b0;
            for (;; ++i) {
                const int64_t w = weigh(i);
                if (left < w) break;
                left -= w;
            }
            paged_req(P, i, req);
            const PagedWeights<RT> W(P, req.pos, fixed);
            // the last row tile that begins at or before `left`
            int lo = 0, hi = tiles(P, req) - 1;
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if (W.before(mid) * P.cache.H <= left) lo = mid;
                else hi = mid - 1;
            }
            b = i;
            r = lo;
            left -= W.before(lo) * P.cache.H;
            head = (int)(left / W.of(lo));
            at = range.begin - (left - head * W.of(lo));
        }
        const int from = __ffs(__ballot_sync(full, here)) - 1;
        b = __shfl_sync(full, b, from);
        head = __shfl_sync(full, head, from);
        r = __shfl_sync(full, r, from);
        at = __shfl_sync(full, at, from);
        req.first = __shfl_sync(full, req.first, from);
        req.n = __shfl_sync(full, req.n, from);
        req.pos = __shfl_sync(full, req.pos, from);
    }

    // The next part, or false.
    __device__ __forceinline__ bool next(const PagedAttnParams &P, PagedPart &p) {
        if (at >= range.end) return false;
        while (r >= tiles(P, req)) {       // the next request that has rows
            ++b;
            r = 0;
            paged_req(P, b, req);
        }
        const int64_t w = PagedWeights<RT>(P, req.pos, fixed).of(r);
        p.b = b;
        p.r = r;
        p.head = head;
        p.req = req;
        p.at = at;
        p.w = w;
        const int row0 = r * RT;
        p.rows = min(RT, req.n * P.G - row0);
        const int most = P.cache.max_blocks * P.cache.block_size;       // fits: checked on the host
        p.e0 = paged_end(P, req.pos, row0);
        p.e1 = paged_end(P, req.pos, row0 + p.rows - 1);
        p.hi = (int)min(p.e1, (uint32_t)most);
        p.lo = P.window > 0 ? (int)min(p.e0 - min(p.e0, (uint32_t)P.window), (uint32_t)p.hi) : 0;
        const int t0 = p.lo / PT, t1 = (p.hi + PT - 1) / PT;
        p.skip = min((min(P.sinks, p.hi) + PT - 1) / PT, t0);
        p.base = t0 - p.skip;
        p.nt = p.skip + max(t1 - t0, 0);
        const int64_t xa = max(range.begin - at, (int64_t)0), xb = min(range.end - at, w);
        p.begins = xa == 0;
        p.ends = xb == w;
        p.tile = p.begins ? 0 : (int)((double)xa * p.nt / (double)w);
        p.stop = p.ends ? p.nt : (int)((double)xb * p.nt / (double)w);
        at += w;
        if (++head == P.cache.H) {
            head = 0;
            ++r;
        }
        return true;
    }
};

// The statuses of the requests, by the first CTA's threads.
__device__ __forceinline__ void paged_status(const PagedAttnParams &P, int threads) {
    if (!P.status || blockIdx.x != 0) return;
    for (int b = threadIdx.x; b < P.B; b += threads) {
        PagedReq q;
        const int bad = paged_req(P, b, q);
        if (bad) atomicMax(P.status + b, bad);
    }
}

// The block that the table has for position p of request b.
__device__ __forceinline__ int paged_page(const PagedAttnParams &P, int b, int p) {
    return __ldg(P.cache.block_table + (int64_t)b * P.cache.max_blocks + P.by_page((uint32_t)p));
}

// Where CTA `cta` leaves a part of an item: slot 0 if it came into the item from the middle,
// slot 1 if it began the item. rows x (d values, then reference and sum apart).
__device__ __forceinline__ float *paged_slot(const PagedAttnParams &P, int cta, int slot, int rows,
                                             int d) {
    return P.ws + ((int64_t)cta * 2 + slot) * rows * (d + 2);
}

// A CTA's note for the joining kernel: of the item it began and did not finish (its last), if any, the
// request's first row (else -1), the item's first row in the request, its rows, and its K/V head with
// the CTA that has its end. One thread calls it, at the CTA's end.
constexpr int kNoteCtas = 12;       // bits
__device__ __forceinline__ void paged_note(const PagedAttnParams &P, const PagedRange &r,
                                           const PagedPart &last, int rows_tile, bool any) {
    int4 note = make_int4(-1, 0, 0, 0);
    if (any && last.begins && !last.ends)
        note = make_int4(last.req.first, last.r * rows_tile, last.rows,
                         last.head << kNoteCtas | paged_owner(r, last.at + last.w - 1));
    P.notes[blockIdx.x] = note;
}

// Row i of a request (whose first is `first` of the batch) and K/V head as an index of lse [T, Hq].
__device__ __forceinline__ int64_t paged_row(const PagedAttnParams &P, int first, int head, int i) {
    const int t = (int)P.by_group((uint32_t)i);
    return (int64_t)(first + t) * P.Hq + head * P.G + (i - t * P.G);
}
// Where it begins among the queries.
__device__ __forceinline__ const unsigned short *paged_query(const PagedAttnParams &P, int first,
                                                             int head, int i) {
    const int t = (int)P.by_group((uint32_t)i);
    return static_cast<const unsigned short *>(P.q) + (first + t) * P.q_stride +
           (int64_t)(head * P.G + (i - t * P.G)) * P.cache.D;
}
// Four values of an output row.
template <int T>
__device__ __forceinline__ void paged_store4(void *out, int64_t e, float4 v) {
    uint2 w;
    const float x[4] = {v.x, v.y, v.z, v.w};
    if constexpr (T == 1) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
    }
    unsigned short *p = reinterpret_cast<unsigned short *>(out) + e;
    if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
        *reinterpret_cast<uint2 *>(p) = w;
    } else {   // an output that begins off an 8-byte boundary
        p[0] = (unsigned short)w.x;
        p[1] = (unsigned short)(w.x >> 16);
        p[2] = (unsigned short)w.y;
        p[3] = (unsigned short)(w.y >> 16);
    }
}

// The running softmax of a row. p = 2^(x - m) with a reference m that is raised to the largest
// score less kPagedHeadroom, and again only when a score passes m by kPagedRescale: rescaling is
// rare, and no p passes 2^15, which a half holds; a half's last step is 2^-24, so keys down to 2^-31
// of the largest keep their weight in the product with V. The factor cancels in the result.
constexpr float kPagedNoMax = -3.40282347e38f;    // below any score; not -inf, whose differences are NaN
constexpr float kPagedHeadroom = 7.f, kPagedRescale = 15.f;
// Rounded down here and up there, so that no p passes 2^15 where scores are beyond 2^20 either.
__device__ __forceinline__ float paged_limit(float m) { return __fadd_rd(m, kPagedRescale); }
__device__ __forceinline__ float paged_reference(float m, float x) {
    return fmaxf(m, __fadd_ru(x, -kPagedHeadroom));
}
// The factor of a row's scores stays a positive float32: 0 and infinity would make NaN of -inf and 0.
__device__ __forceinline__ float paged_factor(float f) {
    return fminf(fmaxf(f, 1.4e-45f), 3.40282347e38f);
}
__device__ __forceinline__ float paged_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Bits of the 32 positions from j0 on that a row of this end sees, among those below `hi`.
__device__ __forceinline__ unsigned paged_bits(uint32_t j0, uint32_t end, int hi, int window,
                                               int sinks) {
    auto below = [&](uint32_t n) -> unsigned {      // positions j0 .. n - 1
        return n <= j0 ? 0u : n - j0 >= 32 ? 0xffffffffu : (1u << (n - j0)) - 1u;
    };
    unsigned seen = below(min(end, (uint32_t)hi));
    if (window > 0) seen &= ~below(end - min(end, (uint32_t)window)) | below((uint32_t)sinks);
    return seen;
}
// Whether rows of ends e0 (the first's) to e1 all see all of the n positions from j0 on, as far as
// those are there.
__device__ __forceinline__ bool all_see(const PagedAttnParams &P, uint32_t e0, uint32_t e1, int j0,
                                        int n) {
    return (uint32_t)(j0 + n) <= e0 &&
           (P.window == 0 || (uint32_t)j0 + (uint32_t)P.window >= e1 || j0 + n <= P.sinks);
}

// A 16-byte copy to shared memory; zeros when !ok.
__device__ __forceinline__ void copy16(uint32_t smem, const void *gmem, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

template <int I>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (I == 1) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <int I>
__device__ __forceinline__ float value16(uint32_t x) {
    return I == 1 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((unsigned short)x));
}
// Two 8-bit codes (the low 16 bits) as halves, exactly.
template <int KIND>
__device__ __forceinline__ uint32_t halves2(uint32_t two) {
    if constexpr (KIND == 1) {
        uint32_t r;
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
            : "=r"(r)
            : "r"(two));
        return r;
    } else {       // e5m2 is a half's upper byte
        return __byte_perm(two, 0u, 0x1404);
    }
}
// Whether one of the elements in a word is NaN or infinite.
template <int I, int KIND>
__device__ __forceinline__ bool odd_word(uint32_t w) {
    if constexpr (KIND == 1) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    if constexpr (KIND == 2) return __vcmpeq4(w & 0x7c7c7c7cu, 0x7c7c7c7cu) != 0;
    constexpr uint32_t ex = I == 1 ? 0x7f807f80u : 0x7c007c00u;
    return __vcmpeq2(w & ex, ex) != 0;
}

// D up to the next size that the kernels are built for.
inline int paged_padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Few rows (paged_few.cuh): CTAs an SM holds, by shared memory and registers; the launches, mt
// groups of 16 rows an item.
constexpr int paged_few_ctas(bool fp8, int DP) {
    return DP * (fp8 ? 1 : 2) <= 64 ? 3 : DP * (fp8 ? 1 : 2) <= 256 ? 2 : 1;
}
cudaError_t launch_paged_few_bf16(const PagedAttnParams &p, int mt, int grid, cudaStream_t st);
cudaError_t launch_paged_few_f16(const PagedAttnParams &p, int mt, int grid, cudaStream_t st);

// Launches on the tcgen05 tensor cores (paged_tc.cuh).
constexpr int paged_tc_rows(int DP) { return DP == 256 ? 128 : 256; }   // of an item
cudaError_t launch_paged_tc_bf16(const PagedAttnParams &p, int grid, cudaStream_t st);
cudaError_t launch_paged_tc_f16(const PagedAttnParams &p, int grid, cudaStream_t st);

}  // namespace specv
