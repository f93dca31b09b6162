// What the tree-attention kernels share: how the work is dealt to the CTAs and how the parts
// of an item are joined. Internal.
//
// The work of a call is a list of items (request, K/V head, tile of query rows), each a row of
// tiles: its context in tiles of kTile positions, then one tile for the tree's own nodes. A
// context tile counts as one unit of work; the tree's tile, with what an item costs besides
// (its queries in, its result out), as `cost` units, of which the tile takes place in the first.
// The units of all items, in order, are cut into equal ranges, one for each CTA of a single
// wave, whatever the requests' lengths (which only the device knows). The CTAs may stand in
// columns, one for each item of a request (K/V head and row tile), each column cutting all
// requests alike: then the heads of a position are read at the same time. In the NHD layout they
// lie side by side, eight bytes of block scales each, and were fetched over and over when every
// head passed a position at a time of its own (64 chains, 8 heads: 1.14 GB for 0.54). A CTA therefore works on
// end of one item, some whole items, and the start of another. Whole items are finished in
// place. The parts of an item that a cut goes through are written to the workspace (row sums
// and maxima and the unnormalised rows, float32), and a second kernel joins them in their
// order: all SMs share that, where the last CTA to arrive at an item of many parts would take
// longer for it than for its own part (80 us of 180 for 8 items of 256 rows in 19 parts each).
#pragma once

#include "fp4_device.cuh"

namespace specv {

constexpr int kTile = 128;          // context positions of a tile

// A context length as the kernels use it.
__device__ __forceinline__ int attn_ctx(const TreeAttnParams &P, int b) {
    const int most = P.cache.max_blocks * P.cache.block_size;   // fits: checked on the host
    return min(max(__ldg(P.ctx_len + b), 0), most);
}

// A CTA's range of units, and where it begins.
struct AttnRange {
    int64_t total, begin, end;   // units of a column; this CTA's [begin, end)
    int ctas;                    // CTAs of a column that have a range: each at least one unit
    int b, item, tile;           // place of `begin`: request, item in it, unit in that
};

// `items`: items of a request in a column. Every warp computes it for itself (one warp scan).
__device__ __forceinline__ AttnRange attn_range(const TreeAttnParams &P, int items, int cost,
                                                int columns) {
    auto units = [&](int b) { return (attn_ctx(P, b) + kTile - 1) / kTile + cost; };
    const unsigned full = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int per = (P.B + 31) / 32, b0 = lane * per, b1 = min(P.B, b0 + per);
    int64_t mine = 0;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) mine += (int64_t)units(b) * items;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(full, sum, o);
        if (lane >= o) sum += v;
    }
    AttnRange r;
    r.total = __shfl_sync(full, sum, 31);
    const int cta = blockIdx.x / columns;
    r.ctas = (int)min((int64_t)(gridDim.x / columns), r.total);
    r.b = r.item = r.tile = 0;
    r.begin = r.end = 0;
    if (cta >= r.ctas) return r;
    r.begin = r.total * cta / r.ctas;
    r.end = r.total * (cta + 1) / r.ctas;
    const int64_t before = sum - mine;
    const bool here = before <= r.begin && r.begin < sum;
    if (here) {
        int64_t left = r.begin - before;
        int b = b0;
        for (;; ++b) {
            const int n = units(b);
            if (left < (int64_t)n * items) {
                r.item = (int)(left / n);
                r.tile = (int)(left - (int64_t)r.item * n);
                break;
            }
            left -= (int64_t)n * items;
        }
        r.b = b;
    }
    const int src = __ffs(__ballot_sync(full, here)) - 1;
    r.b = __shfl_sync(full, r.b, src);
    r.item = __shfl_sync(full, r.item, src);
    r.tile = __shfl_sync(full, r.tile, src);
    return r;
}

// The CTA (of a column) whose range holds unit s.
__device__ __forceinline__ int attn_owner(const AttnRange &r, int64_t s) {
    return (int)(((s + 1) * r.ctas - 1) / r.total);
}

// A CTA's part of an item: its tiles [tile, stop) of the item's nt.
struct AttnPart {
    int b, item, tile, stop, nt, ctx;
    int64_t first;                // unit of the item's first tile
};

// Steps through a CTA's parts, in order.
struct AttnWalk {
    AttnRange r;
    int64_t at;
    int b, item, tile, items, cost, column;   // column: 0 if there is one only

    // `all`: items of a request.
    __device__ __forceinline__ AttnWalk(const TreeAttnParams &P, int all, int cost_, int columns)
        : r(attn_range(P, columns > 1 ? 1 : all, cost_, columns)), at(r.begin), b(r.b),
          item(r.item), tile(r.tile), items(columns > 1 ? 1 : all), cost(cost_),
          column(blockIdx.x % columns) {}
    // The next part, or false. Units past the tree's first start nothing.
    __device__ __forceinline__ bool next(const TreeAttnParams &P, AttnPart &p) {
        while (at < r.end) {
            const int ctx = attn_ctx(P, b), nt = (ctx + kTile - 1) / kTile + 1;
            const int left = nt - 1 + cost - tile;
            const bool starts = tile < nt;
            p.b = b;
            p.item = item + column;
            p.tile = tile;
            p.nt = nt;
            p.ctx = ctx;
            p.first = at - tile;
            p.stop = (int)min((int64_t)nt, tile + (r.end - at));
            at += left;
            tile = 0;
            if (++item == items) {
                item = 0;
                ++b;
            }
            if (starts) return true;
        }
        return false;
    }
};

// Where CTA `cta` leaves a part of an item: slot 0 if it came into the item from the middle,
// slot 1 if it began the item. rows x (d values, then max and sum apart).
__device__ __forceinline__ float *attn_slot(const TreeAttnParams &P, int cta, int slot, int rows,
                                            int d) {
    return P.ws + ((int64_t)cta * 2 + slot) * rows * (d + 2);
}

// A CTA's note for the joining kernel: the item it began and did not finish (its last), if any,
// and the CTA that has the item's last part. One thread calls it, at the CTA's end.
__device__ __forceinline__ void attn_note(const TreeAttnParams &P, const AttnRange &r,
                                          const AttnPart &last, bool any) {
    int4 note = make_int4(-1, 0, 0, 0);
    if (any && last.tile == 0 && last.stop < last.nt)
        note = make_int4(last.b, last.item,
                         attn_owner(r, last.first + last.nt - 1) * P.columns +
                             (int)blockIdx.x % P.columns,
                         0);
    P.notes[blockIdx.x] = note;
}

// Four values of an output row.
template <int T>
__device__ __forceinline__ void store_out4(void *out, int64_t e, float4 v) {
    uint2 w;
    if (T == 1) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
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

// Element offset of row r of item (b, head): [B, N, Hq, D] with r = n * G + g.
__device__ __forceinline__ int64_t attn_row(const TreeAttnParams &P, int b, int head, int r) {
    const int n = r / P.G, g = r - n * P.G;
    return ((int64_t)b * P.N + n) * P.Hq + head * P.G + g;
}

// A row's reference before the first key: the lowest number, so that any score passes it. (Not
// -inf: its difference from a masked score would be NaN.)
constexpr float kNoMax = -3.40282347e38f;

// A row's probabilities are 2^(x - m) with a reference m that is raised to its largest score less
// kHeadroom, and raised again only when a score passes m by kRescale. So the largest score met
// when m was raised stands at 2^7 and none above 2^15, which a half holds; a half's last step is
// 2^-24, so keys down to 2^-31 of that one keep their weight in the product with V. (With m at the
// largest score they ended at 2^-24: the result lost what many such keys weigh together, while
// the row's sum had it.) The factor cancels in the result and in m + log2(sum).
constexpr float kHeadroom = 7.f, kRescale = 15.f;

// What a score has to pass for its row's reference m to be raised. Rounded down, for the same reason
// as the reference is rounded up.
__device__ __forceinline__ float attn_limit(float m) { return __fadd_rd(m, kRescale); }

// The reference for a largest score x that passed m. Rounded up: m steps by more than the
// headroom where scores are beyond 2^27, and no probability may pass 2^15.
__device__ __forceinline__ float attn_reference(float m, float x) {
    return fmaxf(m, __fadd_ru(x, -kHeadroom));
}
constexpr float kLn2 = 0.6931471805599453f;

// The factor of a row's scores, kept a positive float32 number (2^-149 at least): 0, which the
// smallest factors of a row of zeros come to, would make NaN of the -inf of a masked score, and
// infinity would of a score of zero.
__device__ __forceinline__ float attn_factor(float f) {
    return fminf(fmaxf(f, 1.4e-45f), 3.40282347e38f);
}

// log sum exp from a maximum in powers of two and a sum.
__device__ __forceinline__ float attn_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace specv
