// What the tree-attention kernels share: how the work is dealt to the CTAs and how the parts
// of an item are joined. Internal.
//
// The work of a call is a list of items (request, K/V head, tile of query rows), each a row of
// tiles: its context in tiles of kTile positions, then one tile for the tree's own nodes. The
// tiles of all items, in order, are cut into equal ranges, one for each CTA of a single wave,
// whatever the requests' lengths (which only the device knows). A CTA therefore works on the
// end of one item, some whole items, and the start of another. Whole items are finished in
// place. The parts of an item that a cut goes through are written to the workspace (row sums
// and maxima and the unnormalised rows, float32); the CTA that arrives last joins them in
// their order, so the result does not depend on which that is.
#pragma once

#include "fp4_device.cuh"

namespace specv {

constexpr int kTile = 128;          // context positions of a tile

// A context length as the kernels use it.
__device__ __forceinline__ int attn_ctx(const TreeAttnParams &P, int b) {
    const int most = P.cache.max_blocks * P.cache.block_size;   // fits: checked on the host
    return min(max(__ldg(P.ctx_len + b), 0), most);
}
__device__ __forceinline__ int attn_tiles(const TreeAttnParams &P, int b) {
    return (attn_ctx(P, b) + kTile - 1) / kTile + 1;
}

// A CTA's range of tiles, and where it begins.
struct AttnRange {
    int64_t total, begin, end;   // tiles of the call; this CTA's [begin, end)
    int ctas;                    // CTAs that have a range: each has at least one tile
    int b, item, tile;           // place of `begin`
};

// `items`: items of a request. Every warp computes it for itself (one warp scan).
__device__ __forceinline__ AttnRange attn_range(const TreeAttnParams &P, int items) {
    const unsigned full = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int per = (P.B + 31) / 32, b0 = lane * per, b1 = min(P.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += (int64_t)attn_tiles(P, b) * items;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(full, sum, o);
        if (lane >= o) sum += v;
    }
    AttnRange r;
    r.total = __shfl_sync(full, sum, 31);
    r.ctas = (int)min((int64_t)gridDim.x, r.total);
    r.b = r.item = r.tile = 0;
    r.begin = r.end = 0;
    if ((int)blockIdx.x >= r.ctas) return r;
    r.begin = r.total * blockIdx.x / r.ctas;
    r.end = r.total * (blockIdx.x + 1) / r.ctas;
    const int64_t before = sum - mine;
    const bool here = before <= r.begin && r.begin < sum;
    if (here) {
        int64_t left = r.begin - before;
        int b = b0;
        for (;; ++b) {
            const int n = attn_tiles(P, b);
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

// The CTA whose range holds tile s.
__device__ __forceinline__ int attn_owner(const AttnRange &r, int64_t s) {
    return (int)(((s + 1) * r.ctas - 1) / r.total);
}

// Where CTA `cta` leaves a part of an item: slot 0 if it came into the item from the middle,
// slot 1 if it began the item. rows x (d values, then max and sum apart).
__device__ __forceinline__ float *attn_slot(const TreeAttnParams &P, int cta, int slot, int rows,
                                            int d) {
    return P.ws + ((int64_t)cta * 2 + slot) * rows * (d + 2);
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

constexpr float kNoMax = -1e30f;            // running maximum before the first key
constexpr float kLn2 = 0.6931471805599453f;

// log sum exp from a maximum in powers of two and a sum.
__device__ __forceinline__ float attn_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The last of an item's parts to arrive joins them. Called by all threads of the CTA after they
// have written their part; `first` = the item's first tile, `n` its tiles. Returns after the
// join, or at once when other parts are still missing.
template <int T, int D>
__device__ __forceinline__ void attn_join(const TreeAttnParams &P, const AttnRange &R,
                                          int64_t first, int n, int b, int head, int row0,
                                          int rows, int rows_tile, int *s_flag) {
    const int c0 = attn_owner(R, first), c1 = attn_owner(R, first + n - 1);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int seen = atomicAdd(P.arrive + c0, 1);
        const int last = seen == c1 - c0;
        if (last) P.arrive[c0] = 0;   // for the next call
        __threadfence();
        *s_flag = last;
    }
    __syncthreads();
    if (!*s_flag) return;
    for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
        const int r = i / (D / 4), d4 = i - r * (D / 4);
        float m = kNoMax, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            const float *part = attn_slot(P, c, c == c0, rows_tile, D);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + r * D) + d4);
            const float pm = __ldcg(part + rows_tile * D + r);
            const float pl = __ldcg(part + rows_tile * (D + 1) + r);
            const float mx = fmaxf(m, pm), a = exp2f(m - mx), w = exp2f(pm - mx);
            o.x = o.x * a + v.x * w;
            o.y = o.y * a + v.y * w;
            o.z = o.z * a + v.z * w;
            o.w = o.w * a + v.w * w;
            l = l * a + pl * w;
            m = mx;
        }
        const float f = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = attn_row(P, b, head, row0 + r);
        store_out4<T>(P.out, at * D + d4 * 4, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
        if (P.lse && d4 == 0) P.lse[at] = attn_lse(m, l);
    }
}

}  // namespace specv
