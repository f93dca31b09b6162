// New tokens into the paged cache: queries and keys normalised and rotated, keys and values written
// to their positions' places, in one pass.
//
// The rows and the arithmetic are those of qk_rope.cu (rope_device.cuh): a warp takes a share of one
// token's heads, here the query heads, then the key heads, then the value heads, which are only
// converted. Where a token belongs is found by its warp: a search among the requests' first rows,
// 32 at a time, so that 1024 requests take two dependent loads, then one block-table entry.
// DRAM bounds it: each row once in and once out, and nothing between. Writing K and V where they
// belong instead of in rows saves the copy's read and write of both. 32380 new tokens of 32 + 16 heads
// x 128 in bfloat16 with head norms take 144 us, 5.5 TB/s (81% of the measured copy); 15 tokens 4 us,
// dependent loads from a cold cache.

#pragma once

#include "rope_device.cuh"

namespace specv {
namespace {

using namespace rope;

// Whether request b has row r among its rows, which are within those given.
__device__ __forceinline__ bool has_row(const KvAppendParams &P, int b, int r) {
    const int s = __ldg(P.row_start + b), e = __ldg(P.row_start + b + 1);
    return s >= 0 && e <= P.T && s <= r && r < e;
}

// The request that has row r, or -1; all lanes of a warp, B >= 1. The search takes it that row_start
// does not fall. What it finds is looked at: a request out of range beside others may lead it astray,
// so that they are gone through one after another where it found none (rows of no request pay for that).
__device__ __forceinline__ int owner_of(const KvAppendParams &P, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = P.B;
    do {      // the last of n requests from lo on whose first row is not past r
        const int step = (n + 31) / 32, at = lane * step;
        const bool le = at < n && __ldg(P.row_start + lo + at) <= r;
        const int c = max(1, __popc(__ballot_sync(0xffffffffu, le)));
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
    } while (n > 1);
    if (has_row(P, lo, r)) return lo;
    for (int b = 0; b < P.B; b += 32) {
        const unsigned has = __ballot_sync(0xffffffffu, b + lane < P.B && has_row(P, b + lane, r));
        if (has) return b + __ffs(has) - 1;
    }
    return -1;
}

// KIND: 0 elements of type T, 1 e4m3, 2 e5m2.
template <int KIND>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
    uint16_t r;
    if constexpr (KIND == 1)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

template <int T, int KIND>
struct NewRows {
    using E_t = typename Elem<T>::type;
    static constexpr int E = T == 0 ? 4 : 8;
    const KvAppendParams &P;
    int64_t row;
    char *slot[2];          // K, V: head 0 of the token's place; null if it has none
    int64_t head;           // bytes from one head to the next there
    float scale[2];

    // 0 q, 1 k, 2 v; head within it
    __device__ __forceinline__ int kind(int &r) const {
        if (r < P.Hq) return 0;
        r -= P.Hq;
        if (r < P.cache.H) return 1;
        r -= P.cache.H;
        return 2;
    }
    __device__ __forceinline__ const E_t *src(int r) const {
        const int i = kind(r);
        return reinterpret_cast<const E_t *>(P.x[i]) + row * P.stride[i] + (int64_t)r * P.cache.D;
    }
    __device__ __forceinline__ bool turns(int r) const { return r < P.Hq + P.cache.H; }
    __device__ __forceinline__ bool norm() const { return P.w[1] != nullptr; }
    __device__ __forceinline__ const E_t *weight(int r) const {
        return reinterpret_cast<const E_t *>(P.w[r >= P.Hq]);
    }
    // A row's place: its address, null if it has none, and for a row of an 8-bit cache the scale.
    struct Place {
        char *at;
        bool codes;
        float scale;
    };
    __device__ __forceinline__ Place place(int r) const {
        const int i = kind(r);
        if (i == 0)
            return Place{reinterpret_cast<char *>(reinterpret_cast<E_t *>(P.q_out) +
                                                  row * P.q_out_stride + (int64_t)r * P.cache.D),
                         false, 1.f};
        char *to = i == 1 ? slot[0] : slot[1];
        return Place{to ? to + r * head : nullptr, KIND != 0, i == 1 ? scale[0] : scale[1]};
    }
    __device__ __forceinline__ void put(const Place &p, int v, const float (&x)[E]) const {
        if (!p.at) return;
        if (KIND == 0 || !p.codes) {
            *reinterpret_cast<uint4 *>(p.at + v * 16) = pack<T>(x);
            return;
        }
        uint32_t w[E / 4];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __fdiv_rn(x[e + k], p.scale);
            w[e / 4] = fp8x2<KIND>(y[0], y[1]) | fp8x2<KIND>(y[2], y[3]) << 16;
        }
        if constexpr (E == 8)
            *reinterpret_cast<uint2 *>(p.at + v * 8) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p.at + v * 4) = w[0];
    }
    __device__ __forceinline__ void put1(const Place &p, int e, float x) const {
        if (!p.at) return;
        if (KIND == 0 || !p.codes)
            reinterpret_cast<E_t *>(p.at)[e] = from_f32<T>(x);
        else
            reinterpret_cast<uint8_t *>(p.at)[e] = (uint8_t)fp8x2<KIND>(__fdiv_rn(x, p.scale), 0.f);
    }
};

// A warp's token: its rows, where it goes, and its position; no rows if it is no request's.
template <int T, int KIND>
__device__ __forceinline__ NewRows<T, KIND> warp_rows(const KvAppendParams &P, int shares, int per,
                                                      int &row0, int &row1, int &pos) {
    const spec_kv_cache &C = P.cache;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    NewRows<T, KIND> io{P, w / shares, {nullptr, nullptr}, 0, {1.f, 1.f}};
    if (P.status && P.row_start && blockIdx.x == 0)
        for (int b = threadIdx.x; b < P.B; b += kWarps * 32) {
            const int s = P.row_start[b], e = P.row_start[b + 1];
            if (s < 0 || e > P.T || s > e) atomicMax(P.status + b, SPEC_REQ_BAD_RANGE);
        }
    row0 = (int)(w - io.row * shares) * per;
    row1 = min(row0 + per, P.Hq + 2 * C.H);
    pos = 0;
    int b = -1, first = 0;
    if (io.row < P.T) {
        if (P.row_start) {
            b = owner_of(P, (int)io.row);
            if (b >= 0) first = __ldg(P.row_start + b);
        } else {
            b = (int)(io.row / P.N);
            first = b * P.N;
        }
    }
    if (b < 0) {
        row0 = row1 = 0;
        return io;
    }
    // two's complement addition, so that no pair of inputs is undefined
    pos = (int)((uint32_t)__ldg(P.seq_pos + b) + (uint32_t)((int)io.row - first));
    const int page = pos < 0 ? -1 : (int)((uint32_t)pos / (uint32_t)C.block_size);
    const int block = page >= 0 && page < C.max_blocks
                          ? __ldg(C.block_table + (int64_t)b * C.max_blocks + page)
                          : -1;
    if (block >= 0 && block < C.num_blocks) {
        const int off = pos - page * C.block_size;
        const int64_t e = KIND == 0 ? (int64_t)sizeof(typename Elem<T>::type) : 1;
        const int64_t in = (C.layout == SPEC_KV_NHD ? (int64_t)off * C.H : off) * C.D;
        io.slot[0] = static_cast<char *>(C.k) + (block * C.k_block_stride + in) * e;
        io.slot[1] = static_cast<char *>(C.v) + (block * C.v_block_stride + in) * e;
        io.head = (C.layout == SPEC_KV_NHD ? C.D : (int64_t)C.block_size * C.D) * e;
    } else if (P.status && row0 == 0 && (threadIdx.x & 31) == 0) {
        atomicMax(P.status + b, SPEC_REQ_BAD_SLOT);
    }
    if (KIND != 0) {
        if (C.k_scale) io.scale[0] = __ldg(C.k_scale);
        if (C.v_scale) io.scale[1] = __ldg(C.v_scale);
    }
    return io;
}

template <int T, int KIND, int LPR, int MODE>
__global__ void __launch_bounds__(kWarps * 32)
    kv_append_vec(KvAppendParams P, int shares, int per) {
    extern __shared__ float2 s_cs[];
    const int warp = threadIdx.x >> 5, half = P.rot / 2, D = P.cache.D;
    int row0, row1, pos;
    const NewRows<T, KIND> io = warp_rows<T, KIND>(P, shares, per, row0, row1, pos);
    float *across = reinterpret_cast<float *>(s_cs + kWarps * half) +
                    warp * (32 / LPR) * across_pitch<T>(D);
    share_vec<T, LPR, MODE>(io, row0, row1, pos, D, P.rot, P.eps, P.inv_freq, s_cs + warp * half,
                            across);
}

template <int T, int KIND>
__global__ void __launch_bounds__(kWarps * 32)
    kv_append_any(KvAppendParams P, int shares, int per, int pitch) {
    extern __shared__ float s_any[];
    float *buf = s_any + (threadIdx.x >> 5) * pitch;
    int row0, row1, pos;
    const NewRows<T, KIND> io = warp_rows<T, KIND>(P, shares, per, row0, row1, pos);
    share_any<T>(io, row0, row1, pos, P.cache.D, P.rot, P.pairs, P.eps, P.inv_freq,
                 reinterpret_cast<float2 *>(buf), buf + P.rot);
}

template <int T, int KIND, int LPR>
cudaError_t launch_vec(const KvAppendParams &p, const Plan &n, cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8;
    const int mode = p.pairs ? M_PAIRS : p.rot / 2 % E == 0 ? M_HALVES : M_ACROSS;
    const size_t smem = smem_vec<T>(mode, LPR, p.cache.D, p.rot);
    const unsigned grid = (unsigned)n.grid;
    if (mode == M_PAIRS)
        kv_append_vec<T, KIND, LPR, M_PAIRS><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    else if (mode == M_HALVES)
        kv_append_vec<T, KIND, LPR, M_HALVES><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    else
        kv_append_vec<T, KIND, LPR, M_ACROSS><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    return cudaGetLastError();
}

template <int T, int KIND>
cudaError_t launch_kind(const KvAppendParams &p, cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8, es = T == 0 ? 4 : 2;
    const int D = p.cache.D;
    bool vec = D % E == 0 && D / E <= 64 && vec16(p.q_out) && p.q_out_stride * es % 16 == 0;
    for (int i = 0; i < 3; ++i) vec = vec && vec16(p.x[i]) && p.stride[i] * es % 16 == 0;
    vec = vec && vec16(p.w[0]) && vec16(p.w[1]);
    const Plan n = plan(p.T, p.Hq + 2 * p.cache.H, D, E, vec, p.sms);
    if (n.grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (!vec) {
        kv_append_any<T, KIND><<<(unsigned)n.grid, kWarps * 32, smem_any(D, p.rot), st>>>(
            p, n.shares, n.per, any_pitch(D, p.rot));
        return cudaGetLastError();
    }
    switch (n.lpr) {
        case 4: return launch_vec<T, KIND, 4>(p, n, st);
        case 8: return launch_vec<T, KIND, 8>(p, n, st);
        case 16: return launch_vec<T, KIND, 16>(p, n, st);
        default: return launch_vec<T, KIND, 32>(p, n, st);
    }
}

}  // namespace

template <int T>
cudaError_t launch_kv_append_type(const KvAppendParams &p, cudaStream_t st) {
    if (p.cache.kind == SPEC_CACHE_SAME) return launch_kind<T, 0>(p, st);
    if (p.cache.kind == SPEC_CACHE_FP8_E4M3) return launch_kind<T, 1>(p, st);
    return launch_kind<T, 2>(p, st);
}

}  // namespace specv
