// The norm of a head and the rotation by a position, as the kernels that write queries and keys
// share them: angles, element types, and a warp's share of one token's heads. Internal.
//
// The kernel brings an IO with
//   const E_t *src(int r)      row r of the token (its heads one after another);
//   bool turns(int r)          whether the row is normalised and rotated (values are not);
//   const E_t *weight(int r)   norm weights; norm(): whether there are any;
//   Place place(int r)         where row r goes, once for all of it;
//   void put(Place p, int v, const float (&x)[E])   its vector v (E elements of 16 bytes);
//   void put1(Place p, int e, float x)              element e, for rows that 16-byte vectors do not fit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "spec_device.cuh"
#include "spec_internal.h"

namespace specv {
namespace rope {

constexpr int kWarps = 4;           // of a CTA
constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;   // floor(2^64 / (2 pi))

// inv_freq / (2 pi) of a turn as a fraction of 2^64 (modulo one turn).
__device__ __forceinline__ uint64_t turn_step(float f) {
    const uint32_t u = __float_as_uint(f);
    const int e = (int)((u >> 23) & 0xffu);
    const uint32_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - (e ? e : 1);   // |f| = m * 2^-s
    const uint64_t lo = (uint64_t)m * kInv2Pi, hi = __umul64hi((uint64_t)m, kInv2Pi);
    uint64_t t;
    if (s <= 0)
        t = s > -64 ? lo << -s : 0;
    else if (s < 64)
        t = (lo >> s) | (hi << (64 - s));
    else
        t = s < 128 ? hi >> (s - 64) : 0;
    return (u >> 31) ? 0 - t : t;
}

// (cos, sin) of pair i at `pos`.
__device__ __forceinline__ float2 cos_sin(const float *inv_freq, int i, int pos) {
    const float f = __ldg(inv_freq + i);
    const uint64_t turn = (uint64_t)(int64_t)pos * turn_step(f);
    const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);       // the nearest
    const int rest = (int)((int64_t)(turn - ((uint64_t)quarter << 62)) >> 30);   // of 2^34
    float s, c;
    sincospif((float)rest * 1.1641532182693481e-10f, &s, &c);   // 2^-33: a turn is 2 half turns
    if (!(fabsf(f) < INFINITY)) s = c = NAN;
    const float2 r = quarter & 1 ? make_float2(-s, c) : make_float2(c, s);
    return quarter & 2 ? make_float2(-r.x, -r.y) : r;
}

template <int T>
struct Elem;
template <>
struct Elem<0> {
    using type = float;
};
template <>
struct Elem<1> {
    using type = __nv_bfloat16;
};
template <>
struct Elem<2> {
    using type = __half;
};

template <int T>
__device__ __forceinline__ float to_f32(typename Elem<T>::type x) {
    if constexpr (T == 0) return x;
    if constexpr (T == 1) return __bfloat162float(x);
    if constexpr (T == 2) return __half2float(x);
}
template <int T>
__device__ __forceinline__ typename Elem<T>::type from_f32(float x) {
    if constexpr (T == 0) return x;
    if constexpr (T == 1) return __float2bfloat16_rn(x);
    if constexpr (T == 2) return __float2half_rn(x);
}

// Elements of a 16-byte vector as floats, and back.
template <int T>
__device__ __forceinline__ void unpack(const uint4 &a, float *x) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == 0) {
            x[i] = __uint_as_float(w[i]);
        } else if constexpr (T == 1) {
            x[2 * i] = bf_lo(w[i]);
            x[2 * i + 1] = bf_hi(w[i]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <int T>
__device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == 0) {
            w[i] = __float_as_uint(x[i]);
        } else if constexpr (T == 1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// How a lane's two vectors rotate: with each other (halves whose length is a multiple of a
// vector), each within itself (pairs), or with elements of other lanes, through shared memory
// (other halves: 16384 tokens of 40 heads x 128 with 90 rotated take 84 us, 181 with a warp per
// row and its two-byte loads).
enum Mode { M_HALVES = 0, M_PAIRS = 1, M_ACROSS = 2 };

// Floats between two rows of the ACROSS form's shared memory.
template <int T>
__host__ __device__ constexpr int across_pitch(int D) {
    return D + D / (2 * (T == 0 ? 4 : 8)) + 1;
}

// Rows [row0, row1) of a token at `pos`, by one warp. LPR: lanes per head row; cs: rot / 2 float2s
// of this warp's in shared memory; across: (32 / LPR) rows of the pitch below (ACROSS only).
template <int T, int LPR, int MODE, typename IO>
__device__ __forceinline__ void share_vec(IO &io, int row0, int row1, int pos, int D, int rot, float eps,
                                          const float *inv_freq, float2 *cs, float *across) {
    constexpr bool PAIRS = MODE == M_PAIRS, ACROSS = MODE == M_ACROSS;
    constexpr int E = T == 0 ? 4 : 8;    // elements of a vector
    constexpr int G = 32 / LPR;          // rows a warp holds at a time
    const int lane = threadIdx.x & 31, j = lane % LPR, g = lane / LPR;
    const int half = rot / 2, nv = D / E, hv = half / E;
    // this lane's vectors, -1 if none
    int va, vb;
    if (PAIRS || ACROSS) {
        va = 2 * j;
        vb = 2 * j + 1;
    } else if (j < hv) {
        va = j;
        vb = j + hv;
    } else {
        va = 2 * j;          // 2 hv + 2 (j - hv)
        vb = 2 * j + 1;
    }
    if (va >= nv) va = -1;
    if (vb >= nv) vb = -1;
    using E_t = typename Elem<T>::type;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    auto fetch = [&](int r) {
        if (r >= row1) return;
        const E_t *x = io.src(r);
        if (va >= 0) a = *reinterpret_cast<const uint4 *>(x + va * E);
        if (vb >= 0) b = *reinterpret_cast<const uint4 *>(x + vb * E);
    };
    fetch(row0 + g);         // in flight while the angles are formed
    for (int i = lane; i < half; i += 32) cs[i] = cos_sin(inv_freq, i, pos);
    __syncwarp();
    // Element e of the lane's vectors rotates with (c, s)[e]: pair e of the halves, or pair
    // e of the E pairs in the two neighbouring vectors. ACROSS: element e becomes itself times
    // c plus its partner times s, and s has the sign.
    constexpr int K = ACROSS ? 2 * E : E;
    float c[K], s[K];
#pragma unroll
    for (int e = 0; e < K; ++e) {
        const int at = j * K + e;
        const int i = ACROSS ? (at < half ? at : at < rot ? at - half : half)
                             : (PAIRS || j < hv ? at : half);
        const float2 v = i < half ? cs[i] : make_float2(1.f, 0.f);
        c[e] = v.x;
        s[e] = ACROSS && at < half ? -v.y : v.y;
    }
    // ACROSS: the rows between norm and rotation. A word is left out after each lane's share, so
    // that the lanes' equal elements lie in different banks.
    float *buf = across + g * across_pitch<T>(D);
    const float inv_d = 1.f / (float)D;
    for (int r0 = row0; r0 < row1; r0 += G) {
        const int r = r0 + g;
        const bool live = r < row1, turns = io.turns(r);
        float x[E], y[E];
        unpack<T>(a, x);
        unpack<T>(b, y);
        fetch(r + G);
        if (io.norm()) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sum = fmaf(x[e], x[e], sum);
                sum = fmaf(y[e], y[e], sum);   // a lane without a vector holds zeros
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (turns) {
                const float n = rsqrtf(fmaf(sum, inv_d, eps));
                const E_t *w = io.weight(r);
                float u[E];
                if (va >= 0) {
                    unpack<T>(__ldg(reinterpret_cast<const uint4 *>(w + va * E)), u);
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = x[e] * n * u[e];
                }
                if (vb >= 0) {
                    unpack<T>(__ldg(reinterpret_cast<const uint4 *>(w + vb * E)), u);
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = y[e] * n * u[e];
                }
            }
        }
        if (ACROSS) {
            float *mine = buf + j * (2 * E + 1);
            if (va >= 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) mine[e] = x[e];
            }
            if (vb >= 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) mine[E + e] = y[e];
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) {
                const int at = j * 2 * E + e;
                if (at >= rot || !turns) continue;
                const int to = at < half ? at + half : at - half;
                const float p = buf[to + to / (2 * E)];
                float &v = e < E ? x[e % E] : y[e % E];
                v = v * c[e] + p * s[e];
            }
            __syncwarp();
        } else if (PAIRS) {
            if (turns) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float p = x[e], q = x[e + 1];
                    x[e] = p * c[e / 2] - q * s[e / 2];
                    x[e + 1] = q * c[e / 2] + p * s[e / 2];
                    const float t = y[e], v = y[e + 1];
                    y[e] = t * c[E / 2 + e / 2] - v * s[E / 2 + e / 2];
                    y[e + 1] = v * c[E / 2 + e / 2] + t * s[E / 2 + e / 2];
                }
            }
        } else if (j < hv && turns) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float p = x[e], q = y[e];
                x[e] = p * c[e] - q * s[e];
                y[e] = q * c[e] + p * s[e];
            }
        }
        if (live) {
            const auto to = io.place(r);
            if (va >= 0) io.put(to, va, x);
            if (vb >= 0) io.put(to, vb, y);
        }
    }
}

// The same for any head size and alignment: the row's elements in shared memory (row) between
// norm and rotation.
template <int T, typename IO>
__device__ __forceinline__ void share_any(IO &io, int row0, int row1, int pos, int D, int rot, int pairs,
                                          float eps, const float *inv_freq, float2 *cs, float *row) {
    using E_t = typename Elem<T>::type;
    const int lane = threadIdx.x & 31, half = rot / 2;
    for (int i = lane; i < half; i += 32) cs[i] = cos_sin(inv_freq, i, pos);
    for (int r = row0; r < row1; ++r) {
        const E_t *x = io.src(r);
        const auto to = io.place(r);
        const bool turns = io.turns(r);
        const int turned = turns ? half : 0;
        float sum = 0.f;
        for (int e = lane; e < D; e += 32) {
            const float v = to_f32<T>(x[e]);
            row[e] = v;
            sum = fmaf(v, v, sum);
        }
        if (turns && io.norm()) {
            const E_t *w = io.weight(r);
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            const float n = rsqrtf(fmaf(sum, 1.f / (float)D, eps));
            for (int e = lane; e < D; e += 32) row[e] = row[e] * n * to_f32<T>(w[e]);
        }
        __syncwarp();
        for (int i = lane; i < turned; i += 32) {
            const int ia = pairs ? 2 * i : i, ic = pairs ? 2 * i + 1 : i + half;
            const float2 t = cs[i];
            const float p = row[ia], q = row[ic];
            io.put1(to, ia, p * t.x - q * t.y);
            io.put1(to, ic, q * t.x + p * t.y);
        }
        for (int e = 2 * turned + lane; e < D; e += 32) io.put1(to, e, row[e]);
        __syncwarp();
    }
}

inline bool vec16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// How a launch shares out `rows` head rows a token.
struct Plan {
    int lpr, shares, per;     // lanes per row; warps of a token, rows of each
    int64_t grid;
};
inline Plan plan(int64_t tokens, int rows, int D, int E, bool vec, int sms) {
    Plan p;
    const int units = (D / E + 1) / 2;
    p.lpr = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
    const int at_once = vec ? 32 / p.lpr : 1;
    // rows in rounds of `at_once`; as few rounds a warp as keep 16 warps an SM busy
    const int rounds = (rows + at_once - 1) / at_once;
    const int64_t want = (int64_t)16 * sms;
    int64_t shares = (want + tokens - 1) / tokens;
    shares = shares < 1 ? 1 : shares > rounds ? rounds : shares;
    p.per = (int)((rounds + shares - 1) / shares) * at_once;
    p.shares = (rows + p.per - 1) / p.per;
    p.grid = (tokens * p.shares + kWarps - 1) / kWarps;
    return p;
}
// Dynamic shared memory of a CTA.
template <int T>
size_t smem_vec(int mode, int lpr, int D, int rot) {
    const size_t cs = sizeof(float2) * (size_t)(kWarps * (rot / 2));
    return mode == M_ACROSS ? cs + sizeof(float) * (size_t)(kWarps * (32 / lpr) * across_pitch<T>(D))
                            : cs;
}
inline int any_pitch(int D, int rot) { return rot + (D + 1) / 2 * 2; }     // even: float2s first
inline size_t smem_any(int D, int rot) { return sizeof(float) * (size_t)kWarps * any_pitch(D, rot); }

}  // namespace rope
}  // namespace specv
