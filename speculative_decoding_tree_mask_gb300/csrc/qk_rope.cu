// Norm of every query and key head and the rotation by the node's position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w over the D elements of a head;
//   (a, c) <- (a cos t - c sin t, c cos t + a sin t), t = position * inv_freq[i].
//
// The operator moves each row once in and once out and computes about ten operations an
// element, so DRAM bounds it. A head row is held by a group of 4 to 32 lanes: each lane owns a
// pair of 16-byte vectors whose elements rotate together (vectors j and j + rot/2 for halves,
// neighbours for pairs), so the rotation needs no exchange and the sum of squares a few
// shuffles. The position is the same for all heads of a token, so a warp takes (a share of) the
// heads of one token: it forms the token's rot/2 sines and cosines once, in shared memory, and
// keeps its lanes' own in registers for all its rows. Heads are shared out over more warps
// when there are few tokens, so that a small call still fills the GPU. 16384 tokens of 40 heads
// x 128 in bfloat16 take 58 us, 5.8 TB/s in and out (86% of the measured copy), by pairs 59 us; 256
// tokens 4.3 us.
// Sizes and alignments that 16-byte vectors do not fit take a warp per row.
//
// The angle: turns = position * inv_freq / (2 pi). inv_freq / (2 pi) becomes a 64-bit fixed
// point fraction of a turn (one integer product with floor(2^64 / (2 pi))), the product with the
// position is taken modulo one turn by 64-bit wrap-around, its nearest quarter turn is taken off,
// and 32 bits of the rest become a float: no 64-bit floating point, whose rate is low. The step's
// two cuts cost |position| (|inv_freq| + 1) 2^-64 of a turn, the rest's 2^-34. (A float of the
// whole turn would have 24 bits of it: 2^-26 of a turn near a half turn, where the sine is small.)

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "spec_device.cuh"
#include "spec_internal.h"

namespace specv {
namespace {

constexpr int kWarps = 4;
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

// Work of warp `w`: a share of the heads of one token.
struct Share {
    int64_t token;
    int row0, row1, pos;   // rows: the query heads, then the key heads
};
__device__ __forceinline__ Share warp_share(const QkRopeParams &P, int shares, int per) {
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    Share s;
    s.token = w / shares;
    s.row0 = (int)(w - s.token * shares) * per;
    s.row1 = min(s.row0 + per, P.H[0] + P.H[1]);
    if (s.token >= P.tokens) s.row1 = s.row0 = 0;
    const int64_t t = s.token < P.tokens ? s.token : 0;
    const int b = (int)(t / P.N), n = (int)(t - (int64_t)b * P.N);
    // two's complement addition, so that no pair of inputs is undefined
    s.pos = (int)((uint32_t)P.seq_pos[b] + (uint32_t)(P.depth ? P.depth[t] : n));
    return s;
}

// How a lane's two vectors rotate: with each other (halves whose length is a multiple of a
// vector), each within itself (pairs), or with elements of other lanes, through shared memory
// (other halves: 16384 tokens of 40 heads x 128 with 90 rotated take 84 us, 181 with a warp per
// row and its two-byte loads).
enum Mode { M_HALVES = 0, M_PAIRS = 1, M_ACROSS = 2 };

// T: element type; LPR: lanes per head row.
template <int T, int LPR, int MODE>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_vec(QkRopeParams P, int shares, int per) {
    constexpr bool PAIRS = MODE == M_PAIRS, ACROSS = MODE == M_ACROSS;
    constexpr int E = T == 0 ? 4 : 8;    // elements of a vector
    constexpr int G = 32 / LPR;          // rows a warp holds at a time
    extern __shared__ float2 s_cs[];
    const int lane = threadIdx.x & 31, j = lane % LPR, g = lane / LPR;
    const int half = P.rot / 2, nv = P.D / E, hv = half / E;
    float2 *cs = s_cs + (threadIdx.x >> 5) * half;
    const Share sh = warp_share(P, shares, per);
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
        if (r >= sh.row1) return;
        const int kind = r >= P.H[0];
        const E_t *x = reinterpret_cast<const E_t *>(P.x[kind]) + sh.token * P.stride[kind] +
                       (int64_t)(r - (kind ? P.H[0] : 0)) * P.D;
        if (va >= 0) a = *reinterpret_cast<const uint4 *>(x + va * E);
        if (vb >= 0) b = *reinterpret_cast<const uint4 *>(x + vb * E);
    };
    fetch(sh.row0 + g);      // in flight while the angles are formed
    for (int i = lane; i < half; i += 32) cs[i] = cos_sin(P.inv_freq, i, sh.pos);
    __syncwarp();
    // Element e of the lane's vectors rotates with (c, s)[e]: pair e of the halves, or pair
    // e of the E pairs in the two neighbouring vectors. ACROSS: element e becomes itself times
    // c plus its partner times s, and s has the sign.
    constexpr int K = ACROSS ? 2 * E : E;
    float c[K], s[K];
#pragma unroll
    for (int e = 0; e < K; ++e) {
        const int at = j * K + e;
        const int i = ACROSS ? (at < half ? at : at < P.rot ? at - half : half)
                             : (PAIRS || j < hv ? at : half);
        const float2 v = i < half ? cs[i] : make_float2(1.f, 0.f);
        c[e] = v.x;
        s[e] = ACROSS && at < half ? -v.y : v.y;
    }
    // ACROSS: the rows between norm and rotation. A word is left out after each lane's share, so
    // that the lanes' equal elements lie in different banks.
    const int pitch = P.D + P.D / (2 * E) + 1;
    float *buf = reinterpret_cast<float *>(s_cs + kWarps * half) +
                 ((threadIdx.x >> 5) * G + g) * pitch;
    const float inv_d = 1.f / (float)P.D;
    for (int r0 = sh.row0; r0 < sh.row1; r0 += G) {
        const int r = r0 + g;
        const bool live = r < sh.row1;
        const int kind = r >= P.H[0];
        float x[E], y[E];
        unpack<T>(a, x);
        unpack<T>(b, y);
        fetch(r + G);
        if (P.w[0]) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sum = fmaf(x[e], x[e], sum);
                sum = fmaf(y[e], y[e], sum);   // a lane without a vector holds zeros
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float n = rsqrtf(fmaf(sum, inv_d, P.eps));
            const E_t *w = reinterpret_cast<const E_t *>(P.w[kind]);
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
                if (at >= P.rot) continue;
                const int to = at < half ? at + half : at - half;
                const float p = buf[to + to / (2 * E)];
                float &v = e < E ? x[e % E] : y[e % E];
                v = v * c[e] + p * s[e];
            }
            __syncwarp();
        } else if (PAIRS) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float p = x[e], q = x[e + 1];
                x[e] = p * c[e / 2] - q * s[e / 2];
                x[e + 1] = q * c[e / 2] + p * s[e / 2];
                const float t = y[e], v = y[e + 1];
                y[e] = t * c[E / 2 + e / 2] - v * s[E / 2 + e / 2];
                y[e + 1] = v * c[E / 2 + e / 2] + t * s[E / 2 + e / 2];
            }
        } else if (j < hv) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float p = x[e], q = y[e];
                x[e] = p * c[e] - q * s[e];
                y[e] = q * c[e] + p * s[e];
            }
        }
        if (live) {
            E_t *o = reinterpret_cast<E_t *>(P.y[kind]) + sh.token * P.ystride[kind] +
                     (int64_t)(r - (kind ? P.H[0] : 0)) * P.D;
            if (va >= 0) *reinterpret_cast<uint4 *>(o + va * E) = pack<T>(x);
            if (vb >= 0) *reinterpret_cast<uint4 *>(o + vb * E) = pack<T>(y);
        }
    }
}

// Any head size and alignment: a warp per row, its elements in shared memory between
// the norm and the rotation.
template <int T>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_any(QkRopeParams P, int shares, int per) {
    using E_t = typename Elem<T>::type;
    extern __shared__ float s_any[];
    const int lane = threadIdx.x & 31, D = P.D, half = P.rot / 2;
    float *buf = s_any + (threadIdx.x >> 5) * (2 * half + (D + 1) / 2 * 2);   // even: float2s
    float2 *cs = reinterpret_cast<float2 *>(buf);
    float *row = buf + 2 * half;
    const Share sh = warp_share(P, shares, per);
    for (int i = lane; i < half; i += 32) cs[i] = cos_sin(P.inv_freq, i, sh.pos);
    for (int r = sh.row0; r < sh.row1; ++r) {
        const int kind = r >= P.H[0];
        const int64_t head = (int64_t)(r - (kind ? P.H[0] : 0)) * D;
        const E_t *x = reinterpret_cast<const E_t *>(P.x[kind]) + sh.token * P.stride[kind] + head;
        E_t *o = reinterpret_cast<E_t *>(P.y[kind]) + sh.token * P.ystride[kind] + head;
        const E_t *w = reinterpret_cast<const E_t *>(P.w[kind]);
        float sum = 0.f;
        for (int e = lane; e < D; e += 32) {
            const float v = to_f32<T>(x[e]);
            row[e] = v;
            sum = fmaf(v, v, sum);
        }
        float n = 1.f;
        if (w) {
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            n = rsqrtf(fmaf(sum, 1.f / (float)D, P.eps));
            for (int e = lane; e < D; e += 32) row[e] = row[e] * n * to_f32<T>(w[e]);
        }
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            const int ia = P.pairs ? 2 * i : i, ic = P.pairs ? 2 * i + 1 : i + half;
            const float2 t = cs[i];
            const float p = row[ia], q = row[ic];
            o[ia] = from_f32<T>(p * t.x - q * t.y);
            o[ic] = from_f32<T>(q * t.x + p * t.y);
        }
        for (int e = P.rot + lane; e < D; e += 32) o[e] = from_f32<T>(row[e]);
        __syncwarp();
    }
}

bool vec16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int T, int LPR>
cudaError_t launch_vec(const QkRopeParams &p, int64_t grid, int shares, int per,
                       cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8;
    const size_t smem = sizeof(float2) * (size_t)(kWarps * (p.rot / 2));
    if (p.pairs) {
        qk_rope_vec<T, LPR, M_PAIRS><<<(unsigned)grid, kWarps * 32, smem, st>>>(p, shares, per);
    } else if (p.rot / 2 % E == 0) {
        qk_rope_vec<T, LPR, M_HALVES><<<(unsigned)grid, kWarps * 32, smem, st>>>(p, shares, per);
    } else {
        const size_t rows = sizeof(float) * (size_t)(kWarps * (32 / LPR) *
                                                     (p.D + p.D / (2 * E) + 1));
        qk_rope_vec<T, LPR, M_ACROSS><<<(unsigned)grid, kWarps * 32, smem + rows, st>>>(p, shares,
                                                                                      per);
    }
    return cudaGetLastError();
}

template <int T>
cudaError_t launch_type(const QkRopeParams &p, cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8, es = T == 0 ? 4 : 2;
    bool vec = p.D % E == 0 && p.D / E <= 64;
    for (int i = 0; i < 2; ++i)
        vec = vec && vec16(p.x[i]) && vec16(p.y[i]) && vec16(p.w[i]) &&
              p.stride[i] * es % 16 == 0 && p.ystride[i] * es % 16 == 0;
    const int units = (p.D / E + 1) / 2;
    const int lpr = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
    const int at_once = vec ? 32 / lpr : 1, rows = p.H[0] + p.H[1];
    // rows in rounds of `at_once`; as few rounds a warp as keep 16 warps an SM busy
    const int rounds = (rows + at_once - 1) / at_once;
    const int64_t want = (int64_t)16 * p.sms;
    int64_t shares = (want + p.tokens - 1) / p.tokens;
    shares = shares < 1 ? 1 : shares > rounds ? rounds : shares;
    const int per = (int)((rounds + shares - 1) / shares) * at_once;
    shares = (rows + per - 1) / per;
    const int64_t grid = (p.tokens * shares + kWarps - 1) / kWarps;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (!vec) {
        const size_t smem = sizeof(float) * (size_t)kWarps * (p.rot + (p.D + 1) / 2 * 2);
        qk_rope_any<T><<<(unsigned)grid, kWarps * 32, smem, st>>>(p, (int)shares, per);
        return cudaGetLastError();
    }
    switch (lpr) {
        case 4: return launch_vec<T, 4>(p, grid, (int)shares, per, st);
        case 8: return launch_vec<T, 8>(p, grid, (int)shares, per, st);
        case 16: return launch_vec<T, 16>(p, grid, (int)shares, per, st);
        default: return launch_vec<T, 32>(p, grid, (int)shares, per, st);
    }
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeParams &p, cudaStream_t st) {
    if (p.tokens <= 0) return cudaSuccess;
    if (p.dtype == 0) return launch_type<0>(p, st);
    if (p.dtype == 1) return launch_type<1>(p, st);
    return launch_type<2>(p, st);
}

}  // namespace specv
