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
// x 128 in bfloat16 take 57 us, 5.8 TB/s in and out (86% of the measured copy), by pairs 58 us; 256
// tokens 3.8 us, one call after another.
// Sizes and alignments that 16-byte vectors do not fit take a warp per row.
//
// The angle: turns = position * inv_freq / (2 pi). inv_freq / (2 pi) becomes a 64-bit fixed
// point fraction of a turn (one integer product with floor(2^64 / (2 pi))), the product with the
// position is taken modulo one turn by 64-bit wrap-around, its nearest quarter turn is taken off,
// and 32 bits of the rest become a float: no 64-bit floating point, whose rate is low. The step's
// two cuts cost |position| (|inv_freq| + 1) 2^-64 of a turn, the rest's 2^-34. (A float of the
// whole turn would have 24 bits of it: 2^-26 of a turn near a half turn, where the sine is small.)

#include "rope_device.cuh"

namespace specv {
namespace {

using namespace rope;

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

// The rows of a token where they are and where they go.
template <int T>
struct TokenRows {
    using E_t = typename Elem<T>::type;
    static constexpr int E = T == 0 ? 4 : 8;
    const QkRopeParams &P;
    int64_t token;

    __device__ __forceinline__ const E_t *src(int r) const {
        const int kind = r >= P.H[0];
        return reinterpret_cast<const E_t *>(P.x[kind]) + token * P.stride[kind] +
               (int64_t)(r - (kind ? P.H[0] : 0)) * P.D;
    }
    __device__ __forceinline__ E_t *place(int r) const {
        const int kind = r >= P.H[0];
        return reinterpret_cast<E_t *>(P.y[kind]) + token * P.ystride[kind] +
               (int64_t)(r - (kind ? P.H[0] : 0)) * P.D;
    }
    __device__ __forceinline__ bool turns(int) const { return true; }
    __device__ __forceinline__ bool norm() const { return P.w[0] != nullptr; }
    __device__ __forceinline__ const E_t *weight(int r) const {
        return reinterpret_cast<const E_t *>(P.w[r >= P.H[0]]);
    }
    __device__ __forceinline__ void put(E_t *to, int v, const float (&x)[E]) const {
        *reinterpret_cast<uint4 *>(to + v * E) = pack<T>(x);
    }
    __device__ __forceinline__ void put1(E_t *to, int e, float x) const { to[e] = from_f32<T>(x); }
};

// T: element type; LPR: lanes per head row.
template <int T, int LPR, int MODE>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_vec(QkRopeParams P, int shares, int per) {
    extern __shared__ float2 s_cs[];
    const int warp = threadIdx.x >> 5, half = P.rot / 2;
    const Share sh = warp_share(P, shares, per);
    TokenRows<T> io{P, sh.token};
    float *across = reinterpret_cast<float *>(s_cs + kWarps * half) +
                    warp * (32 / LPR) * across_pitch<T>(P.D);
    share_vec<T, LPR, MODE>(io, sh.row0, sh.row1, sh.pos, P.D, P.rot, P.eps, P.inv_freq,
                            s_cs + warp * half, across);
}

// Any head size and alignment: a warp per row.
template <int T>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_any(QkRopeParams P, int shares, int per,
                                                           int pitch) {
    extern __shared__ float s_any[];
    float *buf = s_any + (threadIdx.x >> 5) * pitch;
    const Share sh = warp_share(P, shares, per);
    TokenRows<T> io{P, sh.token};
    share_any<T>(io, sh.row0, sh.row1, sh.pos, P.D, P.rot, P.pairs, P.eps, P.inv_freq,
                 reinterpret_cast<float2 *>(buf), buf + P.rot);
}

template <int T, int LPR>
cudaError_t launch_vec(const QkRopeParams &p, const Plan &n, cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8;
    const int mode = p.pairs ? M_PAIRS : p.rot / 2 % E == 0 ? M_HALVES : M_ACROSS;
    const size_t smem = smem_vec<T>(mode, LPR, p.D, p.rot);
    const unsigned grid = (unsigned)n.grid;
    if (mode == M_PAIRS)
        qk_rope_vec<T, LPR, M_PAIRS><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    else if (mode == M_HALVES)
        qk_rope_vec<T, LPR, M_HALVES><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    else
        qk_rope_vec<T, LPR, M_ACROSS><<<grid, kWarps * 32, smem, st>>>(p, n.shares, n.per);
    return cudaGetLastError();
}

template <int T>
cudaError_t launch_type(const QkRopeParams &p, cudaStream_t st) {
    constexpr int E = T == 0 ? 4 : 8, es = T == 0 ? 4 : 2;
    bool vec = p.D % E == 0 && p.D / E <= 64;
    for (int i = 0; i < 2; ++i)
        vec = vec && vec16(p.x[i]) && vec16(p.y[i]) && vec16(p.w[i]) &&
              p.stride[i] * es % 16 == 0 && p.ystride[i] * es % 16 == 0;
    const Plan n = plan(p.tokens, p.H[0] + p.H[1], p.D, E, vec, p.sms);
    if (n.grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (!vec) {
        qk_rope_any<T><<<(unsigned)n.grid, kWarps * 32, smem_any(p.D, p.rot), st>>>(
            p, n.shares, n.per, any_pitch(p.D, p.rot));
        return cudaGetLastError();
    }
    switch (n.lpr) {
        case 4: return launch_vec<T, 4>(p, n, st);
        case 8: return launch_vec<T, 8>(p, n, st);
        case 16: return launch_vec<T, 16>(p, n, st);
        default: return launch_vec<T, 32>(p, n, st);
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
