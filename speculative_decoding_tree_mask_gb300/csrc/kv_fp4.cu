// The 4-bit paged KV cache: rows quantised as they are written, and read back.
//
// A block of 16 consecutive elements of a head is the unit of both kernels, one thread each:
//   s = e4m3(amax * c),  code = e2m1(x * m),  c = RN(r * RN(1/6)), m = RN(RN(1/s) * r),
// with r = RN(1 / tensor scale); back, value = code * s * tensor scale. The quotients are
// products with rounded reciprocals by definition, so that every implementation that follows
// the formulas in float32 stores the same codes. Consecutive threads take consecutive blocks,
// so a warp reads 1 KB of 16-bit rows and writes 256 bytes of codes and 32 of scales side by
// side. Reading back is bound by DRAM once there are enough rows (16 x 16384 positions, 8 heads
// x 128, to bfloat16: 195 us, 6.4 TB/s). A commit writes few slots a request: 2048 slots of 32
// heads x 128 take 16 us where their bytes need 6, in dependent loads (length, node and block,
// row) and about 290 instructions a block.

#include "fp4_device.cuh"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kSmemRequests = 2048;   // requests whose last slot and position fit in shared memory
// Commit: blocks of 16 elements a thread handles at a time, CTAs an SM holds. With their read-back,
// 2048 slots of 32 heads x 128 and 4 x 4097 rows of 8 heads x 80: 33 and 28 us with 2 and 3; 36 and 32
// with 1 and 6; 40 and 41 with 1 and 8; 35 and 31 with 4 and 2.
constexpr int kCommitItems = 2, kCommitUnit = kThreads * kCommitItems, kCommitCtas = 3;
// Load: blocks a thread handles, 4 when that fills the GPU, else 1 (333 positions of two
// requests, 4 heads x 64: 2.9 us against 4.3); a CTA has one unit of them (16 x 16384 positions,
// 8 heads x 128: 195 us; 222 with CTAs that stride over the units, 312 with one block a thread).
constexpr int kLoadItems = 4, kLoadCtas = 8;

// A thread's 16 elements as floats. vec: 32, 16 (byte alignment of every block) or 0.
template <int T>
__device__ __forceinline__ void load16(const void *base, int64_t e, int vec, uint32_t (&w)[16]) {
    constexpr int W = T == 0 ? 16 : 8;   // 32-bit words
    const char *p = reinterpret_cast<const char *>(base) + e * (T == 0 ? 4 : 2);
    if (vec == 32) {
#pragma unroll
        for (int i = 0; i < W; i += 8)
            asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]),
                           "=r"(w[i + 4]), "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                         : "l"(p + i * 4));
    } else if (vec == 16) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + i * 4));
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (T == 0) {
                w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
            } else {
                const unsigned short *q = reinterpret_cast<const unsigned short *>(p) + 2 * i;
                w[i] = (uint32_t)__ldg(q) | (uint32_t)__ldg(q + 1) << 16;
            }
        }
    }
}

template <int T>
__device__ __forceinline__ void floats16(const uint32_t (&w)[16], float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < (T == 0 ? 16 : 8); ++i) {
        if (T == 0) {
            x[i] = __uint_as_float(w[i]);
        } else if (T == 1) {
            x[2 * i] = bf_lo(w[i]);
            x[2 * i + 1] = bf_hi(w[i]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// One block: codes in c, the scale's code returned. r = RN(1 / tensor scale).
__device__ __forceinline__ uint32_t quantise16(const float (&x)[16], float r, uint2 &c) {
    float a = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) a = fmax_nan(a, fabsf(x[i]));
    const uint32_t sf = f32_to_e4m3(a * (r * (1.f / 6.f)));
    // the scale's float: exact through a half
    const uint32_t h = e4m3x2_to_f16x2(sf);
    const float s = __half2float(__ushort_as_half((unsigned short)h));
    const float m = s > 0.f ? __frcp_rn(s) * r : 0.f;   // s 0: codes 0; s NaN: any codes
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x[i] * m;
    c.x = f32x8_to_e2m1x8(y);
    c.y = f32x8_to_e2m1x8(y + 8);
    return sf;
}

// ---- commit ----------------------------------------------------------------------------------

// The last slot request b writes, or -1.
__device__ __forceinline__ int last_slot(const KvFp4Params &P, int b) {
    if (P.kv_commit && __ldg(P.kv_commit + (int64_t)b * P.N) < 0) return -1;
    return P.last ? min(__ldg(P.last + b), P.N - 1) : P.N - 1;
}

// SPEC_REQ_BAD_SLOT if a slot of request b has no place, else 0. One warp.
__device__ __forceinline__ void commit_status(const KvFp4Params &P, int b, int last, int lane) {
    bool bad = false;
    for (int j = lane; j <= last; j += 32) {
        const int node = P.kv_commit ? __ldg(P.kv_commit + (int64_t)b * P.N + j) : j;
        int off;
        bad |= node < 0 || node >= P.N ||
               fp4_block(P.cache, P.by_page, b, (int64_t)P.pos[b] + j, &off) < 0;
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) P.status[b] = bad ? SPEC_REQ_BAD_SLOT : 0;
}

// Units of `slots` consecutive slots x all 16-element blocks of K and V of a request (or a
// piece of one slot when that is more than a unit), slot groups outermost: the slots that every
// request writes come first, and the CTAs, a wave of them striding over the units, stop at the
// last slot that any request writes. A unit costs two round trips, its nodes and cache blocks
// and then its rows; the first is made while the unit before waits for its rows.
template <int T>
__global__ void __launch_bounds__(kThreads, kCommitCtas)
    commit_kernel(KvFp4Params P, int slots, int pieces, int vec) {
    extern __shared__ int2 s_req[];      // (last slot, position) of each request
    __shared__ int s_max;
    constexpr int I = kCommitItems;
    const spec_fp4_cache &c = P.cache;
    const int tid = threadIdx.x, B = P.B;
    const bool cached = B <= kSmemRequests;
    const int per_head = c.D / 16, row = c.H * per_head;   // blocks of a head, of a K row
    int most = P.N - 1;
    if (cached) {
        if (tid == 0) s_max = -1;
        __syncthreads();
        int m = -1;
        for (int b = tid; b < B; b += kThreads) {
            const int2 r = make_int2(last_slot(P, b), __ldg(P.pos + b));
            s_req[b] = r;
            m = max(m, r.x);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((tid & 31) == 0) atomicMax(&s_max, m);
        __syncthreads();
        most = s_max;
    }
    auto request = [&](int b) {
        return cached ? s_req[b] : make_int2(last_slot(P, b), __ldg(P.pos + b));
    };
    if (P.status)
        for (int b = (gridDim.x - 1 - blockIdx.x) * (kThreads / 32) + tid / 32; b < B;
             b += gridDim.x * (kThreads / 32))
            commit_status(P, b, request(b).x, tid & 31);
    const float rk = __frcp_rn(c.k_scale ? __ldg(c.k_scale) : 1.f);
    const float rv = __frcp_rn(c.v_scale ? __ldg(c.v_scale) : 1.f);
    const int64_t units = (most < 0 ? 0 : most / slots + 1) * (int64_t)B * pieces;
    // One block of 16 elements: where it comes from and goes.
    struct Item {
        int node, blk, off, e;   // e: block of the K row, or of the V row behind it; -1: nothing
    };
    int b = 0;
    // this thread's items of the next unit at or after u that writes something
    auto find = [&](int64_t u, Item (&it)[I]) -> int64_t {
        for (; u < units; u += gridDim.x) {
            const int64_t gb = pieces == 1 ? u : u / pieces, group = gb / B;
            b = (int)(gb - group * B);
            const int2 req = request(b);
            const int j0 = (int)group * slots;
            if (j0 > req.x) continue;
            const int n = min(slots, req.x - j0 + 1);
            const int lo = (int)(u - gb * pieces) * kCommitUnit, hi = min(n * 2 * row, lo + kCommitUnit);
#pragma unroll
            for (int q = 0; q < I; ++q) {
                const int i = lo + tid + q * kThreads;
                it[q].e = -1;
                it[q].node = it[q].blk = it[q].off = 0;
                if (i >= hi) continue;
                const int sl = slots == 1 ? 0 : (int)(P.by_row(i) >> 1), j = j0 + sl;
                it[q].e = i - sl * 2 * row;
                it[q].node = P.kv_commit ? __ldg(P.kv_commit + (int64_t)b * P.N + j) : j;
                it[q].blk = fp4_block(c, P.by_page, b, (int64_t)req.y + j, &it[q].off);
            }
            return u;
        }
        return units;
    };
    Item it[I];
    int64_t u = find(blockIdx.x, it);
    while (u < units) {
        uint32_t w[I][16];
        int64_t place[I];        // of the block in the cache, -1: nothing
        bool isv[I];
#pragma unroll
        for (int q = 0; q < I; ++q) {
            isv[q] = it[q].e >= row;
            const int e = isv[q] ? it[q].e - row : it[q].e, head = (int)P.by_head(max(e, 0));
            place[q] = -1;
            if (it[q].e < 0 || it[q].node < 0 || it[q].node >= P.N || it[q].blk < 0) continue;
            place[q] = (int64_t)fp4_row(c, it[q].blk, it[q].off, head) * per_head +
                       (e - head * per_head);
            load16<T>(P.src[isv[q]], ((int64_t)b * P.N + it[q].node) * P.stride[isv[q]] + e * 16,
                      vec, w[q]);
        }
        u = find(u + gridDim.x, it);
#pragma unroll
        for (int q = 0; q < I; ++q) {
            if (place[q] < 0) continue;
            float x[16];
            floats16<T>(w[q], x);
            uint2 code;
            const uint32_t sf = quantise16(x, isv[q] ? rv : rk, code);
            reinterpret_cast<uint2 *>(isv[q] ? c.v : c.k)[place[q]] = code;
            reinterpret_cast<uint8_t *>(isv[q] ? c.v_sf : c.k_sf)[place[q]] = (uint8_t)sf;
        }
    }
}

// ---- load ------------------------------------------------------------------------------------

template <int T>
__device__ __forceinline__ void store16(void *base, int64_t e, int vec, const float (&x)[16]) {
    constexpr int W = T == 0 ? 16 : 8;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (T == 0) {
            w[i] = __float_as_uint(x[i]);
        } else if (T == 1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    char *p = reinterpret_cast<char *>(base) + e * (T == 0 ? 4 : 2);
    if (vec == 32) {
#pragma unroll
        for (int i = 0; i < W; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             p + i * 4),
                         "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                         "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                         : "memory");
    } else if (vec == 16) {
#pragma unroll
        for (int i = 0; i < W; i += 4)
            *reinterpret_cast<uint4 *>(p + i * 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (T == 0) {
                reinterpret_cast<uint32_t *>(p)[i] = w[i];
            } else {
                reinterpret_cast<unsigned short *>(p)[2 * i] = (unsigned short)w[i];
                reinterpret_cast<unsigned short *>(p)[2 * i + 1] = (unsigned short)(w[i] >> 16);
            }
        }
    }
}

// Units of I x kThreads consecutive 16-element blocks of one request's K or V output rows.
template <int T, int I>
__global__ void __launch_bounds__(kThreads, T == 0 ? 6 : kLoadCtas)
    load_kernel(KvFp4Params P, int64_t per, int vec) {
    const spec_fp4_cache &c = P.cache;
    const int tid = threadIdx.x;
    const uint32_t per_head = c.D / 16, row = (uint32_t)c.H * per_head;
    const int64_t each = P.max_len * row;                 // blocks of K (and of V) of a request
    const float ks = c.k_scale ? __ldg(c.k_scale) : 1.f;
    const float vs = c.v_scale ? __ldg(c.v_scale) : 1.f;
    for (int64_t u = blockIdx.x; u < 2 * per * P.B; u += gridDim.x) {
        const int64_t bk = u / per, lo = (u - bk * per) * (kThreads * I);
        const int b = (int)(bk >> 1), isv = (int)(bk & 1);
        const int64_t tok0 = lo / row;
        const uint32_t rem0 = (uint32_t)(lo - tok0 * row);
        const int start = __ldg(P.pos + b), count = __ldg(P.last + b);
        const uint2 *codes = reinterpret_cast<const uint2 *>(isv ? c.v : c.k);
        const uint8_t *scales = reinterpret_cast<const uint8_t *>(isv ? c.v_sf : c.k_sf);
        uint2 code[I];
        uint32_t sf[I];
        bool seen = true;
#pragma unroll
        for (int q = 0; q < I; ++q) {
            const uint32_t i = tid + q * kThreads, k = rem0 + i, tok = P.by_row(k);
            const uint32_t e = k - tok * row;
            code[q] = make_uint2(0, 0);
            sf[q] = 0;
            if (lo + i >= each || tok0 + tok >= count) continue;
            int off = 0;
            const int blk = fp4_block(c, P.by_page, b, start + tok0 + tok, &off);
            if (blk < 0) {
                seen = false;
                continue;
            }
            const uint32_t head = P.by_head(e);
            const int64_t place =
                (int64_t)fp4_row(c, blk, off, (int)head) * per_head + (e - head * per_head);
            code[q] = __ldg(codes + place);
            sf[q] = __ldg(scales + place);
        }
        if (P.status && (!seen || count < 0 || count > P.max_len))
            P.status[b] = SPEC_REQ_BAD_SLOT;
#pragma unroll
        for (int q = 0; q < I; ++q) {
            const int64_t i = lo + tid + q * kThreads;
            if (i >= each) continue;
            const uint32_t h = e4m3x2_to_f16x2(sf[q]);
            const float s = __half2float(__ushort_as_half((unsigned short)h));
            const float ts = isv ? vs : ks;
            float x[16];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint32_t r[4];
                e2m1x8_to_f16x2(w ? code[q].y : code[q].x, r);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r[y]));
                    // code * block scale is exact; the tensor scale rounds once
                    x[w * 8 + 2 * y] = f.x * s * ts;
                    x[w * 8 + 2 * y + 1] = f.y * s * ts;
                }
            }
            store16<T>(P.out[isv], (b * each + i) * 16, vec, x);
        }
    }
}

KvFp4Params with_divisors(const KvFp4Params &given) {
    KvFp4Params p = given;
    p.by_head = FastDiv((uint32_t)p.cache.D / 16);
    p.by_row = FastDiv((uint32_t)p.cache.H * (p.cache.D / 16));
    p.by_page = FastDiv((uint32_t)p.cache.block_size);
    return p;
}

// Alignment that every block's 16 elements share: 32 or 16 bytes, or 0.
int align_of(const void *p, int64_t stride_bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes;
    return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 0;
}

template <int T>
cudaError_t commit_type(const KvFp4Params &p, cudaStream_t st) {
    constexpr int es = T == 0 ? 4 : 2;
    const int a = align_of(p.src[0], p.stride[0] * es), b = align_of(p.src[1], p.stride[1] * es);
    const int row2 = 2 * p.cache.H * (p.cache.D / 16);
    const int slots = row2 >= kCommitUnit ? 1 : kCommitUnit / row2;
    const int pieces = (slots * row2 + kCommitUnit - 1) / kCommitUnit;
    const int64_t units = ((int64_t)(p.N - 1) / slots + 1) * p.B * pieces;
    const int64_t cap = (int64_t)p.sms * kCommitCtas;
    const size_t smem = p.B <= kSmemRequests ? sizeof(int2) * (size_t)p.B : 0;
    commit_kernel<T><<<(unsigned)(units < cap ? units : cap), kThreads, smem, st>>>(
        p, slots, pieces, a < b ? a : b);
    return cudaGetLastError();
}

template <int T>
cudaError_t load_type(const KvFp4Params &p, cudaStream_t st) {
    const int a = align_of(p.out[0], 0), b = align_of(p.out[1], 0);
    const int64_t each = p.max_len * p.cache.H * (p.cache.D / 16);
    const bool many = 2 * each * p.B >= (int64_t)p.sms * kLoadCtas * kThreads * kLoadItems;
    const int unit = kThreads * (many ? kLoadItems : 1);
    // a request has a unit even when it has no rows: its count is checked there
    const int64_t per = each > 0 ? (each + unit - 1) / unit : 1;
    const int64_t units = 2 * per * p.B;
    const unsigned grid = (unsigned)(units < INT32_MAX ? units : INT32_MAX);
    if (many)
        load_kernel<T, kLoadItems><<<grid, kThreads, 0, st>>>(p, per, a < b ? a : b);
    else
        load_kernel<T, 1><<<grid, kThreads, 0, st>>>(p, per, a < b ? a : b);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_commit_fp4(const KvFp4Params &given, cudaStream_t st) {
    if (given.B <= 0) return cudaSuccess;
    const KvFp4Params p = with_divisors(given);
    if (p.dtype == 0) return commit_type<0>(p, st);
    if (p.dtype == 1) return commit_type<1>(p, st);
    return commit_type<2>(p, st);
}

cudaError_t launch_kv_load_fp4(const KvFp4Params &given, cudaStream_t st) {
    if (given.B <= 0) return cudaSuccess;
    const KvFp4Params p = with_divisors(given);
    if (p.status) {
        const cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(int32_t) * (size_t)p.B, st);
        if (e != cudaSuccess) return e;
    }
    if (p.dtype == 0) return load_type<0>(p, st);
    if (p.dtype == 1) return load_type<1>(p, st);
    return load_type<2>(p, st);
}

}  // namespace specv
