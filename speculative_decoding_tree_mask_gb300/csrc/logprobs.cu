// Log probabilities of given tokens, entropy and the likeliest tokens of logits rows.
//
//   m = max z,  t_v = (z_v - m) log2(e) / T,  S = sum 2^t,  D = sum 2^t t,
//   log p(v) = (z_v - m) / T - ln S,   H = ln S - ln 2 D / S,
// all out of one pass over the row: the running maximum rescales S and D when it rises (D by
// 2^d (D + d S), d the step down), which per thread is rare. t is held at -200 and above, where 2^t
// is zero already: the -inf of a masked token would make 0 * -inf of its term of D.
//
// The likeliest K tokens need no second pass and no sorting of the row. Every thread keeps its own
// maximum and, for each group of vectors it reads, the group's maximum (shared memory). The K-th
// largest of the threads' maxima is a bound: K tokens at least are not below it, hardly more in all.
// (Maxima of eight threads each are sorted sooner, but let more pass: K = 32 took 278 us for 248.)
// Only groups that reach it are read again, a few KB from L2, a vector a thread and all at once (by
// the threads they belong to, one after another, 4096 rows took 291 us for 236); what passes is sorted,
// 64-bit keys of the value and the lower index, so that no arrival order changes the result. Where
// too many tokens pass (equal logits), the K-th key of those at hand is the next bound.
//
// DRAM bounds it: 4096 rows of 152064 bfloat16 logits, 8 tokens each, 229 us, 5.4 TB/s (80% of the
// measured copy), without tokens 200 us; 2048 rows of float32 216 us, 5.8 TB/s. What is left is each
// row's end, during which its CTA loads nothing: six CTAs an SM are what registers allow (four took 20 us
// more). Times that are compared here are of single replays, about 7 us above these.
// (The next row's first 8 to 64 KB brought to L2 meanwhile: no difference.) A row has a CTA, or with few
// rows a cluster of up to eight CTAs (20 rows of 50257: 11 us, 19 with a CTA each), whose parts meet in
// distributed shared memory (no workspace, no atomics on memory).

#include "spec_device.cuh"
#include "spec_internal.h"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;          // vectors of a thread in flight
constexpr int kGroups = 32;         // groups of a thread whose maxima are kept
constexpr int kCandidates = 1024;
constexpr int kHits = 512;          // groups read again together
constexpr float kFar = -200.f;
constexpr float kLn2 = 0.6931471805599453f;
// CTAs of an SM: while one orders its likeliest tokens the others have to keep the loads in flight.
constexpr int kCtas = 6;

// `bytes` (a multiple of 16) from p (16-byte aligned) on to L2.
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t order_of(float x) {     // increasing in x; -0 counts as 0
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
constexpr uint32_t kLowest = 0x007fffffu;                   // order_of(-inf)

// 32 keys of a warp, the largest in lane 0.
template <typename K>
__device__ __forceinline__ K sort_down(K v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const K o = __shfl_xor_sync(0xffffffffu, v, j);
            v = ((lane & j) == 0) == ((lane & k) == 0) ? (v > o ? v : o) : (v < o ? v : o);
        }
    return v;
}
// The 32 largest of two sorted sets, sorted.
template <typename K>
__device__ __forceinline__ K merge_down(K a, K b) {
    const int lane = threadIdx.x & 31;
    const K r = __shfl_sync(0xffffffffu, b, 31 - lane);
    K v = a > r ? a : r;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const K o = __shfl_xor_sync(0xffffffffu, v, j);
        v = (lane & j) == 0 ? (v > o ? v : o) : (v < o ? v : o);
    }
    return v;
}

struct Sums {                       // of a thread, a warp, a CTA
    float m, s, d;
    int flags;
};
__device__ __forceinline__ Sums join(const Sums &x, const Sums &y, float k) {
    Sums r;
    r.m = fmaxf(x.m, y.m);
    r.flags = x.flags | y.flags;
    r.s = r.d = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Sums &p = i ? y : x;
        if (p.m == -INFINITY) continue;
        const float t = fmaxf((p.m - r.m) * k, kFar), f = ex2(t);
        r.s = fmaf(f, p.s, r.s);
        r.d = fmaf(f, fmaf(t, p.s, p.d), r.d);
    }
    return r;
}

struct Acc {
    float m = -INFINITY, negm = 0.f;
    float2 s = {0.f, 0.f}, d = {0.f, 0.f};
    int flags = 0;

    __device__ __forceinline__ void raise(float v, float k) {
        if (m != -INFINITY) {
            const float t = fmaxf((m - v) * k, kFar), f = ex2(t);
            d = make_float2(f * fmaf(t, s.x, d.x), f * fmaf(t, s.y, d.y));
            s = make_float2(f * s.x, f * s.y);
        }
        m = v;
        negm = -v;
    }
    // two terms by their differences from m
    __device__ __forceinline__ void add(float a, float b, float k) {
        uint64_t kk, t2, e2, s2, d2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(kk) : "f"(k));
        asm("mov.b64 %0, {%1, %2};" : "=l"(t2) : "f"(a), "f"(b));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(t2) : "l"(kk));
        float t, u;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(t), "=f"(u) : "l"(t2));
        t = fmaxf(t, kFar);
        u = fmaxf(u, kFar);
        asm("mov.b64 %0, {%1, %2};" : "=l"(t2) : "f"(t), "f"(u));
        asm("mov.b64 %0, {%1, %2};" : "=l"(e2) : "f"(ex2(t)), "f"(ex2(u)));
        asm("mov.b64 %0, {%1, %2};" : "=l"(s2) : "f"(s.x), "f"(s.y));
        asm("mov.b64 %0, {%1, %2};" : "=l"(d2) : "f"(d.x), "f"(d.y));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s2) : "l"(e2));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d2) : "l"(e2), "l"(t2));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(s.x), "=f"(s.y) : "l"(s2));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(d2));
    }
    __device__ __forceinline__ void scalar(float x, float k) {
        if (x != x) {
            flags |= SPEC_ROW_NAN;
            return;
        }
        if (x > m) raise(x, k);
        const float t = fmaxf((x + negm) * k, kFar), e = ex2(t);
        s.x += e;
        d.x = fmaf(e, t, d.x);
    }
};

// A vector's elements into the sums; returns its largest (NaN if one is).
template <int DT>
__device__ __forceinline__ float take(Acc &a, const uint4 w, float k) {
    float big;
    if constexpr (DT == 1) {
        const uint32_t mm = bmax2_nan(bmax2_nan(w.x, w.y), bmax2_nan(w.z, w.w));
        big = fmax_nan(bf_lo(mm), bf_hi(mm));
    } else {
        big = fmax_nan(fmax_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                       fmax_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    if (!(big <= a.m)) {
        if (big != big)
            a.flags |= SPEC_ROW_NAN;
        else
            a.raise(big, k);
    }
    if constexpr (DT == 1) {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float x, y;
            bf_add2(ws[q], a.negm, x, y);
            a.add(x, y, k);
        }
    } else {
        a.add(__uint_as_float(w.x) + a.negm, __uint_as_float(w.y) + a.negm, k);
        a.add(__uint_as_float(w.z) + a.negm, __uint_as_float(w.w) + a.negm, k);
    }
    return big;
}

struct Shared {
    Sums part[kWarps];
    Sums sums;                                // of the CTA
    uint32_t maxima[kWarps][32];
    unsigned long long best[32];              // the CTA's likeliest, sorted; 0: none
    unsigned long long bound;
    int count, hits;
    unsigned short hit[kHits];                // a thread's group: group << 8 | thread
    unsigned long long key[kCandidates];
};

// DT: 0 f32, 1 bf16; TOP: the likeliest tokens are wanted.
template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(LogprobsParams P, int cluster) {
    constexpr int kEsz = DT == 1 ? 2 : 4, E = 16 / kEsz;
    __shared__ Shared S;
    extern __shared__ float group_max[];      // [groups][kThreads]
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster > 1 ? cluster_rank() : 0;
    const int64_t slot = blockIdx.x / (unsigned)cluster;
    const int b = (int)(slot / P.P);
    const int node = P.node ? __ldg(P.node + slot) : (int)(slot - (int64_t)b * P.P);
    const bool good = node >= 0 && node < P.N;
    if (!good) {       // nothing to score, or a row that is not there
        if (rank != 0) return;
        const bool none = node == -1;
        const float x = none ? 0.f : NAN;
        for (int c = tid; c < P.C; c += kThreads) P.logprob[slot * P.C + c] = x;
        for (int c = tid; c < P.top; c += kThreads) {
            P.top_ids[slot * P.top + c] = -1;
            P.top_logprobs[slot * P.top + c] = none ? -INFINITY : NAN;
        }
        if (tid == 0) {
            if (P.entropy) P.entropy[slot] = x;
            if (P.flags) P.flags[slot] = none ? 0 : SPEC_ROW_BAD_NODE;
        }
        return;
    }
    const int64_t V = P.V;
    const float k = P.k;
    const char *row = reinterpret_cast<const char *>(P.logits) +
                      ((int64_t)b * P.N + node) * V * kEsz;
    // a scalar head up to 16-byte alignment, vectors, a scalar tail
    int head = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kEsz;
    if (head > V) head = (int)V;
    const int nv = (int)((V - head) / E), tail = head + nv * E;
    const uint4 *vec = reinterpret_cast<const uint4 *>(row + head * kEsz);
    const int v0 = (int)((int64_t)nv * rank / cluster), v1 = (int)((int64_t)nv * (rank + 1) / cluster);
    // the CTA's rounds of kUnroll vectors a thread, `per` of them a group
    const int rounds = (v1 - v0 + kUnroll * kThreads - 1) / (kUnroll * kThreads);
    const int per = (rounds + kGroups - 1) / kGroups;
    Acc a;
    // the first CTA's first threads have the head's element, then the tail's
    const int at = rank != 0 ? -1 : tid < head ? tid : tid - head < V - tail ? tail + tid - head : -1;
    float lone = -INFINITY;
    if (at >= 0) {
        lone = load_elem<DT>(row, at);
        a.scalar(lone, k);
    }
    {
        const uint32_t none = DT == 1 ? 0xff80ff80u : 0xff800000u;    // -inf
        float big = -INFINITY;
        int left = per;
        float *to = group_max + tid;
        for (int i = v0 + tid; i - tid < v1; i += kUnroll * kThreads) {
            // float32: the next round to L2 meanwhile (2048 rows of 152064, 8 tokens: 247 us -> 224;
            // bfloat16, twice the instructions a byte, loses by it: 4096 rows 234 -> 240; so do rows
            // of several CTAs, with few rounds each: 192 of 50257 19 -> 21)
            if (DT == 0 && cluster == 1 && tid == 0) {
                const int next = i + kUnroll * kThreads;
                if (next < v1) prefetch_l2(vec + next, min(kUnroll * kThreads, v1 - next) * 16);
            }
            uint4 w[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                w[u] = i + u * kThreads < v1 ? ldg_stream(vec + i + u * kThreads)
                                             : make_uint4(none, none, none, none);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) big = fmaxf(big, take<DT>(a, w[u], k));
            if (TOP && --left == 0) {
                *to = big;
                to += kThreads;
                left = per;
                big = -INFINITY;
            }
        }
        if (TOP && left != per) *to = big;
    }

    Sums p{a.m, a.s.x + a.s.y, a.d.x + a.d.y, a.flags};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sums q;
        q.m = shfl_xor(p.m, o);
        q.s = shfl_xor(p.s, o);
        q.d = shfl_xor(p.d, o);
        q.flags = shfl_xor(p.flags, o);
        p = join(p, q, k);
    }
    if (lane == 0) S.part[warp] = p;
    if (TOP) {
        S.maxima[warp][lane] = sort_down(order_of(a.m));
        if (tid == 0) S.count = S.hits = 0;
    }
    __syncthreads();
    if (warp == 0) {
        p = lane < kWarps ? S.part[lane] : Sums{-INFINITY, 0.f, 0.f, 0};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            Sums q;
            q.m = shfl_xor(p.m, o);
            q.s = shfl_xor(p.s, o);
            q.d = shfl_xor(p.d, o);
            q.flags = shfl_xor(p.flags, o);
            p = join(p, q, k);
        }
        if (lane == 0) S.sums = p;
        if (TOP) {
            uint32_t v = S.maxima[0][lane];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v = merge_down(v, S.maxima[w][lane]);
            v = __shfl_sync(0xffffffffu, v, P.top - 1);
            if (lane == 0) S.bound = (unsigned long long)v << 32;
        }
    }
    __syncthreads();
    if (TOP && S.sums.flags == 0) {
        for (;;) {
            const unsigned long long bound = S.bound;
            const uint32_t low = (uint32_t)(bound >> 32);
            auto offer = [&](float x, int index) {
                const uint32_t o = order_of(x);
                const unsigned long long key = (unsigned long long)o << 32 | (uint32_t)~index;
                if (o > kLowest && key >= bound) {
                    const int n = atomicAdd(&S.count, 1);
                    if (n < kCandidates) S.key[n] = key;
                }
            };
            auto offer_vector = [&](int i) {
                const uint4 w = __ldg(vec + i);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                const int e0 = head + i * E;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (DT == 1) {
                        offer(bf_lo(ws[q]), e0 + 2 * q);
                        offer(bf_hi(ws[q]), e0 + 2 * q + 1);
                    } else {
                        offer(__uint_as_float(ws[q]), e0 + q);
                    }
                }
            };
            const int of_group = per * kUnroll;      // vectors of a group
            if (order_of(a.m) >= low) {
                if (at >= 0) offer(lone, at);
                const int groups = (rounds + per - 1) / max(per, 1);
                for (int g = 0; g < groups; ++g) {
                    if (order_of(group_max[g * kThreads + tid]) < low) continue;
                    const int k = atomicAdd(&S.hits, 1);
                    if (k < kHits) {
                        S.hit[k] = (unsigned short)(g << 8 | tid);
                        continue;
                    }
                    for (int n = g * of_group; n < (g + 1) * of_group; ++n)
                        if (v0 + n * kThreads + tid < v1) offer_vector(v0 + n * kThreads + tid);
                }
            }
            __syncthreads();
            // a vector a thread: all that are read again are under way at once
            const int hits = min(S.hits, kHits) * of_group;
            for (int k = tid; k < hits; k += kThreads) {
                const int hit = S.hit[k / of_group], n = (hit >> 8) * of_group + k % of_group;
                const int i = v0 + n * kThreads + (hit & (kThreads - 1));
                if (i < v1) offer_vector(i);
            }
            __syncthreads();
            const int count = S.count;
            __syncthreads();      // all have it: it can begin again
            if (warp == 0) {
                const int n = min(count, kCandidates);
                unsigned long long v = 0ull;
                for (int i = 0; i < n; i += 32)
                    v = merge_down(v, sort_down(i + lane < n ? S.key[i + lane] : 0ull));
                S.best[lane] = v;
                if (lane == P.top - 1) S.bound = v;
                if (lane == 0) S.count = S.hits = 0;
            }
            __syncthreads();
            // more than fit: those at or above the K-th of the ones at hand are fewer
            if (count <= kCandidates) break;
        }
    }
    if (cluster > 1) cluster_sync();
    if (rank == 0 && warp == 0) {
        Sums all = S.sums;
        unsigned long long best = TOP ? S.best[lane] : 0ull;
        for (int r = 1; r < cluster; ++r) {
            const uint32_t from = cluster_addr(&S.sums, r);
            Sums q;
            q.m = ld_cluster_f32(from);
            q.s = ld_cluster_f32(from + 4);
            q.d = ld_cluster_f32(from + 8);
            q.flags = ld_cluster_s32(from + 12);
            all = join(all, q, k);
            if (TOP) {
                const uint32_t at32 = cluster_addr(&S.best[lane], r);
                const unsigned long long o = (uint32_t)ld_cluster_s32(at32) |
                                             (unsigned long long)(uint32_t)ld_cluster_s32(at32 + 4)
                                                 << 32;
                best = merge_down(best, o);
            }
        }
        int flags = all.flags;
        if (all.m == INFINITY) flags |= SPEC_ROW_POSINF;
        if (all.m == -INFINITY && !(flags & SPEC_ROW_NAN)) flags |= SPEC_ROW_ALL_NEGINF;
        const float log_s = logf(all.s);
        for (int c = lane; c < P.C; c += 32) {
            const int t = __ldg(P.tokens + slot * P.C + c);
            float lp = 0.f;
            if (flags) {
                lp = NAN;
            } else if (t >= 0 && t < V) {
                lp = (load_elem<DT>(row, t) - all.m) * P.inv_t - log_s;
            }
            if (t < -1 || t >= V) {
                lp = NAN;
                if (P.flags) atomicOr(&S.part[0].flags, SPEC_ROW_BAD_TOKEN);
            } else if (t == -1) {
                lp = 0.f;
            }
            P.logprob[slot * P.C + c] = lp;
        }
        if (TOP && lane < P.top) {
            const bool is = flags == 0 && best != 0ull;
            P.top_ids[slot * P.top + lane] = is ? (int)~(uint32_t)best : -1;
            P.top_logprobs[slot * P.top + lane] =
                flags ? NAN
                      : is ? (value_of((uint32_t)(best >> 32)) - all.m) * P.inv_t - log_s : -INFINITY;
        }
        __syncwarp();
        if (lane == 0) {
            if (P.entropy) P.entropy[slot] = flags ? NAN : log_s - kLn2 * all.d / all.s;
            if (P.flags) P.flags[slot] = flags | (S.part[0].flags & SPEC_ROW_BAD_TOKEN);
        }
    }
    if (cluster > 1) cluster_sync();      // the others' sums have been read
}

template <int DT, bool TOP>
cudaError_t launch(const LogprobsParams &p, cudaStream_t st) {
    const int64_t slots = (int64_t)p.B * p.P;
    // few rows: as many CTAs a row, up to eight, as one wave holds
    int cluster = 1;
    for (int c = 8; c > 1; c /= 2)
        if (slots * c <= (int64_t)p.sms * kCtas) {
            cluster = c;
            break;
        }
    constexpr int E = DT == 1 ? 8 : 4;
    const int64_t rounds = (p.V / E / cluster + 1 + kUnroll * kThreads - 1) / (kUnroll * kThreads);
    const size_t smem = TOP ? (size_t)(rounds < kGroups ? rounds : kGroups) * kThreads * sizeof(float)
                            : 0;
    const dim3 grid((unsigned)(slots * cluster));
    if (cluster > 1)
        return launch_dependent_cluster(logprobs_kernel<DT, TOP>, grid, dim3(kThreads), smem, st,
                                        cluster, p, cluster);
    return launch_dependent(logprobs_kernel<DT, TOP>, grid, dim3(kThreads), smem, st, p, 1);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams &p, int dtype, cudaStream_t st) {
    if ((int64_t)p.B * p.P <= 0) return cudaSuccess;
    if (dtype == SPEC_BF16)
        return p.top > 0 ? launch<1, true>(p, st) : launch<1, false>(p, st);
    return p.top > 0 ? launch<0, true>(p, st) : launch<0, false>(p, st);
}

}  // namespace specv
