// Paged attention: how a call is run, and the joining of items that were cut.
#include "paged_attn.cuh"

namespace specv {
namespace {

// The most rows of the kernel for few. With 24 rows (chains of six, 32 and 8 heads x 128) it takes 259 us
// for 64 chains over up to 8192 positions where the tensor cores take 255, but 246 against 306 over an
// 8-bit cache, 39 against 54 for 16 chains over 1000, and with 32 rows at D = 64 164 against 212. Beside a
// launch on the tensor cores 16, one token of up to 16 heads a group: a mixed batch (below) took 6 us more
// with 32.
int few_rows(int D) { return paged_padded(D) == 256 ? 16 : 32; }
int few_beside(int G, int D) { return G <= 16 ? 16 : few_rows(D); }

// The parts of cut items into the result. A thread has a float4 of a row and, of the parts,
// every PG-th, eight of them in flight together; the PG threads of a float4 meet in shared
// memory. PG is 1 for items of few parts and many rows.
constexpr int kJoinThreads = 256;
template <int T, int DP, int PG>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(PagedAttnParams P, int rows_tile) {
    constexpr int F = DP / 4, kPer = kJoinThreads / (F * PG);       // rows of a CTA
    __shared__ float4 s_o[PG > 1 ? kJoinThreads : 1];
    __shared__ float2 s_ml[PG > 1 ? kJoinThreads : 1];
    grid_dep_wait();
    const int c0 = blockIdx.y;
    const int4 note = P.notes[c0];
    if (note.x < 0) return;
    const int c1 = note.w & ((1 << kNoteCtas) - 1), rows = note.z;
    const int d4 = threadIdx.x % F, group = threadIdx.x / F % PG;
    const int first = blockIdx.x * kPer + threadIdx.x / (F * PG);
    // PG 1: more rows than the CTA holds, one after another, two under way
#pragma unroll 2
    for (int r = first; r < (PG == 1 ? rows : first + 1); r += gridDim.x * kPer) {
        float m = kPagedNoMax, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0 + group; c <= c1 && r < rows; c += 8 * PG) {
            float4 v[8];
            float pm[8], pl[8], top = m;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                pm[u] = kPagedNoMax;
                const int k = c + u * PG;
                if (k > c1) continue;
                const float *part = paged_slot(P, k, k == c0, rows_tile, DP);
                v[u] = __ldcg(reinterpret_cast<const float4 *>(part + r * DP) + d4);
                pm[u] = __ldcg(part + rows_tile * DP + r);
                pl[u] = __ldcg(part + rows_tile * (DP + 1) + r);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) top = fmaxf(top, pm[u]);
            const float a = ex2(m - top);
            m = top;
            l *= a;
            o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (c + u * PG > c1) continue;
                const float w = ex2(pm[u] - top);
                o.x = fmaf(v[u].x, w, o.x);
                o.y = fmaf(v[u].y, w, o.y);
                o.z = fmaf(v[u].z, w, o.z);
                o.w = fmaf(v[u].w, w, o.w);
                l = fmaf(pl[u], w, l);
            }
        }
        if (PG > 1) {
            s_o[threadIdx.x] = o;
            s_ml[threadIdx.x] = make_float2(m, l);
            __syncthreads();
            if (group != 0 || r >= rows) return;
            float top = m;
#pragma unroll
            for (int u = 1; u < PG; ++u) top = fmaxf(top, s_ml[threadIdx.x + u * F].x);
            const float a = ex2(m - top);
            o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
            l *= a;
            m = top;
#pragma unroll
            for (int u = 1; u < PG; ++u) {
                const float2 ml = s_ml[threadIdx.x + u * F];
                const float4 v = s_o[threadIdx.x + u * F];
                const float w = ex2(ml.x - top);
                o.x = fmaf(v.x, w, o.x);
                o.y = fmaf(v.y, w, o.y);
                o.z = fmaf(v.z, w, o.z);
                o.w = fmaf(v.w, w, o.w);
                l = fmaf(ml.y, w, l);
            }
        }
        const float f = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = paged_row(P, note.x, note.w >> kNoteCtas, note.y + r);
        if (d4 * 4 < P.cache.D)
            paged_store4<T>(P.out, at * P.cache.D + d4 * 4,
                            make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
        if (P.lse && d4 == 0) P.lse[at] = paged_lse(m, l);
    }
}

// How requests are run: by the warps' matrix unit up to 32 rows an item (16 where D is above 128: its
// registers hold no more), beyond on the tcgen05 tensor cores.
struct Plan {
    int mt, rows, grid;     // groups of 16 rows of an item, 0: tcgen05; rows; CTAs
};
Plan plan(int64_t R, int D, int kind, int sms) {      // R: most rows a head
    Plan p;
    const int DP = paged_padded(D);
    p.mt = R > few_rows(D) ? 0 : R > 16 ? 2 : 1;
    p.rows = p.mt ? 16 * p.mt : paged_tc_rows(DP);
    p.grid = sms * (p.mt ? paged_few_ctas(kind != SPEC_CACHE_SAME, DP) : 1);
    return p;
}

template <int T, int DP>
cudaError_t launch_join(const PagedAttnParams &p, const Plan &n, cudaStream_t st) {
    constexpr int F = DP / 4, PG = DP == 256 ? 4 : 8;
    const int64_t R = (int64_t)p.max_new * p.G < p.rows_most ? (int64_t)p.max_new * p.G : p.rows_most;
    const int rows = (int)(R < n.rows ? R : n.rows), per = kJoinThreads / F;
    const int64_t items = (int64_t)p.B * p.cache.H;
    if (n.grid > 8 * items && rows <= 32)
        return launch_dependent(paged_join_kernel<T, DP, PG>,
                                dim3((rows * PG + per - 1) / per, n.grid), dim3(kJoinThreads), 0, st,
                                p, n.rows);
    // (one wave of CTAs that have eight SM's worth of them at most)
    const int wide = (rows + per - 1) / per, most = 8 * p.sms / n.grid > 1 ? 8 * p.sms / n.grid : 1;
    return launch_dependent(paged_join_kernel<T, DP, 1>, dim3(wide < most ? wide : most, n.grid),
                            dim3(kJoinThreads), 0, st, p, n.rows);
}

int64_t notes_bytes(const Plan &n) { return ((int64_t)n.grid * sizeof(int4) + 255) / 256 * 256; }
int64_t plan_bytes(const Plan &n, int D) {
    const int64_t bytes = (int64_t)n.grid * 2 * n.rows * (paged_padded(D) + 2) * (int64_t)sizeof(float);
    return notes_bytes(n) + (bytes + 255) / 256 * 256;
}

// One launch and its joining, over requests of more than rows_over and at most rows_most rows.
cudaError_t run(PagedAttnParams p, const Plan &n, int rows_over, int rows_most, cudaStream_t st) {
    const int DP = paged_padded(p.cache.D);
    p.rows_over = rows_over;
    p.rows_most = rows_most;
    p.notes = static_cast<int4 *>(p.workspace);
    p.ws = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + notes_bytes(n));
    const bool bf16 = p.dtype == SPEC_BF16;
    const cudaError_t e = n.mt == 0 ? bf16 ? launch_paged_tc_bf16(p, n.grid, st)
                                           : launch_paged_tc_f16(p, n.grid, st)
                          : bf16 ? launch_paged_few_bf16(p, n.mt, n.grid, st)
                                 : launch_paged_few_f16(p, n.mt, n.grid, st);
    if (e != cudaSuccess) return e;
    if (bf16)
        return DP == 64    ? launch_join<1, 64>(p, n, st)
               : DP == 128 ? launch_join<1, 128>(p, n, st)
                           : launch_join<1, 256>(p, n, st);
    return DP == 64    ? launch_join<2, 64>(p, n, st)
           : DP == 128 ? launch_join<2, 128>(p, n, st)
                       : launch_join<2, 256>(p, n, st);
}

}  // namespace

// A batch may hold requests of few rows and of many; which, the device knows alone. Where it may
// hold both, both kernels are launched and take their own: 22 decoding requests over up to 12000
// positions beside a chunk of 512 tokens (D = 64, 8 K/V heads) take 170 us, 37 less than when the tensor
// cores had a tile of 256 rows for four.
int64_t paged_attn_workspace(int max_new, int G, int D, int sms) {
    const int64_t R = (int64_t)max_new * G;
    int64_t most = 256;       // whatever the cache's type and the batch
    for (int kind = 0; kind < 2; ++kind) {
        int64_t bytes = plan_bytes(plan(R, D, kind, sms), D);
        if (R > few_rows(D)) bytes += plan_bytes(plan(few_beside(G, D), D, kind, sms), D);
        most = bytes > most ? bytes : most;
    }
    return most;
}

cudaError_t launch_paged_attn(const PagedAttnParams &given, cudaStream_t st) {
    if (given.B <= 0 || given.T <= 0) return cudaSuccess;
    PagedAttnParams p = given;
    const int64_t R = (int64_t)p.max_new * p.G;
    const Plan n = plan(R, p.cache.D, p.cache.kind, p.sms);
    const int few = few_beside(p.G, p.cache.D);
    // the fewest rows that a request may have, the others having the most
    const int64_t least = p.T - (int64_t)(p.B - 1) * p.max_new;
    const bool both = n.mt == 0 && least * p.G <= few;
    const cudaError_t e = run(p, n, both ? few : 0, INT32_MAX, st);
    if (!both || e != cudaSuccess) return e;
    p.workspace = static_cast<char *>(p.workspace) + plan_bytes(n, p.cache.D);
    return run(p, plan(few, p.cache.D, p.cache.kind, p.sms), 0, few, st);
}

}  // namespace specv
