// C ABI of the verification library (declared in include/spec_verify.h): handle and
// workspace, host-side argument checks, kernel orchestration and per-kernel timing.

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "spec_internal.h"
#include "spec_verify.h"

// Built with SPEC_NVTX, every entry point of the ABI is an NVTX range named after it, so a
// timeline profiler shows the host side of each call around its kernels. Otherwise the
// ranges compile to nothing.
#ifdef SPEC_NVTX
#include <nvtx3/nvToolsExt.h>
namespace {
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};
}  // namespace
#define SPEC_RANGE(name) NvtxRange spec_range_(name)
#else
#define SPEC_RANGE(name) ((void)0)
#endif

using namespace specv;

namespace {

constexpr int kMaxRecords = 16384;
constexpr int64_t kMaxV = int64_t(1) << 21;
constexpr float kLog2eF = 1.4426950408889634f;

}  // namespace

struct spec_ctx {
    int device = 0;
    int max_B = 0, max_N = 0;
    int64_t max_V = 0;
    void *ws = nullptr;
    float *m = nullptr, *s = nullptr, *pc = nullptr, *mq = nullptr, *sq = nullptr,
          *qc = nullptr;
    int32_t *arg = nullptr, *flags = nullptr, *dflags = nullptr;
    float2 *chunk = nullptr;              // row-chunk partials of the target rows
    RowPart *piece = nullptr;             // small batches: per-piece row statistics
    int32_t *count = nullptr;             // ... and per-row arrivals (zero between calls)
    int32_t *dbg = nullptr;               // debug builds: violation bits per request [max_B]
    int inject_row = -1, inject_value = 0;   // debug builds: one armed counter injection
    int inject_lost = 0;                  // ... and one armed loss of an attention's waits
    int slots = 0;                        // CTAs of the split row-statistics kernel in a wave
    int sms = 0;                          // streaming multiprocessors of the device
    const int32_t *n_active = nullptr;   // node budget set by spec_set_node_budget
    bool prof = false;
    bool ev_ready = false;
    int nrec = 0;
    cudaEvent_t ev[2 * kMaxRecords];
    int cls[kMaxRecords];
};

namespace {

// Makes the handle's device current for the duration of a call and restores the caller's.
class DeviceScope {
  public:
    explicit DeviceScope(int dev) {
        ok_ = cudaGetDevice(&prev_) == cudaSuccess;
        if (ok_ && prev_ != dev) ok_ = cudaSetDevice(dev) == cudaSuccess;
        switched_ = ok_ && prev_ != dev;
    }
    ~DeviceScope() {
        if (switched_) cudaSetDevice(prev_);
    }
    bool ok() const { return ok_; }

  private:
    int prev_ = 0;
    bool ok_ = false, switched_ = false;
};

template <typename F>
int timed(spec_handle h, int cls, cudaStream_t st, F &&launch) {
    int slot = -1;
    if (h->prof && h->nrec < kMaxRecords) {
        slot = h->nrec++;
        h->cls[slot] = cls;
        cudaEventRecord(h->ev[2 * slot], st);
    }
    const cudaError_t e = launch();
    if (slot >= 0) cudaEventRecord(h->ev[2 * slot + 1], st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t esize(int dtype) { return dtype == SPEC_BF16 ? 2 : 4; }

// Lazy calls read logits where they live: memory of the handle's device, or page-locked
// host memory that the device reaches at the same address (read over the host link).
// Anything else (another GPU's memory, pageable host memory, a registration mapped at
// another address) is refused.
// Whether p is host memory the device can read (pinned and mapped).
bool host_memory(const void *p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeHost;
}

bool readable_by_device(const void *p, int device) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (a.type == cudaMemoryTypeDevice) return a.device == device;
    if (a.type == cudaMemoryTypeManaged) return true;
    return a.type == cudaMemoryTypeHost && a.devicePointer == p;
}

int check_common(spec_handle h, const void *logits, int dtype, int B, int N, int64_t V,
                 const int32_t *tok, const int32_t *parent, const int32_t *accept_len,
                 const int32_t *out_tokens, const int32_t *kv_commit, const int32_t *bonus,
                 const int32_t *status) {
    if (!h) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B) return SPEC_ERR_ARG;
    if (N < 1 || N > h->max_N || N > kMaxN) return SPEC_ERR_ARG;
    if (V < 1 || V > h->max_V) return SPEC_ERR_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (!logits || !tok || !parent || !accept_len || !out_tokens || !kv_commit || !bonus ||
        !status)
        return SPEC_ERR_ARG;
    if (!aligned(logits, esize(dtype))) return SPEC_ERR_ARG;
    const void *ints[] = {tok, parent, accept_len, out_tokens, kv_commit, bonus, status};
    for (const void *p : ints)
        if (!aligned(p, 4)) return SPEC_ERR_ARG;
    return SPEC_OK;
}

// Small batches: split every row over the most CTAs (8, 4 or 2) that still fit in one wave,
// so that the row-statistics kernel keeps every SM streaming. Only for row counts the
// workspace's per-piece arrays can hold.
void set_split(spec_handle h, RowStatsParams &rp) {
    rp.split = 1;
    if ((int64_t)rp.rows > (int64_t)h->max_B * h->max_N) return;
    rp.piece = h->piece;
    rp.count = h->count;
    for (int s = kRowChunks; s > 1; s /= 2)
        if ((int64_t)rp.rows * s <= h->slots) {
            rp.split = s;
            break;
        }
}

// Dense drafts, few requests: run each request's walk on a cluster of the most CTAs (8, 4 or
// 2) that still fit one wave of the walk kernel (one CTA per SM), so that its full-row passes
// over the target and draft rows are spread over that many SMs. Point drafts keep one CTA.
int walk_cluster(spec_handle h, int B, bool point) {
    if (point) return 1;
    const int64_t wave = h->sms;
    for (int c = 8; c > 1; c /= 2)
        if ((int64_t)B * c <= wave) return c;
    return 1;
}

// Debug builds, before a verify call's kernels: zero the request's violation words and every
// split-row arrival counter (so a counter an earlier call left wrong cannot spill over), then
// apply an injection armed by spec_debug_inject_arrival. Release builds do nothing.
int debug_prologue(spec_handle h, int B, int rows, cudaStream_t st) {
#ifdef SPEC_DEBUG
    const int64_t cap = (int64_t)h->max_B * h->max_N;
    if (cudaMemsetAsync(h->dbg, 0, sizeof(int32_t) * (size_t)B, st) != cudaSuccess ||
        cudaMemsetAsync(h->count, 0, sizeof(int32_t) * (size_t)cap, st) != cudaSuccess)
        return SPEC_ERR_CUDA;
    if (h->inject_row >= 0 && h->inject_row < rows && h->inject_row < cap) {
        if (cudaMemcpyAsync(h->count + h->inject_row, &h->inject_value, sizeof(int32_t),
                            cudaMemcpyHostToDevice, st) != cudaSuccess)
            return SPEC_ERR_CUDA;
        if (cudaStreamSynchronize(st) != cudaSuccess) return SPEC_ERR_CUDA;
        h->inject_row = -1;
    }
#else
    (void)h;
    (void)B;
    (void)rows;
    (void)st;
#endif
    return SPEC_OK;
}

WalkOutputs outputs(int32_t *accept_len, int32_t *out_tokens, int32_t *kv_commit,
                    int32_t *bonus, int32_t *status) {
    WalkOutputs o;
    o.accept_len = accept_len;
    o.out_tokens = out_tokens;
    o.kv_commit = kv_commit;
    o.bonus = bonus;
    o.status = status;
    return o;
}

int greedy_impl(spec_handle h, const void *logits, int dtype, int B, int N, int64_t V,
                const int32_t *tok, const int32_t *parent, WalkOutputs out, cudaStream_t st) {
    const int drc = debug_prologue(h, B, B * N, st);
    if (drc != SPEC_OK) return drc;
    RowStatsParams rp{};
    rp.x = logits;
    rp.V = V;
    rp.rows = B * N;
    rp.N = N;
    rp.k = 0.f;
    rp.m = h->m;
    rp.s = nullptr;
    rp.arg = h->arg;
    rp.flags = h->flags;
    rp.n_active = h->n_active;
    rp.dbg = h->dbg;
    set_split(h, rp);
    int rc = timed(h, SPEC_K_ROW_STATS, st,
                   [&] { return launch_row_stats(rp, dtype, ROW_GREEDY, st); });
    if (rc != SPEC_OK) return rc;
    GreedyWalkParams gp;
    gp.B = B;
    gp.N = N;
    gp.V = V;
    gp.parent = parent;
    gp.tok = tok;
    gp.arg = h->arg;
    gp.flags = h->flags;
    gp.out = out;
    gp.n_active = h->n_active;
    gp.dbg = h->dbg;
    return timed(h, SPEC_K_WALK_GREEDY, st, [&] { return launch_walk_greedy(gp, st); });
}

}  // namespace

extern "C" {

const char *spec_error_string(int code) {
    switch (code) {
        case SPEC_OK: return "ok";
        case SPEC_ERR_ARG: return "invalid argument or outside the handle's limits";
        case SPEC_ERR_UNSUPPORTED: return "unsupported request";
        case SPEC_ERR_CUDA: return "CUDA call or kernel launch failed";
        case SPEC_ERR_WORKSPACE: return "workspace allocation failed";
        default: return "unknown error code";
    }
}

int spec_verify_init(spec_handle *out, int max_B, int max_N, int64_t max_V, int device) {
    SPEC_RANGE("spec_verify_init");
    if (!out) return SPEC_ERR_ARG;
    *out = nullptr;
    if (max_B < 1 || max_N < 1 || max_V < 1) return SPEC_ERR_ARG;
    if (max_N > kMaxN || max_V > kMaxV) return SPEC_ERR_UNSUPPORTED;
    if ((int64_t)max_B * max_N > (int64_t(1) << 30)) return SPEC_ERR_ARG;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev)
        return SPEC_ERR_CUDA;
    DeviceScope ds(device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    spec_ctx *h = new (std::nothrow) spec_ctx();
    if (!h) return SPEC_ERR_WORKSPACE;
    h->device = device;
    h->max_B = max_B;
    h->max_N = max_N;
    h->max_V = max_V;
    const size_t rows = (size_t)max_B * max_N;
    const size_t bytes =
        rows * (9 * 4 + kRowChunks * sizeof(float2) + kRowChunks * sizeof(RowPart) + 4) +
        sizeof(int32_t) * (size_t)max_B;
    if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return SPEC_ERR_WORKSPACE;
    }
    char *p = static_cast<char *>(h->ws);   // cudaMalloc: 256-byte aligned
    auto take = [&](size_t n) {
        char *q = p;
        p += n;
        return q;
    };
    h->chunk = reinterpret_cast<float2 *>(take(rows * kRowChunks * sizeof(float2)));
    h->piece = reinterpret_cast<RowPart *>(take(rows * kRowChunks * sizeof(RowPart)));
    h->m = reinterpret_cast<float *>(take(rows * 4));
    h->s = reinterpret_cast<float *>(take(rows * 4));
    h->pc = reinterpret_cast<float *>(take(rows * 4));
    h->mq = reinterpret_cast<float *>(take(rows * 4));
    h->sq = reinterpret_cast<float *>(take(rows * 4));
    h->qc = reinterpret_cast<float *>(take(rows * 4));
    h->arg = reinterpret_cast<int32_t *>(take(rows * 4));
    h->flags = reinterpret_cast<int32_t *>(take(rows * 4));
    h->dflags = reinterpret_cast<int32_t *>(take(rows * 4));
    h->count = reinterpret_cast<int32_t *>(take(rows * 4));
    h->dbg = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * (size_t)max_B));
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        cudaMemset(h->count, 0, rows * 4) != cudaSuccess ||
        cudaMemset(h->dbg, 0, sizeof(int32_t) * (size_t)max_B) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(h->ws);
        delete h;
        return SPEC_ERR_CUDA;
    }
    h->slots = kSplitCtasPerSm * sms;   // one wave of the split row-statistics kernel
    h->sms = sms;
    *out = h;
    return SPEC_OK;
}

int spec_verify_destroy(spec_handle h) {
    SPEC_RANGE("spec_verify_destroy");
    if (!h) return SPEC_OK;
    DeviceScope ds(h->device);
    if (h->ev_ready)
        for (int i = 0; i < 2 * kMaxRecords; ++i) cudaEventDestroy(h->ev[i]);
    cudaFree(h->ws);
    delete h;
    return SPEC_OK;
}

int spec_build_tree_mask(spec_handle h, const int32_t *parent, int B, int N, uint64_t *anc_mask,
                         int32_t *depth, int32_t *status, void *stream) {
    SPEC_RANGE("spec_build_tree_mask");
    if (!h) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B || N < 1 || N > h->max_N || N > kMaxN) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (!parent || !anc_mask || !depth || !status) return SPEC_ERR_ARG;
    if (!aligned(parent, 4) || !aligned(anc_mask, 8) || !aligned(depth, 4) || !aligned(status, 4))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return timed(h, SPEC_K_TREE_MASK, st, [&] {
        return launch_tree_mask(parent, B, N, anc_mask, depth, status, st);
    });
}

int spec_verify_greedy(spec_handle h, const void *logits, int dtype, int B, int N, int64_t V,
                       const int32_t *draft_token, const int32_t *parent, int32_t *accept_len,
                       int32_t *out_tokens, int32_t *kv_commit, int32_t *bonus, int32_t *status,
                       void *stream) {
    SPEC_RANGE("spec_verify_greedy");
    int rc = check_common(h, logits, dtype, B, N, V, draft_token, parent, accept_len,
                          out_tokens, kv_commit, bonus, status);
    if (rc != SPEC_OK || B == 0) return rc;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    return greedy_impl(h, logits, dtype, B, N, V, draft_token, parent,
                       outputs(accept_len, out_tokens, kv_commit, bonus, status),
                       static_cast<cudaStream_t>(stream));
}

int spec_verify_sample(spec_handle h, const void *logits, int dtype, int B, int N, int64_t V,
                       const int32_t *draft_token, const int32_t *parent, const void *draft,
                       int draft_kind, int draft_dtype, float temperature,
                       const float *uniforms, int32_t *accept_len, int32_t *out_tokens,
                       int32_t *kv_commit, int32_t *bonus, int32_t *status, void *stream) {
    SPEC_RANGE("spec_verify_sample");
    int rc = check_common(h, logits, dtype, B, N, V, draft_token, parent, accept_len,
                          out_tokens, kv_commit, bonus, status);
    if (rc != SPEC_OK) return rc;
    if (!(temperature >= 0.f) || std::isinf(temperature)) return SPEC_ERR_ARG;
    const float k = temperature > 0.f ? kLog2eF / temperature : 0.f;
    if (temperature > 0.f && !std::isfinite(k)) return SPEC_ERR_ARG;
    if (draft_kind != SPEC_DRAFT_POINT && draft_kind != SPEC_DRAFT_PROBS_F32 &&
        draft_kind != SPEC_DRAFT_LOGITS)
        return SPEC_ERR_ARG;
    if (draft_kind == SPEC_DRAFT_LOGITS && draft_dtype != SPEC_F32 && draft_dtype != SPEC_BF16)
        return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    WalkOutputs out = outputs(accept_len, out_tokens, kv_commit, bonus, status);
    if (temperature == 0.f)
        return greedy_impl(h, logits, dtype, B, N, V, draft_token, parent, out, st);
    if (!uniforms || !aligned(uniforms, 4)) return SPEC_ERR_ARG;
    const bool dense = draft_kind != SPEC_DRAFT_POINT;
    if (dense) {
        if (!draft) return SPEC_ERR_ARG;
        const size_t de = draft_kind == SPEC_DRAFT_LOGITS ? esize(draft_dtype) : 4;
        if (!aligned(draft, de)) return SPEC_ERR_ARG;
    }
    rc = debug_prologue(h, B, B * N, st);
    if (rc != SPEC_OK) return rc;

    RowStatsParams rp{};
    rp.x = logits;
    rp.V = V;
    rp.rows = B * N;
    rp.N = N;
    rp.k = k;
    rp.parent = parent;
    rp.tok = draft_token;
    rp.skip_leaves = 0;
    rp.pc_normalized = 0;
    rp.m = h->m;
    rp.s = h->s;
    rp.arg = nullptr;
    rp.flags = h->flags;
    rp.pc = h->pc;
    rp.n_active = h->n_active;
    rp.chunk = h->chunk;
    rp.dbg = h->dbg;
    if (!dense) {
        set_split(h, rp);
        rc = timed(h, SPEC_K_ROW_STATS, st,
                   [&] { return launch_row_stats(rp, dtype, ROW_SAMPLE, st); });
        if (rc != SPEC_OK) return rc;
    } else {
        // The draft rows of the inner nodes are streamed in the same launch as the target rows.
        RowStatsParams dp = rp;
        dp.x = draft;
        dp.chunk = nullptr;   // partials are kept for the target rows only
        dp.skip_leaves = 1;
        dp.flags = h->dflags;
        dp.pc = h->qc;
        int mode = ROW_PROBS, ddt = SPEC_F32;
        if (draft_kind == SPEC_DRAFT_LOGITS) {
            mode = ROW_SAMPLE;
            ddt = draft_dtype;
            dp.m = h->mq;
            dp.s = h->sq;
        } else {
            dp.m = nullptr;
            dp.s = nullptr;
        }
        rc = timed(h, SPEC_K_ROW_STATS, st, [&] {
            return launch_row_stats_pair(rp, dtype, dp, ddt, mode, st);
        });
        if (rc != SPEC_OK) return rc;
    }

    SampleWalkParams wp{};
    wp.B = B;
    wp.N = N;
    wp.V = V;
    wp.dtype = dtype;
    wp.logits = logits;
    wp.parent = parent;
    wp.tok = draft_token;
    wp.uniforms = uniforms;
    wp.k = k;
    wp.m = h->m;
    wp.s = h->s;
    wp.pc = h->pc;
    wp.flags = h->flags;
    wp.draft_kind = draft_kind;
    wp.draft_dtype = draft_dtype;
    wp.draft = draft;
    wp.mq = h->mq;
    wp.sq = h->sq;
    wp.qc = h->qc;
    wp.dflags = h->dflags;
    wp.out = out;
    wp.n_active = h->n_active;
    wp.chunk = draft_kind == SPEC_DRAFT_POINT ? h->chunk : nullptr;
    wp.cluster = walk_cluster(h, B, draft_kind == SPEC_DRAFT_POINT);
    wp.dbg = h->dbg;
    return timed(h, SPEC_K_WALK_SAMPLE, st, [&] { return launch_walk_sample(wp, st); });
}

int spec_verify_greedy_lazy(spec_handle h, const void *logits, int dtype, int B, int N,
                            int64_t V, const int32_t *draft_token, const int32_t *parent,
                            int32_t *accept_len, int32_t *out_tokens, int32_t *kv_commit,
                            int32_t *bonus, int32_t *status, void *stream) {
    SPEC_RANGE("spec_verify_greedy_lazy");
    int rc = check_common(h, logits, dtype, B, N, V, draft_token, parent, accept_len,
                          out_tokens, kv_commit, bonus, status);
    if (rc != SPEC_OK || B == 0) return rc;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    if (!readable_by_device(logits, h->device)) return SPEC_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = debug_prologue(h, B, 0, st);
    if (rc != SPEC_OK) return rc;
    LazyGreedyParams lp;
    lp.B = B;
    lp.N = N;
    lp.V = V;
    lp.dtype = dtype;
    lp.logits = logits;
    lp.parent = parent;
    lp.tok = draft_token;
    lp.out = outputs(accept_len, out_tokens, kv_commit, bonus, status);
    lp.n_active = h->n_active;
    lp.dbg = h->dbg;
    return timed(h, SPEC_K_LAZY_GREEDY, st, [&] { return launch_lazy_greedy(lp, st); });
}

int spec_verify_sample_lazy(spec_handle h, const void *logits, int dtype, int B, int N,
                            int64_t V, const int32_t *draft_token, const int32_t *parent,
                            const void *draft, int draft_kind, int draft_dtype, float temperature,
                            const float *uniforms, int32_t *accept_len, int32_t *out_tokens,
                            int32_t *kv_commit, int32_t *bonus, int32_t *status, void *stream) {
    SPEC_RANGE("spec_verify_sample_lazy");
    int rc = check_common(h, logits, dtype, B, N, V, draft_token, parent, accept_len,
                          out_tokens, kv_commit, bonus, status);
    if (rc != SPEC_OK) return rc;
    if (!(temperature >= 0.f) || std::isinf(temperature)) return SPEC_ERR_ARG;
    const float k = temperature > 0.f ? kLog2eF / temperature : 0.f;
    if (temperature > 0.f && !std::isfinite(k)) return SPEC_ERR_ARG;
    if (draft_kind != SPEC_DRAFT_POINT && draft_kind != SPEC_DRAFT_PROBS_F32 &&
        draft_kind != SPEC_DRAFT_LOGITS)
        return SPEC_ERR_ARG;
    if (draft_kind == SPEC_DRAFT_LOGITS && draft_dtype != SPEC_F32 && draft_dtype != SPEC_BF16)
        return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (temperature == 0.f)
        return spec_verify_greedy_lazy(h, logits, dtype, B, N, V, draft_token, parent,
                                       accept_len, out_tokens, kv_commit, bonus, status, stream);
    if (!uniforms || !aligned(uniforms, 4)) return SPEC_ERR_ARG;
    if (draft_kind != SPEC_DRAFT_POINT) {
        if (!draft) return SPEC_ERR_ARG;
        const size_t de = draft_kind == SPEC_DRAFT_LOGITS ? esize(draft_dtype) : 4;
        if (!aligned(draft, de)) return SPEC_ERR_ARG;
    }
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    if (!readable_by_device(logits, h->device) ||
        (draft && !readable_by_device(draft, h->device)))
        return SPEC_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = debug_prologue(h, B, 0, st);
    if (rc != SPEC_OK) return rc;
    SampleWalkParams wp{};
    wp.B = B;
    wp.N = N;
    wp.V = V;
    wp.dtype = dtype;
    wp.logits = logits;
    wp.parent = parent;
    wp.tok = draft_token;
    wp.uniforms = uniforms;
    wp.k = k;
    wp.draft_kind = draft_kind;
    wp.draft_dtype = draft_dtype;
    wp.draft = draft;
    wp.lazy = 1;
    wp.host_rows = host_memory(logits);
    wp.out = outputs(accept_len, out_tokens, kv_commit, bonus, status);
    wp.n_active = h->n_active;
    wp.dbg = h->dbg;
    return timed(h, SPEC_K_LAZY_SAMPLE, st, [&] { return launch_walk_sample(wp, st); });
}

int spec_set_node_budget(spec_handle h, const int32_t *n_active) {
    SPEC_RANGE("spec_set_node_budget");
    if (!h) return SPEC_ERR_ARG;
    if (n_active && !aligned(n_active, 4)) return SPEC_ERR_ARG;
    h->n_active = n_active;
    return SPEC_OK;
}

int spec_budget_update(spec_handle h, const spec_budget_params *params,
                       const int32_t *accept_len, const int32_t *status, const int32_t *parent,
                       int B, int N, spec_budget_state *state, int32_t *n_active, void *stream) {
    SPEC_RANGE("spec_budget_update");
    if (!h || !params || !state || !n_active) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B || N < 1 || N > h->max_N || N > kMaxN) return SPEC_ERR_ARG;
    const spec_budget_params &q = *params;
    if (!(q.target > 0.0 && q.target <= 1.0) || !(q.alpha > 0.0 && q.alpha <= 1.0) ||
        !(q.band >= 0.0) || !std::isfinite(q.band))
        return SPEC_ERR_ARG;
    if (q.n_min < 1 || q.n_min > q.n_max || q.n_max > N || q.step < 1) return SPEC_ERR_ARG;
    if (B > 0 && (!accept_len || !status || !parent)) return SPEC_ERR_ARG;
    const void *ints[] = {accept_len, status, parent, n_active};
    for (const void *p : ints)
        if (p && !aligned(p, 4)) return SPEC_ERR_ARG;
    if (!aligned(state, alignof(spec_budget_state))) return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BudgetParams bp;
    bp.prm = q;
    bp.accept_len = accept_len;
    bp.status = status;
    bp.parent = parent;
    bp.B = B;
    bp.N = N;
    bp.state = state;
    bp.n_active = n_active;
    return timed(h, SPEC_K_BUDGET, st, [&] { return launch_budget_update(bp, st); });
}

int spec_kv_commit(spec_handle h, const void *src_k, const void *src_v, int src_dtype, int B,
                   int N, int H, int D, const int32_t *kv_commit, const int32_t *accept_len,
                   void *cache_k, void *cache_v, int cache_kind, int layout, int block_size,
                   int64_t num_blocks, const int32_t *block_table, int max_blocks,
                   const int32_t *seq_pos, const float *k_scale, const float *v_scale,
                   int scale_per_token, int32_t *commit_status, void *stream) {
    SPEC_RANGE("spec_kv_commit");
    if (!h) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B || N < 1 || N > h->max_N || N > kMaxN) return SPEC_ERR_ARG;
    if (H < 1 || D < 1 || (int64_t)H * D > (int64_t(1) << 24)) return SPEC_ERR_ARG;
    if (src_dtype != SPEC_F32 && src_dtype != SPEC_BF16 && src_dtype != SPEC_F16)
        return SPEC_ERR_ARG;
    if (cache_kind != SPEC_CACHE_SAME && cache_kind != SPEC_CACHE_FP8_E4M3 &&
        cache_kind != SPEC_CACHE_FP8_E5M2)
        return SPEC_ERR_ARG;
    if (layout != SPEC_KV_NHD && layout != SPEC_KV_HND) return SPEC_ERR_ARG;
    if (scale_per_token != SPEC_SCALE_TENSOR && scale_per_token != SPEC_SCALE_PER_TOKEN)
        return SPEC_ERR_ARG;
    if (block_size < 1 || num_blocks < 1 || num_blocks > INT32_MAX || max_blocks < 1)
        return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (!src_k || !src_v || !kv_commit || !accept_len || !cache_k || !cache_v || !block_table ||
        !seq_pos)
        return SPEC_ERR_ARG;
    const size_t se = src_dtype == SPEC_F32 ? 4 : 2;
    const size_t ce = cache_kind == SPEC_CACHE_SAME ? se : 1;
    if (!aligned(src_k, se) || !aligned(src_v, se) || !aligned(cache_k, ce) ||
        !aligned(cache_v, ce))
        return SPEC_ERR_ARG;
    const void *ints[] = {kv_commit, accept_len, block_table, seq_pos};
    for (const void *p : ints)
        if (!aligned(p, 4)) return SPEC_ERR_ARG;
    if ((k_scale && !aligned(k_scale, 4)) || (v_scale && !aligned(v_scale, 4)) ||
        (commit_status && !aligned(commit_status, 4)))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    KvCommitParams kp;
    kp.src_k = src_k;
    kp.src_v = src_v;
    kp.src_dtype = src_dtype;
    kp.B = B;
    kp.N = N;
    kp.H = H;
    kp.D = D;
    kp.kv_commit = kv_commit;
    kp.accept_len = accept_len;
    kp.cache_k = cache_k;
    kp.cache_v = cache_v;
    kp.cache_kind = cache_kind;
    kp.layout = layout;
    kp.block_size = block_size;
    kp.num_blocks = num_blocks;
    kp.block_table = block_table;
    kp.max_blocks = max_blocks;
    kp.seq_pos = seq_pos;
    kp.k_scale = k_scale;
    kp.v_scale = v_scale;
    kp.scale_per_token = scale_per_token;
    kp.status = commit_status;
    kp.sms = h->sms;
    // 8 elements per thread step: rows of D elements and 16-byte aligned bases.
    const bool vec = D % 8 == 0 && aligned(src_k, 16) && aligned(src_v, 16) &&
                     aligned(cache_k, 16) && aligned(cache_v, 16);
#ifdef SPEC_DEBUG
    // debug builds combine statuses with atomicMax, from zero
    if (commit_status &&
        cudaMemsetAsync(commit_status, 0, sizeof(int32_t) * (size_t)B, st) != cudaSuccess)
        return SPEC_ERR_CUDA;
#endif
    return timed(h, SPEC_K_KV_COMMIT, st, [&] { return launch_kv_commit(kp, vec, st); });
}

// ---- the tree step over a 4-bit cache --------------------------------------------------------

namespace {

bool float_type(int dtype) {
    return dtype == SPEC_F32 || dtype == SPEC_BF16 || dtype == SPEC_F16;
}

// Rows of H heads x D elements, `stride` elements from token to token.
bool rows_ok(const void *p, int64_t stride, int H, int D, int dtype) {
    return p && aligned(p, dtype == SPEC_F32 ? 4 : 2) && stride >= (int64_t)H * D &&
           stride <= (int64_t(1) << 32);
}

bool null_or_aligned(const void *p, size_t a) { return !p || aligned(p, a); }

// The parts of a 4-bit cache that the host can check; a batch of none needs no block table.
int check_cache(const spec_fp4_cache *c, int B) {
    if (!c) return SPEC_ERR_ARG;
    if (c->H < 1 || c->H > (1 << 16) || c->D < 16 || c->D % 16 != 0 || c->D > 512) return SPEC_ERR_ARG;
    if (c->layout != SPEC_KV_NHD && c->layout != SPEC_KV_HND) return SPEC_ERR_ARG;
    if (c->block_size < 1 || c->num_blocks < 1 || c->max_blocks < 1) return SPEC_ERR_ARG;
    if (c->num_blocks > INT32_MAX || (int64_t)c->block_size * c->H > INT32_MAX ||
        c->num_blocks > int64_t(UINT32_MAX) / ((int64_t)c->block_size * c->H) ||
        (int64_t)c->max_blocks * c->block_size > INT32_MAX - 1024)   // tiles past the end count too
        return SPEC_ERR_ARG;
    if (!c->k || !c->v || !c->k_sf || !c->v_sf || (B > 0 && !c->block_table))
        return SPEC_ERR_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_sf, 16) ||
        !aligned(c->v_sf, 16) || !null_or_aligned(c->block_table, 4) ||
        !null_or_aligned(c->k_scale, 4) || !null_or_aligned(c->v_scale, 4))
        return SPEC_ERR_ARG;
    return SPEC_OK;
}

}  // namespace

int spec_qk_norm_rope(spec_handle h, const void *q, int64_t q_stride, const void *k,
                      int64_t k_stride, int dtype, int B, int N, int Hq, int Hkv, int D,
                      const void *q_weight, const void *k_weight, float eps,
                      const float *inv_freq, int rot, int style, const int32_t *seq_pos,
                      const int32_t *depth, void *q_out, int64_t q_out_stride, void *k_out,
                      int64_t k_out_stride, void *stream) {
    SPEC_RANGE("spec_qk_norm_rope");
    if (!h) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B || N < 1 || (int64_t)B * N > INT32_MAX) return SPEC_ERR_ARG;
    if (!float_type(dtype) || Hq < 1 || Hkv < 1 || D < 1 || D > 1024 || Hq > (1 << 20) ||
        Hkv > (1 << 20))
        return SPEC_ERR_ARG;
    if (rot < 0 || rot > D || rot % 2 != 0) return SPEC_ERR_ARG;
    if (style != SPEC_ROPE_HALVES && style != SPEC_ROPE_PAIRS) return SPEC_ERR_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return SPEC_ERR_ARG;
    if ((q_weight == nullptr) != (k_weight == nullptr)) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (!rows_ok(q, q_stride, Hq, D, dtype) || !rows_ok(k, k_stride, Hkv, D, dtype) ||
        !rows_ok(q_out, q_out_stride, Hq, D, dtype) ||
        !rows_ok(k_out, k_out_stride, Hkv, D, dtype))
        return SPEC_ERR_ARG;
    if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride))
        return SPEC_ERR_ARG;
    const size_t e = dtype == SPEC_F32 ? 4 : 2;
    if (!null_or_aligned(q_weight, e) || !null_or_aligned(k_weight, e)) return SPEC_ERR_ARG;
    if ((rot > 0 && !inv_freq) || !null_or_aligned(inv_freq, 4) || !seq_pos ||
        !aligned(seq_pos, 4) || !null_or_aligned(depth, 4))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    QkRopeParams p;
    p.x[0] = q;
    p.x[1] = k;
    p.stride[0] = q_stride;
    p.stride[1] = k_stride;
    p.y[0] = q_out;
    p.y[1] = k_out;
    p.ystride[0] = q_out_stride;
    p.ystride[1] = k_out_stride;
    p.w[0] = q_weight;
    p.w[1] = k_weight;
    p.H[0] = Hq;
    p.H[1] = Hkv;
    p.dtype = dtype;
    p.tokens = (int64_t)B * N;
    p.N = N;
    p.D = D;
    p.rot = rot;
    p.pairs = style == SPEC_ROPE_PAIRS;
    p.eps = eps;
    p.inv_freq = inv_freq;
    p.seq_pos = seq_pos;
    p.depth = depth;
    p.sms = h->sms;
    return timed(h, SPEC_K_QK_ROPE, st, [&] { return launch_qk_rope(p, st); });
}

int spec_kv_commit_fp4(spec_handle h, const void *src_k, int64_t k_stride, const void *src_v,
                       int64_t v_stride, int src_dtype, int B, int N,
                       const spec_fp4_cache *cache, const int32_t *kv_commit,
                       const int32_t *accept_len, const int32_t *seq_pos,
                       int32_t *commit_status, void *stream) {
    SPEC_RANGE("spec_kv_commit_fp4");
    if (!h) return SPEC_ERR_ARG;
    const int rc = check_cache(cache, B);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || B > h->max_B || N < 1 || (int64_t)B * N > INT32_MAX) return SPEC_ERR_ARG;
    if (kv_commit && (N > h->max_N || N > kMaxN || !accept_len)) return SPEC_ERR_ARG;
    if (!float_type(src_dtype)) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    if (!rows_ok(src_k, k_stride, cache->H, cache->D, src_dtype) ||
        !rows_ok(src_v, v_stride, cache->H, cache->D, src_dtype) || !seq_pos)
        return SPEC_ERR_ARG;
    if (!null_or_aligned(kv_commit, 4) || !null_or_aligned(accept_len, 4) ||
        !aligned(seq_pos, 4) || !null_or_aligned(commit_status, 4))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    KvFp4Params p = {};
    p.cache = *cache;
    p.src[0] = src_k;
    p.src[1] = src_v;
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.dtype = src_dtype;
    p.B = B;
    p.N = N;
    p.kv_commit = kv_commit;
    p.last = accept_len;
    p.pos = seq_pos;
    p.status = commit_status;
    p.sms = h->sms;
    return timed(h, SPEC_K_KV_COMMIT_FP4, st, [&] { return launch_kv_commit_fp4(p, st); });
}

int spec_kv_load_fp4(spec_handle h, const spec_fp4_cache *cache, int B, const int32_t *start,
                     const int32_t *count, int64_t max_len, void *out_k, void *out_v,
                     int out_dtype, int32_t *status, void *stream) {
    SPEC_RANGE("spec_kv_load_fp4");
    if (!h) return SPEC_ERR_ARG;
    const int rc = check_cache(cache, B);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || B > h->max_B || max_len < 0 || max_len > INT32_MAX) return SPEC_ERR_ARG;
    if (!float_type(out_dtype)) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    const size_t e = out_dtype == SPEC_F32 ? 4 : 2;
    if (!start || !count || !aligned(start, 4) || !aligned(count, 4) ||
        !null_or_aligned(status, 4))
        return SPEC_ERR_ARG;
    if (max_len > 0 && (!out_k || !out_v || !aligned(out_k, e) || !aligned(out_v, e)))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    KvFp4Params p = {};
    p.cache = *cache;
    p.out[0] = out_k;
    p.out[1] = out_v;
    p.dtype = out_dtype;
    p.B = B;
    p.max_len = max_len;
    p.last = count;
    p.pos = start;
    p.status = status;
    p.sms = h->sms;
    return timed(h, SPEC_K_KV_LOAD_FP4, st, [&] { return launch_kv_load_fp4(p, st); });
}

namespace {

// Sizes of a tree attention call.
int check_attention(spec_handle h, int B, int N, int Hq, int H, int D) {
    if (!h) return SPEC_ERR_ARG;
    if (B < 0 || B > h->max_B || N < 1 || N > h->max_N || N > kMaxN) return SPEC_ERR_ARG;
    if (H < 1 || Hq < H || Hq % H != 0 || Hq > (1 << 16)) return SPEC_ERR_ARG;
    return D == 64 || D == 128 || D == 256 ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

}  // namespace

int spec_tree_attention_workspace(spec_handle h, int B, int N, int Hq, int H, int D,
                                  int64_t *bytes) {
    SPEC_RANGE("spec_tree_attention_workspace");
    const int rc = check_attention(h, B, N, Hq, H, D);
    if (rc != SPEC_OK) return rc;
    if (!bytes) return SPEC_ERR_ARG;
    *bytes = tree_attn_workspace(N * (Hq / H), D, h->sms);
    return SPEC_OK;
}

int spec_tree_attention_fp4(spec_handle h, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, int dtype, int B,
                            int N, int Hq, const spec_fp4_cache *cache, const int32_t *ctx_len,
                            const uint64_t *anc_mask, float scale, void *out, float *lse,
                            int32_t *status, void *workspace, int64_t workspace_bytes,
                            void *stream) {
    SPEC_RANGE("spec_tree_attention_fp4");
    if (!h) return SPEC_ERR_ARG;
    int rc = check_cache(cache, B);
    if (rc != SPEC_OK) return rc;
    rc = check_attention(h, B, N, Hq, cache->H, cache->D);
    if (rc != SPEC_OK) return rc;
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    const int H = cache->H, D = cache->D;
    if (!rows_ok(q, q_stride, Hq, D, dtype) || !rows_ok(k, k_stride, H, D, dtype) ||
        !rows_ok(v, v_stride, H, D, dtype) || !ctx_len || !anc_mask || !out)
        return SPEC_ERR_ARG;
    if (!aligned(ctx_len, 4) || !aligned(anc_mask, 8) || !aligned(out, 2) ||
        !null_or_aligned(lse, 4) || !null_or_aligned(status, 4))
        return SPEC_ERR_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < tree_attn_workspace(N * (Hq / H), D, h->sms))
        return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TreeAttnParams p;
    p.cache = *cache;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.dtype = dtype;
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.G = Hq / H;
    p.ctx_len = ctx_len;
    p.mask = anc_mask;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    p.status = status;
    p.workspace = workspace;
    p.sms = h->sms;
    p.lose = h->inject_lost;
    h->inject_lost = 0;
    // a page found outside the cache raises the request's status from zero
    if (status && cudaMemsetAsync(status, 0, sizeof(int32_t) * (size_t)B, st) != cudaSuccess)
        return SPEC_ERR_CUDA;
    return timed(h, SPEC_K_TREE_ATTN, st, [&] { return launch_tree_attn(p, st); });
}

int spec_row_stats(spec_handle h, const void *logits, int dtype, int rows, int N, int64_t V,
                   float temperature, const int32_t *draft_token, const int32_t *parent,
                   float *row_max, float *row_sum, int32_t *row_argmax, int32_t *row_flags,
                   float *child_prob, void *stream) {
    SPEC_RANGE("spec_row_stats");
    if (!h) return SPEC_ERR_ARG;
    if (rows < 0 || N < 1 || N > kMaxN || V < 1 || V > kMaxV) return SPEC_ERR_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_ARG;
    if (!(temperature >= 0.f) || std::isinf(temperature)) return SPEC_ERR_ARG;
    const float k = temperature > 0.f ? kLog2eF / temperature : 0.f;
    if (temperature > 0.f && !std::isfinite(k)) return SPEC_ERR_ARG;
    const bool gather = draft_token && parent && child_prob;
    if (gather && (temperature == 0.f || rows % N != 0)) return SPEC_ERR_ARG;
    if (rows == 0) return SPEC_OK;
    if (!logits || !row_max || !row_sum || !row_argmax || !row_flags) return SPEC_ERR_ARG;
    if (!aligned(logits, esize(dtype))) return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    RowStatsParams rp{};
    rp.x = logits;
    rp.V = V;
    rp.rows = rows;
    rp.N = N;
    rp.k = k;
    rp.parent = gather ? parent : nullptr;
    rp.tok = gather ? draft_token : nullptr;
    rp.skip_leaves = 0;
    rp.pc_normalized = 1;
    rp.m = row_max;
    rp.s = row_sum;
    rp.arg = row_argmax;
    rp.flags = row_flags;
    rp.pc = gather ? child_prob : nullptr;
    set_split(h, rp);
    if (rp.split > 1) {
        const int drc = debug_prologue(h, 0, rows, st);
        if (drc != SPEC_OK) return drc;
    }
    const int mode = temperature > 0.f ? ROW_SAMPLE : ROW_GREEDY;
    return timed(h, SPEC_K_ROW_STATS, st, [&] { return launch_row_stats(rp, dtype, mode, st); });
}

int spec_profile_begin(spec_handle h) {
    if (!h) return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    if (!h->ev_ready) {
        for (int i = 0; i < 2 * kMaxRecords; ++i)
            if (cudaEventCreate(&h->ev[i]) != cudaSuccess) return SPEC_ERR_CUDA;
        h->ev_ready = true;
    }
    h->nrec = 0;
    h->prof = true;
    return SPEC_OK;
}

int spec_profile_end(spec_handle h, float *ms_per_class, int32_t *launches_per_class) {
    if (!h || !ms_per_class || !launches_per_class) return SPEC_ERR_ARG;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    for (int c = 0; c < SPEC_K_COUNT; ++c) {
        ms_per_class[c] = 0.f;
        launches_per_class[c] = 0;
    }
    int rc = SPEC_OK;
    for (int i = 0; i < h->nrec; ++i) {
        float ms = 0.f;
        if (cudaEventSynchronize(h->ev[2 * i + 1]) != cudaSuccess ||
            cudaEventElapsedTime(&ms, h->ev[2 * i], h->ev[2 * i + 1]) != cudaSuccess) {
            rc = SPEC_ERR_CUDA;
            continue;
        }
        ms_per_class[h->cls[i]] += ms;
        launches_per_class[h->cls[i]] += 1;
    }
    h->prof = false;
    h->nrec = 0;
    return rc;
}

int spec_debug_build(void) {
    SPEC_RANGE("spec_debug_build");
#ifdef SPEC_DEBUG
    return 1;
#else
    return 0;
#endif
}

int spec_debug_inject_arrival(spec_handle h, int row, int value) {
    SPEC_RANGE("spec_debug_inject_arrival");
#ifdef SPEC_DEBUG
    if (!h || row < 0 || (int64_t)row >= (int64_t)h->max_B * h->max_N) return SPEC_ERR_ARG;
    h->inject_row = row;
    h->inject_value = value;
    return SPEC_OK;
#else
    (void)h;
    (void)row;
    (void)value;
    return SPEC_ERR_UNSUPPORTED;
#endif
}

int spec_debug_inject_lost_wait(spec_handle h) {
    SPEC_RANGE("spec_debug_inject_lost_wait");
#ifdef SPEC_DEBUG
    if (!h) return SPEC_ERR_ARG;
    h->inject_lost = 1;
    return SPEC_OK;
#else
    (void)h;
    return SPEC_ERR_UNSUPPORTED;
#endif
}

int spec_debug_words(spec_handle h, int32_t *words, int B, void *stream) {
    SPEC_RANGE("spec_debug_words");
#ifdef SPEC_DEBUG
    if (!h || B < 0 || B > h->max_B || (B > 0 && !words)) return SPEC_ERR_ARG;
    if (B == 0) return SPEC_OK;
    DeviceScope ds(h->device);
    if (!ds.ok()) return SPEC_ERR_CUDA;
    return cudaMemcpyAsync(words, h->dbg, sizeof(int32_t) * (size_t)B, cudaMemcpyDeviceToDevice,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
#else
    (void)h;
    (void)words;
    (void)B;
    (void)stream;
    return SPEC_ERR_UNSUPPORTED;
#endif
}

}  // extern "C"
