// gg_api_moe.cpp -- the C entry points around the grouped GEMMs: router,
// dispatch and combine, gradient clipping (declared in include/gg_moe.h).
// As in gg_api.cpp, every argument is checked on the host before any device
// work is queued, and nothing is allocated.
#include <hip/hip_runtime.h>

#include <cmath>

#include "gg_host.hpp"
#include "gg_step.hpp"

using namespace gg;

namespace {

// Token counts: a block of 256 threads per token stays within a launch's
// 2^32 threads, and tokens * top_k (at most 2^28) within int32.
constexpr int64_t kMaxTokens = 1 << 23;
constexpr int32_t kMaxTopK = 32;
constexpr int32_t kMaxWidth = 1 << 20;

// Rows that a plan's groups are padded to.
bool is_granule(int32_t g) { return g >= 1 && g <= 256 && (g & (g - 1)) == 0; }

gg_status check_tokens(int64_t tokens, int32_t num_experts, int32_t top_k) {
    if (num_experts < 1 || num_experts > 1024)
        return fail(GG_ERR_SHAPE, "num_experts must be in 1..1024 (got %d)", num_experts);
    if (tokens < 0 || top_k < 1)
        return fail(GG_ERR_SHAPE, "tokens must be >= 0 and top_k >= 1");
    if (tokens > kMaxTokens || top_k > kMaxTopK)
        return fail(GG_ERR_UNSUPPORTED, "tokens is limited to 2^23 and top_k to 32");
    return GG_OK;
}

gg_status check_route(const void* logits, gg_dtype dtype, int64_t ld, int64_t tokens,
                      int32_t num_experts, int32_t top_k, gg_score score, float scale,
                      uint32_t flags, const char* name) {
    if (!is_out_dtype(dtype))
        return fail(GG_ERR_DTYPE, "dtype must be GG_BF16, GG_F16 or GG_F32");
    gg_status st = check_tokens(tokens, num_experts, top_k);
    if (st != GG_OK)
        return st;
    if (top_k > num_experts)
        return fail(GG_ERR_SHAPE, "top_k %d exceeds num_experts %d", top_k, num_experts);
    if (ld < num_experts || ld > INT32_MAX)
        return fail(GG_ERR_LAYOUT, "ld must be in num_experts .. 2^31-1 (got %lld)", (long long)ld);
    if (score != GG_SOFTMAX && score != GG_SIGMOID)
        return fail(GG_ERR_MODE, "score must be GG_SOFTMAX or GG_SIGMOID");
    if (!std::isfinite(scale))
        return fail(GG_ERR_VALUE, "scale must be finite");
    if (flags & ~(uint32_t)GG_FLAG_NORMALIZE)
        return fail(GG_ERR_MODE, "unsupported flags 0x%x for %s", flags, name);
    if (!logits && tokens > 0)
        return fail(GG_ERR_NULL, "logits must be non-NULL");
    if (off(logits, size_of(dtype)))
        return fail(GG_ERR_ALIGN, "logits must be aligned to its element");
    return GG_OK;
}

gg_status check_rows(int64_t tokens, int32_t width, int32_t top_k, int64_t m_rows, int64_t ld,
                     const char* pitch) {
    gg_status st = check_tokens(tokens, 1, top_k);
    if (st != GG_OK)
        return st;
    if (width < 1 || m_rows < 0 || m_rows > INT32_MAX)
        return fail(GG_ERR_SHAPE, "width must be positive and m_rows in 0..2^31-1");
    if (width > kMaxWidth)
        return fail(GG_ERR_UNSUPPORTED, "width is limited to 2^20");
    if (ld < width || ld > INT32_MAX)
        return fail(GG_ERR_LAYOUT, "%s must be in width .. 2^31-1 (got %lld)", pitch, (long long)ld);
    return GG_OK;
}

}  // namespace

extern "C" {

size_t gg_route_workspace_size(int64_t tokens, int32_t num_experts) {
    if (tokens < 0 || tokens > kMaxTokens || num_experts < 1 || num_experts > 1024)
        return round256(kWsHeader);
    return round256(route_workspace(tokens, num_experts));
}

gg_status gg_route(const void* logits, gg_dtype dtype, int64_t ld, int64_t tokens,
                   int32_t num_experts, const float* bias, int32_t top_k, gg_score score,
                   float scale, uint32_t flags, int32_t* ids, float* prob, int32_t* counts,
                   int32_t* routed, float* balance, void* workspace, size_t workspace_bytes,
                   void* stream) {
    gg_status st = check_route(logits, dtype, ld, tokens, num_experts, top_k, score, scale, flags,
                               "gg_route");
    if (st != GG_OK)
        return st;
    if (((!ids || !prob) && tokens > 0) || !counts || !routed)
        return fail(GG_ERR_NULL, "ids, prob, counts and routed must be non-NULL");
    if (off(ids, 4) || off(prob, 4) || off(counts, 4) || off(routed, 4) || off(balance, 4) || off(bias, 4))
        return fail(GG_ERR_ALIGN, "ids, prob, counts, routed, balance and bias must be 4-byte aligned");
    st = check_workspace(workspace, workspace_bytes, gg_route_workspace_size(tokens, num_experts));
    if (st != GG_OK)
        return st;
    RouteArgs p = {};
    p.logits = logits;
    p.ld = ld;
    p.T = tokens;
    p.E = num_experts;
    p.k = top_k;
    p.bias = bias;
    p.softmax = score == GG_SOFTMAX;
    p.normalize = (flags & GG_FLAG_NORMALIZE) != 0;
    p.scale = scale;
    p.ids = ids;
    p.prob = prob;
    p.counts = counts;
    p.routed = routed;
    p.balance = balance;
    p.ws = (int32_t*)workspace;
    return go("gg_route", tokens, num_experts, [&](LaunchInfo* li) {
        return launch_route(p, (int)dtype, (hipStream_t)stream, li);
    });
}

gg_status gg_route_bwd(const void* logits, gg_dtype dtype, int64_t ld, int64_t tokens,
                       int32_t num_experts, int32_t top_k, gg_score score, float scale,
                       uint32_t flags, const int32_t* ids, const int32_t* counts,
                       const int32_t* routed, const float* dprob, const int32_t* row_of,
                       int64_t m_rows, const float* dbalance, void* dlogits, void* stream) {
    gg_status st = check_route(logits, dtype, ld, tokens, num_experts, top_k, score, scale, flags,
                               "gg_route_bwd");
    if (st != GG_OK)
        return st;
    if (!counts || !routed || ((!ids || !dlogits) && tokens > 0))
        return fail(GG_ERR_NULL, "ids, counts, routed and dlogits must be non-NULL");
    if (!dprob && tokens > 0 && !(row_of && m_rows == 0))
        return fail(GG_ERR_NULL, "dprob must be non-NULL");
    if (row_of && (m_rows < 0 || m_rows > INT32_MAX))
        return fail(GG_ERR_SHAPE, "m_rows must be in 0..2^31-1");
    if (off(ids, 4) || off(counts, 4) || off(routed, 4) || off(dprob, 4) || off(row_of, 4) ||
        off(dbalance, 4) || off(dlogits, size_of(dtype)))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    RouteBwdArgs p = {};
    p.logits = logits;
    p.ld = ld;
    p.T = tokens;
    p.E = num_experts;
    p.k = top_k;
    p.ids = ids;
    p.counts = counts;
    p.routed = routed;
    p.softmax = score == GG_SOFTMAX;
    p.normalize = (flags & GG_FLAG_NORMALIZE) != 0;
    p.scale = scale;
    p.dprob = dprob;
    p.row_of = row_of;
    p.m_rows = m_rows;
    p.dbalance = dbalance;
    p.dlogits = dlogits;
    return go("gg_route_bwd", tokens, num_experts, [&](LaunchInfo* li) {
        return launch_route_bwd(p, (int)dtype, (hipStream_t)stream, li);
    });
}

size_t gg_plan_workspace_size(int64_t tokens, int32_t num_experts) {
    if (tokens < 0 || tokens > kMaxTokens || num_experts < 1 || num_experts > 1024)
        return round256(kWsHeader);
    return round256(plan_workspace(tokens, num_experts));
}

int64_t gg_plan_max_rows(int64_t tokens, int32_t top_k, int32_t num_experts, int32_t granule) {
    if (tokens < 0 || tokens > kMaxTokens || top_k < 1 || top_k > kMaxTopK || num_experts < 1 ||
        num_experts > 1024 || !is_granule(granule))
        return 0;
    const int64_t n = tokens * top_k, e = n < num_experts ? n : num_experts;
    return (n + (granule - 1) * e) / granule * granule;
}

gg_status gg_plan(const int32_t* ids, int64_t tokens, int32_t top_k, int32_t num_experts,
                  int32_t granule, int64_t m_rows, const float* prob, int32_t* counts,
                  int32_t* padded_offsets, int32_t* row_of, float* prob_rows, void* workspace,
                  size_t workspace_bytes, void* stream) {
    gg_status st = check_tokens(tokens, num_experts, top_k);
    if (st != GG_OK)
        return st;
    if (!is_granule(granule))
        return fail(GG_ERR_SHAPE, "granule must be a power of two in 1..256 (got %d)", granule);
    if (m_rows < 0 || m_rows > INT32_MAX)
        return fail(GG_ERR_SHAPE, "m_rows must be in 0..2^31-1");
    if (((!ids || !row_of) && tokens > 0) || !counts || !padded_offsets)
        return fail(GG_ERR_NULL, "ids, counts, padded_offsets and row_of must be non-NULL");
    if ((prob != nullptr) != (prob_rows != nullptr) && tokens > 0 && m_rows > 0)
        return fail(GG_ERR_MODE, "give both of prob and prob_rows, or neither");
    if (off(ids, 4) || off(prob, 4) || off(counts, 4) || off(padded_offsets, 4) || off(row_of, 4) ||
        off(prob_rows, 4))
        return fail(GG_ERR_ALIGN, "every array must be 4-byte aligned");
    st = check_workspace(workspace, workspace_bytes, gg_plan_workspace_size(tokens, num_experts));
    if (st != GG_OK)
        return st;
    PlanArgs p = {};
    p.ids = ids;
    p.T = tokens;
    p.m_rows = m_rows;
    p.E = num_experts;
    p.k = top_k;
    p.granule = granule;
    p.prob = prob;
    p.counts = counts;
    p.ends = padded_offsets;
    p.row_of = row_of;
    p.prob_rows = prob ? prob_rows : nullptr;
    p.ws = (int32_t*)workspace;
    return go("gg_plan", tokens, num_experts,
              [&](LaunchInfo* li) { return launch_plan(p, (hipStream_t)stream, li); });
}

gg_status gg_permute(const void* x, gg_dtype dtype, int64_t ldx, int64_t tokens, int32_t width,
                     const int32_t* row_of, int32_t top_k, const int32_t* counts,
                     const int32_t* padded_offsets, int32_t num_experts, int64_t m_rows,
                     void* x_rows, void* stream) {
    if (!is_out_dtype(dtype) && !is_fp8(dtype))
        return fail(GG_ERR_DTYPE, "dtype must be GG_BF16, GG_F16, GG_F32, GG_F8E4M3 or GG_F8E5M2");
    gg_status st = check_rows(tokens, width, top_k, m_rows, ldx, "ldx");
    if (st == GG_OK)
        st = check_tokens(tokens, num_experts, top_k);
    if (st != GG_OK)
        return st;
    if (((!x || !row_of) && tokens > 0) || !counts || !padded_offsets || (!x_rows && m_rows > 0))
        return fail(GG_ERR_NULL, "x, row_of, counts, padded_offsets and x_rows must be non-NULL");
    if (off(x, size_of(dtype)) || off(x_rows, size_of(dtype)) || off(row_of, 4) || off(counts, 4) ||
        off(padded_offsets, 4))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    RowsArgs p = {};
    p.tokens = x;
    p.ld = ldx;
    p.T = tokens;
    p.m_rows = m_rows;
    p.width = width;
    p.k = top_k;
    p.E = num_experts;
    p.row_of = row_of;
    p.counts = counts;
    p.ends = padded_offsets;
    p.rows_out = x_rows;
    return go("gg_permute", tokens, width, [&](LaunchInfo* li) {
        return launch_permute(p, (int)dtype, (hipStream_t)stream, li);
    });
}

gg_status gg_combine(const void* y_rows, gg_dtype dtype, int64_t m_rows, int32_t width,
                     const int32_t* row_of, int64_t tokens, int32_t top_k, const float* weights,
                     void* out, int64_t ldo, void* stream) {
    if (!is_out_dtype(dtype))
        return fail(GG_ERR_DTYPE, "dtype must be GG_BF16, GG_F16 or GG_F32");
    gg_status st = check_rows(tokens, width, top_k, m_rows, ldo, "ldo");
    if (st != GG_OK)
        return st;
    if ((!y_rows && m_rows > 0) || ((!row_of || !out) && tokens > 0))
        return fail(GG_ERR_NULL, "y_rows, row_of and out must be non-NULL");
    if (off(y_rows, size_of(dtype)) || off(out, size_of(dtype)) || off(row_of, 4) || off(weights, 4))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    RowsArgs p = {};
    p.out = out;
    p.ld = ldo;
    p.T = tokens;
    p.m_rows = m_rows;
    p.width = width;
    p.k = top_k;
    p.row_of = row_of;
    p.rows_in = y_rows;
    p.weights = weights;
    return go("gg_combine", tokens, width, [&](LaunchInfo* li) {
        return launch_combine(p, (int)dtype, (hipStream_t)stream, li);
    });
}

gg_status gg_combine_bwd(const void* dout, gg_dtype dtype, int64_t ldd, int64_t tokens,
                         int32_t width, const void* y_rows, int64_t m_rows, const float* weights,
                         const int32_t* row_of, int32_t top_k, const int32_t* counts,
                         const int32_t* padded_offsets, int32_t num_experts, void* dy_rows,
                         float* dweights, void* stream) {
    if (!is_out_dtype(dtype))
        return fail(GG_ERR_DTYPE, "dtype must be GG_BF16, GG_F16 or GG_F32");
    gg_status st = check_rows(tokens, width, top_k, m_rows, ldd, "ldd");
    if (st == GG_OK)
        st = check_tokens(tokens, num_experts, top_k);
    if (st != GG_OK)
        return st;
    if (((!dout || !row_of || !weights || !dweights) && tokens > 0) || !counts || !padded_offsets ||
        ((!y_rows || !dy_rows) && m_rows > 0))
        return fail(GG_ERR_NULL, "every array must be non-NULL");
    if (off(dout, size_of(dtype)) || off(y_rows, size_of(dtype)) || off(dy_rows, size_of(dtype)) ||
        off(row_of, 4) || off(weights, 4) || off(dweights, 4) || off(counts, 4) || off(padded_offsets, 4))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    RowsArgs p = {};
    p.tokens = dout;
    p.ld = ldd;
    p.T = tokens;
    p.m_rows = m_rows;
    p.width = width;
    p.k = top_k;
    p.E = num_experts;
    p.row_of = row_of;
    p.counts = counts;
    p.ends = padded_offsets;
    p.rows_in = y_rows;
    p.rows_out = dy_rows;
    p.weights = weights;
    p.dweights = dweights;
    return go("gg_combine_bwd", tokens, width, [&](LaunchInfo* li) {
        return launch_combine_bwd(p, (int)dtype, (hipStream_t)stream, li);
    });
}

size_t gg_grad_workspace_size(void) { return round256(grad_workspace()); }

static gg_status check_grads(const int64_t* ptrs, const int64_t* ends, const int32_t* dtypes,
                             int32_t n, int64_t total, const double* sumsq) {
    if (n < 0 || n > (1 << 24) || total < 0 || (n == 0 && total != 0))
        return fail(GG_ERR_SHAPE, "n must be in 0..2^24 and total >= 0 (0 without tensors)");
    if (total > ((int64_t)1 << 40))
        return fail(GG_ERR_UNSUPPORTED, "total is limited to 2^40 elements");
    if (((!ptrs || !ends || !dtypes) && n > 0) || !sumsq)
        return fail(GG_ERR_NULL, "ptrs, ends, dtypes and sumsq must be non-NULL");
    if (off(ptrs, 8) || off(ends, 8) || off(dtypes, 4) || off(sumsq, 8))
        return fail(GG_ERR_ALIGN, "ptrs, ends and sumsq must be 8-byte aligned, dtypes 4-byte");
    return GG_OK;
}

gg_status gg_grad_norm(const int64_t* ptrs, const int64_t* ends, const int32_t* dtypes, int32_t n,
                       int64_t total, double* sumsq, int32_t accumulate, void* workspace,
                       size_t workspace_bytes, void* stream) {
    gg_status st = check_grads(ptrs, ends, dtypes, n, total, sumsq);
    if (st == GG_OK)
        st = check_workspace(workspace, workspace_bytes, gg_grad_workspace_size());
    if (st != GG_OK)
        return st;
    GradArgs p = {};
    p.ptrs = ptrs;
    p.ends = ends;
    p.dtypes = dtypes;
    p.n = n;
    p.total = total;
    p.sumsq = sumsq;
    p.accumulate = accumulate ? 1 : 0;
    p.ws = (int32_t*)workspace;
    return go("gg_grad_norm", n, total,
              [&](LaunchInfo* li) { return launch_grad_norm(p, (hipStream_t)stream, li); });
}

gg_status gg_grad_clip(const int64_t* ptrs, const int64_t* ends, const int32_t* dtypes, int32_t n,
                       int64_t total, const double* sumsq, float max_norm, float eps, float* norm,
                       const int64_t* out_ptrs, void* stream) {
    gg_status st = check_grads(ptrs, ends, dtypes, n, total, sumsq);
    if (st != GG_OK)
        return st;
    if (!norm)
        return fail(GG_ERR_NULL, "norm must be non-NULL");
    if (off(norm, 4) || off(out_ptrs, 8))
        return fail(GG_ERR_ALIGN, "norm must be 4-byte, out_ptrs 8-byte aligned");
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps))
        return fail(GG_ERR_VALUE, "max_norm must be >= 0, eps >= 0 and finite");
    GradArgs p = {};
    p.ptrs = ptrs;
    p.out_ptrs = out_ptrs ? out_ptrs : ptrs;
    p.ends = ends;
    p.dtypes = dtypes;
    p.n = n;
    p.total = total;
    p.sumsq = (double*)sumsq;
    p.max_norm = max_norm;
    p.eps = eps;
    p.norm = norm;
    return go("gg_grad_clip", n, total,
              [&](LaunchInfo* li) { return launch_grad_clip(p, (hipStream_t)stream, li); });
}

}  // extern "C"
