// gg_api_forward.cpp -- the C entry points of the experts' forward pass: MXFP4
// quantisation, the gated activation, the grouped MXFP4 product, a layer for a
// few tokens (declared in include/gg_moe.h).  As in gg_api.cpp, every argument
// is checked on the host before any device work is queued, and nothing is
// allocated.
#include <hip/hip_runtime.h>

#include <cmath>

#include "gg_forward.hpp"
#include "gg_host.hpp"

using namespace gg;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int32_t kMaxK = 1 << 21;           // as of the other grouped products
constexpr int32_t kFewTokens = 64, kFewTopK = 32, kFewWidth = 1 << 16;

// (rows, width) of a row-wise call; pitch: row pitch of at least `wide`.
gg_status check_matrix(int64_t rows, int32_t width, const char* name, int64_t pitch, int64_t wide,
                       const char* pitch_name) {
    if (rows < 0 || width < 32 || width % 32 != 0)
        return fail(GG_ERR_SHAPE, "rows must be >= 0 and %s a positive multiple of 32 (got %lld, %d)", name,
                    (long long)rows, width);
    if (rows > kMaxRows || width > kMaxWidth)
        return fail(GG_ERR_UNSUPPORTED, "rows is limited to 2^30 and %s to 2^20", name);
    if (pitch < wide || pitch > INT32_MAX)
        return fail(GG_ERR_LAYOUT, "%s must be in %lld .. 2^31-1 (got %lld)", pitch_name, (long long)wide,
                    (long long)pitch);
    return GG_OK;
}

gg_status check_act(gg_act act, float geglu_alpha, float clamp_min, float clamp_max, float linear_offset,
                    float situ_beta1, float situ_beta2, uint32_t flags, const char* name, ActArgs* out) {
    if (act != GG_DSWIGLU && act != GG_DGEGLU && act != GG_DSITUGLU)
        return fail(GG_ERR_MODE, "act must be GG_DSWIGLU, GG_DGEGLU or GG_DSITUGLU");
    if (flags & ~(uint32_t)GG_FLAG_GATE_FIRST)
        return fail(GG_ERR_MODE, "unsupported flags 0x%x for %s", flags, name);
    if (act == GG_DGEGLU && (std::isnan(geglu_alpha) || std::isnan(linear_offset) || !(clamp_min <= clamp_max)))
        return fail(GG_ERR_VALUE, "GeGLU constants must not be NaN, nor clamp_min exceed clamp_max");
    if (act == GG_DSITUGLU &&
        !(situ_beta1 > 0 && situ_beta2 > 0 && std::isfinite(situ_beta1) && std::isfinite(situ_beta2)))
        return fail(GG_ERR_VALUE, "situ_beta1 and situ_beta2 must be positive and finite");
    out->act = act;
    out->gate_first = (flags & GG_FLAG_GATE_FIRST) != 0;
    out->alpha = geglu_alpha;
    out->lo = clamp_min;
    out->hi = clamp_max;
    out->offset = linear_offset;
    out->b1 = situ_beta1;
    out->b2 = situ_beta2;
    return GG_OK;
}

gg_status check_quant(const void* x, gg_dtype dtype, int64_t ld, const char* pitch, int64_t rows, int32_t width,
                      const uint8_t* codes, const uint8_t* scales, const int32_t* end) {
    if (!is_out_dtype(dtype))
        return fail(GG_ERR_DTYPE, "dtype must be GG_BF16, GG_F16 or GG_F32");
    gg_status st = check_matrix(rows, width, "width", ld, width, pitch);
    if (st != GG_OK)
        return st;
    if ((!x || !codes || !scales) && rows > 0)
        return fail(GG_ERR_NULL, "the rows, codes and scales must be non-NULL");
    if (off(x, size_of(dtype)) || off(end, 4))
        return fail(GG_ERR_ALIGN, "the rows must be aligned to their element, end to 4 bytes");
    return GG_OK;
}

}  // namespace

extern "C" {

gg_status gg_mx4_quant(const void* x, gg_dtype dtype, int64_t ldx, int64_t rows, int32_t width, uint8_t* codes,
                       uint8_t* scales, const int32_t* end, void* stream) {
    gg_status st = check_quant(x, dtype, ldx, "ldx", rows, width, codes, scales, end);
    if (st != GG_OK)
        return st;
    const QuantArgs p = {const_cast<void*>(x), ldx, rows, width, codes, scales, end};
    return go("gg_mx4_quant", rows, width,
              [&](LaunchInfo* li) { return launch_quant(p, (int)dtype, (hipStream_t)stream, li); });
}

gg_status gg_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t width, void* out,
                         gg_dtype dtype, int64_t ldo, const int32_t* end, void* stream) {
    gg_status st = check_quant(out, dtype, ldo, "ldo", rows, width, codes, scales, end);
    if (st != GG_OK)
        return st;
    const QuantArgs p = {out, ldo, rows, width, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), end};
    return go("gg_mx4_dequant", rows, width,
              [&](LaunchInfo* li) { return launch_dequant(p, (int)dtype, (hipStream_t)stream, li); });
}

gg_status gg_glu(const void* c, gg_dtype c_dtype, int64_t ldc, const float* prob, int64_t rows, int32_t n, void* y,
                 gg_dtype y_dtype, int64_t ldy, gg_act act, float geglu_alpha, float clamp_min, float clamp_max,
                 float linear_offset, float situ_beta1, float situ_beta2, uint32_t flags, const int32_t* end,
                 void* stream) {
    if (!is_out_dtype(c_dtype) || !is_out_dtype(y_dtype))
        return fail(GG_ERR_DTYPE, "c_dtype and y_dtype must be GG_BF16, GG_F16 or GG_F32");
    gg_status st = check_matrix(rows, n, "n", ldc, 2 * (int64_t)n, "ldc");
    if (st == GG_OK)
        st = check_matrix(rows, n, "n", ldy, n, "ldy");
    GluArgs p = {};
    if (st == GG_OK)
        st = check_act(act, geglu_alpha, clamp_min, clamp_max, linear_offset, situ_beta1, situ_beta2, flags,
                       "gg_glu", &p.act);
    if (st != GG_OK)
        return st;
    if ((!c || !y) && rows > 0)
        return fail(GG_ERR_NULL, "c and y must be non-NULL");
    if (off(c, size_of(c_dtype)) || off(y, size_of(y_dtype)) || off(prob, 4) || off(end, 4))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    p.c = c;
    p.ldc = ldc;
    p.rows = rows;
    p.n = n;
    p.prob = prob;
    p.y = y;
    p.ldy = ldy;
    p.end = end;
    return go("gg_glu", rows, n, [&](LaunchInfo* li) {
        return launch_glu(p, (int)c_dtype, (int)y_dtype, (hipStream_t)stream, li);
    });
}

size_t gg_gemm_mx4_workspace_size(void) { return round256(kWsHeader); }

gg_status gg_gemm_mx4(const uint8_t* a_fp4, const uint8_t* sfa, int64_t m_rows, int32_t k, const uint8_t* b_fp4,
                      const uint8_t* sfb, const int64_t* b_ptrs, const int64_t* sfb_ptrs, int32_t n,
                      const int32_t* offsets, int32_t L, const float* alpha, const float* bias, void* d,
                      gg_dtype d_dtype, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    if (!is_out_dtype(d_dtype))
        return fail(GG_ERR_DTYPE, "d_dtype must be GG_BF16, GG_F16 or GG_F32");
    if (L < 1 || L > 1024)
        return fail(GG_ERR_SHAPE, "L must be in 1..1024 (got %d)", L);
    if (m_rows < 0 || m_rows > INT32_MAX)
        return fail(GG_ERR_SHAPE, "m_rows must be in 0..2^31-1");
    if (k < 128 || k % 128 != 0 || n < 32 || n % 32 != 0)
        return fail(GG_ERR_SHAPE, "k must be a positive multiple of 128, n of 32 (got %d, %d)", k, n);
    if (k > kMaxK || n > kMaxK)
        return fail(GG_ERR_UNSUPPORTED, "k and n are limited to 2^21");
    const bool dense = b_fp4 || sfb, ptrs = b_ptrs || sfb_ptrs;
    if (dense == ptrs)
        return fail(GG_ERR_MODE, "give exactly one of (b_fp4, sfb) and (b_ptrs, sfb_ptrs)");
    if ((dense && (!b_fp4 || !sfb)) || (ptrs && (!b_ptrs || !sfb_ptrs)))
        return fail(GG_ERR_NULL, "weights need both codes and scales");
    if (!offsets || ((!a_fp4 || !sfa || !d) && m_rows > 0))
        return fail(GG_ERR_NULL, "a_fp4, sfa, offsets and d must be non-NULL");
    if (!aligned16(a_fp4) || !aligned16(b_fp4) || !aligned16(d))
        return fail(GG_ERR_ALIGN, "a_fp4, b_fp4 and d must be 16-byte aligned");
    if (off(sfa, 4) || off(sfb, 4) || off(alpha, 4) || off(bias, 4) || off(offsets, 4))
        return fail(GG_ERR_ALIGN, "sfa, sfb, offsets, alpha and bias must be 4-byte aligned");
    if (off(b_ptrs, 8) || off(sfb_ptrs, 8))
        return fail(GG_ERR_ALIGN, "b_ptrs and sfb_ptrs must be 8-byte aligned");
    if (flags)
        return fail(GG_ERR_MODE, "unsupported flags 0x%x for gg_gemm_mx4", flags);
    gg_status st = check_workspace(workspace, workspace_bytes, gg_gemm_mx4_workspace_size());
    if (st != GG_OK)
        return st;
    GemmMx4Args p = {};
    p.a = a_fp4;
    p.sfa = sfa;
    p.m_rows = m_rows;
    p.K = k;
    p.N = n;
    p.L = L;
    p.b_dense = b_fp4;
    p.sfb_dense = sfb;
    p.b_ptrs = b_ptrs;
    p.sfb_ptrs = sfb_ptrs;
    p.ends = offsets;
    p.alpha = alpha;
    p.bias = bias;
    p.d = d;
    p.d_dtype = d_dtype;
    p.ws = (int32_t*)workspace;
    if (gemm_mx4_blocks(p) > kMaxGemmBlocks)
        return fail(GG_ERR_UNSUPPORTED, "m_rows x n has more tiles than one launch holds");
    return go("gg_gemm_mx4", m_rows, n,
              [&](LaunchInfo* li) { return launch_gemm_mx4(p, (hipStream_t)stream, li); });
}

size_t gg_moe_few_workspace_size(int32_t tokens, int32_t top_k, int32_t hidden, int32_t inner) {
    if (tokens < 0 || tokens > kFewTokens || top_k < 1 || top_k > kFewTopK || hidden < 32 || hidden > kFewWidth ||
        inner < 32 || inner > kFewWidth)
        return 0;
    return round256(few_workspace(tokens, top_k, hidden, inner));
}

gg_status gg_moe_few(const void* x, int64_t ldx, int32_t tokens, int32_t hidden, const int32_t* ids,
                     const float* prob, int32_t top_k, int32_t num_experts, const void* w1, const uint8_t* sf1,
                     const float* bias1, const void* w2, const uint8_t* sf2, const float* bias2, gg_dtype w_dtype,
                     int32_t inner, void* y, gg_dtype y_dtype, int64_t ldy, gg_act act, float geglu_alpha,
                     float clamp_min, float clamp_max, float linear_offset, float situ_beta1, float situ_beta2,
                     uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
    if (w_dtype != GG_BF16 && w_dtype != GG_MXFP4)
        return fail(GG_ERR_DTYPE, "w_dtype must be GG_BF16 or GG_MXFP4");
    if (!is_out_dtype(y_dtype))
        return fail(GG_ERR_DTYPE, "y_dtype must be GG_BF16, GG_F16 or GG_F32");
    if (tokens < 0 || top_k < 1 || num_experts < 1 || num_experts > 1024)
        return fail(GG_ERR_SHAPE, "tokens must be >= 0, top_k >= 1 and num_experts in 1..1024");
    if (hidden < 32 || hidden % 32 != 0 || inner < 32 || inner % 32 != 0)
        return fail(GG_ERR_SHAPE, "hidden and inner must be positive multiples of 32 (got %d, %d)", hidden, inner);
    if (tokens > kFewTokens || top_k > kFewTopK || hidden > kFewWidth || inner > kFewWidth)
        return fail(GG_ERR_UNSUPPORTED, "tokens is limited to 64, top_k to 32, hidden and inner to 2^16");
    if (ldx < hidden || ldx % 8 != 0 || ldx > (1 << 23) || ldy < hidden || ldy > INT32_MAX)
        return fail(GG_ERR_LAYOUT, "ldx must be a multiple of 8 in hidden .. 2^23, ldy in hidden .. 2^31-1");
    const bool mx4 = w_dtype == GG_MXFP4;
    if (((!x || !ids || !prob || !y) && tokens > 0) || !w1 || !w2 || (mx4 && (!sf1 || !sf2)))
        return fail(GG_ERR_NULL, "x, ids, prob, w1, w2, y (and the scales of MXFP4) must be non-NULL");
    if (!mx4 && (sf1 || sf2))
        return fail(GG_ERR_MODE, "bf16 weights take no scales");
    if (!aligned16(x) || !aligned16(w1) || !aligned16(w2))
        return fail(GG_ERR_ALIGN, "x, w1 and w2 must be 16-byte aligned");
    if (off(ids, 4) || off(prob, 4) || off(bias1, 4) || off(bias2, 4) || off(y, size_of(y_dtype)))
        return fail(GG_ERR_ALIGN, "every array must be aligned to its element");
    FewArgs p = {};
    gg_status st = check_act(act, geglu_alpha, clamp_min, clamp_max, linear_offset, situ_beta1, situ_beta2, flags,
                             "gg_moe_few", &p.act);
    if (st == GG_OK)
        st = check_workspace(workspace, workspace_bytes, gg_moe_few_workspace_size(tokens, top_k, hidden, inner));
    if (st != GG_OK)
        return st;
    p.x = x;
    p.ldx = ldx;
    p.ldy = ldy;
    p.T = tokens;
    p.H = hidden;
    p.I = inner;
    p.E = num_experts;
    p.k = top_k;
    p.ids = ids;
    p.prob = prob;
    p.w1 = w1;
    p.sf1 = sf1;
    p.bias1 = bias1;
    p.w2 = w2;
    p.sf2 = sf2;
    p.bias2 = bias2;
    p.y = y;
    p.y_dtype = y_dtype;
    p.mx4 = mx4;
    p.ws = (char*)workspace;
    return go("gg_moe_few", tokens, hidden,
              [&](LaunchInfo* li) { return launch_few(p, (hipStream_t)stream, li); });
}

}  // extern "C"
