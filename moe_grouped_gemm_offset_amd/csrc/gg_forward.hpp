// gg_forward.hpp -- parameter blocks and launchers of the experts' forward pass
// (MXFP4 quantisation, gated activation, grouped MXFP4 product, a layer for a
// few tokens), shared between gg_api_forward.cpp and the kernel translation
// units.  Not part of the ABI.
#pragma once
#include "gg_internal.hpp"

namespace gg {

struct ActArgs {
    int act;                  // gg_act
    int gate_first;
    float alpha, lo, hi, offset;          // GG_DGEGLU
    float b1, b2;                         // GG_DSITUGLU
};

struct QuantArgs {
    void* x;                  // (rows, width), row pitch ld: source, or the values
    int64_t ld, rows;
    int width;
    uint8_t* codes;
    uint8_t* scales;
    const int32_t* end;       // [1] or null
};

struct GluArgs {
    const void* c;            // (rows, 2n), row pitch ldc
    int64_t ldc, rows;
    int n;
    const float* prob;        // [rows] or null
    void* y;                  // (rows, n), row pitch ldy
    int64_t ldy;
    ActArgs act;
    const int32_t* end;       // [1] or null
};

struct GemmMx4Args {
    const uint8_t* a;
    const uint8_t* sfa;
    int64_t m_rows;
    int K, N, L;
    const uint8_t* b_dense;
    const uint8_t* sfb_dense;
    const int64_t* b_ptrs;
    const int64_t* sfb_ptrs;
    const int32_t* ends;      // [L]
    const float* alpha;       // [L] or null
    const float* bias;        // (L, N) or null
    void* d;                  // (m_rows, N)
    int d_dtype;
    int32_t* ws;
};

struct FewArgs {
    const void* x;            // (T, H) bf16, row pitch ldx
    int64_t ldx, ldy;
    int T, H, I, E, k;
    const int32_t* ids;       // (T, k)
    const float* prob;        // (T, k)
    const void* w1;           // bf16, or MXFP4 codes with sf1
    const uint8_t* sf1;
    const float* bias1;       // (E, 2I) or null
    const void* w2;
    const uint8_t* sf2;
    const float* bias2;       // (E, H) or null
    void* y;                  // (T, H), row pitch ldy
    int y_dtype, mx4;
    int parts;                // bf16 values that hold an h
    uint32_t k_magic;         // i * k_magic >> 16 = i / k
    ActArgs act;
    char* ws;
};

// Bytes of workspace that a gg_moe_few call uses.
size_t few_workspace(int64_t T, int64_t k, int64_t H, int64_t I);
// Blocks that a gg_gemm_mx4 call launches, and the most that one launch may (of 256
// threads; a launch holds 2^32 threads).
constexpr int64_t kMaxGemmBlocks = 1 << 23;
int64_t gemm_mx4_blocks(const GemmMx4Args& p);
hipError_t launch_quant(const QuantArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_dequant(const QuantArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_glu(const GluArgs& p, int c_dtype, int y_dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_gemm_mx4(const GemmMx4Args& p, hipStream_t s, LaunchInfo* info);
// (info: of both passes, two)
hipError_t launch_few(const FewArgs& p, hipStream_t s, LaunchInfo* info);

}  // namespace gg
