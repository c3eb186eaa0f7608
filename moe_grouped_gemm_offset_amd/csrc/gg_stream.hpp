// gg_stream.hpp -- what the kernels share that stream weights from memory into
// the operand registers of the matrix instructions (gg_moe_few.hip, the thin
// kernel of gg_gemm_mx4.hip).
#pragma once
#include "gg_lane.hpp"
#include "gg_tile.hpp"

namespace gg {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 buf16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// lo, of rows 0 .. 7 (pieces 0 .. 3 in lanes 0 .. 7 of every 16, 4 .. 7 in lanes
// 8 .. 15), and hi, of rows 8 .. 15: the pieces of the lane's own row, of the
// first and of the second half of the line.  (New values, so that loads into
// lo and hi can follow at once: tied to the old ones they would be loaded
// elsewhere, awaited and moved.)
__device__ __forceinline__ void own_rows(bool low, u32x4 lo, u32x4 hi, u32x4 (&out)[2]) {
    auto far = [](uint32_t v) { return lane_dpp<0x128>(v); };    // lane ^ 8
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t a = far(lo[i]), b = far(hi[i]);           // (in every lane)
        out[0][i] = low ? lo[i] : b;
        out[1][i] = low ? a : hi[i];
    }
}

// The value that lanes 16 j .. 16 j + 15 hold, in every 16 lanes.
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&out)[4]) {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    out[0] = a[0], out[1] = a[1], out[2] = b[0], out[3] = b[1];
}

}  // namespace gg
