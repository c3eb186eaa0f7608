// gg_mx4.hip -- rows to MXFP4 and back (gg_mx4_quant, gg_mx4_dequant).
//
// Four lanes hold a block of 32 values, eight each.  The largest magnitude is
// found on the bit patterns (ordered like the magnitudes, with infinities and
// NaNs on top), so the scale is exact: with the largest = (1 + f) 2^E and
// 6 = 1.5 * 2^2, the smallest e with 6 * 2^e >= largest is E - 2, or E - 1
// where f > 1/2.  The conversion instruction divides by 2^e, rounds to nearest
// even and packs; the division is exact, so this is the only rounding.
//
// Bound by memory: 65536 rows of 4096 bf16 values, 680 MB, to MXFP4 in 113 us (6.0
// TB/s), back in 97 (7.0, the codes partly from the last-level cache).
#include <type_traits>

#include "gg_act.hpp"

namespace gg {

namespace {

typedef uint32_t Word __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The largest magnitude of eight elements as fp32 bits (of 16-bit types two at a
// time: their patterns are ordered alike).
template <int DT>
__device__ __forceinline__ uint32_t top_of(const Eight<DT>& x) {
    if constexpr (DT == GG_F32) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t a = __builtin_bit_cast(uint32_t, x.get(i)) & 0x7FFFFFFFu;
            top = a > top ? a : top;
        }
        return top;
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        auto abs2 = [&](int i) { return __builtin_bit_cast(u16x2, (uint32_t)x.v[0].raw[i] & 0x7FFF7FFFu); };
        const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(abs2(0), abs2(1)),
                                                  __builtin_elementwise_max(abs2(2), abs2(3)));
        const uint16_t top = m[0] > m[1] ? m[0] : m[1];
        return __builtin_bit_cast(uint32_t, to_f32<DT>(top));
    }
}

// Eight elements over 2^e, scale = 2^e, as codes: rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t codes_of(const Eight<DT>& x, float scale) {
    uint32_t c = 0;
    if constexpr (DT == GG_F32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.get(0), x.get(1), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.get(2), x.get(3), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.get(4), x.get(5), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.get(6), x.get(7), scale, 3);
    } else if constexpr (DT == GG_BF16) {
        typedef __bf16 Two __attribute__((ext_vector_type(2)));
        auto two = [&](int i) { return __builtin_bit_cast(Two, (uint32_t)x.v[0].raw[i]); };
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(0), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(1), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(2), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(3), scale, 3);
    } else {
        typedef _Float16 Two __attribute__((ext_vector_type(2)));
        auto two = [&](int i) { return __builtin_bit_cast(Two, (uint32_t)x.v[0].raw[i]); };
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, two(0), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, two(1), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, two(2), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, two(3), scale, 3);
    }
    return c;
}

template <int DT, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) quant_kernel(QuantArgs p, Eights e) {
    typedef typename Elem<DT>::T T;
    const T* const x = (const T*)p.x;
    for_eights<FLAT>(e, p.ld, p.end, [&](const Run& run) {
        Eight<DT> in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            in[u].load(x + run.at[u]);
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t top = group_all<4>(top_of<DT>(in[u]), OpMaxU());
            const bool odd = top >= 0x7F800000u;         // an infinity or a NaN
            // the exponent field, one more where f > 1/2, less 2
            const uint32_t up = (top + 0x3FFFFFu) >> 23;
            const uint32_t s = odd ? 255u : (up > 2u ? up - 2u : 0u);
            const uint32_t c = codes_of<DT>(in[u], __builtin_bit_cast(float, s << 23));
            if (run.live[u]) {
                *(Word*)(p.codes + run.v[u] * 4) = odd ? 0u : c;
                if ((threadIdx.x & 3) == 0)
                    p.scales[run.v[u] >> 2] = (uint8_t)s;
            }
        }
    });
}

template <int DT, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) dequant_kernel(QuantArgs p, Eights e) {
    typedef typename Elem<DT>::T T;
    T* const out = (T*)p.x;
    for_eights<FLAT>(e, p.ld, p.end, [&](const Run& run) {
        uint32_t c[kUnroll], s[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            c[u] = *(const Word*)(p.codes + run.v[u] * 4);
            s[u] = p.scales[run.v[u] >> 2];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const float scale = __builtin_bit_cast(float, s[u] << 23);
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 1);
            const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 2);
            const f32x2 g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, 3);
            const float f[8] = {a[0], a[1], b[0], b[1], d[0], d[1], g[0], g[1]};
            Eight<DT> o;
            o.set(f);
            if (run.live[u])
                o.store(out + run.at[u]);
        }
    });
}

template <class Launch>
hipError_t by_dtype(const char* name, const QuantArgs& p, int dtype, LaunchInfo* info, Launch launch) {
    const Eights e = eights_of(p.rows, p.width);
    const unsigned grid = eights_grid(e);
    if (grid == 0)
        return hipSuccess;
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "%s<%s>", name, dtype_name(dtype));
        info->tm = kRowStep;
        info->tn = 8;
        info->waves = kRowThreads / 64;
        info->grid = grid;
    }
    auto by_pitch = [&](auto DT) {
        if (p.ld == p.width)
            launch(DT, std::true_type(), e, grid);
        else
            launch(DT, std::false_type(), e, grid);
    };
    if (dtype == GG_BF16)
        by_pitch(std::integral_constant<int, GG_BF16>());
    else if (dtype == GG_F16)
        by_pitch(std::integral_constant<int, GG_F16>());
    else
        by_pitch(std::integral_constant<int, GG_F32>());
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant(const QuantArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    return by_dtype("quant_kernel", p, dtype, info, [&](auto DT, auto FLAT, const Eights& e, unsigned grid) {
        hipLaunchKernelGGL((quant_kernel<decltype(DT)::value, decltype(FLAT)::value>), dim3(grid), dim3(kRowThreads), 0, s,
                           p, e);
    });
}

hipError_t launch_dequant(const QuantArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    return by_dtype("dequant_kernel", p, dtype, info, [&](auto DT, auto FLAT, const Eights& e, unsigned grid) {
        hipLaunchKernelGGL((dequant_kernel<decltype(DT)::value, decltype(FLAT)::value>), dim3(grid), dim3(kRowThreads), 0, s,
                           p, e);
    });
}

}  // namespace gg
