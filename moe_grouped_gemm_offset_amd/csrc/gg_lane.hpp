// gg_lane.hpp -- device helpers of the row-wise kernels (routing, dispatch,
// clipping): element conversions, vector access at element alignment, and
// reductions over groups of lanes of a wave.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_moe.h"

namespace gg {

// ---- elements ------------------------------------------------------------

template <int DT>
struct Elem {                                        // GG_BF16 and GG_F16
    typedef uint16_t T;
};
template <>
struct Elem<GG_F32> {
    typedef uint32_t T;
};

template <int DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::T u) {
    if constexpr (DT == GG_BF16)
        return __builtin_bit_cast(float, (uint32_t)u << 16);
    else if constexpr (DT == GG_F16)
        return (float)__builtin_bit_cast(_Float16, u);
    else
        return __builtin_bit_cast(float, u);
}

// fp32 to the element, to nearest even (the only rounding these kernels make)
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T from_f32(float f) {
    if constexpr (DT == GG_BF16)
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    else if constexpr (DT == GG_F16)
        return __builtin_bit_cast(uint16_t, (_Float16)f);
    else
        return __builtin_bit_cast(uint32_t, f);
}

// ---- vectors ---------------------------------------------------------------
// 16 bytes of elements in one access that needs no more than the element's own
// alignment: rows of an odd width start anywhere, and global memory takes
// unaligned vectors.

typedef uint32_t Raw16 __attribute__((ext_vector_type(4), aligned(1)));

template <int DT, int N>
struct Vec {
    static_assert(N * (int)sizeof(typename Elem<DT>::T) == 16, "16 bytes");
    typedef Raw16 T;
    T raw;

    // NT: values that are not used again soon pass the caches by
    template <bool NT = false>
    __device__ __forceinline__ void load(const typename Elem<DT>::T* p) {
        raw = NT ? __builtin_nontemporal_load((const T*)p) : *(const T*)p;
    }
    template <bool NT = false>
    __device__ __forceinline__ void store(typename Elem<DT>::T* p) const {
        if constexpr (NT)
            __builtin_nontemporal_store(raw, (T*)p);
        else
            *(T*)p = raw;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (DT == GG_F32)
            return __builtin_bit_cast(float, (uint32_t)raw[i]);
        else
            return to_f32<DT>((uint16_t)(raw[i >> 1] >> (16 * (i & 1))));
    }
    // Moves element d + i to i (0 <= d < N; what comes in at the top is
    // unspecified).  (Words by name: of an array of them the compiler may make
    // memory in LDS, indexed by d.)
    __device__ __forceinline__ void drop(int d) {
        const int words = DT == GG_F32 ? d : d >> 1;
        const bool two = words & 2, one = words & 1;
        const uint32_t a = two ? raw[2] : raw[0], b = two ? raw[3] : raw[1], c = raw[2], e = raw[3];
        const uint32_t w0 = one ? b : a, w1 = one ? c : b, w2 = one ? e : c;
        if constexpr (DT == GG_F32) {
            raw = T{w0, w1, w2, e};
        } else {
            const uint32_t sh = 16 * (d & 1);
            raw = T{__builtin_amdgcn_alignbit(w1, w0, sh), __builtin_amdgcn_alignbit(w2, w1, sh),
                    __builtin_amdgcn_alignbit(e, w2, sh), __builtin_amdgcn_alignbit(e, e, sh)};
        }
    }
    __device__ __forceinline__ void set(const float (&f)[N]) {
        if constexpr (DT == GG_F32) {
#pragma unroll
            for (int i = 0; i < N; i++)
                raw[i] = __builtin_bit_cast(uint32_t, f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2)
                raw[i >> 1] = (uint32_t)from_f32<DT>(f[i]) | (uint32_t)from_f32<DT>(f[i + 1]) << 16;
        }
    }
};

// ---- lanes -----------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t lane_dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// Combines v over each aligned group of W lanes (4 <= W <= 64, a power of
// two) with a commutative op; every lane gets the result, the same bits in
// each.  Whole waves only: every lane must be active.
template <int W, class T, class Op>
__device__ __forceinline__ T group_all(T v, Op op) {
    static_assert(sizeof(T) == 4 && W >= 4 && W <= 64, "32-bit values, groups of 4 to 64 lanes");
    auto u = [](T x) { return __builtin_bit_cast(uint32_t, x); };
    auto t = [](uint32_t x) { return __builtin_bit_cast(T, x); };
    v = op(v, t(lane_dpp<0xB1>(u(v))));              // lane ^ 1
    v = op(v, t(lane_dpp<0x4E>(u(v))));              // lane ^ 2
    if constexpr (W >= 8)
        v = op(v, t(lane_dpp<0x141>(u(v))));         // 7 - lane within eight
    if constexpr (W >= 16)
        v = op(v, t(lane_dpp<0x140>(u(v))));         // 15 - lane within sixteen
    if constexpr (W >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
        v = op(t(r[0]), t(r[1]));
    }
    if constexpr (W >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
        v = op(t(r[0]), t(r[1]));
    }
    return v;
}

// Orders the LDS accesses of a wave's lanes around it (the hardware keeps a
// wave's LDS accesses in order; this keeps the compiler from forwarding a
// lane's own value past another lane's write).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct OpMaxU {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct OpMaxF {
    // (NaN if either is; fmaxf would first quiet both, an instruction each)
    __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_elementwise_maximum(a, b); }
};
struct OpAddF {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Lowest lane of this lane's group of W for which the predicate holds, as an
// index within the group (-1 if there is none).
template <int W>
__device__ __forceinline__ int group_first(bool pred, int lane) {
    const uint64_t m = __ballot(pred);
    if constexpr (W == 64)
        return __ffsll((unsigned long long)m) - 1;
    else
        return __ffs((int)((uint32_t)(m >> (lane & ~(W - 1))) & (uint32_t)((1ull << W) - 1))) - 1;
}

// Sum of v over the wave, in every lane (the same tree at every call).
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int h = 32; h > 0; h >>= 1)
        v += __shfl_xor(v, h);
    return v;
}

// Sum of v over a block of THREADS, in every thread, through tmp[THREADS /
// 64] in LDS; the same order at every call.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double* tmp) {
    v = wave_sum(v);
    __syncthreads();                                 // tmp may still be read
    if ((threadIdx.x & 63) == 0)
        tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = tmp[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; w++)
        s += tmp[w];
    return s;
}

}  // namespace gg
