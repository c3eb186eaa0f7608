// gg_act.hpp -- the gated activations, forward, in fp32 (their backward is
// gg_dglu_epi.hpp), and the row-wise walk that gg_glu and the quantiser share.
#pragma once
#include "gg_forward.hpp"
#include "gg_lane.hpp"

namespace gg {

// 1 / (1 + exp(-x)) from the exponential of -|x|, which neither overflows nor
// cancels; good to 6 units of 2^-24 down to results of 2^-126.
__device__ __forceinline__ float sigmoid_full(float x) {
    const float e = exp_below<true>(-fabsf(x)), d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.0f), r, r);
    return __builtin_signbitf(x) ? e * r : r;
}

// The activation of a gate and an input (without prob).  (minimum and maximum
// keep a NaN.  SiTU-GLU is bound by its arithmetic: 49663 rows of 2336 outputs, 226 us
// for SwiGLU's 118.  A tanh of an exponential and a polynomial without branches took
// 300: most arguments are small, where the library's branch is short.)
template <int ACT>
__device__ __forceinline__ float act_forward(float g, float u, const ActArgs& a) {
    if constexpr (ACT == GG_DSWIGLU) {
        return g * sigmoid_full(g) * u;
    } else if constexpr (ACT == GG_DGEGLU) {
        const float gc = __builtin_elementwise_minimum(g, a.hi);
        const float uc = __builtin_elementwise_maximum(__builtin_elementwise_minimum(u, a.hi), a.lo);
        return gc * sigmoid_full(a.alpha * gc) * (uc + a.offset);
    } else {
        return a.b1 * tanhf(g / a.b1) * sigmoid_full(g) * (a.b2 * tanhf(u / a.b2));
    }
}

// Calls f(std::integral_constant<int, act>).
template <class F>
void for_act(int act, F f) {
    if (act == GG_DSWIGLU)
        f(std::integral_constant<int, GG_DSWIGLU>());
    else if (act == GG_DGEGLU)
        f(std::integral_constant<int, GG_DGEGLU>());
    else
        f(std::integral_constant<int, GG_DSITUGLU>());
}

// ---- rows as a run of eights -------------------------------------------------
// Kernels over (rows, width) elements take eight elements of a row a lane (width
// is a multiple of 32), kUnroll of them at a time (65536 rows of 4096 in bf16, one, two
// and four at a time: to MXFP4 117, 113 and 113 us, back 114, 97 and 100; the
// activation to 2048 columns 130, 132 and 138), the block's threads side by side: eight v of the
// matrix is row v / per_row.  The division goes by the block's first eight (a 64-bit
// reciprocal, exact for v * per_row < 2^64) and by the distance from it within the
// row.
constexpr int kRowThreads = 256;
constexpr int kUnroll = 2;
constexpr int kRowStep = kRowThreads * kUnroll;

struct Eights {
    int64_t rows;
    uint32_t per_row;         // eights of a row, 4 .. 2^17
    uint32_t magic;           // floor(2^32 / per_row) + 1
    uint64_t magic64;         // floor(2^64 / per_row) + 1
};

inline Eights eights_of(int64_t rows, int width) {
    Eights e;
    e.rows = rows;
    e.per_row = (uint32_t)(width / 8);
    e.magic = (uint32_t)((1ull << 32) / e.per_row + 1);
    e.magic64 = (uint64_t)(((unsigned __int128)1 << 64) / e.per_row + 1);
    return e;
}

// Blocks for them: a block goes on to its next run past 2^22 blocks (launches
// hold 2^32 threads).
inline unsigned eights_grid(const Eights& e) {
    const int64_t n = (e.rows * e.per_row + kRowStep - 1) / kRowStep;
    return (unsigned)(n < (1 << 22) ? n : 1 << 22);
}

// The thread's eights of a run (clamped to the matrix's last where !live): row and
// first column, the eight's own index, and the first element's in rows of pitch
// ld.
struct Run {
    int64_t row[kUnroll], v[kUnroll], at[kUnroll];
    uint32_t col[kUnroll];
    bool live[kUnroll];
};

// Calls f(run) for every run of the block.  FLAT: rows follow each other without a
// gap (ld is the width), and f wants neither rows nor columns.
template <bool FLAT, class F>
__device__ __forceinline__ void for_eights(const Eights& e, int64_t ld, const int32_t* end, F f) {
    int64_t rows = e.rows;
    if (end) {
        const int64_t n = *end;
        rows = n < 0 ? 0 : (n < rows ? n : rows);
    }
    const int64_t total = rows * e.per_row;
    for (int64_t base = (int64_t)blockIdx.x * kRowStep; base < total; base += (int64_t)gridDim.x * kRowStep) {
        const uint32_t left = (uint32_t)(total - base < kRowStep ? total - base : kRowStep) - 1;
        int64_t row0 = 0;
        uint32_t at0 = 0;
        if constexpr (!FLAT) {
            row0 = (int64_t)__umul64hi((uint64_t)base, e.magic64);
            at0 = (uint32_t)(base - row0 * e.per_row);
        }
        Run r;
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t i = threadIdx.x + u * kRowThreads;
            r.live[u] = i <= left;
            const uint32_t j = r.live[u] ? i : left;
            r.v[u] = base + j;
            if constexpr (FLAT) {
                r.at[u] = r.v[u] * 8;
            } else {
                // (at < 2 per_row from kRowStep on, at < 2 kRowStep below)
                const uint32_t at = at0 + j;
                const uint32_t over = e.per_row >= kRowStep ? (at >= e.per_row ? 1u : 0u) : __umulhi(at, e.magic);
                r.row[u] = row0 + over;
                r.col[u] = (at - over * e.per_row) * 8;
                r.at[u] = r.row[u] * ld + r.col[u];
            }
        }
        f(r);
    }
}

// Eight elements, loaded and stored as 16-byte vectors at element alignment.
template <int DT>
struct Eight {
    static constexpr int kVec = 16 / (int)sizeof(typename Elem<DT>::T), kN = 8 / kVec;
    Vec<DT, kVec> v[kN];
    __device__ __forceinline__ void load(const typename Elem<DT>::T* p) {
#pragma unroll
        for (int i = 0; i < kN; i++)
            v[i].template load<true>(p + i * kVec);
    }
    __device__ __forceinline__ void store(typename Elem<DT>::T* p) const {
#pragma unroll
        for (int i = 0; i < kN; i++)
            v[i].template store<true>(p + i * kVec);
    }
    __device__ __forceinline__ float get(int i) const { return v[i / kVec].get(i % kVec); }
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < kN; i++) {
            float g[kVec];
#pragma unroll
            for (int j = 0; j < kVec; j++)
                g[j] = f[i * kVec + j];
            v[i].set(g);
        }
    }
};

}  // namespace gg
