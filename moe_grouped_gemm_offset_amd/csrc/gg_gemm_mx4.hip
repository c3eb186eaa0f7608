// gg_gemm_mx4.hip -- the grouped product of MXFP4 rows and weights
// (gg_gemm_mx4): d = alpha_g deq(a) deq(b_g)^T + bias_g over ragged groups.
//
// Two kernels, chosen by the rows that a group has on average:
//  * gemm_kernel, tiles of 256 x 256 on the two-buffer main loop of the 8-bit
//    kernels.  v_mfma_scale_f32_32x32x64_f8f6f4 takes 4-bit operands at twice
//    the 8-bit rate: a lane supplies one block of 32 values, 16 bytes, so a
//    64-byte stage of a row is 128 values in two steps, and a load unit 256.
//  * thin_kernel, for groups of few rows, where reading the weights is what
//    costs: blocks of 64 weight rows whose waves split the reduction axis, the
//    weights going from memory into the operand registers (as in
//    gg_moe_few.hip).
// Groups have any number of rows: every block counts the tiles of the groups
// (a scan over the ends by each of its waves) and finds its own.
#include <type_traits>

#include "gg_forward.hpp"
#include "gg_lane.hpp"
#include "gg_tile.hpp"

namespace gg {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));

// ---- tiles of ragged groups --------------------------------------------------

struct TileAt {
    int g;                    // group, -1: none
    int m0, rows;             // first row and rows of the tile (at most TM)
    int nt;                   // tile of columns
};

// Tile of block `q` where groups are cut into tiles of TM rows and tiles_n
// columns.  Ends are taken as a running maximum within 0 .. m_rows, so ranges
// are disjoint and in bounds whatever the array holds.  Lane l of every wave
// has groups l * per .. ; per is 1 up to 64 groups.  Blocks of one XCD (every
// eighth) get neighbouring tiles, in bands of 4 tiles of rows within a group.
template <int TM>
__device__ __forceinline__ TileAt tile_at(const int32_t* ends, int L, int m_rows, int tiles_n, int q) {
    const int lane = threadIdx.x & 63, per = (L + 63) >> 6, g0 = lane * per;
    auto end_of = [&](int g) { return min(max(ends[g], 0), m_rows); };
    int top = 0;
    for (int i = 0; i < per; i++)
        if (g0 + i < L)
            top = max(top, end_of(g0 + i));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int below = __shfl_up(top, d);
        top = lane >= d ? max(top, below) : top;
    }
    int start = __shfl_up(top, 1);                     // where the lane's first group begins
    start = lane ? start : 0;
    int tiles = 0, at = start;
    for (int i = 0; i < per; i++)
        if (g0 + i < L) {
            const int end = max(at, end_of(g0 + i));
            tiles += (end - at + TM - 1) / TM;
            at = end;
        }
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int below = __shfl_up(upto, d);
        upto += lane >= d ? below : 0;
    }
    TileAt t;
    t.g = -1;
    const int64_t P = (int64_t)__builtin_amdgcn_readlane(upto, 63) * tiles_n;
    if (q >= P)
        return t;
    const int each = (int)(P >> 3), more = (int)(P & 7), x = q & 7;
    int j = x * each + min(x, more) + (q >> 3);        // the q-th block's tile
    int mt = j / tiles_n;
    const int owner = __ffsll((unsigned long long)__ballot(upto > mt)) - 1;
    int before = __builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(tiles, owner);
    int begin = __builtin_amdgcn_readlane(start, owner), end = begin, n = 0;
    int g = owner * per;
    for (; g < L; g++) {
        end = max(begin, uniform(end_of(g)));
        n = (end - begin + TM - 1) / TM;
        if (mt < before + n)
            break;
        before += n;
        begin = end;
    }
    j -= before * tiles_n;
    const int band = j / (4 * tiles_n), high = min(4, n - 4 * band);
    j -= band * 4 * tiles_n;
    mt = 4 * band + j % high;
    t.g = g < L ? g : -1;
    t.nt = j / high;
    t.m0 = begin + mt * TM;
    t.rows = min(TM, end - t.m0);
    return t;
}

// Blocks that the tiles cannot exceed (every group may have a part of a tile).
inline int64_t tile_bound(const GemmMx4Args& p, int tm, int tn) {
    const int64_t groups = p.m_rows < p.L ? p.m_rows : p.L;
    return (p.m_rows / tm + groups) * ((p.N + tn - 1) / tn);
}

// The error word, by the first wave of block 0.
__device__ __forceinline__ void check_ends(const GemmMx4Args& p) {
    if (blockIdx.x != 0 || threadIdx.x >= 64)
        return;
    bool low = false, high = false;
    for (int g = threadIdx.x; g < p.L; g += 64) {
        low |= p.ends[g] < (g ? p.ends[g - 1] : 0);
        high |= p.ends[g] > p.m_rows;
    }
    const int code = (__ballot(low) ? GG_DEVERR_DECREASING : 0) | (__ballot(high) ? GG_DEVERR_LAST : 0);
    if (threadIdx.x == 0)
        p.ws[0] = code;
}

// Codes and scales of group g's weights from row n0 on.
__device__ __forceinline__ const char* weights_at(const GemmMx4Args& p, int g, int n0) {
    const char* b = p.b_dense ? (const char*)p.b_dense + (int64_t)g * p.N * (p.K / 2) : (const char*)p.b_ptrs[g];
    return b + (int64_t)n0 * (p.K / 2);
}
__device__ __forceinline__ const char* scales_at(const GemmMx4Args& p, int g, int n0) {
    const char* s = p.sfb_dense ? (const char*)p.sfb_dense + (int64_t)g * p.N * (p.K / 32) : (const char*)p.sfb_ptrs[g];
    return s + (int64_t)n0 * (p.K / 32);
}

// ---- the tiled kernel --------------------------------------------------------

using GemmCfg = Cfg<256, 256, 2, 2>;

// Scales of 4 stages (16 bytes of every tile row, 2 load units) at a time, in
// two alternating buffers behind the unit buffers: row r of A in slot r, of B
// in slot TM + r.  A wave's load moves the 16 bytes of 64 rows; units 2g + 1
// and 2g + 2 carry the A and the B half of group g + 1.  Then 16 bytes of
// zeros, the scales of the stage past an odd number of them (the next row's
// bytes, which the loads bring there, may be the scale of NaN).
template <class C>
struct Scales4 {
    static constexpr int kBuf = (C::TM + C::TN) * 16;
    static constexpr int kBase = 2 * C::kUnit, kZero = kBase + 2 * kBuf;
    static constexpr int kSmem = kZero + 16 > C::kLds ? kZero + 16 : C::kLds;
    static_assert(C::TM == 256 && C::TN == 256 && C::kWaves == 4, "a wave's load is 64 rows");
};

template <class C>
struct FragMx4 {
    u32x4 a[2][C::MB], b[2][C::NB];                    // the two steps of a stage
    uint32_t sa[C::MB], sb[C::NB];                     // scale words, as read
};

__device__ __forceinline__ i32x8 low4(u32x4 v) {
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// acc += deq(a) deq(b)^T over K values of rows whose codes are K / 2 bytes
// apart (scales K / 32); rows past rows_valid / cols_valid count as zeros.
// ODD: K is an odd number of stages of 128.
template <class C, bool ODD>
__device__ __forceinline__ void mx4_mainloop(char* smem, const char* a, const char* sfa, const char* b,
                                             const char* sfb, int K, int rows_valid, int cols_valid,
                                             int am0, int bn0, f32x16 (&acc)[C::MB][C::NB]) {
    constexpr int TM = C::TM, TN = C::TN, MB = C::MB, NB = C::NB;
    using S = Scales4<C>;
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, wu = uniform(w);
    const int lr = l & 31, lq = l >> 5;
    const int64_t ld = K / 2;
    const uint32_t KB = K / 32;
    const int nk = K / 128;
    // waves 0 and 1 load A's scales, 2 and 3 B's
    const bool of_a = wu < 2;
    const int valid = of_a ? (rows_valid < TM ? rows_valid : TM) : (cols_valid < TN ? cols_valid : TN);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(uniform_ptr(of_a ? sfa : sfb), (uint32_t)uniform(valid * (int)KB));
    const uint32_t sc_lds = lds_addr(smem) + S::kBase + (of_a ? 0 : TM * 16) + (wu & 1) * 1024;
    const uint32_t sc_off = (uint32_t)(64 * (wu & 1) + l) * KB;
    auto scale_load = [&](int grp, int half) {
        dma16(rs, sc_lds + (grp & 1) * S::kBuf + half * 2048, sc_off + half * 128 * KB + 16 * grp);
    };
    LoadK<C, TM> la;
    LoadK<C, TN> lb;
    la.init(ld, rows_valid);
    lb.init(ld, cols_valid);
    constexpr int kLA = LoadK<C, TM>::kN, kLB = LoadK<C, TN>::kN;
    auto issue = [&](uint32_t st, int u, int i) {
        const int64_t kb = (int64_t)u * 128;
        if (i < kLA)
            la.template issue<ODD>(st, a + kb, ld - kb, i);
        else if (i < kLA + kLB)
            lb.template issue<ODD>(st + TM * kRowBytes, b + kb, ld - kb, i - kLA);
        else                                           // (unit 0: group 0's again)
            scale_load(u > 0 ? (u - 1) / 2 + 1 : 0, u > 0 ? (u - 1) & 1 : 0);
    };
    const uint32_t sh = 8 * lq;
    auto read = [&](const char* st, int kt, FragMx4<C>& f, int g) {
        const bool is_a = g < MB;
        const int r = is_a ? am0 + 32 * g + lr : bn0 + 32 * (g - MB) + lr;
        const char* s = is_a ? st : st + TM * kRowBytes;
        const u32x4 x0 = ld_lds16(s, lds_off(r, 4 * (kt & 1) + lq));
        const u32x4 x1 = ld_lds16(s, lds_off(r, 4 * (kt & 1) + 2 + lq));
        int base = S::kBase + ((kt >> 2) & 1) * S::kBuf + 4 * (kt & 3), at = (is_a ? r : TM + r) * 16;
        if constexpr (ODD) {
            const int keep = kt < nk ? -1 : 0;
            base = kt < nk ? base : S::kZero;
            at &= keep;
        }
        const uint32_t word = *reinterpret_cast<const uint32_t*>(smem + base + at);
        if (is_a) {
            f.a[0][g] = x0;
            f.a[1][g] = x1;
            f.sa[g] = word;
        } else {
            f.b[0][g - MB] = x0;
            f.b[1][g - MB] = x1;
            f.sb[g - MB] = word;
        }
    };
    // Byte 2 s + lq of a row's word is the scale of the block that the lane
    // feeds in step s: shifted by lq, then picked by the instruction.
    auto mma = [&](const FragMx4<C>& f, int m0, int m1) {
#pragma unroll
        for (int m = 0; m < 2 * MB * NB; m++) {
            if (m < m0 || m >= m1)
                continue;
            const int i = (m / NB) % MB, j = m % NB;
            const int sa = (int)(f.sa[i] >> sh), sb = (int)(f.sb[j] >> sh);
            if (m < MB * NB)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    low4(f.a[0][i]), low4(f.b[0][j]), acc[i][j], 4, 4, 0, sa, 0, sb);
            else
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    low4(f.a[1][i]), low4(f.b[1][j]), acc[i][j], 4, 4, 2, sa, 2, sb);
        }
    };
    if (ODD && threadIdx.x == 0)
        *reinterpret_cast<u32x4*>(smem + S::kZero) = u32x4{0};
    FragMx4<C> frag[2];
    scale_load(0, 0);
    scale_load(0, 1);
    pipeline<C, kLA + kLB + 1, 2 * MB * NB, MB + NB>(smem, nk, frag, issue, read, mma);
}

template <int DT, bool ODD, bool BIAS>
__global__ void __launch_bounds__(GemmCfg::kThreads, 1) gemm_kernel(GemmMx4Args p) {
    using C = GemmCfg;
    constexpr int TM = C::TM, TN = C::TN, MB = C::MB, NB = C::NB;
    __shared__ __attribute__((aligned(1024))) char smem[Scales4<C>::kSmem];
    check_ends(p);
    const TileAt t = tile_at<TM>(p.ends, p.L, (int)p.m_rows, (p.N + TN - 1) / TN, blockIdx.x);
    if (t.g < 0)
        return;
    const int g = uniform(t.g), rows = uniform(t.rows), n0 = uniform(t.nt) * TN;
    const int64_t m0 = uniform(t.m0);
    const int cols = p.N - n0;
    const int w = threadIdx.x >> 6, wm = w / C::WN, wn = w % C::WN;
    const int am0 = wm * (TM / C::WM), bn0 = wn * (TN / C::WN);
    f32x16 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; i++)
#pragma unroll
        for (int j = 0; j < NB; j++)
            acc[i][j] = f32x16{0};
    mx4_mainloop<C, ODD>(smem, (const char*)p.a + m0 * (p.K / 2), (const char*)p.sfa + m0 * (p.K / 32),
                         weights_at(p, g, n0), scales_at(p, g, n0), p.K, rows, cols, am0, bn0, acc);
    const float alpha = p.alpha ? p.alpha[g] : 1.0f;
    struct Bias {
        float v[BIAS ? 8 : 1];
    };
    auto load = [&](int, int, int c) {
        Bias b = {};
        if constexpr (BIAS) {
            const int col = n0 + bn0 + c;
            const float* from = p.bias + (int64_t)g * p.N + (col < p.N ? col : 0);
#pragma unroll
            for (int k = 0; k < 8; k++)
                b.v[k] = from[k];
        }
        return b;
    };
    auto store = [&](int, int r, int c, float (&v)[8], const Bias& b) {
        const int row = am0 + r, col = n0 + bn0 + c;
        if (row < rows && col < p.N) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                v[k] = BIAS ? fmaf(alpha, v[k], b.v[k]) : alpha * v[k];
            store8(p.d, DT, (m0 + row) * p.N + col, v);
        }
    };
    for_each_row8<C, BIAS ? 4 : 1, 64, 0, -1, true>(acc, (float*)(smem + w * kEpiWaveBytes), load, store);
}

// ---- the thin kernel ---------------------------------------------------------

constexpr int kThinWaves = 8, kThinThreads = 64 * kThinWaves, kThinCols = 64, kRB = kThinCols / 16;

// NB: blocks of 16 rows of d in a tile.
template <int NB>
__global__ void __launch_bounds__(kThinThreads, NB == 1 ? 4 : 2) thin_kernel(GemmMx4Args p) {
    __shared__ __attribute__((aligned(16))) f32x4 sum[kThinWaves][kRB][64];
    check_ends(p);
    const TileAt t = tile_at<16 * NB>(p.ends, p.L, (int)p.m_rows, (p.N + kThinCols - 1) / kThinCols, blockIdx.x);
    if (t.g < 0)
        return;
    const int g = uniform(t.g), rows = uniform(t.rows), n0 = uniform(t.nt) * kThinCols;
    const int64_t m0 = uniform(t.m0);
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int cols = min(kThinCols, p.N - n0), nb = (rows + 15) >> 4;
    const uint32_t pitch = p.K / 2, spitch = p.K / 32;
    const char* const w = (const char*)uniform_ptr(weights_at(p, g, n0));
    const char* const sw = (const char*)uniform_ptr(scales_at(p, g, n0));
    const char* const x = (const char*)p.a + m0 * pitch;
    const char* const sx = (const char*)p.sfa + m0 * spitch;
    uint32_t wr[kRB], xr[NB];
#pragma unroll
    for (int rb = 0; rb < kRB; rb++)
        wr[rb] = min(16 * rb + r, cols - 1);
#pragma unroll
    for (int b = 0; b < NB; b++)
        xr[b] = min(16 * b + r, rows - 1);
    f32x4 acc[kRB][NB];
#pragma unroll
    for (int rb = 0; rb < kRB; rb++)
#pragma unroll
        for (int b = 0; b < NB; b++)
            acc[rb][b] = f32x4{0};
    // H halves of 128 values from k0 on; a scale word has the bytes of its four
    // blocks, a lane's is byte q
    auto chunk = [&](int k0, auto Hc) {
        constexpr int H = decltype(Hc)::value;
        u32x4 wv[H][kRB], xv[H][NB];
        uint32_t ws[H][kRB], xs[H][NB];
#pragma unroll
        for (int h = 0; h < H; h++)
#pragma unroll
            for (int rb = 0; rb < kRB; rb++)
                wv[h][rb] = *(const u32x4*)(w + wr[rb] * pitch + (uint32_t)(k0 / 2 + 64 * h + 16 * q));
#pragma unroll
        for (int h = 0; h < H; h++)
#pragma unroll
            for (int rb = 0; rb < kRB; rb++)
                ws[h][rb] = *(const uint32_t*)(sw + wr[rb] * spitch + (uint32_t)(k0 / 32 + 4 * h));
#pragma unroll
        for (int b = 0; b < NB; b++)
            if (b < nb) {
#pragma unroll
                for (int h = 0; h < H; h++) {
                    xv[h][b] = *(const u32x4*)(x + xr[b] * pitch + (uint32_t)(k0 / 2 + 64 * h + 16 * q));
                    xs[h][b] = *(const uint32_t*)(sx + xr[b] * spitch + (uint32_t)(k0 / 32 + 4 * h));
                }
            }
#pragma unroll
        for (int h = 0; h < H; h++)
#pragma unroll
            for (int b = 0; b < NB; b++)
                if (b < nb) {
#pragma unroll
                    for (int rb = 0; rb < kRB; rb++)
                        acc[rb][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            low4(wv[h][rb]), low4(xv[h][b]), acc[rb][b], 4, 4, 0, (int)(ws[h][rb] >> (8 * q)),
                            0, (int)(xs[h][b] >> (8 * q)));
                }
    };
    int k0 = wave * 256;
    for (; k0 + 256 <= p.K; k0 += kThinWaves * 256)
        chunk(k0, std::integral_constant<int, 2>());
    if (k0 < p.K)
        chunk(k0, std::integral_constant<int, 1>());
    const float alpha = p.alpha ? p.alpha[g] : 1.0f;
#pragma unroll
    for (int b = 0; b < NB; b++) {
        if (b >= nb)
            break;
        if (b)
            __syncthreads();                           // sum may still be read
#pragma unroll
        for (int rb = 0; rb < kRB; rb++)
            sum[wave][rb][lane] = acc[rb][b];
        __syncthreads();
        if (wave < kRB) {
            f32x4 v = sum[0][wave][lane];
#pragma unroll
            for (int j = 1; j < kThinWaves; j++)
                v += sum[j][wave][lane];
            // register i of a lane is weight row 4 q + i, row r of d
            const int row = 16 * b + r, col = 16 * wave + 4 * q;
            if (row < rows && col < cols) {
                const float* const bias = p.bias ? p.bias + (int64_t)g * p.N + n0 + col : nullptr;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    v[i] = bias ? fmaf(alpha, v[i], bias[i]) : alpha * v[i];
                const int64_t at = (m0 + row) * p.N + n0 + col;
                if (p.d_dtype == GG_F32)
                    *(f32x4*)((float*)p.d + at) = v;
                else {
                    uint32_t lo, hi;
                    if (p.d_dtype == GG_BF16) {
                        lo = pack_bf16x2(v[0], v[1]);
                        hi = pack_bf16x2(v[2], v[3]);
                    } else {
                        lo = (uint32_t)f32_to_f16(v[0]) | (uint32_t)f32_to_f16(v[1]) << 16;
                        hi = (uint32_t)f32_to_f16(v[2]) | (uint32_t)f32_to_f16(v[3]) << 16;
                    }
                    *(u32x2*)((uint16_t*)p.d + at) = u32x2{lo, hi};
                }
            }
        }
    }
}

}  // namespace

// Blocks of 16 rows of the thin kernel's tiles, 0: the tiled kernel.
static int thin_blocks(const GemmMx4Args& p) {
    const int64_t each = p.m_rows / p.L;               // rows of a group, on average
    return each <= 16 ? 1 : each <= 64 ? 4 : 0;
}

int64_t gemm_mx4_blocks(const GemmMx4Args& p) {
    const int nb = thin_blocks(p);
    const int64_t tiles = nb ? tile_bound(p, 16 * nb, kThinCols) : tile_bound(p, GemmCfg::TM, GemmCfg::TN);
    return tiles > 1 ? tiles : 1;                      // (one block writes the error word)
}

hipError_t launch_gemm_mx4(const GemmMx4Args& p, hipStream_t s, LaunchInfo* info) {
    const int nb = thin_blocks(p);
    const dim3 grid((unsigned)gemm_mx4_blocks(p));
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "%s<D %s>", nb ? "thin_kernel" : "gemm_kernel",
                 dtype_name(p.d_dtype));
        info->tm = nb ? 16 * nb : GemmCfg::TM;
        info->tn = nb ? kThinCols : GemmCfg::TN;
        info->waves = nb ? kThinWaves : GemmCfg::kWaves;
        info->grid = grid.x;
    }
    if (nb == 1)
        hipLaunchKernelGGL((thin_kernel<1>), grid, dim3(kThinThreads), 0, s, p);
    else if (nb)
        hipLaunchKernelGGL((thin_kernel<4>), grid, dim3(kThinThreads), 0, s, p);
    else {
        const dim3 block(GemmCfg::kThreads);
        auto by_shape = [&](auto DTc) {
            constexpr int DT = decltype(DTc)::value;
            auto by_bias = [&](auto ODDc) {
                constexpr bool ODD = decltype(ODDc)::value;
                if (p.bias)
                    hipLaunchKernelGGL((gemm_kernel<DT, ODD, true>), grid, block, 0, s, p);
                else
                    hipLaunchKernelGGL((gemm_kernel<DT, ODD, false>), grid, block, 0, s, p);
            };
            p.K % 256 ? by_bias(std::true_type()) : by_bias(std::false_type());
        };
        if (p.d_dtype == GG_BF16)
            by_shape(std::integral_constant<int, GG_BF16>());
        else if (p.d_dtype == GG_F16)
            by_shape(std::integral_constant<int, GG_F16>());
        else
            by_shape(std::integral_constant<int, GG_F32>());
    }
    return hipGetLastError();
}

}  // namespace gg
