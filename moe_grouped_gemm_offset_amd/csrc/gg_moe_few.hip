// gg_moe_few.hip -- a whole mixture-of-experts layer for up to 64 tokens
// (gg_moe_few): every weight of a chosen expert is read once, so the layer
// costs what reading them costs.
//
// Two passes of one kernel, then the sum over a token's choices:
//   first    c = w1_e x, h = prob act(c + bias1), for every (token, choice)
//   second   w2_e h + prob bias2, for every (token, choice)
// A block takes 64 rows of one chosen expert's matrix and all of its tokens;
// its 8 waves split the reduction axis and add up in LDS.  Weights go from
// memory into the registers that the matrix instruction reads, as its 16-row
// operand (16x16x32, bf16): a lane loads 16 bytes of a row at a time, four
// lanes 64 consecutive ones, and the other half of the line next.  The tokens
// are the 16 columns.  4-bit weights are widened to bf16, which holds each
// exactly.  Four blocks of 16 rows share a column operand, so what comes from
// the cache is at most what comes from memory.
//
// h is kept as hi + lo, two bf16 values with 16 bits between them (in one, the
// rounding would show in an fp32 result): the second pass takes 8 choices as
// 16 columns, eight of hi and eight of lo, and adds them up at the end.
#include <type_traits>

#include "gg_act.hpp"
#include "gg_tile.hpp"

namespace gg {

namespace {

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
constexpr int kFewRows = 64, kRB = kFewRows / 16;
constexpr int kMaxPairs = 64 * 32;                    // tokens * top_k
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Workspace: the error word's header, h of every choice (hi, then lo), the
// choices' results.
__host__ __device__ inline size_t few_h_bytes(int64_t pairs, int64_t I) { return (size_t)(pairs * I * 4); }

// The expert of a block and its choices (indexes of (token, choice) in list).
struct Chosen {
    uint32_t map[32];         // a bit per expert
    int n;
    uint16_t list[kMaxPairs];
};

// Finds the a-th of the chosen experts in ascending order and lists its
// choices; -1 where there are fewer.
__device__ __forceinline__ int choose(const FewArgs& p, int a, Chosen& s) {
    constexpr int kEach = kMaxPairs / kFewThreads;
    const int t = threadIdx.x, lane = t & 63, pairs = p.T * p.k;
    int id[kEach];
#pragma unroll
    for (int c = 0; c < kEach; c++) {
        const int i = t + c * kFewThreads;
        id[c] = i < pairs ? p.ids[i] : -1;
    }
    if (t < 32)
        s.map[t] = 0;
    if (t == 0)
        s.n = 0;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kEach; c++)
        if ((uint32_t)id[c] < (uint32_t)p.E)
            atomicOr(&s.map[id[c] >> 5], 1u << (id[c] & 31));
    __syncthreads();
    const uint32_t word = lane < 32 ? s.map[lane] : 0;
    int upto = __popc(word);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int below = __shfl_up(upto, d);
        upto += lane >= d ? below : 0;
    }
    const uint64_t past = __ballot(upto > a);
    if (past == 0)
        return -1;
    const int at = __ffsll((unsigned long long)past) - 1;
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
    const int before = __builtin_amdgcn_readlane(upto, at) - __popc(bits);
    for (int i = before; i < a; i++)
        bits &= bits - 1;
    const int e = 32 * at + __ffs((int)bits) - 1;
#pragma unroll
    for (int c = 0; c < kEach; c++)
        if (id[c] == e)
            s.list[atomicAdd(&s.n, 1)] = (uint16_t)(t + c * kFewThreads);
    __syncthreads();
    return e;
}

__device__ __forceinline__ u32x4 load16(const void* base, uint32_t bytes) {
    return *(const u32x4*)((const char*)base + bytes);
}

// Eight 4-bit codes times 2^(s - 127), scale = s << 23.
__device__ __forceinline__ bf16x8 widen(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// acc[rb][b] += rows 16 rb .. of the block's 64 times columns 16 b .., over the
// wave's chunks of the reduction axis: 128 bytes of every row, in two halves.
// w: the block's first row, row_at[rb] the lane's row's offset from it (sf,
// scale_at likewise); x: the columns' matrix, col_at[b] the lane's column's
// offset; all in bytes.
template <bool MX4, int NB>
__device__ __forceinline__ void stream(const char* w, const uint32_t (&row_at)[kRB], const uint8_t* sf,
                                       const uint32_t (&scale_at)[kRB], const char* x,
                                       const uint32_t (&col_at)[NB], int nb, int K,
                                       f32x4 (&acc)[kRB][NB]) {
    constexpr int kChunk = MX4 ? 256 : 64, kHalf = kChunk / 2;
    constexpr int F = MX4 ? 4 : 1;                     // operands a lane's 16 bytes make
    const int wave = uniform(threadIdx.x >> 6), q = (threadIdx.x & 63) >> 4;
    auto chunk = [&](int k0, auto TAILc) {
        constexpr bool TAIL = decltype(TAILc)::value;
        u32x4 wv[2][kRB];
        uint32_t sc[2][kRB];
        bool in[2];
        // the lane's first value of each half, 0 past the row's end
        uint32_t at[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            at[h] = (uint32_t)(k0 + h * kHalf + q * (kHalf / 4));
            in[h] = !TAIL || at[h] < (uint32_t)K;
            at[h] = in[h] ? at[h] : 0u;
#pragma unroll
            for (int rb = 0; rb < kRB; rb++)
                wv[h][rb] = load16(w, row_at[rb] + (MX4 ? at[h] / 2 : at[h] * 2));
        }
        if constexpr (MX4) {
#pragma unroll
            for (int rb = 0; rb < kRB; rb++) {
                if constexpr (TAIL) {
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        sc[h][rb] = (uint32_t)sf[scale_at[rb] + at[h] / 32] << 23;
                } else {
                    const u32x2 v = *(const u32x2u*)(sf + scale_at[rb] + (uint32_t)k0 / 32);
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        sc[h][rb] = __builtin_amdgcn_ubfe(v[h], 8 * q, 8) << 23;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4 xv[NB][F];
#pragma unroll
            for (int b = 0; b < NB; b++)
                if (b < nb) {
#pragma unroll
                    for (int f = 0; f < F; f++) {
                        xv[b][f] = load16(x, col_at[b] + at[h] * 2 + f * 16);
                        if (TAIL && !in[h])
                            xv[b][f] = u32x4{0};
                    }
                }
            if constexpr (TAIL) {
                if (!in[h]) {
#pragma unroll
                    for (int rb = 0; rb < kRB; rb++)
                        wv[h][rb] = u32x4{0}, sc[h][rb] = 0;
                }
            }
#pragma unroll
            for (int f = 0; f < F; f++) {
                bf16x8 wf[kRB];
#pragma unroll
                for (int rb = 0; rb < kRB; rb++) {
                    if constexpr (MX4)
                        wf[rb] = widen(wv[h][rb][f], __builtin_bit_cast(float, sc[h][rb]));
                    else
                        wf[rb] = __builtin_bit_cast(bf16x8, wv[h][rb]);
                }
#pragma unroll
                for (int b = 0; b < NB; b++)
                    if (b < nb) {
#pragma unroll
                        for (int rb = 0; rb < kRB; rb++)
                            acc[rb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wf[rb], __builtin_bit_cast(bf16x8, xv[b][f]), acc[rb][b], 0, 0, 0);
                    }
            }
        }
    };
    int k0 = wave * kChunk;
    for (; k0 + kChunk <= K; k0 += kFewWaves * kChunk)
        chunk(k0, std::false_type());
    if (k0 < K)
        chunk(k0, std::true_type());
}

// ACT: the first pass and its activation, or -1: the second pass.
template <bool MX4, int NB, int ACT>
__global__ void __launch_bounds__(kFewThreads, NB <= 2 ? 4 : 2) few_kernel(FewArgs p) {
    constexpr bool FIRST = ACT >= 0;
    __shared__ Chosen s;
    __shared__ __attribute__((aligned(16))) f32x4 sum[kFewWaves][kRB][64];
    if (FIRST && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *(int32_t*)p.ws = 0;                           // the error word
    const int e = uniform(choose(p, blockIdx.y, s));
    if (e < 0)
        return;
    const int n = uniform(s.n), pairs = p.T * p.k;
    const int R = FIRST ? 2 * p.I : p.H, K = FIRST ? p.H : p.I, row0 = blockIdx.x * kFewRows;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int rows = R - row0 < kFewRows ? R - row0 : kFewRows;
    const int64_t first = (int64_t)e * R + row0;
    const uint32_t pitch = (uint32_t)(MX4 ? K / 2 : K * 2);
    const char* const w = (const char*)(FIRST ? p.w1 : p.w2) + first * pitch;
    const uint8_t* const sf = (FIRST ? p.sf1 : p.sf2) + first * (K / 32);
    uint32_t row_at[kRB], scale_at[kRB];
#pragma unroll
    for (int rb = 0; rb < kRB; rb++) {
        const int row = min(16 * rb + r, rows - 1);
        row_at[rb] = row * pitch;
        scale_at[rb] = (uint32_t)(row * (K / 32));
    }
    char* const hbuf = p.ws + kWsHeader;
    float* const out = (float*)(hbuf + few_h_bytes(pairs, p.I));
    // columns of a 16-column operand block: 16 tokens, or 8 choices twice
    constexpr int kCols = FIRST ? 16 : 8;
    const char* const x = FIRST ? (const char*)p.x : hbuf;
    for (int c0 = 0; c0 < n; c0 += kCols * NB) {
        const int nb = min(NB, (n - c0 + kCols - 1) / kCols);
        uint32_t col_at[NB];
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const uint32_t i = s.list[min(c0 + kCols * b + (FIRST ? r : r & 7), n - 1)];
            col_at[b] = FIRST ? (uint32_t)((i / p.k) * p.ldx * 2)
                              : (uint32_t)(((r < 8 ? 0 : pairs) + i) * p.I * 2);
        }
        f32x4 acc[kRB][NB];
#pragma unroll
        for (int rb = 0; rb < kRB; rb++)
#pragma unroll
            for (int b = 0; b < NB; b++)
                acc[rb][b] = f32x4{0};
        stream<MX4, NB>(w, row_at, sf, scale_at, x, col_at, nb, K, acc);
#pragma unroll
        for (int b = 0; b < NB; b++) {
            if (b >= nb)
                break;
            __syncthreads();                           // sum may still be read
#pragma unroll
            for (int rb = 0; rb < kRB; rb++)
                sum[wave][rb][lane] = acc[rb][b];
            __syncthreads();
            // register i of a lane is row 16 rb + 4 q + i, column r
            const int c = c0 + kCols * b + (FIRST ? r : r & 7);
            const bool live = c < n;
            const int pair = s.list[live ? c : n - 1];
            if constexpr (FIRST) {
                if (wave < 2) {                        // rows 16 wave .. of the 32 pairs
                    f32x4 v[2];
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        v[half] = sum[0][2 * half + wave][lane];
#pragma unroll
                        for (int j = 1; j < kFewWaves; j++)
                            v[half] += sum[j][2 * half + wave][lane];
                        if (p.bias1) {
                            const float* bias = p.bias1 + first + 32 * half + 16 * wave + 4 * q;
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                v[half][i] += bias[i];
                        }
                    }
                    const float pr = p.prob[pair];
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float g = p.act.gate_first ? v[0][i] : v[1][i];
                        const float u = p.act.gate_first ? v[1][i] : v[0][i];
                        const float h = act_forward<ACT>(g, u, p.act) * pr;
                        const uint16_t a = from_f32<GG_BF16>(h);
                        const float rest = h - to_f32<GG_BF16>(a);
                        // (nothing is left of an infinity)
                        const uint16_t d = from_f32<GG_BF16>(fabsf(h) < INFINITY ? rest : 0.0f);
                        hi[i >> 1] = i & 1 ? hi[i >> 1] | (uint32_t)a << 16 : a;
                        lo[i >> 1] = i & 1 ? lo[i >> 1] | (uint32_t)d << 16 : d;
                    }
                    if (live) {
                        char* const h = hbuf + ((int64_t)pair * p.I + row0 / 2 + 16 * wave + 4 * q) * 2;
                        *(u32x2*)h = u32x2{hi[0], hi[1]};
                        *(u32x2*)(h + (int64_t)pairs * p.I * 2) = u32x2{lo[0], lo[1]};
                    }
                }
            } else {
                if (wave < kRB) {
                    f32x4 v = sum[0][wave][lane];
#pragma unroll
                    for (int j = 1; j < kFewWaves; j++)
                        v += sum[j][wave][lane];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        v[i] += __shfl_xor(v[i], 8);   // hi and lo
                    const int row = row0 + 16 * wave + 4 * q;
                    if (live && r < 8 && row < R) {
                        if (p.bias2) {
                            const float pr = p.prob[pair];
                            const float* bias = p.bias2 + (int64_t)e * p.H + row;
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                v[i] = fmaf(pr, bias[i], v[i]);
                        }
                        *(f32x4*)(out + (int64_t)pair * p.H + row) = v;
                    }
                }
            }
        }
    }
}

// y[t] = the sum of the results of t's choices, in their order.
template <int DT>
__global__ void __launch_bounds__(256) few_sum_kernel(FewArgs p) {
    const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= p.H)
        return;
    const float* const in = (const float*)(p.ws + kWsHeader + few_h_bytes((int64_t)p.T * p.k, p.I));
    f32x4 y = {0};
    for (int j = 0; j < p.k; j++) {
        const int i = t * p.k + j;
        if ((uint32_t)p.ids[i] < (uint32_t)p.E)
            y += *(const f32x4*)(in + (int64_t)i * p.H + c);
    }
    typedef typename Elem<DT>::T T;
    T* const out = (T*)p.y + t * p.ldy + c;
#pragma unroll
    for (int i = 0; i < 4; i++)
        out[i] = from_f32<DT>(y[i]);
}

template <class F>
void for_blocks(int nb, F f) {
    if (nb <= 1)
        f(std::integral_constant<int, 1>());
    else if (nb == 2)
        f(std::integral_constant<int, 2>());
    else
        f(std::integral_constant<int, 4>());
}

}  // namespace

size_t few_workspace(int64_t T, int64_t k, int64_t H, int64_t I) {
    return kWsHeader + few_h_bytes(T * k, I) + (size_t)(T * k * H * 4);
}

hipError_t launch_few(const FewArgs& p, hipStream_t s, LaunchInfo* info) {
    const int pairs = p.T * p.k;
    if (p.T == 0)
        return hipSuccess;
    // Columns that an expert is likely to have: twice its share and a few more,
    // at most one a token.  (More take another pass over its weights.)
    const int share = 2 * ((pairs + p.E - 1) / p.E) + 8, cols = share < p.T ? share : p.T;
    const int active = pairs < p.E ? pairs : p.E;
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "few_kernel<%s> x 2 + sum", p.mx4 ? "mxfp4" : "bf16");
        info->tm = kFewRows;
        info->tn = cols;
        info->waves = kFewWaves;
        info->grid = (int64_t)(p.I / 32) * active;
    }
    const dim3 block(kFewThreads), first(p.I / 32, active), second((p.H + kFewRows - 1) / kFewRows, active);
    auto by_weights = [&](auto MX4) {
        constexpr bool mx4 = decltype(MX4)::value;
        for_blocks((cols + 15) / 16, [&](auto NB) {
            for_act(p.act.act, [&](auto ACT) {
                hipLaunchKernelGGL((few_kernel<mx4, decltype(NB)::value, decltype(ACT)::value>), first, block,
                                   0, s, p);
            });
        });
        for_blocks((cols + 7) / 8, [&](auto NB) {
            hipLaunchKernelGGL((few_kernel<mx4, decltype(NB)::value, -1>), second, block, 0, s, p);
        });
    };
    p.mx4 ? by_weights(std::true_type()) : by_weights(std::false_type());
    const dim3 sum((p.H + 1023) / 1024, p.T);
    if (p.y_dtype == GG_BF16)
        hipLaunchKernelGGL((few_sum_kernel<GG_BF16>), sum, dim3(256), 0, s, p);
    else if (p.y_dtype == GG_F16)
        hipLaunchKernelGGL((few_sum_kernel<GG_F16>), sum, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((few_sum_kernel<GG_F32>), sum, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gg
