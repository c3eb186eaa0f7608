// gg_moe_few.hip -- a whole mixture-of-experts layer for up to 64 tokens
// (gg_moe_few): the layer costs what reading the chosen experts' weights costs, as
// long as a block has columns for all choices of its expert.  It has 4 to 32, shared by
// the parts of h in the second pass; more choices take another pass over the weights
// (60 tokens, 7 of 8 experts of 5024 x 2304 in bf16, fp32 y, some 52 choices an expert:
// 2 passes and 6, 408 us for the 85 of reading them once).
//
//   first    c = w1_e x, h = prob act(c + bias1), for every (token, choice)
//   second   w2_e h + prob bias2, for every (token, choice)
//   sum      y = the sum over a token's choices
//
// A wave takes 32 rows of one chosen expert's matrix (in the first pass 16 input
// rows and the 16 gate rows that go with them) and streams them from memory into
// the registers that the matrix instruction reads, as its 16-row operand
// (16x16x32, bf16); 4-bit weights are widened to bf16, which holds each exactly.
// The tokens of the expert are the 16 columns.
//
// Tokens that share experts (few_kernel, few_sum_kernel): a block stands for an
// expert, so that its weights are read once; the waves share the columns in LDS.
// They have different rows, or, where there are too few rows to fill the device,
// WK of them the same rows and parts of the reduction axis, added up in LDS.
// (The sum by the last block of some rows, which saves the launch, took longer:
// every block then awaits its results and counts itself, 5 us of one token's
// second pass for the 4 of the launch, 60 us of 64 tokens'.)
//
// Few tokens, whose choices share little (lone_first_kernel, lone_second_kernel): a
// wave takes rows of one choice's expert, with its columns in LDS of its own, so
// none waits for another on the way, and a token's choices meet in one block of
// the second pass, which leaves no third.  One token over 64 experts of 4096 x
// 2048, 8 choices, weights from memory: MXFP4 49 us for 54, bf16 127 for 140.  (From
// memory, here and below: after 256 MB were overwritten, which are written back under
// the weights' loads.  Without that, other experts at each call, 855 MB in turn: 28 and
// 72 us.)
//
// What a CU's load path takes is lines: a vector load of 8 rows x 128 bytes
// costs half of one of 16 rows x 64 bytes.  So 16 bf16 rows x 128 bytes come in
// two loads of 8 whole lines, and lanes r and r + 8 of every 16 then exchange a
// half (a DPP move a register), which leaves each lane 16-byte pieces of its own
// row.  4-bit rows come as halves of lines, a quarter of the bytes for the same
// arithmetic: there the moves cost what the lines save (64 experts of 4096 x 2048, one
// token, both passes: 28.7 us with them, 28.2 without).  Their scales come in one load for
// 2 lines, 4 bytes a lane, and go to the lanes by row swaps.
//
// h is kept as the sum of `parts` bf16 values, 2 for a 16-bit y (16 bits of h),
// 3 for an fp32 one (24 bits): the second pass takes them as so many columns and
// adds the columns' results up.
#include <cmath>
#include <type_traits>

#include "gg_act.hpp"
#include "gg_stream.hpp"

namespace gg {

namespace {

constexpr int kMaxPairs = 64 * 32;                    // tokens * top_k
constexpr int kParts = 3;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Workspace: the error word's header, h of every choice (its parts one after
// the other), the choices' results.
__host__ __device__ inline size_t few_h_bytes(int64_t pairs, int64_t I) {
    return (size_t)(pairs * I * 2 * kParts);
}

// The choices of a block's expert: of each its index in (token, choice) order,
// and its token in the upper half.
struct Choices {
    // (all waves list the same for themselves)
    uint32_t* list;
    int n, first;

    // Up to num_experts choices the block stands for choice a, and the first
    // choice of an expert has them all; with more it stands for expert a.
    static __device__ __forceinline__ bool by_pair(const FewArgs& p) { return p.T * p.k <= p.E; }

    __device__ __forceinline__ void add(const FewArgs& p, int at, int id, int e) {
        const int i = at + (int)(threadIdx.x & 63);
        const bool hit = i < p.T * p.k && id == e;
        const uint64_t m = __ballot(hit);
        if (hit)                                       // (i / k by a reciprocal, exact below 2^11)
            list[n + __popcll(m & ((1ull << (threadIdx.x & 63)) - 1))] = (uint32_t)i * p.k_magic >> 16 << 16 | i;
        if (first < 0 && m)
            first = at + __ffsll((unsigned long long)m) - 1;
        n += __popcll(m);
    }
    __device__ __forceinline__ void collect(const FewArgs& p, int e) {
        constexpr int kAtOnce = 8;
        const int pairs = p.T * p.k, lane = threadIdx.x & 63;
        if (pairs <= 64) {
            add(p, 0, p.ids[min(lane, pairs - 1)], e);
        } else {
            for (int at = 0; at < pairs; at += 64 * kAtOnce) {
                int id[kAtOnce];
#pragma unroll
                for (int c = 0; c < kAtOnce; c++)
                    id[c] = p.ids[min(at + 64 * c + lane, pairs - 1)];
#pragma unroll
                for (int c = 0; c < kAtOnce; c++)
                    add(p, at + 64 * c, id[c], e);
            }
        }
        wave_sync();
    }
};

// What the next bf16 part of h is rounded from: h, but no more than bf16's largest
// where h is finite (an fp32 number past it would become an infinity, and h less
// that one too).
__device__ __forceinline__ float part_of(float h) {
    constexpr float top = 0x1.FEp127f;
    return fabsf(h) < INFINITY ? __builtin_amdgcn_fmed3f(h, -top, top) : h;
}
// What a part leaves of h (nothing of an infinity).
__device__ __forceinline__ float less_part(float h) {
    return fabsf(h) < INFINITY ? h - bf16_to_f32(f32_to_bf16(part_of(h))) : 0.0f;
}

// A sum over all parts of h, from that over the first parts alone: an infinite
// weight makes a NaN of a part that is 0, and of parts of different signs, where its
// product with h is an infinity, as with the first part.  (Finite weights give a NaN
// in both or in neither.)
__device__ __forceinline__ float over_parts(float all, float first) { return all == all ? all : first; }

// Eight 4-bit codes times 2^(s - 127), scale = s << 23.
__device__ __forceinline__ bf16x8 widen(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Blocks of NW waves, WK of them along the reduction axis; 16 NB columns of LDS
// for the WK parts together, XC for each.
template <bool MX4_, int NW_, int WK_, int NB_>
struct Few {
    static constexpr bool MX4 = MX4_;
    static constexpr int NW = NW_, WK = WK_, NB = NB_, WR = NW / WK, kThreads = 64 * NW;
    static constexpr int XC = 16 * NB / WK;
    // a piece: 2 or 4 lines of every row, and as many values of the columns
    static constexpr int kLines = MX4 ? 2 : 4, kBytes = 128 * kLines, kValues = MX4 ? 2 * kBytes : kBytes / 2;
    static constexpr int kHalf = MX4 ? 128 : 32, F = MX4 ? 4 : 1;   // operands of 16 bytes
    static constexpr int kPitch = 2 * kValues + 16;              // of a column in LDS
    static constexpr int kX = 16 * NB * kPitch;
    static constexpr int kPer = 2 * kValues / 16;                // 16-byte pieces of a column
    static constexpr int kStage = 16 * NB * kPer / kThreads;     // of them a thread
    static constexpr int kSum = NW * 2 * NB * 1024;
    static constexpr int kLds = 2 * kX > kSum ? 2 * kX : kSum;
    static_assert(kStage * kThreads == 16 * NB * kPer, "whole pieces a thread");
};

// ACT: the first pass and its activation, or -1: the second pass, over PARTS
// columns a choice.
template <class C, int ACT, int PARTS>
__global__ void __launch_bounds__(C::kThreads, 2) few_kernel(FewArgs p) {
    constexpr bool FIRST = ACT >= 0, MX4 = C::MX4;
    constexpr int NB = C::NB, WK = C::WK, XC = C::XC, kPass = XC / PARTS;
    __shared__ __attribute__((aligned(16))) char smem[C::kLds];
    __shared__ uint32_t list[kMaxPairs];
    const int pairs = p.T * p.k;
    char* const hbuf = p.ws + kWsHeader;
    float* const out = (float*)(hbuf + few_h_bytes(pairs, p.I));
    const bool by_pair = Choices::by_pair(p);
    const int e = by_pair ? scalar_read(p.ids + blockIdx.y) : (int)blockIdx.y;
    if (FIRST && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *(int32_t*)p.ws = 0;                           // the error word
    if ((uint32_t)e >= (uint32_t)p.E)
        return;
    Choices choices{list, 0, -1};
    choices.collect(p, e);
    const int n = uniform(choices.n);
    if (n == 0 || (by_pair && uniform(choices.first) != (int)blockIdx.y))
        return;
    const int R = FIRST ? 2 * p.I : p.H, K = FIRST ? p.H : p.I;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wr = wave / WK, wk = wave % WK;
    // the wave's rows: 16 from row0 on and 16 from row0 + second on
    const int units = R / 32;
    const int unit = min((int)blockIdx.x * C::WR + wr, units - 1);
    const int row0 = FIRST ? unit / 2 * 64 + unit % 2 * 16 : unit * 32, second = FIRST ? 32 : 16;
    const int64_t first = (int64_t)e * R + row0;
    const uint32_t pitch = (uint32_t)(MX4 ? K / 2 : K * 2), KB = K / 32;
    const __amdgpu_buffer_rsrc_t rw =
        make_rsrc(uniform_ptr((const char*)(FIRST ? p.w1 : p.w2) + first * pitch), (second + 16) * pitch);
    const uint8_t* const sf = (FIRST ? p.sf1 : p.sf2) + first * KB;
    // Load i of a row block's line: bf16, rows 8 i + r % 8, piece q (lanes 0 .. 7)
    // or 4 + q; 4-bit, row r, half i, piece q.
    const uint32_t piece = 16 * (MX4 ? q : q + 4 * (r >> 3));
    uint32_t row_at[2][2];
#pragma unroll
    for (int rb = 0; rb < 2; rb++)
#pragma unroll
        for (int i = 0; i < 2; i++)
            row_at[rb][i] = (MX4 ? (uint32_t)(rb * second + r) * pitch + 64 * i
                                 : (uint32_t)(rb * second + 8 * i + (r & 7)) * pitch) + piece;
    const int pieces = (int)((pitch + C::kBytes - 1) / C::kBytes), steps = (pieces + WK - 1) / WK;
    // Blocks start at different pieces: at the same one they would all read the
    // same few of the memory's channels (rows are powers of two apart: 441 us for
    // 355 on the bf16 first pass of 64 tokens over 64 experts of 4096 x 2048).
    const int start = (blockIdx.x + e) % steps;
    auto turn = [&](int t) { return t >= steps ? steps : (t + start >= steps ? t + start - steps : t + start); };

    constexpr int kLines = C::kLines;
    u32x4 w[kLines][2][2];
    uint32_t sc[2], next_sc[2];
    // Line j of the wave's piece of step t.  Past the row's end: zeros (bf16), or
    // whatever the next row has there (4-bit: finite, at scales of 2^-127 against
    // columns of zeros).
    auto load_line = [&](int t, int j) {
        const uint32_t at = (uint32_t)(t * WK + wk) * C::kBytes;
        const bool in = MX4 || at + 128 * j + piece < pitch;
#pragma unroll
        for (int rb = 0; rb < 2; rb++)
#pragma unroll
            for (int i = 0; i < 2; i++)
                w[j][rb][i] = buf16(rw, in ? row_at[rb][i] + at + 128 * j : kInvalid);
    };
    // The scales of half line q of step t, of row r: 4 bytes, 0 past the row's end.
    // (Loaded at the array's last 4 bytes where they would pass its end.)
    const int64_t sf_left = ((int64_t)p.E * R - first) * KB - 4;
    const uint32_t sf_last = sf_left < INT32_MAX ? (uint32_t)sf_left : INT32_MAX;
    auto load_scales = [&](int t, uint32_t (&v)[2]) {
        if constexpr (MX4) {
            typedef uint32_t Four __attribute__((aligned(1)));
#pragma unroll
            for (int rb = 0; rb < 2; rb++) {
                const uint32_t at = (uint32_t)(rb * second + r) * KB + (uint32_t)(t * WK + wk) * 16 + 4 * q;
                v[rb] = *(const Four*)(sf + min(at, sf_last));
            }
        }
    };
    auto row_scales = [&](int t, const uint32_t (&v)[2], uint32_t (&out)[2][4]) {
#pragma unroll
        for (int rb = 0; rb < 2; rb++) {
            const uint32_t in_row = (uint32_t)(t * WK + wk) * 16 + 4 * q;
            const uint32_t at = (uint32_t)(rb * second + r) * KB + in_row;
            const uint32_t past = at > sf_last ? at - sf_last : 0;
            uint32_t x = v[rb] >> (8 * (past & 3));
            if (in_row + 4 > KB)
                x = in_row < KB ? x & ((1u << (8 * (KB - in_row))) - 1) : 0;
            spread4(x, out[rb]);
        }
    };

    auto load_weights = [&](int t) {
        load_scales(t, sc);
#pragma unroll
        for (int j = 0; j < kLines; j++)
            load_line(t, j);
    };
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(FIRST ? p.x : hbuf);
    for (int c0 = 0; c0 < n; c0 += kPass) {
        const int here = min(kPass, n - c0);
        // the thread's pieces of the columns, choice by choice within a part
        uint32_t x_at[C::kStage], x_lds[C::kStage];
        int x_k[C::kStage];
#pragma unroll
        for (int i = 0; i < C::kStage; i++) {
            const int c = threadIdx.x + i * C::kThreads, col = c / C::kPer, xk = col / XC, own = col % XC;
            const int part = own / kPass, which = own % kPass, k = xk * C::kValues + c % C::kPer * 8;
            const bool live = part < PARTS && which < here;
            const uint32_t choice = list[c0 + (live ? which : 0)], pair = choice & 0xFFFF;
            x_k[i] = live ? k : INT32_MAX / 2;
            x_at[i] = ((FIRST ? (choice >> 16) * (uint32_t)p.ldx : (part * pairs + pair) * (uint32_t)p.I) + k) * 2;
            x_lds[i] = col * C::kPitch + c % C::kPer * 16;
        }
        // What a thread finishes: four rows of a choice (in the first pass four
        // inputs and their gates), with their biases and the choice's prob, which
        // are loaded before the product for a thread's first.
        struct Item {
            int q, rb, which, wrow, u, pair;
        };
        struct Extra {
            float prob;
            f32x4 bias[2];
        };
        auto item = [&](int it) {
            Item m;
            m.q = it & 3;
            m.rb = FIRST ? 0 : it >> 2 & 1;
            const int c = it / (FIRST ? 4 : 8);
            m.wrow = c % C::WR;
            m.which = c / C::WR;
            m.u = blockIdx.x * C::WR + m.wrow;
            m.pair = list[c0 + min(m.which, here - 1)] & 0xFFFF;
            return m;
        };
        auto extra = [&](const Item& m) {
            Extra x = {p.prob[m.pair], {f32x4{0}, f32x4{0}}};
            const float* const bias = FIRST ? p.bias1 : p.bias2;
            if (bias && m.u < units) {
                const int row = FIRST ? m.u / 2 * 64 + m.u % 2 * 16 + 4 * m.q : m.u * 32 + 16 * m.rb + 4 * m.q;
#pragma unroll
                for (int rb = 0; rb < (FIRST ? 2 : 1); rb++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        x.bias[rb][i] = bias[(int64_t)e * R + row + 32 * rb + i];
            }
            return x;
        };
        u32x4 xr[C::kStage];
        auto load_x = [&](int t) {
            const int k0 = t * WK * C::kValues;
#pragma unroll
            for (int i = 0; i < C::kStage; i++)
                xr[i] = buf16(rx, k0 + x_k[i] < K ? x_at[i] + k0 * 2 : kInvalid);
        };
        auto store_x = [&](int t) {
#pragma unroll
            for (int i = 0; i < C::kStage; i++)
                *(u32x4*)(smem + (t & 1) * C::kX + x_lds[i]) = xr[i];
        };
        f32x4 acc[2][NB];
#pragma unroll
        for (int rb = 0; rb < 2; rb++)
#pragma unroll
            for (int b = 0; b < NB; b++)
                acc[rb][b] = f32x4{0};
        // a lane's column of each block of 16 (the first where there is none)
        uint32_t col_at[NB];
#pragma unroll
        for (int b = 0; b < NB; b++)
            col_at[b] = (wk * XC + (16 * b + r < kPass * PARTS && (16 * b + r) % kPass < here ? 16 * b + r : 0)) *
                            C::kPitch + q * (2 * C::kHalf / 4);

        // The columns of every wave before any wave's weights: a CU's vector loads
        // return in the order they were issued.
        load_x(turn(0));
        unit_barrier();
        load_weights(turn(0));
        const Extra early = extra(item(threadIdx.x));
        store_x(0);
        lds_wait();
        unit_barrier();
        for (int t = 0; t < steps; t++) {
            const int next = turn(t + 1);
            load_x(next);
            load_scales(next, next_sc);
            uint32_t scale[2][4];
            if constexpr (MX4)
                row_scales(turn(t), sc, scale);
            const char* const xb = smem + (t & 1) * C::kX;
#pragma unroll
            for (int j = 0; j < kLines; j++) {
                u32x4 wv[2][2];
#pragma unroll
                for (int rb = 0; rb < 2; rb++) {
                    if constexpr (MX4)
                        wv[rb][0] = w[j][rb][0], wv[rb][1] = w[j][rb][1];
                    else
                        own_rows(r < 8, w[j][rb][0], w[j][rb][1], wv[rb]);
                }
                if constexpr (!MX4)
                    load_line(next, j);
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int f = 0; f < C::F; f++) {
                        bf16x8 wf[2];
#pragma unroll
                        for (int rb = 0; rb < 2; rb++) {
                            if constexpr (MX4)
                                wf[rb] = widen(wv[rb][h][f], __builtin_bit_cast(float, __builtin_amdgcn_ubfe(
                                                                 scale[rb][(2 * j + h) & 3], 8 * q, 8) << 23));
                            else
                                wf[rb] = __builtin_bit_cast(bf16x8, wv[rb][h]);
                        }
#pragma unroll
                        for (int b = 0; b < NB; b++) {
                            const bf16x8 xf = __builtin_bit_cast(
                                bf16x8, *(const u32x4*)(xb + col_at[b] + (2 * j + h) * 2 * C::kHalf + f * 16));
#pragma unroll
                            for (int rb = 0; rb < 2; rb++)
                                acc[rb][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[rb], xf, acc[rb][b], 0, 0, 0);
                        }
                    }
                // (once the line is used up: the loads go into its registers)
                if constexpr (MX4)
                    load_line(next, j);
                __builtin_amdgcn_sched_barrier(0);
            }
            store_x(t + 1);
            sc[0] = next_sc[0], sc[1] = next_sc[1];
            lds_wait();
            unit_barrier();
        }
        // Sums over the waves of a row, and over the parts: register i of a lane is
        // row 4 q + i of its block, column r.
        f32x4 (*const sum)[2][NB][64] = (f32x4 (*)[2][NB][64])smem;
#pragma unroll
        for (int rb = 0; rb < 2; rb++)
#pragma unroll
            for (int b = 0; b < NB; b++)
                sum[wave][rb][b][lane] = acc[rb][b];
        __syncthreads();
        auto total = [&](int wrow, int rb, int qq, int col) {
            f32x4 v = sum[wrow * WK][rb][col >> 4][qq * 16 + (col & 15)];
#pragma unroll
            for (int j = 1; j < WK; j++)
                v += sum[wrow * WK + j][rb][col >> 4][qq * 16 + (col & 15)];
            return v;
        };
        if constexpr (FIRST) {
            for (int it = threadIdx.x; it < C::WR * here * 4; it += C::kThreads) {
                const Item m = item(it);
                if (m.u >= units)
                    continue;
                const Extra x = it < C::kThreads ? early : extra(m);
                f32x4 v[2];
#pragma unroll
                for (int rb = 0; rb < 2; rb++)
                    v[rb] = total(m.wrow, rb, m.q, m.which) + x.bias[rb];
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float g = p.act.gate_first ? v[0][i] : v[1][i];
                    h[i] = act_forward<ACT>(g, p.act.gate_first ? v[1][i] : v[0][i], p.act) * x.prob;
                }
                char* at = hbuf + ((int64_t)m.pair * p.I + m.u * 16 + 4 * m.q) * 2;
                for (int part = 0; part < p.parts; part++, at += (int64_t)pairs * p.I * 2) {
                    *(u32x2*)at = u32x2{pack_bf16x2(part_of(h[0]), part_of(h[1])),
                                        pack_bf16x2(part_of(h[2]), part_of(h[3]))};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        h[i] = less_part(h[i]);
                }
            }
        } else {
            for (int it = threadIdx.x; it < C::WR * here * 8; it += C::kThreads) {
                const Item m = item(it);
                if (m.u >= units)
                    continue;
                const Extra x = it < C::kThreads ? early : extra(m);
                const f32x4 of_first = total(m.wrow, m.rb, m.q, m.which);
                f32x4 v = of_first;
#pragma unroll
                for (int part = 1; part < PARTS; part++)
                    v += total(m.wrow, m.rb, m.q, part * kPass + m.which);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    v[i] = fmaf(x.prob, x.bias[0][i], over_parts(v[i], of_first[i]));
                *(f32x4*)(out + (int64_t)m.pair * p.H + m.u * 32 + 16 * m.rb + 4 * m.q) = v;
            }
        }
        __syncthreads();                               // the columns' LDS is free again
    }
}

// y[t] = the sum of the results of t's choices, in their order (the loads of
// kAtOnce of them at once).
template <int DT>
__global__ void __launch_bounds__(256) few_sum_kernel(FewArgs p) {
    constexpr int kAtOnce = 8;
    const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= p.H)
        return;
    const float* const in = (const float*)(p.ws + kWsHeader + few_h_bytes((int64_t)p.T * p.k, p.I));
    f32x4 y = {0};
    for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
        f32x4 v[kAtOnce];
        bool live[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; j++) {
            const int i = t * p.k + min(j0 + j, p.k - 1);
            live[j] = j0 + j < p.k && (uint32_t)scalar_read(p.ids + i) < (uint32_t)p.E;
            v[j] = *(const f32x4*)(in + (int64_t)i * p.H + c);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; j++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                y[i] = live[j] ? y[i] + v[j][i] : y[i];
    }
    const int64_t at = t * p.ldy + c;
    if constexpr (DT == GG_F32) {
        typedef f32x4 Out __attribute__((aligned(4)));
        *(Out*)((float*)p.y + at) = y;
    } else {
        typedef u32x2 Out __attribute__((aligned(2)));
        auto two = [](float a, float b) { return (uint32_t)from_f32<DT>(a) | (uint32_t)from_f32<DT>(b) << 16; };
        *(Out*)((uint16_t*)p.y + at) = u32x2{two(y[0], y[1]), two(y[2], y[3])};
    }
}

// A call without tokens.
__global__ void __launch_bounds__(64) few_none_kernel(int32_t* ws) {
    if (threadIdx.x == 0)
        *ws = 0;                                       // the error word
}

// The most choices that a token's block has waves for.
constexpr int kLoneK = 8;

// Whether the choices go each for itself: up to 4 tokens, or half as many choices
// as experts, and not more choices than experts (from memory, us, apart / shared;
// experts of 4096 x 2048: 4 tokens, 8 of 64, MXFP4 129 / 139, bf16 313 / 327; 8 tokens, 4 of
// 64, 131 / 138 and 314 / 322; 6 tokens, 8 of 64, 167 / 161 and 430 / 396).
bool lone(const FewArgs& p) {
    const int pairs = p.T * p.k;
    return p.k <= kLoneK && pairs <= p.E && (p.T <= 4 || 2 * pairs <= p.E);
}

// Few tokens with choices of their own: a wave takes 16 RB rows of one choice's
// expert (the blocks of 16 `apart` rows from one another), or every WK-th piece of
// them, against COLS columns, at its own pace: no wave waits for another before
// their sum.  Its columns pass through its own region of LDS.
template <bool MX4, int RB, int COLS>
struct Lone {
    // a piece: 2 lines of every row (4: 50 for 49 us, and 130 for 127, of the calls
    // at the head), and as many values of the columns
    static constexpr int LINES = 2;
    static constexpr int F = MX4 ? 4 : 1, kBytes = 128 * LINES, kValues = MX4 ? 2 * kBytes : kBytes / 2;
    static constexpr int kCol = 2 * kValues + 16, kX = COLS * kCol, kLds = 2 * kX;
    static constexpr int kPer = 2 * kValues / 16, kStage = (COLS * kPer + 63) / 64;

    // The wave's sums: register i of a lane is row 4 q + i of its block, column r.
    // The rows are those of expert e (R each, of K values) from row0 on; column c's
    // values are at x0 + c x_next (bytes).  `seed` chooses the piece that is first.
    static __device__ __forceinline__ void run(char* lds, const void* w_all, const uint8_t* sf_all, int E, int R, int K,
                                               int e, int row0, int apart, __amdgpu_buffer_rsrc_t rx, uint32_t x0,
                                               uint32_t x_next, int wk, int WK, int seed, f32x4 (&acc)[RB]) {
        const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
        const int64_t first = (int64_t)e * R + row0;
        const uint32_t pitch = (uint32_t)(MX4 ? K / 2 : K * 2), KB = K / 32;
        const __amdgpu_buffer_rsrc_t rw =
            make_rsrc(uniform_ptr((const char*)w_all + first * pitch), ((RB - 1) * apart + 16) * pitch);
        const uint8_t* const sf = sf_all + first * KB;
        const uint32_t piece = 16 * (MX4 ? q : q + 4 * (r >> 3));
        uint32_t row_at[RB][2];
#pragma unroll
        for (int rb = 0; rb < RB; rb++)
#pragma unroll
            for (int i = 0; i < 2; i++)
                row_at[rb][i] = (MX4 ? (uint32_t)(rb * apart + r) * pitch + 64 * i
                                     : (uint32_t)(rb * apart + 8 * i + (r & 7)) * pitch) + piece;
        const int pieces = (int)((pitch + kBytes - 1) / kBytes), steps = (pieces + WK - 1) / WK;
        const int start = seed % steps;
        auto turn = [&](int i) { return i >= steps ? steps : (i + start >= steps ? i + start - steps : i + start); };
        u32x4 w[LINES][RB][2], xr[kStage];
        uint32_t sc[RB], next_sc[RB];
        // (past the row's end as in few_kernel, the scales too)
        auto load_line = [&](int i, int l) {
            const uint32_t at = (uint32_t)(i * WK + wk) * kBytes + 128 * l;
            const bool in = MX4 || at + piece < pitch;
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    w[l][rb][h] = buf16(rw, in ? row_at[rb][h] + at : kInvalid);
        };
        const int64_t sf_left = ((int64_t)E * R - first) * KB - 4;
        const uint32_t sf_last = sf_left < INT32_MAX ? (uint32_t)sf_left : INT32_MAX;
        auto scale_at = [&](int i) { return (uint32_t)(i * WK + wk) * 16 + 4 * q; };
        auto load_scales = [&](int i, uint32_t (&v)[RB]) {
            typedef uint32_t Four __attribute__((aligned(1)));
            if constexpr (MX4)
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
                    v[rb] = *(const Four*)(sf + min((rb * apart + r) * KB + scale_at(i), sf_last));
        };
        auto row_scales = [&](int i, int rb, uint32_t v, uint32_t (&out)[4]) {
            const uint32_t in_row = scale_at(i), at = (rb * apart + r) * KB + in_row;
            const uint32_t past = at > sf_last ? at - sf_last : 0;
            uint32_t x = v >> (8 * (past & 3));
            if (in_row + 4 > KB)
                x = in_row < KB ? x & ((1u << (8 * (KB - in_row))) - 1) : 0;
            spread4(x, out);
        };
        uint32_t x_at[kStage], x_lds[kStage];
        int x_k[kStage];
#pragma unroll
        for (int i = 0; i < kStage; i++) {
            const int c = lane + 64 * i, col = c / kPer, k = c % kPer * 8;
            x_k[i] = col < COLS ? k : INT32_MAX / 2;
            x_at[i] = x0 + col * x_next + k * 2;
            x_lds[i] = min(col, COLS - 1) * kCol + k * 2;
        }
        auto load_x = [&](int i) {
            const int k0 = (i * WK + wk) * kValues;
#pragma unroll
            for (int c = 0; c < kStage; c++)
                xr[c] = buf16(rx, k0 + x_k[c] < K ? x_at[c] + k0 * 2 : kInvalid);
        };
        auto store_x = [&](int i) {
#pragma unroll
            for (int c = 0; c < kStage; c++)
                if (COLS * kPer % 64 == 0 || lane + 64 * c < COLS * kPer)
                    *(u32x4*)(lds + (i & 1) * kX + x_lds[c]) = xr[c];
            wave_sync();
        };
        const uint32_t col_at = (r < COLS ? r : 0) * kCol + q * (MX4 ? 64 : 16);
#pragma unroll
        for (int rb = 0; rb < RB; rb++)
            acc[rb] = f32x4{0};
        load_x(turn(0));
        load_scales(turn(0), sc);
#pragma unroll
        for (int l = 0; l < LINES; l++)
            load_line(turn(0), l);
        for (int i = 0; i < steps; i++) {
            const int next = turn(i + 1);
            store_x(i);
            load_x(next);
            load_scales(next, next_sc);
            const char* const xb = lds + (i & 1) * kX + col_at;
            uint32_t scale[RB][4];
            if constexpr (MX4)
#pragma unroll
                for (int rb = 0; rb < RB; rb++)
                    row_scales(turn(i), rb, sc[rb], scale[rb]);
#pragma unroll
            for (int l = 0; l < LINES; l++) {
                u32x4 wv[RB][2];
#pragma unroll
                for (int rb = 0; rb < RB; rb++) {
                    if constexpr (MX4)
                        wv[rb][0] = w[l][rb][0], wv[rb][1] = w[l][rb][1];
                    else
                        own_rows(r < 8, w[l][rb][0], w[l][rb][1], wv[rb]);
                }
                if constexpr (!MX4)
                    load_line(next, l);
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int f = 0; f < F; f++) {
                        const bf16x8 xf = __builtin_bit_cast(
                            bf16x8, *(const u32x4*)(xb + (2 * l + h) * (MX4 ? 256 : 64) + f * 16));
#pragma unroll
                        for (int rb = 0; rb < RB; rb++) {
                            bf16x8 wf;
                            if constexpr (MX4)
                                wf = widen(wv[rb][h][f], __builtin_bit_cast(float, __builtin_amdgcn_ubfe(
                                                             scale[rb][2 * l + h], 8 * q, 8) << 23));
                            else
                                wf = __builtin_bit_cast(bf16x8, wv[rb][h]);
                            acc[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf, acc[rb], 0, 0, 0);
                        }
                    }
                if constexpr (MX4)
                    load_line(next, l);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int rb = 0; rb < RB; rb++)
                sc[rb] = next_sc[rb];
        }
    }
};

// h of choice blockIdx.y: a block takes 4 / WK times 16 inputs and their gates.
template <bool MX4, int WK, int ACT>
__global__ void __launch_bounds__(256) lone_first_kernel(FewArgs p) {
    using S = Lone<MX4, 2, 1>;
    constexpr int NW = 4, WR = NW / WK;
    __shared__ __attribute__((aligned(16))) char smem[NW][S::kLds];
    __shared__ f32x4 sum[NW][2][4];
    const int pair = blockIdx.y;
    if (blockIdx.x == 0 && pair == 0 && threadIdx.x == 0)
        *(int32_t*)p.ws = 0;                           // the error word
    const int e = scalar_read(p.ids + pair);
    if ((uint32_t)e >= (uint32_t)p.E)
        return;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int units = p.I / 16;
    const int unit = min((int)blockIdx.x * WR + wave / WK, units - 1);
    const uint32_t token = (uint32_t)pair * p.k_magic >> 16;
    // a finishing thread's row of its unit, and what it needs there
    const int mu = blockIdx.x * WR + threadIdx.x / 16, mr = threadIdx.x % 16;
    const bool finishes = threadIdx.x < 16 * WR && mu < units;
    float v[2] = {0, 0}, prob = 0;
    if (finishes) {
        prob = p.prob[pair];
        if (p.bias1)
#pragma unroll
            for (int rb = 0; rb < 2; rb++)
                v[rb] = p.bias1[(int64_t)e * 2 * p.I + mu / 2 * 64 + mu % 2 * 16 + 32 * rb + mr];
    }
    f32x4 acc[2];
    S::run(smem[wave], p.w1, p.sf1, p.E, 2 * p.I, p.H, e, unit / 2 * 64 + unit % 2 * 16, 32, make_rsrc(p.x),
           token * (uint32_t)p.ldx * 2, 0, wave % WK, WK, blockIdx.x + e, acc);
    if (r == 0)
#pragma unroll
        for (int rb = 0; rb < 2; rb++)
            sum[wave][rb][q] = acc[rb];
    __syncthreads();
    if (!finishes)
        return;
#pragma unroll
    for (int rb = 0; rb < 2; rb++)
#pragma unroll
        for (int i = 0; i < WK; i++)
            v[rb] += sum[threadIdx.x / 16 * WK + i][rb][mr >> 2][mr & 3];
    const float g = p.act.gate_first ? v[0] : v[1];
    float h = act_forward<ACT>(g, p.act.gate_first ? v[1] : v[0], p.act) * prob;
    uint16_t* at = (uint16_t*)(p.ws + kWsHeader) + (int64_t)pair * p.I + mu * 16 + mr;
    for (int part = 0; part < p.parts; part++, at += (int64_t)p.T * p.k * p.I) {
        *at = f32_to_bf16(part_of(h));
        h = less_part(h);
    }
}

// y[t], in place of the second pass and the sum: a block takes 16 rows of the
// token's experts, its waves a choice each, or one of WK parts of it.
template <bool MX4, int DT>
__global__ void __launch_bounds__(64 * kLoneK) lone_second_kernel(FewArgs p, int WK) {
    constexpr int NW = kLoneK, PARTS = DT == GG_F32 ? 3 : 2;
    using S = Lone<MX4, 1, PARTS>;
    __shared__ __attribute__((aligned(16))) char smem[NW][S::kLds];
    __shared__ f32x4 sum[NW][PARTS][4];
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int t = blockIdx.y, row0 = 16 * blockIdx.x, wk = wave % WK, j = wave / WK;
    const int pair = t * p.k + min(j, p.k - 1);
    const int e = scalar_read(p.ids + pair);
    f32x4 acc[1] = {f32x4{0}};
    if (j < p.k && (uint32_t)e < (uint32_t)p.E) {
        f32x4 bias = {0};
        if (p.bias2 && wk == 0) {
            const float prob = p.prob[pair];
            const float* const from = p.bias2 + (int64_t)e * p.H + row0 + 4 * q;
#pragma unroll
            for (int i = 0; i < 4; i++)
                bias[i] = prob * from[i];
        }
        S::run(smem[wave], p.w2, p.sf2, p.E, p.H, p.I, e, row0, 0, make_rsrc(p.ws + kWsHeader),
               (uint32_t)pair * p.I * 2, (uint32_t)(p.T * p.k) * p.I * 2, wk, WK, blockIdx.x + wave, acc);
        if (r == 0)
            acc[0] += bias;
    }
    if (r < PARTS)
        sum[wave][r][q] = acc[0];
    __syncthreads();
    if (threadIdx.x < 16) {
        const int c = threadIdx.x;
        float y = 0.0f, of_first = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; i++) {
            of_first += sum[i][0][c >> 2][c & 3];
#pragma unroll
            for (int part = 0; part < PARTS; part++)
                y += sum[i][part][c >> 2][c & 3];
        }
        y = over_parts(y, of_first);
        const int64_t at = t * p.ldy + row0 + c;
        if constexpr (DT == GG_F32)
            ((float*)p.y)[at] = y;
        else
            ((uint16_t*)p.y)[at] = (uint16_t)from_f32<DT>(y);
    }
}

// Calls f(Few<...>()) with a block's shape for `units` pairs of row blocks, of rows
// of K, of `active` experts (at most) and about `cols` columns of each.
//  * Eight waves and room for 32 columns where more than `room` are likely and there
//    are blocks enough (both passes, us, against four waves: 64 tokens, 8 of 64
//    experts of 4096 x 2048 in bf16 553 and 622; 26 tokens, 7 of 8 of 4736 x 1184 in
//    MXFP4 62 and 83; short rows need more blocks: 17 tokens, 4 of 8 of 2528 x 320
//    in MXFP4, 79 of them in the second pass, 31 and 23).
//  * Four waves for MXFP4; two for bf16 (two and four: 18 tokens, 7 of 60 of 5120 x
//    1728, 517 and 537; 15 tokens, 6 of 32 of 4224 x 672, 112 and 123), where an
//    expert's last block of four would have two or three waves idle (52 tokens, 8 of
//    128 of 6112 x 416 in MXFP4 172 and 184), and where blocks of four would be fewer
//    than half the CUs (46 tokens, 5 of 8 of 1888 x 1216 in bf16 52 and 62).
//  * Fewer blocks and columns: parts of the reduction axis (3 tokens over 8 experts
//    of 2048 x 1024 in bf16, first and second pass: 18.4 + 10.2 undivided, 12.4 + 6.6
//    in two, 13.2 + 8.0 in four; 3 tokens, 6 of 16 of 5696 x 256 38 in two and 29 in
//    four), as far as the columns fit and the parts have a piece each.
template <bool MX4, class F>
void for_shape(int units, int K, int active, int cols, int room, F f) {
    const int cus = cu_count();
    const int64_t blocks = (int64_t)((units + 3) / 4) * active, wide = (int64_t)units * active / 8;
    const int pieces = (K + (MX4 ? 511 : 255)) / (MX4 ? 512 : 256);
    const int idle = -units & 3;                       // waves of an expert's last block of 4
    if (cols > room && wide >= (pieces < 4 ? cus / 2 : cus / 4))
        return f(Few<MX4, 8, 1, 2>());
    if constexpr (MX4)
        if (blocks >= cus / 2 && (cols > 8 || pieces < 2 || blocks >= cus * 3 / 4) && (idle < 2 || units >= 32))
            return f(Few<MX4, 4, 1, 1>());
    if (blocks >= cus * 3 / 4 || cols > 8 || pieces < 2)
        f(Few<MX4, 2, 1, 1>());
    else if (blocks * 2 >= cus * 3 / 4 || cols > 4 || pieces < 4)
        f(Few<MX4, 4, 2, 1>());
    else
        f(Few<MX4, 4, 4, 1>());
}

}  // namespace

size_t few_workspace(int64_t T, int64_t k, int64_t H, int64_t I) {
    return kWsHeader + few_h_bytes(T * k, I) + (size_t)(T * k * H * 4);
}

// Reports a pass: rows x choices of a block, its waves, and which kernel it is (parts
// of the reduction axis as "K in", of h as "h in").
template <class... Args>
static void few_info(LaunchInfo* info, int pass, int tm, int tn, int waves, dim3 grid, const char* format,
                     Args... args) {
    if (!info)
        return;
    info += pass;
    snprintf(info->kernel, sizeof info->kernel, format, args...);
    info->tm = tm;
    info->tn = tn;
    info->waves = waves;
    info->grid = (int64_t)grid.x * grid.y;
}
static const char* few_name(bool mx4) { return dtype_name(mx4 ? GG_MXFP4 : GG_BF16); }

// Both passes for choices that go each for itself.  WK of the first: parts of the
// reduction axis until half of the CUs have a block (blocks undivided, us with 1, 2
// and 4 parts, MXFP4: 256, 49.1 48.5 48.7; 132, 22.9 24.3 23.8; 64, 14.9 13.3 13.7; 32, 18.0
// 15.6 13.8.  bf16: 127 128 142; 50 53 52; 22 18 17; 30 22 19).
template <bool MX4>
void launch_lone(const FewArgs& p, hipStream_t s, LaunchInfo* info) {
    using std::integral_constant;
    const int units = p.I / 16, pairs = p.T * p.k, enough = cu_count() / 2;
    auto first = [&](auto WKc) {
        constexpr int WK = decltype(WKc)::value;
        const dim3 grid((units * WK + 3) / 4, pairs);
        few_info(info, 0, 128 / WK, 1, 4, grid, "lone_first_kernel<%s, K in %d>", few_name(MX4), WK);
        for_act(p.act.act, [&](auto ACT) {
            hipLaunchKernelGGL((lone_first_kernel<MX4, WK, decltype(ACT)::value>), grid, dim3(256), 0, s, p);
        });
    };
    const int blocks = units * pairs / 4;
    if (blocks >= enough)
        first(integral_constant<int, 1>());
    else if (blocks * 2 >= enough)
        first(integral_constant<int, 2>());
    else
        first(integral_constant<int, 4>());
    int wk = 1;                                        // of the second: what k leaves
    while (2 * wk * p.k <= kLoneK)
        wk *= 2;
    const dim3 grid(p.H / 16, p.T);
    few_info(info, 1, 16, p.k, kLoneK, grid, "lone_second_kernel<%s, K in %d, h in %d>", few_name(MX4), wk, p.parts);
    auto second = [&](auto DT) {
        hipLaunchKernelGGL((lone_second_kernel<MX4, decltype(DT)::value>), grid, dim3(64 * kLoneK), 0, s, p, wk);
    };
    if (p.y_dtype == GG_BF16)
        second(integral_constant<int, GG_BF16>());
    else if (p.y_dtype == GG_F16)
        second(integral_constant<int, GG_F16>());
    else
        second(integral_constant<int, GG_F32>());
}

hipError_t launch_few(const FewArgs& args, hipStream_t s, LaunchInfo* info) {
    FewArgs p = args;
    const int pairs = p.T * p.k;
    if (p.T == 0) {
        hipLaunchKernelGGL(few_none_kernel, dim3(1), dim3(64), 0, s, (int32_t*)p.ws);
        return hipGetLastError();
    }
    p.parts = p.y_dtype == GG_F32 ? 3 : 2;
    p.k_magic = 65536u / p.k + 1;
    // Columns that an expert is likely to have: its share and one and a half times
    // that one's root, at most one a token.  (More take another pass over its
    // weights.)
    const double share = (double)pairs / p.E;
    const int likely = (int)ceil(share + 1.5 * sqrt(share)), cols = likely < p.T ? likely : p.T;
    const int active = pairs < p.E ? pairs : p.E;
    if (lone(p)) {
        p.mx4 ? launch_lone<true>(p, s, info) : launch_lone<false>(p, s, info);
        return hipGetLastError();
    }
    auto by_weights = [&](auto MX4) {
        constexpr bool mx4 = decltype(MX4)::value;
        // (bf16: eight waves from 9 columns on for long rows, as above; 63 tokens, 6 of
        // 64 experts of 768 x 576, 56 us and 49 without)
        for_shape<mx4>(p.I / 16, p.H, active, cols, mx4 || p.H < 2048 ? 16 : 8, [&](auto shape) {
            using C = decltype(shape);
            const dim3 grid((p.I / 16 + C::WR - 1) / C::WR, active);
            few_info(info, 0, 32 * C::WR, C::XC, C::NW, grid, "few_kernel<%s, first, K in %d>", few_name(mx4), C::WK);
            for_act(p.act.act, [&](auto ACT) {
                hipLaunchKernelGGL((few_kernel<C, decltype(ACT)::value, 1>), grid, dim3(C::kThreads), 0, s, p);
            });
        });
        for_shape<mx4>(p.H / 32, p.I, active, cols * p.parts, 16, [&](auto shape) {
            using C = decltype(shape);
            const dim3 grid((p.H / 32 + C::WR - 1) / C::WR, active);
            few_info(info, 1, 32 * C::WR, C::XC / p.parts, C::NW, grid,
                     "few_kernel<%s, second, K in %d, h in %d>, few_sum_kernel", few_name(mx4), C::WK, p.parts);
            if (p.parts == 2)
                hipLaunchKernelGGL((few_kernel<C, -1, 2>), grid, dim3(C::kThreads), 0, s, p);
            else
                hipLaunchKernelGGL((few_kernel<C, -1, 3>), grid, dim3(C::kThreads), 0, s, p);
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
