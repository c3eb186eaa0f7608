// gg_moe_few.hip -- a whole mixture-of-experts layer for up to 64 tokens
// (gg_moe_few): every weight of a chosen expert is read once, so the layer
// costs what reading them costs.
//
// Two passes of one kernel, then the sum over a token's choices:
//   first    c = w1_e x, h = prob act(c + bias1), for every (token, choice)
//   second   w2_e h + prob bias2, for every (token, choice)
// (The sum by the last block of some rows, which saves the launch, took longer:
// every block then awaits its results and counts itself, 5 us of one token's
// second pass for the 4 of the launch, 60 us of 64 tokens'.)
// A wave takes 32 rows of one chosen expert's matrix (in the first pass 16 input
// rows and the 16 gate rows that go with them) and streams them from memory into
// the registers that the matrix instruction reads, as its 16-row operand
// (16x16x32, bf16); 4-bit weights are widened to bf16, which holds each exactly.
// The tokens of the expert are the 16 columns, from LDS, where the block's waves
// share them.  The waves of a block have different rows, or, where there are too
// few rows to fill the device, WK of them the same rows and parts of the
// reduction axis, added up in LDS.
//
// What a CU's load path takes is lines: a vector load of 8 rows x 128 bytes
// costs half of one of 16 rows x 64 bytes.  So 16 rows x 128 bytes come in two
// loads of 8 whole lines, and lanes r and r + 8 of every 16 then exchange a half
// (a DPP move a register), which leaves each lane 16-byte pieces of its own row.
// The scales of 4 lines (32 bytes of a row) come in one load, 8 bytes a lane, and
// go to the lanes by row swaps.
//
// h is kept as the sum of `parts` bf16 values, 2 for a 16-bit y (16 bits of h),
// 3 for an fp32 one (24 bits): the second pass takes them as so many columns and
// adds the columns' results up.
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
    const int start = (blockIdx.x + blockIdx.y) % steps;
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
                    *(u32x2*)at = u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
#pragma unroll
                    for (int i = 0; i < 4; i++)        // (nothing is left of an infinity)
                        h[i] = fabsf(h[i]) < INFINITY ? h[i] - bf16_to_f32(f32_to_bf16(h[i])) : 0.0f;
                }
            }
        } else {
            for (int it = threadIdx.x; it < C::WR * here * 8; it += C::kThreads) {
                const Item m = item(it);
                if (m.u >= units)
                    continue;
                const Extra x = it < C::kThreads ? early : extra(m);
                f32x4 v = total(m.wrow, m.rb, m.q, m.which);
#pragma unroll
                for (int part = 1; part < PARTS; part++)
                    v += total(m.wrow, m.rb, m.q, part * kPass + m.which);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    v[i] = fmaf(x.prob, x.bias[0][i], v[i]);
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

// Calls f(Few<...>()) with a block's shape for `rows` rows of `active` experts
// (at most) and about `cols` columns of each: parts of the reduction axis until
// three quarters of the CUs have a block, as far as the columns then fit (3
// tokens over 8 experts of 2048 x 1024 in bf16, first and second pass: 18.4 + 10.2
// us undivided, 12.4 + 6.6 in two, 13.2 + 8.0 in four; one token over 64 of 4096 x
// 2048 in MXFP4, 256 blocks undivided: 17.5 + 11.1, 18.7 + 11.4, 20.2 + 14.0); room
// for 32 columns where 16 are too few.
template <bool MX4, class F>
void for_shape(int rows, int active, int cols, F f) {
    const int64_t blocks = (int64_t)(rows / 32) * active / 4, enough = cu_count() * 3 / 4;
    if (cols > 16)
        f(Few<MX4, 8, 1, 2>());
    else if (blocks >= enough || cols > 8)
        f(Few<MX4, 4, 1, 1>());
    else if (blocks * 2 >= enough || cols > 4)
        f(Few<MX4, 4, 2, 1>());
    else
        f(Few<MX4, 4, 4, 1>());
}

}  // namespace

size_t few_workspace(int64_t T, int64_t k, int64_t H, int64_t I) {
    return kWsHeader + few_h_bytes(T * k, I) + (size_t)(T * k * H * 4);
}

hipError_t launch_few(const FewArgs& args, hipStream_t s, LaunchInfo* info) {
    FewArgs p = args;
    const int pairs = p.T * p.k;
    if (p.T == 0)
        return hipSuccess;
    p.parts = p.y_dtype == GG_F32 ? 3 : 2;
    p.k_magic = 65536u / p.k + 1;
    // Columns that an expert is likely to have: twice its share and a few more,
    // at most one a token.  (More take another pass over its weights.)
    const int share = pairs / p.E * 2 + 4, cols = share < p.T ? share : p.T;
    const int active = pairs < p.E ? pairs : p.E;
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "few_kernel<%s> x 2 + sum", p.mx4 ? "mxfp4" : "bf16");
        info->tm = 128;
        info->tn = cols;
        info->waves = 4;
        info->grid = (int64_t)(p.I / 64) * active;
    }
    auto by_weights = [&](auto MX4) {
        constexpr bool mx4 = decltype(MX4)::value;
        for_shape<mx4>(2 * p.I, active, cols, [&](auto shape) {
            using C = decltype(shape);
            const dim3 grid((p.I / 16 + C::WR - 1) / C::WR, active);
            for_act(p.act.act, [&](auto ACT) {
                hipLaunchKernelGGL((few_kernel<C, decltype(ACT)::value, 1>), grid, dim3(C::kThreads), 0, s, p);
            });
        });
        for_shape<mx4>(p.H, active, cols * p.parts, [&](auto shape) {
            using C = decltype(shape);
            const dim3 grid((p.H / 32 + C::WR - 1) / C::WR, active);
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
