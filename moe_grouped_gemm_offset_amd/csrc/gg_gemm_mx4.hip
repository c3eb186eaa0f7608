// gg_gemm_mx4.hip -- the grouped product of MXFP4 rows and weights
// (gg_gemm_mx4): d = alpha_g deq(a) deq(b_g)^T + bias_g over ragged groups.
//
// Two kernels (shape_of has the rule and what both measured):
//  * gemm_kernel, tiles of 128 x 128 or 256 x 256 on the two-buffer main loop of the
//    8-bit kernels.  v_mfma_scale_f32_32x32x64_f8f6f4 takes 4-bit operands at twice
//    the 8-bit rate: a lane supplies one block of 32 values, 16 bytes, so a
//    64-byte stage of a row is 128 values in two steps, and a load unit 256.  A
//    CU has two of the small tiles at a time, one's start and end under the
//    other's products, and reads twice the bytes a product; the large tile has
//    the fewest.  64 groups of 4096 x 4096: 65536 rows 664 us (3310 TFLOP/s; the
//    matrix instructions take half of a block's clocks: 3.3k clocks a unit for 2.05k of
//    them, 15k a tile for its start and end), 512 rows 100 us (5.8 TB/s of weights).
//  * thin_kernel, for so few tiles that most CUs would have none: the reduction
//    axis in four, the weights going from memory into the operand registers (as
//    in gg_moe_few.hip).
// Groups have any number of rows: every block counts the tiles of the groups
// (a scan over the ends by each of its waves) and finds its own.
#include <cmath>
#include <type_traits>

#include "gg_forward.hpp"
#include "gg_lane.hpp"
#include "gg_stream.hpp"

namespace gg {

namespace {

// ---- tiles of ragged groups --------------------------------------------------

struct TileAt {
    int g;                    // group, -1: none
    int m0, rows;             // first row and rows of the tile (at most TM)
    int nt;                   // tile of columns
};

// v of the lane D before within 16 (first 15: 0), of lane 15 of the 16 lanes
// before, of lane 31: the steps of a scan over the wave in the vector ALU.
template <int CTRL, int ROWS>
__device__ __forceinline__ int step_from(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// Inclusive scan over the lanes of a wave, of values that 0 leaves as they are.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, step_from<0x111, 0xF>(v));
    v = op(v, step_from<0x112, 0xF>(v));
    v = op(v, step_from<0x114, 0xF>(v));
    v = op(v, step_from<0x118, 0xF>(v));
    v = op(v, step_from<0x142, 0xA>(v));               // row_bcast:15
    return op(v, step_from<0x143, 0xC>(v));            // row_bcast:31
}

// Tile of block `q` where groups are cut into tiles of TM rows and tiles_n
// columns.  Ends are taken as a running maximum within 0 .. m_rows, so ranges
// are disjoint and in bounds whatever the array holds.  Lane l of every wave
// has groups l * per .. ; per is 1 up to 64 groups.  Blocks of one XCD (every
// eighth) get neighbouring tiles, in bands of 4 tiles of rows within a group.
template <int TM>
__device__ __forceinline__ TileAt tile_at(const int32_t* ends, int L, int m_rows, int tiles_n, int q) {
    const int lane = threadIdx.x & 63, per = (L + 63) >> 6, g0 = lane * per;
    auto end_of = [&](int g) { return min(max(ends[g], 0), m_rows); };
    // (unsigned: a group of 2^31 - 1 rows and TM - 1 more)
    auto tiles_of = [](int rows) { return (int)(((uint32_t)rows + TM - 1) / TM); };
    int top = 0;
    for (int i = 0; i < per; i++)
        if (g0 + i < L)
            top = max(top, end_of(g0 + i));
    top = wave_scan(top, [](int a, int b) { return max(a, b); });
    int start = __shfl_up(top, 1);                     // where the lane's first group begins
    start = lane ? start : 0;
    int tiles = 0;
    if (per == 1) {
        tiles = tiles_of(top - start);
    } else {
        for (int i = 0, at = start; i < per; i++)
            if (g0 + i < L) {
                const int end = max(at, end_of(g0 + i));
                tiles += tiles_of(end - at);
                at = end;
            }
    }
    const int upto = wave_scan(tiles, [](int a, int b) { return a + b; });
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
    int begin = __builtin_amdgcn_readlane(start, owner), end = __builtin_amdgcn_readlane(top, owner);
    int n = tiles_of(end - begin), g = owner * per;
    if (per > 1)
        for (end = begin; g < L; g++) {
            end = max(begin, uniform(end_of(g)));
            n = tiles_of(end - begin);
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

using BigTile = Cfg<256, 256, 2, 2>;
using SmallTile = Cfg<128, 128, 2, 2>;

// Scales of 8 stages (32 bytes of every tile row, 4 load units) at a time, in two
// alternating buffers behind the unit buffers: row r of A in slot r, of B in slot
// TM + r.  A wave's load moves the 32 bytes of 32 rows, two lanes a row; units
// 4g + 1 .. 4g + 4 carry 64 rows of A and of B each of group g + 1.  (16 bytes of 64 rows a
// load, as many loads, cost the load path twice the lines: a third of all that a
// unit takes.)  The two halves of a slot change places in every second 8 rows, so
// that the words of 32 rows are read with 2-way bank conflicts.
template <class C>
struct Scales4 {
    static constexpr int kBuf = (C::TM + C::TN) * 32, kBase = 2 * C::kUnit;
    static constexpr int kSmem = kBase + 2 * kBuf > C::kLds ? kBase + 2 * kBuf : C::kLds;
    static constexpr int kSlices = C::TM / 64;         // units that carry a group
    static_assert(C::TM == C::TN && kSlices <= 4 && C::kWaves == 4, "a wave's load is 32 rows");
};

template <class C>
struct FragMx4 {
    u32x4 a[2][C::MB], b[2][C::NB];                    // the two steps of a stage
    uint32_t sa[C::MB], sb[C::NB];                     // scale words, as read
};

__device__ __forceinline__ i32x8 low4(u32x4 v) {
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// acc[i][j] += the transpose of the wave's (32 i, 32 j) block of deq(a) deq(b)^T
// (a lane then owns a row of the block and four consecutive columns a register
// group) over K values of rows whose codes are K / 2 bytes apart (scales K / 32);
// rows past rows_valid / cols_valid count as zeros.
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
    // Slice s of a group: rows 64 s + 32 (w & 1) + l / 2 of A (waves 0 and 1) and of
    // B (2 and 3).  (What is past a row's end belongs to no stage.)
    const bool of_a = wu < 2;
    const int valid = of_a ? (rows_valid < TM ? rows_valid : TM) : (cols_valid < TN ? cols_valid : TN);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(uniform_ptr(of_a ? sfa : sfb), (uint32_t)uniform(valid * (int)KB));
    const uint32_t sc_lds = lds_addr(smem) + S::kBase + (of_a ? 0 : TM * 32) + (wu & 1) * 1024;
    const uint32_t sc_off = (uint32_t)(32 * (wu & 1) + (l >> 1)) * KB + 16 * ((l ^ l >> 4) & 1);
    auto scale_load = [&](int grp, int s) {
        dma16(rs, sc_lds + (grp & 1) * S::kBuf + s * 2048, sc_off + s * 64 * KB + 32 * grp);
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
            scale_load(u > 0 ? (u - 1) / 4 + 1 : 0, u > 0 ? (u - 1) % S::kSlices : 0);
    };
    const uint32_t sh = 8 * lq;
    const int sc_a = (am0 + lr) * 32, sc_b = (TM + bn0 + lr) * 32, sc_half = lr << 1 & 16;
    auto read = [&](const char* st, int kt, FragMx4<C>& f, int g) {
        const bool is_a = g < MB;
        const int r = is_a ? am0 + 32 * g + lr : bn0 + 32 * (g - MB) + lr;
        const char* s = is_a ? st : st + TM * kRowBytes;
        const u32x4 x0 = ld_lds16(s, lds_off(r, 4 * (kt & 1) + lq));
        const u32x4 x1 = ld_lds16(s, lds_off(r, 4 * (kt & 1) + 2 + lq));
        // (word w of a slot is in its half (w / 4) ^ (row / 8 % 2))
        const char* base = smem + S::kBase + ((kt >> 3) & 1) * S::kBuf + 4 * (kt & 3);
        int at = (is_a ? sc_a + 1024 * g : sc_b + 1024 * (g - MB)) + ((kt << 2 & 16) ^ sc_half);
        if constexpr (ODD) {
            // past an odd number of stages: a word of the codes, which are zeros
            // there (the next row's scales, which the loads bring, may be NaN's)
            base = kt < nk ? base : st + lds_off(0, 4);
            at = kt < nk ? at : 0;
        }
        const uint32_t word = *reinterpret_cast<const uint32_t*>(base + at);
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
                    low4(f.b[0][j]), low4(f.a[0][i]), acc[i][j], 4, 4, 0, sb, 0, sa);
            else
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    low4(f.b[1][j]), low4(f.a[1][i]), acc[i][j], 4, 4, 2, sb, 2, sa);
        }
    };
    FragMx4<C> frag[2];
#pragma unroll
    for (int i = 0; i < S::kSlices; i++)
        scale_load(0, i);
    pipeline<C, kLA + kLB + 1, 2 * MB * NB, MB + NB>(smem, nk, frag, issue, read, mma);
}

template <class C, int DT, bool ODD, bool BIAS>
__global__ void __launch_bounds__(C::kThreads, C::TM == 256 ? 1 : 2) gemm_kernel(GemmMx4Args p) {
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
    // Rounded, then through the wave's own region of LDS, so that a store has whole
    // lines: kLanes lanes the 128 or 256 bytes of a row of the wave's.  Rows and columns off the tile are masked by
    // the descriptor.  (Against staging fp32 and rounding behind it, a third of the
    // LDS instructions: a tile of 256 x 256 5k clocks, 9k where every CU writes, for 15k.)
    constexpr int kSize = DT == GG_F32 ? 4 : 2, kJ = NB < 8 / kSize ? NB : 8 / kSize, kPasses = NB / kJ;
    constexpr int kRow = 32 * kJ * kSize, kPitch = kRow + 16, kRows = TM / C::WM, kWave = kRows * kPitch;
    constexpr int kLanes = kRow / 16, kAtOnce = 64 / kLanes;   // of a row; rows a store
    static_assert(C::kWaves * kWave <= Scales4<C>::kSmem, "the waves' regions");
    char* const lds = smem + w * kWave;
    const int lane = threadIdx.x & 63, lr = lane & 31, lq = lane >> 5;
    const uint32_t pitch = (uint32_t)p.N * kSize;
    const int left = rows - am0 < 0 ? 0 : (rows - am0 < kRows ? rows - am0 : kRows);
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(uniform_ptr((char*)p.d + (m0 + am0) * pitch),
                                                (uint32_t)uniform((int)(left * pitch)));
#pragma unroll
    for (int pass = 0; pass < kPasses; pass++) {
#pragma unroll
        for (int jj = 0; jj < kJ; jj++) {
            const int j = pass * kJ + jj, col = n0 + bn0 + 32 * j + 4 * lq;
            f32x4 bias[4];
#pragma unroll
            for (int g4 = 0; g4 < 4; g4++)
                if constexpr (BIAS) {
                    const float* const from = p.bias + (int64_t)g * p.N + (col < p.N ? col + 8 * g4 : 0);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        bias[g4][k] = from[k];
                }
#pragma unroll
            for (int i = 0; i < MB; i++)
#pragma unroll
                for (int g4 = 0; g4 < 4; g4++) {
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        v[k] = BIAS ? fmaf(alpha, acc[i][j][4 * g4 + k], bias[g4][k]) : alpha * acc[i][j][4 * g4 + k];
                    char* const at = lds + (32 * i + lr) * kPitch + (32 * jj + 8 * g4 + 4 * lq) * kSize;
                    if constexpr (DT == GG_F32)
                        *(f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
                    else if constexpr (DT == GG_BF16)
                        *(u32x2*)at = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    else
                        *(u32x2*)at = u32x2{(uint32_t)f32_to_f16(v[0]) | (uint32_t)f32_to_f16(v[1]) << 16,
                                            (uint32_t)f32_to_f16(v[2]) | (uint32_t)f32_to_f16(v[3]) << 16};
                }
        }
        wave_sync();
        const int col = n0 + bn0 + 32 * kJ * pass + 16 / kSize * (lane % kLanes);
        const uint32_t at = lane / kLanes * pitch + (uint32_t)col * kSize;
#pragma unroll
        for (int i = 0; i < kRows; i += kAtOnce) {
            typedef int i32x4 __attribute__((ext_vector_type(4)));
            const i32x4 v = *(const i32x4*)(lds + (i + lane / kLanes) * kPitch + 16 * (lane % kLanes));
            __builtin_amdgcn_raw_buffer_store_b128(v, rd, col < p.N ? at + i * pitch : kInvalid, 0, 2);
        }
        wave_sync();                                   // the region is free again
    }
}

// ---- the thin kernel ---------------------------------------------------------

constexpr int kThinWaves = 4, kThinThreads = 64 * kThinWaves;

// 32 rows of the weights and NB blocks of 16 rows of a to a block, a quarter of the
// reduction axis to a wave, in pieces of 2 lines (512 values) of each row; the next
// piece's loads go into the registers that a line leaves.  The waves' sums are
// added up in LDS.
//
// What a CU's load path takes is lines, so every load is one of whole lines: codes
// 8 rows x 128 bytes (own_rows brings each lane its own row's), scales as 8 rows x
// 128 bytes for 8 pieces, through a region of LDS of the wave's own.
template <int NB>
__global__ void __launch_bounds__(kThinThreads, 2) thin_kernel(GemmMx4Args p) {
    constexpr int WK = kThinWaves, kCols = 32, kBlocks = 2 + NB;             // (two blocks of b, NB of a)
    constexpr int kAhead = 8, kPitch = 16 * kAhead + 16;                     // pieces of scales; a row of them in LDS
    constexpr int kScales = 16 * kBlocks * kPitch, kSum = 2 * NB * 1024;
    __shared__ __attribute__((aligned(16))) char smem[kThinWaves][kScales > kSum ? kScales : kSum];
    check_ends(p);
    const TileAt t = tile_at<16 * NB>(p.ends, p.L, (int)p.m_rows, (p.N + kCols - 1) / kCols, blockIdx.x);
    if (t.g < 0)
        return;
    const int g = uniform(t.g), rows = uniform(t.rows);
    const int64_t m0 = uniform(t.m0);
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int n0 = uniform(t.nt) * kCols;
    const uint32_t pitch = p.K / 2, KB = p.K / 32;
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(uniform_ptr(weights_at(p, g, n0)), 32 * pitch);
    const __amdgpu_buffer_rsrc_t rsw = make_rsrc(uniform_ptr(scales_at(p, g, n0)), 32 * KB);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(uniform_ptr((const char*)p.a + m0 * pitch), rows * pitch);
    const __amdgpu_buffer_rsrc_t rsx = make_rsrc(uniform_ptr((const char*)p.sfa + m0 * KB), rows * KB);
    const int pieces = (p.K + 511) / 512, steps = (pieces + WK - 1) / WK;
    const int first = wave * steps;                     // the wave's pieces: first .. first + steps - 1
    // block c: rows 16 c .. of the weights, then of a
    auto rsrc = [&](int c) { return c < 2 ? rw : rx; };
    auto scale_rsrc = [&](int c) { return c < 2 ? rsw : rsx; };
    auto row_of = [&](int c, int row) { return (uint32_t)(c < 2 ? 16 * c + row : 16 * (c - 2) + row); };

    u32x4 v[2][kBlocks][2], sv[kBlocks][2];
    // Line j of piece i: rows 8 h + r % 8, 16 bytes at 16 (q + 4 (r / 8)).  (Past the
    // rows of a: zeros.  Past the row's end, where no step uses it, whatever the
    // next row has there.)
    const uint32_t lane_at = (r & 7) * pitch + 16 * (q + 4 * (r >> 3));
    auto load_line = [&](int i, int j) {
        const uint32_t at = lane_at + (uint32_t)i * 256 + 128 * j;
#pragma unroll
        for (int c = 0; c < kBlocks; c++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                v[j][c][h] = buf16(rsrc(c), row_of(c, 8 * h) * pitch + at);
    };
    // The scales of pieces i .. i + 7: rows 8 h + lane / 8, those of piece i + lane % 8.
    auto load_scales = [&](int i) {
        const uint32_t at = (lane >> 3) * KB + (uint32_t)(i + (lane & 7)) * 16;
#pragma unroll
        for (int c = 0; c < kBlocks; c++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                sv[c][h] = buf16(scale_rsrc(c), row_of(c, 8 * h) * KB + at);
    };
    auto store_scales = [&] {
#pragma unroll
        for (int c = 0; c < kBlocks; c++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                *(u32x4*)(smem[wave] + (16 * c + 8 * h + (lane >> 3)) * kPitch + 16 * (lane & 7)) = sv[c][h];
        wave_sync();
    };
    f32x4 acc[2][NB];
#pragma unroll
    for (int rb = 0; rb < 2; rb++)
#pragma unroll
        for (int b = 0; b < NB; b++)
            acc[rb][b] = f32x4{0};
    load_scales(first);
    load_line(first, 0);
    load_line(first, 1);
    for (int i0 = first; i0 < first + steps; i0 += kAhead) {
        store_scales();
        load_scales(i0 + kAhead);
        const int end = min(i0 + kAhead, first + steps);
        for (int i = i0; i < end; i++) {
            u32x4 sc[kBlocks];
#pragma unroll
            for (int c = 0; c < kBlocks; c++)
                sc[c] = *(const u32x4*)(smem[wave] + (16 * c + r) * kPitch + 16 * (i - i0));
            // Halves of the piece within the row (its end is a multiple of one); past
            // them scales of 2^-127 on both sides, which leave nothing of any codes.
            const int halves = (int)(KB - (uint32_t)i * 16) / 4;
#pragma unroll
            for (int c = 0; c < kBlocks; c++)
#pragma unroll
                for (int h = 0; h < 4; h++)
                    sc[c][h] = h < halves ? sc[c][h] >> (8 * q) : 0;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                u32x4 own[kBlocks][2];
#pragma unroll
                for (int c = 0; c < kBlocks; c++)
                    own_rows(r < 8, v[j][c][0], v[j][c][1], own[c]);
                load_line(i + 1, j);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int b = 0; b < NB; b++)
#pragma unroll
                        for (int rb = 0; rb < 2; rb++)
                            acc[rb][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                low4(own[rb][h]), low4(own[2 + b][h]), acc[rb][b], 4, 4, 0,
                                (int)sc[rb][2 * j + h], 0, (int)sc[2 + b][2 * j + h]);
            }
        }
    }
    const float alpha = p.alpha ? p.alpha[g] : 1.0f;
    // register i of a lane: weight row 16 rb + 4 q + i, row 16 b + r of a
    auto store = [&](int rb, int b, f32x4 v) {
        const int row = 16 * b + r, col = n0 + 16 * rb + 4 * q;
        if (row >= rows)
            return;
        const float* const bias = p.bias ? p.bias + (int64_t)g * p.N + col : nullptr;
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = bias ? fmaf(alpha, v[i], bias[i]) : alpha * v[i];
        const int64_t at = (m0 + row) * p.N + col;
        if (p.d_dtype == GG_F32) {
            *(f32x4*)((float*)p.d + at) = v;
        } else {
            auto two = [&](float a, float b) {
                return p.d_dtype == GG_BF16 ? pack_bf16x2(a, b)
                                            : (uint32_t)f32_to_f16(a) | (uint32_t)f32_to_f16(b) << 16;
            };
            *(u32x2*)((uint16_t*)p.d + at) = u32x2{two(v[0], v[1]), two(v[2], v[3])};
        }
    };
    auto sum = [&](int w, int rb, int b) { return (f32x4*)smem[w] + (rb * NB + b) * 64 + lane; };
#pragma unroll
    for (int rb = 0; rb < 2; rb++)
#pragma unroll
        for (int b = 0; b < NB; b++)
            *sum(wave, rb, b) = acc[rb][b];
    __syncthreads();
    // block (rb, b) by wave rb NB + b
    if (wave < 2 * NB) {
        const int rb = wave / NB, b = wave % NB;
        f32x4 v = *sum(0, rb, b);
#pragma unroll
        for (int k = 1; k < WK; k++)
            v += *sum(k, rb, b);
        store(rb, b, v);
    }
}

// How a call is cut into tiles.  tn 32: thin_kernel.
struct Shape {
    int tm, tn;
    bool thin() const { return tn == 32; }
};

// Thin while its blocks do not outnumber the CUs (one group, thin and in tiles of
// 128: 16 rows of 8192 x 8192, 256 blocks, 12.5 and 24 us; 64 rows of 4096 x 4096,
// 256, 11.4 and 13.3; 96 rows, 384, 17 and 13; 4 groups of 16 rows, 512, 18.7 and
// 15.6).
// Else the tile for which the blocks take less, by what they take in us with u
// units of 256 values: of 256 x 256, one on a CU, 8 + 1.8 u; of 128 x 128, of which
// the next starts as soon as one of two ends, 2.1 + 0.57 u; with an fp32 d 11 and
// 2.7 in place of 8 and 2.1.  (In tiles of 256 and of 128: one group of 16384 rows,
// 4096 x 4096, 146 and 164 us, of 4096 rows, 2048 x 2048, 23 and 16; 8 groups, 8192
// rows, 4096 x 1024 46 and 34, 2048 x 2048 42 and 31; 64 groups of 4096 x 4096, 65536
// rows 660 and 786, 16384 rows 250 and 260, 512 rows 136 and 100; fp32, 8 groups,
// 5003 rows, 2080 x 1920, 26.0 and 24.0.)
// Where a launch does not hold the blocks of 128 x 128, 256 x 256 too.
// The rows of a group are known on the device only: counted as tiles are all the
// rows together and half a tile more for each group but one, and at least one a
// group.
Shape shape_of(const GemmMx4Args& p) {
    const double groups = (double)(p.m_rows < p.L ? p.m_rows : p.L), cus = cu_count(), units = p.K / 256.0;
    auto tiles = [&](int tm, int tn) {
        const double rows = (double)((p.m_rows + tm - 1) / tm) + (groups - 1) / 2;
        return (rows > groups ? rows : groups) * ((p.N + tn - 1) / tn);
    };
    const int tm = p.m_rows / p.L <= 16 ? 16 : 32;
    if (tiles(tm, 32) <= cus)
        return Shape{tm, 32};
    const bool wide = p.d_dtype == GG_F32;
    const double big = ceil(tiles(256, 256) / cus) * ((wide ? 11 : 8) + 1.8 * units);
    const double small = (tiles(128, 128) / cus + 0.5) * ((wide ? 2.7 : 2.1) + 0.57 * units);
    const bool holds = tile_bound(p, 128, 128) <= kMaxGemmBlocks;
    return small < big && holds ? Shape{128, 128} : Shape{256, 256};
}

}  // namespace

int64_t gemm_mx4_blocks(const GemmMx4Args& p) {
    const Shape c = shape_of(p);
    const int64_t tiles = tile_bound(p, c.tm, c.tn);
    return tiles > 1 ? tiles : 1;                      // (one block writes the error word)
}

hipError_t launch_gemm_mx4(const GemmMx4Args& p, hipStream_t s, LaunchInfo* info) {
    const Shape c = shape_of(p);
    const dim3 grid((unsigned)gemm_mx4_blocks(p));
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "%s<D %s>", c.thin() ? "thin_kernel" : "gemm_kernel",
                 dtype_name(p.d_dtype));
        info->tm = c.tm;
        info->tn = c.tn;
        info->waves = c.thin() ? kThinWaves : BigTile::kWaves;
        info->grid = grid.x;
    }
    if (c.thin()) {
        if (c.tm == 16)
            hipLaunchKernelGGL((thin_kernel<1>), grid, dim3(kThinThreads), 0, s, p);
        else
            hipLaunchKernelGGL((thin_kernel<2>), grid, dim3(kThinThreads), 0, s, p);
    } else {
        const dim3 block(BigTile::kThreads);
        auto by_shape = [&](auto DTc) {
            constexpr int DT = decltype(DTc)::value;
            auto by_bias = [&](auto tile, auto ODDc) {
                using C = decltype(tile);
                constexpr bool ODD = decltype(ODDc)::value;
                if (p.bias)
                    hipLaunchKernelGGL((gemm_kernel<C, DT, ODD, true>), grid, block, 0, s, p);
                else
                    hipLaunchKernelGGL((gemm_kernel<C, DT, ODD, false>), grid, block, 0, s, p);
            };
            auto by_k = [&](auto tile) {
                p.K % 256 ? by_bias(tile, std::true_type()) : by_bias(tile, std::false_type());
            };
            c.tm == 256 ? by_k(BigTile()) : by_k(SmallTile());
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
