// gg_dispatch.hip -- tokens to the expert-sorted rows the grouped GEMMs take,
// and back: the row of every (token, choice), the copies, the weighted sum
// of a token's rows and that sum's gradients.
#include <type_traits>

#include "gg_lane.hpp"
#include "gg_step.hpp"

namespace gg {

namespace {

// ---- the plan --------------------------------------------------------------
//
// A row's place in its expert's group is the number of earlier tokens that
// chose the expert.  Tokens go in chunks of 256: per chunk an LDS bitmap,
// one bit per (expert, token), is set with integer ORs (their order does not
// matter), and a token's rank is the population count of the bits below its
// own.  A block takes a run of chunks.  plan_count_kernel writes each
// block's counts, plan_assign_kernel sums those of the blocks before it and
// numbers the rows.  With one block there is nothing to join and
// plan_assign_kernel counts for itself.
//
// An id outside 0 .. E-1, or one that its token has already used, has no row.
// A second use shows as a bit that was set before; only a chunk with one
// looks for the first uses.
//
// Bound by latency: 8192 tokens x 8 choices of 64 experts 4.7 + 6.9 us, 7
// tokens 3.9 us.  Two chunks of tokens still go through one block.

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kChunk = 256;                          // tokens of a bitmap
constexpr int kWords = kChunk / 32;
constexpr int kMaxExperts = 1024;

// i / k for slots i of a chunk (i < 256 * 32, k <= 32): with m = ceil(2^18 /
// k), i m / 2^18 exceeds i / k by less than i k / (2^18 k) < 1 / k.
struct SlotDiv {
    uint32_t m;
    __device__ explicit SlotDiv(int k) : m(((1u << 18) + k - 1) / k) {}
    __device__ __forceinline__ int operator()(int i) const { return (int)(((uint32_t)i * m) >> 18); }
};

// Whether slot i of the chunk's ids (token t of it) is its token's first use
// of its expert.
__device__ __forceinline__ bool first_use(const int32_t* ids, int i, int t, int k, int e) {
    for (int q = t * k; q < i; q++)
        if (ids[q] == e)
            return false;
    return true;
}

// Sets the bits of a chunk of n tokens (bit t % 32 of bits[t / 32 * E + e]);
// every thread of the block calls it.  bits holds zeros on entry.  Returns
// whether a token uses an expert twice; f |= a flag for ids that are neither
// an expert nor -1, or used twice.
__device__ __forceinline__ bool plan_bits(const PlanArgs& p, const int32_t* ids, int n, SlotDiv div,
                                          uint32_t* bits, int32_t* twice, int& f) {
    for (int i = threadIdx.x; i < n * p.k; i += kPlanThreads) {
        const int e = ids[i], t = div(i);
        if (e >= 0 && e < p.E) {
            const uint32_t bit = 1u << (t & 31);
            if (atomicOr(&bits[(t >> 5) * p.E + e], bit) & bit) {
                *twice = 1;
                f |= GG_DEVERR_IDS;
            }
        } else if (e != -1) {
            f |= GG_DEVERR_IDS;
        }
    }
    __syncthreads();
    return *twice != 0;
}

__device__ __forceinline__ int plan_ones(const uint32_t* bits, int E, int e) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kWords; w++)
        c += __popc(bits[w * E + e]);
    return c;
}

__device__ __forceinline__ void plan_clear(uint32_t* bits, int E) {
    for (int i = threadIdx.x; i < E * kWords; i += kPlanThreads)
        bits[i] = 0;
    __syncthreads();
}

// Workspace: header (int32 0: the error word), then [blocks][E] int32 counts
// and [blocks] flags.
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(PlanArgs p, int64_t run) {
    __shared__ uint32_t bits[kMaxExperts * kWords];
    __shared__ int32_t flags, twice;
    const int e = threadIdx.x;
    if (e == 0)
        flags = twice = 0;
    const SlotDiv div(p.k);
    int count = 0, f = 0;
    const int64_t t1 = min(p.T, (int64_t)(blockIdx.x + 1) * run);
    for (int64_t t = blockIdx.x * run; t < t1; t += kChunk) {
        plan_clear(bits, p.E);
        plan_bits(p, p.ids + t * p.k, (int)min((int64_t)kChunk, t1 - t), div, bits, &twice, f);
        if (e < p.E)
            count += plan_ones(bits, p.E, e);
        __syncthreads();
    }
    if (f)
        atomicOr(&flags, f);
    __syncthreads();
    int32_t* part = p.ws + kWsHeader / 4;
    if (e < p.E)
        part[(int64_t)blockIdx.x * p.E + e] = count;
    if (e == 0)
        part[(int64_t)gridDim.x * p.E + blockIdx.x] = flags;
}

__global__ void __launch_bounds__(kPlanThreads) plan_assign_kernel(PlanArgs p, int64_t run, int blocks,
                                                                   int lanes) {
    __shared__ uint32_t bits[kMaxExperts * kWords];
    __shared__ int32_t base[kMaxExperts];            // row of the block's next token of an expert
    __shared__ int32_t stop[kMaxExperts];            // end of the group, within m_rows
    __shared__ int32_t fill[kMaxExperts];            // first padding row
    __shared__ int32_t wave_sums[kPlanWaves];
    __shared__ int32_t flags, twice;
    const int e = threadIdx.x, E = p.E, lane = e & 63, wave = e >> 6;
    const SlotDiv div(p.k);
    if (e == 0)
        flags = twice = 0;
    base[e] = stop[e] = 0;
    plan_clear(bits, E);
    int f = 0;
    // counts of the blocks before this one, and of all
    int before = 0, all = 0;
    bool dup = false;
    if (blocks > 1) {
        // `lanes` threads along the experts (a power of two >= E), the rest
        // along the blocks
        const int x = e & (lanes - 1), rows = kPlanThreads / lanes;
        const int32_t* part = p.ws + kWsHeader / 4;
        int b0 = 0, a0 = 0;
        if (x < E) {
#pragma unroll 8
            for (int b = e / lanes; b < blocks; b += rows) {
                const int c = part[(int64_t)b * E + x];
                b0 += b < (int)blockIdx.x ? c : 0;
                a0 += c;
            }
            atomicAdd(&base[x], b0);
            atomicAdd(&stop[x], a0);
        }
        if (blockIdx.x == 0 && e < blocks)
            f |= part[(int64_t)blocks * E + e];
        __syncthreads();
        before = base[e];
        all = stop[e];
        __syncthreads();
    } else {
        for (int64_t t = 0; t < p.T; t += kChunk) {
            if (t)
                plan_clear(bits, E);
            dup = plan_bits(p, p.ids + t * p.k, (int)min((int64_t)kChunk, p.T - t), div, bits, &twice, f);
            if (e < E)
                all += plan_ones(bits, E, e);
            __syncthreads();
        }
    }
    // the padded groups' ends: a scan over the experts (below 2^31: at most
    // 2^28 choices and 255 rows of padding for each expert)
    const int padded = e < E ? (all + p.granule - 1) & -p.granule : 0;
    int sum = padded;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
        const int v = __shfl_up(sum, h);
        sum += lane >= h ? v : 0;
    }
    if (lane == 63)
        wave_sums[wave] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPlanWaves; w++)
        sum += w < wave ? wave_sums[w] : 0;
    // groups are cut off where the rows end
    const int limit = (int)(p.m_rows & -(int64_t)p.granule);
    const int b0 = min(sum - padded, limit), b1 = min(sum, limit);
    const int kept = min(all, b1 - b0);
    if (e < E) {
        base[e] = b0 + min(before, b1 - b0);
        stop[e] = b1;
        fill[e] = b0 + kept;
        if (blockIdx.x == 0) {
            p.counts[e] = kept;
            p.ends[e] = b1;
            if (kept < all)
                f |= GG_DEVERR_LAST;
        }
    }
    __syncthreads();
    const int64_t t1 = min(p.T, (int64_t)(blockIdx.x + 1) * run);
    int seen = 0;
    for (int64_t t0 = blockIdx.x * run; t0 < t1; t0 += kChunk) {
        const int32_t* ids = p.ids + t0 * p.k;
        const int n = (int)min((int64_t)kChunk, t1 - t0);
        // a single chunk's bits are there already; the first chunk of
        // several blocks' finds cleared ones
        if (blocks > 1 || p.T > kChunk) {
            if (t0 != blockIdx.x * run || blocks == 1)
                plan_clear(bits, E);
            dup = plan_bits(p, ids, n, div, bits, &twice, seen);
        }
        for (int i = threadIdx.x; i < n * p.k; i += kPlanThreads) {
            const int x = ids[i], t = div(i);
            int row = -1;
            if (x >= 0 && x < E && (!dup || first_use(ids, i, t, p.k, x))) {
                int rank = __popc(bits[(t >> 5) * E + x] & ((1u << (t & 31)) - 1u));
                for (int w = 0; w < (t >> 5); w++)
                    rank += __popc(bits[w * E + x]);
                if (rank < stop[x] - base[x])
                    row = base[x] + rank;
            }
            const int64_t slot = t0 * p.k + i;
            p.row_of[slot] = row;
            if (p.prob_rows && row >= 0)
                p.prob_rows[row] = p.prob[slot];
        }
        if (t0 + kChunk < t1) {
            __syncthreads();
            if (e < E)
                base[e] += min(plan_ones(bits, E, e), stop[e] - base[e]);
            __syncthreads();
        }
    }
    // padding rows, the experts dealt to the blocks
    if (p.prob_rows)
        for (int x = blockIdx.x * kPlanWaves + wave; x < E; x += gridDim.x * kPlanWaves)
            for (int r = fill[x] + lane; r < stop[x]; r += 64)
                p.prob_rows[r] = 0.0f;
    if (blockIdx.x == 0) {
        if (f)
            atomicOr(&flags, f);
        __syncthreads();
        if (e == 0)
            p.ws[0] = flags;
    }
}

// ---- rows ------------------------------------------------------------------
//
// Token rows and expert rows are walked in 16-byte vectors at element
// alignment.  Where a row is no whole number of them, permute and combine
// start the last one a vector before the row's end: what it shares with the
// one before is computed and written twice, the same values (1001 tokens x 3
// rows of 2047 fp32: 5.9 us for 8.0 with single elements at the end).  Only
// rows shorter than a vector go element by element.  A block is tx vectors of
// a row by 256 / tx tokens.
//
// Bound by memory: every token row is read or written once, every expert row
// once.  Measured, bf16 (a copy kernel's best on the same card is 6.6 TB/s):
// - permute, 8192 tokens x 8 rows of 4096 (604 MB, and 67 MB of zeros): 111 us,
//   6.1 TB/s.  Scattering, so that a token row is read once.
// - combine, the same sizes: 99 us, 6.1 TB/s.  A row at a time per thread:
//   with 2, 4 or 8 rows' loads at once 102 us, and 252 for 231 at two rows of
//   7168 a token; enough waves are in flight.
// - combine_bwd, 32768 tokens x 2 rows of 7168 (2.35 GB): 421 us, 5.6 TB/s.
//   Here a block keeps a token (its sums end in one place), so 8 vectors of
//   rows at once are needed: one at a time 516 us.  A slot without a row (past
//   k, or a dropped choice) loads row 0, which the cache holds: 65536 rows of
//   4096 in 1, 2, 3, 4, 5, 6, 7, 8 and 9 choices a token run at 5.1, 5.5, 5.5,
//   5.3, 5.2, 5.2, 4.9, 4.8 and 4.3 TB/s, nothing at 3, 5 and 6, 10% at 9,
//   whose second turn has one row in eight slots.

constexpr int kRowThreads = 256;
constexpr int kPadParts = 8;                         // blocks that share an expert's padding rows

template <int DT>
struct RowElem {
    typedef typename Elem<DT>::T T;
    static constexpr int N = 16 / (int)sizeof(T);
};

// Which of its block's tokens a wave works on (a scalar: tx is 64 at least).
__device__ __forceinline__ int wave_token(int tx) {
    return __builtin_amdgcn_readfirstlane((int)threadIdx.x / tx);
}

// x_rows[row_of[t, j]] = x[t], zeros in the padding.  SIZE: bytes of an
// element; the values are copied as they are.  Every row of x is read once
// and written k times.
template <int SIZE, bool NT>
__global__ void __launch_bounds__(kRowThreads) permute_kernel(RowsArgs p, int tx, int pads) {
    typedef Raw16 V;
    const int col = threadIdx.x % tx + (int)blockIdx.y * tx;
    const int64_t bytes = (int64_t)p.width * SIZE;
    if ((int64_t)col * 16 >= bytes)
        return;
    const bool whole = bytes >= 16;
    const int64_t at = whole ? min((int64_t)col * 16, bytes - 16) : 0;
    char* out = (char*)p.rows_out;
    auto put = [&](int64_t r, V v) {
        if constexpr (NT)
            __builtin_nontemporal_store(v, (V*)(out + r * bytes + at));
        else
            *(V*)(out + r * bytes + at) = v;
    };
    if ((int)blockIdx.x < pads) {
        const int e = blockIdx.x / kPadParts, part = blockIdx.x % kPadParts;
        const int ty = kRowThreads / tx;
        const int begin = e ? p.ends[e - 1] : 0;
        const int64_t r1 = min((int64_t)p.ends[e], p.m_rows);
        for (int64_t r = (int64_t)max(begin, 0) + max(p.counts[e], 0) + part * ty + threadIdx.x / tx; r < r1;
             r += kPadParts * ty) {
            if (whole)
                put(r, V{0, 0, 0, 0});
            else
                for (int64_t b = at; b < bytes; b++)
                    out[r * bytes + b] = 0;
        }
        return;
    }
    const int64_t t = (int64_t)(blockIdx.x - pads) * (kRowThreads / tx) + wave_token(tx);
    if (t >= p.T)
        return;
    const char* in = (const char*)p.tokens + t * p.ld * SIZE;
    const int32_t* row_of = p.row_of + t * p.k;
    V v = {0, 0, 0, 0};
    if (whole)
        v = *(const V*)(in + at);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        int r[8];                                    // eight rows' numbers before the stores
#pragma unroll
        for (int j = 0; j < 8; j++)
            r[j] = row_of[min(j0 + j, p.k - 1)];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (j0 + j >= p.k || r[j] < 0 || r[j] >= p.m_rows)
                continue;
            if (whole)
                put(r[j], v);
            else
                for (int64_t b = at; b < bytes; b++)
                    out[r[j] * bytes + b] = in[b];
        }
    }
}

// out[t] = sum_j w[t, j] y[row_of[t, j]], in fp32 in the order of j, rounded
// once.
template <int DT, bool NT>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(RowsArgs p, int tx) {
    typedef typename Elem<DT>::T T;
    constexpr int N = RowElem<DT>::N;
    const int at = (threadIdx.x % tx + (int)blockIdx.y * tx) * N;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / tx) + wave_token(tx);
    if (t >= p.T || at >= p.width)
        return;
    const T* y = (const T*)p.rows_in;
    T* out = (T*)p.out + t * p.ld;
    const int32_t* row_of = p.row_of + t * p.k;
    const float* w = p.weights ? p.weights + t * p.k : nullptr;
    if (p.width >= N) {
        const int c = min(at, p.width - N);
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; i++)
            acc[i] = 0.0f;
        for (int j = 0; j < p.k; j++) {
            const int64_t r = row_of[j];
            if (r < 0 || r >= p.m_rows)
                continue;
            Vec<DT, N> v;
            v.template load<NT>(y + r * p.width + c);
            const float wj = w ? w[j] : 1.0f;
#pragma unroll
            for (int i = 0; i < N; i++)
                acc[i] = fmaf(wj, v.get(i), acc[i]);
        }
        Vec<DT, N> v;
        v.set(acc);
        v.template store<NT>(out + c);
    } else {
        for (int i = 0; i < p.width; i++) {
            float acc = 0.0f;
            for (int j = 0; j < p.k; j++) {
                const int64_t r = row_of[j];
                if (r >= 0 && r < p.m_rows)
                    acc = fmaf(w ? w[j] : 1.0f, to_f32<DT>(y[r * p.width + i]), acc);
            }
            out[i] = from_f32<DT>(acc);
        }
    }
}

// dy[row_of[t, j]] = w[t, j] dout[t] (rounded once; zeros in the padding),
// dw[t, j] = <dout[t], y[row_of[t, j]]> in fp32.  A block a token; KB rows by
// U vectors of loads at once.  The first `pads` blocks clear the padding.
template <int DT, int KB, int U, bool NT>
__global__ void __launch_bounds__(kRowThreads) combine_bwd_kernel(RowsArgs p, int pads) {
    typedef typename Elem<DT>::T T;
    constexpr int N = RowElem<DT>::N;
    __shared__ float part[kRowThreads / 64][KB];
    T* dy = (T*)p.rows_out;
    const int tid = threadIdx.x, threads = blockDim.x;
    const int vecs = p.width / N;                    // whole ones; the rest is `rest` elements
    const int rest = p.width - vecs * N;
    if ((int)blockIdx.x < pads) {
        const int e = blockIdx.x / kPadParts, sub = blockIdx.x % kPadParts;
        const int begin = e ? p.ends[e - 1] : 0;
        const int64_t r1 = min((int64_t)p.ends[e], p.m_rows);
        for (int64_t r = (int64_t)max(begin, 0) + max(p.counts[e], 0) + sub; r < r1; r += kPadParts) {
            Vec<DT, N> z;
            z.raw = 0;
            for (int i = tid; i < vecs; i += threads)
                z.template store<NT>(dy + r * p.width + i * N);
            if (tid < rest)
                dy[r * p.width + vecs * N + tid] = 0;
        }
        return;
    }
    const int64_t t = blockIdx.x - pads;
    const T* dout = (const T*)p.tokens + t * p.ld;
    const T* y = (const T*)p.rows_in;
    for (int j0 = 0; j0 < p.k; j0 += KB) {
        const int kb = min(KB, p.k - j0);
        int row[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; j++) {
            const int64_t at = t * p.k + j0 + min(j, kb - 1);
            row[j] = p.row_of[at];
            row[j] = j < kb && row[j] < p.m_rows ? row[j] : -1;
            w[j] = p.weights[at];
            dot[j] = 0.0f;
        }
        // (with no rows at all there is nothing to load)
        for (int i0 = tid; p.m_rows > 0 && i0 < vecs; i0 += U * threads) {
            Vec<DT, N> d[U], v[U][KB];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int c = min(i0 + u * threads, vecs - 1) * N;
                d[u].template load<NT>(dout + c);
#pragma unroll
                for (int j = 0; j < KB; j++)
                    v[u][j].template load<NT>(y + (int64_t)max(row[j], 0) * p.width + c);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (i0 + u * threads >= vecs)
                    break;
                const int c = (i0 + u * threads) * N;
#pragma unroll
                for (int j = 0; j < KB; j++) {
                    if (row[j] < 0)
                        continue;
                    Vec<DT, N> o;
                    float f[N];
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        dot[j] = fmaf(d[u].get(i), v[u][j].get(i), dot[j]);
                        f[i] = w[j] * d[u].get(i);
                    }
                    o.set(f);
                    o.template store<NT>(dy + (int64_t)row[j] * p.width + c);
                }
            }
        }
        if (tid < rest) {
            const int c = vecs * N + tid;
            const float d = to_f32<DT>(dout[c]);
#pragma unroll
            for (int j = 0; j < KB; j++)
                if (row[j] >= 0) {
                    const int64_t at = (int64_t)row[j] * p.width + c;
                    dot[j] = fmaf(d, to_f32<DT>(y[at]), dot[j]);
                    dy[at] = from_f32<DT>(w[j] * d);
                }
        }
#pragma unroll
        for (int j = 0; j < KB; j++) {
            const float s = group_all<64>(dot[j], OpAddF());
            if ((tid & 63) == 0)
                part[tid >> 6][j] = s;
        }
        __syncthreads();
        if (tid < kb) {
            float s = part[0][tid];
            for (int x = 1; x < threads / 64; x++)
                s += part[x][tid];
            p.dweights[t * p.k + j0 + tid] = s;
        }
        __syncthreads();
    }
}

// Threads of a block along a row of `vecs` vectors: a power of two, whole waves,
// up to 256.
int row_threads(int64_t vecs) {
    int tx = 64;
    while (tx < vecs && tx < kRowThreads)
        tx *= 2;
    return tx;
}

}  // namespace

// ---- launches --------------------------------------------------------------

static int64_t plan_blocks(int64_t T) {
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    return chunks <= 2 ? 1 : chunks > 256 ? 256 : chunks;
}

size_t plan_workspace(int64_t T, int E) {
    return kWsHeader + (size_t)plan_blocks(T) * ((size_t)E + 1) * 4;
}

hipError_t launch_plan(const PlanArgs& p, hipStream_t s, LaunchInfo* info) {
    int64_t blocks = plan_blocks(p.T);
    const int64_t chunks = (p.T + kChunk - 1) / kChunk;
    const int64_t run = (chunks + blocks - 1) / blocks * kChunk;     // tokens of a block
    if (blocks > 1)
        blocks = (p.T + run - 1) / run;
    hipError_t e = hipSuccess;
    if (blocks > 1) {
        hipLaunchKernelGGL(plan_count_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), 0, s, p, run);
        e = hipGetLastError();
    }
    if (e == hipSuccess) {
        int lanes = 64;
        while (lanes < p.E)
            lanes *= 2;
        hipLaunchKernelGGL(plan_assign_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), 0, s, p, run,
                           (int)blocks, lanes);
        e = hipGetLastError();
    }
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "%splan_assign_kernel",
                 blocks > 1 ? "plan_count_kernel + " : "");
        info->tm = (int)run;
        info->tn = p.E;
        info->waves = kPlanThreads / 64;
        info->grid = blocks;
    }
    return e;
}

static void rows_info(LaunchInfo* info, const char* name, int dtype, int tokens, int cols, int64_t grid) {
    if (!info)
        return;
    snprintf(info->kernel, sizeof info->kernel, "%s<%s>", name, dtype_name(dtype));
    info->tm = tokens;
    info->tn = cols;
    info->waves = kRowThreads / 64;
    info->grid = grid;
}

static int elem_bytes(int dtype) { return dtype == GG_F32 ? 4 : dtype == GG_BF16 || dtype == GG_F16 ? 2 : 1; }

// Whether the expert rows of a call are more than the 256 MB cache in front
// of the memory holds.  Non-temporal accesses then pass it by: 537 MB of
// rows permute in 112 us for 126, combine in 100 for 117, combine_bwd (940
// MB) in 420 for 446.  Below it they lose what the cache would have held: 134
// MB permute in 33 us for 28, 67 MB combine_bwd in 37 for 28.
static bool past_cache(const RowsArgs& p, int size) {
    return p.T * p.k * (int64_t)p.width * size > (int64_t)256 << 20;
}

// f(std::integral_constant) of a type, of a truth value.
template <class F>
static void by_dtype(int dtype, F f) {
    if (dtype == GG_BF16)
        f(std::integral_constant<int, GG_BF16>());
    else if (dtype == GG_F16)
        f(std::integral_constant<int, GG_F16>());
    else
        f(std::integral_constant<int, GG_F32>());
}
template <class F>
static void by_bool(bool b, F f) {
    if (b)
        f(std::true_type());
    else
        f(std::false_type());
}

hipError_t launch_permute(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    const int size = elem_bytes(dtype);
    const int64_t vecs = ((int64_t)p.width * size + 15) / 16;
    const int tx = row_threads(vecs), ty = kRowThreads / tx;
    const int pads = p.E * kPadParts;
    const dim3 grid((unsigned)(pads + (p.T + ty - 1) / ty), (unsigned)((vecs + tx - 1) / tx));
    by_bool(past_cache(p, size), [&](auto NT) {
        if (size == 1)
            hipLaunchKernelGGL((permute_kernel<1, NT.value>), grid, dim3(kRowThreads), 0, s, p, tx, pads);
        else if (size == 2)
            hipLaunchKernelGGL((permute_kernel<2, NT.value>), grid, dim3(kRowThreads), 0, s, p, tx, pads);
        else
            hipLaunchKernelGGL((permute_kernel<4, NT.value>), grid, dim3(kRowThreads), 0, s, p, tx, pads);
    });
    rows_info(info, "permute_kernel", dtype, ty, tx * 16 / size, (int64_t)grid.x * grid.y);
    return hipGetLastError();
}

hipError_t launch_combine(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    if (p.T == 0)
        return hipSuccess;
    const int size = elem_bytes(dtype);
    const int64_t vecs = ((int64_t)p.width * size + 15) / 16;
    const int tx = row_threads(vecs), ty = kRowThreads / tx;
    const dim3 grid((unsigned)((p.T + ty - 1) / ty), (unsigned)((vecs + tx - 1) / tx));
    by_dtype(dtype, [&](auto DT) {
        by_bool(past_cache(p, size), [&](auto NT) {
            hipLaunchKernelGGL((combine_kernel<DT.value, NT.value>), grid, dim3(kRowThreads), 0, s, p, tx);
        });
    });
    rows_info(info, "combine_kernel", dtype, ty, tx * 16 / size, (int64_t)grid.x * grid.y);
    return hipGetLastError();
}

hipError_t launch_combine_bwd(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    const int size = elem_bytes(dtype);
    const int pads = p.E * kPadParts;
    const dim3 grid((unsigned)(pads + p.T));
    const int64_t vecs = ((int64_t)p.width * size + 15) / 16;
    const dim3 threads((unsigned)(vecs >= kRowThreads ? kRowThreads : (vecs + 63) / 64 * 64));
    by_dtype(dtype, [&](auto DT) {
        by_bool(past_cache(p, size), [&](auto NT) {
            if (p.k <= 2)
                hipLaunchKernelGGL((combine_bwd_kernel<DT.value, 2, 4, NT.value>), grid, threads, 0, s, p, pads);
            else if (p.k <= 4)
                hipLaunchKernelGGL((combine_bwd_kernel<DT.value, 4, 2, NT.value>), grid, threads, 0, s, p, pads);
            else
                hipLaunchKernelGGL((combine_bwd_kernel<DT.value, 8, 1, NT.value>), grid, threads, 0, s, p, pads);
        });
    });
    rows_info(info, "combine_bwd_kernel", dtype, 1, p.width, grid.x);
    return hipGetLastError();
}

}  // namespace gg
