// gg_route.hip -- the router: top-k choice of experts, their weights, tokens
// per expert and the balance loss; and the gradient of the logits.
//
// Both kernels give each token a group of LPT lanes, each lane EPL
// consecutive experts, so that one pass over the logits holds a token's row
// in registers.  Statistics, weights and gradients are in fp32.
//
// Measured at 65536 tokens x 256 experts, bf16, 8 choices (34 MB of logits;
// medians):
// - route_kernel 20.2 us (sigmoid) and route_join_kernel 5.0 us.  Bound by the
//   vector ALU: a wave spends some 500 vector instructions, 35 of them
//   transcendental, on four tokens, two fifths in the 8 steps of the choice;
//   79% of its cycles issue one.  Occupancies of 4, 6 and 8 waves a SIMD give
//   the same time.  Twice the experts a lane (8 lanes x 32) halves what the
//   reductions cost a token but leaves half the passes to hide latency: 2.2 us
//   more.
// - route_bwd_kernel 18.4 us (softmax) and 21.1 (sigmoid, whose slope takes a
//   second value an expert).  88 MB from and to memory by the counters, 13 us
//   at a copy's rate: the latency of the chain ids -> rows -> dprob is the
//   rest.  8 lanes a token take 8 us more, 32 lanes 3.
// A few tokens (5 x 256): 5 us, the launch and four dependent loads.
#include <cfloat>
#include <type_traits>

#include "gg_lane.hpp"
#include "gg_step.hpp"

namespace gg {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
constexpr float kTiny = 1e-20f;          // added to sums of sigmoids, which can underflow

// Exponentials.  The hardware's, of a log2(e) rounded to fp32, is off by up to
// |a| 2^-24 of itself: FULL brings back what that rounding left out, as a - t
// ln(2) with ln(2) in two parts, and is good to 2 units of 2^-24.  It is used
// where a caller sees the exponential itself, the weights and fp32 gradients
// (weights at logits of -25 to -45: off by 5 units at most for 44).  Without it are
// the sums over all experts, whose large terms have small arguments, the loss,
// which is a mean over them, and gradients that are rounded to 16 bits: there
// it would cost route_kernel 20.1 -> 24.6 us and route_bwd_kernel 19.0 -> 20.1
// (65536 x 256 bf16).

// exp(a) of a <= 0: 0 far below the normal numbers, a NaN kept.
template <bool FULL>
__device__ __forceinline__ float exp_below(float a) {
    if constexpr (!FULL)
        return __expf(a);
    a = __builtin_elementwise_maximum(a, -110.0f);
    const float t = a * 1.44269504f;
    const float e = __builtin_amdgcn_exp2f(t);
    const float rest = fmaf(t, 1.90465421e-9f, fmaf(t, -0.693147182f, a));
    return fmaf(e, rest, e);
}

// sigmoid(-|x|), at most 1/2, with x's sign.  A sigmoid and its slope come out
// of it without 1 minus what rounds to 1: sigmoid(x) is the tail t or 1 - t,
// the slope t (1 - t).  (From the sigmoid itself the slope is off by 6% at x =
// 16 and 0 from 17 on.)
template <bool FULL>
__device__ __forceinline__ float signed_tail(float x) {
    const float e = exp_below<FULL>(-fabsf(x)), d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);              // to 1 ulp; a step of Newton's makes it half
    if constexpr (FULL)
        r = fmaf(fmaf(-d, r, 1.0f), r, r);
    return __builtin_copysignf(e * r, x);
}
__device__ __forceinline__ float tail_sigmoid(float t) {
    return __builtin_signbitf(t) ? -t : 1.0f - t;
}
__device__ __forceinline__ float tail_slope(float t) {
    return fmaf(-t, t, fabsf(t));
}

// Order of the choice as unsigned integers: fp32 order with -0 = +0 (bias is
// never -0).  kNever, a key of -inf, is never chosen; 0: taken.  ODD: the wave
// has a logit that is +inf or NaN.  An invalid operation of this hardware gives
// a NaN whose sign is set, which the plain order has below -inf.
constexpr uint32_t kNever = 0x007FFFFFu;             // the key of -inf

template <bool ODD>
__device__ __forceinline__ uint32_t order_key(float logit, float bias) {
    const float sum = logit + bias;
    const uint32_t u = __builtin_bit_cast(uint32_t, sum);
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    if (ODD && sum != sum)
        return bias == -INFINITY ? kNever : 0xFFFFFFFFu;
    return key;
}

// Words of LDS from a lane's first element to the next lane's, where a group
// keeps EPL of each lane: 16-byte vectors that lanes write at once then fall
// into different banks.
template <int EPL>
constexpr int lane_pitch() {
    return EPL + 4;
}

// How a lane loads its experts: kWholeRows are whole vectors, kOddRows are
// not but hold one, kShortRows are shorter than one.
enum RowKind { kWholeRows = 0, kOddRows = 1, kShortRows = 2 };

template <int DT>
constexpr int row_vector() {
    return 16 / (int)sizeof(typename Elem<DT>::T);
}

// The EPL experts of a lane, -inf past the row's end and where !live.  The
// loads are unconditional, at clamped addresses: a branch around a load
// makes the wave wait for it before the next.
template <int DT, int EPL, int KIND>
__device__ __forceinline__ void load_row(const typename Elem<DT>::T* row, int first, int E, bool live,
                                         float (&x)[EPL]) {
    constexpr int N = row_vector<DT>();
    // `first` as a value of its own in every pass over this: compares with it
    // would otherwise be kept from pass to pass, a register pair each
    asm volatile("" : "+v"(first));
    if constexpr (KIND == kShortRows) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            x[i] = to_f32<DT>(row[min(first + i, E - 1)]);
    } else {
        // (odd rows: the vector that crosses the row's end is read N before
        // the end and moved down by what came before it)
        Vec<DT, N> v[EPL / N];
#pragma unroll
        for (int c = 0; c < EPL; c += N)
            v[c / N].load(row + min(first + c, E - N));
#pragma unroll
        for (int c = 0; c < EPL; c += N) {
            if constexpr (KIND == kOddRows)
                v[c / N].drop(first + c - min(first + c, E - N));
#pragma unroll
            for (int i = 0; i < N; i++)
                x[c + i] = v[c / N].get(i);
        }
    }
    // past the row's end, or no row: waves of whole rows skip this
    if (__ballot(!live || first + EPL > E))
#pragma unroll
        for (int i = 0; i < EPL; i++)
            x[i] = live && first + i < E ? x[i] : -INFINITY;
}

template <int DT, int EPL, int KIND>
__device__ __forceinline__ void store_row(typename Elem<DT>::T* row, int first, int E,
                                          const float (&x)[EPL]) {
    constexpr int N = row_vector<DT>();
#pragma unroll
    for (int c = 0; c < EPL; c += N) {
        if (first + c + N <= E) {
            Vec<DT, N> v;
            float f[N];
#pragma unroll
            for (int i = 0; i < N; i++)
                f[i] = x[c + i];
            v.set(f);
            v.store(row + first + c);
        } else if constexpr (KIND != kWholeRows) {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (first + c + i < E)
                    row[first + c + i] = from_f32<DT>(x[c + i]);
        }
    }
}

// Largest of a lane's values, NaN if one is.
template <int EPL>
__device__ __forceinline__ float lane_top(const float (&x)[EPL]) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < EPL; i++)
        m = __builtin_elementwise_maximum(m, x[i]);
    return m;
}

// 1 / a sum of scores.
__device__ __forceinline__ float inverse_sum(float sum, bool softmax) {
    return softmax ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f / (sum + kTiny);
}

// A token's softmax or sigmoid over its row: x becomes the scores, `inv` what
// turns them into the balance probabilities (softmax: x are exp(x - top), so
// that p = x inv is the softmax as well; a row of -inf gives all zeros, one
// with a NaN all NaN).  m is the lane's lane_top.
template <int LPT, int EPL, bool FULL>
__device__ __forceinline__ void row_scores(float (&x)[EPL], bool softmax, float m, float& top, float& inv) {
    float sum = 0.0f;
    if (softmax) {
        m = group_all<LPT>(m, OpMaxF());
        top = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            x[i] = exp_below<FULL>(x[i] - top);
            sum += x[i];
        }
        sum = group_all<LPT>(sum, OpAddF());
        inv = inverse_sum(sum, true);
    } else {
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            x[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
            sum += x[i];
        }
        sum = group_all<LPT>(sum, OpAddF());
        inv = inverse_sum(sum, false);
    }
}

// Largest of the chosen logits (0 if there is none, NaN if one is).
template <int LPT, int NJ>
__device__ __forceinline__ float choice_top(const float (&v)[NJ]) {
    const float m = group_all<LPT>(lane_top(v), OpMaxF());
    return m == -INFINITY ? 0.0f : m;
}

}  // namespace

// Workspace: header (int32 0: the error word, always 0; 1: the finishing
// ticket; 4 + 2q, 5 + 2q: quarter q's routed tokens as a double), then the
// blocks' counts and probability sums as pairs, 16 experts (a 128-byte line)
// of a block after another's: [ceil(E / 16)][blocks][16], the blocks' routed
// tokens, and what the joining blocks have made of a quarter of the blocks
// each, [4][E].
struct RoutePair {
    int32_t count;
    float sum;
};
struct RouteJoined {
    double sum;
    int64_t count;
};
constexpr int kMaxRouteBlocks = 768;                 // three to a CU, then more passes each
constexpr int kLine = 16, kQuarters = 4;

__host__ __device__ inline int64_t route_lines(int E) { return (E + kLine - 1) / kLine; }
__device__ inline RoutePair* route_pairs(int32_t* ws) { return (RoutePair*)(ws + kWsHeader / 4); }
__device__ inline int32_t* route_routed(int32_t* ws, int E, int blocks) {
    return (int32_t*)(route_pairs(ws) + route_lines(E) * blocks * kLine);
}
__device__ inline RouteJoined* route_joined(int32_t* ws, int E, int blocks) {
    return (RouteJoined*)(route_routed(ws, E, blocks) + (blocks + 3) / 4 * 4);
}

// One token per group of LPT lanes and pass.  The choice: every lane keeps
// the largest key of its EPL; a step takes the group's largest (ties: the
// lowest lane, so the lowest experts), rescans that lane's keys -- in LDS,
// one per lane of the group -- for the expert, removes it and hands the lane
// its next largest.
template <int DT, int LPT, int EPL, int KIND, int SCORE>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs p) {
    static_assert(EPL <= LPT, "a group rescans one lane's keys in one read");
    constexpr int TPW = 64 / LPT;                    // tokens per wave
    constexpr int NJ = LPT >= 32 ? 1 : 32 / LPT;     // choices a lane may hold
    constexpr int kCap = LPT * EPL;
    constexpr int kPitch = lane_pitch<EPL>();
    __shared__ __align__(16) uint32_t keys[kWaves * 64 * kPitch];
    __shared__ __align__(16) float bias[LPT * kPitch];
    __shared__ int32_t hist[kCap];
    __shared__ int32_t nrouted;
    typedef typename Elem<DT>::T T;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // a scalar: loops over it are the wave's
    const int g = lane & (LPT - 1), sub = lane / LPT;
    const int first = g * EPL;
    const int E = p.E, k = p.k;
    constexpr bool softmax = SCORE == GG_SOFTMAX;
    const bool stats = p.balance != nullptr;
    uint32_t* group_keys = keys + (wave * TPW + sub) * LPT * kPitch;

    for (int e = tid; e < kCap; e += kThreads)
        hist[e] = 0;
    if (tid == 0) {
        nrouted = 0;
        if (blockIdx.x == 0)
            p.ws[0] = p.ws[1] = 0;
    }
    // +inf and NaN as the largest finite bias: a logit of -inf stays one
    for (int e = tid; e < kCap; e += kThreads) {
        const float b = p.bias && e < E ? p.bias[e] : 0.0f;
        bias[e / EPL * kPitch + e % EPL] = b <= FLT_MAX ? b + 0.0f : FLT_MAX;
    }
    // (fp32: a group adds T / (blocks x groups) probabilities here, 171 at 2^23
    // tokens of 8 experts; the blocks' sums are joined in fp64)
    float psum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++)
        psum[i] = 0.0f;
    __syncthreads();

    const int T_ = (int)p.T;                         // at most 2^23
    const int step = (int)gridDim.x * kWaves * TPW;
    for (int t0 = ((int)blockIdx.x * kWaves + wave) * TPW; t0 < T_; t0 += step) {
        const int t = t0 + sub;
        const bool live = t < T_;
        const T* row = (const T*)p.logits + (live ? t : 0) * p.ld;
        float x[EPL];
        load_row<DT, EPL, KIND>(row, first, E, live, x);
        uint32_t best = 0;
        auto make_keys = [&](auto odd) {
#pragma unroll
            for (int c = 0; c < EPL; c += 4) {
                u32x4 four;
                const f32x4 b = *(const f32x4*)(bias + g * kPitch + c);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    four[i] = order_key<odd.value>(x[c + i], b[i]);
                    best = best > four[i] ? best : four[i];
                }
                *(u32x4*)(group_keys + g * kPitch + c) = four;
            }
        };
        // (the wave's choice of the two: 1% of this case; as one instruction
        // more in every key 2%)
        const float m = lane_top(x);
        const bool odd = __ballot(!(m < INFINITY)) != 0;
        if (odd)
            make_keys(std::true_type());
        else
            make_keys(std::false_type());
        uint32_t most = group_all<LPT>(best, OpMaxU());
        float top = 0.0f, inv = 0.0f;
        if (stats || (softmax && !p.normalize)) {
            row_scores<LPT, EPL, false>(x, softmax, m, top, inv);
            if (stats) {
                // no choice: no part in the loss, though a bias of -inf may
                // have taken out a NaN, which 0 times does not
                const float share = most > kNever ? inv : 0.0f;
                if (odd)
#pragma unroll
                    for (int i = 0; i < EPL; i++)
                        x[i] = most > kNever ? x[i] : 0.0f;
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    psum[i] = fmaf(x[i], share, psum[i]);
            }
        }
        if constexpr (EPL < LPT)
            group_keys[g * kPitch + EPL] = 0;        // read and written by the lanes past EPL
        // the choice; lane j % LPT keeps choice j, NJ of them if top_k > LPT
        int32_t e[NJ];
        float v[NJ];
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            int32_t id = -1;
            uint32_t kept = 0;
            const int n = __builtin_amdgcn_readfirstlane(min(LPT, k - s * LPT));
            for (int j = 0; j < n; j++) {
                wave_sync();
                const int from = group_first<LPT>(best == most, lane);
                uint32_t* mine = group_keys + from * kPitch + min(g, EPL);
                uint32_t key = *mine;
                const int at = group_first<LPT>(key == most, lane);
                key = g == at ? 0u : key;
                *mine = key;
                const uint32_t next = group_all<LPT>(key, OpMaxU());
                best = g == from ? next : best;
                id = g == j ? from * EPL + at : id;
                kept = g == j ? most : kept;
                most = group_all<LPT>(best, OpMaxU());
            }
            e[s] = live && kept > kNever ? id : -1;
            v[s] = -INFINITY;
            if (s * LPT < k) {
                v[s] = to_f32<DT>(row[max(e[s], 0)]);
                v[s] = e[s] >= 0 ? v[s] : -INFINITY;
            }
        }
        wave_sync();
        float norm = softmax ? inv : 1.0f;
        if (p.normalize && softmax)
            top = choice_top<LPT, NJ>(v);
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            if (s * LPT >= k)                        // no lane's: the wave skips it
                continue;
            v[s] = softmax ? exp_below<true>(v[s] - top) : tail_sigmoid(signed_tail<true>(v[s]));
            sum += v[s];
        }
        if (p.normalize) {
            sum = group_all<LPT>(sum, OpAddF());
            norm = inverse_sum(sum, softmax);
        }
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            const int j = g + s * LPT;
            if (!live || j >= k)
                continue;
            p.ids[t * k + j] = e[s];
            p.prob[t * k + j] = e[s] >= 0 ? p.scale * (v[s] * norm) : 0.0f;
            if (e[s] >= 0) {
                atomicAdd(&hist[e[s]], 1);
                if (j == 0)
                    atomicAdd(&nrouted, 1);
            }
        }
    }
    __syncthreads();
    // the block's probability sums: every group's, added in the groups' order
    float* sums = (float*)keys;
    if (stats) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            sums[(wave * TPW + sub) * kCap + first + i] = psum[i];
    }
    __syncthreads();
    const bool last = gridDim.x == 1;
    const int groups = (int)min((int64_t)kWaves * TPW, p.T);     // that had a token
    const int blocks = gridDim.x;
    double loss = 0.0;
    for (int e = tid; e < E; e += kThreads) {
        float s = 0.0f;
        if (stats)
            for (int w = 0; w < groups; w++)
                s += sums[w * kCap + e];
        if (last) {
            p.counts[e] = hist[e];
            loss += (double)hist[e] * (double)s;
        } else {
            route_pairs(p.ws)[((int64_t)(e / kLine) * blocks + blockIdx.x) * kLine + e % kLine] = {hist[e], s};
        }
    }
    if (!last) {
        if (tid == 0)
            route_routed(p.ws, E, blocks)[blockIdx.x] = nrouted;
        return;
    }
    // a single block finishes here
    __syncthreads();
    loss = block_sum<kThreads>(loss, (double*)keys);
    if (tid == 0) {
        p.routed[0] = nrouted;
        if (stats) {
            const double n = nrouted > 0 ? (double)nrouted : 1.0;
            p.balance[0] = (float)((double)E * loss / ((double)k * n * n));
        }
    }
}

// Joins the blocks' counts and probability sums: a block takes 16 experts
// over a quarter of the blocks, eight lanes a line; the one that finishes
// last adds up the quarters and the loss.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) route_join_kernel(RouteArgs p, int blocks) {
    constexpr int kRows = kJoinThreads / 8;          // lines read at once
    constexpr int kEach = kMaxRouteBlocks / kQuarters / kRows;
    static_assert(kEach * kRows * kQuarters == kMaxRouteBlocks, "a quarter's lines are whole rows");
    __shared__ RouteJoined part[kJoinThreads / 64][kLine];
    __shared__ double tmp[kJoinThreads / 64];
    __shared__ int32_t is_last;
    const int tid = threadIdx.x, E = p.E, lane = tid & 63, wave = tid >> 6;
    const int group = blockIdx.x, quarter = blockIdx.y;
    const int b0 = quarter * (kMaxRouteBlocks / kQuarters);
    const RoutePair* lines = route_pairs(p.ws) + (int64_t)group * blocks * kLine + (tid & 7) * 2;
    // all loads at once, at clamped addresses
    RoutePair in[kEach][2];
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const RoutePair* q = lines + min(b0 + i * kRows + tid / 8, blocks - 1) * kLine;
        in[i][0] = q[0];
        in[i][1] = q[1];
    }
    int32_t c[2] = {0, 0};
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const bool have = b0 + i * kRows + tid / 8 < blocks;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            c[h] += have ? in[i][h].count : 0;
            s[h] += have ? (double)in[i][h].sum : 0.0;
        }
    }
    double routed = 0.0;
    if (group == 0) {
        const int32_t* n = route_routed(p.ws, E, blocks);
        const int b = b0 + tid;
        routed = tid < kMaxRouteBlocks / kQuarters && b < blocks ? (double)n[b] : 0.0;
        routed = block_sum<kJoinThreads>(routed, tmp);
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int x = 8; x < 64; x <<= 1) {
            c[h] += __shfl_xor(c[h], x);
            s[h] += __shfl_xor(s[h], x);
        }
        if (lane < 8)
            part[wave][lane * 2 + h] = {s[h], c[h]};
    }
    __syncthreads();
    RouteJoined* joined = route_joined(p.ws, E, blocks);
    double* header = (double*)p.ws + 2;              // each quarter's routed tokens
    if (tid < 64) {                                  // one wave stores, then takes the ticket
        const int e = group * kLine + tid;
        if (tid < kLine && e < E) {
            RouteJoined j = part[0][tid];
#pragma unroll
            for (int w = 1; w < kJoinThreads / 64; w++) {
                j.sum += part[w][tid].sum;
                j.count += part[w][tid].count;
            }
            RouteJoined* to = &joined[(int64_t)quarter * E + e];
            __hip_atomic_store(&to->sum, j.sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&to->count, j.count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (group == 0 && tid == 0)
            __hip_atomic_store(&header[quarter], routed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __threadfence();
        if (tid == 0)
            is_last = __hip_atomic_fetch_add(&p.ws[1], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      (int)(gridDim.x * gridDim.y) - 1;
    }
    __syncthreads();
    if (!is_last)
        return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    double loss = 0.0;
    for (int e = tid; e < E; e += kJoinThreads) {
        RouteJoined j = {0.0, 0};
#pragma unroll
        for (int q = 0; q < kQuarters; q++) {
            j.sum += __hip_atomic_load(&joined[(int64_t)q * E + e].sum, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            j.count += __hip_atomic_load(&joined[(int64_t)q * E + e].count, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
        }
        p.counts[e] = (int32_t)j.count;
        loss += (double)j.count * j.sum;
    }
    double n = 0.0;
#pragma unroll
    for (int q = 0; q < kQuarters; q++)
        n += __hip_atomic_load(&header[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    loss = block_sum<kJoinThreads>(loss, tmp);
    if (tid == 0) {
        p.routed[0] = (int32_t)n;
        if (p.balance) {
            n = n > 0.0 ? n : 1.0;
            p.balance[0] = (float)((double)E * loss / ((double)p.k * n * n));
        }
    }
}

// The gradient of the logits.  The chosen experts' gradients go into an LDS
// row, a lane each, and every lane takes its EPL from there.
template <int DT, int LPT, int EPL, int KIND, int SCORE>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteBwdArgs p) {
    constexpr bool softmax = SCORE == GG_SOFTMAX;
    constexpr bool kFull = DT == GG_F32;
    constexpr int TPW = 64 / LPT;
    constexpr int NJ = LPT >= 32 ? 1 : 32 / LPT;
    constexpr int kCap = LPT * EPL, kPitch = lane_pitch<EPL>();
    __shared__ __align__(16) float at_all[4 * 64 * kPitch];
    typedef typename Elem<DT>::T T;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // a scalar: loops over it are the wave's
    const int g = lane & (LPT - 1), sub = lane / LPT;
    const int first = g * EPL, E = p.E, k = p.k;
    float* at = at_all + (wave * TPW + sub) * LPT * kPitch;

    // c = dL/dp of the balance loss
    __shared__ __align__(16) float c[LPT * kPitch];
    const float n = fmaxf((float)p.routed[0], 1.0f);
    const float cb = p.dbalance ? p.dbalance[0] * (float)E / ((float)k * n * n) : 0.0f;
    for (int e = tid; e < kCap; e += 256)
        c[e / EPL * kPitch + e % EPL] = e < E ? cb * (float)p.counts[e] : 0.0f;
    __syncthreads();

    // Whether every expert's score has a gradient: the balance loss and plain
    // softmax weights are over all of them.  Otherwise only the choices have
    // one, and a NaN elsewhere (an expert that a bias of -inf took out) is not
    // in any of their terms.
    const bool every = p.dbalance || (softmax && !p.normalize);
    const int64_t rows = p.row_of ? p.m_rows : p.T * k;
    const int T_ = (int)p.T;                         // at most 2^23
    const int step = (int)gridDim.x * 4 * TPW;
    for (int t0 = ((int)blockIdx.x * 4 + wave) * TPW; t0 < T_; t0 += step) {
        const int t = t0 + sub;
        const bool live = t < T_;
        const T* row = (const T*)p.logits + (live ? t : 0) * p.ld;

        // a lane per choice: its expert, G = scale * dprob, its logit (loads at
        // clamped addresses, as in load_row)
        int32_t e[NJ], r[NJ];
        float G[NJ], v[NJ];
        bool any = false;
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            const int j = g + s * LPT;
            e[s] = r[s] = -1;
            if (s * LPT < k) {
                const int i = live && j < k ? t * k + j : 0;
                e[s] = p.ids[i];
                r[s] = p.row_of ? p.row_of[i] : i;
            }
        }
        float x[EPL];
        load_row<DT, EPL, KIND>(row, first, E, live, x);
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            G[s] = 0.0f;
            v[s] = -INFINITY;
            if (s * LPT < k) {
                const bool have = r[s] >= 0 && r[s] < rows;
                e[s] = live && g + s * LPT < k && e[s] < E ? e[s] : -1;
                if (rows > 0)
                    G[s] = p.dprob[have ? r[s] : 0];
                v[s] = to_f32<DT>(row[max(e[s], 0)]);
                G[s] = have && e[s] >= 0 ? p.scale * G[s] : 0.0f;
                v[s] = e[s] >= 0 ? v[s] : -INFINITY;
                any |= e[s] >= 0;
            }
        }
#pragma unroll
        for (int i = 0; i < EPL; i += 4)
            *(f32x4*)(at + g * kPitch + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        wave_sync();

        float top = 0.0f, inv = 0.0f, pc = 0.0f;
        if (every) {
            if constexpr (softmax)
                row_scores<LPT, EPL, kFull>(x, true, lane_top(x), top, inv);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const f32x4 four = *(const f32x4*)(c + g * kPitch + i);
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    float score = x[i + h];
                    if constexpr (!softmax) {        // x become the tails
                        x[i + h] = signed_tail<kFull>(score);
                        score = tail_sigmoid(x[i + h]);
                        sum += score;
                    }
                    pc = fmaf(score, four[h], pc);
                }
            }
            if constexpr (!softmax)
                inv = inverse_sum(group_all<LPT>(sum, OpAddF()), false);
            pc = group_all<LPT>(pc, OpAddF()) * inv;
        }

        // weights q (before scale) and their mean gradient sum q G
        if (p.normalize && softmax)
            top = choice_top<LPT, NJ>(v);
        float chosen = 0.0f, qg = 0.0f, slope[NJ] = {};
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            if (s * LPT >= k)                        // no lane's: the wave skips it
                continue;
            const float tail = softmax ? 0.0f : signed_tail<kFull>(v[s]);
            slope[s] = every ? 1.0f : tail_slope(tail);
            v[s] = softmax ? exp_below<kFull>(v[s] - top) : tail_sigmoid(tail);
            chosen += v[s];
            qg = fmaf(v[s], G[s], qg);
        }
        chosen = group_all<LPT>(chosen, OpAddF());
        qg = group_all<LPT>(qg, OpAddF());
        const float norm = p.normalize ? inverse_sum(chosen, softmax) : softmax ? inv : 1.0f;
        const float mean = qg * norm;
        // what a choice adds: to dx (softmax), to ds (sigmoid; dx if !every)
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            if (e[s] < 0)
                continue;
            const float centred = p.normalize ? G[s] - mean : G[s];
            const float d = softmax ? v[s] * norm * centred : centred * norm * slope[s];
            atomicAdd(&at[e[s] / EPL * kPitch + e[s] % EPL], d);
        }
        wave_sync();
        const bool routed = group_first<LPT>(any, lane) >= 0;
        const float pull = pc + (softmax && !p.normalize ? mean : 0.0f);
        if (live) {
            auto gradients = [&](auto of) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    const f32x4 a = *(const f32x4*)(at + g * kPitch + i), b = *(const f32x4*)(c + g * kPitch + i);
#pragma unroll
                    for (int h = 0; h < 4; h++)
                        x[i + h] = routed ? of(x[i + h], a[h], b[h]) : 0.0f;
                }
            };
            // a row without a choice has no gradient
            if (!every)
                gradients([&](float, float a, float) { return a; });
            else if constexpr (softmax)
                gradients([&](float v, float a, float b) { return fmaf(v * inv, b - pull, a); });
            else
                gradients([&](float v, float a, float b) { return fmaf(b - pc, inv, a) * tail_slope(v); });
            store_row<DT, EPL, KIND>((T*)p.dlogits + (int64_t)t * E, first, E, x);
        }
        wave_sync();
    }
}

// ---- launches --------------------------------------------------------------

// Blocks of a route call: a block takes kWaves waves of tokens a pass.  Two
// passes of a single block cost less than joining two blocks (64 tokens of
// 256 experts: 8.3 us a call for 11.1); three cost as much (96: 10.5, 11.0).
static int64_t route_tokens_per_block(int E) { return kWaves * (E <= 64 ? 8 : E <= 256 ? 4 : E <= 512 ? 2 : 1); }

int64_t route_blocks(int64_t T, int E) {
    const int64_t per = route_tokens_per_block(E);
    if (T <= 2 * per)
        return 1;
    const int64_t b = (T + per - 1) / per;
    return b < 1 ? 1 : b > kMaxRouteBlocks ? kMaxRouteBlocks : b;
}

size_t route_workspace(int64_t T, int E) {
    const size_t b = (size_t)route_blocks(T, E);
    return kWsHeader + (size_t)route_lines(E) * b * kLine * sizeof(RoutePair) + (b + 3) / 4 * 16 +
           kQuarters * (size_t)E * sizeof(RouteJoined);
}

// Calls f with the kernels' parameters for E experts of a type: lanes a token,
// experts a lane, how the rows load.  A lane has 16 experts at most, 8 up to 128
// of them.  One table for both kernels, which agree from 65 experts on (the
// measurements above); up to 64 they do not, at 65536 x 64 fp32 the choice
// takes 9.8 us with 8 lanes x 8 and 11.5 with 4 x 16, the gradient 11.6 with 8
// x 8 and 10.2 with 16 x 4.
template <int DT, class F>
static hipError_t by_experts(int E, F f) {
    constexpr int N = row_vector<DT>();
#define GG_KIND(LPT, EPL)                                                     \
    (E % N == 0 ? f(std::integral_constant<int, LPT>(), std::integral_constant<int, EPL>(),    \
                    std::integral_constant<int, kWholeRows>())                                     \
                : f(std::integral_constant<int, LPT>(), std::integral_constant<int, EPL>(),    \
                    std::integral_constant<int, kOddRows>()))
    if (E < N)
        return f(std::integral_constant<int, 8>(), std::integral_constant<int, 8>(),
                 std::integral_constant<int, kShortRows>());
    if (E <= 64)
        return GG_KIND(8, 8);
    if (E <= 128)
        return GG_KIND(16, 8);
    if (E <= 256)
        return GG_KIND(16, 16);
    if (E <= 512)
        return GG_KIND(32, 16);
    return GG_KIND(64, 16);
#undef GG_KIND
}

template <int DT>
static hipError_t route_dt(const RouteArgs& p, hipStream_t s, LaunchInfo* info) {
    const int64_t blocks = route_blocks(p.T, p.E);
    int lanes = 0;
    hipError_t e = by_experts<DT>(p.E, [&](auto LPT, auto EPL, auto KIND) {
        lanes = LPT.value;
        if (p.softmax)
            hipLaunchKernelGGL((route_kernel<DT, LPT.value, EPL.value, KIND.value, GG_SOFTMAX>),
                               dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
        else
            hipLaunchKernelGGL((route_kernel<DT, LPT.value, EPL.value, KIND.value, GG_SIGMOID>),
                               dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
        return hipGetLastError();
    });
    if (e == hipSuccess && blocks > 1) {
        hipLaunchKernelGGL(route_join_kernel, dim3((unsigned)route_lines(p.E), kQuarters),
                           dim3(kJoinThreads), 0, s, p, (int)blocks);
        e = hipGetLastError();
    }
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "route_kernel<%s, %d lanes a token>%s",
                 dtype_name(DT), lanes, blocks > 1 ? " + join" : "");
        info->tm = (int)route_tokens_per_block(p.E);
        info->tn = p.E;
        info->waves = kWaves;
        info->grid = blocks;
    }
    return e;
}

hipError_t launch_route(const RouteArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    return dtype == GG_BF16 ? route_dt<GG_BF16>(p, s, info)
           : dtype == GG_F16 ? route_dt<GG_F16>(p, s, info) : route_dt<GG_F32>(p, s, info);
}

template <int DT>
static hipError_t route_bwd_dt(const RouteBwdArgs& p, hipStream_t s, LaunchInfo* info) {
    return by_experts<DT>(p.E, [&](auto LPT, auto EPL, auto KIND) {
        const int64_t per = 4 * (64 / LPT.value);
        int64_t blocks = (p.T + per - 1) / per;
        if (blocks > 2048)
            blocks = 2048;                           // eight to a CU, then more passes each
        if (p.softmax)
            hipLaunchKernelGGL((route_bwd_kernel<DT, LPT.value, EPL.value, KIND.value, GG_SOFTMAX>),
                               dim3((unsigned)blocks), dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((route_bwd_kernel<DT, LPT.value, EPL.value, KIND.value, GG_SIGMOID>),
                               dim3((unsigned)blocks), dim3(256), 0, s, p);
        if (info) {
            snprintf(info->kernel, sizeof info->kernel, "route_bwd_kernel<%s, %d lanes a token>",
                     dtype_name(DT), LPT.value);
            info->tm = (int)per;
            info->tn = p.E;
            info->waves = 4;
            info->grid = blocks;
        }
        return hipGetLastError();
    });
}

hipError_t launch_route_bwd(const RouteBwdArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    if (p.T == 0)
        return hipSuccess;
    return dtype == GG_BF16 ? route_bwd_dt<GG_BF16>(p, s, info)
           : dtype == GG_F16 ? route_bwd_dt<GG_F16>(p, s, info) : route_bwd_dt<GG_F32>(p, s, info);
}

}  // namespace gg
