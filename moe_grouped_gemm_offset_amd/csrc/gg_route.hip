// gg_route.hip -- the router: top-k choice of experts, their weights, tokens
// per expert and the balance loss; and the gradient of the logits.
//
// Both kernels give each token a group of LPT lanes, each lane EPL
// consecutive experts, so that one pass over the logits holds a token's row
// in registers.  Statistics, weights and gradients are in fp32.
#include <cfloat>

#include "gg_internal.hpp"
#include "gg_lane.hpp"

namespace gg {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr float kTiny = 1e-20f;          // added to sums of sigmoids, which can underflow

__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}

// Order of the choice as unsigned integers: fp32 order with -0 = +0 and NaN on
// top.  kNever and below: a logit or key of -inf, never chosen; 0: taken.
constexpr uint32_t kNever = 0x007FFFFFu;             // the key of -inf

__device__ __forceinline__ uint32_t order_key(float logit, float bias) {
    const float s = logit + bias + 0.0f;
    const uint32_t u = s != s ? 0x7FC00000u : __builtin_bit_cast(uint32_t, s);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The EPL experts of a lane, -inf past the row's end.
template <int DT, int EPL>
__device__ __forceinline__ void load_row(const typename Elem<DT>::T* row, int first, int E, bool live,
                                         float (&x)[EPL]) {
    constexpr int N = EPL * (int)sizeof(typename Elem<DT>::T) >= 16
                          ? 16 / (int)sizeof(typename Elem<DT>::T) : EPL;
#pragma unroll
    for (int c = 0; c < EPL; c += N) {
        if (live && first + c + N <= E) {
            Vec<DT, N> v;
            v.load(row + first + c);
#pragma unroll
            for (int i = 0; i < N; i++)
                x[c + i] = v.get(i);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                x[c + i] = live && first + c + i < E ? to_f32<DT>(row[first + c + i]) : -INFINITY;
        }
    }
}

template <int DT, int EPL>
__device__ __forceinline__ void store_row(typename Elem<DT>::T* row, int first, int E,
                                          const float (&x)[EPL]) {
    constexpr int N = EPL * (int)sizeof(typename Elem<DT>::T) >= 16
                          ? 16 / (int)sizeof(typename Elem<DT>::T) : EPL;
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
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (first + c + i < E)
                    row[first + c + i] = from_f32<DT>(x[c + i]);
        }
    }
}

// 1 / a sum of scores.
__device__ __forceinline__ float inverse_sum(float sum, bool softmax) {
    return softmax ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f / (sum + kTiny);
}

// A token's softmax or sigmoid over its row: x becomes the scores, `inv` what
// turns them into the balance probabilities (softmax: x are exp(x - top), so
// that p = x inv is the softmax as well; a row of -inf gives all zeros).
template <int LPT, int EPL>
__device__ __forceinline__ void row_scores(float (&x)[EPL], bool softmax, float& top, float& inv) {
    float sum = 0.0f;
    if (softmax) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < EPL; i++)
            m = fmaxf(m, x[i]);
        m = group_all<LPT>(m, OpMaxF());
        top = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            x[i] = __expf(x[i] - top);
            sum += x[i];
        }
        sum = group_all<LPT>(sum, OpAddF());
        inv = inverse_sum(sum, true);
    } else {
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            x[i] = sigmoid(x[i]);
            sum += x[i];
        }
        sum = group_all<LPT>(sum, OpAddF());
        inv = inverse_sum(sum, false);
    }
}

// Largest of the chosen logits (0 if there is none).
template <int LPT, int NJ>
__device__ __forceinline__ float choice_top(const float (&v)[NJ]) {
    float m = v[0];
#pragma unroll
    for (int s = 1; s < NJ; s++)
        m = fmaxf(m, v[s]);
    m = group_all<LPT>(m, OpMaxF());
    return m == -INFINITY ? 0.0f : m;
}

}  // namespace

// Workspace: header (int32 1: the finishing ticket), then per block the
// int32 counts and fp32 probability sums of the E experts and the routed
// tokens, [blocks][2E + 1], then a double per expert.
__host__ __device__ inline int64_t route_partial(int E) { return 2 * (int64_t)E + 1; }

// One token per group of LPT lanes and pass.  The choice: every lane keeps
// the largest key of its EPL; a step takes the group's largest (ties: the
// lowest lane, so the lowest experts), rescans that lane's keys -- in LDS,
// one per lane of the group -- for the expert, removes it and hands the lane
// its next largest.
template <int DT, int LPT, int EPL>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs p) {
    static_assert(EPL <= LPT, "a group rescans one lane's keys in one read");
    constexpr int TPW = 64 / LPT;                    // tokens per wave
    constexpr int NJ = LPT >= 32 ? 1 : 32 / LPT;     // choices a lane may hold
    constexpr int kPitch = EPL + 4;                  // words of a lane's keys
    constexpr int kCap = LPT * EPL;
    __shared__ __align__(16) uint32_t keys[kWaves * 64 * kPitch];
    __shared__ int32_t hist[kCap];
    __shared__ int32_t sel[kWaves][TPW][32];
    __shared__ int32_t nrouted;
    typedef typename Elem<DT>::T T;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane & (LPT - 1), sub = lane / LPT;
    const int first = g * EPL;
    const int E = p.E, k = p.k;
    const bool softmax = p.softmax, stats = p.balance != nullptr;
    uint32_t* group_keys = keys + (wave * 64 + sub * LPT) * kPitch;
    uint32_t* my_keys = group_keys + g * kPitch;
    int32_t* my_sel = sel[wave][sub];

    for (int e = tid; e < kCap; e += kThreads)
        hist[e] = 0;
    if (tid == 0) {
        nrouted = 0;
        if (blockIdx.x == 0)
            p.ws[1] = 0;
    }
    float bias[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        // +inf and NaN as the largest finite bias: a logit of -inf stays one
        const float v = p.bias && first + i < E ? p.bias[first + i] : 0.0f;
        bias[i] = v <= FLT_MAX ? v : FLT_MAX;
    }
    float psum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++)
        psum[i] = 0.0f;
    __syncthreads();

    const int64_t step = (int64_t)gridDim.x * kWaves * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * TPW; t0 < p.T; t0 += step) {
        const int64_t t = t0 + sub;
        const bool live = t < p.T;
        const T* row = (const T*)p.logits + (live ? t : 0) * p.ld;
        float x[EPL];
        load_row<DT, EPL>(row, first, E, live, x);
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const uint32_t key = order_key(x[i], bias[i]);
            my_keys[i] = key;
            best = best > key ? best : key;
        }
        wave_sync();
        for (int j = 0; j < k; j++) {
            const uint32_t top = group_all<LPT>(best, OpMaxU());
            const int from = group_first<LPT>(best == top, lane);
            uint32_t* theirs = group_keys + from * kPitch;
            uint32_t v = g < EPL ? theirs[g] : 0u;
            const int at = group_first<LPT>(v == top && g < EPL, lane);
            if (g == at) {
                v = 0;
                theirs[g] = 0;
            }
            const uint32_t next = group_all<LPT>(v, OpMaxU());
            if (g == from)
                best = next;
            if (g == 0)
                my_sel[j] = top > kNever ? from * EPL + at : -1;
            wave_sync();
        }
        // the chosen experts, a lane each (NJ of them if top_k > LPT)
        int32_t e[NJ];
        float v[NJ];
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            const int j = g + s * LPT;
            e[s] = live && j < k ? my_sel[j] : -1;
            v[s] = e[s] >= 0 ? to_f32<DT>(row[e[s]]) : -INFINITY;
        }
        float top = 0.0f, inv = 0.0f;
        if (stats || (softmax && !p.normalize)) {
            row_scores<LPT, EPL>(x, softmax, top, inv);
            if (stats) {
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    psum[i] = fmaf(x[i], inv, psum[i]);
            }
        }
        float norm = softmax ? inv : 1.0f;
        if (p.normalize && softmax)
            top = choice_top<LPT, NJ>(v);
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            v[s] = softmax ? __expf(v[s] - top) : sigmoid(v[s]);
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
    int32_t* part = p.ws + kWsHeader / 4 + blockIdx.x * route_partial(E);
    double loss = 0.0;
    for (int e = tid; e < E; e += kThreads) {
        float s = 0.0f;
        if (stats)
            for (int w = 0; w < kWaves * TPW; w++)
                s += sums[w * kCap + e];
        if (last) {
            p.counts[e] = hist[e];
            loss += (double)hist[e] * (double)s;
        } else {
            part[e] = hist[e];
            part[E + e] = __builtin_bit_cast(int32_t, s);
        }
    }
    if (!last) {
        if (tid == 0)
            part[2 * E] = nrouted;
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

// Joins the blocks' counts and probability sums: 16 experts a block, 64
// runs of blocks each; the block that finishes last adds up the loss.
constexpr int kJoinExperts = 16, kJoinRuns = 64, kJoinThreads = kJoinExperts * kJoinRuns;

__global__ void __launch_bounds__(kJoinThreads) route_join_kernel(RouteArgs p, int blocks) {
    __shared__ int32_t cnt[kJoinRuns][kJoinExperts];
    __shared__ double sum[kJoinRuns][kJoinExperts];
    __shared__ double tmp[kJoinThreads / 64];
    __shared__ int32_t is_last;
    const int tid = threadIdx.x, E = p.E;
    const int run = tid / kJoinExperts, lane = tid % kJoinExperts;
    const int e = blockIdx.x * kJoinExperts + lane;
    const int32_t* part = p.ws + kWsHeader / 4;
    const int64_t pitch = route_partial(E);
    const int each = (blocks + kJoinRuns - 1) / kJoinRuns;
    const int b1 = min(blocks, (run + 1) * each);
    int32_t c = 0;
    double s = 0.0;
    if (e < E) {
        for (int b = run * each; b < b1; b++) {
            c += part[b * pitch + e];
            s += (double)__builtin_bit_cast(float, part[b * pitch + E + e]);
        }
    }
    cnt[run][lane] = c;
    sum[run][lane] = s;
    __syncthreads();
    double* terms = (double*)(p.ws + kWsHeader / 4 + ((int64_t)blocks * pitch + 1) / 2 * 2);
    if (run == 0 && e < E) {
        for (int r = 1; r < kJoinRuns; r++) {
            c += cnt[r][lane];
            s += sum[r][lane];
        }
        p.counts[e] = c;
        __hip_atomic_store(&terms[e], (double)c * s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __threadfence();                             // before this block's ticket
    }
    __syncthreads();
    if (tid == 0)
        is_last = __hip_atomic_fetch_add(&p.ws[1], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                  (int)gridDim.x - 1;
    __syncthreads();
    if (!is_last)
        return;
    double loss = 0.0;
    int32_t n = 0;
    for (int i = tid; i < E; i += kJoinThreads)
        loss += __hip_atomic_load(&terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int b = tid; b < blocks; b += kJoinThreads)
        n += part[b * pitch + 2 * E];
    loss = block_sum<kJoinThreads>(loss, tmp);
    n = (int32_t)block_sum<kJoinThreads>((double)n, tmp);
    if (tid == 0) {
        p.routed[0] = n;
        if (p.balance) {
            const double m = n > 0 ? (double)n : 1.0;
            p.balance[0] = (float)((double)E * loss / ((double)p.k * m * m));
        }
    }
}

// The gradient of the logits.  The chosen experts' gradients go into an LDS
// row, a lane each, and every lane takes its EPL from there.  A block walks
// over tokens, so that a lane's counts are loaded once.
template <int DT, int LPT, int EPL>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteBwdArgs p) {
    constexpr int TPW = 64 / LPT;
    constexpr int NJ = LPT >= 32 ? 1 : 32 / LPT;
    constexpr int kPitch = EPL + 4;
    __shared__ __align__(16) float at_all[4 * 64 * kPitch];
    typedef typename Elem<DT>::T T;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane & (LPT - 1), sub = lane / LPT;
    const int first = g * EPL, E = p.E, k = p.k;
    float* at = at_all + (wave * 64 + sub * LPT) * kPitch;
    float* my_at = at + g * kPitch;

    // c = dL/dp of the balance loss
    float c[EPL];
    const float n = fmaxf((float)p.routed[0], 1.0f);
    const float cb = p.dbalance ? p.dbalance[0] * (float)E / ((float)k * n * n) : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; i++)
        c[i] = p.dbalance && first + i < E ? cb * (float)p.counts[first + i] : 0.0f;

    const int64_t step = (int64_t)gridDim.x * 4 * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * TPW; t0 < p.T; t0 += step) {
        const int64_t t = t0 + sub;
        const bool live = t < p.T;
        const T* row = (const T*)p.logits + (live ? t : 0) * p.ld;

        // a lane per choice: its expert, G = scale * dprob, its logit
        int32_t e[NJ];
        float G[NJ], v[NJ];
        bool any = false;
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            const int j = g + s * LPT;
            e[s] = -1;
            G[s] = 0.0f;
            if (live && j < k) {
                const int64_t i = t * k + j;
                e[s] = p.ids[i];
                if (e[s] >= E)
                    e[s] = -1;
                const int64_t r = p.row_of ? (int64_t)p.row_of[i] : i;
                if (!p.row_of || (r >= 0 && r < p.m_rows))
                    G[s] = p.scale * p.dprob[r];
            }
        }
        float x[EPL];
        load_row<DT, EPL>(row, first, E, live, x);
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            v[s] = e[s] >= 0 ? to_f32<DT>(row[e[s]]) : -INFINITY;
            any |= e[s] >= 0;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            my_at[i] = 0.0f;
        wave_sync();

        float top = 0.0f, inv = 0.0f;
        row_scores<LPT, EPL>(x, p.softmax, top, inv);
        float pc = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            pc = fmaf(x[i], c[i], pc);
        pc = group_all<LPT>(pc, OpAddF()) * inv;

        // weights q (before scale) and their mean gradient sum q G
        if (p.normalize && p.softmax)
            top = choice_top<LPT, NJ>(v);
        float chosen = 0.0f, qg = 0.0f;
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            v[s] = p.softmax ? __expf(v[s] - top) : sigmoid(v[s]);
            if (e[s] < 0)
                v[s] = G[s] = 0.0f;
            chosen += v[s];
            qg = fmaf(v[s], G[s], qg);
        }
        chosen = group_all<LPT>(chosen, OpAddF());
        qg = group_all<LPT>(qg, OpAddF());
        const float norm = p.normalize ? inverse_sum(chosen, p.softmax) : p.softmax ? inv : 1.0f;
        const float mean = qg * norm;
        // what a choice adds: to dx (softmax), to ds (sigmoid)
#pragma unroll
        for (int s = 0; s < NJ; s++) {
            if (e[s] < 0)
                continue;
            const float centred = p.normalize ? G[s] - mean : G[s];
            const float d = p.softmax ? v[s] * norm * centred : centred * norm;
            atomicAdd(&at[e[s] / EPL * kPitch + e[s] % EPL], d);
        }
        wave_sync();
        const bool routed = group_first<LPT>(any, lane) >= 0;
        const float pull = pc + (p.softmax && !p.normalize ? mean : 0.0f);
        if (live) {
            float dx[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                const float a = my_at[i];
                if (p.softmax)
                    dx[i] = fmaf(x[i] * inv, c[i] - pull, a);
                else
                    dx[i] = fmaf(c[i] - pc, inv, a) * x[i] * (1.0f - x[i]);
                if (!routed)
                    dx[i] = 0.0f;
            }
            store_row<DT, EPL>((T*)p.dlogits + t * E, first, E, dx);
        }
        wave_sync();
    }
}

// ---- launches --------------------------------------------------------------

// Blocks of a route call: a block takes kWaves waves of tokens a pass; up to
// 512 of them (two to a CU), then more passes each.
static int64_t route_tokens_per_block(int E) { return kWaves * (E <= 64 ? 8 : E <= 256 ? 4 : E <= 512 ? 2 : 1); }

int64_t route_blocks(int64_t T, int E) {
    const int64_t per = route_tokens_per_block(E);
    const int64_t b = (T + per - 1) / per;
    return b < 1 ? 1 : b > 512 ? 512 : b;
}

size_t route_workspace(int64_t T, int E) {
    return kWsHeader + ((size_t)route_blocks(T, E) * route_partial(E) + 1) / 2 * 8 + 8 * (size_t)E;
}

template <int DT>
static hipError_t route_dt(const RouteArgs& p, hipStream_t s, LaunchInfo* info) {
    const int64_t blocks = route_blocks(p.T, p.E);
    const dim3 grid((unsigned)blocks), th(kThreads);
    int lpt;
    if (p.E <= 64) {
        lpt = 8;
        hipLaunchKernelGGL((route_kernel<DT, 8, 8>), grid, th, 0, s, p);
    } else if (p.E <= 128) {
        lpt = 16;
        hipLaunchKernelGGL((route_kernel<DT, 16, 8>), grid, th, 0, s, p);
    } else if (p.E <= 256) {
        lpt = 16;
        hipLaunchKernelGGL((route_kernel<DT, 16, 16>), grid, th, 0, s, p);
    } else if (p.E <= 512) {
        lpt = 32;
        hipLaunchKernelGGL((route_kernel<DT, 32, 16>), grid, th, 0, s, p);
    } else {
        lpt = 64;
        hipLaunchKernelGGL((route_kernel<DT, 64, 16>), grid, th, 0, s, p);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && blocks > 1) {
        hipLaunchKernelGGL(route_join_kernel, dim3((unsigned)((p.E + kJoinExperts - 1) / kJoinExperts)),
                           dim3(kJoinThreads), 0, s, p, (int)blocks);
        e = hipGetLastError();
    }
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "route_kernel<%s, %d lanes a token>%s",
                 dtype_name(DT), lpt, blocks > 1 ? " + join" : "");
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

template <int DT, int LPT, int EPL>
static hipError_t route_bwd_go(const RouteBwdArgs& p, hipStream_t s, LaunchInfo* info) {
    const int64_t per = 4 * (64 / LPT);
    int64_t blocks = (p.T + per - 1) / per;
    if (blocks > 2048)
        blocks = 2048;                               // eight to a CU, then more passes each
    hipLaunchKernelGGL((route_bwd_kernel<DT, LPT, EPL>), dim3((unsigned)blocks), dim3(256), 0, s, p);
    if (info) {
        snprintf(info->kernel, sizeof info->kernel, "route_bwd_kernel<%s, %d lanes a token>",
                 dtype_name(DT), LPT);
        info->tm = (int)per;
        info->tn = p.E;
        info->waves = 4;
        info->grid = blocks;
    }
    return hipGetLastError();
}

template <int DT>
static hipError_t route_bwd_dt(const RouteBwdArgs& p, hipStream_t s, LaunchInfo* info) {
    if (p.E <= 64)
        return route_bwd_go<DT, 8, 8>(p, s, info);
    if (p.E <= 128)
        return route_bwd_go<DT, 16, 8>(p, s, info);
    if (p.E <= 256)
        return route_bwd_go<DT, 16, 16>(p, s, info);
    if (p.E <= 512)
        return route_bwd_go<DT, 32, 16>(p, s, info);
    return route_bwd_go<DT, 64, 16>(p, s, info);
}

hipError_t launch_route_bwd(const RouteBwdArgs& p, int dtype, hipStream_t s, LaunchInfo* info) {
    if (p.T == 0)
        return hipSuccess;
    return dtype == GG_BF16 ? route_bwd_dt<GG_BF16>(p, s, info)
           : dtype == GG_F16 ? route_bwd_dt<GG_F16>(p, s, info) : route_bwd_dt<GG_F32>(p, s, info);
}

}  // namespace gg
