// gg_clip.hip -- the 2-norm over many tensors, and their clipping by it.
//
// The tensors are one range of elements, cut at `ends` (cumulative element
// counts).  Blocks take equal pieces of the range and find, by a search over
// `ends`, the tensors that a piece covers, so that a thousand small tensors
// and a few large ones make the same kind of work, with no table to build on
// the host.  Squares are summed in 64 bits: no overflow or underflow of a
// square for any fp32 value, and no error of the sum's length.
#include "gg_internal.hpp"
#include "gg_lane.hpp"

namespace gg {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;

// Elements of a piece: about kMaxBlocks pieces, of 2048 elements at least
// (one vector of fp16 per thread) and 32768 at most.
__host__ __device__ inline int64_t piece_size(int64_t total) {
    int64_t c = (total / kMaxBlocks + 2047) / 2048 * 2048;
    return c < 2048 ? 2048 : c > 32768 ? 32768 : c;
}

// First tensor whose end is past element `at` (n if there is none), by a
// 64-way search; the whole wave calls it.
__device__ __forceinline__ int find_tensor(const int64_t* ends, int n, int64_t at) {
    const int lane = threadIdx.x & 63;
    int lo = 0, width = n;
    while (width > 0) {
        const int step = (width + 63) / 64;
        const int64_t q = (int64_t)lo + (int64_t)(lane + 1) * step - 1;
        const int64_t last = (int64_t)lo + width - 1;
        const bool past = q <= last ? ends[q] > at : true;
        const int hit = __ffsll((unsigned long long)__ballot(past)) - 1;
        if (hit < 0)
            return n;
        lo += hit * step;
        if (lo >= n)
            return n;
        if (step == 1)
            return ends[lo] > at ? lo : n;
        width = (int)min((int64_t)step, last - lo + 1);
    }
    return n;
}

// Calls f(i, dtype, a, b) for every tensor i and its elements a .. b-1 within
// the range's elements lo .. hi-1.
template <class F>
__device__ __forceinline__ void walk(const GradArgs& p, int64_t lo, int64_t hi, F f) {
    int i = find_tensor(p.ends, p.n, lo);
    while (i < p.n) {
        const int64_t begin = i ? p.ends[i - 1] : 0, end = p.ends[i];
        if (begin >= hi)
            break;
        const int64_t a = max(lo, begin) - begin, b = min(hi, end) - begin;
        if (a < b)
            f(i, p.dtypes[i], a, b);
        i++;
    }
}

template <int DT>
__device__ __forceinline__ double sum_squares(const void* base, int64_t a, int64_t b) {
    typedef typename Elem<DT>::T T;
    constexpr int N = 16 / (int)sizeof(T);
    const T* q = (const T*)base;
    double s = 0.0;
    const int64_t whole = a + (b - a) / N * N;
    for (int64_t i = a + threadIdx.x * N; i < whole; i += kThreads * N) {
        Vec<DT, N> v;
        v.load(q + i);
#pragma unroll
        for (int j = 0; j < N; j++)
            s = fma((double)v.get(j), (double)v.get(j), s);
    }
    const int64_t i = whole + threadIdx.x;
    if (i < b)
        s = fma((double)to_f32<DT>(q[i]), (double)to_f32<DT>(q[i]), s);
    return s;
}

template <int DT>
__device__ __forceinline__ void scale_range(const void* base, void* out, int64_t a, int64_t b, float factor) {
    typedef typename Elem<DT>::T T;
    constexpr int N = 16 / (int)sizeof(T);
    const T* q = (const T*)base;
    T* o = (T*)out;
    const int64_t whole = a + (b - a) / N * N;
    for (int64_t i = a + threadIdx.x * N; i < whole; i += kThreads * N) {
        Vec<DT, N> v;
        float f[N];
        v.load(q + i);
#pragma unroll
        for (int j = 0; j < N; j++)
            f[j] = v.get(j) * factor;
        v.set(f);
        v.store(o + i);
    }
    const int64_t i = whole + threadIdx.x;
    if (i < b)
        o[i] = from_f32<DT>(to_f32<DT>(q[i]) * factor);
}

// Workspace: header, then a double per block.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(GradArgs p, int64_t piece) {
    __shared__ double tmp[kThreads / 64];
    double s = 0.0;
    for (int64_t lo = (int64_t)blockIdx.x * piece; lo < p.total; lo += (int64_t)gridDim.x * piece)
        walk(p, lo, min(p.total, lo + piece), [&](int i, int dt, int64_t a, int64_t b) {
            const void* q = (const void*)p.ptrs[i];
            if (dt == GG_BF16)
                s += sum_squares<GG_BF16>(q, a, b);
            else if (dt == GG_F16)
                s += sum_squares<GG_F16>(q, a, b);
            else if (dt == GG_F32)
                s += sum_squares<GG_F32>(q, a, b);
        });
    const double all = block_sum<kThreads>(s, tmp);
    if (threadIdx.x == 0) {
        if (gridDim.x == 1)
            p.sumsq[0] = p.accumulate ? p.sumsq[0] + all : all;
        else
            ((double*)(p.ws + kWsHeader / 4))[blockIdx.x] = all;
    }
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(GradArgs p, int blocks) {
    __shared__ double tmp[kThreads / 64];
    const double* part = (const double*)(p.ws + kWsHeader / 4);
    double s = 0.0;
    for (int b = threadIdx.x; b < blocks; b += kThreads)
        s += part[b];
    const double all = block_sum<kThreads>(s, tmp);
    if (threadIdx.x == 0)
        p.sumsq[0] = p.accumulate ? p.sumsq[0] + all : all;
}

__global__ void __launch_bounds__(kThreads) grad_clip_kernel(GradArgs p, int64_t piece) {
    const double norm = sqrt(p.sumsq[0]);
    // min(1, max_norm / (norm + eps)), a NaN kept
    const float ratio = (float)((double)p.max_norm / (norm + (double)p.eps));
    const float factor = ratio >= 1.0f ? 1.0f : ratio;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.norm[0] = (float)norm;
        p.norm[1] = factor;
    }
    const bool in_place = p.out_ptrs == p.ptrs;
    if (in_place && factor == 1.0f)
        return;                                      // every value stays as it is
    for (int64_t lo = (int64_t)blockIdx.x * piece; lo < p.total; lo += (int64_t)gridDim.x * piece)
        walk(p, lo, min(p.total, lo + piece), [&](int i, int dt, int64_t a, int64_t b) {
            const void* q = (const void*)p.ptrs[i];
            void* o = (void*)p.out_ptrs[i];
            if (dt == GG_BF16)
                scale_range<GG_BF16>(q, o, a, b, factor);
            else if (dt == GG_F16)
                scale_range<GG_F16>(q, o, a, b, factor);
            else if (dt == GG_F32)
                scale_range<GG_F32>(q, o, a, b, factor);
        });
}

int64_t grad_blocks(int64_t total) {
    const int64_t c = piece_size(total), b = (total + c - 1) / c;
    return b < 1 ? 1 : b > kMaxBlocks ? kMaxBlocks : b;
}

}  // namespace

size_t grad_workspace() { return kWsHeader + 8 * (size_t)kMaxBlocks; }

static void grad_info(LaunchInfo* info, const char* name, int64_t piece, int64_t blocks) {
    if (!info)
        return;
    snprintf(info->kernel, sizeof info->kernel, "%s", name);
    info->tm = 1;
    info->tn = (int)piece;
    info->waves = kThreads / 64;
    info->grid = blocks;
}

hipError_t launch_grad_norm(const GradArgs& p, hipStream_t s, LaunchInfo* info) {
    const int64_t piece = piece_size(p.total), blocks = grad_blocks(p.total);
    hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, p, piece);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && blocks > 1) {
        hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, s, p, (int)blocks);
        e = hipGetLastError();
    }
    grad_info(info, "grad_norm_kernel", piece, blocks);
    return e;
}

hipError_t launch_grad_clip(const GradArgs& p, hipStream_t s, LaunchInfo* info) {
    const int64_t piece = piece_size(p.total), blocks = grad_blocks(p.total);
    hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, p, piece);
    grad_info(info, "grad_clip_kernel", piece, blocks);
    return hipGetLastError();
}

}  // namespace gg
