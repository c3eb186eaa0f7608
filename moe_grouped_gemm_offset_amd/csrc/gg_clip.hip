// gg_clip.hip -- the 2-norm over many tensors, and their clipping by it.
//
// The tensors are one range of elements, cut at `ends` (cumulative element
// counts).  Blocks take equal pieces of the range and find, by a search over
// `ends`, the tensors that a piece covers: equal work by elements, with no
// table to build on the host.  Within a piece a block takes its tensors one
// after another, each a chain of dependent loads (end, type and address,
// values), so that what costs there is the number of tensors, not their sizes:
// 256 tensors of 16 elements are one piece, 115 us for the norm and 158 for
// the scaling; 1000 of 128 elements 17, 4 and 23 us.  Squares are summed in 64
// bits: no overflow or underflow of a square for any fp32 value, and no error
// of the sum's length.
//
// Memory bound where the tensors are large: 64 of 4096 x 2048 bf16, out of
// place, 162 and 338 us (medians), 6.6 and 6.4 TB/s.  What sets the rate is how
// the blocks are cut.  Each at its fastest: the norm, which only reads, 6.9
// TB/s with 2048 blocks of non-temporal loads, 5.2 without the hint and with
// one load in flight; the scaling, which writes as much as it reads, wants many
// short blocks: pieces of 8192 elements 6.5, of 32768 5.8, of 4096 4.9.  Walking the pieces backwards,
// or loads that stay in the cache, change nothing at 64 MB to 1 GB: the scaling
// finds nothing of the norm's pass.  96 tensors of mixed types, 40000 elements
// on average (10 MB): 5.1, 4.7 and 7.4 us, the latency of the search, the
// addresses and the values behind one another.
#include "gg_lane.hpp"
#include "gg_step.hpp"

namespace gg {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;
constexpr int kNormPiece = 32768, kClipPiece = 8192, kClipBlocks = 1 << 20;

// Elements of a piece: about kMaxBlocks pieces, of 4096 elements at least and
// `most` at most.  (A block's start is what a small piece costs: with 2048 and
// twice the blocks, 3.8 M elements in 96 tensors take 7.0 and 8.1 us for 5.3
// and 7.4; with 8192 as long as with 4096.  Tensors of a few elements are the
// other way round: twice as many of them follow one another in a block.)
int64_t piece_size(int64_t total, int64_t most) {
    int64_t c = (total / kMaxBlocks + 2047) / 2048 * 2048;
    return c < 4096 ? 4096 : c > most ? most : c;
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

// Elements a .. b-1 of a tensor in vectors, kUnroll of a thread's loads at
// once; f(v, i) takes the vector at element i, g(i) a single one at the end.
constexpr int kUnroll = 4;

template <int DT, class F, class G>
__device__ __forceinline__ void sweep(const typename Elem<DT>::T* q, int64_t a, int64_t b, F f, G g) {
    constexpr int N = 16 / (int)sizeof(typename Elem<DT>::T), kStep = kThreads * N;
    const int64_t whole = a + (b - a) / N * N;
    int64_t i = a + threadIdx.x * N;
    for (; i + (kUnroll - 1) * kStep < whole; i += kUnroll * kStep) {
        Vec<DT, N> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            v[u].template load<true>(q + i + u * kStep);
#pragma unroll
        for (int u = 0; u < kUnroll; u++)
            f(v[u], i + u * kStep);
    }
    for (; i < whole; i += kStep) {
        Vec<DT, N> v;
        v.template load<true>(q + i);
        f(v, i);
    }
    if (whole + threadIdx.x < b)
        g(whole + threadIdx.x);
}

template <int DT>
__device__ __forceinline__ double sum_squares(const void* base, int64_t a, int64_t b) {
    typedef typename Elem<DT>::T T;
    constexpr int N = 16 / (int)sizeof(T);
    const T* q = (const T*)base;
    double s = 0.0;
    auto add = [&](float v) { s = fma((double)v, (double)v, s); };
    sweep<DT>(
        q, a, b,
        [&](const Vec<DT, N>& v, int64_t) {
#pragma unroll
            for (int j = 0; j < N; j++)
                add(v.get(j));
        },
        [&](int64_t i) { add(to_f32<DT>(q[i])); });
    return s;
}

template <int DT>
__device__ __forceinline__ void scale_range(const void* base, void* out, int64_t a, int64_t b, float factor) {
    typedef typename Elem<DT>::T T;
    constexpr int N = 16 / (int)sizeof(T);
    const T* q = (const T*)base;
    T* o = (T*)out;
    sweep<DT>(
        q, a, b,
        [&](Vec<DT, N>& v, int64_t i) {
            float f[N];
#pragma unroll
            for (int j = 0; j < N; j++)
                f[j] = v.get(j) * factor;
            v.set(f);
            v.template store<true>(o + i);
        },
        [&](int64_t i) { o[i] = from_f32<DT>(to_f32<DT>(q[i]) * factor); });
}

// Workspace: header (int32 0: the error word, always 0), then a double per
// block.
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
        if (blockIdx.x == 0)
            p.ws[0] = 0;
        if (gridDim.x == 1)
            p.sumsq[0] = p.accumulate ? p.sumsq[0] + all : all;
        else
            ((double*)(p.ws + kWsHeader / 4))[blockIdx.x] = all;
    }
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(GradArgs p, int blocks) {
    __shared__ double tmp[kThreads / 64];
    const double* part = (const double*)(p.ws + kWsHeader / 4);
    double s = 0.0, v[kMaxBlocks / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxBlocks / kThreads; i++)  // all loads at once, at clamped addresses
        v[i] = part[min(i * kThreads + (int)threadIdx.x, blocks - 1)];
#pragma unroll
    for (int i = 0; i < kMaxBlocks / kThreads; i++)
        s += i * kThreads + (int)threadIdx.x < blocks ? v[i] : 0.0;
    const double all = block_sum<kThreads>(s, tmp);
    if (threadIdx.x == 0)
        p.sumsq[0] = p.accumulate ? p.sumsq[0] + all : all;
}

__global__ void __launch_bounds__(kThreads) grad_clip_kernel(GradArgs p, int64_t piece) {
    const double norm = sqrt(p.sumsq[0]);
    // 1 where the limit is not passed (0 / 0 and infinity / infinity among
    // it), else max_norm / (norm + eps); a NaN is kept
    const double with_eps = norm + (double)p.eps;
    const float ratio = (float)((double)p.max_norm / with_eps);
    const float factor = (double)p.max_norm >= with_eps || ratio >= 1.0f ? 1.0f : ratio;
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

int64_t grad_blocks(int64_t total, int64_t piece, int64_t most) {
    const int64_t b = (total + piece - 1) / piece;
    return b < 1 ? 1 : b > most ? most : b;
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
    const int64_t piece = piece_size(p.total, kNormPiece), blocks = grad_blocks(p.total, piece, kMaxBlocks);
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
    const int64_t piece = piece_size(p.total, kClipPiece), blocks = grad_blocks(p.total, piece, kClipBlocks);
    hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, p, piece);
    grad_info(info, "grad_clip_kernel", piece, blocks);
    return hipGetLastError();
}

}  // namespace gg
