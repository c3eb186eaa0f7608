// gg_step.hpp -- parameter blocks and launchers of the calls around the grouped
// GEMMs (router, dispatch and combine, gradient clipping), shared between
// gg_api_moe.cpp and the kernel translation units.  Not part of the ABI.
#pragma once
#include "gg_internal.hpp"

namespace gg {

// The router (gg_route, gg_route_bwd).
struct RouteArgs {
    const void* logits;       // (T, E), row pitch ld
    int64_t ld, T;
    int E, k;
    const float* bias;        // [E] or null: added for the choice only
    int softmax, normalize;
    float scale;
    int32_t* ids;             // (T, k)
    float* prob;              // (T, k)
    int32_t* counts;          // [E]
    int32_t* routed;          // [1]
    float* balance;           // [1] or null
    int32_t* ws;
};

struct RouteBwdArgs {
    const void* logits;
    int64_t ld, T;
    int E, k;
    const int32_t* ids;
    const int32_t* counts;
    const int32_t* routed;
    int softmax, normalize;
    float scale;
    const float* dprob;       // (T, k), or [m_rows] with row_of
    const int32_t* row_of;    // (T, k) or null
    int64_t m_rows;
    const float* dbalance;    // [1] or null
    void* dlogits;            // (T, E)
};

// Dispatch to the expert-sorted rows and back.
struct PlanArgs {
    const int32_t* ids;       // (T, k)
    int64_t T, m_rows;
    int E, k, granule;
    const float* prob;        // (T, k) or null
    int32_t* counts;          // [E]
    int32_t* ends;            // [E]
    int32_t* row_of;          // (T, k)
    float* prob_rows;         // [m_rows] or null
    int32_t* ws;
};

struct RowsArgs {
    const void* tokens;       // (T, width), row pitch ld: x (permute), dout (combine_bwd)
    void* out;                // (T, width), row pitch ld (combine)
    int64_t ld, T, m_rows;
    int width, k, E;
    const int32_t* row_of;    // (T, k)
    const int32_t* counts;    // [E]
    const int32_t* ends;      // [E]
    const void* rows_in;      // (m_rows, width): y
    void* rows_out;           // (m_rows, width): x_rows, dy_rows
    const float* weights;     // (T, k) or null
    float* dweights;          // (T, k)
};

// Gradient norm and clipping over many tensors.
struct GradArgs {
    const int64_t* ptrs;      // [n] tensors
    const int64_t* out_ptrs;  // [n] (the tensors themselves: in place)
    const int64_t* ends;      // [n] cumulative element counts
    const int32_t* dtypes;    // [n]
    int n;
    int64_t total;
    double* sumsq;            // [1]
    int accumulate;
    float max_norm, eps;
    float* norm;              // [2]: norm, factor
    int32_t* ws;
};

// Bytes of workspace that a route, plan or norm call uses.
size_t route_workspace(int64_t T, int E);
size_t plan_workspace(int64_t T, int E);
size_t grad_workspace();
// Launchers: the HIP status of the launch; *info, where given, says what was
// launched.
hipError_t launch_route(const RouteArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_route_bwd(const RouteBwdArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_plan(const PlanArgs& p, hipStream_t s, LaunchInfo* info);
hipError_t launch_permute(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_combine(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_combine_bwd(const RowsArgs& p, int dtype, hipStream_t s, LaunchInfo* info);
hipError_t launch_grad_norm(const GradArgs& p, hipStream_t s, LaunchInfo* info);
hipError_t launch_grad_clip(const GradArgs& p, hipStream_t s, LaunchInfo* info);

}  // namespace gg
