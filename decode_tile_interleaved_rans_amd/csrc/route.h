// Launch interface of the expert routing kernels (route.hip): tokens sorted by expert, summed back
// with their weights, and the gradients.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ep {

constexpr int kRouteMaxExperts = 1024;

// The choices of T tokens, k experts each.
struct RouteArgs {
    const void* ids;        // [T][k] int32 or int64 expert numbers; any other than 0 .. E - 1 is dropped
    int id_bytes;           // 4 or 8
    int64_t T;
    int k, E;
    int32_t* offsets;       // out [E + 1]
    int32_t* pos;           // out [T][k]: row of the choice, or -1 - row behind the experts' when dropped
};

// Scratch of launch_sort_tokens (0 when the choices fit one block).
size_t sort_tokens_scratch(int64_t T, int k, int E);

// offsets, pos and rows [T k][row_bytes]: rows[pos[t][j]] = x[t], zeros in the rows of dropped choices.
// Rows of x are ldx_bytes apart. T k < 2^31. rows may be null (offsets and pos only).
hipError_t launch_sort_tokens(const RouteArgs& r, const void* x, int64_t ldx_bytes, int64_t row_bytes, void* rows,
                              void* scratch, hipStream_t stream);

// One token's rows and weights, shared by the sum and its gradient.
struct CombineArgs {
    const void* ys;         // [R][H]
    const int32_t* pos;     // [T][k]
    const float* w;         // [T][k] or null (ones)
    int64_t T, H, R;
    int k;
    int dtype;              // ep_dtype EP_F32, EP_BF16 or EP_F16, of ys, y, dy and d_ys
};

// y [T][H] = sum over j, in order, of w[t][j] ys[pos[t][j]] (dropped choices left out), fp32 sums.
hipError_t launch_combine_tokens(const CombineArgs& c, void* y, hipStream_t stream);

// d_ys [R][H]: row pos[t][j] = w[t][j] dy[t], zeros in the rows of dropped choices; d_w [T][k] =
// <dy[t], ys[pos[t][j]]> (0 for a dropped choice), fp32 sums. Either may be null; ys may be null
// when d_w is.
hipError_t launch_combine_tokens_grad(const CombineArgs& c, const void* dy, void* d_ys, float* d_w, hipStream_t stream);

}  // namespace ep
