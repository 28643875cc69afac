// Launch interface of the expert layer for few tokens (mlp.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ep {

constexpr int kMlpMaxTokens = 64;       // one bit each of an expert's mask
constexpr int kMlpMaxChoices = 1024;    // T k

// y[t] = sum over j of w[t][j] (W_out[e] h + b_out[e]), h = silu(g) u, (g, u) = W_in[e] x[t] + b_in[e], e = ids[t][j].
struct MlpArgs {
    const void* x;              // [T] rows of H elements of `act`, ldx apart
    const void* ids;            // [T][k] int32 or int64 expert numbers; any other than 0 .. E - 1 is dropped
    const float* w;             // [T][k] or null (ones)
    const void* w_in;           // [E][2 I][H] of `act` or MXFP4 codes [E][2 I][Hp / 2]; rows 0 .. I - 1 give g, the others u
    const uint8_t* s_in;        // null, or the codes' scales [E][Hp / 128][2 I][4]
    const uint16_t* b_in;       // [E][2 I] bf16 or null
    const void* w_out;          // [E][N][I] of `act` or codes [E][N][Ip / 2]
    const uint8_t* s_out;       // null, or [E][Ip / 128][N][4]
    const uint16_t* b_out;      // [E][N] bf16 or null
    void* scratch;              // mlp_scratch() bytes, 16-byte aligned
    void* y;                    // [T][N] of `act`
    int64_t ldx;
    int T, k, E, H, I, N;
    int id_bytes;               // 4 or 8
    int act;                    // ep_dtype EP_BF16 or EP_F16
};

// mx: the weights are MXFP4.
size_t mlp_scratch(int64_t T, int64_t k, int64_t E, int64_t I, int64_t N, bool mx);

// T at most kMlpMaxTokens, T k at most kMlpMaxChoices, E at most kRouteMaxExperts.
hipError_t launch_mlp(const MlpArgs& a, hipStream_t stream);

}  // namespace ep
