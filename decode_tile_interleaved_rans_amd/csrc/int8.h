// Launch interface of the INT8 row quantizer and of the INT8 matrix products (int8.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ep {

// Largest K of an INT8 product, the largest multiple of 16 below 2^17: that many products of two codes, each at
// most 2^14 in magnitude (-128 squared), stay below 2^31, so the int32 sums are exact. A longer row would be
// laid out to 2^17 codes, which nothing tells from a row whose sum leaves int32.
constexpr int64_t kI8MaxK = 131056;

// Per-row INT8 quantization of rows of `src` elements (ep_dtype EP_F32, EP_BF16 or EP_F16):
// Q [M][K], S [M]; see quantize_rows_i8 in int8.hip for the rule. Rows of X are ldx elements apart;
// any alignment of the element size.
hipError_t launch_quantize_rows_i8(const void* X, int src, int M, int K, int64_t ldx, int8_t* Q, float* S,
                                   hipStream_t stream);

// Y[m][n] = sx[m] sw[n] sum_k X[m][k] W[n][k] (+ bias[n]), int32 sums, fp32 epilogue.
struct GemmI8Args {
    const int8_t* X;        // [M][ldx]
    const float* sx;        // [M]
    const int8_t* W;        // [N][ldw]; with experts [experts][N][ldw]
    const float* sw;        // [N]; with experts [experts][N]
    const uint16_t* bias;   // [N] bf16 or null; with experts [experts][N]
    void* Y;                // [M][ldy] elements of `out`
    const int32_t* offsets; // experts: [experts + 1] row ranges, ascending from 0; else null
    int M, N, K, ldx, ldw, ldy;
    int experts;            // 0: one weight for all rows
    int out;                // ep_dtype EP_BF16, EP_F16 or EP_F32
    int rows;               // rows that the tile and the grid are made for: M, or, with offsets that begin past 0, no
                            // less than the rows from offsets[0] on
};

// Requires K % 16 == 0 and 16-byte aligned rows (ldx, ldw multiples of 16, aligned bases) and K at most
// kI8MaxK. With experts, rows [offsets[e], offsets[e + 1]) are multiplied by expert
// e's weight and rows from offsets[experts] on are set to zero.
hipError_t launch_gemm_i8(const GemmI8Args& g, hipStream_t stream);

// dst [count][N] = bias[i] [N] for i < count <= 32; a null bias gives -0, which added to a sum leaves its bits.
hipError_t launch_gather_bias(const uint16_t* const* bias, int count, int N, uint16_t* dst, hipStream_t stream);

// dst [rows][ld] = src [rows][K] with zeros in columns K .. ld - 1 (ld a multiple of 16, dst 16-byte
// aligned, src of any alignment, rows contiguous).
hipError_t launch_pad_rows_i8(const int8_t* src, int64_t rows, int K, int8_t* dst, int ld, hipStream_t stream);

}  // namespace ep
