// Launch interface of the MXFP4 row quantizer, its inverse and the MXFP4 matrix products (mxfp4.hip).
//
// MXFP4: 32 consecutive elements of a row share a scale 2^(b - 127), b a byte (255: NaN); an element is a code of
// four bits, a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, two to a byte, the even element in the low half. Rows are
// padded with zero codes to Kp, whole 128 elements. Codes are [rows][Kp / 2], scales [Kp / 128][rows][4]: the four
// scales of a row's 128 elements are one dword, and those of consecutive rows are consecutive, so that the scales of
// a product's tile are one contiguous piece per 128 of K (row by row they would be pieces of 8 bytes, a cache line
// each).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ep {

constexpr int64_t kMxMaxK = 1 << 22;        // of a row: the byte offsets of a tile's 256 rows stay below 2^31
constexpr int64_t kMxMaxRows = 1 << 27;     // of a matrix: so do those of the scales of 256 of K

// `rows` rows of K elements of src (ep_dtype EP_F32, EP_BF16 or EP_F16), ldx elements apart, any alignment of the
// element, as rows / M matrices of M rows: Q [rows][Kp / 2], S [rows / M][Kp / 128][M][4]. Q and S 4-byte aligned.
hipError_t launch_quantize_rows_mx(const void* X, int src, int64_t rows, int64_t M, int64_t K, int64_t ldx, uint8_t* Q,
                                   uint8_t* S, hipStream_t stream);

// The values of the first K columns of such codes, [rows][K] of dst (EP_F32, EP_BF16 or EP_F16); Kp is their padded
// width (a multiple of 128, at least K).
hipError_t launch_dequantize_rows_mx(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t M, int64_t Kp, int64_t K,
                                     int dst, void* Y, hipStream_t stream);

// Y[m][n] = sum over blocks b of 2^(sx[m][b] + sw[n][b] - 254) sum_{k in b} X[m][k] W[n][k] (+ bias[n]), fp32 sums,
// rounded once.
struct GemmMxArgs {
    const uint8_t* X;       // [M][K / 2]
    const uint8_t* sx;      // [K / 128][M][4]
    const uint8_t* W;       // [N][K / 2]; with experts [experts][N][K / 2]
    const uint8_t* sw;      // [K / 128][N][4]; with experts [experts][K / 128][N][4]
    const uint16_t* bias;   // [N] bf16 or null; with experts [experts][N]
    void* Y;                // [M][ldy] elements of `out`
    const int32_t* offsets; // experts: [experts + 1] row ranges, ascending from 0; else null
    int M, N, K, ldy;       // K a multiple of 128
    int experts;            // 0: one weight for all rows
    int out;                // ep_dtype EP_BF16, EP_F16 or EP_F32
    int rows;               // rows that the grid is made for: M
};

// Requires 16-byte aligned X and W, 4-byte aligned scales, K at most kMxMaxK, M and N at most kMxMaxRows. With
// experts, rows [offsets[e], offsets[e + 1]) are multiplied by expert e's weight and rows from offsets[experts] on
// are set to zero.
hipError_t launch_gemm_mx(const GemmMxArgs& g, hipStream_t stream);

}  // namespace ep
