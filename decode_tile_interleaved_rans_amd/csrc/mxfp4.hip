// gfx950 MXFP4 row quantizer, its inverse, and MXFP4 matrix products: Y[m][n] = sum over blocks b of 32 of
// 2^(sx[m][b] + sw[n][b] - 254) sum_{k in b} X[m][k] W[n][k] (+ bias[n]) on the matrix cores, which take the codes
// and the scale bytes as they are (v_mfma_scale_f32_16x16x128_f8f6f4 and 32x32x64), fp32 sums. The format and its layout stand in
// mxfp4.h.
//
// Operand lane layout of the 16-row instruction (checked on the device): lane l supplies 32 codes (16 bytes) of A row l % 16 and of B column
// l % 16, K group l / 16, and a scale byte for each, and receives C[4 (l / 16) + i][l % 16], i < 4. A and B take the
// same K positions per lane, so equal k meet whatever the order. W is the A operand and X the B operand: a lane then
// holds four consecutive output columns of one row. A scale byte of 255 gives NaN, whatever the codes.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "entropack.h"
#include "kernels.h"
#include "mx_tiles.h"
#include "mxfp4.h"
#include "tiles.h"

namespace ep {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// --------------------------------------------------------------------------- quantizer and inverse
// A block's scale byte is b = max(0, e - 2), e the biased exponent of max |x| as an fp32 number: 2^(b - 127) = 2^(floor
// (log2 max |x|) - 2), which puts the largest magnitude into [4, 8) of the codes' range. Codes are x / 2^(b - 127)
// rounded to nearest, ties to the even code, at most 6 in magnitude (v_cvt_scalef32_pk_fp4_f32 does just that, for
// subnormal numbers and scales too: checked on the device against the definition at and next to every rounding
// border of every scale). A block with an infinity or a NaN gets b = 255 and codes 0, so that every product with it
// is NaN instead of a plausible number.
//
// Every block of 32 stands alone, so a wave takes 16 rows x 128 columns: four lanes to a block, eight elements
// to a lane, four rows to a load; the maximum goes over the four lanes (DPP). The scales of 16 rows
// leave in one store of 64 bytes. Bound by HBM: 4096 x 10240 BF16 in 20 us, 5.3 TB/s; one row takes a launch (4 us).
template <int SRC> struct Elem { typedef uint16_t type; };
template <> struct Elem<EP_F32> { typedef uint32_t type; };

template <int SRC>
__device__ __forceinline__ float elem_value(uint32_t bits) {
    if constexpr (SRC == EP_F32) return __uint_as_float(bits);
    if constexpr (SRC == EP_BF16) return __uint_as_float(bits << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

template <int SRC>
struct Eight {
    typename Elem<SRC>::type e[8];
    typedef uint32_t Words __attribute__((ext_vector_type(2 * sizeof(typename Elem<SRC>::type)), aligned(sizeof(typename Elem<SRC>::type))));
    // rows of any alignment of the element, past the caches: 4096 x 10240 BF16 quantized in 20 us for 23.5 with ordinary loads
    // and stores, the values of the codes written in 17 for 25
    __device__ __forceinline__ void load(const void* p) {
        const Words w = __builtin_nontemporal_load(static_cast<const Words*>(p));
        __builtin_memcpy(e, &w, sizeof e);
    }
    __device__ __forceinline__ void store(void* p) const {
        Words w;
        __builtin_memcpy(&w, e, sizeof e);
        __builtin_nontemporal_store(w, static_cast<Words*>(p));
    }
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// What a wave works on: rows r0 ... of matrix e, the 128 columns of chunk c.
struct MxPart {
    int64_t e, r0, c;
};
__device__ __forceinline__ MxPart mx_part(int64_t unit, int64_t row_groups, int64_t col_groups) {
    const int64_t cg = unit % col_groups, rest = unit / col_groups;
    return MxPart{rest / row_groups, 16 * (rest % row_groups), 4 * cg + (threadIdx.x >> 6)};
}

template <int SRC>
__global__ __launch_bounds__(256) void quantize_rows_mx(const void* Xv, int64_t M, int64_t K, int64_t ldx, uint8_t* Q, uint8_t* S,
                                                        int64_t chunks, int64_t row_groups, int64_t units) {
    typedef typename Elem<SRC>::type T;
    const int64_t col_groups = (chunks + 3) / 4;
    const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const MxPart at = mx_part(u, row_groups, col_groups);
        if (at.c >= chunks) continue;
        const int64_t k = 128 * at.c + 8 * p;
        const int left = (int)(K - k < 8 ? (K - k > 0 ? K - k : 0) : 8);      // elements of the row from k on
        Eight<SRC> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = at.r0 + 4 * j + g;
            const T* x = static_cast<const T*>(Xv) + (at.e * M + m) * ldx + k;
            if (m < M && left == 8) {
                v[j].load(x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j].e[i] = m < M && i < left ? x[i] : 0;
            }
        }
        uint32_t scale = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = at.r0 + 4 * j + g;
            float f[8];
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = elem_value<SRC>(v[j].e[i]);
                const uint32_t b = __float_as_uint(f[i]) & 0x7FFFFFFFu;
                a = a > b ? a : b;
            }
            uint32_t o = dpp<0xB1>(a);                                      // the lane beside, then the pair beside
            a = a > o ? a : o;
            o = dpp<0x4E>(a);
            a = a > o ? a : o;
            const bool bad = a >= 0x7F800000u;
            const uint32_t e8 = a >> 23, b8 = bad ? 255u : e8 > 2 ? e8 - 2 : 0u;
            const float unit = __uint_as_float((bad ? 127u : b8) << 23);      // exponent bits 0 stand for 2^-127 here
            uint32_t q = 0;
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0], f[1], unit, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], unit, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], unit, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], unit, 3);
            q = bad ? 0u : q;
            if (m < M) __builtin_nontemporal_store(q, reinterpret_cast<uint32_t*>(Q + (at.e * M + m) * (chunks * 64) + k / 2));
            uint32_t s = b8 << (8 * (p >> 2));                              // the row's four scales, in all its 16 lanes
            s |= dpp<0x124>(s);
            s |= dpp<0x128>(s);
            if (p == j) scale = s;                                          // lane p < 4 keeps row 4 p + g
        }
        const int64_t m = at.r0 + 4 * p + g;
        if (p < 4 && m < M) __builtin_memcpy(S + ((at.e * chunks + at.c) * M + m) * 4, &scale, 4);
    }
}

// The inverse: a lane turns the eight codes of a dword into values, exactly in BF16 and FP32 (up to scale bytes
// of 252, the largest that the quantizer gives; above it 6 times the scale passes their range), rounded once in FP16.
template <int DST>
__device__ __forceinline__ void eight_values(uint32_t q, float unit, Eight<DST>* out) {
    auto two = [&](auto sel) {
        constexpr int s = decltype(sel)::value;
        if constexpr (DST == EP_BF16) {
            const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, s));
            out->e[2 * s] = (uint16_t)v, out->e[2 * s + 1] = (uint16_t)(v >> 16);
        } else if constexpr (DST == EP_F16) {
            const uint32_t v = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, s));
            out->e[2 * s] = (uint16_t)v, out->e[2 * s + 1] = (uint16_t)(v >> 16);
        } else {
            const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, unit, s);
            out->e[2 * s] = __float_as_uint(v[0]), out->e[2 * s + 1] = __float_as_uint(v[1]);
        }
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    two(std::integral_constant<int, 2>{});
    two(std::integral_constant<int, 3>{});
}

template <int DST>
__global__ __launch_bounds__(256) void dequantize_rows_mx(const uint8_t* Q, const uint8_t* S, int64_t M, int64_t chunks, int64_t K,
                                                          void* Yv, int64_t row_groups, int64_t units) {
    typedef typename Elem<DST>::type T;
    const int64_t col_groups = (chunks + 3) / 4;
    const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const MxPart at = mx_part(u, row_groups, col_groups);
        const int64_t k = 128 * at.c + 8 * p;
        if (at.c >= chunks || k >= K) continue;
        uint32_t q[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = at.r0 + 4 * j + g;
            q[j] = s[j] = 0;
            if (m < M) {
                __builtin_memcpy(&q[j], Q + (at.e * M + m) * (chunks * 64) + k / 2, 4);
                __builtin_memcpy(&s[j], S + ((at.e * chunks + at.c) * M + m) * 4, 4);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = at.r0 + 4 * j + g;
            if (m >= M) continue;
            Eight<DST> v;
            // a byte of 255 makes the unit an infinity, which the conversion takes for the format's NaN
            eight_values<DST>(q[j], __uint_as_float((s[j] >> (8 * (p >> 2)) & 255u) << 23), &v);
            T* y = static_cast<T*>(Yv) + (at.e * M + m) * K + k;
            if (K - k >= 8) {
                v.store(y);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < K - k) y[i] = v.e[i];
            }
        }
    }
}

struct MxGrid {
    int64_t chunks, row_groups, units;
    unsigned blocks;
};
MxGrid mx_grid(int64_t rows, int64_t M, int64_t K) {
    MxGrid g;
    g.chunks = (K + 127) / 128;
    g.row_groups = (M + 15) / 16;
    g.units = rows / M * g.row_groups * ((g.chunks + 3) / 4);
    g.blocks = (unsigned)(g.units < (1 << 22) ? g.units : 1 << 22);          // a grid may have at most 2^32 - 1 threads
    return g;
}

// ------------------------------------------------------------------------------- tiled product
// The ring of the INT8 product (int8.hip) on rows of 128 bytes, 256 codes, a step: both operand tiles go from global
// memory straight into LDS, S stages deep, and the fragments of the next sub-step are read behind the current
// MFMAs. The K group of a lane takes neighbouring chunks of the row in the sub-steps of a step, so that its scale bytes
// are neighbours in one dword and the instruction picks the byte. The scales of a stage are two dwords per row, loaded
// into LDS beside the codes: [2][rows], a contiguous piece of each 128 columns.
//
// 4096 x 8192 x 8192 takes 117-124 us (boxes differ), 4.4-4.7 PFLOP/s, of which 20 go to the starts of the two rounds of
// tiles and their 67 MB of outputs. Per 4096 of K it takes 53 us, 5.1 PFLOP/s: the matrix cores alone, without any memory,
// reach 7.2 on random codes, where the card holds 1.7-1.9 GHz (9.9 on zeros). They are busy for 65% of the cycles.
template <int ROWS>
constexpr int scale_words() { return 2 * ROWS < 64 ? 64 : 2 * ROWS; }

// The scale loads of one stage, dealt over the waves: every wave issues kEach loads, of its own part of X's or W's
// scales or, behind the last, of zeros into the spare KiB.
template <int BM, int BN, int NW>
struct ScaleDma {
    static constexpr int kX = scale_words<BM>() / 64, kW = scale_words<BN>() / 64, kEach = (kX + kW + NW - 1) / NW;
    const uint8_t *x, *w;           // the scales of the tile's first row, chunk 0
    int64_t px, pw;                 // bytes between chunks
    int rx, rw;                     // rows of the tile that are there
    __device__ __forceinline__ void load(int step, int chunks, uint8_t* lds, uint8_t* spare, int wave) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = wave + NW * j;                                    // uniform
            const bool isx = i < kX, any = i < kX + kW;
            const int at = 64 * (isx ? i : i - kX) + lane, rows = isx ? BM : BN;
            const int c = isx ? at / BM : at / BN, r = isx ? at % BM : at % BN;
            const int64_t pitch = isx ? px : pw;
            const uint8_t* base = (isx ? x : w) + 2 * (int64_t)step * pitch;
            const bool in = any && at < 2 * rows && r < (isx ? rx : rw) && 2 * step + c < chunks;
            const uint32_t off = in ? (uint32_t)(c * (int)pitch + 4 * r) : kOob;
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0x7FFFFFFF, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(any ? lds + 256 * i : spare), 4, off, 0, 0, 0);
        }
    }
};

// The matrix instruction of a tile: MR = 16 (v_mfma_scale_f32_16x16x128_f8f6f4) or 32 (v_mfma_scale_f32_32x32x64_f8f6f4,
// lane l with row l % 32, K group l / 32 of two, C[8 (i / 4) + 4 (l / 32) + i % 4][l % 32]). A step of 256 codes takes
// kSub sub-steps; in sub-step s a lane of K group g reads chunk kSub g + s of the row.
template <int MR>
struct Instr {
    static constexpr int kSub = MR == 16 ? 2 : 4, kQuads = MR * MR / 256;    // quads: four consecutive rows of C in a lane
    typedef float Acc __attribute__((ext_vector_type(4 * kQuads)));
    static __device__ __forceinline__ int row() { return threadIdx.x & (MR - 1); }
    static __device__ __forceinline__ int group() { return (threadIdx.x & 63) / MR; }
};

// Slot (before the swizzle) of the chunk that K group g reads in sub-step s: the groups of one sub-step side by side for
// MR = 16, whose 64 lanes cover all banks only then (a third of the cycles of LDS went to conflicts with the chunks in
// their own order); chunk_of is the inverse.
template <int MR>
__device__ __forceinline__ int slot_of(int g, int s) { return MR == 16 ? 4 * s + g : 4 * g + s; }
template <int MR>
__device__ __forceinline__ int chunk_of(int slot) { return MR == 16 ? 2 * (slot & 3) + (slot >> 2) : slot; }

// Fragments of T parts of MR rows from row r0 of an operand tile, sub-step s of a stage.
template <int MR, int T>
__device__ __forceinline__ void read_frags(const uint8_t* tile, int r0, int s, i32x4 (&f)[T]) {
    const int r = r0 + Instr<MR>::row();
    const uint8_t* p = tile + r * 128 + ((slot_of<MR>(Instr<MR>::group(), s) ^ chunk_swizzle(r)) << 4);
#pragma unroll
    for (int i = 0; i < T; ++i) f[i] = *reinterpret_cast<const i32x4*>(p + MR * 128 * i);
}

// Their scales, byte s for sub-step s; ROWS rows in the tile.
template <int MR, int ROWS, int T>
__device__ __forceinline__ void read_scales(const uint8_t* scales, int r0, int (&s)[T]) {
    const int g = Instr<MR>::group();
    const uint8_t* p = scales + 4 * ((MR == 16 ? g >> 1 : g) * ROWS + r0 + Instr<MR>::row());
#pragma unroll
    for (int i = 0; i < T; ++i) s[i] = *reinterpret_cast<const int*>(p + 4 * MR * i) >> (MR == 16 ? 16 * (g & 1) : 0);
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

template <int MR, int H, int TI, int TJ>
__device__ __forceinline__ void multiply(const i32x4 (&x)[TI], const i32x4 (&w)[TJ], const int (&sx)[TI], const int (&sw)[TJ],
                                         typename Instr<MR>::Acc (&acc)[TI][TJ]) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
            if constexpr (MR == 16)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(w[j]), widen(x[i]), acc[i][j], 4, 4, H, sw[j], H, sx[i]);
            else
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(w[j]), widen(x[i]), acc[i][j], 4, 4, H, sw[j], H, sx[i]);
}

// Four consecutive columns of a part, from column n of the matrix on, with the bias; count of them are in the matrix.
__device__ __forceinline__ void load_bias(const GemmMxArgs& g, int e, int n, int count, float (&bias)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) bias[c] = c < count ? __uint_as_float((uint32_t)g.bias[(int64_t)e * g.N + n + c] << 16) : 0.0f;
}

// The epilogue of a wave's TI x TJ parts of MR x MR: rows m0 + MR i + the lane's, columns n0 + MR j + 8 q + 4 (K group),
// stored from the registers, four columns a lane: the small tiles.
template <int OUT, int MR, int TI, int TJ>
__device__ __forceinline__ void store_tile(const GemmMxArgs& g, const TileAt& t, int m0, int n0,
                                           const typename Instr<MR>::Acc (&acc)[TI][TJ]) {
    const bool vec = vec_out(g);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < Instr<MR>::kQuads; ++q) {
            const int n = n0 + MR * j + 8 * q + 4 * Instr<MR>::group(), count = g.N - n < 4 ? g.N - n : 4;
            if (count <= 0) continue;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (g.bias) load_bias(g, t.e, n, count, bias);
#pragma unroll
            for (int i = 0; i < TI; ++i) {
                const int m = m0 + MR * i + Instr<MR>::row();
                if (m >= t.m_end) continue;
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = g.bias ? acc[i][j][4 * q + c] + bias[c] : acc[i][j][4 * q + c];
                store4<OUT>(g.Y, (int64_t)m * g.ldy + n, v, count, vec);
            }
        }
}

// The same through LDS, MR rows at a time in a region of the wave's own, so that it stores whole rows of its columns, 16
// bytes a lane (of any alignment): from the registers a store instruction touches 16 or 32 rows with 32 or 16 bytes each,
// and 4096 x 8192 outputs of a single step of K took 31 us, now 20 (4096 x 8192 x 8192: 149 and 129).
template <int OUT, int MR, int TJ>
constexpr int stage_pitch() { return MR * TJ * (OUT == EP_F32 ? 4 : 2) + 16; }
template <int OUT, int MR, int TI, int TJ>
__device__ __forceinline__ void store_staged(const GemmMxArgs& g, const TileAt& t, int m0, int n0,
                                             const typename Instr<MR>::Acc (&acc)[TI][TJ], uint8_t* lds) {
    constexpr int kEs = OUT == EP_F32 ? 4 : 2, kPitch = stage_pitch<OUT, MR, TJ>(), kPieces = MR * TJ * kEs / 16, kOf = 16 / kEs;
    const int lane = threadIdx.x & 63, cols = g.N - n0;
    float bias[TJ][Instr<MR>::kQuads][4];
    if (g.bias) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int q = 0; q < Instr<MR>::kQuads; ++q) {
                const int c = MR * j + 8 * q + 4 * Instr<MR>::group();
                load_bias(g, t.e, n0 + c, cols - c, bias[j][q]);
            }
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int q = 0; q < Instr<MR>::kQuads; ++q) {
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = g.bias ? acc[i][j][4 * q + c] + bias[j][q][c] : acc[i][j][4 * q + c];
                uint8_t* at = lds + Instr<MR>::row() * kPitch + (MR * j + 8 * q + 4 * Instr<MR>::group()) * kEs;
                store4<OUT>(at, 0, v, 4, true);
            }
        __builtin_amdgcn_wave_barrier();                     // LDS serves a wave's instructions in their order
        const int rows = t.m_end - (m0 + MR * i);
#pragma unroll
        for (int p = 0; p < (MR * kPieces + 63) / 64; ++p) {
            const int at = 64 * p + lane, r = at / kPieces, c = at % kPieces;
            if (r >= MR || r >= rows || kOf * c >= cols) continue;
            const uint8_t* from = lds + r * kPitch + 16 * c;
            uint8_t* to = static_cast<uint8_t*>(g.Y) + ((int64_t)(m0 + MR * i + r) * g.ldy + n0) * kEs + 16 * c;
            if (kOf * (c + 1) <= cols)
                __builtin_memcpy(to, __builtin_assume_aligned(from, 16), 16);
            else
                for (int e = 0; e < cols - kOf * c; ++e) __builtin_memcpy(to + kEs * e, from + kEs * e, kEs);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int BM, int BN>
constexpr int stage_bytes() { return (BM + BN) * 128 + 4 * scale_words<BM>() + 4 * scale_words<BN>(); }

// The tile t. smem: the rings of the K groups, then a spare KiB.
template <int BM, int BN, int MR, int WGM, int WGN, int S, int KS>
__device__ __forceinline__ void tile_product(const GemmMxArgs& g, const TileAt& t, uint8_t* smem) {
    constexpr int NW = WGM * WGN;                            // waves of a K group
    constexpr int TI = BM / WGM / MR, TJ = BN / WGN / MR, SUB = Instr<MR>::kSub, Q = Instr<MR>::kQuads;
    static_assert(TI * WGM * MR == BM && TJ * WGN * MR == BN, "whole parts per wave");
    constexpr int kScalesX = (BM + BN) * 128, kScalesW = kScalesX + 4 * scale_words<BM>();
    constexpr int kStage = stage_bytes<BM, BN>();
    constexpr int kLoads = Dma<BM, NW>::kLoads + Dma<BN, NW>::kLoads + ScaleDma<BM, BN, NW>::kEach;      // per wave and stage
    constexpr int kRing = S * kStage;                        // of a K group
    constexpr int kSums = (KS - 1) * BM * BN * 4;
    static_assert(kSums <= KS * kRing, "the sums of the other K groups reuse the rings");
    uint8_t* spare = smem + KS * kRing;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) % NW);
    const int kg = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / NW);   // K group of the wave
    uint8_t* lds = smem + kg * kRing;
    const int wm = (wave / WGN) * (BM / WGM), wn = (wave % WGN) * (BN / WGN);
    const int ld = g.K / 2, chunks = g.K / 128;              // bytes of a row
    Dma<BM, NW> dx;
    Dma<BN, NW> dw;
    dx.init(g.X, ld, t.m0, t.m_end, wave);
    dw.init(g.W + (int64_t)t.e * g.N * ld, ld, t.n0, g.N, wave);
    dx.chunk = 16 * chunk_of<MR>(dx.chunk / 16);
    dw.chunk = 16 * chunk_of<MR>(dw.chunk / 16);
    const ScaleDma<BM, BN, NW> ds{g.sx + 4 * (int64_t)t.m0, g.sw + 4 * ((int64_t)t.e * chunks * g.N + t.n0), 4 * (int64_t)g.M,
                                  4 * (int64_t)g.N, t.m_end - t.m0, g.N - t.n0};

    typename Instr<MR>::Acc acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = 0.0f;

    const int nk = (ld + 128 * KS - 1) / (128 * KS);
    int step = kg;                                           // of the next loads
    auto load = [&](uint8_t* stage) {                        // past K zeros are written, so no step has a tail
        dx.load(128 * step, ld, stage, spare, wave);
        dw.load(128 * step, ld, stage + BM * 128, spare, wave);
        ds.load(step, chunks, stage + kScalesX, spare, wave);
        step += KS;
    };
#pragma unroll
    for (int p = 0; p < S; ++p) load(lds + p * kStage);
    wait_loads<(S - 1) * kLoads>();                          // this wave's part of the first stage landed
    __syncthreads();
    i32x4 x[2][TI], w[2][TJ];
    int sx[TI], sw[TJ];
    read_frags<MR, TI>(lds, wm, 0, x[0]);
    read_frags<MR, TJ>(lds + BM * 128, wn, 0, w[0]);
    read_scales<MR, BM, TI>(lds + kScalesX, wm, sx);
    read_scales<MR, BN, TJ>(lds + kScalesW, wn, sw);
    uint8_t* cur = lds;
    for (int kt = 0; kt < nk; ++kt) {
        uint8_t* nxt = cur + kStage == lds + kRing ? lds : cur + kStage;
        auto within = [&](auto at) {                         // sub-step s, the fragments of s + 1 read behind its MFMAs
            constexpr int s = decltype(at)::value;
            __builtin_amdgcn_sched_barrier(0);
            read_frags<MR, TI>(cur, wm, s + 1, x[(s + 1) & 1]);
            read_frags<MR, TJ>(cur + BM * 128, wn, s + 1, w[(s + 1) & 1]);
            multiply<MR, s, TI, TJ>(x[s & 1], w[s & 1], sx, sw, acc);
            interleave<TI + TJ, TI * TJ, 0x100>();
        };
        within(std::integral_constant<int, 0>{});
        if constexpr (SUB == 4) {
            within(std::integral_constant<int, 1>{});
            within(std::integral_constant<int, 2>{});
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<(S - 2) * kLoads>();                      // all of this stage read, the next one landed
        __syncthreads();
        load(cur);
        int nsx[TI], nsw[TJ];
        read_frags<MR, TI>(nxt, wm, 0, x[0]);
        read_frags<MR, TJ>(nxt + BM * 128, wn, 0, w[0]);
        read_scales<MR, BM, TI>(nxt + kScalesX, wm, nsx);
        read_scales<MR, BN, TJ>(nxt + kScalesW, wn, nsw);
        multiply<MR, SUB - 1, TI, TJ>(x[1], w[1], sx, sw, acc);
        interleave<kLoads, TI * TJ * 3 / 4, 0x20>();
        interleave<TI + TJ + (TI + 1) / 2 + (TJ + 1) / 2, TI * TJ - TI * TJ * 3 / 4, 0x100>();
#pragma unroll
        for (int i = 0; i < TI; ++i) sx[i] = nsx[i];
#pragma unroll
        for (int j = 0; j < TJ; ++j) sw[j] = nsw[j];
        cur = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                      // no load may still write LDS when the block ends
    if constexpr (KS > 1) {
        static_assert(Q == 1, "small tiles");
        __syncthreads();                                     // every group is done with its ring
        f32x4* sums = reinterpret_cast<f32x4*>(smem) + (wave * TI * TJ) * 64 + (threadIdx.x & 63);
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) sums[((kg - 1) * NW * TI * TJ + i * TJ + j) * 64] = acc[i][j];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int q = 0; q < KS - 1; ++q)
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int j = 0; j < TJ; ++j) acc[i][j] += sums[(q * NW * TI * TJ + i * TJ + j) * 64];
    }

    auto store = [&](auto out) {
        constexpr int OUT = decltype(out)::value, kRegion = MR * stage_pitch<OUT, MR, TJ>();
        if constexpr (KS == 1 && NW * kRegion <= kRing) {
            __syncthreads();                                 // every wave is done with the ring
            store_staged<OUT, MR, TI, TJ>(g, t, t.m0 + wm, t.n0 + wn, acc, smem + wave * kRegion);
        } else {
            store_tile<OUT, MR, TI, TJ>(g, t, t.m0 + wm, t.n0 + wn, acc);
        }
    };
    if (g.out == EP_BF16) store(std::integral_constant<int, EP_BF16>{});
    else if (g.out == EP_F16) store(std::integral_constant<int, EP_F16>{});
    else store(std::integral_constant<int, EP_F32>{});
}

// A tile of 256 rows of which an expert has at most 128 is one of 128 rows with a stage more (4096 tokens, 4 of 64 experts of
// 2048 x 2048, 256 rows each on average: 78.6 us, as full tiles 83.2; 512 rows each of 32 of 2048 x 4096: 103.3 and 103.7).
template <int BM, int BN, int MR, int WGM, int WGN, int S, int KS, bool EXPERTS>
__global__ __launch_bounds__(64 * WGM * WGN * KS) void gemm_mx(GemmMxArgs g) {
    constexpr int kFull = KS * S * stage_bytes<BM, BN>();
    if constexpr (EXPERTS && BM == 256) {
        constexpr int kHalf = 3 * stage_bytes<BM / 2, BN>();
        __shared__ __align__(1024) uint8_t smem[(kFull > kHalf ? kFull : kHalf) + 1024];
        const TileAt t = expert_tile<BM, BN>(g);
        if (!t.any) return;
        if (t.e == g.experts) zero_rows(g, t, BM, BN);
        else if (t.m_end - t.m0 <= BM / 2) tile_product<BM / 2, BN, MR, WGM, WGN, 3, 1>(g, t, smem);
        else tile_product<BM, BN, MR, WGM, WGN, S, KS>(g, t, smem);
    } else if constexpr (EXPERTS) {
        __shared__ __align__(1024) uint8_t smem[kFull + 1024];
        const TileAt t = expert_tile<BM, BN>(g);
        if (!t.any) return;
        if (t.e == g.experts) zero_rows(g, t, BM, BN);
        else tile_product<BM, BN, MR, WGM, WGN, S, KS>(g, t, smem);
    } else {
        __shared__ __align__(1024) uint8_t smem[kFull + 1024];
        tile_product<BM, BN, MR, WGM, WGN, S, KS>(g, block_tile<BM, BN>(g), smem);
    }
}

template <int BM, int BN, int MR, int WGM, int WGN, int S, int KS, bool EXPERTS>
hipError_t tiled_go(const GemmMxArgs& g, hipStream_t stream) {
    int64_t blocks = row_tiles(g, BM) * (((int64_t)g.N + BN - 1) / BN);
    if (EXPERTS) blocks = (blocks + 7) / 8 * 8;                // an eighth of the tiles for each XCD
    if (blocks * (64 * WGM * WGN * KS) > kMaxThreads) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_mx<BM, BN, MR, WGM, WGN, S, KS, EXPERTS>), dim3((unsigned)blocks), dim3(64 * WGM * WGN * KS), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows_mx(const void* X, int src, int64_t rows, int64_t M, int64_t K, int64_t ldx, uint8_t* Q,
                                   uint8_t* S, hipStream_t stream) {
    if (rows <= 0 || K <= 0) return hipSuccess;
    const MxGrid g = mx_grid(rows, M, K);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(g.blocks), dim3(256), 0, stream, X, M, K, ldx, Q, S, g.chunks, g.row_groups, g.units);
        return hipGetLastError();
    };
    switch (src) {
        case EP_F32: return go(quantize_rows_mx<EP_F32>);
        case EP_BF16: return go(quantize_rows_mx<EP_BF16>);
        case EP_F16: return go(quantize_rows_mx<EP_F16>);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_dequantize_rows_mx(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t M, int64_t Kp, int64_t K,
                                     int dst, void* Y, hipStream_t stream) {
    if (rows <= 0 || K <= 0) return hipSuccess;
    const MxGrid g = mx_grid(rows, M, Kp);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(g.blocks), dim3(256), 0, stream, Q, S, M, g.chunks, K, Y, g.row_groups, g.units);
        return hipGetLastError();
    };
    switch (dst) {
        case EP_F32: return go(dequantize_rows_mx<EP_F32>);
        case EP_BF16: return go(dequantize_rows_mx<EP_BF16>);
        case EP_F16: return go(dequantize_rows_mx<EP_F16>);
        default: return hipErrorInvalidValue;
    }
}

// The kernels of kMxTiles. The instruction of 16 rows takes less power than that of 32 (7.2 PFLOP/s of random codes without
// memory, 6.4), which tells in the largest tiles; in 128 x 128 and 64 x 64, where waves have 64 x 32 or 32 x 32 of
// them, the one of 32 rows is ahead by 4 to 10%.
template <int I, int MR, int WGM, int WGN, int S>
constexpr hipError_t (*tile_go())(const GemmMxArgs&, hipStream_t) {
    return tiled_go<kMxTiles[I].bm, kMxTiles[I].bn, MR, WGM, WGN, S, kMxTiles[I].ks, false>;
}
hipError_t (*const kTileGo[])(const GemmMxArgs&, hipStream_t) = {
    tile_go<0, 16, 2, 4, 2>(), tile_go<1, 16, 2, 4, 2>(), tile_go<2, 16, 4, 2, 3>(), tile_go<3, 32, 2, 4, 3>(), tile_go<4, 16, 4, 2, 3>(),
    tile_go<5, 32, 2, 2, 4>(), tile_go<6, 16, 1, 2, 4>(), tile_go<7, 16, 1, 2, 3>(), tile_go<8, 16, 1, 2, 4>(),
};
static_assert(sizeof kTileGo / sizeof *kTileGo == kMxTileCount, "a kernel for each tile");

hipError_t launch_gemm_mx(const GemmMxArgs& g, hipStream_t stream) {
    if (g.M <= 0 || g.N <= 0) return hipSuccess;
    const int64_t cus = device_cus();
    if (!g.experts) return kTileGo[mx_tile(g.M, g.N, g.K, cus)](g, stream);
    // Experts: how many rows each has is known to the device only, so the tile goes by the average. Measured with rows
    // spread unevenly (a factor of e^0.5 as standard deviation), weights that come from HBM, in us: 2 rows each on 16 x 64 23.2 (32
    // experts of 4096 x 2048; 64 x 128: 24.1) and 12.1 at 1 row each of 64 of 1024 x 2048 (64 x 128: 14.2); 8 rows on 64 x 128 28.8 (16 x 64:
    // 30.8) and 81.6 (128 of 2816 x 2048; 16 x 64: 88.4); 24 rows on 128 x 128, two blocks to a CU, 33.3 and 17.2 (64 of 1024 x 2048; 64 x 128:
    // 36.2 and 21.3); 64 rows on 64 x 128 40.0 and 34.1 (32 of 2048 x 4096; 128 x 128, where the larger experts begin a second
    // row tile: 45.7 and over 40); 100 rows on 128 x 128 43.3 and 121 (128 of 2816 x 2048; 64 x 128: 50.6, 256 x 256: 136). Above that
    // whichever of 256 x 256 and 256 x 192 fills its rounds better: 200 rows 62 and 56 (128 x 128: 66 and 63), 400 rows of 8 of
    // 8192 x 4096 on 256 x 192 86 (256 x 256: 99), 800 rows of 128 of 2816 x 2048 on 256 x 256 505 (256 x 192: 545).
    const int64_t used = g.M < g.experts ? g.M : g.experts, rows = mx_over(g.M, used);
    if (rows > 150) {
        // a partly filled tile per expert: half a tile on average
        const int64_t tiles = (2 * g.M + 256 * used) / 512;
        return mx_cost(kMxTiles[1], tiles, g.N, g.K, cus) < mx_cost(kMxTiles[0], tiles, g.N, g.K, cus)
                   ? tiled_go<256, 192, 16, 2, 4, 2, 1, true>(g, stream)
                   : tiled_go<256, 256, 16, 2, 4, 2, 1, true>(g, stream);
    }
    if (rows <= 2) return tiled_go<16, 64, 16, 1, 4, 4, 1, true>(g, stream);
    if (rows <= 20 || (rows > 40 && rows <= 64)) return tiled_go<64, 128, 32, 2, 4, 3, 1, true>(g, stream);
    return tiled_go<128, 128, 32, 2, 4, 2, 1, true>(g, stream);
}

}  // namespace ep
