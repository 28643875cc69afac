// gfx950 INT8 row quantizer and INT8 matrix products: Y[m][n] = sx[m] sw[n] sum_k X[m][k] W[n][k]
// (+ bias[n]), int32 sums on the matrix cores (v_mfma_i32_16x16x64_i8), fp32 epilogue. The weight is
// the INT8 container of the decoder (codes and one scale per output channel), the activations carry
// one scale per row, so both scales leave the sum and the sum itself is exact: any split or order
// of K gives the same bits.
//
// Operand lane layout (v_mfma_i32_16x16x64_i8, checked on the device): lane l supplies 16 codes of
// A row l % 16 and of B column l % 16, K group l / 16, and receives C[4 (l / 16) + i][l % 16],
// i < 4. A and B take the same 16 K positions per lane, so equal k meet whatever the order. W is
// the A operand and X the B operand: a lane then holds four consecutive output columns of one row.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "entropack.h"
#include "int8.h"
#include "kernels.h"

namespace ep {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;   // of a grid
constexpr uint32_t kOob = 0x80000000u;      // an offset past every resource: the load returns 0

__device__ __forceinline__ uint16_t to_bf16(float v) {
    return (uint16_t)(__builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, 0.0f}, bf16x2)) & 0xFFFFu);
}
__device__ __forceinline__ uint16_t to_f16(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// ------------------------------------------------------------------------------- row quantizer
// a = max |x| over the row (raised to 2^-100 when smaller, unless zero), scale = a / 127 (fp32),
// code = 127 x / a rounded to nearest, ties to even, decided exactly. A zero row gets scale 0 and
// codes 0; a row with an infinity or a NaN gets scale NaN and codes 0, so that every product with
// it is NaN instead of a plausible number.
//
// The quotient is formed as x (127 / a), off by at most 1.5e-5 at 127 (two roundings); where it
// falls within 5e-5 of a rounding border f + 1/2 the code is decided by comparing 254 |x| with
// (2 f + 1) a in fp64, where both products are exact (at most 32 bits).
//
// One row per block of 256 threads or, for short rows, per wave; the row stays in registers between
// the maximum and the codes (CH chunks of 8 elements per thread; CH = 0 reads it twice), so it is
// read once from memory. Memory bound: 4096 x 10240 BF16 in 26-29 us, 126 MB at 4.3-4.8 TB/s (a 1 GiB copy
// reaches 5.2).
constexpr float kMagic = 12582912.0f;       // 1.5 * 2^23: v + kMagic holds rne(v) in its low mantissa bits

template <int SRC> struct Elem { typedef uint16_t type; };
template <> struct Elem<EP_F32> { typedef uint32_t type; };

template <int SRC>
__device__ __forceinline__ float elem_value(uint32_t bits) {
    if constexpr (SRC == EP_F32) return __uint_as_float(bits);
    if constexpr (SRC == EP_BF16) return __uint_as_float(bits << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}
template <int SRC> __device__ __forceinline__ uint32_t abs_bits(uint32_t b) { return b & (SRC == EP_F32 ? 0x7FFFFFFFu : 0x7FFFu); }
template <int SRC> constexpr uint32_t inf_bits() { return SRC == EP_F32 ? 0x7F800000u : SRC == EP_BF16 ? 0x7F80u : 0x7C00u; }

// Eight consecutive elements, loaded at any alignment of the element; the last chunk of a row that is no
// multiple of eight long starts eight before its end and gives some codes twice (the same ones), so no
// row needs a tail of single elements (4096 x 10241 BF16 element by element: 62 us). V = 1: rows shorter
// than eight.
template <int SRC, int V>
struct Chunk {
    typename Elem<SRC>::type e[V];
};
template <int SRC, int V>
__device__ __forceinline__ Chunk<SRC, V> load_chunk(const typename Elem<SRC>::type* x) {
    Chunk<SRC, V> c;
    __builtin_memcpy(&c, x, sizeof c);
    return c;
}

template <int SRC, int V>
__device__ __forceinline__ uint32_t chunk_max(const Chunk<SRC, V>& c, uint32_t a) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t b = abs_bits<SRC>(c.e[i]);
        a = a > b ? a : b;
    }
    return a;
}

// The codes of a chunk, one byte each (low byte first).
template <int SRC, int V>
__device__ __forceinline__ void chunk_codes(const Chunk<SRC, V>& c, float inv, float amax, uint32_t* out) {
    uint32_t m[V];
    bool close = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float t = elem_value<SRC>(c.e[i]) * inv;
        const float r = t + kMagic;
        m[i] = __float_as_uint(r);
        close |= fabsf(t - (r - kMagic)) > 0.49995f;
    }
    if (close) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // floor f of the magnitude, then 127 |x| / a against the border f + 1/2: both products exact
            const float x = elem_value<SRC>(c.e[i]), f = floorf(fabsf(x * inv));
            if (fabsf(fabsf(x * inv) - f - 0.5f) > 5e-5f) continue;
            const double l = 254.0 * (double)fabsf(x), r = (double)(2.0f * f + 1.0f) * (double)amax;
            const int n = (int)f, q = l > r || (l == r && (n & 1)) ? n + 1 : n;
            m[i] = (uint32_t)(x < 0.0f ? -q : q);
        }
    }
#pragma unroll
    for (int i = 0; i < (V + 3) / 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4 && 4 * i + j < V; ++j) w |= (m[4 * i + j] & 0xFFu) << (8 * j);
        out[i] = w;
    }
}

// TPR threads per row (64 or 256), V elements per chunk (8 or 1), CH chunks per thread held in registers.
template <int SRC, int TPR, int V, int CH>
__global__ __launch_bounds__(256) void quantize_rows_i8(const void* Xv, int M, int K, int64_t ldx, int8_t* Q, float* S) {
    typedef typename Elem<SRC>::type T;
    __shared__ uint32_t wmax[4];
    const int t = threadIdx.x % TPR;
    // m is uniform in the block for TPR 256 (block barriers below), in the wave for TPR 64; a grid may
    // have at most 2^32 - 1 threads, so the blocks stride over the rows
    for (int64_t m = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR; m < M; m += (int64_t)gridDim.x * (256 / TPR)) {
        const T* x = static_cast<const T*>(Xv) + m * ldx;
        int8_t* q = Q + m * K;
        constexpr int R = CH > 0 ? CH : 1;
        Chunk<SRC, V> v[R];
        uint32_t a = 0;
        auto start = [K](auto k) { return k < K - V ? k : (decltype(k))(K - V); };
        if constexpr (CH > 0) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = V * (t + TPR * c);
                if (k < K) v[c] = load_chunk<SRC, V>(x + start(k));
                else
#pragma unroll
                    for (int i = 0; i < V; ++i) v[c].e[i] = 0;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) a = chunk_max<SRC, V>(v[c], a);
        } else {
            for (int64_t k = V * t; k < K; k += V * TPR) a = chunk_max<SRC, V>(load_chunk<SRC, V>(x + start(k)), a);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint32_t b = (uint32_t)__shfl_xor((int)a, o);
            a = a > b ? a : b;
        }
        if constexpr (TPR == 256) {
            if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = a;
            __syncthreads();
            a = wmax[0];
#pragma unroll
            for (int i = 1; i < 4; ++i) a = a > wmax[i] ? a : wmax[i];
            __syncthreads();                                       // wmax is free for the next row
        }
        float amax = elem_value<SRC>(a);
        const bool bad = a >= inf_bits<SRC>();
        if (a == 0 || bad) {
            if (t == 0) S[m] = bad ? __builtin_nanf("") : 0.0f;
            // in the codes' own pieces: a row may have 2^31 - 1 codes, and padding tokens are rows of zeros
            auto clear = [&](auto k) { __builtin_memset(q + start(k), 0, V); };
            if constexpr (CH > 0) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int k = V * (t + TPR * c);
                    if (k < K) clear(k);
                }
            } else {
                for (int64_t k = V * t; k < K; k += V * TPR) clear(k);
            }
            continue;
        }
        amax = fmaxf(amax, 0x1p-100f);
        if (t == 0) S[m] = amax / 127.0f;
        const float inv = 127.0f / amax;
        auto store = [&](auto k, const Chunk<SRC, V>& c) {
            uint32_t o[(V + 3) / 4];
            chunk_codes<SRC, V>(c, inv, amax, o);
            __builtin_memcpy(q + start(k), o, V);
        };
        if constexpr (CH > 0) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = V * (t + TPR * c);
                if (k < K) store(k, v[c]);
            }
        } else {
            for (int64_t k = V * t; k < K; k += V * TPR) store(k, load_chunk<SRC, V>(x + start(k)));
        }
    }
}

template <int SRC, int TPR, int V, int CH>
hipError_t quantize_go(const void* X, int M, int K, int64_t ldx, int8_t* Q, float* S, hipStream_t stream) {
    const int64_t groups = ((int64_t)M + 256 / TPR - 1) / (256 / TPR);
    const unsigned blocks = (unsigned)(groups < (1 << 20) ? groups : 1 << 20);
    hipLaunchKernelGGL((quantize_rows_i8<SRC, TPR, V, CH>), dim3(blocks), dim3(256), 0, stream, X, M, K, ldx, Q, S);
    return hipGetLastError();
}

template <int SRC>
hipError_t quantize_src(const void* X, int M, int K, int64_t ldx, int8_t* Q, float* S, hipStream_t stream) {
    if (K < 8) return quantize_go<SRC, 64, 1, 1>(X, M, K, ldx, Q, S, stream);
    if (K <= 512) return quantize_go<SRC, 64, 8, 1>(X, M, K, ldx, Q, S, stream);
    if (K <= 1024) return quantize_go<SRC, 64, 8, 2>(X, M, K, ldx, Q, S, stream);
    if (K <= 2048) return quantize_go<SRC, 256, 8, 1>(X, M, K, ldx, Q, S, stream);
    if (K <= 4096) return quantize_go<SRC, 256, 8, 2>(X, M, K, ldx, Q, S, stream);
    if (K <= 8192) return quantize_go<SRC, 256, 8, 4>(X, M, K, ldx, Q, S, stream);
    if (K <= 16384) return quantize_go<SRC, 256, 8, 8>(X, M, K, ldx, Q, S, stream);
    return quantize_go<SRC, 256, 8, 0>(X, M, K, ldx, Q, S, stream);
}

// ------------------------------------------------------------------------------- rows to 16 bytes
// Codes whose rows are not 16-byte aligned (K % 16, or a base address inside a row) are copied once
// to rows of ld >= K codes with zeros behind; the zeros add nothing to the sums. The piece that a row ends
// in is read like the others where the next row's codes lie behind it, and masked; only the last row's is
// read byte by byte.
__global__ __launch_bounds__(256) void pad_rows_i8(const int8_t* src, int64_t rows, int K, int8_t* dst, int ld) {
    const int cpr = ld / 16;
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= rows * cpr) return;
    const int64_t r = c / cpr;
    const int k0 = 16 * (int)(c % cpr);
    const uint8_t* s = reinterpret_cast<const uint8_t*>(src) + r * (int64_t)K + k0;
    uint32_t w[4] = {0, 0, 0, 0};
    const int left = K - k0;                                   // codes of the row from here on
    if (left > 0 && r * (int64_t)K + k0 + 16 <= rows * (int64_t)K) {
        __builtin_memcpy(w, s, 16);                            // one load of any alignment
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = left - 4 * i;                        // valid bytes of this word
            w[i] = n >= 4 ? w[i] : n > 0 ? w[i] & ((1u << (8 * n)) - 1) : 0;
        }
    } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) w[i / 4] |= (uint32_t)s[i] << (8 * (i % 4));
    }
    *reinterpret_cast<uint4*>(dst + r * (int64_t)ld + k0) = make_uint4(w[0], w[1], w[2], w[3]);
}

struct BiasList {
    const uint16_t* p[32];
};
__global__ __launch_bounds__(256) void gather_bias(BiasList b, int N, uint16_t* dst) {
    const uint16_t* src = b.p[blockIdx.y];
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < N; n += (int64_t)gridDim.x * 256)
        dst[(int64_t)blockIdx.y * N + n] = src ? src[n] : 0x8000u;
}

// ------------------------------------------------------------------------------- tile of a block
// The output tile of a block: rows [m0, m0 + BM) up to m_end, columns [n0, n0 + BN), of expert e
// (0 without experts). e == experts stands for the rows behind the last expert's, which are zeroed;
// `any` is false for a block without a tile (the grid holds the largest tile count that the row
// count allows, since the split over the experts is known to the device only).
struct TileAt {
    int m0, m_end, n0, e;
    bool any;
};

// Rows of expert e (e == experts: the rows behind), clamped to [0, M] so that no offset can lead
// out of the buffers.
__device__ __forceinline__ void expert_rows(const GemmI8Args& g, int e, int* a, int* b) {
    const int lo = g.offsets[e], hi = e < g.experts ? g.offsets[e + 1] : g.M;
    *a = lo < 0 ? 0 : lo < g.M ? lo : g.M;
    *b = hi < *a ? *a : hi < g.M ? hi : g.M;
}

// The row tiles of 64 experts from e0 on, one expert per lane: its rows [a, b), its tile count and the
// sum of the counts of the lanes up to it. Returns the 64 experts' total.
template <int BM>
__device__ __forceinline__ int expert_counts(const GemmI8Args& g, int e0, int* a, int* b, int* cnt, int* upto) {
    const int lane = threadIdx.x & 63;
    *a = *b = 0;
    if (e0 + lane <= g.experts) expert_rows(g, e0 + lane, a, b);
    *cnt = (*b - *a + BM - 1) / BM;
    int sum = *cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(sum, o);
        if (lane >= o) sum += v;
    }
    *upto = sum;
    return __builtin_amdgcn_readlane(sum, 63);
}

// Every wave looks its tile up on its own. Tiles are numbered expert by expert, within an expert in groups
// of 8 row tiles that walk the column tiles together. Consecutive block ids land on different XCDs, so
// each XCD takes a contiguous eighth of the numbers: the rows and the weight of a group then meet in
// one L2. Against tiles dealt out round robin, column tiles innermost (same weights every call): 4096 tokens
// on 4 of 32 experts (2048 x 4096) 183 us for 261, 1024 tokens 73 for 80, 8 of 128 (1408 x 2048) 175 for 178, 2 of
// 8 (8192 x 4096) 307 for 373, with groups of one row tile 355; 16 tokens (4096 x 2048) 30.7 for 31.4.
template <int BM, int BN>
__device__ __forceinline__ TileAt expert_tile(const GemmI8Args& g) {
    constexpr int G = 8;
    const int tiles_n = (g.N + BN - 1) / BN;
    int a, b, cnt, upto;
    int total = expert_counts<BM>(g, 0, &a, &b, &cnt, &upto);
    for (int e0 = 64; e0 <= g.experts; e0 += 64) {
        int a2, b2, c2, u2;
        total += expert_counts<BM>(g, e0, &a2, &b2, &c2, &u2);
    }
    const int64_t all = (int64_t)total * tiles_n;
    const int64_t each = (all + 7) / 8, at = (int64_t)blockIdx.x / 8;
    const int64_t number = (int64_t)(blockIdx.x % 8) * each + at;
    TileAt t{0, 0, 0, 0, false};
    if (at >= each || number >= all) return t;
    int before = 0;
    for (int e0 = 0; e0 <= g.experts; e0 += 64) {
        if (e0 > 0) {
            before += __builtin_amdgcn_readlane(upto, 63);
            expert_counts<BM>(g, e0, &a, &b, &cnt, &upto);
        }
        const int64_t mine = (int64_t)(before + upto - cnt) * tiles_n;     // tiles before this lane's expert
        const uint64_t hit = __ballot(number >= mine && number < mine + (int64_t)cnt * tiles_n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int in = (int)(number - __shfl(mine, l)), tms = __shfl(cnt, l);
            const int per = G * tiles_n, first = in / per * G, size = tms - first < G ? tms - first : G;
            const int tm = first + (in % per) % size, tn = (in % per) / size;
            t.e = __builtin_amdgcn_readfirstlane(e0 + l);
            t.m0 = __builtin_amdgcn_readfirstlane(__shfl(a, l) + BM * tm);
            t.n0 = __builtin_amdgcn_readfirstlane(BN * tn);
            t.m_end = __builtin_amdgcn_readfirstlane(__shfl(b, l));
            t.any = true;
            return t;
        }
    }
    return t;
}

// The output of four sums of one row (columns n .. n + count - 1 of a lane), scaled, biased, rounded once
// and stored; `vec` when rows of Y are aligned to four elements.
template <int OUT>
__device__ __forceinline__ void store4(void* Y, int64_t at, i32x4 acc, const float* sw, float sx, const float* bias, int count,
                                       bool vec) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = (float)acc[i] * sw[i] * sx;
        if (bias) v[i] += bias[i];
    }
    if constexpr (OUT == EP_F32) {
        float* y = static_cast<float*>(Y) + at;
        if (vec && count == 4) *reinterpret_cast<f32x4*>(y) = f32x4{v[0], v[1], v[2], v[3]};
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) y[i] = v[i];
    } else {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = OUT == EP_BF16 ? to_bf16(v[i]) : to_f16(v[i]);
        uint16_t* y = static_cast<uint16_t*>(Y) + at;
        if (vec && count == 4)
            *reinterpret_cast<uint2*>(y) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) y[i] = h[i];
    }
}

// Scales and biases of a lane's four columns from n on (count of them inside the matrix).
__device__ __forceinline__ void load_columns(const GemmI8Args& g, int e, int n, int count, float* sw, float* bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = (int64_t)e * g.N + n + i;
        sw[i] = i < count ? g.sw[c] : 0.0f;
        if (g.bias) bias[i] = i < count ? __uint_as_float((uint32_t)g.bias[c] << 16) : 0.0f;
    }
}

// The epilogue of a wave's TI x TJ parts of 16 x 16: rows m0 + 16 i + lane % 16, columns n0 + 16 j + 4 (lane / 16).
template <int OUT, int TI, int TJ>
__device__ __forceinline__ void store_tile(const GemmI8Args& g, const TileAt& t, int m0, int n0, const i32x4 (&acc)[TI][TJ],
                                           bool vec) {
    const int lane = threadIdx.x & 63;
    float sx[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int m = m0 + 16 * i + (lane & 15);
        sx[i] = m < t.m_end ? g.sx[m] : 0.0f;
    }
    float sw[TJ][4], bias[TJ][4];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
        const int n = n0 + 16 * j + 4 * (lane >> 4);
        load_columns(g, t.e, n, g.N - n < 4 ? g.N - n : 4, sw[j], bias[j]);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int m = m0 + 16 * i + (lane & 15);
        if (m >= t.m_end) continue;
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int n = n0 + 16 * j + 4 * (lane >> 4);
            if (n >= g.N) continue;
            store4<OUT>(g.Y, (int64_t)m * g.ldy + n, acc[i][j], sw[j], sx[i], g.bias ? bias[j] : nullptr,
                        g.N - n < 4 ? g.N - n : 4, vec);
        }
    }
}

__device__ __forceinline__ void zero_rows(const GemmI8Args& g, const TileAt& t, int bm, int bn) {
    const int rows = t.m_end - t.m0 < bm ? t.m_end - t.m0 : bm, cols = g.N - t.n0 < bn ? g.N - t.n0 : bn;
    for (int i = threadIdx.x; i < rows * cols; i += blockDim.x) {
        const int64_t at = (int64_t)(t.m0 + i / cols) * g.ldy + t.n0 + i % cols;
        if (g.out == EP_F32) static_cast<float*>(g.Y)[at] = 0.0f;
        else static_cast<uint16_t*>(g.Y)[at] = 0;
    }
}

__device__ __forceinline__ bool vec_out(const GemmI8Args& g) {
    return g.ldy % 4 == 0 && !(reinterpret_cast<uintptr_t>(g.Y) & (g.out == EP_F32 ? 15 : 7));
}

// Rows [r0, r0 + ROWS) up to r_end of a row-major code matrix as a buffer resource: rows past r_end
// read as zero.
template <int ROWS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* src, int ld, int64_t r0, int64_t r_end) {
    const int64_t left = r_end - r0;
    const int n = (int)(left < ROWS ? left : ROWS);
    const int bytes = __builtin_amdgcn_readfirstlane((n > 0 ? n : 0) * ld);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(src + r0 * ld), 0, bytes, 0x00020000);
}

// ------------------------------------------------------------------------------- tiled product
// A block of WGM x WGN waves owns a BM x BN tile of Y and walks K in steps of 128 codes. Both operand
// tiles go straight from global memory into LDS (buffer_load ... lds, 16 bytes per lane, 8 rows of
// 128 bytes per instruction), in a ring of S stages. The eight 16-byte chunks of a row are swizzled: chunk c of
// row r sits at slot c ^ ((r / 2) % 8), so that the 16 lanes of a fragment read (16 consecutive rows,
// one chunk) cover all banks.
//
// A step has two halves of 64 codes with a fragment set each. While the MFMAs of one half run, the
// wave reads the other set: the second half's behind the first half's MFMAs, the next step's first
// half behind the second half's. So no MFMA waits for LDS, and the one barrier of a step sits between
// the halves: by then every wave has read all of this stage (it may be overwritten: the loads of step
// k + S start there) and the loads of step k + 1, in flight for S - 1 steps, have landed.
//
// At 4096 x 8192 x 8192 (256 x 256 tiles) 204-218 us, 2.5-2.7 POP/s: the MFMAs are busy 73% of the cycles,
// at the 1.7 GHz that the card holds under this load; no LDS bank conflicts. With the fragments read just
// before their MFMAs, in the compiler's order, it took 260 us (2.1 POP/s). Smaller tiles wait for the loads:
// without the MFMAs 512 x 3840 x 10240 takes as long (28 us), though at well under half of what a CU's cache can
// deliver: 128 x 64 tiles load 24 KiB per step of 0.47 us, 85% of it from L2. What counts is the loads' latency,
// with S - 1 steps in flight. Slower: a ring of 64-code
// stages with twice the bytes in flight (half lines: 252 for 226 us), 4 waves of 128 x 128 (237), raised wave
// priority around the MFMAs (228 for 202). Walking the tiles in one persistent block per CU, the next tile's
// loads ahead of the stores, gained 2-3% on several rounds of tiles and lost 1-3% on one.
//
// KS groups of WGM x WGN waves work on one tile, each on its own 128 codes of a step of 128 KS: more
// waves hide the latency of small tiles, without a workspace. Their int32 sums are added through LDS.
__device__ __forceinline__ int chunk_swizzle(int r) { return (r >> 1) & 7; }

// One operand tile of ROWS rows: the lane's byte offset in its first row group, and the loads of step k0.
// The row groups of a wave are 8 NW rows apart, so the swizzle (period 16 rows) is that of the first one.
// Every wave issues the same number of loads, which the waits count: a wave without a row group of its
// own loads zeros (an offset past the resource) into the spare KiB behind the ring.
template <int ROWS, int NW>
struct Dma {
    static constexpr int kLoads = (ROWS / 8 + NW - 1) / NW;
    __amdgpu_buffer_rsrc_t rs;
    uint32_t row_off;           // of the wave's first row group
    int chunk;                  // K chunk that the lane's slot holds
    uint32_t group_step;        // bytes between the wave's row groups
    __device__ __forceinline__ void init(const int8_t* src, int ld, int64_t r0, int64_t r_end, int wave) {
        const int lane = threadIdx.x & 63;
        const int r = 8 * wave + (lane >> 3);
        rs = rows_rsrc<ROWS>(src, ld, r0, r_end);
        row_off = (uint32_t)(r * ld);
        chunk = 16 * ((lane & 7) ^ chunk_swizzle(r));
        group_step = (uint32_t)(8 * NW * ld);
    }
    __device__ __forceinline__ void load(int k0, int K, uint8_t* lds, uint8_t* spare, int wave) const {
        static_assert(NW % 2 == 0 && (ROWS / 8 % NW == 0 || ROWS / 8 < NW), "whole row groups, a swizzle of two of them");
        const int k = k0 + chunk;
        const uint32_t at = row_off + ((uint32_t)k | ((uint32_t)((K - 1 - k) >> 31) & kOob));   // past K reads zero
        if constexpr (ROWS / 8 < NW) {
            const bool mine = wave < ROWS / 8;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(mine ? lds + 1024 * wave : spare), 16, mine ? at : kOob, 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + 1024 * (wave + NW * j)), 16, at + j * group_step, 0, 0, 0);
        }
    }
};

// Fragments of T 16-row parts from row r0 of an operand tile, K half h (64 codes) of a stage.
template <int T>
__device__ __forceinline__ void read_frags(const uint8_t* tile, int r0, int h, i32x4 (&f)[T]) {
    const int lane = threadIdx.x & 63, r = r0 + (lane & 15);
    const uint8_t* p = tile + r * 128 + (((4 * h + (lane >> 4)) ^ chunk_swizzle(r)) << 4);
#pragma unroll
    for (int i = 0; i < T; ++i) f[i] = *reinterpret_cast<const i32x4*>(p + 16 * 128 * i);
}

template <int TI, int TJ>
__device__ __forceinline__ void multiply(const i32x4 (&x)[TI], const i32x4 (&w)[TJ], i32x4 (&acc)[TI][TJ]) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
}

// Scheduling order of a half step: `many` memory instructions of the kind `mask` (0x100 LDS reads, 0x20
// global loads) spread evenly over `mfmas` MFMAs.
template <int MANY, int MFMAS, int MASK, int I = 0>
__device__ __forceinline__ void interleave() {
    if constexpr (I < MANY) {
        __builtin_amdgcn_sched_group_barrier(MASK, 1, 0);
        constexpr int n = MFMAS * (I + 1) / MANY - MFMAS * I / MANY;
        if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x8, n, 0);
        interleave<MANY, MFMAS, MASK, I + 1>();
    }
}

// s_waitcnt vmcnt(n) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}

template <int BM, int BN, int WGM, int WGN, int S, int KS, bool EXPERTS>
__global__ __launch_bounds__(64 * WGM * WGN * KS) void gemm_i8(GemmI8Args g) {
    constexpr int NW = WGM * WGN;                            // waves of a K group
    constexpr int TI = BM / WGM / 16, TJ = BN / WGN / 16;
    constexpr int kStage = (BM + BN) * 128;
    constexpr int kLoads = Dma<BM, NW>::kLoads + Dma<BN, NW>::kLoads;       // per wave and stage
    constexpr bool kSpare = BM / 8 < NW || BN / 8 < NW;
    constexpr int kRing = S * kStage;                        // of a K group
    constexpr int kSums = (KS - 1) * BM * BN * 4;
    static_assert(kSums <= KS * kRing, "the sums of the other K groups reuse the rings");
    __shared__ __align__(1024) uint8_t smem[KS * kRing + (kSpare ? 1024 : 0)];
    uint8_t* spare = smem + KS * kRing;
    TileAt t;
    if constexpr (EXPERTS) {
        t = expert_tile<BM, BN>(g);
        if (!t.any) return;
        if (t.e == g.experts) {
            zero_rows(g, t, BM, BN);
            return;
        }
    } else {
        const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN, nblk = tiles_m * tiles_n;
        // each XCD a contiguous range of the tiles, so that a column's row tiles meet in one L2 (333 x 5003 x 3968,
        // 237 tiles, same weights every call: 16.1 us, dealt out round robin 16.9; 200 x 4100 x 8192: 20.0 and 22.4)
        const int xcd = blockIdx.x % 8, rest = nblk % 8;
        const int b = xcd * (nblk / 8) + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
        constexpr int G = 4;
        const int per_group = G * tiles_n, first_m = (b / per_group) * G;
        const int gsize = tiles_m - first_m < G ? tiles_m - first_m : G;
        t.m0 = __builtin_amdgcn_readfirstlane((first_m + (b % per_group) % gsize) * BM);
        t.n0 = __builtin_amdgcn_readfirstlane(((b % per_group) / gsize) * BN);
        t.m_end = g.M;
        t.e = 0;
    }
    const int wave = (threadIdx.x >> 6) % NW;
    const int kg = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / NW);   // K group of the wave
    uint8_t* lds = smem + kg * kRing;
    const int wm = (wave / WGN) * (BM / WGM), wn = (wave % WGN) * (BN / WGN);
    Dma<BM, NW> dx;
    Dma<BN, NW> dw;
    dx.init(g.X, g.ldx, t.m0, t.m_end, wave);
    dw.init(g.W + (int64_t)t.e * g.N * g.ldw, g.ldw, t.n0, g.N, wave);

    i32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    const int nk = (g.K + 128 * KS - 1) / (128 * KS);
    int k0 = 128 * kg;                                       // of the next loads
#pragma unroll
    for (int p = 0; p < S; ++p) {                            // loads past K write zeros, so no step has a tail
        dx.load(k0, g.K, lds + p * kStage, spare, wave);
        dw.load(k0, g.K, lds + p * kStage + BM * 128, spare, wave);
        k0 += 128 * KS;
    }
    wait_loads<(S - 1) * kLoads>();                          // this wave's part of the first stage landed
    __syncthreads();
    i32x4 x0[TI], w0[TJ], x1[TI], w1[TJ];
    read_frags<TI>(lds, wm, 0, x0);
    read_frags<TJ>(lds + BM * 128, wn, 0, w0);
    uint8_t* cur = lds;
    for (int kt = 0; kt < nk; ++kt) {
        uint8_t* nxt = cur + kStage == lds + kRing ? lds : cur + kStage;
        __builtin_amdgcn_sched_barrier(0);
        read_frags<TI>(cur, wm, 1, x1);
        read_frags<TJ>(cur + BM * 128, wn, 1, w1);
        multiply<TI, TJ>(x0, w0, acc);
        interleave<TI + TJ, TI * TJ, 0x100>();
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<(S - 2) * kLoads>();                      // all of this stage read, the next one landed
        __syncthreads();
        dx.load(k0, g.K, cur, spare, wave);
        dw.load(k0, g.K, cur + BM * 128, spare, wave);
        k0 += 128 * KS;
        read_frags<TI>(nxt, wm, 0, x0);
        read_frags<TJ>(nxt + BM * 128, wn, 0, w0);
        multiply<TI, TJ>(x1, w1, acc);
        interleave<kLoads, TI * TJ * 3 / 4, 0x20>();         // spread widely: 1% over half and half, 4% over reads first
        interleave<TI + TJ, TI * TJ / 4, 0x100>();
        cur = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                      // no load may still write LDS when the block ends
    if constexpr (KS > 1) {
        __syncthreads();                                     // every group is done with its ring
        i32x4* sums = reinterpret_cast<i32x4*>(smem) + (wave * TI * TJ) * 64 + (threadIdx.x & 63);
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

    const bool vec = vec_out(g);
    if (g.out == EP_BF16) store_tile<EP_BF16, TI, TJ>(g, t, t.m0 + wm, t.n0 + wn, acc, vec);
    else if (g.out == EP_F16) store_tile<EP_F16, TI, TJ>(g, t, t.m0 + wm, t.n0 + wn, acc, vec);
    else store_tile<EP_F32, TI, TJ>(g, t, t.m0 + wm, t.n0 + wn, acc, vec);
}

// Tiles of BM rows that the rows split over the experts can need: every range adds at most one partly
// filled tile (the rows behind the last expert's are a range of their own).
int64_t row_tiles(const GemmI8Args& g, int bm) {
    if (!g.experts) return ((int64_t)g.M + bm - 1) / bm;
    const int64_t most = (int64_t)g.rows / bm + g.experts + 1;
    return most < g.rows ? most : g.rows;
}

template <int BM, int BN, int WGM, int WGN, int S, int KS>
hipError_t tiled_go(const GemmI8Args& g, hipStream_t stream) {
    int64_t blocks = row_tiles(g, BM) * (((int64_t)g.N + BN - 1) / BN);
    if (g.experts) blocks = (blocks + 7) / 8 * 8;              // an eighth of the tiles for each XCD
    if (blocks * (64 * WGM * WGN * KS) > kMaxThreads) return hipErrorInvalidValue;
    if (g.experts)
        hipLaunchKernelGGL((gemm_i8<BM, BN, WGM, WGN, S, KS, true>), dim3((unsigned)blocks), dim3(64 * WGM * WGN * KS), 0, stream, g);
    else
        hipLaunchKernelGGL((gemm_i8<BM, BN, WGM, WGN, S, KS, false>), dim3((unsigned)blocks), dim3(64 * WGM * WGN * KS), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows_i8(const void* X, int src, int M, int K, int64_t ldx, int8_t* Q, float* S,
                                   hipStream_t stream) {
    if (M <= 0) return hipSuccess;
    switch (src) {
        case EP_F32: return quantize_src<EP_F32>(X, M, K, ldx, Q, S, stream);
        case EP_BF16: return quantize_src<EP_BF16>(X, M, K, ldx, Q, S, stream);
        case EP_F16: return quantize_src<EP_F16>(X, M, K, ldx, Q, S, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_gather_bias(const uint16_t* const* bias, int count, int N, uint16_t* dst, hipStream_t stream) {
    if (count < 1 || count > 32) return hipErrorInvalidValue;
    BiasList b{};
    for (int i = 0; i < count; ++i) b.p[i] = bias[i];
    const int64_t blocks = ((int64_t)N + 255) / 256;
    hipLaunchKernelGGL(gather_bias, dim3((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)count), dim3(256), 0, stream, b, N, dst);
    return hipGetLastError();
}

hipError_t launch_pad_rows_i8(const int8_t* src, int64_t rows, int K, int8_t* dst, int ld, hipStream_t stream) {
    const int64_t chunks = rows * (ld / 16);
    if (chunks <= 0) return hipSuccess;
    if (chunks > kMaxThreads - 256) return hipErrorInvalidValue;
    hipLaunchKernelGGL(pad_rows_i8, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, stream, src, rows, K, dst, ld);
    return hipGetLastError();
}

// Tile of a product with one weight. A step of 128 K columns takes a block about the time below, whatever
// M, N and K (measured with one block per CU and weights that come from HBM; small tiles are bound by the
// latency and the rate of the loads, the largest by the MFMAs), so the estimate is rounds of tiles over the
// CUs times steps times that. It picks, e.g., 256 x 256 for 4096 x 8192 x 8192 (215 us; 256 x 128: 245, 128 x 128:
// 321), 256 x 192 for 1024 x 11520 x 3840 (50; 256 x 256: 55, 256 x 128: 67), 128 x 128 for 512 x 8192 x 8192 (44; 256 x
// 128: 55, 128 x 64: 59), 128 x 64 for 333 x 5003 x 3968 (17.6; 64 x 64: 20.8, 128 x 128: 23.7), 64 x 64 for 256 x 4096 x
// 4096 (12.8; 32 x 64: 15.9, 128 x 64: 17.2), 32 x 64 for 64 x 8192 x 8192 (19.6; 64 x 64: 24.0), 16 x 64 for 1 x 11520 x
// 3840 (10.9; 32 x 64: 10.8) and 16 x 32 with two K groups for 1 x 8192 x 8192 (15.2; 16 x 64: 16.4) and 1 x 4096 x
// 16384 (16.4; 16 x 64: 24.7). Waves per block: 128 x 128 in 16 or 8 within 4% of each other either way (1024 x 4096 x
// 4096 25.0 and 24.5, 1024 x 11520 x 3840 68.5 and 69.3), 128 x 64 in 8 (333 x 5003 x 3968 17.6; in 4 17.8) and 64 x 64
// in 8 (256 x 4096 x 4096 12.8; in 4 13.4): more of them hide the barrier and the LDS reads of a step. All of one run.
struct TileCost {
    int bm, bn;
    float step_us;
    hipError_t (*go)(const GemmI8Args&, hipStream_t);
};
const TileCost kTiles[] = {
    {256, 256, 1.65f, tiled_go<256, 256, 2, 4, 2, 1>}, {256, 192, 1.33f, tiled_go<256, 192, 2, 4, 2, 1>},
    {256, 128, 0.97f, tiled_go<256, 128, 4, 2, 3, 1>}, {128, 128, 0.65f, tiled_go<128, 128, 4, 4, 3, 1>},
    {128, 64, 0.47f, tiled_go<128, 64, 4, 2, 4, 1>},   {64, 64, 0.365f, tiled_go<64, 64, 2, 4, 4, 1>},
    {32, 64, 0.305f, tiled_go<32, 64, 1, 4, 5, 1>},    {32, 32, 0.245f, tiled_go<32, 32, 1, 2, 4, 2>},
    {16, 64, 0.28f, tiled_go<16, 64, 1, 4, 6, 1>},     {16, 32, 0.235f, tiled_go<16, 32, 1, 2, 6, 2>},
};
constexpr float kTileUs = 1.5f;             // start and epilogue of a tile

hipError_t launch_gemm_i8(const GemmI8Args& g, hipStream_t stream) {
    if (g.M <= 0 || g.N <= 0 || g.rows <= 0) return hipSuccess;
    if (!g.experts) {
        const TileCost* best = nullptr;
        float least = 0.0f;
        for (const TileCost& t : kTiles) {
            const int64_t tiles = (((int64_t)g.M + t.bm - 1) / t.bm) * (((int64_t)g.N + t.bn - 1) / t.bn);
            const float us = (float)((tiles + device_cus() - 1) / device_cus()) * ((float)((g.K + 127) / 128) * t.step_us + kTileUs);
            if (!best || us < least) best = &t, least = us;
        }
        return best->go(g, stream);
    }
    // Experts: how many rows each has is known to the device only, so the tile goes by the average, several
    // small blocks share a CU where the weights' bytes bound the time, and a tile too large to give
    // every CU one makes way for the next. Measured with the same weights every call, in us, and, behind the
    // slash, with weights that come from HBM: 2 rows each on 16 x 64 tiles 34 / 41 (128 experts, 1408 x 2048; 32 x 64:
    // 35 / 43, 64 x 64: 39 / 48), 8 rows on 32 x 64 40 / 51 (32 experts, 4096 x 2048; 16 x 64: 41 / 49), 32 rows on 128 x
    // 128 44 / 67 (32 experts, 2048 x 4096; in 4 waves instead of 16 46 / 69; 64 x 64: 46 / 62), 128 rows on 128 x 256
    // 75 / 85 (128 x 128: 83 / 90, 128 x 192: 93 / 101), and from 192 rows on 128 x 192, two blocks to a CU, so that one's
    // start and end run behind the other's MFMAs: 375 rows of 16 experts of 4096 x 2048 71 / 87 (128 x 256: 84 / 93,
    // 128 x 128: 81 / 94), 2048 rows of 4 of 2048 x 2048 44 / 45 (128 x 256: 47), 256 rows of 128 of 1408 x 2048 175
    // (128 x 256: 192). 512 rows of 32 of 2048 x 4096: 181 / 185, as 128 x 256 (180 / 185); in the profile of six passes
    // 196, in the one before with 128 x 256 185. 256 x 256 tiles, which no call takes here, took 179 /
    // 181 there, 293 for 306 at 1024 rows of 8 of 8192 x 4096 and 70 / 78 at the 375 rows, but 189 for 175 at the 256.
    const int64_t used = g.rows < g.experts ? g.rows : g.experts, rows = (g.rows + used - 1) / used;
    auto fills = [&](int bm, int bn) { return used * ((rows + bm - 1) / bm) * (((int64_t)g.N + bn - 1) / bn) >= device_cus(); };
    if (rows >= 192 && fills(128, 192)) return tiled_go<128, 192, 2, 4, 2, 1>(g, stream);
    if (rows > 64 && fills(128, 256)) return tiled_go<128, 256, 2, 4, 3, 1>(g, stream);
    if (rows > 16 && fills(128, 128)) return tiled_go<128, 128, 4, 4, 2, 1>(g, stream);
    if (rows > 16 && fills(128, 64)) return tiled_go<128, 64, 4, 2, 3, 1>(g, stream);
    if (rows > 4) return tiled_go<32, 64, 1, 4, 3, 1>(g, stream);
    return tiled_go<16, 64, 1, 4, 3, 1>(g, stream);
}

}  // namespace ep
