// Pieces shared by the tiled matrix products on codes (int8.hip, mxfp4.hip): the tile of a block, with one
// weight or one per expert, operand tiles loaded straight into LDS, and the stores of the outputs. A code
// matrix is rows of bytes here; what a byte holds is the product's own.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "entropack.h"

namespace ep {
namespace {

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
template <typename Args>
__device__ __forceinline__ void expert_rows(const Args& g, int e, int* a, int* b) {
    const int lo = g.offsets[e], hi = e < g.experts ? g.offsets[e + 1] : g.M;
    *a = lo < 0 ? 0 : lo < g.M ? lo : g.M;
    *b = hi < *a ? *a : hi < g.M ? hi : g.M;
}

// The row tiles of 64 experts from e0 on, one expert per lane: its rows [a, b), its tile count and the
// sum of the counts of the lanes up to it. Returns the 64 experts' total.
template <int BM, typename Args>
__device__ __forceinline__ int expert_counts(const Args& g, int e0, int* a, int* b, int* cnt, int* upto) {
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
// one L2. Against tiles dealt out round robin, column tiles innermost (INT8, same weights every call): 4096 tokens
// on 4 of 32 experts (2048 x 4096) 183 us for 261, 1024 tokens 73 for 80, 8 of 128 (1408 x 2048) 175 for 178, 2 of
// 8 (8192 x 4096) 307 for 373, with groups of one row tile 355; 16 tokens (4096 x 2048) 30.7 for 31.4.
template <int BM, int BN, typename Args>
__device__ __forceinline__ TileAt expert_tile(const Args& g) {
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

// The tile of a block where one weight meets all rows.
template <int BM, int BN, typename Args>
__device__ __forceinline__ TileAt block_tile(const Args& g) {
    const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN, nblk = tiles_m * tiles_n;
    // each XCD a contiguous range of the tiles, so that a column's row tiles meet in one L2 (INT8, 333 x 5003 x 3968,
    // 237 tiles, same weights every call: 16.1 us, dealt out round robin 16.9; 200 x 4100 x 8192: 20.0 and 22.4)
    const int xcd = blockIdx.x % 8, rest = nblk % 8;
    const int b = xcd * (nblk / 8) + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    constexpr int G = 4;
    const int per_group = G * tiles_n, first_m = (b / per_group) * G;
    const int gsize = tiles_m - first_m < G ? tiles_m - first_m : G;
    TileAt t;
    t.m0 = __builtin_amdgcn_readfirstlane((first_m + (b % per_group) % gsize) * BM);
    t.n0 = __builtin_amdgcn_readfirstlane(((b % per_group) / gsize) * BN);
    t.m_end = g.M;
    t.e = 0;
    t.any = true;
    return t;
}

// Four values of one row (columns n .. n + count - 1 of a lane), rounded once and stored; `vec` when rows of Y
// are aligned to four elements.
template <int OUT>
__device__ __forceinline__ void store4(void* Y, int64_t at, const float* v, int count, bool vec) {
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

template <typename Args>
__device__ __forceinline__ void zero_rows(const Args& g, const TileAt& t, int bm, int bn) {
    const int rows = t.m_end - t.m0 < bm ? t.m_end - t.m0 : bm, cols = g.N - t.n0 < bn ? g.N - t.n0 : bn;
    for (int i = threadIdx.x; i < rows * cols; i += blockDim.x) {
        const int64_t at = (int64_t)(t.m0 + i / cols) * g.ldy + t.n0 + i % cols;
        if (g.out == EP_F32) static_cast<float*>(g.Y)[at] = 0.0f;
        else static_cast<uint16_t*>(g.Y)[at] = 0;
    }
}

template <typename Args>
__device__ __forceinline__ bool vec_out(const Args& g) {
    return g.ldy % 4 == 0 && !(reinterpret_cast<uintptr_t>(g.Y) & (g.out == EP_F32 ? 15 : 7));
}

// ------------------------------------------------------------------------------- operand tiles
// Rows [r0, r0 + ROWS) up to r_end of a row-major code matrix as a buffer resource: rows past r_end
// read as zero.
template <int ROWS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint8_t* src, int ld, int64_t r0, int64_t r_end) {
    const int64_t left = r_end - r0;
    const int n = (int)(left < ROWS ? left : ROWS);
    const int bytes = __builtin_amdgcn_readfirstlane((n > 0 ? n : 0) * ld);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(src + r0 * ld), 0, bytes, 0x00020000);
}

// The eight 16-byte chunks of a 128-byte row of a stage: chunk c of row r sits at slot c ^ chunk_swizzle(r), so that
// the 16 lanes of a fragment read (16 consecutive rows, one chunk) cover all banks.
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
    __device__ __forceinline__ void init(const uint8_t* src, int ld, int64_t r0, int64_t r_end, int wave) {
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

// Tiles of BM rows that the rows split over the experts can need: every range adds at most one partly
// filled tile (the rows behind the last expert's are a range of their own).
template <typename Args>
int64_t row_tiles(const Args& g, int bm) {
    if (!g.experts) return ((int64_t)g.M + bm - 1) / bm;
    const int64_t most = (int64_t)g.rows / bm + g.experts + 1;
    return most < g.rows ? most : g.rows;
}

}  // namespace
}  // namespace ep
