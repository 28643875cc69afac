// gfx950 expert layer for few tokens: y[t] = sum over j of w[t][j] (W_out[e] h + b_out[e]), h = silu(g) u, (g, u) = W_in[e] x[t] +
// b_in[e], e = ids[t][j], in two kernels, without a sort, a host wait or atomics on memory. With few tokens the weights of
// the experts that some token chose are all that counts: both kernels stream them once from memory straight into the
// matrix operands and split K over the waves of a block.
//
// A token that names an expert twice meets it once, with the sum of the two weights. w[t][j] goes into h before its one
// rounding to the activations' type (the same relative error as rounding h itself): a column of the second
// product is then a token, not a choice, its sum runs over all experts in the matrix accumulators, and nothing has to
// be added up afterwards.
//
// Operand lane layout (v_mfma_f32_16x16x32, checked on the device): lane l supplies eight elements of A row l % 16 and
// of B column l % 16, K group l / 16, and receives C[4 (l / 16) + i][l % 16], i < 4. A and B take the same K positions per
// lane, so equal k meet whatever the order. A is the weight, B the tokens.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "entropack.h"
#include "kernels.h"
#include "mlp.h"
#include "route.h"
#include "tiles.h"

namespace ep {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------------------------------ the choices
// The tokens of every expert as a mask of 64 bits, in LDS.
__device__ __forceinline__ int64_t choice(const MlpArgs& a, int c) {
    return a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[c] : (int64_t) static_cast<const int32_t*>(a.ids)[c];
}
__device__ __forceinline__ void fill_masks(const MlpArgs& a, unsigned long long* masks) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) masks[e] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < a.T * a.k; c += blockDim.x) {
        const int64_t e = choice(a, c);
        if (e >= 0 && e < a.E) atomicOr(&masks[e], 1ull << (c / a.k));
    }
    __syncthreads();
}

// The experts with tokens, in ascending order, are the slots; a slot's tokens have consecutive rows in h. One
// expert per lane, 64 at a time: f(lane has one, e, mask, slot, first row) for every one; returns their number.
template <typename F>
__device__ __forceinline__ int each_slot(const MlpArgs& a, const unsigned long long* masks, F&& f) {
    const int lane = threadIdx.x & 63;
    int slots = 0, rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const unsigned long long m = e0 + lane < a.E ? masks[e0 + lane] : 0;
        const uint64_t hit = __ballot(m != 0);
        int upto = __popcll(m);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            if (lane >= o) upto += v;
        }
        f(m != 0, e0 + lane, m, slots + __popcll(hit & ((1ull << lane) - 1)), rows + upto - __popcll(m));
        slots += __popcll(hit);
        rows += __builtin_amdgcn_readlane(upto, 63);
    }
    return slots;
}

// The weight of token t's choices of expert e together, added in their order.
__device__ __forceinline__ float share(const MlpArgs& a, int t, int e) {
    float s = 0.0f;
    for (int j = 0; j < a.k; ++j)
        if (choice(a, t * a.k + j) == e) s += a.w ? a.w[t * a.k + j] : 1.0f;
    return s;
}

// ------------------------------------------------------------------------------------ the operands
template <int ACT>
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 c) {
    if constexpr (ACT == EP_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// Eight elements of a row of K from k on, zeros past its end; rows at any alignment of the element.
__device__ __forceinline__ u32x4 row_piece(const uint16_t* row, int64_t k, int64_t K) {
    u32x4 v = {0, 0, 0, 0};
    if (k + 8 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) v[i / 2] |= (uint32_t)row[k + i] << (16 * (i % 2));
    }
    return v;
}

// K goes in chunks of 128, four MFMA steps each. In step s the lane's eight elements are 32 s + 8 (l / 16) + i of the
// chunk for 16-bit weights (a load covers 64 bytes of each row), 32 (l / 16) + 8 s + i for MXFP4 (the lane's 16 bytes
// of codes are one block, with one scale).
template <bool MX>
__device__ __forceinline__ int k_of(int s) {
    const int g = (threadIdx.x & 63) >> 4;
    return MX ? 32 * g + 8 * s : 32 * s + 8 * g;
}

// A chunk of a weight row per lane, as it comes from memory.
template <bool MX>
struct Piece {
    u32x4 v[MX ? 1 : 4];
    uint32_t scale;
};
// One row per lane (l % 16) of a weight matrix.
template <int ACT, bool MX>
struct Rows {
    const uint8_t* w;
    const uint8_t* s;
    int64_t K, apart;           // apart: bytes between the scales of two chunks
    // row `row` of expert e's [n][K] matrix
    __device__ __forceinline__ void init(const void* W, const uint8_t* S, int e, int64_t n, int64_t K_, int64_t row) {
        K = K_;
        if constexpr (MX) {
            const int64_t chunks = (K + 127) / 128;
            w = static_cast<const uint8_t*>(W) + (e * n + row) * chunks * 64 + 16 * ((threadIdx.x & 63) >> 4);
            s = S + (e * chunks * n + row) * 4;
            apart = 4 * n;
        } else {
            w = static_cast<const uint8_t*>(W) + (e * n + row) * K * 2;
        }
    }
    __device__ __forceinline__ void load(int c, Piece<MX>* p) const {
        if constexpr (MX) {
            p->v[0] = *reinterpret_cast<const u32x4*>(w + 64 * (int64_t)c);
            p->scale = *reinterpret_cast<const uint32_t*>(s + c * apart);
        } else {
            const int64_t k0 = 128 * (int64_t)c;
#pragma unroll
            for (int i = 0; i < 4; ++i) p->v[i] = row_piece(reinterpret_cast<const uint16_t*>(w), k0 + k_of<false>(i), K);
        }
    }
};
// The operand of step s. MXFP4 values are exact in BF16, and in FP16 from 2^-14 to 65504.
template <int ACT, bool MX>
__device__ __forceinline__ u32x4 operand(const Piece<MX>& p, int s) {
    if constexpr (!MX) {
        return p.v[s];
    } else {
        const float unit = __uint_as_float((p.scale >> (8 * ((threadIdx.x & 63) >> 4)) & 255u) << 23);
        const uint32_t q = p.v[0][s];
        u32x4 v;
        if constexpr (ACT == EP_BF16) {
            v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, 0));
            v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, 1));
            v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, 2));
            v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, unit, 3));
        } else {
            v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, 0));
            v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, 1));
            v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, 2));
            v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, unit, 3));
        }
        return v;
    }
}

template <int ACT>
__device__ __forceinline__ uint16_t to_act(float v) {
    return ACT == EP_BF16 ? to_bf16(v) : to_f16(v);
}
__device__ __forceinline__ float bf16_at(const uint16_t* p, int64_t i) { return p ? __uint_as_float((uint32_t)p[i] << 16) : 0.0f; }

__host__ __device__ inline int64_t padded(int64_t n) { return (n + 127) / 128 * 128; }

// ----------------------------------------------------------------------------------- first product
// A block: 16 columns of h (their gate and up rows) of one slot's expert, for up to 16 TT of its tokens at a time. Its
// waves take the chunks of K in turn; their sums meet in LDS.
template <int ACT, bool MX, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void mlp_in(MlpArgs a) {
    __shared__ unsigned long long masks[kRouteMaxExperts];
    __shared__ float sums[NW][2 * TT][256];
    __shared__ int tokens[kMlpMaxTokens];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int tiles = (int)(padded(a.I) / 16);
    const int slot = blockIdx.x / tiles, i0 = 16 * (int)(blockIdx.x % tiles);
    fill_masks(a, masks);
    int e = -1, base = 0;
    unsigned long long mask = 0;
    each_slot(a, masks, [&](bool any, int e_, unsigned long long m, int s, int row) {
        const uint64_t mine = __ballot(any && s == slot);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            e = __builtin_amdgcn_readlane(e_, l);
            base = __builtin_amdgcn_readlane(row, l);
            mask = (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)m, l) |
                   (unsigned long long)(uint32_t)__builtin_amdgcn_readlane((int)(m >> 32), l) << 32;
        }
    });
    if (e < 0) return;
    const int n = __popcll(mask);
    if (threadIdx.x < 64 && (mask >> lane & 1)) tokens[__popcll(mask & ((1ull << lane) - 1))] = lane;
    __syncthreads();
    const int64_t ldh = padded(a.I);
    const int chunks = (a.H + 127) / 128;
    const int r = i0 + (lane & 15), row = r < a.I ? r : a.I - 1;            // columns past I: zeros, stored below
    Rows<ACT, MX> gate, up;
    gate.init(a.w_in, a.s_in, e, 2 * (int64_t)a.I, a.H, row);
    up.init(a.w_in, a.s_in, e, 2 * (int64_t)a.I, a.H, a.I + (int64_t)row);
    for (int n0 = 0; n0 < n; n0 += 16 * TT) {
        const uint16_t* x[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int at = n0 + 16 * i + (lane & 15);
            x[i] = at < n ? static_cast<const uint16_t*>(a.x) + tokens[at] * a.ldx : nullptr;
        }
        f32x4 g[TT], u[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) g[i] = u[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (i0 < a.I) {
            Piece<MX> pg, pu;
            if (wave < chunks) gate.load(wave, &pg), up.load(wave, &pu);
            for (int c = wave; c < chunks; c += NW) {
                u32x4 xv[TT][4];
#pragma unroll
                for (int i = 0; i < TT; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        xv[i][s] = x[i] ? row_piece(x[i], 128 * (int64_t)c + k_of<MX>(s), a.H) : u32x4{0, 0, 0, 0};
                Piece<MX> ng = pg, nu = pu;
                if (c + NW < chunks) gate.load(c + NW, &ng), up.load(c + NW, &nu);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const u32x4 wg = operand<ACT, MX>(pg, s), wu = operand<ACT, MX>(pu, s);
#pragma unroll
                    for (int i = 0; i < TT; ++i) {
                        g[i] = mfma<ACT>(wg, xv[i][s], g[i]);
                        u[i] = mfma<ACT>(wu, xv[i][s], u[i]);
                    }
                }
                pg = ng, pu = nu;
            }
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            *reinterpret_cast<f32x4*>(&sums[wave][2 * i][4 * lane]) = g[i];
            *reinterpret_cast<f32x4*>(&sums[wave][2 * i + 1][4 * lane]) = u[i];
        }
        __syncthreads();
        for (int i = wave; i < TT; i += NW) {
            const int at = n0 + 16 * i + (lane & 15), col = i0 + 4 * (lane >> 4);
            if (at < n) {
                f32x4 gs = {0.0f, 0.0f, 0.0f, 0.0f}, us = gs;
#pragma unroll
                for (int v = 0; v < NW; ++v) {
                    gs += *reinterpret_cast<const f32x4*>(&sums[v][2 * i][4 * lane]);
                    us += *reinterpret_cast<const f32x4*>(&sums[v][2 * i + 1][4 * lane]);
                }
                const float part = share(a, tokens[at], e);
                uint16_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t b = (int64_t)e * 2 * a.I + col + q;
                    const bool in = col + q < a.I;
                    const float gv = in ? gs[q] + bf16_at(a.b_in, b) : 0.0f, uv = in ? us[q] + bf16_at(a.b_in, b + a.I) : 0.0f;
                    o[q] = in ? to_act<ACT>(part * (gv / (1.0f + expf(-gv)) * uv)) : 0;
                }
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.h) + (base + at) * ldh + col) =
                    make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
            }
        }
        __syncthreads();                                                    // the sums are free for the next tokens
    }
}

// ---------------------------------------------------------------------------------- second product
// A block: 16 columns of y for all tokens, column t of the product being token t. Its waves take the chunks of all
// slots' K in turn; a token that did not choose a slot's expert has zeros there.
template <int ACT, bool MX, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void mlp_out(MlpArgs a) {
    __shared__ unsigned long long masks[kRouteMaxExperts];
    __shared__ unsigned long long slot_mask[kMlpMaxChoices];
    __shared__ int slot_at[kMlpMaxChoices];                                 // expert << 11 | first row
    __shared__ float sums[NW][TT][256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n0 = 16 * (int)blockIdx.x;
    fill_masks(a, masks);
    const int slots = each_slot(a, masks, [&](bool any, int e, unsigned long long m, int s, int row) {
        if (any && wave == 0) slot_mask[s] = m, slot_at[s] = e << 11 | row;
    });
    __syncthreads();
    const int64_t ldh = padded(a.I);
    const int chunks = (int)(ldh / 128);
    const int r = n0 + (lane & 15), row = r < a.N ? r : a.N - 1;
    f32x4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto load = [&](int s, int c, Piece<MX>* p) {
        Rows<ACT, MX> w;
        w.init(a.w_out, a.s_out, slot_at[s] >> 11, a.N, a.I, row);
        w.load(c, p);
    };
    int s = chunks > 0 ? wave / chunks : slots, c = chunks > 0 ? wave % chunks : 0;
    Piece<MX> p;
    if (s < slots) load(s, c, &p);
    while (s < slots) {
        int ns = s, nc = c + NW;
        while (nc >= chunks) nc -= chunks, ++ns;
        const unsigned long long m = slot_mask[s];
        const int base = slot_at[s] & 2047;
        u32x4 hv[TT][4];
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int t = 16 * i + (lane & 15);
            const uint16_t* h = static_cast<const uint16_t*>(a.h) + (base + __popcll(m & ((1ull << t) - 1))) * ldh + 128 * (int64_t)c;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                hv[i][q] = m >> t & 1 ? *reinterpret_cast<const u32x4*>(h + k_of<MX>(q)) : u32x4{0, 0, 0, 0};
        }
        Piece<MX> np = p;
        if (ns < slots) load(ns, nc, &np);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const u32x4 w = operand<ACT, MX>(p, q);
#pragma unroll
            for (int i = 0; i < TT; ++i) acc[i] = mfma<ACT>(w, hv[i][q], acc[i]);
        }
        p = np, s = ns, c = nc;
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) *reinterpret_cast<f32x4*>(&sums[wave][i][4 * lane]) = acc[i];
    __syncthreads();
    for (int i = wave; i < TT; i += NW) {
        const int t = 16 * i + (lane & 15), col = n0 + 4 * (lane >> 4);
        if (t >= a.T || col >= a.N) continue;
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NW; ++v) y += *reinterpret_cast<const f32x4*>(&sums[v][i][4 * lane]);
        if (a.b_out)
            for (int j = 0; j < a.k; ++j) {
                const int64_t e = choice(a, t * a.k + j);
                if (e < 0 || e >= a.E) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (col + q < a.N) y[q] += (a.w ? a.w[t * a.k + j] : 1.0f) * bf16_at(a.b_out, e * a.N + col + q);
            }
        const float v[4] = {y[0], y[1], y[2], y[3]};
        const bool vec = a.N % 4 == 0 && !(reinterpret_cast<uintptr_t>(a.y) & 7);
        store4<ACT>(a.y, (int64_t)t * a.N + col, v, a.N - col < 4 ? a.N - col : 4, vec);
    }
}

template <int ACT, bool MX>
hipError_t mlp_go(const MlpArgs& a, hipStream_t stream) {
    const int64_t slots = (int64_t)a.T * a.k < a.E ? (int64_t)a.T * a.k : a.E;
    const int64_t in_blocks = slots * (padded(a.I) / 16), out_blocks = ((int64_t)a.N + 15) / 16;
    if (in_blocks * 256 > kMaxThreads || out_blocks * 512 > kMaxThreads) return hipErrorInvalidValue;
    if (in_blocks > 0) {
        if (a.T <= 16) hipLaunchKernelGGL((mlp_in<ACT, MX, 1, 4>), dim3((unsigned)in_blocks), dim3(256), 0, stream, a);
        else if (a.T <= 32) hipLaunchKernelGGL((mlp_in<ACT, MX, 2, 4>), dim3((unsigned)in_blocks), dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((mlp_in<ACT, MX, 4, 4>), dim3((unsigned)in_blocks), dim3(256), 0, stream, a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (a.T <= 16) hipLaunchKernelGGL((mlp_out<ACT, MX, 1, 8>), dim3((unsigned)out_blocks), dim3(512), 0, stream, a);
    else if (a.T <= 32) hipLaunchKernelGGL((mlp_out<ACT, MX, 2, 8>), dim3((unsigned)out_blocks), dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((mlp_out<ACT, MX, 4, 8>), dim3((unsigned)out_blocks), dim3(512), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

size_t mlp_scratch(int64_t T, int64_t k, int64_t I) { return (size_t)(T * k * padded(I) * 2); }

hipError_t launch_mlp(const MlpArgs& a, hipStream_t stream) {
    if (a.T <= 0 || a.N <= 0) return hipSuccess;
    const bool mx = a.s_out != nullptr;                                     // s_in may be null where H is 0
    if (a.act == EP_BF16) return mx ? mlp_go<EP_BF16, true>(a, stream) : mlp_go<EP_BF16, false>(a, stream);
    if (a.act == EP_F16) return mx ? mlp_go<EP_F16, true>(a, stream) : mlp_go<EP_F16, false>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace ep
