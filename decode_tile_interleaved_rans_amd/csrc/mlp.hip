// gfx950 expert layer for few tokens: y[t] = sum over j of w[t][j] (W_out[e] h + b_out[e]), h = silu(g) u, (g, u) = W_in[e] x[t] +
// b_in[e], e = ids[t][j], in two kernels, without a sort or a host wait. With few tokens the weights of the experts that
// some token chose are all that counts: both kernels stream them from memory straight into the matrix operands and split K
// over the waves of a block, whose sums are added in a fixed order.
//
// A token that names an expert twice meets it once, with the sum of the two weights. h is rounded once to the activations'
// type, which the matrix instruction takes: y is then 0.0023 off (relative, L2; 16 tokens on 4 of 32 experts of 4096 x 2048 in BF16),
// where its own rounding alone makes 0.0017. h as the sum of two such numbers brings that back, but was measured 6 to 25%
// slower (that layer 215 -> 250 us, 64 tokens on 2 of 8 experts of 8192 x 4096 in MXFP4 162 -> 203). w[t][j] is not in h: it
// multiplies the 32-bit sums of the second product where a wave leaves an expert, since in FP16 w h may pass 65504 or fall below
// 2^-14 where h does not.
//
// What bounds it: 16 tokens on 4 of 32 experts of 4096 x 2048 in BF16 read 1.4 GB in 214-226 us, over 6 TB/s (a read of 400 MB in
// this pattern alone reaches 6.0). In MXFP4 the tokens' loads count as well: 64 tokens on 8 of 128 experts of 2048 x 1408
// take 160-172 us (boxes differ) for 0.58 GB. Small layers are bound by latency: each kernel takes 6 to 8 us beside the transfer of
// its weights (one token on 4 of 32 experts of 2048 x 1408 in BF16 27 us for 69 MB).
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
__device__ __forceinline__ int64_t choice(const MlpArgs& a, int c) {
    return a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[c] : (int64_t) static_cast<const int32_t*>(a.ids)[c];
}

// s_waitcnt lgkmcnt(0) and a barrier: what waves exchange through LDS is there, and loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The routing of a call, in LDS of every block of the first kernel. The experts with tokens, in ascending order, are the
// slots; the tokens of a slot, in ascending order, are consecutive rows of h.
struct Routing {
    float weight[kMlpMaxChoices];                   // of a row: its choices' weights, added in their order
    uint16_t expert[kMlpMaxChoices];                // of a slot
    uint16_t first[kMlpMaxChoices + 1];             // a slot's first row; behind the last slot, the number of rows
    uint8_t token[kMlpMaxChoices];                  // of a row
    int slots;
};
struct RoutingWork {
    unsigned long long masks[kRouteMaxExperts];     // the tokens of an expert
    float weight[kMlpMaxChoices];                   // of a choice
    int16_t id[kMlpMaxChoices];                     // of a choice, -1 where it is dropped
    uint16_t slot[kRouteMaxExperts];                // of an expert with tokens
};
__device__ __forceinline__ void route(const MlpArgs& a, Routing& r, RoutingWork& w) {
    const int n = a.T * a.k;
    int64_t e = -1;
    if (threadIdx.x < n) e = choice(a, threadIdx.x);  // in flight while the masks are cleared
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) w.masks[i] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
        if (c >= (int)blockDim.x) e = choice(a, c);
        const bool in = e >= 0 && e < a.E;
        w.id[c] = in ? (int16_t)e : (int16_t)-1;
        w.weight[c] = a.w ? a.w[c] : 1.0f;
        if (in) atomicOr(&w.masks[e], 1ull << (c / a.k));
    }
    __syncthreads();
    if (threadIdx.x < 64) {                          // 64 experts at a time, one per lane
        const int lane = threadIdx.x;
        int slots = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const unsigned long long m = e0 + lane < a.E ? w.masks[e0 + lane] : 0;
            const uint64_t hit = __ballot(m != 0);
            if (!hit) continue;
            int upto = __popcll(m);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(upto, o);
                if (lane >= o) upto += v;
            }
            if (m) {
                const int slot = slots + __popcll(hit & ((1ull << lane) - 1));
                r.expert[slot] = (uint16_t)(e0 + lane);
                r.first[slot] = (uint16_t)(rows + upto - __popcll(m));
                w.slot[e0 + lane] = (uint16_t)slot;
            }
            slots += __popcll(hit);
            rows += __builtin_amdgcn_readlane(upto, 63);
        }
        if (lane == 0) r.slots = slots, r.first[slots] = (uint16_t)rows;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
        const int e = w.id[c], t = c / a.k;
        if (e < 0) continue;
        bool again = false;                          // the token has named the expert before
        for (int o = t * a.k; o < c; ++o) again |= w.id[o] == e;
        if (again) continue;
        float sum = w.weight[c];
        for (int o = c + 1; o < (t + 1) * a.k; ++o)
            if (w.id[o] == e) sum += w.weight[o];
        const int row = r.first[w.slot[e]] + __popcll(w.masks[e] & ((1ull << t) - 1));
        r.weight[row] = sum;
        r.token[row] = (uint8_t)t;
    }
    __syncthreads();
}

// The start of part i of n things in `parts` parts whose sizes differ by one at most.
__device__ __forceinline__ int part_start(int n, int parts, int i) {
    const int each = n / parts, more = n - each * parts;
    return i * each + (i < more ? i : more);
}

// What the first kernel leaves for the second, before h in the scratch.
struct Plan {
    int slots;
    float weight[kMlpMaxChoices];                                           // of a row, as in Routing
    uint16_t expert[kMlpMaxChoices], first[kMlpMaxChoices + 1];              // of a slot, as in Routing
    uint8_t token[kMlpMaxChoices];                                          // of a row
};

// ------------------------------------------------------------------------------------ the operands
template <int ACT>
__device__ __forceinline__ f32x4 mfma(u32x4 w, u32x4 x, f32x4 c) {
    if constexpr (ACT == EP_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// K goes in chunks of 128, four MFMA steps each. In step s the lane's eight elements are 32 s + 8 (l / 16) + i of the
// chunk for 16-bit weights (a load covers 64 bytes of each row), 32 (l / 16) + 8 s + i for MXFP4 (the lane's 16 bytes
// of codes are one block, with one scale).
template <bool MX>
__device__ __forceinline__ int k_of(int s) {
    const int g = (threadIdx.x & 63) >> 4;
    return MX ? 32 * g + 8 * s : 32 * s + 8 * g;
}

// One row of K 16-bit elements per lane, at any alignment of the element. load() reads what the lane needs of chunk c without
// a branch, so that the loads of the next chunk stay in flight behind the current products: a lane whose eight elements
// reach past the row's end reads its last eight. fix() puts those right where they are used: zeros past the end.
struct Row16 {
    const uint16_t* p;
    int K;
    template <bool MX>
    __device__ __forceinline__ void load(int c, u32x4 (&v)[4]) const {
        if (K >= 8) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = 128 * c + k_of<MX>(s);
                __builtin_memcpy(&v[s], p + (k < K - 8 ? k : K - 8), 16);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) v[s] = u32x4{0, 0, 0, 0};
            if (c == 0 && k_of<MX>(0) == 0) {        // the one lane of a row that has any
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (i < K) v[0][i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
            }
        }
    }
    template <bool MX>
    __device__ __forceinline__ void fix(int c, u32x4 (&v)[4]) const {
        if (128 * (c + 1) <= K) return;
        const int r = K >= 8 ? -K & 7 : 0;           // elements before those of the lane that straddles the end
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int left = K - (128 * c + k_of<MX>(s));
            u32x4 t = v[s];
            if (r & 4) t = u32x4{t[2], t[3], 0, 0};
            if (r & 2) t = u32x4{t[1], t[2], t[3], 0};
            if (r & 1) t = u32x4{t[0] >> 16 | t[1] << 16, t[1] >> 16 | t[2] << 16, t[2] >> 16 | t[3] << 16, t[3] >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[s][i] = left >= 8 ? v[s][i] : left > 0 ? t[i] : 0;
        }
    }
};

// A chunk of a weight row per lane, as it comes from memory.
template <bool MX>
struct Chunk {
    u32x4 v[MX ? 1 : 4];
    uint32_t scale;
};
// One row per lane (l % 16) of a weight matrix.
template <bool MX>
struct Rows {
    Row16 r;
    const uint8_t *w, *s;
    int64_t apart;              // bytes between the scales of two chunks
    // row `row` of expert e's [n][K] matrix
    __device__ __forceinline__ void init(const void* W, const uint8_t* S, int e, int64_t n, int K, int64_t row) {
        if constexpr (MX) {
            const int64_t chunks = (K + 127) / 128;
            w = static_cast<const uint8_t*>(W) + (e * n + row) * chunks * 64 + 16 * ((threadIdx.x & 63) >> 4);
            s = S + (e * chunks * n + row) * 4;
            apart = 4 * n;
        } else {
            r = Row16{static_cast<const uint16_t*>(W) + (e * n + row) * K, K};
        }
    }
    __device__ __forceinline__ void load(int c, Chunk<MX>* p) const {
        if constexpr (MX) {
            p->v[0] = *reinterpret_cast<const u32x4*>(w + 64 * (int64_t)c);
            p->scale = *reinterpret_cast<const uint32_t*>(s + c * apart);
        } else {
            r.load<false>(c, p->v);
        }
    }
};
// The operand of step s. MXFP4 values are exact in BF16, and in FP16 from 2^-14 to 65504.
template <int ACT, bool MX>
__device__ __forceinline__ u32x4 operand(const Chunk<MX>& p, int s) {
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

// The scratch: Plan, a counter for every tile of y's columns, the splits' sums of y, h.
struct Layout {
    int tiles, width, splits;   // of the second product: tiles of columns, their columns together, splits of K
};
struct Scratch {
    Plan* plan;
    int* done;
    float* part;                // [splits][T][width]
    uint16_t* h;                // [rows][ldh]
};
__host__ __device__ inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
__host__ __device__ inline int64_t part_at(const Layout& l) { return up16(sizeof(Plan)) + up16(4 * (int64_t)l.tiles); }
__host__ __device__ inline int64_t h_at(const Layout& l, int64_t T) {
    return part_at(l) + (l.splits > 1 ? l.splits * T * l.width * 4 : 0);
}
__device__ __forceinline__ Scratch scratch_of(const MlpArgs& a, const Layout& l) {
    uint8_t* p = static_cast<uint8_t*>(a.scratch);
    return Scratch{reinterpret_cast<Plan*>(p), reinterpret_cast<int*>(p + up16(sizeof(Plan))), reinterpret_cast<float*>(p + part_at(l)),
                   reinterpret_cast<uint16_t*>(p + h_at(l, a.T))};
}

// The operands of a chunk of K: M weight tiles of 16 rows and 16 TT tokens. A wave has two sets of them and fills one
// while it multiplies the other.
template <int ACT, bool MX, int M, int TT>
struct Piece {
    Chunk<MX> w[M];
    u32x4 x[TT][4];
    __device__ __forceinline__ void load(const Rows<MX> (&rows)[M], const Row16 (&xs)[TT], int c) {
#pragma unroll
        for (int m = 0; m < M; ++m) rows[m].load(c, &w[m]);
#pragma unroll
        for (int t = 0; t < TT; ++t) xs[t].template load<MX>(c, x[t]);
    }
    // rows of Kw (16-bit weights) and Kx elements
    __device__ __forceinline__ void multiply(int Kw, int Kx, int c, f32x4 (&acc)[M][TT]) {
        if constexpr (!MX) {
#pragma unroll
            for (int m = 0; m < M; ++m) Row16{nullptr, Kw}.fix<false>(c, w[m].v);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) Row16{nullptr, Kx}.template fix<MX>(c, x[t]);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const u32x4 o = operand<ACT, MX>(w[m], s);
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[m][t] = mfma<ACT>(o, x[t][s], acc[m][t]);
            }
    }
};

// ----------------------------------------------------------------------------------- first product
// A unit of work is 16 P columns of h (their gate and up rows) of one slot's expert for all its tokens, 16 TT in a pass over
// the weights (more tokens take further passes, whose weights come from L2). A block takes a contiguous range of the
// units; in each its waves take the chunks of K in turn, those of the next unit in flight behind the current one's
// products, and their sums meet in LDS, where one wave finishes 16 columns of 16 tokens while the others go on.
template <int ACT, bool MX, int P, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void mlp_in(MlpArgs a, Layout lay) {
    constexpr int COLS = 16 * P, kSums = NW * 2 * P * TT * 1024;
    __shared__ Routing r;
    __shared__ __align__(16) uint8_t work[sizeof(RoutingWork) > kSums ? sizeof(RoutingWork) : kSums];
    float (*sums)[2 * P * TT][256] = reinterpret_cast<float (*)[2 * P * TT][256]>(work);
    const Scratch to = scratch_of(a, lay);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t ldh = padded(a.I);
    const int tiles = (int)(ldh / COLS), chunks = (a.H + 127) / 128;
    route(a, r, *reinterpret_cast<RoutingWork*>(work));
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s < r.slots; s += blockDim.x) to.plan->expert[s] = r.expert[s];
        for (int s = threadIdx.x; s <= r.slots; s += blockDim.x) to.plan->first[s] = r.first[s];
        for (int i = threadIdx.x; i < r.first[r.slots]; i += blockDim.x) to.plan->token[i] = r.token[i], to.plan->weight[i] = r.weight[i];
        for (int i = threadIdx.x; i < lay.tiles; i += blockDim.x) to.done[i] = 0;
        if (threadIdx.x == 0) to.plan->slots = r.slots;
    }
    const int units = r.slots * tiles;
    const int u0 = part_start(units, (int)gridDim.x, (int)blockIdx.x), u1 = part_start(units, (int)gridDim.x, (int)blockIdx.x + 1);
    if (u0 >= u1) return;

    // Unit, first token of the pass, chunk: what is loaded next, and what is multiplied next, in the same order. All waves
    // take as many steps per pass; those without a chunk left in it do nothing in the last.
    struct At {
        int u, from, c, e, base, n;
    };
    auto open = [&](At& t) {
        const int s = t.u / tiles;
        t.e = __builtin_amdgcn_readfirstlane((int)r.expert[s]);
        t.base = __builtin_amdgcn_readfirstlane((int)r.first[s]);
        t.n = __builtin_amdgcn_readfirstlane((int)r.first[s + 1]) - t.base;
        t.from = 0;
    };
    auto next = [&](At& t) {                         // true at the end of a pass
        t.c += NW;
        if (t.c - wave < chunks) return false;
        t.c = wave;
        t.from += 16 * TT;
        if (t.from >= t.n && ++t.u < u1) open(t);
        return true;
    };
    At l{u0, 0, wave, 0, 0, 0};
    Rows<MX> rows[2 * P];
    Row16 x[TT];
    auto point = [&]() {                             // the rows of l
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = COLS * (l.u % tiles) + 16 * i + (lane & 15);
            const int row = c < a.I ? c : a.I - 1;   // columns past I are not used
            rows[2 * i].init(a.w_in, a.s_in, l.e, 2 * (int64_t)a.I, a.H, row);
            rows[2 * i + 1].init(a.w_in, a.s_in, l.e, 2 * (int64_t)a.I, a.H, a.I + (int64_t)row);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {               // lanes without a token read the last one's
            const int at = l.from + 16 * i + (lane & 15);
            x[i] = Row16{static_cast<const uint16_t*>(a.x) + r.token[l.base + (at < l.n ? at : l.n - 1)] * a.ldx, a.H};
        }
    };
    typedef Piece<ACT, MX, 2 * P, TT> Ops;
    auto load = [&](Ops& o) {
        if (l.u >= u1 || chunks == 0) return;
        o.load(rows, x, l.c < chunks ? l.c : chunks - 1);
        if (next(l) && l.u < u1) point();
    };
    open(l);
    At m = l;
    point();
    f32x4 acc[2 * P][TT];
    auto clear = [&]() {
#pragma unroll
        for (int q = 0; q < 2 * P; ++q)
#pragma unroll
            for (int i = 0; i < TT; ++i) acc[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();
    int turn = 0;                                    // of the waves at finishing
    auto step = [&](Ops& o) {                        // false at the end of the range
        if (m.c < chunks) o.multiply(a.H, a.H, m.c, acc);
        const At t = m;
        const bool end = next(m);
        load(o);
        if (!end) return true;
        lds_barrier();                               // the last pass's sums are read
#pragma unroll
        for (int q = 0; q < 2 * P; ++q)
#pragma unroll
            for (int i = 0; i < TT; ++i) *reinterpret_cast<f32x4*>(&sums[wave][q * TT + i][4 * lane]) = acc[q][i];
        clear();
        lds_barrier();
#pragma unroll
        for (int j = 0; j < P * TT; ++j) {           // 16 columns of 16 tokens
            if (wave != (turn + j) % NW) continue;
            const int q = j / TT, i = j % TT;
            const int at = t.from + 16 * i + (lane & 15), col = COLS * (t.u % tiles) + 16 * q + 4 * (lane >> 4);
            if (at >= t.n) continue;
            f32x4 gs = {0.0f, 0.0f, 0.0f, 0.0f}, us = gs;
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                gs += *reinterpret_cast<const f32x4*>(&sums[v][2 * q * TT + i][4 * lane]);
                us += *reinterpret_cast<const f32x4*>(&sums[v][(2 * q + 1) * TT + i][4 * lane]);
            }
            if (a.b_in) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int64_t b = (int64_t)t.e * 2 * a.I + (col + v < a.I ? col + v : a.I - 1);
                    gs[v] += bf16_at(a.b_in, b);
                    us[v] += bf16_at(a.b_in, b + a.I);
                }
            }
            uint16_t o4[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) o4[v] = col + v < a.I ? to_act<ACT>(gs[v] / (1.0f + expf(-gs[v])) * us[v]) : 0;
            *reinterpret_cast<uint2*>(to.h + (t.base + at) * ldh + col) = make_uint2(o4[0] | (uint32_t)o4[1] << 16, o4[2] | (uint32_t)o4[3] << 16);
        }
        turn += P * TT;
        return m.u < u1;
    };
    Ops o0, o1;
    load(o0);
    load(o1);
    while (step(o0) && step(o1)) {}
}

// ---------------------------------------------------------------------------------- second product
// A block: 16 M columns of y and one of the splits of all slots' chunks of K, of which each wave takes a contiguous
// part. A wave multiplies a slot's rows of h, 16 TT in a pass, and adds the sums, times the rows' weights, to its own y
// [token][columns] in LDS when it leaves the slot. The waves' y are added in their order; with several splits the block
// that finishes last adds the splits' in theirs.
template <int ACT, bool MX, int M, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void mlp_out(MlpArgs a, Layout lay) {
    constexpr int COLS = 16 * M;
    extern __shared__ __align__(16) float ys[];      // [NW][T][COLS]
    __shared__ uint16_t expert[kMlpMaxChoices], first[kMlpMaxChoices + 1];
    __shared__ uint8_t token[kMlpMaxChoices];
    __shared__ float weight[kMlpMaxChoices];
    __shared__ bool last;
    const Scratch from = scratch_of(a, lay);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n0 = COLS * (int)blockIdx.x, split = (int)blockIdx.y, splits = lay.splits;
    const int64_t ldh = padded(a.I);
    const int chunks = (int)(ldh / 128);
    int slots = 0;
    if (a.I > 0 && a.k > 0) {
        const int most = a.T * a.k < a.E ? a.T * a.k : a.E;
        for (int i = threadIdx.x; i < most; i += blockDim.x) expert[i] = from.plan->expert[i], first[i + 1] = from.plan->first[i + 1];
        for (int i = threadIdx.x; i < a.T * a.k; i += blockDim.x) token[i] = from.plan->token[i], weight[i] = from.plan->weight[i];
        if (threadIdx.x == 0) first[0] = 0;
        slots = __builtin_amdgcn_readfirstlane(from.plan->slots);
    }
    for (int i = threadIdx.x; i < NW * a.T * COLS; i += blockDim.x) ys[i] = 0.0f;
    __syncthreads();
    const int items = slots * chunks, parts = NW * splits, part = split * NW + wave;
    const int begin = part_start(items, parts, part), end = part_start(items, parts, part + 1);

    // Item (slot and chunk) and first token of the pass: what is loaded next, and what is multiplied next. A slot's items of
    // this wave are first ... stop - 1, taken once per pass.
    struct At {
        int it, first, stop, s, from, base, n;
    };
    auto open = [&](At& t) {
        t.first = t.it;
        t.s = t.it / chunks;
        t.stop = t.s * chunks + chunks < end ? t.s * chunks + chunks : end;
        t.base = __builtin_amdgcn_readfirstlane((int)first[t.s]);
        t.n = __builtin_amdgcn_readfirstlane((int)first[t.s + 1]) - t.base;
        t.from = 0;
    };
    auto next = [&](At& t) {                         // true at the end of a pass
        if (++t.it < t.stop) return false;
        t.from += 16 * TT;
        if (t.from < t.n) t.it = t.first;
        else if (t.it < end) open(t);
        return true;
    };
    At l{begin, 0, 0, 0, 0, 0, 0};
    Rows<MX> rows[M];
    Row16 h[TT];
    auto point = [&]() {
        const int e = __builtin_amdgcn_readfirstlane((int)expert[l.s]);
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int c = n0 + 16 * i + (lane & 15);
            rows[i].init(a.w_out, a.s_out, e, a.N, a.I, c < a.N ? c : a.N - 1);
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {               // lanes without a token read the last one's
            const int at = l.from + 16 * i + (lane & 15);
            h[i] = Row16{from.h + (l.base + (at < l.n ? at : l.n - 1)) * ldh, (int)ldh};
        }
    };
    typedef Piece<ACT, MX, M, TT> Ops;
    auto load = [&](Ops& o) {
        if (l.it >= end) return;
        o.load(rows, h, l.it - l.s * chunks);
        if (next(l) && l.it < end) point();
    };
    f32x4 acc[M][TT];
#pragma unroll
    for (int q = 0; q < M; ++q)
#pragma unroll
        for (int i = 0; i < TT; ++i) acc[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (begin < end) {
        open(l);
        At m = l;
        point();
        auto step = [&](Ops& o) {                    // false at the end
            o.multiply(a.I, (int)ldh, m.it - m.s * chunks, acc);
            const At t = m;
            const bool left = next(m);
            load(o);
            if (left) {
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    const int at = t.from + 16 * i + (lane & 15), row = t.base + (at < t.n ? at : t.n - 1);
                    float* y = ys + (wave * a.T + token[row]) * COLS + 4 * (lane >> 4);
#pragma unroll
                    for (int q = 0; q < M; ++q) {
                        if (at < t.n) *reinterpret_cast<f32x4*>(y + 16 * q) += weight[row] * acc[q][i];
                        acc[q][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                }
            }
            return m.it < end;
        };
        Ops o0, o1;
        load(o0);
        load(o1);
        while (step(o0) && step(o1)) {}
    }
    __syncthreads();
    const int quads = 4 * M, width = lay.width;
    if (splits > 1) {
        for (int i = threadIdx.x; i < quads * a.T; i += blockDim.x) {
            const int t = i / quads, c = 4 * (i % quads);
            f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < NW; ++v) y += *reinterpret_cast<const f32x4*>(ys + (v * a.T + t) * COLS + c);
            *reinterpret_cast<f32x4*>(from.part + ((int64_t)split * a.T + t) * width + n0 + c) = y;
        }
        // the splits' blocks may run on other XCDs: what this block wrote has reached its L2 (vmcnt(0)) and is released
        // before it counts itself done, and what the others wrote is acquired with the count
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(&from.done[blockIdx.x], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
        __syncthreads();
        if (!last) return;
    }
    for (int i = threadIdx.x; i < quads * a.T; i += blockDim.x) {
        const int t = i / quads, c = 4 * (i % quads), col = n0 + c;
        if (col >= a.N) continue;
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
        if (splits > 1) {
            for (int v0 = 0; v0 < splits; v0 += 8) {  // eight loads in flight; added in order
                f32x4 p[8];
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    p[v] = *reinterpret_cast<const f32x4*>(from.part + ((int64_t)(v0 + v < splits ? v0 + v : v0) * a.T + t) * width + col);
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    if (v0 + v < splits) y += p[v];
            }
        } else {
#pragma unroll
            for (int v = 0; v < NW; ++v) y += *reinterpret_cast<const f32x4*>(ys + (v * a.T + t) * COLS + c);
        }
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

// Launch shapes. Measured on 19 layers of MXFP4 and as many of 16-bit weights, one to 64 tokens on 2 of 8 ... 8 of 128 experts of 1024
// x 512 ... 8192 x 4096, weights that come from HBM, in us; "a / b" stands for a as chosen and b as the alternative.
//
// From 12 tokens per expert on, a pass takes 32 tokens in both products (64 tokens, 2 of 8 of 4096 x 2048: MXFP4 58 / 66, BF16
// 110 / 117; 32 x 2048 x 1408 on 8 of 128, 2 per expert: 112, with 32 tokens 120). In the first product of 16-bit weights it does so for
// more than 16 tokens however few an expert has (64 tokens, 4 of 32 of 4096 x 2048: 362 / 381).
//
// First product: blocks of two waves with 32 columns of h, where 64 tokens' experts differ in their passes a grid of 24 waves
// to a CU (64 x 2048 x 1408 on 8 of 128 in MXFP4: 185 / 192 with 12), up to 32 tokens of 12 (16 tokens: 96 / 98 with 24; blocks of four waves
// 102; two chunks of K at a time for four waves 105). Below 512 units blocks of eight waves with 16 columns (one token,
// 4096 x 2048, 2 of 8: 17.0 / 19.4), and passes of 32 tokens blocks of four waves, a grid of 16 to a CU (64 tokens, 2 of 8 of 4096 x
// 2048: 60.3, with 12 or 24 the same; of 8192 x 4096 178, 12 181). 16-bit weights take 16 columns: above 16 tokens in passes of 32, a grid of 24 waves to a CU (64 tokens, 4
// of 32 of 4096 x 2048: 362 / 374 with 16), up to 16 tokens from 1024 units on in blocks of eight waves, one to a CU (16
// tokens, 4 of 32 of 4096 x 2048: 214 / 217), else in blocks of four and a grid of 16 waves to a CU (16 x 1024 x 512 on 2 of 16: 8 to 32
// all 23.4). A grid's waves to a CU are not those that run at once: the registers hold 16 with 16 columns in MXFP4, 8 in passes of 32
// tokens and 12 else, and the blocks past those start as others end, which evens experts of unlike passes out at the price of
// their routing.
//
// Second product: 16 columns in blocks of 16 waves where there is little work for 256 blocks, unsplit (one token, 8 of 128 of
// 2048 x 1408 in MXFP4: 22.3, 64 columns 23.9; 16 tokens, 2 of 8 of 4096 x 2048: 36.0 / 39.7), and for 16-bit weights in
// splits until there are 256 blocks (4 x 2048 x 768 on 8 of 128 in BF16: 63.7, unsplit 66.6). More work in MXFP4 takes 64 columns
// of y in blocks of eight waves, which reads h four times less often (64 x 2048 x 1408 on 8 of 128: 160 / 168), and
// passes of 32 tokens take 32 columns (64 tokens, 2 of 8 of 8192 x 4096 in BF16: 356, 16 columns 385).
//
// Work is counted in items, a slot's 128 of K. `many` of them are, for 16-bit weights, 128: splits gain nothing at 88 (one token, 8
// of 128 of 2048 x 1408: 42.4 / 42.3 unsplit; two, 4 of 32: 40.1 / 39.1) and 5% at 192 and 256 (the case above; 24 x 2048 x 2048 on 2 of 16: 83.7 /
// 88.5). In MXFP4, up to 2048 columns of y, which make at most 128 blocks of 16, 256 (24 x 2048 x 2048 on 2 of 16, 256 items: 64 columns in
// splits 38.9 / 39.5; 4 x 2048 x 768 on 8 of 128, 192: 32.6 / 31.8); wider y fill the CUs with blocks of 16 columns, and 64 columns are worth their
// splits from 512 on (32 x 4096 x 2048 on 4 of 32, 512: 106.7 / 107.6, though 8 tokens of that layer take 69.7 / 68.6; 16 tokens, 2 of 8,
// 128: 41.1 / 36.0).
struct Shape {
    Layout lay;
    bool two;                   // 32 tokens to a pass
    int outs;                   // tiles of 16 columns in a block of the second product
    int64_t slots;              // most there can be
};
Shape shape_of(int64_t T, int64_t k, int64_t E, int64_t I, int64_t N, bool mx) {
    Shape s;
    s.slots = T * k < E ? T * k : E;
    s.two = T > 16 && T * k >= 12 * E;
    const int64_t items = s.slots * (padded(I) / 128);
    const bool many = items >= (mx ? (N > 2048 ? 512 : 256) : 128);
    s.outs = s.two ? 2 : mx && many ? 4 : 1;
    s.lay.tiles = (int)((N + 16 * s.outs - 1) / (16 * s.outs));
    s.lay.width = s.lay.tiles * 16 * s.outs;
    const int most = s.two ? 4 : 8;
    s.lay.splits = (many || (s.two && items > 0)) && s.lay.tiles <= 128 ? (most * s.lay.tiles < 256 ? most : 256 / s.lay.tiles) : 1;
    return s;
}

template <int ACT, bool MX, int P, int TT, int NW>
hipError_t in_go(const MlpArgs& a, const Shape& s, int waves, hipStream_t stream) {
    const int64_t room = (int64_t)device_cus() * waves / NW, units = s.slots * (padded(a.I) / (16 * P));
    hipLaunchKernelGGL((mlp_in<ACT, MX, P, TT, NW>), dim3((unsigned)(units < room ? units : room)), dim3(64 * NW), 0, stream, a, s.lay);
    return hipGetLastError();
}
template <int ACT, bool MX, int M, int TT, int NW>
hipError_t out_go(const MlpArgs& a, const Layout& lay, hipStream_t stream) {
    hipLaunchKernelGGL((mlp_out<ACT, MX, M, TT, NW>), dim3((unsigned)lay.tiles, (unsigned)lay.splits), dim3(64 * NW),
                       (size_t)NW * a.T * 64 * M, stream, a, lay);
    return hipGetLastError();
}
template <int ACT, bool MX>
hipError_t mlp_go(const MlpArgs& a, hipStream_t stream) {
    const Shape s = shape_of(a.T, a.k, a.E, a.I, a.N, MX);
    const int64_t units = s.slots * (padded(a.I) / (MX ? 32 : 16));
    if (units > 0) {
        hipError_t e;
        if constexpr (MX) {
            if (s.two) e = in_go<ACT, true, 2, 2, 4>(a, s, 16, stream);
            else if (units < 512) e = in_go<ACT, true, 1, 1, 8>(a, s, 16, stream);
            else e = in_go<ACT, true, 2, 1, 2>(a, s, a.T > 32 ? 24 : 12, stream);
        } else {
            if (a.T > 16) e = in_go<ACT, false, 1, 2, 4>(a, s, 24, stream);
            else if (units >= 1024) e = in_go<ACT, false, 1, 1, 8>(a, s, 8, stream);
            else e = in_go<ACT, false, 1, 1, 4>(a, s, 16, stream);
        }
        if (e != hipSuccess) return e;
    }
    if (s.outs == 2) return out_go<ACT, MX, 2, 2, 8>(a, s.lay, stream);
    if constexpr (MX)
        if (s.outs == 4) return out_go<ACT, true, 4, 1, 8>(a, s.lay, stream);
    return out_go<ACT, MX, 1, 1, 16>(a, s.lay, stream);
}

}  // namespace

size_t mlp_scratch(int64_t T, int64_t k, int64_t E, int64_t I, int64_t N, bool mx) {
    if (T * k == 0 || I == 0) return 0;
    return (size_t)(h_at(shape_of(T, k, E, I, N, mx).lay, T) + T * k * padded(I) * 2);
}

hipError_t launch_mlp(const MlpArgs& a, hipStream_t stream) {
    if (a.T <= 0 || a.N <= 0) return hipSuccess;
    const bool mx = a.s_out != nullptr;                                     // s_in may be null where H is 0
    if (a.act == EP_BF16) return mx ? mlp_go<EP_BF16, true>(a, stream) : mlp_go<EP_BF16, false>(a, stream);
    if (a.act == EP_F16) return mx ? mlp_go<EP_F16, true>(a, stream) : mlp_go<EP_F16, false>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace ep
