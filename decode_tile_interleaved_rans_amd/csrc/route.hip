// gfx950 kernels of the expert routing: tokens sorted by the experts they chose, the experts' rows
// summed back per token with their weights, and the gradients of both.
//
// Every choice (t, j) gets a row of its own: choices are ordered by expert and within an expert by
// t k + j (a stable counting sort), dropped choices (no valid expert) last. pos[t][j] is that row, or
// -1 - row for a dropped choice, so that every kernel that walks the tokens also meets the rows that
// no expert owns and can clear them: no kernel needs a second pass or the inverse order, and each
// token's hidden vector is read once however many experts chose it. Nothing is summed by atomics on
// floating values: results do not depend on scheduling.
//
// All of it is memory bound but the order itself: 16384 tokens of 4096 BF16 columns, 4 of 64 experts, 2% dropped,
// each call repeated by itself: order 9 us, rows 130 us (671 MB, 5.1 TB/s), sum 135 us (660 MB, 4.9 TB/s), the
// gradient of the sum 239 us (1.2 GB, 5.0 TB/s); a copy reaches 5.2. In passes of sort and sum the order takes
// 11.5, the rows 107 and the sum, while the rows' last lines still leave the caches, 167. A few tokens: one
// launch of 4.7 us for order and rows.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "entropack.h"
#include "route.h"

namespace ep {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxSortBlocks = 128;

// ------------------------------------------------------------------------------- order of choices
__device__ __forceinline__ int choice_key(const RouteArgs& r, int64_t i) {
    const int64_t id = r.id_bytes == 8 ? static_cast<const int64_t*>(r.ids)[i] : static_cast<const int32_t*>(r.ids)[i];
    return id >= 0 && id < r.E ? (int)id : r.E;
}

// Lanes of the wave whose key equals this lane's, among the lanes with `on`.
__device__ __forceinline__ uint64_t same_key(int key, bool on, int bits) {
    uint64_t m = __ballot(on);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? one : ~one;
    }
    return m;
}

// LDS of a sorting block: per wave the count of each of the E + 1 keys in the current chunk of 1024
// choices, then the row where the next choice of each key goes.
struct SortLds {
    uint16_t* cnt;          // [kSortWaves][E + 1]
    int* base;              // [E + 1]
};
__host__ __device__ inline size_t sort_lds_bytes(int E) {
    return (size_t)kSortWaves * (((size_t)E + 2) & ~(size_t)1) * 2 + ((size_t)E + 1) * 4;
}
__device__ __forceinline__ SortLds sort_lds(uint8_t* smem, int E) {
    SortLds s;
    s.base = reinterpret_cast<int*>(smem);
    s.cnt = reinterpret_cast<uint16_t*>(smem + ((size_t)E + 1) * 4);
    return s;
}

// Inclusive sum over the block's threads.
__device__ __forceinline__ int block_scan(int v, int* wave_sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    if (lane == 63) wave_sum[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += wave_sum[w];
    __syncthreads();
    return v;
}

// The rank of this thread's choice among the block's earlier choices of the same key, this chunk only;
// leaves in cnt[w][key] the choices of the chunk in waves before w and returns the chunk's total of
// key threadIdx.x in *total.
__device__ __forceinline__ int chunk_rank(const SortLds& s, int E, int key, bool on, int bits, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kSortWaves * (E + 1); i += kSortThreads) s.cnt[i] = 0;
    __syncthreads();
    const uint64_t m = same_key(key, on, bits);
    const int before = __popcll(m & ((1ull << lane) - 1));
    if (on && before == 0) s.cnt[wave * (E + 1) + key] = (uint16_t)__popcll(m);
    __syncthreads();
    *total = 0;
    for (int b = threadIdx.x; b <= E; b += kSortThreads) {
        int sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = s.cnt[w * (E + 1) + b];
            s.cnt[w * (E + 1) + b] = (uint16_t)sum;
            sum += c;
        }
        if (b == (int)threadIdx.x) *total = sum;               // keys below E (<= 1024): one per thread
    }
    __syncthreads();
    return on ? before + s.cnt[wave * (E + 1) + key] : 0;
}

__device__ __forceinline__ int key_bits(int E) { return 32 - __builtin_clz((unsigned)E); }   // keys 0 .. E

// counts [blocks][E + 1]: the choices of each key in a block's part (`part` choices, a multiple of 1024).
__global__ __launch_bounds__(kSortThreads) void count_choices(RouteArgs r, int64_t n, int64_t part, int* counts) {
    extern __shared__ __align__(16) uint8_t smem[];
    int* c = reinterpret_cast<int*>(smem);
    for (int b = threadIdx.x; b <= r.E; b += kSortThreads) c[b] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * part, i1 = i0 + part < n ? i0 + part : n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&c[choice_key(r, i)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= r.E; b += kSortThreads) counts[(int64_t)blockIdx.x * (r.E + 1) + b] = c[b];
}

// Positions of a block's part: where each key starts follows from all blocks' counts.
__global__ __launch_bounds__(kSortThreads) void place_choices(RouteArgs r, int64_t n, int64_t part, const int* counts,
                                                              int blocks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int wave_sum[kSortWaves];
    __shared__ int total[kRouteMaxExperts];
    const SortLds s = sort_lds(smem, r.E);
    const int keys = r.E + 1;
    for (int b = threadIdx.x; b < keys; b += kSortThreads) {
        s.base[b] = 0;
        if (b < r.E) total[b] = 0;
    }
    __syncthreads();
    // several threads per key, each over some of the blocks (integer sums: any order)
    const int groups = keys < kSortThreads ? kSortThreads / keys : 1;
    for (int u = threadIdx.x; u < keys * groups; u += kSortThreads) {
        const int b = u % keys, g = u / keys;
        int all = 0, before = 0;
        for (int k = g; k < blocks; k += groups) {
            const int c = counts[(int64_t)k * keys + b];
            all += c;
            if (k < (int)blockIdx.x) before += c;
        }
        if (before) atomicAdd(&s.base[b], before);
        if (b < r.E && all) atomicAdd(&total[b], all);
    }
    __syncthreads();
    const int mine = (int)threadIdx.x < r.E ? total[threadIdx.x] : 0;
    const int upto = block_scan(mine, wave_sum);
    if ((int)threadIdx.x < r.E) {
        s.base[threadIdx.x] += upto - mine;
        if (blockIdx.x == 0) r.offsets[threadIdx.x + 1] = upto;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) r.offsets[0] = 0;
    if (threadIdx.x == kSortThreads - 1) s.base[r.E] += upto;  // dropped choices follow the last expert's
    __syncthreads();
    const int bits = key_bits(r.E);
    const int64_t i0 = blockIdx.x * part, i1 = i0 + part < n ? i0 + part : n;
    for (int64_t c0 = i0; c0 < i1; c0 += kSortThreads) {
        const int64_t i = c0 + threadIdx.x;
        const bool on = i < i1;
        const int key = on ? choice_key(r, i) : 0;
        int added;
        const int rank = chunk_rank(s, r.E, key, on, bits, &added);
        if (on) {
            const int row = s.base[key] + rank;
            r.pos[i] = key < r.E ? row : -1 - row;
        }
        __syncthreads();
        if ((int)threadIdx.x < r.E) s.base[threadIdx.x] += added;
        // the dropped of this chunk: all choices that went to no expert
        const int experts_added = block_scan((int)threadIdx.x < r.E ? added : 0, wave_sum);
        if (threadIdx.x == kSortThreads - 1)
            s.base[r.E] += (int)(i1 - c0 < kSortThreads ? i1 - c0 : kSortThreads) - experts_added;
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------- rows of the experts
// Where piece c (U elements or bytes) of a row of n starts: the last one ends with the row and repeats part
// of the one before it (the same values), so rows of any length and alignment move in whole pieces.
template <int U>
__device__ __forceinline__ int64_t piece_start(int64_t c, int64_t n) {
    return U * c < n - U ? U * c : n - U;
}

// Each thread takes U bytes (16, or 1 for rows shorter than that) of a token's vector and stores them once
// per choice.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int U> struct Piece { typedef u32x4 type; };
template <> struct Piece<1> { typedef uint8_t type; };
template <int U>
__device__ __forceinline__ void copy_piece(const uint8_t* x, int64_t ldx, int64_t t, int64_t c, const int32_t* pos, int k,
                                           int64_t row_bytes, int64_t R, uint8_t* rows) {
    const int64_t at = piece_start<U>(c, row_bytes);
    typename Piece<U>::type v;
    __builtin_memcpy(&v, x + t * ldx + at, U);
    for (int j = 0; j < k; ++j) {
        const int p = pos[j];
        const int64_t row = p < 0 ? -1 - (int64_t)p : p;
        const typename Piece<U>::type o = v & (typename Piece<U>::type)(p < 0 ? 0u : ~0u);   // a dropped choice's row is zero
        if (row < R) __builtin_memcpy(rows + row * row_bytes + at, &o, U);
    }
}

template <int U>
__global__ __launch_bounds__(256) void scatter_rows(const uint8_t* x, int64_t ldx, int64_t T, int k, int64_t row_bytes, int tpb,
                                                    const int32_t* pos, int64_t R, uint8_t* rows) {
    const int64_t pieces = (row_bytes + U - 1) / U;
    for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < T; t0 += (int64_t)gridDim.x * tpb) {
        if (tpb == 1) {
            for (int64_t c = threadIdx.x; c < pieces; c += 256) copy_piece<U>(x, ldx, t0, c, pos + t0 * k, k, row_bytes, R, rows);
            continue;
        }
        const int64_t t1 = t0 + tpb < T ? t0 + tpb : T;
        const int p32 = (int)pieces;                           // tpb > 1: at most 128 pieces per token
        for (int u = threadIdx.x; u < (int)(t1 - t0) * p32; u += 256) {
            const int64_t t = t0 + u / p32;
            copy_piece<U>(x, ldx, t, u % p32, pos + t * k, k, row_bytes, R, rows);
        }
    }
}

// Up to 1024 choices: every block orders all of them by itself (a chunk of one choice per thread) and
// copies its own tokens, so a decoding step takes one launch. Block 0 writes offsets and pos.
template <int U>
__global__ __launch_bounds__(kSortThreads) void sort_small(RouteArgs r, const uint8_t* x, int64_t ldx, int64_t row_bytes, int tpb,
                                                           uint8_t* rows) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int wave_sum[kSortWaves];
    __shared__ int32_t dst[kSortThreads];
    const SortLds s = sort_lds(smem, r.E);
    const int n = (int)(r.T * r.k);
    const bool on = (int)threadIdx.x < n;
    const int key = on ? choice_key(r, threadIdx.x) : 0;
    int mine;
    const int rank = chunk_rank(s, r.E, key, on, key_bits(r.E), &mine);
    if ((int)threadIdx.x >= r.E) mine = 0;
    const int upto = block_scan(mine, wave_sum);
    if ((int)threadIdx.x < r.E) s.base[threadIdx.x] = upto - mine;
    if (threadIdx.x == kSortThreads - 1) s.base[r.E] = upto;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) r.offsets[0] = 0;
        if ((int)threadIdx.x < r.E) r.offsets[threadIdx.x + 1] = upto;
    }
    __syncthreads();
    if (on) {
        const int row = s.base[key] + rank;
        const int p = key < r.E ? row : -1 - row;
        dst[threadIdx.x] = p;
        if (blockIdx.x == 0) r.pos[threadIdx.x] = p;
    }
    if (!rows) return;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * tpb, t1 = t0 + tpb < r.T ? t0 + tpb : r.T;
    const int64_t pieces = (row_bytes + U - 1) / U;
    for (int64_t u = threadIdx.x; u < (t1 - t0) * pieces; u += kSortThreads) {
        const int64_t t = t0 + u / pieces;
        copy_piece<U>(x, ldx, t, u % pieces, dst + t * r.k, r.k, row_bytes, n, rows);
    }
}

// ------------------------------------------------------------------------------- rows back to tokens
template <int DT> struct Store { typedef uint16_t type; };
template <> struct Store<EP_F32> { typedef float type; };

template <int DT>
__device__ __forceinline__ float widen(typename Store<DT>::type v) {
    if constexpr (DT == EP_F32) return v;
    else if constexpr (DT == EP_BF16) return __uint_as_float((uint32_t)v << 16);
    else return (float)__builtin_bit_cast(_Float16, v);
}
template <int DT>
__device__ __forceinline__ typename Store<DT>::type narrow(float v) {
    if constexpr (DT == EP_F32) return v;
    else if constexpr (DT == EP_BF16)
        return (uint16_t)(__builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v, 0.0f}, bf16x2)) & 0xFFFFu);
    else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// V consecutive elements: 16 bytes at any alignment of the element, or one for rows shorter than that.
template <int DT, int V>
struct Vec {
    typename Store<DT>::type e[V];
};
template <int DT, int V>
__device__ __forceinline__ Vec<DT, V> load_vec(const typename Store<DT>::type* p) {
    Vec<DT, V> v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}
template <int DT, int V>
__device__ __forceinline__ void store_vec(typename Store<DT>::type* p, const Vec<DT, V>& v) {
    __builtin_memcpy(p, &v, sizeof v);
}

constexpr int kRowsAtOnce = 4;              // rows of a token loaded together

template <int DT, int V>
__global__ __launch_bounds__(256) void combine_tokens(CombineArgs c, typename Store<DT>::type* y, int tpb) {
    typedef typename Store<DT>::type E;
    const E* ys = static_cast<const E*>(c.ys);
    const int64_t pieces = (c.H + V - 1) / V;
    auto piece = [&](int64_t t, int64_t p) {
        const int32_t* pos = c.pos + t * c.k;
        const float* w = c.w ? c.w + t * c.k : nullptr;
        const int64_t at = piece_start<V>(p, c.H);
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int j0 = 0; j0 < c.k; j0 += kRowsAtOnce) {
            Vec<DT, V> v[kRowsAtOnce];
            bool on[kRowsAtOnce];
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) {
                const int64_t row = j0 + j < c.k ? pos[j0 + j] : -1;
                on[j] = row >= 0 && row < c.R;
                if (on[j]) v[j] = load_vec<DT, V>(ys + row * c.H + at);
            }
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) {
                if (!on[j]) continue;
                const float wj = w ? w[j0 + j] : 1.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(wj, widen<DT>(v[j].e[i]), acc[i]);
            }
        }
        Vec<DT, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.e[i] = narrow<DT>(acc[i]);
        store_vec<DT, V>(y + t * c.H + at, o);
    };
    for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < c.T; t0 += (int64_t)gridDim.x * tpb) {
        if (tpb == 1) {
            for (int64_t p = threadIdx.x; p < pieces; p += 256) piece(t0, p);
            continue;
        }
        const int64_t t1 = t0 + tpb < c.T ? t0 + tpb : c.T;
        const int p32 = (int)pieces;
        for (int u = threadIdx.x; u < (int)(t1 - t0) * p32; u += 256) piece(t0 + u / p32, u % p32);
    }
}

// TPT threads per token (16 lanes, a wave, or the block). dy is read once per kRowsAtOnce choices; the dot
// products are summed per thread in column order, then across the lanes and waves in a fixed order.
template <int DT, int V, int TPT>
__global__ __launch_bounds__(256) void combine_tokens_grad(CombineArgs c, const typename Store<DT>::type* dy,
                                                           typename Store<DT>::type* d_ys, float* d_w) {
    typedef typename Store<DT>::type E;
    __shared__ float part[4][kRowsAtOnce];
    const E* ys = static_cast<const E*>(c.ys);
    const int64_t pieces = (c.H + V - 1) / V;
    // t is uniform in the block for TPT 256 (block barriers below), in a group of TPT lanes otherwise
    for (int64_t t = (int64_t)blockIdx.x * (256 / TPT) + threadIdx.x / TPT; t < c.T; t += (int64_t)gridDim.x * (256 / TPT)) {
        for (int j0 = 0; j0 < c.k; j0 += kRowsAtOnce) {
            int64_t row[kRowsAtOnce];
            float w[kRowsAtOnce], dot[kRowsAtOnce];
            bool kept[kRowsAtOnce], in[kRowsAtOnce];
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) {
                const bool has = j0 + j < c.k;
                const int p = has ? c.pos[t * c.k + j0 + j] : 0;
                row[j] = p < 0 ? -1 - (int64_t)p : p;
                in[j] = has && row[j] < c.R;
                kept[j] = in[j] && p >= 0;
                w[j] = has && c.w ? c.w[t * c.k + j0 + j] : 1.0f;
                dot[j] = 0.0f;
            }
            for (int64_t q = threadIdx.x % TPT; q < pieces; q += TPT) {
                const int64_t at = piece_start<V>(q, c.H);
                const int again = (int)(q * V - at);           // elements that the piece before has counted
                const Vec<DT, V> g = load_vec<DT, V>(dy + t * c.H + at);
                Vec<DT, V> v[kRowsAtOnce];
                if (d_w) {
#pragma unroll
                    for (int j = 0; j < kRowsAtOnce; ++j)
                        if (kept[j]) v[j] = load_vec<DT, V>(ys + row[j] * c.H + at);
                }
#pragma unroll
                for (int j = 0; j < kRowsAtOnce; ++j) {
                    if (d_w && kept[j]) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                        if (i >= again) dot[j] = __builtin_fmaf(widen<DT>(g.e[i]), widen<DT>(v[j].e[i]), dot[j]);
                    }
                    if (d_ys && in[j]) {
                        Vec<DT, V> o;
#pragma unroll
                        for (int i = 0; i < V; ++i) o.e[i] = kept[j] ? narrow<DT>(w[j] * widen<DT>(g.e[i])) : narrow<DT>(0.0f);
                        store_vec<DT, V>(d_ys + row[j] * c.H + at, o);
                    }
                }
            }
            if (!d_w) continue;
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j)
#pragma unroll
                for (int o = (TPT < 64 ? TPT : 64) / 2; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
            if constexpr (TPT == 256) {
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < kRowsAtOnce; ++j) part[threadIdx.x >> 6][j] = dot[j];
                __syncthreads();
                if (threadIdx.x < kRowsAtOnce && j0 + (int)threadIdx.x < c.k) {
                    float s = 0.0f;
                    for (int i = 0; i < 4; ++i) s += part[i][threadIdx.x];
                    d_w[t * c.k + j0 + threadIdx.x] = s;
                }
                __syncthreads();
            } else if (threadIdx.x % TPT == 0) {
#pragma unroll
                for (int j = 0; j < kRowsAtOnce; ++j)
                    if (j0 + j < c.k) d_w[t * c.k + j0 + j] = dot[j];
            }
        }
    }
}

// Blocks of a kernel that strides over its tokens: a grid may have at most 2^32 - 1 threads.
unsigned token_blocks(int64_t groups) { return (unsigned)(groups < (1 << 20) ? groups : 1 << 20); }

// Tokens per 256-thread block: several when a token has few pieces.
int tokens_per_block(int64_t pieces) { return pieces >= 256 || pieces <= 0 ? 1 : pieces > 128 ? 1 : (int)(256 / pieces); }

template <int U>
hipError_t sort_go(const RouteArgs& r, const void* x, int64_t ldx, int64_t row_bytes, void* rows, void* scratch,
                   hipStream_t stream) {
    const int64_t n = r.T * r.k, pieces = (row_bytes + U - 1) / U;
    if (n <= kSortThreads) {
        // a block's copying threads take about one 1024-piece round
        int64_t tpb = pieces > 0 ? kSortThreads / pieces : r.T;
        tpb = tpb < 1 ? 1 : tpb > r.T ? r.T : tpb;
        const unsigned blocks = n > 0 && rows && pieces > 0 ? (unsigned)((r.T + tpb - 1) / tpb) : 1u;
        hipLaunchKernelGGL(sort_small<U>, dim3(blocks), dim3(kSortThreads), sort_lds_bytes(r.E), stream, r,
                           static_cast<const uint8_t*>(x), ldx, row_bytes, (int)tpb, n > 0 ? static_cast<uint8_t*>(rows) : nullptr);
        return hipGetLastError();
    }
    const int64_t chunks = (n + kSortThreads - 1) / kSortThreads;
    const int64_t part = (chunks + kMaxSortBlocks - 1) / kMaxSortBlocks * kSortThreads;
    const int blocks = (int)((n + part - 1) / part);
    int* counts = static_cast<int*>(scratch);
    hipLaunchKernelGGL(count_choices, dim3(blocks), dim3(kSortThreads), (r.E + 1) * sizeof(int), stream, r, n, part, counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(place_choices, dim3(blocks), dim3(kSortThreads), sort_lds_bytes(r.E), stream, r, n, part,
                       (const int*)counts, blocks);
    e = hipGetLastError();
    if (e != hipSuccess || !rows || pieces <= 0) return e;
    const int tpb = tokens_per_block(pieces);
    hipLaunchKernelGGL(scatter_rows<U>, dim3(token_blocks((r.T + tpb - 1) / tpb)), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(x), ldx, r.T, r.k, row_bytes, tpb, (const int32_t*)r.pos, n,
                       static_cast<uint8_t*>(rows));
    return hipGetLastError();
}

template <int DT, int V>
hipError_t combine_go(const CombineArgs& c, void* y, hipStream_t stream) {
    const int tpb = tokens_per_block((c.H + V - 1) / V);
    hipLaunchKernelGGL((combine_tokens<DT, V>), dim3(token_blocks((c.T + tpb - 1) / tpb)), dim3(256), 0, stream, c,
                       static_cast<typename Store<DT>::type*>(y), tpb);
    return hipGetLastError();
}

template <int DT, int V, int TPT>
hipError_t grad_tpt(const CombineArgs& c, const void* dy, void* d_ys, float* d_w, hipStream_t stream) {
    typedef typename Store<DT>::type E;
    constexpr int tpb = 256 / TPT;
    hipLaunchKernelGGL((combine_tokens_grad<DT, V, TPT>), dim3(token_blocks((c.T + tpb - 1) / tpb)), dim3(256), 0, stream, c,
                       static_cast<const E*>(dy), static_cast<E*>(d_ys), d_w);
    return hipGetLastError();
}

template <int DT, int V>
hipError_t grad_go(const CombineArgs& c, const void* dy, void* d_ys, float* d_w, hipStream_t stream) {
    const int64_t pieces = (c.H + V - 1) / V;
    if (pieces <= 32) return grad_tpt<DT, V, 16>(c, dy, d_ys, d_w, stream);
    if (pieces <= 128) return grad_tpt<DT, V, 64>(c, dy, d_ys, d_w, stream);
    return grad_tpt<DT, V, 256>(c, dy, d_ys, d_w, stream);
}

}  // namespace

size_t sort_tokens_scratch(int64_t T, int k, int E) {
    return T * k <= kSortThreads ? 0 : (size_t)kMaxSortBlocks * ((size_t)E + 1) * sizeof(int);
}

hipError_t launch_sort_tokens(const RouteArgs& r, const void* x, int64_t ldx_bytes, int64_t row_bytes, void* rows,
                              void* scratch, hipStream_t stream) {
    return row_bytes >= 16 ? sort_go<16>(r, x, ldx_bytes, row_bytes, rows, scratch, stream)
                           : sort_go<1>(r, x, ldx_bytes, row_bytes, rows, scratch, stream);
}

hipError_t launch_combine_tokens(const CombineArgs& c, void* y, hipStream_t stream) {
    if (c.T <= 0 || c.H <= 0) return hipSuccess;
    const bool v = c.H >= (c.dtype == EP_F32 ? 4 : 8);
    switch (c.dtype) {
        case EP_F32: return v ? combine_go<EP_F32, 4>(c, y, stream) : combine_go<EP_F32, 1>(c, y, stream);
        case EP_BF16: return v ? combine_go<EP_BF16, 8>(c, y, stream) : combine_go<EP_BF16, 1>(c, y, stream);
        case EP_F16: return v ? combine_go<EP_F16, 8>(c, y, stream) : combine_go<EP_F16, 1>(c, y, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_combine_tokens_grad(const CombineArgs& c, const void* dy, void* d_ys, float* d_w, hipStream_t stream) {
    if (c.T <= 0) return hipSuccess;
    const bool v = c.H >= (c.dtype == EP_F32 ? 4 : 8);
    switch (c.dtype) {
        case EP_F32: return v ? grad_go<EP_F32, 4>(c, dy, d_ys, d_w, stream) : grad_go<EP_F32, 1>(c, dy, d_ys, d_w, stream);
        case EP_BF16: return v ? grad_go<EP_BF16, 8>(c, dy, d_ys, d_w, stream) : grad_go<EP_BF16, 1>(c, dy, d_ys, d_w, stream);
        case EP_F16: return v ? grad_go<EP_F16, 8>(c, dy, d_ys, d_w, stream) : grad_go<EP_F16, 1>(c, dy, d_ys, d_w, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ep
