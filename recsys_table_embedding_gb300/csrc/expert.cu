// Expert routing: tokens sorted by expert and back.
//
// T tokens, each with K experts e(t,k) in [0,E) (any other value: the pair is
// dropped) and K weights.  The P = T*K pairs are sorted by (expert, pair
// index), so the rows of one expert follow one another in token order:
//   slot[t,k]   place of pair (t,k) among the sorted pairs, -1 when dropped
//   source[s]   pair at place s, -1 beyond the last
//   offset[e]   first place of expert e; offset[E] = M, the pairs not dropped
// and the operators move rows between the two orders:
//   dispatch            rows[slot(t,k),:] = x[t,:]                      rows beyond M are zero
//   combine             out[t,:] = sum_k w[t,k] rows[slot(t,k),:]
//   combine, backward   drows[slot(t,k),:] = w[t,k] dout[t,:],  dw[t,k] = <dout[t,:], rows[slot(t,k),:]>
//   dispatch, backward  dx[t,:] = sum_k drows[slot(t,k),:]
// Sums are in 32 bits in ascending k (the inner product over a fixed tree) and
// rounded once.  Every row is written by one owner: no atomics on results.
#include "token_internal.cuh"

namespace tbe {

constexpr int ROUTE_MAX_EXPERTS = 4096;
constexpr int ROUTE_MAX_K = 1024;

__device__ __forceinline__ int expert_of(const void *ids, int index_type, int64_t p, int64_t P, int E) {
    if (p >= P) return -1;
    const int64_t e = load_index(ids, index_type, p);
    return e >= 0 && e < E ? (int)e : -1;
}

// ---------------------------------------------------------------------------
// Rows of tokens [t0, t1) to their slots, by the threads of a block; 2^lg
// threads take a token.  Bound by memory: a token's row is read once and
// written to each of its slots from registers.
template <typename T, int VEC>
__device__ __forceinline__ void dispatch_tokens(const T *__restrict__ x, int64_t x_stride, const int32_t *slot, int K,
                                                int64_t t0, int64_t t1, int vectors, int lg, T *__restrict__ rows,
                                                int64_t rows_stride) {
    constexpr int U = 4;
    const int step = 1 << lg, lane = threadIdx.x & (step - 1);
    for (int64_t t = t0 + (threadIdx.x >> lg); t < t1; t += blockDim.x >> lg) {
        const T *src = x + t * x_stride;
        for (int c0 = lane; c0 < vectors; c0 += U * step) {
            Raw<T, VEC> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * step < vectors) r[u] = load_raw<T, VEC, true>(src + (int64_t)(c0 + u * step) * VEC);
            for (int k = 0; k < K; ++k) {
                const int s = slot[t * K + k];
                if (s < 0) continue;
                T *dst = rows + (int64_t)s * rows_stride;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * step < vectors) store_raw<T, VEC>(dst + (int64_t)(c0 + u * step) * VEC, r[u]);
            }
        }
    }
}

// Rows [s0, s1) as zeros, by the threads of a block.
template <typename T, int VEC>
__device__ __forceinline__ void zero_rows(T *rows, int64_t stride, int64_t s0, int64_t s1, int vectors) {
    Raw<T, VEC> zero;
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::WORDS; ++i) zero.w[i] = 0;
    for (int64_t s = s0; s < s1; ++s)
        for (int c = threadIdx.x; c < vectors; c += blockDim.x) store_raw<T, VEC>(rows + s * stride + (int64_t)c * VEC, zero);
}

// Block's share of the places [M, P) that no pair has.
__device__ __forceinline__ void tail_share(int64_t M, int64_t P, int64_t block, int64_t blocks, int64_t &s0, int64_t &s1) {
    const int64_t per = (P - M + blocks - 1) / blocks;
    s0 = min(P, M + block * per);
    s1 = min(P, s0 + per);
}

// Exclusive scan of n shared counts over the block (result in place); returns
// their sum.  `warp_sum`: one word per warp.
__device__ __forceinline__ int block_scan(int32_t *v, int n, int32_t *warp_sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + tid;
        const int own = i < n ? v[i] : 0;
        int s = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(FULL, s, d);
            if (lane >= d) s += o;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        int add = carry;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) add += warp_sum[w];
            carry += warp_sum[w];
        }
        if (i < n) v[i] = add + s - own;
    }
    __syncthreads();
    return carry;
}

// ---------------------------------------------------------------------------
// Few pairs (tokens being generated): sort and dispatch in one launch, bound
// by latency.  A block takes a few tokens (`per`) and finds their pairs' places
// by comparing them with all others; one more block writes the experts' offsets.
// One token of 2048 bf16 to 8 of 64 experts: 4.7 us; 1001 of 501 f32 to 3: 13 us.
constexpr int SMALL_PAIRS = 4096;

template <typename T, int VEC>
__global__ void __launch_bounds__(256)
expert_small_kernel(const void *__restrict__ ids, int index_type, int tokens, int K, int E, int32_t *slot,
                    int32_t *source, int32_t *offset, int per, const T *__restrict__ x, int64_t x_stride, int vectors,
                    int lg, T *__restrict__ rows, int64_t rows_stride) {
    extern __shared__ int32_t count[];   // [E], in the last block
    __shared__ int32_t expert[SMALL_PAIRS], warp_sum[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = tokens * K;
    int mine = 0;
#pragma unroll 4
    for (int p = tid; p < P; p += 256) {
        expert[p] = expert_of(ids, index_type, p, P, E);
        mine += expert[p] >= 0;
    }
    if (blockIdx.x + 1 == gridDim.x) {
        for (int e = tid; e < E; e += 256) count[e] = 0;
        __syncthreads();
        for (int p = tid; p < P; p += 256)
            if (expert[p] >= 0) atomicAdd(&count[expert[p]], 1);
        __syncthreads();
        const int M = block_scan(count, E, warp_sum);
        for (int e = tid; e < E; e += 256) offset[e] = count[e];
        if (tid == 0) offset[E] = M;
        return;
    }
    mine = __reduce_add_sync(FULL, mine);
    if (lane == 0) warp_sum[warp] = mine;
    __syncthreads();
    int M = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) M += warp_sum[w];
    const int t0 = blockIdx.x * per, t1 = min(tokens, t0 + per);
    for (int p = t0 * K + warp; p < t1 * K; p += 8) {
        const int e = expert[p];
        int before = 0;
#pragma unroll 4
        for (int j = lane; j < P; j += 32) {
            const int o = expert[j];
            before += o >= 0 && (o < e || (o == e && j < p));
        }
        before = __reduce_add_sync(FULL, before);
        if (lane == 0) {
            slot[p] = e >= 0 ? before : -1;
            if (e >= 0) source[before] = p;
        }
    }
    int64_t s0, s1;
    tail_share(M, P, blockIdx.x, gridDim.x - 1, s0, s1);
    for (int64_t s = s0 + tid; s < s1; s += 256) source[s] = -1;
    if (rows == nullptr) return;
    __syncthreads();   // the block's slots
    dispatch_tokens<T, VEC>(x, x_stride, slot, K, t0, t1, vectors, lg, rows, rows_stride);
    zero_rows<T, VEC>(rows, rows_stride, s0, s1, vectors);
}

// ---------------------------------------------------------------------------
// More pairs: a counting sort over the experts, by tiles, one per SM.  One
// launch counts every tile's pairs per expert; the next adds up the counts
// before its tile and places the tile's pairs in order (every warp with counts
// of its own).  The rows are moved by a launch of small blocks: 32,768 tokens of
// 1024 bf16 to 8 experts each take 15 + 90 us so, 112 us when the tiles' blocks
// move them.
constexpr int PLACE_THREADS = 1024;
constexpr int PLACE_COUNTS = 16384;   // shared counts: warps * experts

__global__ void __launch_bounds__(PLACE_THREADS)
expert_count_kernel(const void *__restrict__ ids, int index_type, int64_t P, int E, int64_t tile,
                    int32_t *__restrict__ counts) {
    extern __shared__ int32_t count[];
    launch_dependents();
    for (int e = threadIdx.x; e < E; e += PLACE_THREADS) count[e] = 0;
    __syncthreads();
    const int64_t p0 = blockIdx.x * tile, p1 = min(P, p0 + tile);
#pragma unroll 4
    for (int64_t p = p0 + threadIdx.x; p < p1; p += PLACE_THREADS) {
        const int e = expert_of(ids, index_type, p, P, E);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLACE_THREADS) counts[(int64_t)blockIdx.x * E + e] = count[e];
}

__global__ void __launch_bounds__(PLACE_THREADS)
expert_place_kernel(const void *__restrict__ ids, int index_type, int64_t P, int E, int64_t tile, int warps,
                    const int32_t *counts, int32_t *slot, int32_t *source, int32_t *offset) {
    extern __shared__ int32_t smem[];
    int32_t *before = smem, *first = smem + E, *place = smem + 2 * E;   // [E], [E], [warps][E]
    __shared__ int32_t warp_sum[PLACE_THREADS / 32];
    launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tiles = gridDim.x;
    const int64_t p0 = min(P, blockIdx.x * tile), p1 = min(P, p0 + tile);
    const int64_t share = ((p1 - p0 + warps - 1) / warps + 31) / 32 * 32;
    const int64_t w0 = min(p1, p0 + warp * share), w1 = warp < warps ? min(p1, w0 + share) : w0;
    for (int i = tid; i < (2 + warps) * E; i += PLACE_THREADS) smem[i] = 0;
    __syncthreads();
    for (int64_t p = w0 + lane; p < w1; p += 32) {
        const int e = expert_of(ids, index_type, p, P, E);
        if (e >= 0) atomicAdd(&place[warp * E + e], 1);
    }
    wait_for_launch_before();
    // counts of the tiles before, and of all: as many threads per expert as there are
    int per = 1;
    while (2 * per * E <= PLACE_THREADS) per *= 2;
    for (int i = tid; i < per * E; i += PLACE_THREADS) {
        const int e = i % E;
        int sum_before = 0, sum = 0;
#pragma unroll 8
        for (int t = i / E; t < tiles; t += per) {
            const int n = counts[(int64_t)t * E + e];
            sum_before += t < (int)blockIdx.x ? n : 0;
            sum += n;
        }
        atomicAdd(&before[e], sum_before);
        atomicAdd(&first[e], sum);
    }
    __syncthreads();
    const int64_t M = block_scan(first, E, warp_sum);
    if (blockIdx.x == 0) {
        for (int e = tid; e < E; e += PLACE_THREADS) offset[e] = first[e];
        if (tid == 0) offset[E] = (int32_t)M;
    }
    for (int e = tid; e < E; e += PLACE_THREADS) {
        int at = first[e] + before[e];
        for (int w = 0; w < warps; ++w) {
            const int n = place[w * E + e];
            place[w * E + e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t p = w0 + lane; p - lane < w1; p += 32) {
        const int e = p < w1 ? expert_of(ids, index_type, p, P, E) : -1;
        const unsigned same = __match_any_sync(FULL, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int at = e >= 0 ? place[warp * E + e] + rank : -1;
        __syncwarp();
        if (e >= 0 && rank == 0) place[warp * E + e] += __popc(same);
        __syncwarp();
        if (p < w1) {
            slot[p] = at;
            if (at >= 0) source[at] = (int32_t)p;
        }
    }
    int64_t s0, s1;
    tail_share(M, P, blockIdx.x, tiles, s0, s1);
    for (int64_t s = s0 + tid; s < s1; s += PLACE_THREADS) source[s] = -1;
}

// Dispatch along a route; a block takes the tokens of 2^lg threads each and
// ends (blocks that stay and take tokens in turn write slower).  32,768 tokens
// of 1024 bf16 to 8 experts each: 90 us, 6.7 TB/s.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
expert_dispatch_kernel(const T *__restrict__ x, int64_t x_stride, const int32_t *slot, const int32_t *pairs,
                       int64_t tokens, int K, int vectors, int lg, T *__restrict__ rows, int64_t rows_stride) {
    const int64_t t0 = (int64_t)blockIdx.x << (8 - lg), t1 = min(tokens, t0 + (1 << (8 - lg)));
    wait_for_launch_before();
    dispatch_tokens<T, VEC>(x, x_stride, slot, K, t0, t1, vectors, lg, rows, rows_stride);
    int64_t s0, s1;
    tail_share(*pairs, tokens * K, blockIdx.x, gridDim.x, s0, s1);
    zero_rows<T, VEC>(rows, rows_stride, s0, s1, vectors);
}

// ---------------------------------------------------------------------------
// Rows from slots: combine, and the gradient of dispatch (no weights).  A
// group of 2^lg lanes takes `strips` column strips of one token; the rows of
// B experts are on their way at once.  Bound by the read of P rows: 32,768
// tokens of 1024 bf16 from 8 experts each take 92-96 us, 6.3-6.5 TB/s.
template <typename T, int VEC, int B>
__global__ void __launch_bounds__(256)
expert_combine_kernel(const T *__restrict__ rows, int64_t rows_stride, const int32_t *__restrict__ slot,
                      const void *__restrict__ weights, int weight_type, int64_t tokens, int K, int vectors, int lg,
                      int strips, T *__restrict__ out, int64_t out_stride) {
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    if (t >= tokens) return;
    int c = (blockIdx.y * strips << lg) + (threadIdx.x & ((1 << lg) - 1));
    for (int i = 0; i < strips && c < vectors; ++i, c += 1 << lg) {
        float acc[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
        for (int k0 = 0; k0 < K; k0 += B) {
            int s[B];
            float w[B];
#pragma unroll
            for (int j = 0; j < B; ++j) s[j] = k0 + j < K ? __ldg(slot + t * K + k0 + j) : -1;
            Raw<T, VEC> r[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (s[j] < 0) continue;
                r[j] = load_raw<T, VEC, true>(rows + (int64_t)s[j] * rows_stride + (int64_t)c * VEC);
                w[j] = weights != nullptr ? load_f32(weights, weight_type, t * K + k0 + j) : 1.f;
            }
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (s[j] < 0) continue;
                float f[VEC];
                widen<T, VEC>(r[j], f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[v] += w[j] * f[v];
            }
        }
        store_raw<T, VEC>(out + t * out_stride + (int64_t)c * VEC, narrow<T, VEC>(acc));
    }
}

// ---------------------------------------------------------------------------
// Gradient of combine: W warps take one token (one, or the whole block where
// tokens are few), B experts at a time, so that the token's gradient row is
// read once for up to eight.  Bound by one read and one write of P rows: 32,768
// tokens of 1024 bf16 to 8 experts each take 179 us, 6.7 TB/s.
template <typename T, int VEC, int W, int B>
__global__ void __launch_bounds__(256, B == 8 ? 2 : 4)
expert_combine_bwd_kernel(const T *__restrict__ dout, int64_t dout_stride, const T *rows, int64_t rows_stride,
                          const int32_t *__restrict__ slot, const int32_t *__restrict__ pairs,
                          const void *__restrict__ weights, int weight_type, int64_t tokens, int K, int vectors,
                          T *drows, int64_t drows_stride, void *__restrict__ dweights) {
    constexpr int TOKENS = 8 / W;
    __shared__ float dots[W > 1 ? 8 : 1][B];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * TOKENS + warp / W;
    if (t < tokens) {
        const T *g_row = dout + t * dout_stride;
        for (int k0 = 0; k0 < K; k0 += B) {
            int s[B];
            float w[B], dot[B];
#pragma unroll
            for (int j = 0; j < B; ++j) s[j] = k0 + j < K ? __ldg(slot + t * K + k0 + j) : -1;
#pragma unroll
            for (int j = 0; j < B; ++j) {
                w[j] = s[j] >= 0 ? load_f32(weights, weight_type, t * K + k0 + j) : 0.f;
                dot[j] = 0.f;
            }
            for (int c = (warp % W) * 32 + lane; c < vectors; c += 32 * W) {
                Raw<T, VEC> r[B];
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (s[j] >= 0) r[j] = load_raw<T, VEC, true>(rows + (int64_t)s[j] * rows_stride + (int64_t)c * VEC);
                float g[VEC];
                widen<T, VEC>(load_raw<T, VEC>(g_row + (int64_t)c * VEC), g);
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (s[j] < 0) continue;
                    float f[VEC], d[VEC];
                    widen<T, VEC>(r[j], f);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        dot[j] += g[v] * f[v];
                        d[v] = w[j] * g[v];
                    }
                    store_raw<T, VEC>(drows + (int64_t)s[j] * drows_stride + (int64_t)c * VEC, narrow<T, VEC>(d));
                }
            }
            float mine = 0.f;   // lane j: the product with expert k0+j's row
#pragma unroll
            for (int j = 0; j < B; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o /= 2) dot[j] += __shfl_xor_sync(FULL, dot[j], o);
                if (lane == j) mine = dot[j];
            }
            if constexpr (W > 1) {
                if (lane < B) dots[warp][lane] = mine;
                __syncthreads();
                if (warp == 0 && lane < B) {
                    mine = 0.f;
#pragma unroll
                    for (int i = 0; i < W; ++i) mine += dots[i][lane];
                }
            }
            if (warp % W == 0 && lane < B && k0 + lane < K) {
                const bool have = __ldg(slot + t * K + k0 + lane) >= 0;
                store_f32(dweights, weight_type, t * K + k0 + lane, have ? mine : 0.f);
            }
            if constexpr (W > 1) __syncthreads();
        }
    }
    int64_t s0, s1;
    tail_share(__ldg(pairs), tokens * K, blockIdx.x, gridDim.x, s0, s1);
    zero_rows<T, VEC>(drows, drows_stride, s0, s1, vectors);
}

// ---------------------------------------------------------------------------
// host

// Tiles of whole tokens, about one per SM (at most 256, whatever the device).
struct RouteTiles {
    int64_t tile;
    int tiles;
};
constexpr int MAX_TILES = 256;

static RouteTiles route_tiles(int64_t tokens, int K, int sms) {
    RouteTiles t;
    const int most = sms < MAX_TILES ? sms : MAX_TILES;
    const int64_t per = (tokens + most - 1) / most;
    t.tile = per * K;
    t.tiles = (int)((tokens + per - 1) / per);
    return t;
}

static tbe_status check_route(const tbe_route *r) {
    if (r == nullptr) return TBE_ERR_NULL_POINTER;
    if (r->tokens < 0 || r->K < 1 || r->K > ROUTE_MAX_K || r->experts < 1 || r->experts > ROUTE_MAX_EXPERTS ||
        r->tokens >= TOKEN_MAX_ROWS / r->K)
        return TBE_ERR_INVALID_ARGUMENT;
    if (r->offset == nullptr || (r->tokens > 0 && (r->slot == nullptr || r->source == nullptr)))
        return TBE_ERR_NULL_POINTER;
    if (!is_aligned(r->slot, 4) || !is_aligned(r->source, 4) || !is_aligned(r->offset, 4))
        return TBE_ERR_MISALIGNED;
    return TBE_OK;
}

// rows [P, H] against tokens [T, H], one type
static tbe_status check_route_rows(const tbe_route *r, const tbe_matrix *tokens, bool tokens_written,
                                   const tbe_matrix *rows, bool rows_written) {
    tbe_status st = check_matrix(tokens, tokens_written);
    if (st == TBE_OK) st = check_matrix(rows, rows_written);
    if (st != TBE_OK) return st;
    if (tokens->rows != r->tokens || rows->rows != r->tokens * r->K || tokens->cols != rows->cols ||
        tokens->cols > TOKEN_MAX_COLS)
        return TBE_ERR_INVALID_ARGUMENT;
    return tokens->dtype == rows->dtype ? TBE_OK : TBE_ERR_UNSUPPORTED_DTYPE;
}

static size_t route_workspace(int64_t P, int E) {
    return P <= SMALL_PAIRS ? 0 : (size_t)MAX_TILES * E * 4;
}

static tbe_status check_route_sort(const tbe_route *r, const void *ids, int index_type, const void *ws,
                                   size_t ws_bytes) {
    if (!known_index(index_type)) return TBE_ERR_INVALID_ARGUMENT;
    const size_t need = route_workspace(r->tokens * r->K, r->experts);
    if ((r->tokens > 0 && ids == nullptr) || (need > 0 && ws == nullptr)) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(ids, index_type == TBE_INDEX_I64 ? 8 : 4) || !is_aligned(ws, 256)) return TBE_ERR_MISALIGNED;
    return ws_bytes < need ? TBE_ERR_BUFFER_TOO_SMALL : TBE_OK;
}

// Calls fn<T, VEC> for the matrices' type and alignment.
#define TBE_ROWS_SWITCH(dtype, vec, ...)                                       \
    do {                                                                       \
        if ((dtype) == TBE_F32) {                                              \
            using T = float;                                                   \
            if ((vec) >= 4) { constexpr int VEC = 4; __VA_ARGS__; }                   \
            else if ((vec) == 2) { constexpr int VEC = 2; __VA_ARGS__; }              \
            else { constexpr int VEC = 1; __VA_ARGS__; }                              \
        } else if ((dtype) == TBE_F16) {                                       \
            using T = __half;                                                  \
            if ((vec) == 8) { constexpr int VEC = 8; __VA_ARGS__; }                   \
            else if ((vec) == 4) { constexpr int VEC = 4; __VA_ARGS__; }              \
            else if ((vec) == 2) { constexpr int VEC = 2; __VA_ARGS__; }              \
            else { constexpr int VEC = 1; __VA_ARGS__; }                              \
        } else {                                                               \
            using T = __nv_bfloat16;                                           \
            if ((vec) == 8) { constexpr int VEC = 8; __VA_ARGS__; }                   \
            else if ((vec) == 4) { constexpr int VEC = 4; __VA_ARGS__; }              \
            else if ((vec) == 2) { constexpr int VEC = 2; __VA_ARGS__; }              \
            else { constexpr int VEC = 1; __VA_ARGS__; }                              \
        }                                                                      \
    } while (0)

static int most_vector(int dtype) { return dtype == TBE_F32 ? 4 : 8; }

// Threads per token as a shift: a warp at most for many tokens, else as many
// as have a vector (`most`: those of a block).
static int token_threads(int64_t tokens, int64_t vectors, int sms, int most) {
    int s = lane_shift(vectors);
    while (s >= 5 && s < most && (1 << s) < vectors && (tokens << (s + 1)) <= (int64_t)sms * 2048) ++s;
    return s;
}

// `after`: right after the route's sort on the same stream.
static void run_dispatch(Launch &L, const tbe_route *r, const tbe_matrix *x, const tbe_matrix *rows, bool after) {
    const tbe_matrix *ms[2] = {x, rows};
    const int vec = vector_of(most_vector(x->dtype), x->cols, ms, 2);
    const int vectors = (int)(x->cols / vec), lg = token_threads(r->tokens, vectors, L.num_sms, 8);
    const dim3 grid((unsigned)(((r->tokens << lg) + 255) / 256));
    TBE_ROWS_SWITCH(x->dtype, vec, launch_with(L, "tbe_expert_dispatch", after, 1, expert_dispatch_kernel<T, VEC>, grid,
        256, 0, (const T *)x->data, x->stride, r->slot, r->offset + r->experts, r->tokens, r->K, vectors, lg,
        (T *)rows->data, rows->stride));
}

// Sort, and with `rows` the dispatch.
static void run_sort(Launch &L, const tbe_route *r, const void *ids, int index_type, void *ws, const tbe_matrix *x,
                     const tbe_matrix *rows) {
    const int64_t P = r->tokens * r->K;
    const int E = r->experts;
    if (P <= SMALL_PAIRS) {
        const int dtype = rows != nullptr ? x->dtype : TBE_F32;
        const tbe_matrix *ms[2] = {x, rows};
        const int vec = rows != nullptr ? vector_of(most_vector(dtype), x->cols, ms, 2) : 1;
        const int vectors = rows != nullptr ? (int)(x->cols / vec) : 0;
        const void *src = rows != nullptr ? x->data : nullptr;
        void *dst = rows != nullptr ? rows->data : nullptr;
        const int64_t src_stride = rows != nullptr ? x->stride : 0, dst_stride = rows != nullptr ? rows->stride : 0;
        const int per = (int)((r->tokens + 4 * L.num_sms - 1) / (4 * L.num_sms));
        int lg = lane_shift(vectors);   // threads a token: all of the block's tokens at once
        while (lg >= 5 && lg < 8 && (1 << lg) < vectors && per << (lg + 1) <= 256) ++lg;
        const unsigned blocks = (unsigned)(per > 0 ? (r->tokens + per - 1) / per : 0) + 1;
        L.before("tbe_expert_small");
        TBE_ROWS_SWITCH(dtype, vec, (expert_small_kernel<T, VEC><<<blocks, 256, (size_t)E * 4, L.stream>>>(
            ids, index_type, (int)r->tokens, r->K, E, r->slot, r->source, r->offset, per, (const T *)src, src_stride,
            vectors, lg, (T *)dst, dst_stride)));
        L.after();
        return;
    }
    const RouteTiles t = route_tiles(r->tokens, r->K, L.num_sms);
    int32_t *counts = (int32_t *)ws;
    L.before("tbe_expert_count");
    expert_count_kernel<<<t.tiles, PLACE_THREADS, (size_t)E * 4, L.stream>>>(ids, index_type, P, E, t.tile, counts);
    L.after();
    int warps = PLACE_THREADS / 32;
    while (warps > 1 && warps * E > PLACE_COUNTS) warps /= 2;
    cached_smem_attr(L.dev, (const void *)expert_place_kernel, (size_t)(PLACE_COUNTS + 2 * ROUTE_MAX_EXPERTS) * 4);
    launch_with(L, "tbe_expert_place", true, 1, expert_place_kernel, dim3(t.tiles), PLACE_THREADS,
                (size_t)(2 + warps) * E * 4, ids, index_type, P, E, t.tile, warps, counts, r->slot, r->source, r->offset);
    if (rows != nullptr) run_dispatch(L, r, x, rows, true);
}

static void run_combine(Launch &L, const tbe_route *r, const tbe_matrix *rows, const void *weights,
                        int weight_type, const tbe_matrix *out) {
    const tbe_matrix *ms[2] = {rows, out};
    const int vec = vector_of(most_vector(out->dtype), out->cols, ms, 2);
    const int vectors = (int)(out->cols / vec), lg = lane_shift(vectors);
    const int64_t all = (vectors + (1 << lg) - 1) >> lg, blocks = ((r->tokens << lg) + 255) / 256;
    // strips per group: all of a token's where that leaves enough groups
    int64_t strips = 1;
    while (strips < all && blocks * ((all + strips) / (2 * strips)) >= 16 * L.num_sms) strips *= 2;
    const dim3 grid((unsigned)blocks, (unsigned)((all + strips - 1) / strips));
    L.before("tbe_expert_combine");
    TBE_ROWS_SWITCH(out->dtype, vec, {
        auto *fn = r->K <= 4 ? expert_combine_kernel<T, VEC, 4> : expert_combine_kernel<T, VEC, 8>;
        fn<<<grid, 256, 0, L.stream>>>((const T *)rows->data, rows->stride, r->slot, weights, weight_type, r->tokens,
                                       r->K, vectors, lg, (int)strips, (T *)out->data, out->stride);
    });
    L.after();
}

static void run_combine_bwd(Launch &L, const tbe_route *r, const tbe_matrix *dout, const tbe_matrix *rows,
                            const void *weights, int weight_type, const tbe_matrix *drows, void *dweights) {
    const tbe_matrix *ms[3] = {dout, rows, drows};
    const int vec = vector_of(most_vector(rows->dtype), rows->cols, ms, 3);
    const int vectors = (int)(rows->cols / vec);
    const bool block = vectors > 32 && r->tokens <= 24 * L.num_sms;
    const unsigned grid = (unsigned)(block ? r->tokens : (r->tokens + 7) / 8);
    L.before("tbe_expert_combine_bwd");
    TBE_ROWS_SWITCH(rows->dtype, vec, {
        auto *fn = r->K <= 4 ? (block ? expert_combine_bwd_kernel<T, VEC, 8, 4> : expert_combine_bwd_kernel<T, VEC, 1, 4>)
                             : (block ? expert_combine_bwd_kernel<T, VEC, 8, 8> : expert_combine_bwd_kernel<T, VEC, 1, 8>);
        fn<<<grid, 256, 0, L.stream>>>((const T *)dout->data, dout->stride, (const T *)rows->data, rows->stride, r->slot,
                                       r->offset + r->experts, weights, weight_type, r->tokens, r->K, vectors,
                                       (T *)drows->data, drows->stride, dweights);
    });
    L.after();
}

static tbe_status check_weights(const void *weights, int dtype) {
    if (weights == nullptr) return TBE_ERR_NULL_POINTER;
    if (!known_dtype(dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    return is_aligned(weights, dtype_bytes(dtype)) ? TBE_OK : TBE_ERR_MISALIGNED;
}

}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_route_workspace_bytes(int64_t tokens, int32_t K, int32_t experts) {
    if (tokens < 0 || K < 1 || K > ROUTE_MAX_K || experts < 1 || experts > ROUTE_MAX_EXPERTS ||
        tokens >= TOKEN_MAX_ROWS / K)
        return 0;
    return route_workspace(tokens * K, experts);
}

tbe_status tbe_route_sort(const tbe_route *route, const void *expert_ids, int32_t index_type,
                          void *workspace, size_t workspace_bytes, const tbe_config *cfg,
                          cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_sort(route, expert_ids, index_type, workspace, workspace_bytes);
    if (st != TBE_OK) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_sort(L, route, expert_ids, index_type, workspace, nullptr, nullptr);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_route_dispatch(const tbe_route *route, const tbe_matrix *x, const tbe_matrix *rows,
                              const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_rows(route, x, false, rows, true);
    if (st != TBE_OK) return st;
    if (route->tokens == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_dispatch(L, route, x, rows, false);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_route_sort_dispatch(const tbe_route *route, const void *expert_ids, int32_t index_type,
                                   const tbe_matrix *x, const tbe_matrix *rows, void *workspace,
                                   size_t workspace_bytes, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_sort(route, expert_ids, index_type, workspace, workspace_bytes);
    if (st == TBE_OK) st = check_route_rows(route, x, false, rows, true);
    if (st != TBE_OK) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_sort(L, route, expert_ids, index_type, workspace, x, route->tokens > 0 ? rows : nullptr);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_route_combine(const tbe_route *route, const tbe_matrix *rows, const void *weights,
                             int32_t weight_dtype, const tbe_matrix *out, const tbe_config *cfg,
                             cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_rows(route, out, true, rows, false);
    if (st != TBE_OK || route->tokens == 0) return st;
    if ((st = check_weights(weights, weight_dtype)) != TBE_OK) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_combine(L, route, rows, weights, weight_dtype, out);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_route_dispatch_backward(const tbe_route *route, const tbe_matrix *grad_rows,
                                       const tbe_matrix *grad_x, const tbe_config *cfg,
                                       cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_rows(route, grad_x, true, grad_rows, false);
    if (st != TBE_OK || route->tokens == 0) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_combine(L, route, grad_rows, nullptr, TBE_F32, grad_x);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_route_combine_backward(const tbe_route *route, const tbe_matrix *grad_out,
                                      const tbe_matrix *rows, const void *weights, int32_t weight_dtype,
                                      const tbe_matrix *grad_rows, void *grad_weights,
                                      const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_route(route);
    if (st == TBE_OK) st = check_route_rows(route, grad_out, false, rows, false);
    if (st == TBE_OK) st = check_route_rows(route, grad_out, false, grad_rows, true);
    if (st != TBE_OK || route->tokens == 0) return st;
    if ((st = check_weights(weights, weight_dtype)) != TBE_OK) return st;
    if ((st = check_weights(grad_weights, weight_dtype)) != TBE_OK) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_combine_bwd(L, route, grad_out, rows, weights, weight_dtype, grad_rows, grad_weights);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
