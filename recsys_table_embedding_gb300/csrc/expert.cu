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
constexpr int SORT_CTA = 512;

// ---------------------------------------------------------------------------
// Sort: a counting sort over the experts.  Tile i holds the pairs
// [i*tile, (i+1)*tile); kernel 1 counts each tile's pairs per expert; kernel 2
// adds up the counts before its tile, and places the tile's pairs, 32 at a
// time in order.

__device__ __forceinline__ int expert_of(const void *ids, int index_type, int64_t p, int64_t P, int E) {
    if (p >= P) return -1;
    const int64_t e = load_index(ids, index_type, p);
    return e >= 0 && e < E ? (int)e : -1;
}

__global__ void __launch_bounds__(SORT_CTA)
expert_count_kernel(const void *__restrict__ ids, int index_type, int64_t P, int E, int64_t tile,
                    int32_t *__restrict__ counts) {
    extern __shared__ int32_t count[];
    for (int e = threadIdx.x; e < E; e += SORT_CTA) count[e] = 0;
    __syncthreads();
    const int64_t p0 = blockIdx.x * tile, p1 = min(P, p0 + tile);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += SORT_CTA) {
        const int e = expert_of(ids, index_type, p, P, E);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += SORT_CTA) counts[(int64_t)blockIdx.x * E + e] = count[e];
}

__global__ void __launch_bounds__(SORT_CTA)
expert_place_kernel(const void *__restrict__ ids, int index_type, int64_t P, int E, int64_t tile,
                    int tiles, const int32_t *__restrict__ counts, int32_t *__restrict__ slot,
                    int32_t *__restrict__ source, int32_t *__restrict__ offset) {
    extern __shared__ int32_t smem[];
    int32_t *base = smem, *total = smem + E;   // next place of each expert; pairs of each expert
    __shared__ int32_t warp_sum[SORT_CTA / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < E; e += SORT_CTA) {
        int before = 0, all = 0;
        for (int i = 0; i < tiles; ++i) {
            const int c = __ldg(counts + (int64_t)i * E + e);
            before += i < (int)blockIdx.x ? c : 0;
            all += c;
        }
        base[e] = before;
        total[e] = all;
    }
    __syncthreads();
    // exclusive scan of total over the experts
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += SORT_CTA) {
        const int e = e0 + tid;
        const int v = e < E ? total[e] : 0;
        int s = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(FULL, s, d);
            if (lane >= d) s += o;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        int add = carry, whole = 0;
        for (int i = 0; i < SORT_CTA / 32; ++i) {
            if (i < warp) add += warp_sum[i];
            whole += warp_sum[i];
        }
        if (e < E) {
            base[e] += add + s - v;
            if (blockIdx.x == 0) offset[e] = add + s - v;
        }
        carry += whole;
        __syncthreads();
    }
    const int64_t M = carry;
    if (blockIdx.x == 0 && tid == 0) offset[E] = (int32_t)M;
    // places of the tile's pairs, warp by warp in order
    const int64_t p0 = blockIdx.x * tile, p1 = min(P, p0 + tile);
    if (warp == 0) {
        for (int64_t p = p0 + lane; p - lane < p1; p += 32) {
            const int e = p < p1 ? expert_of(ids, index_type, p, P, E) : -1;
            const unsigned same = __match_any_sync(FULL, e);
            const int rank = __popc(same & ((1u << lane) - 1));
            int at = -1;
            if (e >= 0) at = base[e] + rank;
            __syncwarp();
            if (e >= 0 && rank == 0) base[e] += __popc(same);
            __syncwarp();
            if (p < p1) {
                slot[p] = at;
                if (at >= 0) source[at] = (int32_t)p;
            }
        }
    }
    for (int64_t p = max(p0, M) + tid; p < p1; p += SORT_CTA) source[p] = -1;
}

// ---------------------------------------------------------------------------
// Rows to slots (dispatch).  A group of 2^lg lanes takes one column chunk of
// one token's row and writes it to the token's slots; the groups of the tokens
// T, T+1, ... T+P-1 write the zero rows beyond M.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
expert_dispatch_kernel(const T *__restrict__ x, int64_t x_stride, const int32_t *__restrict__ slot,
                       const int32_t *__restrict__ pairs, int64_t tokens, int K, int vectors, int lg,
                       T *__restrict__ rows, int64_t rows_stride) {
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    const int c = (blockIdx.y << lg) + (threadIdx.x & ((1 << lg) - 1));
    if (c >= vectors) return;
    if (t < tokens) {
        const Raw<T, VEC> r = load_raw<T, VEC>(x + t * x_stride + (int64_t)c * VEC);
        for (int k = 0; k < K; ++k) {
            const int s = __ldg(slot + t * K + k);
            if (s >= 0) store_raw<T, VEC>(rows + (int64_t)s * rows_stride + (int64_t)c * VEC, r);
        }
        return;
    }
    const int64_t s = t - tokens + __ldg(pairs);
    if (s >= tokens * K) return;
    Raw<T, VEC> zero;
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::WORDS; ++i) zero.w[i] = 0;
    store_raw<T, VEC>(rows + s * rows_stride + (int64_t)c * VEC, zero);
}

// ---------------------------------------------------------------------------
// Rows from slots: combine, and the gradient of dispatch (no weights).
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
expert_combine_kernel(const T *__restrict__ rows, int64_t rows_stride, const int32_t *__restrict__ slot,
                      const void *__restrict__ weights, int weight_type, int64_t tokens, int K,
                      int vectors, int lg, T *__restrict__ out, int64_t out_stride) {
    const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    const int c = (blockIdx.y << lg) + (threadIdx.x & ((1 << lg) - 1));
    if (c >= vectors || t >= tokens) return;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    constexpr int B = 4;
    for (int k0 = 0; k0 < K; k0 += B) {
        Raw<T, VEC> r[B];
        float w[B];
        bool have[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int k = k0 + j;
            const int s = k < K ? __ldg(slot + t * K + k) : -1;
            have[j] = s >= 0;
            if (have[j]) {
                r[j] = load_raw<T, VEC>(rows + (int64_t)s * rows_stride + (int64_t)c * VEC);
                w[j] = weights != nullptr ? load_f32(weights, weight_type, t * K + k) : 1.f;
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (!have[j]) continue;
            float f[VEC];
            widen<T, VEC>(r[j], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += w[j] * f[i];
        }
    }
    store_raw<T, VEC>(out + t * out_stride + (int64_t)c * VEC, narrow<T, VEC>(acc));
}

// ---------------------------------------------------------------------------
// Gradient of combine.  A warp takes one token (blocks of 4 experts at a time:
// the token's gradient row is read once per block, from L1 after the first).
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
expert_combine_bwd_kernel(const T *__restrict__ dout, int64_t dout_stride, const T *__restrict__ rows,
                          int64_t rows_stride, const int32_t *__restrict__ slot,
                          const int32_t *__restrict__ pairs, const void *__restrict__ weights,
                          int weight_type, int64_t tokens, int K, int vectors, T *__restrict__ drows,
                          int64_t drows_stride, void *__restrict__ dweights) {
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= tokens) {
        const int64_t s = t - tokens + __ldg(pairs);
        if (s >= tokens * K) return;
        Raw<T, VEC> zero;
#pragma unroll
        for (int i = 0; i < Raw<T, VEC>::WORDS; ++i) zero.w[i] = 0;
        for (int c = lane; c < vectors; c += 32)
            store_raw<T, VEC>(drows + s * drows_stride + (int64_t)c * VEC, zero);
        return;
    }
    constexpr int B = 4;
    for (int k0 = 0; k0 < K; k0 += B) {
        int s[B];
        float w[B], dot[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int k = k0 + j;
            s[j] = k < K ? __ldg(slot + t * K + k) : -1;
            w[j] = s[j] >= 0 ? load_f32(weights, weight_type, t * K + k) : 0.f;
            dot[j] = 0.f;
        }
        for (int c = lane; c < vectors; c += 32) {
            float g[VEC];
            widen<T, VEC>(load_raw<T, VEC>(dout + t * dout_stride + (int64_t)c * VEC), g);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (s[j] < 0) continue;
                float f[VEC], d[VEC];
                widen<T, VEC>(load_raw<T, VEC>(rows + (int64_t)s[j] * rows_stride + (int64_t)c * VEC), f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    dot[j] += g[i] * f[i];
                    d[i] = w[j] * g[i];
                }
                store_raw<T, VEC>(drows + (int64_t)s[j] * drows_stride + (int64_t)c * VEC, narrow<T, VEC>(d));
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            float v = dot[j];
#pragma unroll
            for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(FULL, v, o);
            if (lane == 0 && k0 + j < K) store_f32(dweights, weight_type, t * K + k0 + j, s[j] >= 0 ? v : 0.f);
        }
    }
}

// ---------------------------------------------------------------------------
// host

struct RouteTiles {
    int64_t tile;
    int tiles;
};

static RouteTiles route_tiles(int64_t P) {
    RouteTiles t;
    t.tile = (P + 255) / 256;
    if (t.tile < 1024) t.tile = 1024;
    t.tiles = (int)((P + t.tile - 1) / t.tile);
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
    return round_up((size_t)route_tiles(P).tiles * E * 4 + 256, 256);
}

static tbe_status check_route_sort(const tbe_route *r, const void *ids, int index_type, const void *ws,
                                   size_t ws_bytes) {
    if (!known_index(index_type)) return TBE_ERR_INVALID_ARGUMENT;
    const size_t need = route_workspace(r->tokens * r->K, r->experts);
    if ((r->tokens > 0 && ids == nullptr) || (need > 0 && ws == nullptr)) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(ids, index_type == TBE_INDEX_I64 ? 8 : 4) || !is_aligned(ws, 256)) return TBE_ERR_MISALIGNED;
    return ws_bytes < need ? TBE_ERR_BUFFER_TOO_SMALL : TBE_OK;
}

static void run_sort(Launch &L, const tbe_route *r, const void *ids, int index_type, void *ws) {
    const int64_t P = r->tokens * r->K;
    const int E = r->experts;
    const RouteTiles t = route_tiles(P);
    int32_t *counts = (int32_t *)ws;
    if (t.tiles > 0) {
        L.before("tbe_expert_count");
        expert_count_kernel<<<t.tiles, SORT_CTA, (size_t)E * 4, L.stream>>>(ids, index_type, P, E, t.tile, counts);
        L.after();
    }
    L.before("tbe_expert_place");
    expert_place_kernel<<<t.tiles > 0 ? t.tiles : 1, SORT_CTA, (size_t)E * 8, L.stream>>>(
        ids, index_type, P, E, t.tile, t.tiles, counts, r->slot, r->source, r->offset);
    L.after();
}

// Calls fn<T, VEC> for the matrices' type and alignment.
#define TBE_ROWS_SWITCH(dtype, vec, CALL)                                      \
    do {                                                                       \
        if ((dtype) == TBE_F32) {                                              \
            using T = float;                                                   \
            if ((vec) >= 4) { constexpr int VEC = 4; CALL; }                   \
            else if ((vec) == 2) { constexpr int VEC = 2; CALL; }              \
            else { constexpr int VEC = 1; CALL; }                              \
        } else if ((dtype) == TBE_F16) {                                       \
            using T = __half;                                                  \
            if ((vec) == 8) { constexpr int VEC = 8; CALL; }                   \
            else if ((vec) == 4) { constexpr int VEC = 4; CALL; }              \
            else if ((vec) == 2) { constexpr int VEC = 2; CALL; }              \
            else { constexpr int VEC = 1; CALL; }                              \
        } else {                                                               \
            using T = __nv_bfloat16;                                           \
            if ((vec) == 8) { constexpr int VEC = 8; CALL; }                   \
            else if ((vec) == 4) { constexpr int VEC = 4; CALL; }              \
            else if ((vec) == 2) { constexpr int VEC = 2; CALL; }              \
            else { constexpr int VEC = 1; CALL; }                              \
        }                                                                      \
    } while (0)

static int most_vector(int dtype) { return dtype == TBE_F32 ? 4 : 8; }

static void run_dispatch(Launch &L, const tbe_route *r, const tbe_matrix *x, const tbe_matrix *rows) {
    const tbe_matrix *ms[2] = {x, rows};
    const int vec = vector_of(most_vector(x->dtype), x->cols, ms, 2);
    const int vectors = (int)(x->cols / vec), lg = lane_shift(vectors);
    // tokens, then one group for each row that may lie beyond M
    const int64_t groups = r->tokens + r->tokens * r->K;
    const dim3 grid((unsigned)(((groups << lg) + 255) / 256), (unsigned)((vectors + (1 << lg) - 1) >> lg));
    L.before("tbe_expert_dispatch");
    TBE_ROWS_SWITCH(x->dtype, vec, (expert_dispatch_kernel<T, VEC><<<grid, 256, 0, L.stream>>>(
        (const T *)x->data, x->stride, r->slot, r->offset + r->experts, r->tokens, r->K, vectors, lg,
        (T *)rows->data, rows->stride)));
    L.after();
}

static void run_combine(Launch &L, const tbe_route *r, const tbe_matrix *rows, const void *weights,
                        int weight_type, const tbe_matrix *out) {
    const tbe_matrix *ms[2] = {rows, out};
    const int vec = vector_of(most_vector(out->dtype), out->cols, ms, 2);
    const int vectors = (int)(out->cols / vec), lg = lane_shift(vectors);
    const dim3 grid((unsigned)(((r->tokens << lg) + 255) / 256), (unsigned)((vectors + (1 << lg) - 1) >> lg));
    L.before("tbe_expert_combine");
    TBE_ROWS_SWITCH(out->dtype, vec, (expert_combine_kernel<T, VEC><<<grid, 256, 0, L.stream>>>(
        (const T *)rows->data, rows->stride, r->slot, weights, weight_type, r->tokens, r->K, vectors, lg,
        (T *)out->data, out->stride)));
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
        run_sort(L, route, expert_ids, index_type, workspace);
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
        run_dispatch(L, route, x, rows);
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
        run_sort(L, route, expert_ids, index_type, workspace);
        if (route->tokens > 0) run_dispatch(L, route, x, rows);
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
        const tbe_matrix *ms[3] = {grad_out, rows, grad_rows};
        const int vec = vector_of(most_vector(rows->dtype), rows->cols, ms, 3);
        const int vectors = (int)(rows->cols / vec);
        const int64_t groups = route->tokens + route->tokens * route->K;
        L.before("tbe_expert_combine_bwd");
        TBE_ROWS_SWITCH(rows->dtype, vec, (expert_combine_bwd_kernel<T, VEC><<<(unsigned)((groups + 7) / 8), 256, 0, L.stream>>>(
            (const T *)grad_out->data, grad_out->stride, (const T *)rows->data, rows->stride, route->slot,
            route->offset + route->experts, weights, weight_dtype, route->tokens, route->K, vectors,
            (T *)grad_rows->data, grad_rows->stride, grad_weights)));
        L.after();
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
