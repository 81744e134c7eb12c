// The experts' products: rows sorted by expert times their expert's matrix, and
// the gradients of both.
//
//   forward    out[s,n] = sum_k x[s,k] W_e[n,k]
//   rows       dx[s,k]  = sum_n dy[s,n] W_e[n,k]
//   weights    dW_e[n,k] = sum_{s of e} dy[s,n] x[s,k]
//
// with the gated block's activation, or its gradient, where the sums end.
#include "token_internal.cuh"

namespace tbe {

// ---- activations: a(g) and a'(g)
struct Slope {
    float value, slope;
};
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }
// Phi(x) = erfc(-x / sqrt 2) / 2, which keeps its relative precision for x << 0
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(-0.70710678118654752f * x); }

__device__ __forceinline__ float act(int kind, float g) {
    return g * (kind == TBE_SILU ? sigmoid(g) : normal_cdf(g));
}
__device__ __forceinline__ Slope act_slope(int kind, float g) {
    if (kind == TBE_SILU) {
        const float s = sigmoid(g);
        return {g * s, s * fmaf(g, 1.0f - s, 1.0f)};
    }
    const float c = normal_cdf(g);
    return {g * c, fmaf(g * 0.3989422804014327f, expf(-0.5f * g * g), c)};
}

// ---- groups
// Rows of a group: offset[e] .. offset[e+1], held to [0, rows], the first from row
// 0 on; no offsets: all.
struct Groups {
    const int32_t *offset;
    int experts;
    int rows;
};
__device__ __forceinline__ int group_start(const Groups &g, int e) {
    if (e == 0) return 0;
    if (g.offset == nullptr) return g.rows;
    return min(max(__ldg(g.offset + e), 0), g.rows);
}

// A tile of rows: group `e` (experts: the rows behind the last), rows [r0, r1).
struct RowTile {
    int e, r0, r1;
};
// Tile number t of all groups' tiles of TILE rows, by a warp; e < 0 beyond the last.
template <int TILE> __device__ __forceinline__ RowTile find_tile(const Groups &g, int t, int lane) {
    int before = 0;
    for (int base = 0; base <= g.experts; base += 32) {
        const int e = base + lane;
        int a = 0, n = 0;
        if (e <= g.experts) {
            a = group_start(g, e);
            const int b = e < g.experts ? group_start(g, e + 1) : g.rows;
            n = b > a ? b - a : 0;
        }
        const int tiles = (n + TILE - 1) / TILE;
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, sum, o);
            if (lane >= o) sum += v;
        }
        const int first = before + sum - tiles;
        const unsigned hit = __ballot_sync(FULL, t >= first && t < first + tiles);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            const int r0 = __shfl_sync(FULL, a + (t - first) * TILE, src);
            const int end = __shfl_sync(FULL, a + n, src);
            return {base + src, r0, min(r0 + TILE, end)};
        }
        before += __shfl_sync(FULL, sum, 31);
    }
    return {-1, 0, 0};
}

// ---------------------------------------------------------------------------
// 64 x 64 tiles of sums in registers, for every type, stride and alignment.

enum Epilogue { STORE = 0, GATED = 1, GATE_GRAD = 2 };

struct RowsProduct {
    const void *x;              // [rows, K]
    int64_t xs;
    const void *w;              // W_e[n,k] at e * we + n * wn + k * wk
    int64_t we, wn, wk;
    void *out;                  // [rows, N]; GATED: hidden [rows, N / 2]; GATE_GRAD: [rows, 2 N]
    int64_t os;
    void *gate_up;              // GATED: written (or nullptr) [rows, N]; GATE_GRAD: read [rows, 2 N]
    int64_t gs;
    int N, K, activation;
    Groups groups;
};

constexpr int SIMPLE_TILE = 64, SIMPLE_K = 16;

template <typename T, int EPI>
__global__ void __launch_bounds__(256) product_rows_simple_kernel(const RowsProduct p) {
    __shared__ float sx[SIMPLE_K][SIMPLE_TILE + 4], sw[SIMPLE_K][SIMPLE_TILE + 4];
    __shared__ RowTile tile;
    if (threadIdx.x < 32) {
        const RowTile t = find_tile<SIMPLE_TILE>(p.groups, blockIdx.x, threadIdx.x);
        if (threadIdx.x == 0) tile = t;
    }
    __syncthreads();
    const RowTile t = tile;
    if (t.e < 0) return;
    const int half = p.N / 2;
    // column j of the tile: GATED tiles hold 32 columns of the gate and the same 32 of the other half
    const int c0 = blockIdx.y * (EPI == GATED ? SIMPLE_TILE / 2 : SIMPLE_TILE);
    const int cols = EPI == GATED ? half : p.N;
    auto column = [&](int j) { return EPI == GATED ? c0 + (j & 31) + (j >> 5) * half : c0 + j; };
    auto inside = [&](int j) { return (EPI == GATED ? c0 + (j & 31) : c0 + j) < cols; };
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    if (t.e < p.groups.experts) {
        const T *x = (const T *)p.x, *w = (const T *)p.w + t.e * p.we;
        for (int k0 = 0; k0 < p.K; k0 += SIMPLE_K) {
            for (int i = threadIdx.x; i < SIMPLE_TILE * SIMPLE_K; i += 256) {
                const int r = i / SIMPLE_K, k = i % SIMPLE_K;
                sx[k][r] = t.r0 + r < t.r1 && k0 + k < p.K ? to_f32(x[(int64_t)(t.r0 + r) * p.xs + k0 + k]) : 0.f;
                // the weight's contiguous direction along the threads
                const int j = p.wk == 1 ? i / SIMPLE_K : i % SIMPLE_TILE, l = p.wk == 1 ? i % SIMPLE_K : i / SIMPLE_TILE;
                sw[l][j] = inside(j) && k0 + l < p.K ? to_f32(w[(int64_t)column(j) * p.wn + (int64_t)(k0 + l) * p.wk]) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < SIMPLE_K; ++k) {
                float a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = sx[k][ty * 4 + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = sw[k][(j & 1) + tx * 2 + (j >> 1) * 32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = t.r0 + ty * 4 + i;
        if (r >= t.r1) continue;
        const bool some = t.e < p.groups.experts;       // rows behind the last group get zeros
        T *out = (T *)p.out + r * p.os;
        if constexpr (EPI == GATED) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = c0 + tx * 2 + j;
                if (c >= half) continue;
                out[c] = from_f32<T>(some ? act(p.activation, acc[i][j]) * acc[i][j + 2] : 0.f);
                if (p.gate_up != nullptr) {
                    T *z = (T *)p.gate_up + r * p.gs;
                    z[c] = from_f32<T>(acc[i][j]);
                    z[half + c] = from_f32<T>(acc[i][j + 2]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + tx * 2 + (j & 1) + (j >> 1) * 32;
                if (c >= p.N) continue;
                if constexpr (EPI == GATE_GRAD) {
                    float dg = 0.f, du = 0.f;
                    if (some) {
                        const T *z = (const T *)p.gate_up + r * p.gs;
                        const Slope a = act_slope(p.activation, to_f32(z[c]));
                        dg = acc[i][j] * to_f32(z[p.N + c]) * a.slope;
                        du = acc[i][j] * a.value;
                    }
                    out[c] = from_f32<T>(dg);
                    out[p.N + c] = from_f32<T>(du);
                } else {
                    out[c] = from_f32<T>(acc[i][j]);
                }
            }
        }
    }
}

struct WeightsProduct {
    const void *dy;             // [rows, N]
    int64_t ds;
    const void *x;              // [rows, K]
    int64_t xs;
    void *out;                  // [experts, N, K]
    int64_t oe, os;
    int N, K, out_f32, accumulate;
    Groups groups;
};

template <typename T> __global__ void __launch_bounds__(256) product_weights_simple_kernel(const WeightsProduct p) {
    __shared__ float sy[SIMPLE_K][SIMPLE_TILE + 4], sx[SIMPLE_K][SIMPLE_TILE + 4];
    const int e = blockIdx.z, n0 = blockIdx.y * SIMPLE_TILE, k0 = blockIdx.x * SIMPLE_TILE;
    const int r0 = group_start(p.groups, e);
    const int r1 = max(r0, group_start(p.groups, e + 1));
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (p.accumulate && r0 == r1) return;
    float acc[4][4] = {};
    for (int s = r0; s < r1; s += SIMPLE_K) {
        for (int i = threadIdx.x; i < SIMPLE_TILE * SIMPLE_K; i += 256) {
            const int c = i % SIMPLE_TILE, r = i / SIMPLE_TILE;
            const bool row = s + r < r1;
            sy[r][c] = row && n0 + c < p.N ? to_f32(((const T *)p.dy)[(int64_t)(s + r) * p.ds + n0 + c]) : 0.f;
            sx[r][c] = row && k0 + c < p.K ? to_f32(((const T *)p.x)[(int64_t)(s + r) * p.xs + k0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < SIMPLE_K; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sy[k][ty * 4 + i];
                b[i] = sx[k][(i & 1) + tx * 2 + (i >> 1) * 32];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + ty * 4 + i;
        if (n >= p.N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + tx * 2 + (j & 1) + (j >> 1) * 32;
            if (k >= p.K) continue;
            const int64_t at = (int64_t)e * p.oe + (int64_t)n * p.os + k;
            if (p.out_f32) {
                float *o = (float *)p.out + at;
                *o = p.accumulate ? *o + acc[i][j] : acc[i][j];
            } else {
                T *o = (T *)p.out + at;
                *o = from_f32<T>(p.accumulate ? to_f32(*o) + acc[i][j] : acc[i][j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// host

constexpr int PRODUCT_MOST_EXPERTS = 4096;

// Experts as a source (written: rows and experts do not overlap).
static tbe_status check_experts(const tbe_experts *w, bool written) {
    if (w == nullptr) return TBE_ERR_NULL_POINTER;
    if (!known_dtype(w->dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (w->experts < 1 || w->experts > PRODUCT_MOST_EXPERTS || w->rows < 1 || w->rows > TOKEN_MAX_COLS || w->cols < 1 ||
        w->cols > TOKEN_MAX_COLS || w->stride < 0 || w->expert_stride < 0)
        return TBE_ERR_INVALID_ARGUMENT;
    // every element's offset fits 62 bits
    if (w->stride > (int64_t)1 << 38 || w->expert_stride > (int64_t)1 << 48) return TBE_ERR_INVALID_ARGUMENT;
    if (written) {
        if (w->rows > 1 && w->stride < w->cols) return TBE_ERR_INVALID_ARGUMENT;
        if (w->experts > 1 && w->expert_stride < (w->rows - 1) * w->stride + w->cols) return TBE_ERR_INVALID_ARGUMENT;
    }
    if (w->data == nullptr) return TBE_ERR_NULL_POINTER;
    return is_aligned(w->data, dtype_bytes(w->dtype)) ? TBE_OK : TBE_ERR_MISALIGNED;
}

static tbe_status check_groups(const tbe_route *route, int64_t rows, int64_t experts) {
    if (rows >= TOKEN_MAX_ROWS) return TBE_ERR_INVALID_ARGUMENT;
    if (route == nullptr) return experts == 1 ? TBE_OK : TBE_ERR_INVALID_ARGUMENT;
    if (route->offset == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(route->offset, 4)) return TBE_ERR_MISALIGNED;
    if (route->tokens < 0 || route->K < 1 || route->experts != experts || route->tokens > TOKEN_MAX_ROWS ||
        route->tokens * route->K != rows)
        return TBE_ERR_INVALID_ARGUMENT;
    return TBE_OK;
}

static Groups groups_of(const tbe_route *route, int64_t rows, int64_t experts) {
    return Groups{route != nullptr ? route->offset : nullptr, (int)experts, (int)rows};
}

static tbe_status check_status(const int32_t *dev_status) {
    return is_aligned(dev_status, 4) ? TBE_OK : TBE_ERR_MISALIGNED;
}

#define TBE_TYPE_SWITCH(dtype, ...)                                            \
    do {                                                                       \
        if ((dtype) == TBE_F32) { using T = float; __VA_ARGS__; }              \
        else if ((dtype) == TBE_F16) { using T = __half; __VA_ARGS__; }        \
        else { using T = __nv_bfloat16; __VA_ARGS__; }                         \
    } while (0)

template <int EPI> static void run_rows(Launch &L, int dtype, const RowsProduct &p) {
    const int64_t tiles = (p.groups.rows + SIMPLE_TILE - 1) / SIMPLE_TILE + p.groups.experts + 1;
    const int cols = EPI == GATED ? p.N / 2 : p.N, width = EPI == GATED ? SIMPLE_TILE / 2 : SIMPLE_TILE;
    const dim3 grid((unsigned)tiles, (unsigned)((cols + width - 1) / width));
    L.before("tbe_product_rows");
    TBE_TYPE_SWITCH(dtype, (product_rows_simple_kernel<T, EPI><<<grid, 256, 0, L.stream>>>(p)));
    L.after();
}

}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_expert_gated_forward(const tbe_route *route, const tbe_matrix *rows, const tbe_experts *weight,
                                    int32_t activation, const tbe_matrix *hidden, const tbe_matrix *gate_up,
                                    int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_matrix(rows, false);
    if (st == TBE_OK) st = check_experts(weight, false);
    if (st == TBE_OK) st = check_matrix(hidden, true);
    if (st == TBE_OK && gate_up != nullptr) st = check_matrix(gate_up, true);
    if (st == TBE_OK) st = check_groups(route, rows->rows, weight->experts);
    if (st == TBE_OK) st = check_status(dev_status);
    if (st != TBE_OK) return st;
    if (rows->cols != weight->cols || weight->rows != 2 * hidden->cols || hidden->rows != rows->rows ||
        (gate_up != nullptr && (gate_up->rows != rows->rows || gate_up->cols != weight->rows)) ||
        (activation != TBE_SILU && activation != TBE_GELU))
        return TBE_ERR_INVALID_ARGUMENT;
    if (rows->dtype != weight->dtype || rows->dtype != hidden->dtype ||
        (gate_up != nullptr && gate_up->dtype != rows->dtype))
        return TBE_ERR_UNSUPPORTED_DTYPE;
    if (rows->rows == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const RowsProduct p{rows->data, rows->stride, weight->data, weight->expert_stride, weight->stride, 1,
                            hidden->data, hidden->stride, gate_up != nullptr ? gate_up->data : nullptr,
                            gate_up != nullptr ? gate_up->stride : 0, (int)weight->rows, (int)weight->cols, activation,
                            groups_of(route, rows->rows, weight->experts)};
        run_rows<GATED>(L, rows->dtype, p);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_expert_forward(const tbe_route *route, const tbe_matrix *rows, const tbe_experts *weight,
                              const tbe_matrix *out, int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_matrix(rows, false);
    if (st == TBE_OK) st = check_experts(weight, false);
    if (st == TBE_OK) st = check_matrix(out, true);
    if (st == TBE_OK) st = check_groups(route, rows->rows, weight->experts);
    if (st == TBE_OK) st = check_status(dev_status);
    if (st != TBE_OK) return st;
    if (rows->cols != weight->cols || out->cols != weight->rows || out->rows != rows->rows)
        return TBE_ERR_INVALID_ARGUMENT;
    if (rows->dtype != weight->dtype || rows->dtype != out->dtype) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (rows->rows == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const RowsProduct p{rows->data, rows->stride, weight->data, weight->expert_stride, weight->stride, 1, out->data,
                            out->stride, nullptr, 0, (int)weight->rows, (int)weight->cols, 0,
                            groups_of(route, rows->rows, weight->experts)};
        run_rows<STORE>(L, rows->dtype, p);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_expert_backward(const tbe_route *route, const tbe_matrix *grad_out, const tbe_experts *weight,
                               const tbe_matrix *gate_up, int32_t activation, const tbe_matrix *grad_rows,
                               int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_matrix(grad_out, false);
    if (st == TBE_OK) st = check_experts(weight, false);
    if (st == TBE_OK && gate_up != nullptr) st = check_matrix(gate_up, false);
    if (st == TBE_OK) st = check_matrix(grad_rows, true);
    if (st == TBE_OK) st = check_groups(route, grad_out->rows, weight->experts);
    if (st == TBE_OK) st = check_status(dev_status);
    if (st != TBE_OK) return st;
    const int64_t wide = gate_up != nullptr ? 2 * weight->cols : weight->cols;
    if (grad_out->cols != weight->rows || grad_rows->cols != wide || grad_rows->rows != grad_out->rows ||
        (gate_up != nullptr && (gate_up->rows != grad_out->rows || gate_up->cols != wide)) ||
        (gate_up != nullptr && activation != TBE_SILU && activation != TBE_GELU))
        return TBE_ERR_INVALID_ARGUMENT;
    if (grad_out->dtype != weight->dtype || grad_out->dtype != grad_rows->dtype ||
        (gate_up != nullptr && gate_up->dtype != grad_out->dtype))
        return TBE_ERR_UNSUPPORTED_DTYPE;
    if (grad_out->rows == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const RowsProduct p{grad_out->data, grad_out->stride, weight->data, weight->expert_stride, 1, weight->stride,
                            grad_rows->data, grad_rows->stride, gate_up != nullptr ? gate_up->data : nullptr,
                            gate_up != nullptr ? gate_up->stride : 0, (int)weight->cols, (int)weight->rows, activation,
                            groups_of(route, grad_out->rows, weight->experts)};
        if (gate_up != nullptr) run_rows<GATE_GRAD>(L, grad_out->dtype, p);
        else run_rows<STORE>(L, grad_out->dtype, p);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

size_t tbe_expert_workspace_bytes(int64_t rows, int64_t experts, int64_t N, int64_t K) { return 0; }

tbe_status tbe_expert_weight_backward(const tbe_route *route, const tbe_matrix *grad_out, const tbe_matrix *rows,
                                      const tbe_experts *grad_weight, int32_t accumulate, void *workspace,
                                      size_t workspace_bytes, int32_t *dev_status, const tbe_config *cfg,
                                      cudaStream_t stream) {
    tbe_status st = check_matrix(grad_out, false);
    if (st == TBE_OK) st = check_matrix(rows, false);
    if (st == TBE_OK) st = check_experts(grad_weight, true);
    if (st == TBE_OK) st = check_groups(route, rows->rows, grad_weight->experts);
    if (st == TBE_OK) st = check_status(dev_status);
    if (st == TBE_OK && !is_aligned(workspace, 256)) st = TBE_ERR_MISALIGNED;
    if (st != TBE_OK) return st;
    if (grad_out->rows != rows->rows || grad_weight->rows != grad_out->cols || grad_weight->cols != rows->cols ||
        (accumulate != 0 && accumulate != 1))
        return TBE_ERR_INVALID_ARGUMENT;
    if (grad_out->dtype != rows->dtype || (grad_weight->dtype != rows->dtype && grad_weight->dtype != TBE_F32))
        return TBE_ERR_UNSUPPORTED_DTYPE;
    const size_t need = tbe_expert_workspace_bytes(rows->rows, grad_weight->experts, grad_weight->rows, grad_weight->cols);
    if (need > 0 && workspace == nullptr) return TBE_ERR_NULL_POINTER;
    if (workspace_bytes < need) return TBE_ERR_BUFFER_TOO_SMALL;
    if (rows->rows == 0 && accumulate) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const WeightsProduct p{grad_out->data, grad_out->stride, rows->data, rows->stride, grad_weight->data,
                               grad_weight->expert_stride, grad_weight->stride, (int)grad_weight->rows,
                               (int)grad_weight->cols, grad_weight->dtype == TBE_F32, accumulate,
                               groups_of(route, rows->rows, grad_weight->experts)};
        const dim3 grid((unsigned)((p.K + SIMPLE_TILE - 1) / SIMPLE_TILE), (unsigned)((p.N + SIMPLE_TILE - 1) / SIMPLE_TILE),
                        (unsigned)grad_weight->experts);
        L.before("tbe_product_weights");
        TBE_TYPE_SWITCH(rows->dtype, (product_weights_simple_kernel<T><<<grid, 256, 0, L.stream>>>(p)));
        L.after();
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
