// The experts' products: rows sorted by expert times their expert's matrix, and
// the gradients of both.
//
//   forward    out[s,n] = sum_k x[s,k] W_e[n,k]
//   rows       dx[s,k]  = sum_n dy[s,n] W_e[n,k]
//   weights    dW_e[n,k] = sum_{s of e} dy[s,n] x[s,k]
//
// with the gated block's activation, or its gradient, where the sums end.
#include <limits.h>

#include "tensor_core.cuh"

namespace tbe {

// ---- activations: a(g) and a'(g)
struct Slope {
    float value, slope;
};
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }
// Phi(x) = erfc(-x / sqrt 2) / 2, which keeps its relative precision for x << 0
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(-0.70710678118654752f * x); }

// One activation for all elements of an array: the branch lies outside the
// loops, whose elements the compiler then interleaves.
template <int N> __device__ __forceinline__ void gate_products(int kind, float (&g)[N], const float (&u)[N]) {
    if (kind == TBE_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = g[j] * normal_cdf(g[j]) * u[j];
    }
}
template <int N> __device__ __forceinline__ void act_slopes(int kind, const float (&g)[N], Slope (&a)[N]) {
    if (kind == TBE_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float s = sigmoid(g[j]);
            a[j] = {g[j] * s, s * fmaf(g[j], 1.0f - s, 1.0f)};
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float c = normal_cdf(g[j]);
            a[j] = {g[j] * c, fmaf(g[j] * 0.3989422804014327f, expf(-0.5f * g[j] * g[j]), c)};
        }
    }
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
                float h[1] = {acc[i][j]};
                const float u[1] = {acc[i][j + 2]};
                gate_products(p.activation, h, u);
                out[c] = from_f32<T>(some ? h[0] : 0.f);
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
                        const float g[1] = {to_f32(z[c])};
                        Slope a[1];
                        act_slopes(p.activation, g, a);
                        dg = acc[i][j] * to_f32(z[p.N + c]) * a[0].slope;
                        du = acc[i][j] * a[0].value;
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
// Tensor cores: 256 x 256 tiles by pairs of CTAs.

// What a product multiplies: rows with the weight as it lies or transposed, or
// the rows' two matrices with one another.
enum Form { ROWS = 0, ROWS_GRAD = 1, WEIGHTS = 2 };

constexpr int TC_TILE = 256, TC_K = 64, TC_EPILOGUE = 8;
constexpr int TC_OPERAND = 128 * TC_K * 2, TC_STAGE = 2 * TC_OPERAND;      // bytes a CTA holds of a step
constexpr int TC_STAGED = 32 * 128;        // bytes of a warp's rows on their way out
constexpr int tc_stages(int form) { return form == WEIGHTS ? 6 : 5; }
// Steps after which the weights' sums leave the tensor core: it cuts the sum off
// at 24 bits after each product of 16 instead of rounding, which makes it too
// small by 2^-28 of itself a row (measured: 9.1e-6 after 8192 rows, 4.7e-7 after
// 512).  Sums of 512 rows are added up in registers.
constexpr int TC_SEGMENT = 512;
// Warps: four that load, issue and clear, eight that finish the sums.  Of the 168
// registers a thread that a CTA of 384 is launched with the first give up what
// the others take: 128 * 56 + 256 * 216 <= 384 * 168.
constexpr int TC_CONTROL = 4, TC_THREADS = 32 * (TC_CONTROL + TC_EPILOGUE);
constexpr int TC_LAUNCH_REGS = 168, TC_CONTROL_REGS = 56, TC_EPILOGUE_REGS = 216;
static_assert(32 * (TC_CONTROL * TC_CONTROL_REGS + TC_EPILOGUE * TC_EPILOGUE_REGS) <= TC_THREADS * TC_LAUNCH_REGS,
              "an increase beyond the launch's registers never ends");

struct TensorProduct {
    void *out;                  // ROWS, ROWS_GRAD: [rows, N] (GATED: hidden [rows, N], N columns of the gate)
    int64_t os, oe;             // WEIGHTS: [experts, M, N]
    void *gate_up;
    int64_t gs;
    int M, N, K;                // K: what the sums run over (WEIGHTS: the rows)
    int tiles_m, tiles_n;       // of a weight (WEIGHTS), of the columns
    int slices;                 // WEIGHTS: parts of each group's rows; several: each with a result of its own
    int activation, accumulate, out_f32;
    int whole_out, whole_gate;  // rows of 16-byte vectors
    int32_t *status;
    Groups groups;
};

struct TensorTile {
    int e, r0, r1;      // rows of the result, [r0, r1)
    int c;              // first column
    int s0, s1;         // what the sums run over
    int slice;
};

struct TensorBars {
    uint64_t full[6], empty[6], tail[6], cleared[6], sums[2], taken[2];
    uint32_t tmem;
};

template <int FORM>
__device__ __forceinline__ TensorTile tensor_tile(const TensorProduct &p, const int *first, int64_t t) {
    TensorTile r;
    if constexpr (FORM == WEIGHTS) {
        const int per = p.tiles_m * p.tiles_n;
        const int64_t g = t / per;
        r.e = (int)(g / p.slices);
        r.slice = (int)(g % p.slices);
        const int i = (int)(t - g * per);
        r.r0 = i / p.tiles_n * TC_TILE;
        r.r1 = p.M;
        r.c = i % p.tiles_n * TC_TILE;
        r.s0 = group_start(p.groups, r.e);
        r.s1 = max(r.s0, group_start(p.groups, r.e + 1));
        if (p.slices > 1) {
            const int each = ((r.s1 - r.s0 + p.slices - 1) / p.slices + TC_K - 1) / TC_K * TC_K;
            r.s0 = min(r.s1, r.s0 + r.slice * each);
            r.s1 = min(r.s1, r.s0 + each);
        }
    } else {
        // the group: first[e] * tiles_n <= t
        int lo = 0, hi = p.groups.experts + 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)first[mid] * p.tiles_n <= t) lo = mid;
            else hi = mid;
        }
        r.e = lo;
        const int64_t i = t - (int64_t)first[lo] * p.tiles_n;
        const int tiles = first[lo + 1] - first[lo];
        // blocks of 16 row tiles, the columns through each: 4096 rows stay in L2 beside the weights
        const int block = (int)(i / (16 * p.tiles_n));
        const int j = (int)(i - (int64_t)block * 16 * p.tiles_n), high = min(16, tiles - block * 16);
        const int a = group_start(p.groups, lo);
        const int end = lo < p.groups.experts ? max(a, group_start(p.groups, lo + 1)) : p.groups.rows;
        r.r0 = a + (block * 16 + j % high) * TC_TILE;
        r.r1 = min(r.r0 + TC_TILE, end);
        r.c = j / high;
        r.s0 = 0;
        r.s1 = lo < p.groups.experts ? p.K : 0;
    }
    return r;
}

// ---- results: a warp's 32 rows of 128 bytes go through shared memory, so that
// they are written a row after the other (16-byte vectors, the row's number
// mixed into their places against bank conflicts).

// 32 columns of this lane's row as T, into the first or second half of its 128 bytes.
template <typename T> __device__ __forceinline__ void pack_columns(const float (&f)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float two[2] = {f[2 * j], f[2 * j + 1]};
        w[j] = narrow<T, 2>(two).w[0];
    }
}
__device__ __forceinline__ void stage_columns(unsigned char *staged, int lane, int half, const uint32_t (&w)[16]) {
    uint4 *row = (uint4 *)(staged + lane * 128);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        row[(half * 4 + j) ^ (lane & 7)] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
// The staged 32 rows x 64 columns to `out` (its first row and column), `rows`
// and `cols` of which exist; whole: rows of 16-byte vectors.
template <typename T>
__device__ __forceinline__ void write_columns(const unsigned char *staged, int lane, T *out, int64_t stride, int rows,
                                              int cols, bool whole) {
    __syncwarp();
    const int unit = lane & 7;
    if (whole && cols % 8 == 0) {
        if (unit * 8 < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = i * 4 + (lane >> 3);
                if (row < rows)
                    *(uint4 *)(out + row * stride + unit * 8) = *(const uint4 *)(staged + row * 128 + ((unit ^ (row & 7)) << 4));
            }
        }
    } else {
        for (int row = 0; row < rows; ++row) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = j * 32 + lane;
                if (c < cols)
                    out[row * stride + c] = *(const T *)(staged + row * 128 + (((c >> 3) ^ (row & 7)) << 4) + (c & 7) * 2);
            }
        }
    }
    __syncwarp();
}

// 32 sums of this lane's row from TMEM; without products: `fill`
__device__ __forceinline__ void load_sums(float (&v)[32], uint32_t from, bool some, float fill) {
    if (some) {
        uint32_t bits[32];
        __syncwarp();
        tc::tmem_ld32(from, bits);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(bits[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = fill;
    }
}

// What a warp writes of a tile of rows: 32 rows from `row`, `rows` of which
// exist, and its half of the tile's columns, from TMEM column `from` on.  `some`:
// there are sums, otherwise `fill` stands for them.
template <typename T, int EPI>
__device__ __forceinline__ void finish_rows(const TensorProduct &p, unsigned char *staged, int lane, uint32_t from,
                                            bool some, float fill, int64_t row, int rows, int c) {
    constexpr int CHUNKS = EPI == GATED ? 1 : 2;        // of 64 columns
#pragma unroll 1
    for (int i = 0; i < CHUNKS; ++i, c += 64, from += 64) {
        const int cols = min(64, p.N - c);
        T *out = (T *)p.out + row * p.os + c;
        if constexpr (EPI == STORE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                uint32_t w[16];
                load_sums(v, from + h * 32, some, fill);
                pack_columns<T>(v, w);
                stage_columns(staged, lane, h, w);
            }
            write_columns<T>(staged, lane, out, p.os, rows, cols, p.whole_out);
        } else if constexpr (EPI == GATED) {
            // the gate's sums, the others 128 columns further, then the product
            if (p.gate_up != nullptr) {
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[32];
                        uint32_t w[16];
                        load_sums(v, from + k * 128 + h * 32, some, fill);
                        pack_columns<T>(v, w);
                        stage_columns(staged, lane, h, w);
                    }
                    write_columns<T>(staged, lane, (T *)p.gate_up + row * p.gs + k * p.N + c, p.gs, rows, cols,
                                     p.whole_gate && (k == 0 || p.N % 8 == 0));
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float g[32], u[32];
                uint32_t w[16];
                load_sums(g, from + h * 32, some, fill);
                load_sums(u, from + 128 + h * 32, some, fill);
                gate_products(p.activation, g, u);
                pack_columns<T>(g, w);
                stage_columns(staged, lane, h, w);
            }
            write_columns<T>(staged, lane, out, p.os, rows, cols, p.whole_out);
        }
    }
}

// This lane's 32 sums as FP32 into its 128 bytes.
__device__ __forceinline__ void stage_sums(unsigned char *staged, int lane, const float (&v)[32]) {
    float4 *row = (float4 *)(staged + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j) row[j ^ (lane & 7)] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
// Four sums of row i * 4 + lane / 8, columns (lane % 8) * 4 on.
__device__ __forceinline__ float4 staged_sums(const unsigned char *staged, int lane, int i) {
    const int row = i * 4 + (lane >> 3);
    return *(const float4 *)(staged + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
}

// The gate and the other half that 32 rows x 32 columns of gradients meet, as
// staged_sums lays them out: eight rows a lane.
template <typename T> struct GateUp {
    Raw<T, 4> g[8], u[8];
    // (rows behind the last group are not read: they may hold anything)
    __device__ __forceinline__ void load(const TensorProduct &p, int lane, bool some, int64_t row, int rows, int c) {
        const int j = c + (lane & 7) * 4, left = p.N - j;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            const T *z = (const T *)p.gate_up + (row + r) * p.gs + j;
            const bool here = some && r < rows;
            if (here && p.whole_gate && left >= 4) {
                g[i] = load_raw<T, 4>(z);
                u[i] = load_raw<T, 4>(z + p.N);
            } else {
                uint16_t h[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[k] = here && k < left ? *(const uint16_t *)(z + k) : 0;
                    h[4 + k] = here && k < left ? *(const uint16_t *)(z + p.N + k) : 0;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    g[i].w[k] = h[2 * k] | (uint32_t)h[2 * k + 1] << 16;
                    u[i].w[k] = h[4 + 2 * k] | (uint32_t)h[5 + 2 * k] << 16;
                }
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void store_four(T *out, const float (&f)[4], int left, bool whole) {
    if (whole && left >= 4) {
        store_raw<T, 4>(out, narrow<T, 4>(f));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left) out[k] = from_f32<T>(f[k]);
    }
}

// The staged 32 rows x 32 columns of dh through the gate: [dg | du].
template <typename T>
__device__ __forceinline__ void write_gate_grad(const TensorProduct &p, const unsigned char *staged, const GateUp<T> &z,
                                                int lane, bool some, float fill, int64_t row, int rows, int c) {
    __syncwarp();
    const int j = c + (lane & 7) * 4, left = p.N - j;
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += 4) {
        float g[16], u[16], dh[16];
        Slope a[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 q = staged_sums(staged, lane, i0 + i);
            float f[4];
            widen<T, 4>(i0 == 0 ? z.g[i] : z.g[4 + i], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) g[4 * i + k] = f[k];
            widen<T, 4>(i0 == 0 ? z.u[i] : z.u[4 + i], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) u[4 * i + k] = f[k];
            dh[4 * i] = q.x; dh[4 * i + 1] = q.y; dh[4 * i + 2] = q.z; dh[4 * i + 3] = q.w;
        }
        act_slopes(p.activation, g, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (i0 + i) * 4 + (lane >> 3);
            float dg[4], du[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dg[k] = some ? dh[4 * i + k] * u[4 * i + k] * a[4 * i + k].slope : fill;
                du[k] = some ? dh[4 * i + k] * a[4 * i + k].value : fill;
            }
            if (r < rows) {
                T *out = (T *)p.out + (row + r) * p.os + j;
                store_four<T>(out, dg, left, p.whole_out);
                store_four<T>(out + p.N, du, left, p.whole_out);
            }
        }
    }
    __syncwarp();
}

// The staged 32 rows x 32 FP32 sums to `out`, added to what is there with `add`.
template <typename O>
__device__ __forceinline__ void write_weights(O *out, const TensorProduct &p, const unsigned char *staged, int lane,
                                              int rows, int cols) {
    __syncwarp();
    const int unit = lane & 7;
    const int64_t stride = p.os;
    const bool whole = p.whole_out, add = p.accumulate;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (lane >> 3);
        if (row >= rows) continue;
        const float4 q = staged_sums(staged, lane, i);
        float f[4] = {q.x, q.y, q.z, q.w};
        O *at = out + row * stride + unit * 4;
        if (whole && unit * 4 + 4 <= cols) {
            if (add) {
                float old[4];
                widen<O, 4>(load_raw<O, 4>(at), old);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] += old[k];
            }
            store_raw<O, 4>(at, narrow<O, 4>(f));
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (unit * 4 + k < cols) at[k] = from_f32<O>(add ? to_f32(at[k]) + f[k] : f[k]);
        }
    }
    __syncwarp();
}

// Tiles of 256 x 256 by a pair of CTAs, each with 128 of the rows: one TMA warp,
// one warp that issues the products of both (the first CTA's), eight that
// finish the sums, which lie in one half of TMEM while the products fill the
// other.  WEIGHTS: a third control warp for groups that end inside a step.
template <typename T, int FORM, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TC_THREADS, 1)
product_tensor_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                      const TensorProduct p) {
    extern __shared__ unsigned char dynamic[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    constexpr int STAGES = tc_stages(FORM);
    unsigned char *staging = smem + STAGES * TC_STAGE;
    TensorBars &bars = *(TensorBars *)(staging + TC_EPILOGUE * TC_STAGED);
    int *first = (int *)(&bars + 1);        // first row tile of each group, and how many there are
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;
    const uint32_t tiles0 = tc::smem_u32(smem), full = tc::smem_u32(bars.full), empty = tc::smem_u32(bars.empty),
                   sums = tc::smem_u32(bars.sums), taken = tc::smem_u32(bars.taken), tail = tc::smem_u32(bars.tail),
                   cleared = tc::smem_u32(bars.cleared);
    if (warp == 0 && lane == 0) {
        tc::prefetch_map(&amap);
        tc::prefetch_map(&bmap);
        for (int i = 0; i < STAGES; ++i) {
            tc::bar_init(full + 8 * i, 1);
            tc::bar_init(cleared + 8 * i, 1);
            tc::bar_init(empty + 8 * i, 1);
            tc::bar_init(tail + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(sums + 8 * i, 1);
            tc::bar_init(taken + 8 * i, 2 * TC_EPILOGUE);
        }
        tc::fence_bar_init();
    }
    if (warp == 1) tc::tmem_alloc2(&bars.tmem, 512);
    if (FORM != WEIGHTS && warp == 3) {
        int before = 0;
        for (int base = 0; base <= p.groups.experts; base += 32) {
            const int e = base + lane;
            int n = 0;
            if (e <= p.groups.experts) {
                const int a = group_start(p.groups, e);
                n = max(0, (e < p.groups.experts ? group_start(p.groups, e + 1) : p.groups.rows) - a);
            }
            const int tiles = (n + TC_TILE - 1) / TC_TILE;
            int sum = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, sum, o);
                if (lane >= o) sum += v;
            }
            if (e <= p.groups.experts) first[e] = before + sum - tiles;
            before += __shfl_sync(FULL, sum, 31);
        }
        if (lane == 0) first[p.groups.experts + 1] = before;
    }
    tc::fence_before();
    __syncthreads();
    cluster_arrive<true>();
    cluster_wait();
    tc::fence_after();
    launch_dependents();
    const uint32_t tmem = bars.tmem;
    const int64_t total = FORM == WEIGHTS ? (int64_t)p.groups.experts * p.slices * p.tiles_m * p.tiles_n
                                          : (int64_t)first[p.groups.experts + 1] * p.tiles_n;
    const int64_t t0 = blockIdx.x >> 1, step = gridDim.x >> 1;
    // EPI GATED: a tile is 128 columns of the gate and the same of the other half
    constexpr int WIDTH = EPI == GATED ? TC_TILE / 2 : TC_TILE;
    auto tile_at = [&](int64_t t) {
        TensorTile r = tensor_tile<FORM>(p, first, t);
        if constexpr (FORM != WEIGHTS) r.c *= WIDTH;
        return r;
    };
    bool alive = true;
    // (a branch each for the two counts of registers: code after a merge gets the fewer)
    if (warp >= TC_CONTROL) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TC_EPILOGUE_REGS));
        const int quarter = warp & 3, half = (warp - TC_CONTROL) >> 2;
        unsigned char *staged = staging + (warp - TC_CONTROL) * TC_STAGED;
        constexpr int SEGMENT = TC_SEGMENT;
        const uint32_t taken0 = tc::of_rank(taken, 0), lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        int turn = 0;
        // the next sums, or false
        auto wait_sums = [&]() {
            if (alive) alive = tc::bar_wait(sums + 8 * (turn & 1), (turn >> 1) & 1);
            alive = __all_sync(FULL, alive);
            tc::fence_after();
        };
        auto release_sums = [&]() {
            tc::fence_before();
            if (lane == 0) tc::bar_arrive_cluster(taken0 + 8 * (turn & 1));
            ++turn;
        };
        const float given_up = __int_as_float(0x7FC00000);      // NaN where products are missing
        for (int64_t t = t0; t < total; t += step) {
            const TensorTile a = tile_at(t);
            const bool some = a.s1 > a.s0;
            const int row = a.r0 + (int)rank * 128 + quarter * 32, rows = min(32, a.r1 - row);
            if constexpr (FORM == WEIGHTS) {
                if (!some && p.accumulate) continue;
                float sum[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int begin = a.s0; begin < a.s1; begin += SEGMENT) {
                    wait_sums();
                    if (alive) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v[32];
                            load_sums(v, lanes + (turn & 1) * 256 + half * 128 + i * 32, true, 0.f);
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[i][j] += v[j];
                        }
                        release_sums();
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = a.c + half * 128 + i * 32, cols = min(32, p.N - c);
                    if (!alive) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[i][j] = given_up;
                    }
                    stage_sums(staged, lane, sum[i]);
                    const int64_t slice = p.slices > 1 ? (int64_t)a.slice * p.groups.experts * p.oe : 0;
                    const int64_t at = slice + (int64_t)a.e * p.oe + (int64_t)row * p.os + c;
                    if (p.out_f32) write_weights((float *)p.out + at, p, staged, lane, rows, cols);
                    else write_weights((T *)p.out + at, p, staged, lane, rows, cols);
                }
            } else {
                if constexpr (EPI == GATE_GRAD) {
                    // a chunk's gate is loaded while the one before it is finished
                    GateUp<T> z;
                    const int c = a.c + half * 128;
                    z.load(p, lane, some, row, rows, c);
                    if (some) wait_sums();
                    const uint32_t from = lanes + (turn & 1) * 256 + half * 128;
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        float v[32];
                        load_sums(v, from + i * 32, some && alive, some ? given_up : 0.f);
                        if (i == 3 && some && alive) release_sums();
                        stage_sums(staged, lane, v);
                        GateUp<T> now = z;
                        if (i < 3) z.load(p, lane, some, row, rows, c + (i + 1) * 32);
                        write_gate_grad<T>(p, staged, now, lane, some, 0.f, row, rows, c + i * 32);
                    }
                    continue;
                }
                if (some) wait_sums();
                finish_rows<T, EPI>(p, staged, lane, lanes + (turn & 1) * 256 + half * (WIDTH / 2), some && alive,
                                    some ? given_up : 0.f, row, rows, a.c + half * (WIDTH / 2));
                if (some && alive) release_sums();
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_CONTROL_REGS));
        if (warp == 0) {
            if (lane == 0) {
                uint32_t stage = 0, phase = 0;
                const uint32_t full0 = tc::of_rank(full, 0);
                for (int64_t t = t0; t < total && alive; t += step) {
                    const TensorTile a = tile_at(t);
                    for (int s = a.s0; s < a.s1; s += TC_K) {
                        if (!tc::bar_wait(empty + 8 * stage, phase ^ 1)) {
                            alive = false;
                            break;
                        }
                        const uint32_t at = tiles0 + stage * TC_STAGE, bt = at + TC_OPERAND;
                        uint32_t bar = full0 + 8 * stage;
                        if (FORM == WEIGHTS && a.s1 - s < TC_K) {
                            // rows of the next group come along: the last warp clears them
                            bar = tail + 8 * stage;
                            tc::bar_expect(bar, TC_STAGE);
                        } else if (rank == 0) {
                            tc::bar_expect(full + 8 * stage, 2 * TC_STAGE);
                        }
                        if constexpr (FORM == WEIGHTS) {
    #pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                tc::load_box<true>(at + j * (TC_OPERAND / 2), &amap, bar, a.r0 + rank * 128 + j * 64, s, 0);
                                tc::load_box<true>(bt + j * (TC_OPERAND / 2), &bmap, bar, a.c + rank * 128 + j * 64, s, 0);
                            }
                        } else {
                            tc::load_box<true>(at, &amap, bar, s, a.r0 + rank * 128, 0);
                            if constexpr (FORM == ROWS) {
                                tc::load_box<true>(bt, &bmap, bar, s, a.c + (EPI == GATED ? rank * p.N : rank * 128), a.e);
                            } else {
    #pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    tc::load_box<true>(bt + j * (TC_OPERAND / 2), &bmap, bar, a.c + rank * 128 + j * 64, s, a.e);
                            }
                        }
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // every stage taken: nothing arrives here any more
                for (int i = 0; i < STAGES && alive; ++i) {
                    alive = tc::bar_wait(empty + 8 * stage, phase ^ 1);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == 1) {
            if (lane == 0 && rank == 0) {
                constexpr bool A_ACROSS = FORM == WEIGHTS, B_ACROSS = FORM != ROWS;
                constexpr int SEGMENT = FORM == WEIGHTS ? TC_SEGMENT : INT_MAX;
                constexpr uint32_t idesc = tc::instruction<T, A_ACROSS, B_ACROSS>(256, 256);
                uint32_t stage = 0, phase = 0;
                int turn = 0;
                for (int64_t t = t0; t < total && alive; t += step) {
                    const TensorTile a = tile_at(t);
                    if (a.s1 <= a.s0) continue;
                    for (int begin = a.s0; begin < a.s1 && alive; begin = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1, ++turn) {
                        const uint32_t acc = turn & 1;
                        const int end = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1;
                        alive = tc::bar_wait(taken + 8 * acc, ((turn >> 1) & 1) ^ 1);
                        tc::fence_after();
                        for (int s = begin; s < end && alive; s += TC_K) {
                            if (!tc::bar_wait(full + 8 * stage, phase)) {
                                alive = false;
                                break;
                            }
                            tc::fence_after();
                            const uint32_t at = tiles0 + stage * TC_STAGE, bt = at + TC_OPERAND;
    #pragma unroll
                            for (int k = 0; k < TC_K / 16; ++k)
                                if (s + 16 * k < a.s1)
                                    tc::mma2(tmem + acc * 256,
                                             tc::operand<A_ACROSS>(at + k * (A_ACROSS ? 2048 : 32), TC_OPERAND / 2),
                                             tc::operand<B_ACROSS>(bt + k * (B_ACROSS ? 2048 : 32), TC_OPERAND / 2), idesc,
                                             s > begin || k > 0);
                            tc::commit2(empty + 8 * stage);
                            if (++stage == STAGES) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                        if (alive) tc::commit2(sums + 8 * acc);
                    }
                }
            }
        } else if (FORM == WEIGHTS && warp == 2) {
            // Steps in which a group ends: rows of the next one are cleared before
            // the products read them (its infinities would reach this group's sums).
            const uint32_t cleared0 = tc::of_rank(cleared, 0);
            uint32_t chunks = 0, turns = 0;      // turns: the phase of each stage's barrier, a bit each
            for (int64_t t = t0; t < total && alive; t += step) {
                const TensorTile a = tile_at(t);
                chunks += (a.s1 - a.s0 + TC_K - 1) / TC_K;
                const int rows = (a.s1 - a.s0) % TC_K;
                if (rows == 0) continue;
                const uint32_t stage = (chunks - 1) % STAGES;
                alive = tc::bar_wait(tail + 8 * stage, (turns >> stage) & 1);
                alive = __all_sync(FULL, alive);
                if (!alive) break;
                uint4 *at = (uint4 *)(smem + stage * TC_STAGE);
                // four blocks of 64 rows of 128 bytes
                const int left = TC_K - rows;
                for (int i = lane; i < 4 * left * 8; i += 32) {
                    const int block = i / (left * 8), j = i % (left * 8);
                    at[block * (TC_OPERAND / 32) + rows * 8 + j] = make_uint4(0, 0, 0, 0);
                }
                tc::fence_smem_writes();
                __syncwarp();
                if (rank == 1) {
                    if (lane == 0) tc::bar_arrive_cluster(cleared0 + 8 * stage);
                } else {
                    alive = tc::bar_wait(cleared + 8 * stage, (turns >> stage) & 1);
                    alive = __all_sync(FULL, alive);
                    if (alive && lane == 0) tc::bar_arrive(full + 8 * stage);
                }
                turns ^= 1u << stage;
            }
        }
    }
    if (!alive) {
        if (p.status != nullptr) atomicOr(p.status + 1, TBE_FLAG_MMA_TIMEOUT);
        tc::wait_out();
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    cluster_arrive<true>();
    cluster_wait();
    tc::fence_after();
    if (warp == 1) tc::tmem_free2(tmem, 512);
    cluster_arrive<true>();
    cluster_wait();
}

// The slices' results added up, in order: a row of a weight a block and 256 * VEC columns.
template <typename O, int VEC>
__global__ void __launch_bounds__(256) product_join_kernel(const float *__restrict__ parts, const TensorProduct p) {
    const int e = blockIdx.x / p.M, row = blockIdx.x - e * p.M;
    const int c = (blockIdx.y * 256 + threadIdx.x) * VEC;
    wait_for_launch_before();
    if (c >= p.N) return;
    if (p.accumulate && group_start(p.groups, e + 1) <= group_start(p.groups, e)) return;
    const int64_t size = (int64_t)p.groups.experts * p.M * p.N;
    const float *from = parts + (int64_t)blockIdx.x * p.N + c;
    O *out = (O *)p.out + e * p.oe + row * p.os + c;
    float sum[VEC] = {};
#pragma unroll 4
    for (int i = 0; i < p.slices; ++i) {
        float f[VEC];
        widen<float, VEC>(load_raw<float, VEC>(from + i * size), f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] += f[k];
    }
    if (p.accumulate) {
        float f[VEC];
        widen<O, VEC>(load_raw<O, VEC>(out), f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum[k] += f[k];
    }
    store_raw<O, VEC>(out, narrow<O, VEC>(sum));
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

namespace tc {
bool make_map(CUtensorMap *map, const void *data, int dtype, int64_t cols, int64_t rows, int64_t depth, int64_t stride,
              int64_t depth_stride, int box_rows) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (Encode)fn;
    }();
    // rows on 16-byte boundaries that do not overlap
    if (encode == nullptr || dtype == TBE_F32 || !is_aligned(data, 16)) return false;
    if (rows <= 1) stride = (int64_t)round_up((size_t)cols, 8);
    if (depth <= 1) depth_stride = (int64_t)round_up((size_t)cols, 8);
    if (stride % 8 != 0 || depth_stride % 8 != 0 || stride < cols || depth_stride < cols || stride >= (int64_t)1 << 38 ||
        depth_stride >= (int64_t)1 << 38)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)depth_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, steps[3] = {1, 1, 1};
    return encode(map, dtype == TBE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void *>(data), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace tc

// Into how many slices the rows of the groups are cut when the weights have few
// tiles for the device's 76 pairs: the number with the least time by tiles at 512
// cycles a step of 64 rows and 3000 a tile, and the parts, written and read, at
// 3 KB a cycle.  At least 512 rows a slice.
static int weight_slices(int64_t rows, int64_t experts, int64_t N, int64_t K) {
    const int64_t tiles = experts * ((N + TC_TILE - 1) / TC_TILE) * ((K + TC_TILE - 1) / TC_TILE), pairs = 76;
    if (tiles >= 4 * pairs) return 1;
    int best = 1;
    double least = 0;
    for (int s = 1; s <= 32 && (s == 1 || rows / (experts * s) >= 512); ++s) {
        const double steps = (double)((rows / experts + s - 1) / s + TC_K - 1) / TC_K;
        const double time = (double)((tiles * s + pairs - 1) / pairs) * (steps * 512 + 3000) +
                            (s > 1 ? 6000 + (double)s * experts * N * K * 8 / 3000 : 0);
        if (s == 1 || time < least) {
            best = s;
            least = time;
        }
    }
    return best;
}

static bool whole_rows(const void *p, int64_t stride, int64_t more, int bytes) {
    return is_aligned(p, 16) && stride * bytes % 16 == 0 && more * bytes % 16 == 0;
}

template <typename T, int FORM, int EPI>
static void launch_tensor(Launch &L, const char *name, const CUtensorMap &a, const CUtensorMap &b, TensorProduct &p) {
    constexpr int WIDTH = EPI == GATED ? TC_TILE / 2 : TC_TILE;
    p.tiles_m = (p.M + TC_TILE - 1) / TC_TILE;
    p.tiles_n = (p.N + WIDTH - 1) / WIDTH;
    const int64_t groups = p.groups.experts + 1 < p.groups.rows ? p.groups.experts + 1 : p.groups.rows;
    const int64_t most = FORM == WEIGHTS ? (int64_t)p.groups.experts * p.slices * p.tiles_m * p.tiles_n
                                         : ((int64_t)p.groups.rows / TC_TILE + groups) * p.tiles_n;
    int64_t pairs = L.num_sms / 2 > 0 ? L.num_sms / 2 : 1;
    if (pairs > most) pairs = most;
    auto *fn = product_tensor_kernel<T, FORM, EPI>;
    // one size whatever the number of experts: a kernel's limit is set once
    const size_t smem = 1024 + (size_t)tc_stages(FORM) * TC_STAGE + TC_EPILOGUE * TC_STAGED + sizeof(TensorBars) +
                        (FORM == WEIGHTS ? 0 : (size_t)(PRODUCT_MOST_EXPERTS + 2) * 4);
    cached_smem_attr(L.dev, (const void *)fn, smem);
    L.before(name);
    fn<<<(unsigned)(2 * pairs), TC_THREADS, smem, L.stream>>>(a, b, p);
    L.after();
}

#define TBE_HALF_SWITCH(dtype, ...)                                            \
    do {                                                                       \
        if ((dtype) == TBE_F16) { using T = __half; __VA_ARGS__; }             \
        else { using T = __nv_bfloat16; __VA_ARGS__; }                         \
    } while (0)

// The product on the tensor cores where TMA takes both operands; false: it does not.
template <int FORM, int EPI>
static bool run_tensor(Launch &L, const tbe_matrix *x, const tbe_experts *w, const tbe_matrix *out,
                       const tbe_matrix *gate_up, int activation, int32_t *status, const Groups &groups) {
    CUtensorMap a, b;
    if (!tc::make_map(&a, x->data, x->dtype, x->cols, x->rows, 1, x->stride, 0, 128) ||
        !tc::make_map(&b, w->data, w->dtype, w->cols, w->rows, w->experts, w->stride, w->expert_stride,
                      FORM == ROWS ? 128 : 64))
        return false;
    TensorProduct p = {};
    p.out = out->data;
    p.os = out->stride;
    p.gate_up = gate_up != nullptr ? gate_up->data : nullptr;
    p.gs = gate_up != nullptr ? gate_up->stride : 0;
    p.N = (int)(FORM == ROWS ? (EPI == GATED ? w->rows / 2 : w->rows) : w->cols);
    p.K = (int)(FORM == ROWS ? w->cols : w->rows);
    p.activation = activation;
    // (the gate's gradient: rows and halves of 8-byte vectors)
    const int64_t second = EPI == GATE_GRAD ? p.N : 0;
    p.whole_out = whole_rows(out->data, out->stride, second, EPI == GATE_GRAD ? 4 : 2);
    p.whole_gate = gate_up != nullptr && whole_rows(gate_up->data, gate_up->stride, second, EPI == GATE_GRAD ? 4 : 2);
    p.status = status;
    p.groups = groups;
    TBE_HALF_SWITCH(x->dtype, (launch_tensor<T, FORM, EPI>(L, "tbe_product_tensor", a, b, p)));
    return true;
}

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
        if (!run_tensor<ROWS, GATED>(L, rows, weight, hidden, gate_up, activation, dev_status, p.groups))
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
        if (!run_tensor<ROWS, STORE>(L, rows, weight, out, nullptr, 0, dev_status, p.groups))
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
        if (gate_up != nullptr) {
            if (!run_tensor<ROWS_GRAD, GATE_GRAD>(L, grad_out, weight, grad_rows, gate_up, activation, dev_status, p.groups))
                run_rows<GATE_GRAD>(L, grad_out->dtype, p);
        } else if (!run_tensor<ROWS_GRAD, STORE>(L, grad_out, weight, grad_rows, nullptr, 0, dev_status, p.groups)) {
            run_rows<STORE>(L, grad_out->dtype, p);
        }
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

size_t tbe_expert_workspace_bytes(int64_t rows, int64_t experts, int64_t N, int64_t K) {
    if (rows < 0 || rows >= TOKEN_MAX_ROWS || experts < 1 || experts > PRODUCT_MOST_EXPERTS || N < 1 ||
        N > TOKEN_MAX_COLS || K < 1 || K > TOKEN_MAX_COLS)
        return 0;
    const int slices = weight_slices(rows, experts, N, K);
    return slices > 1 ? (size_t)slices * experts * N * K * 4 : 0;
}

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
        CUtensorMap a, b;
        if (rows->rows > 0 && tc::make_map(&a, grad_out->data, rows->dtype, grad_out->cols, rows->rows, 1, grad_out->stride, 0, 64) &&
            tc::make_map(&b, rows->data, rows->dtype, rows->cols, rows->rows, 1, rows->stride, 0, 64)) {
            TensorProduct q = {};
            q.out = p.out;
            q.os = p.os;
            q.oe = p.oe;
            q.M = p.N;
            q.N = p.K;
            q.accumulate = accumulate;
            q.out_f32 = p.out_f32;
            q.whole_out = whole_rows(p.out, p.os, grad_weight->experts > 1 ? p.oe : 0, p.out_f32 ? 4 : 2);
            q.status = dev_status;
            q.groups = p.groups;
            q.slices = weight_slices(rows->rows, grad_weight->experts, q.M, q.N);
            TensorProduct part = q;
            if (q.slices > 1) {
                part.out = workspace;
                part.os = q.N;
                part.oe = (int64_t)q.M * q.N;
                part.accumulate = 0;
                part.out_f32 = 1;
                part.whole_out = q.N % 4 == 0;
            }
            TBE_HALF_SWITCH(rows->dtype, (launch_tensor<T, WEIGHTS, STORE>(L, "tbe_product_tensor_weights", a, b, part)));
            if (q.slices > 1) {
                const bool whole = q.whole_out && q.N % 4 == 0;
                const dim3 grid((unsigned)(grad_weight->experts * q.M), (unsigned)((q.N + (whole ? 1023 : 255)) / (whole ? 1024 : 256)));
                TBE_TYPE_SWITCH(grad_weight->dtype, {
                    auto *fn = whole ? product_join_kernel<T, 4> : product_join_kernel<T, 1>;
                    launch_with(L, "tbe_product_join", true, 1, fn, grid, 256, 0, (const float *)workspace, q);
                });
            }
            return L.failed ? TBE_ERR_CUDA : TBE_OK;
        }
        const dim3 grid((unsigned)((p.K + SIMPLE_TILE - 1) / SIMPLE_TILE), (unsigned)((p.N + SIMPLE_TILE - 1) / SIMPLE_TILE),
                        (unsigned)grad_weight->experts);
        L.before("tbe_product_weights");
        TBE_TYPE_SWITCH(rows->dtype, (product_weights_simple_kernel<T><<<grid, 256, 0, L.stream>>>(p)));
        L.after();
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
