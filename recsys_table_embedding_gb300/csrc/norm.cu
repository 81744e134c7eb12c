// Layer norm of rows, and its gradients.
//
//   out = (x - mu) r w + b,   r = 1 / sqrt(var + eps)
//   with d = dy w, h = (x - mu) r:
//   dx = r (d - mean(d) - h mean(d h)),   dw = sum_n dy h,   db = sum_n dy
//
// Every element is used a few times and read once: HBM bounds both passes.  A
// row lies in the registers of a warp, or of a block where a warp's do not
// hold it, between the pass that sums and the pass that writes.
#include "token_internal.cuh"

namespace tbe {

#ifndef TBE_NORM_FWD_NV
#define TBE_NORM_FWD_NV 4
#endif
#ifndef TBE_NORM_RING
#define TBE_NORM_RING 3
#endif
// Elements a thread holds: of a row in the forward pass; of a row of x, one of
// dy, a weight and the two sums in the backward pass.
constexpr int FWD_THREADS = 1024, BWD_THREADS = 512;
// Rows that the backward pass has under way beside the one it works on.
constexpr int BWD_RING = TBE_NORM_RING;

// A 16-byte copy to shared memory, and waiting for all but the latest N groups of them.
__device__ __forceinline__ void copy16(uint4 *shared, const void *global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(shared)), "l"(global)
                 : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A parameter vector of any of the three types; its vectors are read whole
// where it is aligned for them.
struct Param {
    const void *p;      // nullptr: `fill` everywhere
    int dtype;
    int whole;
    float fill;
};

template <int VEC>
__device__ __forceinline__ void load_param(const Param &w, int64_t i, float (&f)[VEC]) {
    if (w.p == nullptr) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = w.fill;
    } else if (!w.whole) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = load_f32(w.p, w.dtype, i + k);
    } else if (w.dtype == TBE_F32) {
        widen<float, VEC>(load_raw<float, VEC>((const float *)w.p + i), f);
    } else if (w.dtype == TBE_F16) {
        widen<__half, VEC>(load_raw<__half, VEC>((const __half *)w.p + i), f);
    } else {
        widen<__nv_bfloat16, VEC>(load_raw<__nv_bfloat16, VEC>((const __nv_bfloat16 *)w.p + i), f);
    }
}

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(FULL, v.x, o);
        v.y += __shfl_xor_sync(FULL, v.y, o);
    }
    return v;
}

// Sum over the threads of a row: a warp, or (BLOCK) the block.  `part`: 32
// words that no thread still reads from an earlier sum; every thread gets the
// same sum, added in the same order.
template <bool BLOCK> __device__ __forceinline__ float2 row_sum2(float2 v, float2 *part) {
    v = warp_sum2(v);
    if constexpr (BLOCK) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = warp_sum2(lane < (int)(blockDim.x >> 5) ? part[lane] : make_float2(0.f, 0.f));
    }
    return v;
}

// ---------------------------------------------------------------------------
// forward

// A thread's NV vectors of its row.  The mean is corrected by the mean distance
// from it, so that rows with an offset far above their spread lose nothing to
// the first sum's rounding.
template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? FWD_THREADS : 256)
layer_norm_fwd_kernel(const T *__restrict__ x, int64_t xs, Param w, Param b, float eps, int64_t rows, int vectors,
                      T *__restrict__ out, int64_t os, float *mean, float *rstd) {
    __shared__ float2 part[2][32];
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31, lanes = BLOCK ? blockDim.x : 32;
    const int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= rows) return;
    Raw<T, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (v < vectors) raw[i] = load_raw<T, VEC, true>(x + row * xs + (int64_t)v * VEC);
    }
    const float n = (float)((int64_t)vectors * VEC);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * lanes < vectors) {
            float f[VEC];
            widen<T, VEC>(raw[i], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) s.x += f[k];
        }
    }
    const float m = row_sum2<BLOCK>(s, part[0]).x / n;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * lanes < vectors) {
            float f[VEC];
            widen<T, VEC>(raw[i], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float c = f[k] - m;
                s.x += c;
                s.y = fmaf(c, c, s.y);
            }
        }
    }
    s = row_sum2<BLOCK>(s, part[1]);
    const float e = s.x / n, var = fmaxf(s.y / n - e * e, 0.f);
    // (a NaN in the row: fmaxf would drop it)
    const float r = s.y == s.y ? 1.0f / sqrtf(var + eps) : s.y;
    if (lane == 0) {
        if (mean != nullptr) mean[row] = m + e;
        if (rstd != nullptr) rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (v < vectors) {
            float f[VEC], g[VEC], o[VEC];
            widen<T, VEC>(raw[i], f);
            load_param<VEC>(w, (int64_t)v * VEC, g);
            load_param<VEC>(b, (int64_t)v * VEC, o);
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = fmaf(((f[k] - m) - e) * r, g[k], o[k]);
            store_raw<T, VEC>(out + row * os + (int64_t)v * VEC, narrow<T, VEC>(o));
        }
    }
}

// Rows that a block's registers do not hold: read three times, the last two
// from L2.
template <typename T, int VEC>
__global__ void __launch_bounds__(FWD_THREADS)
layer_norm_fwd_long_kernel(const T *__restrict__ x, int64_t xs, Param w, Param b, float eps, int vectors,
                           T *__restrict__ out, int64_t os, float *mean, float *rstd) {
    __shared__ float2 part[2][32];
    const int64_t row = blockIdx.x;
    const T *p = x + row * xs;
    const float n = (float)((int64_t)vectors * VEC);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int v = threadIdx.x; v < vectors; v += FWD_THREADS) {
        float f[VEC];
        widen<T, VEC>(load_raw<T, VEC>(p + (int64_t)v * VEC), f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) s.x += f[k];
    }
    const float m = row_sum2<true>(s, part[0]).x / n;
    s = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int v = threadIdx.x; v < vectors; v += FWD_THREADS) {
        float f[VEC];
        widen<T, VEC>(load_raw<T, VEC>(p + (int64_t)v * VEC), f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float c = f[k] - m;
            s.x += c;
            s.y = fmaf(c, c, s.y);
        }
    }
    s = row_sum2<true>(s, part[1]);
    const float e = s.x / n, var = fmaxf(s.y / n - e * e, 0.f);
    const float r = s.y == s.y ? 1.0f / sqrtf(var + eps) : s.y;
    if (threadIdx.x == 0) {
        if (mean != nullptr) mean[row] = m + e;
        if (rstd != nullptr) rstd[row] = r;
    }
    for (int v = threadIdx.x; v < vectors; v += FWD_THREADS) {
        float f[VEC], g[VEC], o[VEC];
        widen<T, VEC>(load_raw<T, VEC, true>(p + (int64_t)v * VEC), f);
        load_param<VEC>(w, (int64_t)v * VEC, g);
        load_param<VEC>(b, (int64_t)v * VEC, o);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = fmaf(((f[k] - m) - e) * r, g[k], o[k]);
        store_raw<T, VEC>(out + row * os + (int64_t)v * VEC, narrow<T, VEC>(o));
    }
}

// ---------------------------------------------------------------------------
// backward

// Where a block's sums of dy h and dy over its rows go: row `part` of the
// workspace [parts][2][D], or (direct: the grid's only block) the gradients.
struct GradSums {
    float *parts;
    void *dw, *db;
    int dtype;
    int direct;
    int64_t cols;
};

__device__ __forceinline__ void store_sums(const GradSums &g, int64_t part, int64_t col, float dw, float db) {
    if (g.direct) {
        if (g.dw != nullptr) store_f32(g.dw, g.dtype, col, dw);
        if (g.db != nullptr) store_f32(g.db, g.dtype, col, db);
    } else {
        float *p = g.parts + part * 2 * g.cols + col;
        p[0] = dw;
        p[g.cols] = db;
    }
}

// The rows' gradient and the block's part of the sums, rows in steps of the
// grid: a thread keeps its columns' sums in registers over its rows.  Rows of
// 16-byte vectors come through shared memory, each thread's vectors in places
// that it alone reads and writes, so that several rows are under way without
// registers or a barrier for them; others are loaded a row ahead.
template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? BWD_THREADS : 256)
layer_norm_bwd_kernel(const T *__restrict__ dy, int64_t ds, const T *__restrict__ x, int64_t xs, Param w,
                      const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int vectors,
                      T *__restrict__ dx, int64_t os, GradSums g) {
    constexpr bool RING = VEC * sizeof(T) == 16;
    __shared__ float2 part[2][32];
    extern __shared__ uint4 ring[];     // RING: [BWD_RING][2 NV][threads]; then warps of rows: sums [2][D]
    launch_dependents();
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31, lanes = BLOCK ? blockDim.x : 32;
    const int64_t step = BLOCK ? (int64_t)gridDim.x : (int64_t)gridDim.x * warps;
    const float n = (float)((int64_t)vectors * VEC);
    float wt[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) aw[i][k] = ab[i][k] = wt[i][k] = 0.f;
        if (lane + i * lanes < vectors) load_param<VEC>(w, (int64_t)(lane + i * lanes) * VEC, wt[i]);
    }
    Raw<T, VEC> rx[NV], ry[NV];
    auto place = [&](int stage, int i) { return ring + (stage * 2 * NV + i) * blockDim.x + threadIdx.x; };
    auto load = [&](int64_t row, int stage) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors && row < rows) {
                const T *px = x + row * xs + (int64_t)v * VEC, *py = dy + row * ds + (int64_t)v * VEC;
                if constexpr (RING) {
                    copy16(place(stage, 2 * i), px);
                    copy16(place(stage, 2 * i + 1), py);
                } else {
                    rx[i] = load_raw<T, VEC, true>(px);
                    ry[i] = load_raw<T, VEC, true>(py);
                }
            }
        }
        if constexpr (RING) copies_issued();
    };
    int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    for (int i = 0; i < (RING ? BWD_RING : 1); ++i) load(row + i * step, i);
    float mu = row < rows ? __ldg(mean + row) : 0.f, r = row < rows ? __ldg(rstd + row) : 0.f;
    int turn = 0, stage = 0;
    for (; row < rows; row += step, turn ^= 1) {
        if constexpr (RING) {
            copies_wait<BWD_RING - 1>();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint4 a = *place(stage, 2 * i), b = *place(stage, 2 * i + 1);
                rx[i].w[0] = a.x; rx[i].w[1] = a.y; rx[i].w[2] = a.z; rx[i].w[3] = a.w;
                ry[i].w[0] = b.x; ry[i].w[1] = b.y; ry[i].w[2] = b.z; ry[i].w[3] = b.w;
            }
        }
        float h[NV][VEC], d[NV][VEC];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * lanes < vectors) {
                widen<T, VEC>(rx[i], h[i]);
                widen<T, VEC>(ry[i], d[i]);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    h[i][k] = (h[i][k] - mu) * r;
                    aw[i][k] = fmaf(d[i][k], h[i][k], aw[i][k]);
                    ab[i][k] += d[i][k];
                    d[i][k] *= wt[i][k];
                    s.x += d[i][k];
                    s.y = fmaf(d[i][k], h[i][k], s.y);
                }
            }
        }
        const float r_now = r;
        if (row + step < rows) {
            mu = __ldg(mean + row + step);
            r = __ldg(rstd + row + step);
        }
        if constexpr (!RING) load(row + step, 0);
        s = row_sum2<BLOCK>(s, part[turn]);
        if constexpr (RING) {
            // (the stage's vectors have been used: the sum depends on them)
            load(row + BWD_RING * step, stage);
            stage = stage + 1 == BWD_RING ? 0 : stage + 1;
        }
        if (dx != nullptr) {
            const float s1 = s.x / n, s2 = s.y / n;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + i * lanes;
                if (v < vectors) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) d[i][k] = r_now * ((d[i][k] - s1) - h[i][k] * s2);
                    store_raw<T, VEC>(dx + row * os + (int64_t)v * VEC, narrow<T, VEC>(d[i]));
                }
            }
        }
    }
    if constexpr (RING) copies_wait<0>();
    if (g.dw == nullptr && g.db == nullptr) return;
    if constexpr (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    store_sums(g, blockIdx.x, (int64_t)v * VEC + k, aw[i][k], ab[i][k]);
            }
        }
    } else {
        // the warps' sums one after the other
        float *sums = (float *)(ring + (RING ? BWD_RING * 2 * NV * blockDim.x : 0));
        for (int t = 0; t < warps; ++t) {
            if (warp == t) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = lane + i * lanes;
                    if (v < vectors) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            float *p = sums + v * VEC + k;
                            p[0] = t == 0 ? aw[i][k] : p[0] + aw[i][k];
                            p[g.cols] = t == 0 ? ab[i][k] : p[g.cols] + ab[i][k];
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < g.cols; c += blockDim.x)
            store_sums(g, blockIdx.x, c, sums[c], sums[g.cols + c]);
    }
}

// Long rows: the rows' gradient, each row read twice (the second time from L2) ...
template <typename T, int VEC>
__global__ void __launch_bounds__(BWD_THREADS)
layer_norm_bwd_long_kernel(const T *__restrict__ dy, int64_t ds, const T *__restrict__ x, int64_t xs, Param w,
                           const float *__restrict__ mean, const float *__restrict__ rstd, int vectors,
                           T *__restrict__ dx, int64_t os) {
    __shared__ float2 part[32];
    const int64_t row = blockIdx.x;
    const float n = (float)((int64_t)vectors * VEC), mu = __ldg(mean + row), r = __ldg(rstd + row);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int v = threadIdx.x; v < vectors; v += BWD_THREADS) {
        float h[VEC], d[VEC], wt[VEC];
        widen<T, VEC>(load_raw<T, VEC>(x + row * xs + (int64_t)v * VEC), h);
        widen<T, VEC>(load_raw<T, VEC>(dy + row * ds + (int64_t)v * VEC), d);
        load_param<VEC>(w, (int64_t)v * VEC, wt);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            const float t = d[k] * wt[k];
            s.x += t;
            s.y = fmaf(t, (h[k] - mu) * r, s.y);
        }
    }
    s = row_sum2<true>(s, part);
    const float s1 = s.x / n, s2 = s.y / n;
#pragma unroll 2
    for (int v = threadIdx.x; v < vectors; v += BWD_THREADS) {
        float h[VEC], d[VEC], wt[VEC];
        widen<T, VEC>(load_raw<T, VEC>(x + row * xs + (int64_t)v * VEC), h);
        widen<T, VEC>(load_raw<T, VEC>(dy + row * ds + (int64_t)v * VEC), d);
        load_param<VEC>(w, (int64_t)v * VEC, wt);
#pragma unroll
        for (int k = 0; k < VEC; ++k) d[k] = r * ((d[k] * wt[k] - s1) - (h[k] - mu) * r * s2);
        store_raw<T, VEC>(dx + row * os + (int64_t)v * VEC, narrow<T, VEC>(d));
    }
}

// ... and the sums over the rows of a part, a strip of 32 vectors a block.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
layer_norm_bwd_columns_kernel(const T *__restrict__ dy, int64_t ds, const T *__restrict__ x, int64_t xs,
                              const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows,
                              int vectors, GradSums g) {
    __shared__ float sums[8][32][2 * VEC + 1];
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, v = blockIdx.x * 32 + lane;
    float aw[VEC] = {}, ab[VEC] = {};
    if (v < vectors) {
#pragma unroll 4
        for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < rows; row += (int64_t)gridDim.y * 8) {
            float h[VEC], d[VEC];
            widen<T, VEC>(load_raw<T, VEC>(x + row * xs + (int64_t)v * VEC), h);
            widen<T, VEC>(load_raw<T, VEC>(dy + row * ds + (int64_t)v * VEC), d);
            const float mu = __ldg(mean + row), r = __ldg(rstd + row);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                aw[k] = fmaf(d[k], (h[k] - mu) * r, aw[k]);
                ab[k] += d[k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        sums[warp][lane][k] = aw[k];
        sums[warp][lane][VEC + k] = ab[k];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * VEC; i += 256) {
        const int l = i / VEC, k = i % VEC;
        if (blockIdx.x * 32 + l >= vectors) continue;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            a += sums[t][l][k];
            b += sums[t][l][VEC + k];
        }
        store_sums(g, blockIdx.y, (int64_t)(blockIdx.x * 32 + l) * VEC + k, a, b);
    }
}

// The parts' sums added up: 32 columns a block, the parts over eight warps.
__global__ void __launch_bounds__(256) layer_norm_bwd_join_kernel(GradSums g, int parts) {
    __shared__ float sums[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    wait_for_launch_before();
    float a = 0.f;
    if (col < g.cols) {
#pragma unroll 8
        for (int p = warp; p < parts; p += 8) a += g.parts[((int64_t)p * 2 + which) * g.cols + col];
    }
    sums[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && col < g.cols) {
        a = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) a += sums[t][lane];
        void *out = which == 0 ? g.dw : g.db;
        if (out != nullptr) store_f32(out, g.dtype, col, a);
    }
}

// ---------------------------------------------------------------------------
// host

// Calls fn with T and VEC for the matrices' type and alignment.
#define TBE_NORM_SWITCH(dtype, vec, ...)                                                  \
    do {                                                                                  \
        if ((dtype) == TBE_F32) {                                                         \
            using T = float;                                                              \
            if ((vec) >= 4) { constexpr int VEC = 4; __VA_ARGS__; }                       \
            else { constexpr int VEC = 1; __VA_ARGS__; }                                  \
        } else if ((dtype) == TBE_F16) {                                                  \
            using T = __half;                                                             \
            if ((vec) == 8) { constexpr int VEC = 8; __VA_ARGS__; }                       \
            else if ((vec) >= 2) { constexpr int VEC = 2; __VA_ARGS__; }                  \
            else { constexpr int VEC = 1; __VA_ARGS__; }                                  \
        } else {                                                                          \
            using T = __nv_bfloat16;                                                      \
            if ((vec) == 8) { constexpr int VEC = 8; __VA_ARGS__; }                       \
            else if ((vec) >= 2) { constexpr int VEC = 2; __VA_ARGS__; }                  \
            else { constexpr int VEC = 1; __VA_ARGS__; }                                  \
        }                                                                                 \
    } while (0)

// The vector that TBE_NORM_SWITCH instantiates for one of vector_of.
static int norm_vector(int dtype, int vec) {
    if (dtype == TBE_F32) return vec >= 4 ? 4 : 1;
    return vec == 8 ? 8 : vec >= 2 ? 2 : 1;
}

static Param param(const void *p, int dtype, int vec, float fill) {
    const size_t bytes = (size_t)vec * dtype_bytes(dtype);
    return Param{p, dtype, is_aligned(p, bytes < 16 ? bytes : 16), fill};
}

static tbe_status check_param(const void *p, int dtype) {
    if (p == nullptr) return TBE_OK;
    if (!known_dtype(dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    return is_aligned(p, dtype_bytes(dtype)) ? TBE_OK : TBE_ERR_MISALIGNED;
}

static tbe_status check_rows(const tbe_matrix *a, const tbe_matrix *b, bool b_written) {
    tbe_status st = check_matrix(a, false);
    if (st == TBE_OK) st = check_matrix(b, b_written);
    if (st != TBE_OK) return st;
    if (a->rows != b->rows || a->cols != b->cols || a->cols > TOKEN_MAX_COLS || a->rows >= TOKEN_MAX_ROWS)
        return TBE_ERR_INVALID_ARGUMENT;
    return a->dtype == b->dtype ? TBE_OK : TBE_ERR_UNSUPPORTED_DTYPE;
}

// Parts of the sums over the rows: a block's each, 32 MB of them at most.
constexpr int64_t NORM_PARTS = 608, NORM_PART_FLOATS = (int64_t)1 << 22;
static int64_t norm_parts(int64_t rows, int64_t cols) {
    int64_t most = NORM_PART_FLOATS / cols;
    if (most > NORM_PARTS) most = NORM_PARTS;
    if (most > rows) most = rows;
    return most > 1 ? most : 1;
}

template <typename T, int VEC, int NV, bool BLOCK>
static void launch_fwd(Launch &L, int threads, const tbe_matrix *x, Param w, Param b, float eps, const tbe_matrix *out,
                       float *mean, float *rstd, int vectors) {
    const int64_t blocks = BLOCK ? x->rows : (x->rows + threads / 32 - 1) / (threads / 32);
    layer_norm_fwd_kernel<T, VEC, NV, BLOCK><<<(unsigned)blocks, threads, 0, L.stream>>>(
        (const T *)x->data, x->stride, w, b, eps, x->rows, vectors, (T *)out->data, out->stride, mean, rstd);
}

template <typename T, int VEC>
static void run_fwd(Launch &L, const tbe_matrix *x, const void *weight, const void *bias, int weight_dtype, float eps,
                    const tbe_matrix *out, float *mean, float *rstd) {
    constexpr int MOST = VEC == 8 ? 4 : 16 / VEC;      // vectors a thread
    const int vectors = (int)(x->cols / VEC);
    const Param w = param(weight, weight_dtype, VEC, 1.f), b = param(bias, weight_dtype, VEC, 0.f);
    L.before("tbe_layer_norm_fwd");
    if (vectors <= 32 * MOST && (x->rows >= 4 * L.num_sms || vectors <= 32)) {
        // a warp a row
        if (vectors <= 32) launch_fwd<T, VEC, 1, false>(L, 256, x, w, b, eps, out, mean, rstd, vectors);
        else if (vectors <= 64) launch_fwd<T, VEC, 2, false>(L, 256, x, w, b, eps, out, mean, rstd, vectors);
        else launch_fwd<T, VEC, MOST, false>(L, 256, x, w, b, eps, out, mean, rstd, vectors);
    } else if (vectors <= FWD_THREADS * MOST) {
        // a block a row: as few vectors a thread as the block's size allows
        const int nv = TBE_NORM_FWD_NV == 1 ? (vectors <= FWD_THREADS / 2 ? 1 : vectors <= FWD_THREADS ? 2 : MOST)
                     : TBE_NORM_FWD_NV == 2 ? (vectors <= 2 * 512 ? 2 : MOST) : MOST;
        const int threads = ((vectors + nv - 1) / nv + 31) / 32 * 32;
        if (nv == 1) launch_fwd<T, VEC, 1, true>(L, threads, x, w, b, eps, out, mean, rstd, vectors);
        else if (nv == 2) launch_fwd<T, VEC, 2, true>(L, threads, x, w, b, eps, out, mean, rstd, vectors);
        else launch_fwd<T, VEC, MOST, true>(L, threads, x, w, b, eps, out, mean, rstd, vectors);
    } else {
        layer_norm_fwd_long_kernel<T, VEC><<<(unsigned)x->rows, FWD_THREADS, 0, L.stream>>>(
            (const T *)x->data, x->stride, w, b, eps, vectors, (T *)out->data, out->stride, mean, rstd);
    }
    L.after();
}

template <typename T, int VEC, int NV, bool BLOCK>
static int64_t launch_bwd(Launch &L, int threads, const tbe_matrix *dy, const tbe_matrix *x, Param w, const float *mean,
                          const float *rstd, const tbe_matrix *dx, GradSums g, int vectors) {
    auto *fn = layer_norm_bwd_kernel<T, VEC, NV, BLOCK>;
    const int rows_a_block = BLOCK ? 1 : threads / 32;
    const size_t ring = VEC * sizeof(T) == 16 ? (size_t)BWD_RING * 2 * NV * threads * 16 : 0;
    const size_t smem = ring + (BLOCK ? 0 : (size_t)g.cols * 8);
    // the limit of the widest call: one size a kernel
    if (ring > 0)
        cached_smem_attr(L.dev, (const void *)fn,
                         (size_t)BWD_RING * 2 * NV * (BLOCK ? BWD_THREADS : 256) * 16 + (BLOCK ? 0 : 4096));
    int64_t blocks = (int64_t)cached_blocks_per_sm(L.dev, (const void *)fn, threads, smem) * L.num_sms;
    const int64_t most = (x->rows + rows_a_block - 1) / rows_a_block, parts = norm_parts(x->rows, x->cols);
    if (blocks > most) blocks = most;
    if (blocks > parts || blocks < 1) blocks = parts;
    g.direct = blocks == 1;
    fn<<<(unsigned)blocks, threads, smem, L.stream>>>(
        (const T *)dy->data, dy->stride, (const T *)x->data, x->stride, w, mean, rstd, x->rows, vectors,
        dx != nullptr ? (T *)dx->data : nullptr, dx != nullptr ? dx->stride : 0, g);
    return blocks;
}

template <typename T, int VEC>
static void run_bwd(Launch &L, const tbe_matrix *dy, const tbe_matrix *x, const void *weight, int weight_dtype,
                    const float *mean, const float *rstd, const tbe_matrix *dx, GradSums g) {
    constexpr int MOST = 16 / VEC, LESS = MOST / 2 > 0 ? MOST / 2 : 1;      // vectors a thread
    const int vectors = (int)(x->cols / VEC);
    const Param w = param(weight, weight_dtype, VEC, 1.f);
    const bool sums = g.dw != nullptr || g.db != nullptr;
    int64_t parts;
    if (vectors <= BWD_THREADS * MOST) {
        L.before("tbe_layer_norm_bwd");
        if (vectors <= 32 * LESS) {
            parts = launch_bwd<T, VEC, LESS, false>(L, 256, dy, x, w, mean, rstd, dx, g, vectors);
        } else if (vectors <= 32 * MOST) {
            parts = launch_bwd<T, VEC, MOST, false>(L, 256, dy, x, w, mean, rstd, dx, g, vectors);
        } else if (vectors <= 256 * LESS) {
            const int threads = ((vectors + LESS - 1) / LESS + 31) / 32 * 32;
            parts = launch_bwd<T, VEC, LESS, true>(L, threads, dy, x, w, mean, rstd, dx, g, vectors);
        } else {
            const int threads = ((vectors + MOST - 1) / MOST + 31) / 32 * 32;
            parts = launch_bwd<T, VEC, MOST, true>(L, threads, dy, x, w, mean, rstd, dx, g, vectors);
        }
        L.after();
    } else {
        if (dx != nullptr) {
            L.before("tbe_layer_norm_bwd_long");
            layer_norm_bwd_long_kernel<T, VEC><<<(unsigned)x->rows, BWD_THREADS, 0, L.stream>>>(
                (const T *)dy->data, dy->stride, (const T *)x->data, x->stride, w, mean, rstd, vectors, (T *)dx->data,
                dx->stride);
            L.after();
        }
        if (!sums) return;
        const int64_t strips = (vectors + 31) / 32;
        parts = norm_parts((x->rows + 31) / 32, x->cols);
        const int64_t enough = (8 * L.num_sms + strips - 1) / strips;
        if (parts > enough) parts = enough;
        g.direct = parts == 1;
        L.before("tbe_layer_norm_bwd_columns");
        layer_norm_bwd_columns_kernel<T, VEC><<<dim3((unsigned)strips, (unsigned)parts), 256, 0, L.stream>>>(
            (const T *)dy->data, dy->stride, (const T *)x->data, x->stride, mean, rstd, x->rows, vectors, g);
        L.after();
    }
    if (sums && parts > 1)
        launch_with(L, "tbe_layer_norm_bwd_join", true, 1, layer_norm_bwd_join_kernel,
                    dim3((unsigned)((x->cols + 31) / 32), 2), 256, 0, g, (int)parts);
}

}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_layer_norm_forward(const tbe_matrix *x, const void *weight, const void *bias, int32_t weight_dtype,
                                  float eps, const tbe_matrix *out, float *mean, float *rstd, const tbe_config *cfg,
                                  cudaStream_t stream) {
    tbe_status st = check_rows(x, out, true);
    if (st == TBE_OK) st = check_param(weight, weight_dtype);
    if (st == TBE_OK) st = check_param(bias, weight_dtype);
    if (st == TBE_OK && !(eps >= 0.f && eps <= 3e38f)) st = TBE_ERR_INVALID_ARGUMENT;
    if (st == TBE_OK && !(is_aligned(mean, 4) && is_aligned(rstd, 4))) st = TBE_ERR_MISALIGNED;
    if (st != TBE_OK || x->rows == 0) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const tbe_matrix *ms[2] = {x, out};
        const int vec = norm_vector(x->dtype, vector_of(x->dtype == TBE_F32 ? 4 : 8, x->cols, ms, 2));
        TBE_NORM_SWITCH(x->dtype, vec, (run_fwd<T, VEC>(L, x, weight, bias, weight_dtype, eps, out, mean, rstd)));
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

size_t tbe_layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || cols > TOKEN_MAX_COLS || rows >= TOKEN_MAX_ROWS) return 0;
    const int64_t parts = norm_parts(rows, cols);
    return parts > 1 ? (size_t)(parts * 2 * cols * 4) : 0;
}

tbe_status tbe_layer_norm_backward(const tbe_matrix *grad_out, const tbe_matrix *x, const void *weight,
                                   int32_t weight_dtype, const float *mean, const float *rstd,
                                   const tbe_matrix *grad_x, void *grad_weight, void *grad_bias,
                                   int32_t grad_weight_dtype, void *workspace, size_t workspace_bytes,
                                   const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_rows(grad_out, x, false);
    if (st == TBE_OK && grad_x != nullptr) st = check_rows(x, grad_x, true);
    if (st == TBE_OK) st = check_param(weight, weight_dtype);
    if (st == TBE_OK) st = check_param(grad_weight, grad_weight_dtype);
    if (st == TBE_OK) st = check_param(grad_bias, grad_weight_dtype);
    if (st != TBE_OK) return st;
    if (x->rows > 0 && (mean == nullptr || rstd == nullptr)) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(mean, 4) || !is_aligned(rstd, 4) || !is_aligned(workspace, 256)) return TBE_ERR_MISALIGNED;
    const bool sums = grad_weight != nullptr || grad_bias != nullptr;
    const size_t need = sums ? tbe_layer_norm_workspace_bytes(x->rows, x->cols) : 0;
    if (need > 0 && workspace == nullptr) return TBE_ERR_NULL_POINTER;
    if (workspace_bytes < need) return TBE_ERR_BUFFER_TOO_SMALL;
    if ((grad_x == nullptr || x->rows == 0) && !sums) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        GradSums g{(float *)workspace, grad_weight, grad_bias, grad_weight_dtype, 0, x->cols};
        if (x->rows == 0) {     // sums over no rows
            L.before("tbe_layer_norm_bwd_join");
            layer_norm_bwd_join_kernel<<<dim3((unsigned)((x->cols + 31) / 32), 2), 256, 0, L.stream>>>(g, 0);
            L.after();
            return L.failed ? TBE_ERR_CUDA : TBE_OK;
        }
        const tbe_matrix *ms[3] = {grad_out, x, grad_x != nullptr ? grad_x : x};
        const int vec = norm_vector(x->dtype, vector_of(x->dtype == TBE_F32 ? 4 : 8, x->cols, ms, 3));
        TBE_NORM_SWITCH(x->dtype, vec, (run_bwd<T, VEC>(L, grad_out, x, weight, weight_dtype, mean, rstd, grad_x, g)));
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
