// Layer norm of rows, and its gradients.
//
//   out = (x - mu) r w + b,   r = 1 / sqrt(var + eps)
//   with d = dy w, h = (x - mu) r:
//   dx = r (d - mean(d) - h mean(d h)),   dw = sum_n dy h,   db = sum_n dy
//
// Every element is used a few times and read once: HBM bounds both passes.  A
// row lies in the registers of a warp, or of a block where a warp's do not
// hold it, between the pass that sums and the pass that writes; the gradient's
// rows come through rings in shared memory.  32,768 x 4096 in bf16, with FP32
// weights: forward 103 us (5.2 TB/s), gradients 157 (5.1 TB/s).
#include "layer_checks.cuh"
#include "pairs.cuh"

namespace tbe {

constexpr int FWD_THREADS = 1024, BWD_THREADS = 512;
// A 16-byte copy to shared memory, and waiting for all but the latest N groups of them.
__device__ __forceinline__ void copy16(uint4 *shared, const void *global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(shared)), "l"(global)
                 : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Rows on their way through shared memory, beside the one worked on: two to eight.
constexpr int RING_MOST = 8;
__device__ __forceinline__ void copies_wait_but(int n) {
    switch (n) {
    case 1: copies_wait<1>(); break;
    case 2: copies_wait<2>(); break;
    case 3: copies_wait<3>(); break;
    case 4: copies_wait<4>(); break;
    case 5: copies_wait<5>(); break;
    case 6: copies_wait<6>(); break;
    default: copies_wait<7>(); break;
    }
}

// A parameter vector of any of the three types; its vectors are read whole
// where it is aligned for them.
struct Param {
    const void *p;      // nullptr: `fill` everywhere
    int dtype;
    int whole;          // aligned for vectors (of 16 bytes at most); 2: of 32 bytes
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
    } else if (VEC == 8 && w.dtype == TBE_F32 && w.whole == 2) {
        // 32 bytes at once: in two loads a warp's span of 1 KB takes twice the wavefronts of L1,
        // which bounded 16-bit rows (32768 x 4096: 130 us, 112 so, before pairs of rows)
        asm("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(f[0]), "=f"(f[1 % VEC]), "=f"(f[2 % VEC]), "=f"(f[3 % VEC]), "=f"(f[4 % VEC]), "=f"(f[5 % VEC]),
              "=f"(f[6 % VEC]), "=f"(f[7 % VEC])
            : "l"((const float *)w.p + i));
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
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) part[warp] = v;
        __syncthreads();
        if (warps <= 8) {
            v = part[0];
            for (int i = 1; i < warps; ++i) {
                v.x += part[i].x;
                v.y += part[i].y;
            }
        } else {
            v = warp_sum2(lane < warps ? part[lane] : make_float2(0.f, 0.f));
        }
    }
    return v;
}

// ---------------------------------------------------------------------------
// forward

// A vector's elements as floats, in pairs where there are several.
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum(float a) { return a; }
__device__ __forceinline__ float sum(Pair a) {
    const float2 f = unpair(a);
    return f.x + f.y;
}
template <int VEC> struct Floats {
    using Value = typename std::conditional<VEC == 1, float, Pair>::type;
    static constexpr int N = VEC > 1 ? VEC / 2 : 1;
    Value p[N];
    static __device__ __forceinline__ Value all(float x) {
        if constexpr (VEC == 1) return x;
        else return pair(x, x);
    }
    __device__ __forceinline__ float at(int k) const {
        if constexpr (VEC == 1) {
            return p[0];
        } else {
            const float2 f = unpair(p[k / 2]);
            return k % 2 ? f.y : f.x;
        }
    }
};
template <int VEC> __device__ __forceinline__ Floats<VEC> floats(const float (&a)[VEC]) {
    Floats<VEC> f;
    if constexpr (VEC == 1) {
        f.p[0] = a[0];
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) f.p[j] = pair(a[2 * j], a[2 * j + 1]);
    }
    return f;
}
template <typename T, int VEC> __device__ __forceinline__ Floats<VEC> floats(const Raw<T, VEC> &r) {
    if constexpr (VEC == 1) {
        float one[1];
        widen<T, 1>(r, one);
        return floats<1>(one);
    } else {
        Floats<VEC> f;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) f.p[j] = widen_pair<T, VEC>(r, j);
        return f;
    }
}
template <typename T, int VEC> __device__ __forceinline__ Raw<T, VEC> raw(const Floats<VEC> &f) {
    if constexpr (VEC == 1) {
        return narrow<T, 1>(f.p);
    } else {
        Raw<T, VEC> r;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) narrow_pair<T, VEC>(r, j, f.p[j]);
        return r;
    }
}

// A thread's NV vectors of its row, held as they lie in memory: few registers and
// small blocks, so that an SM has a dozen rows in some stage at any time.  The
// mean is corrected by the mean distance from it, so that rows with an offset far
// above their spread lose nothing to the first sum's rounding.
template <typename T, int VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS, THREADS != 512 ? 1 : VEC == 8 ? 2 : 3)
layer_norm_fwd_kernel(const T *__restrict__ x, int64_t xs, Param w, Param b, float eps, int64_t rows, int vectors,
                      T *__restrict__ out, int64_t os, float *mean, float *rstd) {
    constexpr bool BLOCK = THREADS > 32;
    using F = Floats<VEC>;
    __shared__ float2 part[2][32];
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31, lanes = BLOCK ? blockDim.x : 32;
    const int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= rows) return;
    Raw<T, VEC> read[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (v < vectors) read[i] = load_raw<T, VEC, true>(x + row * xs + (int64_t)v * VEC);
    }
    const float n = (float)((int64_t)vectors * VEC);
    auto s = F::all(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * lanes < vectors) {
            const F f = floats<T, VEC>(read[i]);
#pragma unroll
            for (int j = 0; j < F::N; ++j) s = add(s, f.p[j]);
        }
    }
    const float m = row_sum2<BLOCK>(make_float2(sum(s), 0.f), part[0]).x / n;
    s = F::all(0.f);
    auto q = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * lanes < vectors) {
            const F f = floats<T, VEC>(read[i]);
#pragma unroll
            for (int j = 0; j < F::N; ++j) {
                const auto c = add(f.p[j], F::all(-m));
                s = add(s, c);
                q = fma(c, c, q);
            }
        }
    }
    const float2 sums = row_sum2<BLOCK>(make_float2(sum(s), sum(q)), part[1]);
    const float e = sums.x / n, var = fmaxf(sums.y / n - e * e, 0.f);
    // (a NaN in the row: fmaxf would drop it)
    const float r = sums.y == sums.y ? 1.0f / sqrtf(var + eps) : sums.y;
    if (lane == 0) {
        if (mean != nullptr) mean[row] = m + e;
        if (rstd != nullptr) rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (v < vectors) {
            float g[VEC], o[VEC];
            load_param<VEC>(w, (int64_t)v * VEC, g);
            load_param<VEC>(b, (int64_t)v * VEC, o);
            const F scale = floats<VEC>(g), shift = floats<VEC>(o);
            F f = floats<T, VEC>(read[i]);
#pragma unroll
            for (int j = 0; j < F::N; ++j)
                f.p[j] = fma(mul(add(add(f.p[j], F::all(-m)), F::all(-e)), F::all(r)), scale.p[j], shift.p[j]);
            store_raw<T, VEC>(out + row * os + (int64_t)v * VEC, raw<T, VEC>(f));
        }
    }
}

// The same for two 16-bit rows a block, whose weights and biases (in FP32 four times
// a row's bytes) are read from L1 and widened once: 32768 x 4096 in bf16 take 103 us
// against 112, 8192 x 16384 in f16 121 against 127.  (Four vectors a thread and 24
// warps an SM; two vectors 123, 16 warps 112.)
constexpr int PAIR_NV = 4;
template <typename T, int NV, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS)
layer_norm_fwd_pair_kernel(const T *__restrict__ x, int64_t xs, Param w, Param b, float eps, int64_t rows, int vectors,
                           T *__restrict__ out, int64_t os, float *mean, float *rstd) {
    constexpr int VEC = 8;
    using F = Floats<VEC>;
    __shared__ float2 part[3][32];
    const int lane = threadIdx.x, lanes = blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * 2;
    const bool second = row + 1 < rows;     // (an odd number's last row is taken twice and written once)
    Raw<T, VEC> read[2][NV];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors) read[k][i] = load_raw<T, VEC, true>(x + (row + (second ? k : 0)) * xs + (int64_t)v * VEC);
        }
    }
    const float n = (float)((int64_t)vectors * VEC);
    Pair s[2] = {pair(0.f, 0.f), pair(0.f, 0.f)}, q[2] = {s[0], s[0]};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * lanes < vectors) {
                const F f = floats<T, VEC>(read[k][i]);
#pragma unroll
                for (int j = 0; j < F::N; ++j) s[k] = add(s[k], f.p[j]);
            }
        }
    }
    const float2 first = row_sum2<true>(make_float2(sum(s[0]), sum(s[1])), part[0]);
    const float m[2] = {first.x / n, first.y / n};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        s[k] = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * lanes < vectors) {
                const F f = floats<T, VEC>(read[k][i]);
#pragma unroll
                for (int j = 0; j < F::N; ++j) {
                    const Pair c = add(f.p[j], F::all(-m[k]));
                    s[k] = add(s[k], c);
                    q[k] = fma(c, c, q[k]);
                }
            }
        }
    }
    float e[2], r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 sums = row_sum2<true>(make_float2(sum(s[k]), sum(q[k])), part[1 + k]);
        e[k] = sums.x / n;
        // (a NaN in the row: fmaxf would drop it)
        r[k] = sums.y == sums.y ? 1.0f / sqrtf(fmaxf(sums.y / n - e[k] * e[k], 0.f) + eps) : sums.y;
        if (lane == 0 && (k == 0 || second)) {
            if (mean != nullptr) mean[row + k] = m[k] + e[k];
            if (rstd != nullptr) rstd[row + k] = r[k];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = lane + i * lanes;
        if (v < vectors) {
            float g[VEC], o[VEC];
            load_param<VEC>(w, (int64_t)v * VEC, g);
            load_param<VEC>(b, (int64_t)v * VEC, o);
            const F scale = floats<VEC>(g), shift = floats<VEC>(o);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                F f = floats<T, VEC>(read[k][i]);
#pragma unroll
                for (int j = 0; j < F::N; ++j)
                    f.p[j] = fma(mul(add(add(f.p[j], F::all(-m[k])), F::all(-e[k])), F::all(r[k])), scale.p[j],
                                 shift.p[j]);
                if (k == 0 || second) store_raw<T, VEC>(out + (row + k) * os + (int64_t)v * VEC, raw<T, VEC>(f));
            }
        }
    }
}

// A thread's vectors of the rows on their way: places of shared memory that it
// alone writes (by asynchronous copies) and reads, so that no barrier is needed
// and no register held while several rows are under way.
template <typename T, int NV, int ROWS> struct Ring {
    static constexpr int VEC = 16 / sizeof(T);
    uint4 *mine;
    int threads, lane, lanes, vectors;
    __device__ __forceinline__ uint4 *place(int stage, int which, int i) const {
        return mine + ((stage * ROWS + which) * NV + i) * threads;
    }
    __device__ __forceinline__ void load(int stage, int which, const T *row) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + i * lanes < vectors) copy16(place(stage, which, i), row + (int64_t)(lane + i * lanes) * VEC);
    }
    __device__ __forceinline__ Floats<VEC> get(int stage, int which, int i) const {
        const uint4 q = *place(stage, which, i);
        Raw<T, VEC> r;
        r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
        return floats<T, VEC>(r);
    }
};

// Rows of up to 128 vectors of 16 bytes, a warp each, in steps of the grid,
// `depth` of them under way; a thread's elements, weights and biases stay in
// registers.  (Rows of blocks are slower so: 32768 x 4096 in bf16 take 152 us.)
template <typename T, int NV>
__global__ void __launch_bounds__(256, 2)
layer_norm_fwd_ring_kernel(const T *__restrict__ x, int64_t xs, Param w, Param b, float eps, int64_t rows, int vectors,
                           T *__restrict__ out, int64_t os, float *mean, float *rstd, int depth) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ uint4 places[];
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    const Ring<T, NV, 1> ring{places + threadIdx.x, (int)blockDim.x, lane, 32, vectors};
    const float n = (float)((int64_t)vectors * VEC);
    int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    for (int i = 0; i < depth; ++i) {
        if (row + i * step < rows) ring.load(i, 0, x + (row + i * step) * xs);
        copies_issued();
    }
    Floats<VEC> f[NV], scale[NV], shift[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float g[VEC] = {}, o[VEC] = {};
        if (lane + i * 32 < vectors) {
            load_param<VEC>(w, (int64_t)(lane + i * 32) * VEC, g);
            load_param<VEC>(b, (int64_t)(lane + i * 32) * VEC, o);
        }
        scale[i] = floats<VEC>(g);
        shift[i] = floats<VEC>(o);
    }
    for (int stage = 0; row < rows; row += step, stage = stage + 1 == depth ? 0 : stage + 1) {
        copies_wait_but(depth - 1);
        Pair s = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * 32 < vectors) {
                f[i] = ring.get(stage, 0, i);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) s = add(s, f[i].p[j]);
            }
        }
        const float m = warp_sum2(make_float2(sum(s), 0.f)).x / n;
        s = pair(0.f, 0.f);
        Pair q = s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * 32 < vectors) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    f[i].p[j] = add(f[i].p[j], pair(-m, -m));
                    s = add(s, f[i].p[j]);
                    q = fma(f[i].p[j], f[i].p[j], q);
                }
            }
        }
        const float2 sums = warp_sum2(make_float2(sum(s), sum(q)));
        const float e = sums.x / n, var = fmaxf(sums.y / n - e * e, 0.f);
        const float r = sums.y == sums.y ? 1.0f / sqrtf(var + eps) : sums.y;
        if (lane == 0) {
            if (mean != nullptr) mean[row] = m + e;
            if (rstd != nullptr) rstd[row] = r;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * 32;
            if (v < vectors) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j)
                    f[i].p[j] = fma(mul(add(f[i].p[j], pair(-e, -e)), pair(r, r)), scale[i].p[j], shift[i].p[j]);
                store_raw<T, VEC>(out + row * os + (int64_t)v * VEC, raw<T, VEC>(f[i]));
            }
        }
        // (the stage's vectors have been used: they are stored)
        if (row + depth * step < rows) ring.load(stage, 0, x + (row + depth * step) * xs);
        copies_issued();
    }
    copies_wait<0>();
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
// grid: a thread keeps its columns' sums in registers over its rows, and the
// next row's loads are under way while a row is summed.
template <typename T, int VEC, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? BWD_THREADS : 256)
layer_norm_bwd_kernel(const T *__restrict__ dy, int64_t ds, const T *__restrict__ x, int64_t xs, Param w,
                      const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int vectors,
                      T *__restrict__ dx, int64_t os, GradSums g) {
    __shared__ float2 part[2][32];
    extern __shared__ float sums[];     // warps of rows: [2][D]
    launch_dependents();
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31, lanes = BLOCK ? blockDim.x : 32;
    const int64_t step = BLOCK ? (int64_t)gridDim.x : (int64_t)gridDim.x * warps;
    const float n = (float)((int64_t)vectors * VEC);
    Floats<VEC> wt[NV], aw[NV], ab[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[VEC] = {};
        aw[i] = ab[i] = floats<VEC>(f);
        if (lane + i * lanes < vectors) load_param<VEC>(w, (int64_t)(lane + i * lanes) * VEC, f);
        wt[i] = floats<VEC>(f);
    }
    Raw<T, VEC> rx[NV], ry[NV];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors && row < rows) {
                const T *px = x + row * xs + (int64_t)v * VEC, *py = dy + row * ds + (int64_t)v * VEC;
                rx[i] = load_raw<T, VEC, true>(px);
                ry[i] = load_raw<T, VEC, true>(py);
            }
        }
    };
    int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    load(row);
    float mu = row < rows ? __ldg(mean + row) : 0.f, r = row < rows ? __ldg(rstd + row) : 0.f;
    int turn = 0;
    for (; row < rows; row += step, turn ^= 1) {
        Floats<VEC> h[NV], d[NV];
        auto sd = Floats<VEC>::all(0.f), sh = sd;
        const auto minus = Floats<VEC>::all(-mu), by = Floats<VEC>::all(r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * lanes < vectors) {
                h[i] = floats<T, VEC>(rx[i]);
                d[i] = floats<T, VEC>(ry[i]);
#pragma unroll
                for (int j = 0; j < Floats<VEC>::N; ++j) {
                    h[i].p[j] = mul(add(h[i].p[j], minus), by);
                    aw[i].p[j] = fma(d[i].p[j], h[i].p[j], aw[i].p[j]);
                    ab[i].p[j] = add(ab[i].p[j], d[i].p[j]);
                    d[i].p[j] = mul(d[i].p[j], wt[i].p[j]);
                    sd = add(sd, d[i].p[j]);
                    sh = fma(d[i].p[j], h[i].p[j], sh);
                }
            }
        }
        const float r_now = r;
        if (row + step < rows) {
            mu = __ldg(mean + row + step);
            r = __ldg(rstd + row + step);
        }
        load(row + step);
        const float2 s = row_sum2<BLOCK>(make_float2(sum(sd), sum(sh)), part[turn]);
        if (dx != nullptr) {
            const float s1 = s.x / n, s2 = s.y / n;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + i * lanes;
                if (v < vectors) {
#pragma unroll
                    for (int j = 0; j < Floats<VEC>::N; ++j)
                        d[i].p[j] = mul(fma(h[i].p[j], Floats<VEC>::all(-s2), add(d[i].p[j], Floats<VEC>::all(-s1))), Floats<VEC>::all(r_now));
                    store_raw<T, VEC>(dx + row * os + (int64_t)v * VEC, raw<T, VEC>(d[i]));
                }
            }
        }
    }
    if (g.dw == nullptr && g.db == nullptr) return;
    if constexpr (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    store_sums(g, blockIdx.x, (int64_t)v * VEC + k, aw[i].at(k), ab[i].at(k));
            }
        }
    } else {
        // the warps' sums one after the other
        for (int t = 0; t < warps; ++t) {
            if (warp == t) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = lane + i * lanes;
                    if (v < vectors) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            float *p = sums + v * VEC + k;
                            p[0] = t == 0 ? aw[i].at(k) : p[0] + aw[i].at(k);
                            p[g.cols] = t == 0 ? ab[i].at(k) : p[g.cols] + ab[i].at(k);
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

// The same for rows of 16-byte vectors, which come through shared memory, `depth`
// of them under way.  KEEP (rows of blocks): a thread's 16 elements of x, dy and
// the weight stay in registers over the row's sums.  Rows of warps, of 32
// elements a thread, read them again, and the weight from shared memory.
template <typename T, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? BWD_THREADS : 256)
layer_norm_bwd_ring_kernel(const T *__restrict__ dy, int64_t ds, const T *__restrict__ x, int64_t xs, Param w,
                           const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int vectors,
                           T *__restrict__ dx, int64_t os, GradSums g, int depth) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr bool KEEP = BLOCK;
    __shared__ float2 part[2][32];
    extern __shared__ uint4 places[];   // the rings; rows of warps: the weight [D], then their sums [2][D]
    launch_dependents();
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = BLOCK ? threadIdx.x : threadIdx.x & 31, lanes = BLOCK ? blockDim.x : 32;
    const int64_t step = BLOCK ? (int64_t)gridDim.x : (int64_t)gridDim.x * warps;
    const Ring<T, NV, 2> ring{places + threadIdx.x, (int)blockDim.x, lane, lanes, vectors};
    float *weight = (float *)(places + depth * 2 * NV * blockDim.x);
    const float n = (float)((int64_t)vectors * VEC);
    int64_t row = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    auto load = [&](int64_t at, int stage) {
        if (at < rows) {
            ring.load(stage, 0, x + at * xs);
            ring.load(stage, 1, dy + at * ds);
        }
        copies_issued();
    };
    for (int i = 0; i < depth; ++i) load(row + i * step, i);
    Floats<VEC> aw[NV], ab[NV], kept_w[KEEP ? NV : 1], kept_h[KEEP ? NV : 1], kept_d[KEEP ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) aw[i].p[j] = ab[i].p[j] = pair(0.f, 0.f);
        if constexpr (KEEP) {
            float f[VEC] = {};
            if (lane + i * lanes < vectors) load_param<VEC>(w, (int64_t)(lane + i * lanes) * VEC, f);
            kept_w[i] = floats<VEC>(f);
        }
    }
    if constexpr (!KEEP) {
        for (int v = threadIdx.x; v < vectors; v += blockDim.x) {
            float f[VEC];
            load_param<VEC>(w, (int64_t)v * VEC, f);
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j)
                ((float4 *)weight)[j * vectors + v] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
        }
        __syncthreads();
    }
    auto weights = [&](int i) {
        if constexpr (KEEP) {
            return kept_w[i];
        } else {
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) {
                const float4 q = ((const float4 *)weight)[j * vectors + lane + i * lanes];
                f[4 * j] = q.x; f[4 * j + 1] = q.y; f[4 * j + 2] = q.z; f[4 * j + 3] = q.w;
            }
            return floats<VEC>(f);
        }
    };
    float mu = row < rows ? __ldg(mean + row) : 0.f, r = row < rows ? __ldg(rstd + row) : 0.f;
    for (int turn = 0, stage = 0; row < rows; row += step, turn ^= 1, stage = stage + 1 == depth ? 0 : stage + 1) {
        copies_wait_but(depth - 1);
        Pair sd = pair(0.f, 0.f), sh = sd;
        const Pair minus = pair(-mu, -mu), by = pair(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * lanes < vectors) {
                const Floats<VEC> f = ring.get(stage, 0, i), d = ring.get(stage, 1, i), wt = weights(i);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const Pair h = mul(add(f.p[j], minus), by), dw = mul(d.p[j], wt.p[j]);
                    aw[i].p[j] = fma(d.p[j], h, aw[i].p[j]);
                    ab[i].p[j] = add(ab[i].p[j], d.p[j]);
                    sd = add(sd, dw);
                    sh = fma(dw, h, sh);
                    if constexpr (KEEP) {
                        kept_h[i].p[j] = h;
                        kept_d[i].p[j] = dw;
                    }
                }
            }
        }
        if (row + step < rows) {
            mu = __ldg(mean + row + step);
            r = __ldg(rstd + row + step);
        }
        const float2 s = row_sum2<BLOCK>(make_float2(sum(sd), sum(sh)), part[turn]);
        if (dx != nullptr) {
            const float s1 = s.x / n, s2 = s.y / n;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + i * lanes;
                if (v < vectors) {
                    Floats<VEC> h, d;
                    if constexpr (KEEP) {
                        h = kept_h[i];
                        d = kept_d[i];
                    } else {
                        h = ring.get(stage, 0, i);
                        d = ring.get(stage, 1, i);
                        const Floats<VEC> wt = weights(i);
#pragma unroll
                        for (int j = 0; j < VEC / 2; ++j) {
                            h.p[j] = mul(add(h.p[j], minus), by);
                            d.p[j] = mul(d.p[j], wt.p[j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j)
                        d.p[j] = mul(fma(h.p[j], pair(-s2, -s2), add(d.p[j], pair(-s1, -s1))), by);
                    store_raw<T, VEC>(dx + row * os + (int64_t)v * VEC, raw<T, VEC>(d));
                }
            }
        }
        // (the stage's vectors have been used)
        load(row + depth * step, stage);
    }
    copies_wait<0>();
    if (g.dw == nullptr && g.db == nullptr) return;
    if constexpr (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = lane + i * lanes;
            if (v < vectors) {
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    store_sums(g, blockIdx.x, (int64_t)v * VEC + k, aw[i].at(k), ab[i].at(k));
            }
        }
    } else {
        // the warps' sums one after the other
        float *sums = weight + g.cols;
        for (int t = 0; t < warps; ++t) {
            if (warp == t) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = lane + i * lanes;
                    if (v < vectors) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            float *p = sums + v * VEC + k;
                            p[0] = t == 0 ? aw[i].at(k) : p[0] + aw[i].at(k);
                            p[g.cols] = t == 0 ? ab[i].at(k) : p[g.cols] + ab[i].at(k);
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
    return Param{p, dtype, !is_aligned(p, bytes < 16 ? bytes : 16) ? 0 : is_aligned(p, 32) ? 2 : 1, fill};
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

struct NormCall {
    const tbe_matrix *x, *out, *dy, *dx;
    Param w, b;
    float eps;
    float *mean, *rstd;         // written (forward), read (backward)
    GradSums sums;
    int vectors;
};

// Blocks that are resident together, `each` rows a block.
static int64_t resident(Launch &L, const void *fn, int threads, size_t smem, int64_t rows, int each) {
    const int64_t blocks = (int64_t)cached_blocks_per_sm(L.dev, fn, threads, smem) * L.num_sms, most = (rows + each - 1) / each;
    return blocks < 1 || blocks > most ? most : blocks;
}

// THREADS: 32 for a warp a row, otherwise the most of a block
template <typename T, int VEC, int NV, int THREADS> static void launch_fwd(Launch &L, int threads, const NormCall &c) {
    const int each = THREADS > 32 ? 1 : threads / 32;
    const int64_t blocks = (c.x->rows + each - 1) / each;
    L.before("tbe_layer_norm_fwd");
    layer_norm_fwd_kernel<T, VEC, NV, THREADS><<<(unsigned)blocks, threads, 0, L.stream>>>(
        (const T *)c.x->data, c.x->stride, c.w, c.b, c.eps, c.x->rows, c.vectors, (T *)c.out->data, c.out->stride, c.mean, c.rstd);
    L.after();
}
// Bytes of shared memory that the rows under way take of an SM: HBM's latency
// under load times its rate is near 100 KB an SM (norm backward of 32768 x 4096
// in bf16: 96 KB reach 0.65 of the copy rate).
constexpr size_t NORM_SMEM = 200 * 1024, NORM_SMEM_MOST = 224 * 1024;
// Rows under way for a kernel whose blocks each need `each` bytes a row and `more` bytes.
static int ring_depth(Launch &L, const void *fn, int threads, size_t each, size_t more) {
    cached_smem_attr(L.dev, fn, NORM_SMEM_MOST);
    int blocks = cached_blocks_per_sm(L.dev, fn, threads, 2 * each + more);
    if (blocks < 1) blocks = 1;
    const int64_t depth = ((int64_t)(NORM_SMEM / blocks) - (int64_t)more) / (int64_t)each;
    return depth < 2 ? 2 : depth > RING_MOST ? RING_MOST : (int)depth;
}

template <typename T, int NV> static void launch_fwd_ring(Launch &L, const NormCall &c) {
    auto *fn = layer_norm_fwd_ring_kernel<T, NV>;
    const size_t each = (size_t)NV * 16 * 256;
    const int depth = ring_depth(L, (const void *)fn, 256, each, 0);
    const int64_t blocks = resident(L, (const void *)fn, 256, each * depth, c.x->rows, 8);
    L.before("tbe_layer_norm_fwd_ring");
    fn<<<(unsigned)blocks, 256, each * depth, L.stream>>>(
        (const T *)c.x->data, c.x->stride, c.w, c.b, c.eps, c.x->rows, c.vectors, (T *)c.out->data, c.out->stride, c.mean,
        c.rstd, depth);
    L.after();
}

static int block_of(int vectors, int nv) { return ((vectors + nv - 1) / nv + 31) / 32 * 32; }

template <typename T, int VEC> static void run_fwd(Launch &L, const NormCall &c) {
    const int vectors = c.vectors;
    const bool many = c.x->rows >= 4 * L.num_sms;
    if constexpr (VEC * sizeof(T) == 16) {
        if (vectors <= 32) return launch_fwd<T, VEC, 1, 32>(L, 256, c);
        if (many && vectors <= 64) return launch_fwd_ring<T, 2>(L, c);
        if (many && vectors <= 128) return launch_fwd_ring<T, 4>(L, c);
        // few rows: as many threads as a row has vectors; many: four vectors a thread
        if (!many && vectors <= 1024) return launch_fwd<T, VEC, 1, 1024>(L, block_of(vectors, 1), c);
        if constexpr (sizeof(T) == 2) {
            if (many && vectors <= 512 * PAIR_NV) {
                const int threads = block_of(vectors, PAIR_NV);
                auto *fn = threads <= 128   ? layer_norm_fwd_pair_kernel<T, PAIR_NV, 128, 6>
                           : threads <= 256 ? layer_norm_fwd_pair_kernel<T, PAIR_NV, 256, 3>
                                            : layer_norm_fwd_pair_kernel<T, PAIR_NV, 512, 2>;
                L.before("tbe_layer_norm_fwd");
                fn<<<(unsigned)((c.x->rows + 1) / 2), threads, 0, L.stream>>>(
                    (const T *)c.x->data, c.x->stride, c.w, c.b, c.eps, c.x->rows, vectors, (T *)c.out->data, c.out->stride,
                    c.mean, c.rstd);
                L.after();
                return;
            }
        }
        if (vectors <= 512 * 4) return launch_fwd<T, VEC, 4, 512>(L, block_of(vectors, 4), c);
        if (vectors <= 1024 * 4) return launch_fwd<T, VEC, 4, 1024>(L, block_of(vectors, 4), c);
    } else {
        constexpr int MOST = 16 / VEC;      // vectors a thread
        if (vectors <= 32) return launch_fwd<T, VEC, 1, 32>(L, 256, c);
        if (many && vectors <= 32 * MOST) return launch_fwd<T, VEC, MOST, 32>(L, 256, c);
        if (vectors <= 512) return launch_fwd<T, VEC, 1, 1024>(L, block_of(vectors, 1), c);
        if (vectors <= 1024 * MOST / 2) return launch_fwd<T, VEC, MOST / 2, 1024>(L, block_of(vectors, MOST / 2), c);
    }
    L.before("tbe_layer_norm_fwd_long");
    layer_norm_fwd_long_kernel<T, VEC><<<(unsigned)c.x->rows, FWD_THREADS, 0, L.stream>>>(
        (const T *)c.x->data, c.x->stride, c.w, c.b, c.eps, vectors, (T *)c.out->data, c.out->stride, c.mean, c.rstd);
    L.after();
}

// Launches the rows' gradient with the sums; returns how many parts these have.
template <typename T, typename Kernel, typename... More>
static int64_t launch_bwd(Launch &L, Kernel fn, bool block, int threads, size_t smem, const NormCall &c, More... more) {
    int64_t blocks = resident(L, (const void *)fn, threads, smem, c.x->rows, block ? 1 : threads / 32);
    const int64_t parts = norm_parts(c.x->rows, c.x->cols);
    if (blocks > parts) blocks = parts;
    GradSums g = c.sums;
    g.direct = blocks == 1;
    L.before("tbe_layer_norm_bwd");
    fn<<<(unsigned)blocks, threads, smem, L.stream>>>(
        (const T *)c.dy->data, c.dy->stride, (const T *)c.x->data, c.x->stride, c.w, c.mean, c.rstd, c.x->rows, c.vectors,
        c.dx != nullptr ? (T *)c.dx->data : nullptr, c.dx != nullptr ? c.dx->stride : 0, g, more...);
    L.after();
    return blocks;
}
template <typename T, int VEC, int NV, bool BLOCK> static int64_t launch_bwd_plain(Launch &L, int threads, const NormCall &c) {
    return launch_bwd<T>(L, layer_norm_bwd_kernel<T, VEC, NV, BLOCK>, BLOCK, threads, BLOCK ? 0 : (size_t)c.x->cols * 8, c);
}
template <typename T, int NV, bool BLOCK> static int64_t launch_bwd_ring(Launch &L, int threads, const NormCall &c) {
    auto *fn = layer_norm_bwd_ring_kernel<T, NV, BLOCK>;
    const size_t each = (size_t)2 * NV * 16 * threads, more = BLOCK ? 0 : (size_t)c.x->cols * 12;
    const int depth = ring_depth(L, (const void *)fn, threads, each, more);
    return launch_bwd<T>(L, fn, BLOCK, threads, each * depth + more, c, depth);
}

template <typename T, int VEC> static void run_bwd(Launch &L, const NormCall &c) {
    constexpr int MOST = 16 / VEC;      // vectors a thread
    const int vectors = c.vectors;
    const bool sums = c.sums.dw != nullptr || c.sums.db != nullptr;
    int64_t parts;
    if (vectors <= BWD_THREADS * MOST) {
        if constexpr (VEC * sizeof(T) == 16) {
            // rows of warps up to 1024 16-bit or 512 32-bit elements, then of blocks
            if (vectors <= 32) parts = launch_bwd_ring<T, 1, false>(L, 256, c);
            else if (vectors <= 64) parts = launch_bwd_ring<T, 2, false>(L, 256, c);
            else if (vectors <= 128) parts = launch_bwd_ring<T, 4, false>(L, 256, c);
            else parts = launch_bwd_ring<T, MOST, true>(L, block_of(vectors, MOST), c);
        } else {
            constexpr int LESS = MOST / 2;
            if (vectors <= 32 * LESS) parts = launch_bwd_plain<T, VEC, LESS, false>(L, 256, c);
            else if (vectors <= 32 * MOST) parts = launch_bwd_plain<T, VEC, MOST, false>(L, 256, c);
            else if (vectors <= 256 * LESS) parts = launch_bwd_plain<T, VEC, LESS, true>(L, block_of(vectors, LESS), c);
            else parts = launch_bwd_plain<T, VEC, MOST, true>(L, block_of(vectors, MOST), c);
        }
    } else {
        if (c.dx != nullptr) {
            L.before("tbe_layer_norm_bwd_long");
            layer_norm_bwd_long_kernel<T, VEC><<<(unsigned)c.x->rows, BWD_THREADS, 0, L.stream>>>(
                (const T *)c.dy->data, c.dy->stride, (const T *)c.x->data, c.x->stride, c.w, c.mean, c.rstd, vectors,
                (T *)c.dx->data, c.dx->stride);
            L.after();
        }
        if (!sums) return;
        const int64_t strips = (vectors + 31) / 32;
        parts = norm_parts((c.x->rows + 31) / 32, c.x->cols);
        const int64_t enough = (8 * L.num_sms + strips - 1) / strips;
        if (parts > enough) parts = enough;
        GradSums g = c.sums;
        g.direct = parts == 1;
        L.before("tbe_layer_norm_bwd_columns");
        layer_norm_bwd_columns_kernel<T, VEC><<<dim3((unsigned)strips, (unsigned)parts), 256, 0, L.stream>>>(
            (const T *)c.dy->data, c.dy->stride, (const T *)c.x->data, c.x->stride, c.mean, c.rstd, c.x->rows, vectors, g);
        L.after();
    }
    if (sums && parts > 1)
        launch_with(L, "tbe_layer_norm_bwd_join", true, 1, layer_norm_bwd_join_kernel,
                    dim3((unsigned)((c.x->cols + 31) / 32), 2), 256, 0, c.sums, (int)parts);
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
    const Span to = span_of(out), from = span_of(x), mu = span_of(mean, x->rows * 4), r = span_of(rstd, x->rows * 4);
    const Span w = span_of(weight, x->cols * dtype_bytes(weight_dtype)), b = span_of(bias, x->cols * dtype_bytes(weight_dtype));
    if (share(to, from, w, b, mu, r) || share(mu, from, w, b, r) || share(r, from, w, b)) return TBE_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const tbe_matrix *ms[2] = {x, out};
        const int vec = norm_vector(x->dtype, vector_of(x->dtype == TBE_F32 ? 4 : 8, x->cols, ms, 2));
        NormCall c = {};
        c.x = x;
        c.out = out;
        c.w = param(weight, weight_dtype, vec, 1.f);
        c.b = param(bias, weight_dtype, vec, 0.f);
        c.eps = eps;
        c.mean = mean;
        c.rstd = rstd;
        c.vectors = (int)(x->cols / vec);
        TBE_NORM_SWITCH(x->dtype, vec, (run_fwd<T, VEC>(L, c)));
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
    const Span dx = span_of(grad_x), dy = span_of(grad_out), from = span_of(x), ws = span_of(workspace, need);
    const Span w = span_of(weight, x->cols * dtype_bytes(weight_dtype)), mu = span_of(mean, x->rows * 4), r = span_of(rstd, x->rows * 4);
    const Span dw = span_of(grad_weight, x->cols * dtype_bytes(grad_weight_dtype)), db = span_of(grad_bias, x->cols * dtype_bytes(grad_weight_dtype));
    if (share(dx, dy, from, w, mu, r, dw, db, ws) || share(dw, dy, from, w, mu, r, db, ws) || share(db, dy, from, w, mu, r, ws) ||
        share(ws, dy, from, w, mu, r))
        return TBE_ERR_INVALID_ARGUMENT;
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
        NormCall c = {};
        c.x = x;
        c.dy = grad_out;
        c.dx = grad_x;
        c.w = param(weight, weight_dtype, vec, 1.f);
        c.mean = const_cast<float *>(mean);
        c.rstd = const_cast<float *>(rstd);
        c.sums = g;
        c.vectors = (int)(x->cols / vec);
        TBE_NORM_SWITCH(x->dtype, vec, (run_bwd<T, VEC>(L, c)));
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
