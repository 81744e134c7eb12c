// Shared by the token operators (token.cu, expert.cu, distill.cu): vectors of
// a row, element conversions, and the host checks of their entry points.
#pragma once

#include <type_traits>

#include "tbe_internal.cuh"

namespace tbe {

// ---- rows as vectors of VEC elements (VEC a power of two, at most 32 bytes)
// A vector is held in registers as it lies in memory and widened when used.
template <typename T, int VEC> struct Raw {
    static constexpr int BYTES = VEC * (int)sizeof(T);
    static constexpr int WORDS = BYTES >= 4 ? BYTES / 4 : 1;
    uint32_t w[WORDS];
};

// STREAM: data that this kernel reads once (evicted first).  The loads are
// plain (not the read-only path), so a kernel may overwrite what it has read.
template <typename T, int VEC, bool STREAM = false>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    Raw<T, VEC> r;
    constexpr int B = Raw<T, VEC>::BYTES;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p) + i;
            const uint4 v = STREAM ? __ldcs(q) : *q;
            r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (B == 8) {
        const uint2 *q = reinterpret_cast<const uint2 *>(p);
        const uint2 v = STREAM ? __ldcs(q) : *q;
        r.w[0] = v.x; r.w[1] = v.y;
    } else if constexpr (B == 4) {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
        r.w[0] = STREAM ? __ldcs(q) : *q;
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
        r.w[0] = STREAM ? __ldcs(q) : *q;
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, VEC> &r) {
    constexpr int B = Raw<T, VEC>::BYTES;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            reinterpret_cast<uint4 *>(p)[i] =
                make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(p) = r.w[0];
    } else {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)r.w[0];
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void widen(const Raw<T, VEC> &r, float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(r.w[i]);
    } else if constexpr (VEC == 1) {
        const uint16_t h = (uint16_t)r.w[0];
        f[0] = to_f32(*reinterpret_cast<const T *>(&h));
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            float2 v;
            if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
                v = bf16x2_to_float2(r.w[i]);
            else
                v = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

// The one rounding of a result to its type (to nearest even).
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> narrow(const float (&f)[VEC]) {
    Raw<T, VEC> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(f[i]);
    } else if constexpr (VEC == 1) {
        const T h = from_f32<T>(f[0]);
        r.w[0] = *reinterpret_cast<const uint16_t *>(&h);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                r.w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                r.w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return r;
}

// element i of an index array (int32 or int64)
__device__ __forceinline__ int64_t load_index(const void *ids, int index_type, int64_t i) {
    return index_type == TBE_INDEX_I64 ? __ldg(reinterpret_cast<const long long *>(ids) + i)
                                       : (int64_t)__ldg(reinterpret_cast<const int *>(ids) + i);
}

// element i of a small array of any of the three types, as a float
__device__ __forceinline__ float load_f32(const void *p, int dtype, int64_t i) {
    if (dtype == TBE_F32) return __ldg(reinterpret_cast<const float *>(p) + i);
    if (dtype == TBE_F16) return __half2float(__ldg(reinterpret_cast<const __half *>(p) + i));
    return __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16 *>(p) + i));
}
__device__ __forceinline__ void store_f32(void *p, int dtype, int64_t i, float x) {
    if (dtype == TBE_F32) reinterpret_cast<float *>(p)[i] = x;
    else if (dtype == TBE_F16) reinterpret_cast<__half *>(p)[i] = __float2half_rn(x);
    else reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// ---- programmatic launch: a kernel launched by launch_after may begin while
// the one before it on the stream runs, and waits for its results
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- clusters
// Stores a word to the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_store(uint32_t *shared, uint32_t rank, uint32_t v) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(shared);
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_store(float *shared, uint32_t rank, float v) {
    cluster_store(reinterpret_cast<uint32_t *>(shared), rank, __float_as_uint(v));
}
// RELEASE: the warp's writes are seen by those that wait
template <bool RELEASE> __device__ __forceinline__ void cluster_arrive() {
    if (RELEASE) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- host: a launch with a cluster and (after) programmatic serialization
template <typename... Formal, typename... Actual>
void launch_with(Launch &L, const char *name, bool after, int cluster, void (*fn)(Formal...), dim3 grid, int threads,
                 size_t smem, Actual... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (after) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    L.before(name);
    cudaLaunchKernelEx(&cfg, fn, static_cast<Formal>(args)...);
    L.after();
}

// ---- host checks
inline bool is_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int dtype_bytes(int dtype) { return dtype == TBE_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == TBE_F32 || dtype == TBE_F16 || dtype == TBE_BF16; }
inline bool known_index(int t) { return t == TBE_INDEX_I32 || t == TBE_INDEX_I64; }

constexpr int64_t TOKEN_MAX_ROWS = (int64_t)1 << 30;   // rows of an activation (positions fit 31 bits)
constexpr int64_t TOKEN_MAX_COLS = (int64_t)1 << 20;   // columns of an activation or a table row

// A matrix as a source (rows may repeat: stride 0 is one row for all) or as a
// destination (rows may not overlap).  An empty matrix needs no pointer.
inline tbe_status check_matrix(const tbe_matrix *m, bool written) {
    if (m == nullptr) return TBE_ERR_NULL_POINTER;
    if (!known_dtype(m->dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (m->rows < 0 || m->cols < 1 || m->stride < 0) return TBE_ERR_INVALID_ARGUMENT;
    if (written && m->rows > 1 && m->stride < m->cols) return TBE_ERR_INVALID_ARGUMENT;
    // every element's offset fits 62 bits
    if (m->rows > 0 && m->stride > ((int64_t)1 << 60) / m->rows) return TBE_ERR_INVALID_ARGUMENT;
    if (m->rows > 0 && m->data == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(m->data, dtype_bytes(m->dtype))) return TBE_ERR_MISALIGNED;
    return TBE_OK;
}

// Largest vector (elements, at most `most`) that divides the columns and that
// every matrix's rows are aligned to (16 bytes at most per access).
inline int vector_of(int most, int64_t cols, const tbe_matrix *const *ms, int n) {
    for (int v = most; v > 1; v /= 2) {
        bool ok = cols % v == 0;
        for (int i = 0; ok && i < n; ++i) {
            const size_t bytes = (size_t)v * dtype_bytes(ms[i]->dtype);
            ok = (ms[i]->rows <= 1 || ms[i]->stride % v == 0) &&
                 is_aligned(ms[i]->data, bytes < 16 ? bytes : 16);
        }
        if (ok) return v;
    }
    return 1;
}

// Lanes per row as a shift: the smallest power of two of lanes, at most a
// warp, that covers `vectors`.
inline int lane_shift(int64_t vectors) {
    int s = 0;
    while (s < 5 && (1 << s) < vectors) ++s;
    return s;
}

// Runs an entry point's body; no C++ exception leaves a C entry point (the
// launch caches allocate host memory).
template <typename F> tbe_status guarded(F &&body) {
    try {
        return body();
    } catch (...) {
        return TBE_ERR_CUDA;
    }
}

}  // namespace tbe
