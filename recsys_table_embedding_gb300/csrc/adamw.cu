// One AdamW step of many tensors in one launch (decoupled weight decay; states
// in FP32, or in 8 bits with a scale for each 256 elements).
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - m lr / (1 - b1^t) / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Each element is read and written once and HBM bounds the step.  A warp takes
// 256 consecutive elements of a tensor, which is also a block of the 8-bit
// states, so that a block's scale is a maximum over a warp; a CTA takes 2048 and
// ends.  The tensors' records are a kernel parameter: no table in device memory
// has to be written, and a captured step carries its own.
#include <math.h>

#include <algorithm>
#include <vector>

#include <cuda_fp8.h>

#include "pairs.cuh"

namespace tbe {

constexpr int ADAM_WARP = 256;                  // elements a warp, and of a block of 8-bit states
constexpr int ADAM_CTA = 8 * ADAM_WARP;
constexpr int ADAM_EACH = ADAM_WARP / 32;       // elements a thread

struct AdamTensor {
    void *param;
    const void *grad;
    void *m, *v;
    float *scales;
    void *copy;
    int64_t n;
    uint32_t first;             // first CTA of the tensor
    uint32_t index;             // place in the caller's list
    uint8_t param_dtype, grad_dtype, copy_dtype, whole;     // whole: vectors of 4 elements are aligned
};

// What the step's numbers come to, on the host or (FromDevice) in the workspace.
struct AdamFactors {
    float keep, rate, root;     // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    uint32_t key;               // of the random numbers
};

// Few tensors travel in 4 KB of parameters, many in 32 (the limit is 32,764 B).
constexpr int ADAM_FEW = 48, ADAM_MANY = 440;
template <int MOST> struct AdamArgs {
    AdamTensor t[MOST];
    int count;
    float b1, c1, b2, c2, eps;  // c = 1 - b
    AdamFactors f;
    const AdamFactors *from_device;     // or nullptr
    const float *grad_scale;            // or nullptr
};
static_assert(sizeof(AdamArgs<ADAM_MANY>) <= 32764, "kernel parameters");

// The finalising mix of MurmurHash3 (Austin Appleby, public domain).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}
__host__ __device__ __forceinline__ uint32_t step_key(uint32_t seed, int64_t step) {
    return mix32(seed + (uint32_t)step * 0x9E3779B9u);
}

// Place of a thread's e-th element among its warp's: vectors of four, or
// (unaligned tensors, their last elements) one after the other across the lanes.
template <bool WHOLE> __device__ __forceinline__ int element(int lane, int e) {
    return WHOLE ? (e >> 2) * 128 + lane * 4 + (e & 3) : e * 32 + lane;
}

template <bool WHOLE>
__device__ __forceinline__ void store_values(void *p, int dtype, int64_t base, int lane, int left,
                                             const float (&f)[ADAM_EACH]) {
    if constexpr (WHOLE) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float part[4] = {f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]};
            const int64_t at = base + j * 128 + lane * 4;
            if (dtype == TBE_F32) store_raw<float, 4>((float *)p + at, narrow<float, 4>(part));
            else if (dtype == TBE_F16) store_raw<__half, 4>((__half *)p + at, narrow<__half, 4>(part));
            else store_raw<__nv_bfloat16, 4>((__nv_bfloat16 *)p + at, narrow<__nv_bfloat16, 4>(part));
        }
    } else {
#pragma unroll
        for (int e = 0; e < ADAM_EACH; ++e)
            if (e * 32 + lane < left) store_f32(p, dtype, base + e * 32 + lane, f[e]);
    }
}

// A thread's elements as they lie in memory (16-bit ones two a word), so that
// every load is under way before the first is used.
template <bool WHOLE> struct Loaded {
    uint32_t w[ADAM_EACH];
    __device__ __forceinline__ void load32(const void *p, int64_t base, int lane, int left) {
        if constexpr (WHOLE) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4 *>((const uint32_t *)p + base + j * 128 + lane * 4));
                w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < ADAM_EACH; ++e)
                w[e] = e * 32 + lane < left ? ((const uint32_t *)p)[base + e * 32 + lane] : 0u;
        }
    }
    __device__ __forceinline__ void load16(const void *p, int64_t base, int lane, int left) {
        if constexpr (WHOLE) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2 *>((const uint16_t *)p + base + j * 128 + lane * 4));
                w[2 * j] = u.x; w[2 * j + 1] = u.y;
            }
        } else {
            uint16_t h[ADAM_EACH];
#pragma unroll
            for (int e = 0; e < ADAM_EACH; ++e)
                h[e] = e * 32 + lane < left ? ((const uint16_t *)p)[base + e * 32 + lane] : (uint16_t)0;
#pragma unroll
            for (int j = 0; j < ADAM_EACH / 2; ++j) w[j] = h[2 * j] | (uint32_t)h[2 * j + 1] << 16;
        }
    }
    __device__ __forceinline__ void load(const void *p, int dtype, int64_t base, int lane, int left) {
        if (dtype == TBE_F32) load32(p, base, lane, left);
        else load16(p, base, lane, left);
    }
    __device__ __forceinline__ void values(int dtype, Pair (&f)[ADAM_EACH / 2]) const {
        if (dtype == TBE_F32) {
#pragma unroll
            for (int j = 0; j < ADAM_EACH / 2; ++j) f[j] = pair(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else if (dtype == TBE_BF16) {
#pragma unroll
            for (int j = 0; j < ADAM_EACH / 2; ++j) {
                const float2 v = bf16x2_to_float2(w[j]);
                f[j] = pair(v.x, v.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < ADAM_EACH / 2; ++j) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                f[j] = pair(v.x, v.y);
            }
        }
    }
};
template <bool WHOLE>
__device__ __forceinline__ void store_pairs(void *p, int dtype, int64_t base, int lane, int left,
                                            const Pair (&a)[ADAM_EACH / 2]) {
    float f[ADAM_EACH];
#pragma unroll
    for (int j = 0; j < ADAM_EACH / 2; ++j) {
        const float2 v = unpair(a[j]);
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
    }
    store_values<WHOLE>(p, dtype, base, lane, left, f);
}

// A thread's codes, four a word.
template <bool WHOLE>
__device__ __forceinline__ void load_codes(const void *p, int64_t base, int lane, int left, uint32_t (&w)[2]) {
    const uint8_t *codes = (const uint8_t *)p + base;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (WHOLE) {
            w[j] = __ldcs(reinterpret_cast<const uint32_t *>(codes + j * 128) + lane);
        } else {
            w[j] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = (4 * j + k) * 32 + lane;
                w[j] |= (i < left ? (uint32_t)codes[i] : 0u) << (8 * k);
            }
        }
    }
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(void *p, int64_t base, int lane, int left, const uint32_t (&w)[2]) {
    uint8_t *codes = (uint8_t *)p + base;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (WHOLE) {
            reinterpret_cast<uint32_t *>(codes + j * 128)[lane] = w[j];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = (4 * j + k) * 32 + lane;
                if (i < left) codes[i] = (uint8_t)(w[j] >> (8 * k));
            }
        }
    }
}

// codes -> values (exact: every e4m3 value is one of FP16's)
__device__ __forceinline__ void decode(const uint32_t (&w)[2], Pair (&f)[ADAM_EACH / 2]) {
#pragma unroll
    for (int j = 0; j < ADAM_EACH / 2; ++j) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3));
        const float2 v = __half22float2(h);
        f[j] = pair(v.x, v.y);
    }
}

// The largest |x| of three, NaN if one is.
__device__ __forceinline__ float largest(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// a + b of products in pairs, which are rounded: the assembler fuses a pair's product and
// sum, but not with scalar sums (no slower here).  The states are the stated formula's to
// the bit, so that codes and scales are those of any other evaluation of it.
__device__ __forceinline__ float2 sum(Pair a, Pair b) {
    const float2 x = unpair(a), y = unpair(b);
    return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// The code of y = |x| / scale, in the lowest byte of the result (others are not 0).  y
// is scaled to whole steps of its binade, 8 to 16 of them (below 2^-6 codes are 2^-9
// apart), which is a product by a power of two; 16 random bits are added behind the
// point, in FP32, and what is left of the point counts codes from the binade's
// first, 8 a binade.  The count is the low bits of 2^23 + t rounded down.  (y is
// 448 at most, but for roundings too small to carry it into the code behind, which
// is NaN's.  Random bits added to the mantissa's are an instruction less, but where
// the sum passes the binade they skip its rounding: eight codes of 268 million, and
// what the next steps make of them.)
__device__ __forceinline__ uint32_t code_of(float y, uint32_t random) {     // random: 128 + random16 / 2^16, as bits
    const uint32_t binade = max(__float_as_uint(y) & 0x7F800000u, 121u << 23);
    const float t = __fmaf_rn(y, __uint_as_float((257u << 23) - binade), __uint_as_float(random) - 128.0f);
    return __float_as_uint(__fadd_rd(t, 8388608.0f)) + (binade >> 20) - (121u << 3);
}

// The codes of a warp's 256 elements and their scale; FLOOR (values >= 0):
// positive ones keep a code above 0.  Elements that are not there are 0.
template <bool FLOOR>
__device__ __forceinline__ void encode(const Pair (&pairs)[ADAM_EACH / 2], const uint32_t (&random)[ADAM_EACH],
                                       uint32_t (&w)[2], float &scale) {
    float x[ADAM_EACH];
#pragma unroll
    for (int j = 0; j < ADAM_EACH / 2; ++j) {
        const float2 v = unpair(pairs[j]);
        x[2 * j] = v.x;
        x[2 * j + 1] = v.y;
    }
    // as bits, which order like the values; infinities and NaN are above them
    uint32_t most = __float_as_uint(largest(largest(largest(x[0], x[1], x[2]), x[3], x[4]), largest(x[5], x[6], x[7]), 0.f));
    most = __reduce_max_sync(FULL, most);
    const bool finite = most < 0x7F800000u;
    if (!finite) {
        most = 0;
#pragma unroll
        for (int e = 0; e < ADAM_EACH; ++e) {
            const uint32_t a = __float_as_uint(x[e]) & 0x7FFFFFFFu;
            if (a < 0x7F800000u) most = max(most, a);
        }
        most = __reduce_max_sync(FULL, most);
    }
    // blocks below 2^-100 become zeros: their reciprocal scale would leave the range
    scale = __uint_as_float(most) < 7.888609052e-31f ? 0.f : __fmul_rn(__uint_as_float(most), 1.0f / 448.0f);
    const float inv = scale > 0.f ? __fdiv_rn(1.0f, scale) : 0.f;
    uint32_t code[ADAM_EACH];
#pragma unroll
    for (int j = 0; j < ADAM_EACH / 2; ++j) {
        const float2 q = unpair(mul(pairs[j], pair(inv, inv)));
        const float y[2] = {fabsf(q.x), fabsf(q.y)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = 2 * j + k;
            code[e] = code_of(y[k], __byte_perm(random[e], 0x4300u, FLOOR ? 0x5432 : 0x5410));
            // (0x4B000000 + code: the larger is the code's own for positive y)
            if (FLOOR) code[e] = max(code[e], 0x4B000000u + min(__float_as_uint(y[k]), 1u));
        }
    }
    if (!finite) {
#pragma unroll
        for (int e = 0; e < ADAM_EACH; ++e)
            if ((__float_as_uint(x[e]) & 0x7FFFFFFFu) >= 0x7F800000u) code[e] = 0x7Fu;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        // the four words' lowest bytes, and (values of either sign) their values' signs
        w[j] = __byte_perm(__byte_perm(code[4 * j], code[4 * j + 1], 0x0040), __byte_perm(code[4 * j + 2], code[4 * j + 3], 0x0040), 0x5410);
        if (!FLOOR)
            w[j] |= __byte_perm(__byte_perm(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]), 0x0073),
                                __byte_perm(__float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]), 0x0073), 0x5410) & 0x80808080u;
    }
}

// One warp's elements of a tensor; `left`: those that there are.
template <bool E4M3, bool WHOLE, int MOST>
__device__ __forceinline__ void adam_block(const AdamArgs<MOST> &a, const AdamTensor &t, int64_t base, int lane,
                                           int left) {
    Loaded<WHOLE> lp, lg, lm, lv;
    uint32_t cm[2], cv[2];
    float sm = 0.f, sv = 0.f;
    float *scales = t.scales + base / ADAM_WARP * 2;
    if constexpr (E4M3) {
        sm = __ldcs(scales);
        sv = __ldcs(scales + 1);
        load_codes<WHOLE>(t.m, base, lane, left, cm);
        load_codes<WHOLE>(t.v, base, lane, left, cv);
    } else {
        lm.load32(t.m, base, lane, left);
        lv.load32(t.v, base, lane, left);
    }
    lp.load(t.param, t.param_dtype, base, lane, left);
    lg.load(t.grad, t.grad_dtype, base, lane, left);
    AdamFactors f = a.f;
    if (a.from_device != nullptr) f = *a.from_device;
    constexpr int N = ADAM_EACH / 2;
    Pair p[N], g[N], m[N], v[N], r[N];
    if constexpr (E4M3) {
        decode(cm, m);
        decode(cv, v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = mul(m[j], pair(sm, sm));
            v[j] = mul(v[j], pair(sv, sv));
            v[j] = mul(v[j], v[j]);
        }
    } else {
        lm.values(TBE_F32, m);
        lv.values(TBE_F32, v);
    }
    lp.values(t.param_dtype, p);
    lg.values(t.grad_dtype, g);
    if (a.grad_scale != nullptr) {
        const float s = __ldg(a.grad_scale);
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = mul(g[j], pair(s, s));
    }
    const Pair b1 = pair(a.b1, a.b1), c1 = pair(a.c1, a.c1), b2 = pair(a.b2, a.b2), c2 = pair(a.c2, a.c2);
    const Pair rate = pair(f.rate, f.rate), root = pair(f.root, f.root), keep = pair(f.keep, f.keep), eps = pair(a.eps, a.eps);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float2 first = sum(mul(m[j], b1), mul(g[j], c1));
        const float2 second = sum(mul(v[j], b2), mul(mul(g[j], g[j]), c2));
        m[j] = pair(first.x, first.y);
        v[j] = pair(second.x, second.y);
        // (the root to the nearest also for 8-bit states: an approximate one saves 23 us of
        // 453 at 135M parameters and changes codes)
        r[j] = pair(__fsqrt_rn(second.x), __fsqrt_rn(second.y));
        const float2 above = unpair(mul(m[j], rate)), below = sum(mul(r[j], root), eps);
        // 8-bit states: the step is bound by its instructions, and the hardware's
        // approximate quotient (2^-22) is enough for a change of the parameter
        const Pair change = E4M3 ? pair(-__fdividef(above.x, below.x), -__fdividef(above.y, below.y))
                                 : pair(-__fdiv_rn(above.x, below.x), -__fdiv_rn(above.y, below.y));
        const float2 after = sum(mul(p[j], keep), change);
        p[j] = pair(after.x, after.y);
    }
    store_pairs<WHOLE>(t.param, t.param_dtype, base, lane, left, p);
    if (t.copy != nullptr) store_pairs<WHOLE>(t.copy, t.copy_dtype, base, lane, left, p);
    if constexpr (E4M3) {
        const uint32_t key = mix32(f.key + t.index), block = mix32((uint32_t)(base / ADAM_WARP) + key);
        uint32_t random[ADAM_EACH];
#pragma unroll
        for (int e = 0; e < ADAM_EACH; ++e)
            random[e] = mix32(block + (uint32_t)element<WHOLE>(lane, e) * 0x9E3779B9u);
        encode<false>(m, random, cm, sm);
        encode<true>(r, random, cv, sv);
        store_codes<WHOLE>(t.m, base, lane, left, cm);
        store_codes<WHOLE>(t.v, base, lane, left, cv);
        if (lane == 0) {
            scales[0] = sm;
            scales[1] = sv;
        }
    } else {
        store_pairs<WHOLE>(t.m, TBE_F32, base, lane, left, m);
        store_pairs<WHOLE>(t.v, TBE_F32, base, lane, left, v);
    }
}

#ifndef TBE_ADAM_MINB
#define TBE_ADAM_MINB 6   // blocks an SM: 453 us at 135M parameters; 3 % more at 7, 7 % at 5
#endif
template <bool E4M3, int MOST>
__global__ void __launch_bounds__(256, E4M3 ? TBE_ADAM_MINB : 4) adamw_kernel(const __grid_constant__ AdamArgs<MOST> a) {
    // the tensor of this CTA: the last whose first CTA is not beyond it
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.t[mid].first <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const AdamTensor &t = a.t[lo];
    const int lane = threadIdx.x & 31;
    const int64_t base = (int64_t)(blockIdx.x - t.first) * ADAM_CTA + (threadIdx.x >> 5) * ADAM_WARP;
    if (a.from_device != nullptr) wait_for_launch_before();
    if (base >= t.n) return;
    const int64_t left = t.n - base;
    if (t.whole && left >= ADAM_WARP) adam_block<E4M3, true>(a, t, base, lane, ADAM_WARP);
    else adam_block<E4M3, false>(a, t, base, lane, left < ADAM_WARP ? (int)left : ADAM_WARP);
}

__host__ __device__ inline double power(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) r *= b;
    return r;
}

__host__ __device__ inline AdamFactors factors(double lr, double b1, double b2, double wd, uint32_t seed, int64_t t) {
    if (t < 1) t = 1;
    AdamFactors f;
    f.keep = (float)(1.0 - lr * wd);
    f.rate = (float)(lr / (1.0 - power(b1, t)));
    f.root = (float)(1.0 / sqrt(1.0 - power(b2, t)));
    f.key = step_key(seed, t);
    return f;
}

// The step's numbers where its step or its rate lies on the device.
__global__ void adamw_factors_kernel(const int64_t *step_device, int64_t step, const float *lr_device, double lr,
                                     double b1, double b2, double wd, uint32_t seed, AdamFactors *out) {
    launch_dependents();
    *out = factors(lr_device != nullptr ? (double)*lr_device : lr, b1, b2, wd, seed,
                   step_device != nullptr ? *step_device : step);
}

// ---------------------------------------------------------------------------
// host

constexpr size_t ADAM_WORKSPACE = 256;
constexpr int64_t ADAM_MOST_CTAS = (int64_t)1 << 30;    // of a launch

static tbe_status check_tensor(const tbe_adamw_tensor &t) {
    if (t.n < 0 || t.n > ((int64_t)1 << 40)) return TBE_ERR_INVALID_ARGUMENT;
    if (!known_dtype(t.param_dtype) || !known_dtype(t.grad_dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (t.copy != nullptr && t.copy_dtype != TBE_F16 && t.copy_dtype != TBE_BF16) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (t.state != TBE_STATE_F32 && t.state != TBE_STATE_E4M3) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (t.n == 0) return TBE_OK;
    if (t.param == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr) return TBE_ERR_NULL_POINTER;
    const bool codes = t.state == TBE_STATE_E4M3;
    if (codes && t.scales == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(t.param, dtype_bytes(t.param_dtype)) || !is_aligned(t.grad, dtype_bytes(t.grad_dtype)) ||
        !is_aligned(t.m, codes ? 1 : 4) || !is_aligned(t.v, codes ? 1 : 4) || !is_aligned(t.scales, 4) ||
        !is_aligned(t.copy, 2))
        return TBE_ERR_MISALIGNED;
    return TBE_OK;
}

// Whether what the step writes of a tensor, or into its workspace, lies in another's memory,
// in a gradient's or over the step's numbers (a tensor that is listed twice, as a shared one
// may be, would be updated twice at once).
static bool overlapping(const tbe_adamw_tensor *tensors, int64_t count, const tbe_adamw_options &o, const void *workspace) {
    struct Range {
        uintptr_t from, to;
        bool written;
    };
    static thread_local std::vector<Range> ranges;
    ranges.clear();
    auto range = [&](const void *p, size_t bytes, bool written) {
        if (p != nullptr) ranges.push_back(Range{(uintptr_t)p, (uintptr_t)p + bytes, written});
    };
    range(o.step_device, 8, false);
    range(o.lr_device, 4, false);
    range(o.grad_scale, 4, false);
    if (o.step_device != nullptr || o.lr_device != nullptr) range(workspace, ADAM_WORKSPACE, true);
    for (int64_t i = 0; i < count; ++i) {
        const tbe_adamw_tensor &t = tensors[i];
        if (t.n == 0) continue;
        const bool codes = t.state == TBE_STATE_E4M3;
        range(t.param, (size_t)t.n * dtype_bytes(t.param_dtype), true);
        range(t.grad, (size_t)t.n * dtype_bytes(t.grad_dtype), false);
        range(t.m, (size_t)t.n * (codes ? 1 : 4), true);
        range(t.v, (size_t)t.n * (codes ? 1 : 4), true);
        if (codes) range(t.scales, (size_t)((t.n + ADAM_WARP - 1) / ADAM_WARP) * 8, true);
        range(t.copy, (size_t)t.n * 2, true);
    }
    std::sort(ranges.begin(), ranges.end(), [](const Range &a, const Range &b) { return a.from < b.from; });
    uintptr_t to = 0, written_to = 0;       // where those before end, and the written ones among them
    for (const Range &r : ranges) {
        if (r.from < (r.written ? to : written_to)) return true;
        to = std::max(to, r.to);
        if (r.written) written_to = std::max(written_to, r.to);
    }
    return false;
}

static bool whole(const tbe_adamw_tensor &t) {
    const size_t state = t.state == TBE_STATE_E4M3 ? 4 : 16;
    return is_aligned(t.param, 4 * dtype_bytes(t.param_dtype)) && is_aligned(t.grad, 4 * dtype_bytes(t.grad_dtype)) &&
           is_aligned(t.m, state) && is_aligned(t.v, state) && is_aligned(t.copy, 8);
}

template <int MOST>
static void launch_tensors(Launch &L, const tbe_adamw_tensor *tensors, int64_t count, int state, AdamArgs<MOST> &a) {
    int64_t i = 0;
    while (i < count) {
        // as many tensors as a launch takes
        int64_t blocks = 0;
        a.count = 0;
        for (; i < count && a.count < MOST; ++i) {
            const tbe_adamw_tensor &t = tensors[i];
            if (t.n == 0 || t.state != state) continue;
            const int64_t more = (t.n + ADAM_CTA - 1) / ADAM_CTA;
            if (blocks > 0 && blocks + more > ADAM_MOST_CTAS) break;
            a.t[a.count++] = AdamTensor{t.param, t.grad, t.m, t.v, t.scales, t.copy, t.n, (uint32_t)blocks, (uint32_t)i,
                                        (uint8_t)t.param_dtype, (uint8_t)t.grad_dtype, (uint8_t)t.copy_dtype, whole(t)};
            blocks += more;
        }
        if (a.count == 0) return;
        auto *fn = state == TBE_STATE_E4M3 ? adamw_kernel<true, MOST> : adamw_kernel<false, MOST>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(256);
        cfg.stream = L.stream;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = a.from_device != nullptr;
        void *args[1] = {&a};
        L.before("tbe_adamw");
        cudaLaunchKernelExC(&cfg, (const void *)fn, args);
        L.after();
    }
}

template <int MOST>
static void run_step(Launch &L, const tbe_adamw_tensor *tensors, int64_t count, const tbe_adamw_options &o,
                     void *workspace) {
    static thread_local AdamArgs<MOST> a;      // 32 KB: not on the caller's stack
    a.b1 = (float)o.beta1;
    a.c1 = (float)(1.0 - o.beta1);
    a.b2 = (float)o.beta2;
    a.c2 = (float)(1.0 - o.beta2);
    a.eps = (float)o.eps;
    a.grad_scale = o.grad_scale;
    a.from_device = nullptr;
    if (o.step_device != nullptr || o.lr_device != nullptr) {
        L.before("tbe_adamw_factors");
        adamw_factors_kernel<<<1, 1, 0, L.stream>>>(o.step_device, o.step, o.lr_device, o.lr, o.beta1, o.beta2,
                                                    o.weight_decay, o.seed, (AdamFactors *)workspace);
        L.after();
        a.from_device = (const AdamFactors *)workspace;
    } else {
        a.f = factors(o.lr, o.beta1, o.beta2, o.weight_decay, o.seed, o.step);
    }
    launch_tensors(L, tensors, count, TBE_STATE_F32, a);
    launch_tensors(L, tensors, count, TBE_STATE_E4M3, a);
}

static bool in_range(double x, double lo, double hi) { return x >= lo && x <= hi; }      // not for NaN

}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_adamw_workspace_bytes(void) { return ADAM_WORKSPACE; }

tbe_status tbe_adamw_step(const tbe_adamw_tensor *tensors, int64_t count, const tbe_adamw_options *options,
                          void *workspace, size_t workspace_bytes, const tbe_config *cfg, cudaStream_t stream) {
    if (options == nullptr || (count > 0 && tensors == nullptr)) return TBE_ERR_NULL_POINTER;
    const tbe_adamw_options &o = *options;
    if (count < 0 || count > (int64_t)1 << 24 || !in_range(o.lr, 0.0, 1e30) || !in_range(o.beta1, 0.0, 1.0) ||
        !in_range(o.beta2, 0.0, 1.0) || o.beta1 == 1.0 || o.beta2 == 1.0 || !in_range(o.eps, 0.0, 1e30) ||
        !in_range(o.weight_decay, 0.0, 1e30) || (o.step_device == nullptr && o.step < 1))
        return TBE_ERR_INVALID_ARGUMENT;
    if (!is_aligned(o.step_device, 8) || !is_aligned(o.lr_device, 4) || !is_aligned(o.grad_scale, 4) ||
        !is_aligned(workspace, 256))
        return TBE_ERR_MISALIGNED;
    if (o.step_device != nullptr || o.lr_device != nullptr) {
        if (workspace == nullptr) return TBE_ERR_NULL_POINTER;
        if (workspace_bytes < ADAM_WORKSPACE) return TBE_ERR_BUFFER_TOO_SMALL;
    }
    int64_t some = 0;
    for (int64_t i = 0; i < count; ++i) {
        const tbe_status st = check_tensor(tensors[i]);
        if (st != TBE_OK) return st;
        some += tensors[i].n > 0;
    }
    if (some == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        if (overlapping(tensors, count, o, workspace)) return TBE_ERR_INVALID_ARGUMENT;
        Launch L(stream, cfg);
        if (some <= ADAM_FEW) run_step<ADAM_FEW>(L, tensors, count, o, workspace);
        else run_step<ADAM_MANY>(L, tensors, count, o, workspace);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
