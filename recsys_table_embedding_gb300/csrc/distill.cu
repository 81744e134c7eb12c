// Distillation loss from a teacher's top logits, forward and backward.
//
// Row n has V student logits z, and K teacher entries (id i_k, logit t_k); an
// entry whose id lies outside [0,V) is not part of the row (a list shorter
// than K is filled with -1).  With temperature c
//   p = softmax(t / c) over the row's entries,  q = softmax(z / c) over V,
//   loss = c^2 sum_k p_k (log p_k - log q_{i_k})          (0 log 0 = 0)
//   dz_j = g c (q_j - sum_{k: i_k = j} p_k)               (g: gradient of the loss)
// A row without an entry of positive probability -- a padding position -- has
// loss 0, lse 0 and gradient 0, and its logits are not read.
//
// Numerics: everything in 32 bits; q from the difference to the row's maximum,
// one rounding of the gradient to the logits' type.
#include "token_internal.cuh"

namespace tbe {

constexpr int DISTILL_MAX_K = 1024;
constexpr float LOG2E = 1.44269504088896340736f;

// 2^x by the hardware's approximation (relative error about 2^-22; results
// below 2^-126 are 0).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x/c - y with one rounding at the size of the result: 1/c in two parts.  An
// infinite x keeps its infinity (the second part of 1/c may be 0).
struct Quotient {
    float hi, lo;
    __device__ __forceinline__ explicit Quotient(float c) : hi(1.f / c) { lo = fmaf(-hi, c, 1.f) / c; }
    __device__ __forceinline__ float minus(float x, float y) const {
        return fmaf(fmaxf(x, -3.0e38f), lo, fmaf(x, hi, -y));
    }
};

struct Teacher {
    const void *ids, *logits;
    int index_type, dtype, K;
    float temperature;
};

// Block-wide maximum / sum over T threads (T/32 <= 32 warps); every thread
// gets the result.  `scratch`: 33 floats.
template <int THREADS, bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float w = __shfl_xor_sync(FULL, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    v = lane < THREADS / 32 ? scratch[lane] : (MAX ? -INFINITY : 0.f);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float w = __shfl_xor_sync(FULL, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    return v;
}

// The teacher's entries of a row in shared memory: ids (-1 for none) and
// (t - max) / c, with the log of the sum of their exponentials.  Returns
// whether the row has an entry of positive probability (a NaN counts: it
// reaches the results).  `bad` counts this thread's ids at or beyond V.
template <int THREADS>
__device__ __forceinline__ bool load_teacher(const Teacher &te, int64_t row, int64_t V, int *ids,
                                             float *logp, float *scratch, float *log_sum, int *bad) {
    float high = -INFINITY;
    bool nan = false;
    int count = 0;
    for (int k = threadIdx.x; k < te.K; k += THREADS) {
        const int64_t at = row * te.K + k;
        const int64_t id = load_index(te.ids, te.index_type, at);
        const bool in = id >= 0 && id < V;
        count += id >= V;
        ids[k] = in ? (int)id : -1;
        const float t = in ? load_f32(te.logits, te.dtype, at) : -INFINITY;
        logp[k] = t;
        high = fmaxf(high, t);
        nan |= t != t;
    }
    *bad = count;
    high = block_reduce<THREADS, true>(high, scratch);
    const bool any_nan = __syncthreads_or(nan);
    if (high == -INFINITY && !any_nan) return false;
    float sum = 0.f;
    for (int k = threadIdx.x; k < te.K; k += THREADS) {
        const float d = ids[k] >= 0 ? (logp[k] - high) / te.temperature : -INFINITY;
        logp[k] = d;
        if (ids[k] >= 0) sum += expf(d);
    }
    *log_sum = logf(block_reduce<THREADS, false>(sum, scratch));
    __syncthreads();
    return true;
}

// sum over the entries of row's teacher with the id of entry k, or a negative
// value when an earlier entry has the same id (which then stands for both).
__device__ __forceinline__ float entry_probability(const int *ids, const float *logp, int K, int k,
                                                   float log_sum) {
    const int id = ids[k];
    float p = expf(logp[k] - log_sum);
    for (int j = 0; j < K; ++j) {
        if (ids[j] != id || j == k) continue;
        if (j < k) return -1.f;
        p += expf(logp[j] - log_sum);
    }
    return p;
}

// The part of a row that is read as 16-byte vectors: [head, head + VEC*vectors).
template <typename T> struct RowSpan {
    int64_t head, vectors;
    __device__ __forceinline__ RowSpan(const T *row, int64_t n, int vec) {
        head = vec == 1 ? 0 : ((16 - ((uintptr_t)row & 15)) & 15) / sizeof(T);
        if (head > n) head = n;
        vectors = (n - head) / vec;
    }
};

struct RunningSum {   // maximum and sum of exponentials of a part of a row
    float m, s;
};

// Adds VEC logits to a running maximum and sum: exp((z - m) / c) = 2^((z - m) scale).
template <int VEC>
__device__ __forceinline__ void add_logits(RunningSum &a, const float (&z)[VEC], float scale) {
    float m = a.m;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = fmaxf(m, z[i]);
    if (m > a.m) {
        a.s *= exp2_approx((a.m - m) * scale);   // a.m = -inf: s is 0 and stays 0
        a.m = m;
    }
    const float ref = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int i = 0; i < VEC; ++i) a.s += exp2_approx((z[i] - ref) * scale);
}

constexpr int FWD_THREADS = 512;

template <typename T, int VEC>
__global__ void __launch_bounds__(FWD_THREADS)
distill_forward_kernel(const T *__restrict__ logits, int64_t stride, int64_t V, Teacher te,
                       float *__restrict__ loss, float *__restrict__ lse, int32_t *status) {
    extern __shared__ int32_t smem[];
    int *ids = smem;
    float *logp = (float *)(smem + te.K);
    __shared__ float scratch[33];
    const int64_t row = blockIdx.x;
    const T *z = logits + row * stride;
    const float c = te.temperature, scale = LOG2E / c;
    float log_sum;
    int bad;
    const bool some = load_teacher<FWD_THREADS>(te, row, V, ids, logp, scratch, &log_sum, &bad);
    if (status != nullptr && bad != 0) atomicAdd(status, bad);
    if (!some) {
        if (threadIdx.x == 0) {
            loss[row] = 0.f;
            lse[row] = 0.f;
        }
        return;
    }
    RunningSum a{-INFINITY, 0.f};
    const RowSpan<T> span(z, V, VEC);
    for (int64_t i = threadIdx.x; i < span.vectors; i += FWD_THREADS) {
        float f[VEC];
        widen<T, VEC>(load_raw<T, VEC, true>(z + span.head + i * VEC), f);
        add_logits<VEC>(a, f, scale);
    }
    const int64_t rest = V - span.vectors * VEC;   // head and tail, fewer than two vectors
    for (int64_t i = threadIdx.x; i < rest; i += FWD_THREADS) {
        const float f[1] = {to_f32(z[i < span.head ? i : i + span.vectors * VEC])};
        add_logits<1>(a, f, scale);
    }
    const float m = block_reduce<FWD_THREADS, true>(a.m, scratch);
    const float s = a.s * (a.m == -INFINITY ? 1.f : exp2_approx((a.m - m) * scale));
    const float log_total = logf(block_reduce<FWD_THREADS, false>(s, scratch));
    float part = 0.f;
    for (int k = threadIdx.x; k < te.K; k += FWD_THREADS) {
        if (ids[k] < 0) continue;
        const float lp = logp[k] - log_sum, p = expf(lp);
        if (p == 0.f) continue;
        const float lq = (to_f32(z[ids[k]]) - m) / c - log_total;
        part += p * (lp - lq);
    }
    part = block_reduce<FWD_THREADS, false>(part, scratch);
    if (threadIdx.x == 0) {
        loss[row] = c * c * part;
        lse[row] = m / c + log_total;
    }
}

constexpr int BWD_THREADS = 256;
constexpr int BWD_CHUNK = 8192;   // logits of a row per block

template <typename T, int VEC>
__global__ void __launch_bounds__(BWD_THREADS)
distill_backward_kernel(const T *logits, int64_t stride, int64_t V, Teacher te, const float *__restrict__ lse,
                        const float *__restrict__ grad_loss, float grad_scale, T *grad, int64_t grad_stride) {
    extern __shared__ int32_t smem[];
    int *ids = smem;
    float *logp = (float *)(smem + te.K), *at_id = (float *)(smem + 2 * te.K);
    __shared__ float scratch[33];
    const int64_t row = blockIdx.y;
    const T *z = logits + row * stride;
    T *dz = grad + row * grad_stride;
    // the chunk begins and ends where a vector does, but for the row's ends
    const RowSpan<T> span(z, V, VEC);
    const int64_t lo = blockIdx.x == 0 ? 0 : span.head + (int64_t)blockIdx.x * BWD_CHUNK;
    const int64_t hi = blockIdx.x + 1 == gridDim.x ? V : min(V, span.head + (int64_t)(blockIdx.x + 1) * BWD_CHUNK);
    if (lo >= V) return;
    const float c = te.temperature;
    float log_sum;
    int bad;
    const bool some = load_teacher<BWD_THREADS>(te, row, V, ids, logp, scratch, &log_sum, &bad);
    const float g = (grad_loss != nullptr ? __ldg(grad_loss + row) * grad_scale : grad_scale) * c;
    const Quotient per_c(c);
    const float shift = some ? __ldg(lse + row) : 0.f;
    // q = exp(z/c - lse)
    auto gradient = [&](float x, float p) { return g * (exp2_approx(per_c.minus(x, shift) * LOG2E) - p); };
    // the logits at the teacher's ids, before an in-place gradient replaces them
    for (int k = threadIdx.x; some && k < te.K; k += BWD_THREADS)
        if (ids[k] >= lo && ids[k] < hi) at_id[k] = to_f32(z[ids[k]]);
    __syncthreads();
    const int64_t first = blockIdx.x == 0 ? span.head : lo;
    const int64_t vectors = hi > first ? (hi - first) / VEC : 0;
    for (int64_t i = threadIdx.x; i < vectors; i += BWD_THREADS) {
        float f[VEC];
        if (some) {
            widen<T, VEC>(load_raw<T, VEC, true>(z + first + i * VEC), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = gradient(f[j], 0.f);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = 0.f;
        }
        store_raw<T, VEC>(dz + first + i * VEC, narrow<T, VEC>(f));
    }
    const int64_t tail = first + vectors * VEC, rest = (first - lo) + (hi - tail);
    for (int64_t i = threadIdx.x; i < rest; i += BWD_THREADS) {
        const int64_t j = i < first - lo ? lo + i : tail + i - (first - lo);
        dz[j] = from_f32<T>(some ? gradient(to_f32(z[j]), 0.f) : 0.f);
    }
    if (!some) return;
    __syncthreads();
    // the teacher's entries in this chunk
    for (int k = threadIdx.x; k < te.K; k += BWD_THREADS) {
        const int id = ids[k];
        if (id < lo || id >= hi) continue;
        const float p = entry_probability(ids, logp, te.K, k, log_sum);
        if (p < 0.f) continue;
        dz[id] = from_f32<T>(gradient(at_id[k], p));
    }
}

// ---------------------------------------------------------------------------
// host

static bool same_buffer(const tbe_matrix *a, const tbe_matrix *b) {
    return a->data == b->data && a->stride == b->stride;
}

// first byte and the byte after the last element
static bool overlap(const tbe_matrix *a, const tbe_matrix *b) {
    auto end = [](const tbe_matrix *m) {
        return (uintptr_t)m->data + ((m->rows - 1) * m->stride + m->cols) * dtype_bytes(m->dtype);
    };
    return (uintptr_t)a->data < end(b) && (uintptr_t)b->data < end(a);
}

static tbe_status check_distill(const tbe_matrix *logits, const tbe_teacher *te) {
    tbe_status st = check_matrix(logits, false);
    if (st != TBE_OK) return st;
    if (te == nullptr) return TBE_ERR_NULL_POINTER;
    if (logits->rows >= TOKEN_MAX_ROWS || logits->cols >= ((int64_t)1 << 31) - 1) return TBE_ERR_INVALID_ARGUMENT;
    if (te->K < 1 || te->K > DISTILL_MAX_K || !known_index(te->index_type)) return TBE_ERR_INVALID_ARGUMENT;
    // also refuses a NaN
    if (!(te->temperature >= 1e-6f && te->temperature <= 1e6f)) return TBE_ERR_INVALID_ARGUMENT;
    if (!known_dtype(te->dtype)) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (logits->rows == 0) return TBE_OK;
    if (te->ids == nullptr || te->logits == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(te->ids, te->index_type == TBE_INDEX_I64 ? 8 : 4) ||
        !is_aligned(te->logits, dtype_bytes(te->dtype)))
        return TBE_ERR_MISALIGNED;
    return TBE_OK;
}

static tbe_status check_floats(const void *p, int64_t n) {
    if (n > 0 && p == nullptr) return TBE_ERR_NULL_POINTER;
    return is_aligned(p, 4) ? TBE_OK : TBE_ERR_MISALIGNED;
}

static tbe_status check_gradient(const tbe_matrix *logits, const tbe_matrix *grad, const float *grad_loss) {
    tbe_status st = check_matrix(grad, true);
    if (st != TBE_OK) return st;
    if (grad->rows != logits->rows || grad->cols != logits->cols) return TBE_ERR_INVALID_ARGUMENT;
    if (grad->dtype != logits->dtype) return TBE_ERR_UNSUPPORTED_DTYPE;
    if (!is_aligned(grad_loss, 4)) return TBE_ERR_MISALIGNED;
    if (logits->rows > 0 && !same_buffer(logits, grad) && overlap(logits, grad)) return TBE_ERR_INVALID_ARGUMENT;
    return TBE_OK;
}

static Teacher teacher_of(const tbe_teacher *te) {
    return Teacher{te->ids, te->logits, te->index_type, te->dtype, te->K, te->temperature};
}

// Rows are read as 16-byte vectors between their unaligned ends; the gradient
// with them when its rows start at the same place within 16 bytes.
static bool same_phase(const tbe_matrix *a, const tbe_matrix *b) {
    const int64_t e = dtype_bytes(a->dtype);
    return ((uintptr_t)a->data - (uintptr_t)b->data) % 16 == 0 &&
           (a->rows <= 1 || (a->stride - b->stride) * e % 16 == 0);
}

template <typename T>
static void run_forward(Launch &L, const tbe_matrix *logits, const Teacher &te, float *loss, float *lse,
                        int32_t *status) {
    L.before("tbe_distill_fwd");
    distill_forward_kernel<T, 16 / sizeof(T)><<<(unsigned)logits->rows, FWD_THREADS, (size_t)te.K * 8, L.stream>>>(
        (const T *)logits->data, logits->stride, logits->cols, te, loss, lse, status);
    L.after();
}

template <typename T>
static void run_backward(Launch &L, const tbe_matrix *logits, const Teacher &te, const float *lse,
                         const float *grad_loss, float grad_scale, const tbe_matrix *grad) {
    const unsigned chunks = (unsigned)((logits->cols + BWD_CHUNK - 1) / BWD_CHUNK);
    // rows in slices of the grid's second extent
    for (int64_t r0 = 0; r0 < logits->rows; r0 += 65535) {
        const int64_t n = logits->rows - r0 < 65535 ? logits->rows - r0 : 65535;
        Teacher t = te;
        t.ids = (const char *)te.ids + r0 * te.K * (te.index_type == TBE_INDEX_I64 ? 8 : 4);
        t.logits = (const char *)te.logits + r0 * te.K * dtype_bytes(te.dtype);
        const T *z = (const T *)logits->data + r0 * logits->stride;
        T *dz = (T *)grad->data + r0 * grad->stride;
        const float *gl = grad_loss != nullptr ? grad_loss + r0 : nullptr;
        const dim3 grid(chunks, (unsigned)n);
        L.before("tbe_distill_bwd");
        if (same_phase(logits, grad))
            distill_backward_kernel<T, 16 / sizeof(T)><<<grid, BWD_THREADS, (size_t)te.K * 12, L.stream>>>(
                z, logits->stride, logits->cols, t, lse + r0, gl, grad_scale, dz, grad->stride);
        else
            distill_backward_kernel<T, 1><<<grid, BWD_THREADS, (size_t)te.K * 12, L.stream>>>(
                z, logits->stride, logits->cols, t, lse + r0, gl, grad_scale, dz, grad->stride);
        L.after();
    }
}

}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_distill_forward(const tbe_matrix *logits, const tbe_teacher *teacher, float *loss, float *lse,
                               int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_floats(loss, logits->rows);
    if (st == TBE_OK) st = check_floats(lse, logits->rows);
    if (st == TBE_OK) st = check_floats(dev_status, 0);
    if (st != TBE_OK || logits->rows == 0) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const Teacher te = teacher_of(teacher);
        if (logits->dtype == TBE_F32) run_forward<float>(L, logits, te, loss, lse, dev_status);
        else if (logits->dtype == TBE_F16) run_forward<__half>(L, logits, te, loss, lse, dev_status);
        else run_forward<__nv_bfloat16>(L, logits, te, loss, lse, dev_status);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_distill_backward(const tbe_matrix *logits, const tbe_teacher *teacher, const float *lse,
                                const float *grad_loss, float grad_scale, const tbe_matrix *grad_logits,
                                const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_floats(lse, logits->rows);
    if (st == TBE_OK) st = check_gradient(logits, grad_logits, grad_loss);
    if (st != TBE_OK || logits->rows == 0) return st;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        const Teacher te = teacher_of(teacher);
        if (logits->dtype == TBE_F32) run_backward<float>(L, logits, te, lse, grad_loss, grad_scale, grad_logits);
        else if (logits->dtype == TBE_F16) run_backward<__half>(L, logits, te, lse, grad_loss, grad_scale, grad_logits);
        else run_backward<__nv_bfloat16>(L, logits, te, lse, grad_loss, grad_scale, grad_logits);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

tbe_status tbe_distill_loss_grad(const tbe_matrix *logits, const tbe_teacher *teacher, const float *grad_loss,
                                 float grad_scale, float *loss, float *lse, const tbe_matrix *grad_logits,
                                 int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_gradient(logits, grad_logits, grad_loss);
    if (st != TBE_OK) return st;
    st = tbe_distill_forward(logits, teacher, loss, lse, dev_status, cfg, stream);
    if (st != TBE_OK) return st;
    return tbe_distill_backward(logits, teacher, lse, grad_loss, grad_scale, grad_logits, cfg, stream);
}

}  // extern "C"
