// Distillation loss from a teacher's top logits, forward and backward.
//
// Row n has V student logits z, and K teacher entries (id i_k, logit t_k); an
// entry whose id lies outside [0,V) is not part of the row (a list shorter
// than K is filled with -1).  With temperature c
//   p = softmax(t / c) over the row's entries,  q = softmax(z / c) over V,
//   loss = c^2 sum_k p_k (log p_k - log q_{i_k})          (0 log 0 = 0)
//   dz_j = g c (q_j - sum_{k: i_k = j} p_k)               (g: gradient of the loss)
// A row without an entry of positive probability -- a padding position -- has
// loss 0, lse 0 and gradient 0, whatever its logits are.
//
// Numerics: everything in 32 bits, from differences of logits; one rounding of
// the gradient to the logits' type.
#include "distill_internal.cuh"
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

// What the kernels over the rows need of a row's teacher, made once per call
// by distill_teacher_kernel: the entries with each id once (its probabilities
// added up; id -1 for the others), the logit at the id (which an in-place
// gradient overwrites), their largest logit `ref` and
// cross = sum_k p_k (log p_k - (z_{i_k} - ref) / c), so that, m being the row's
// maximum, loss = c^2 (cross - ((ref - m) / c - log sum_j exp((z_j - m) / c))):
// differences of logits only, whatever their size.
struct TeacherRows {
    int32_t *ids;         // [rows, K]
    float *prob, *at;     // [rows, K]
    float *cross, *ref;   // [rows]
    int32_t *some;        // [rows]: the row has an entry of positive probability
    float *high, *log_sum;   // [rows], for a gradient by another launch than the sum: lse = high / c + log_sum
};

// Sum over the G lanes of a row (G = 32: a warp; else the whole block).
template <int G, bool MAX> __device__ __forceinline__ float row_reduce(float v, float *scratch) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float w = __shfl_xor_sync(FULL, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    if constexpr (G > 32) {
        const int lane = threadIdx.x & 31;
        __syncthreads();
        if (lane == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < G / 32 ? scratch[lane] : (MAX ? -INFINITY : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            const float w = __shfl_xor_sync(FULL, v, o);
            v = MAX ? fmaxf(v, w) : v + w;
        }
    }
    return v;
}

// A row's teacher by G lanes.  `smem`: 3 K4 vectors of 16 bytes (K4 = K / 4
// rounded up); ids, prob, at: [K], not in `smem` but for `at`, which may be its
// last K4 vectors.  The search for equal ids is K^2 comparisons.
struct TeacherSums {
    float cross, ref;
    bool some;
};

template <typename T, int G>
__device__ __forceinline__ TeacherSums reduce_teacher(const T *z_row, int64_t V, const Teacher &te, int64_t row, bool have,
                                                      int lane, int4 *smem, float *scratch, int32_t *out_ids,
                                                      float *out_prob, float *out_at, int32_t *status) {
    const int K = te.K, K4 = (K + 3) / 4;
    int4 *ids4 = smem;
    int *ids = (int *)ids4;   // [4 * K4], -1 beyond K
    float *p = (float *)(ids4 + K4), *z = (float *)(ids4 + 2 * K4);
    int bad = 0;
    float high = -INFINITY;
    bool nan = false;
#pragma unroll 4
    for (int k = lane; k < (have ? K : 0); k += G) {
        const int64_t id = load_index(te.ids, te.index_type, row * K + k);
        const float given = load_f32(te.logits, te.dtype, row * K + k);
        const bool in = id >= 0 && id < V;
        bad += id >= V;
        const float t = in ? given : -INFINITY;
        ids[k] = in ? (int)id : -1;
        p[k] = t;
        high = fmaxf(high, t);
        nan |= t != t;
    }
    for (int k = K + lane; k < 4 * K4; k += G) ids[k] = -1;
    if (status != nullptr && bad != 0) atomicAdd(status, bad);
    high = row_reduce<G, true>(high, scratch);
    const bool any_nan = G == 32 ? __any_sync(FULL, nan) : __syncthreads_or(nan);
    const bool some = high != -INFINITY || any_nan;
    float sum = 0.f, ref = -INFINITY;
#pragma unroll 4
    for (int k = lane; k < (have && some ? K : 0); k += G) {
        const int id = ids[k];
        const float at = to_f32(z_row[max(id, 0)]);
        const float d = id >= 0 ? (p[k] - high) / te.temperature : -INFINITY;   // log of p, but for the sum
        z[k] = at;
        p[k] = d;
        if (id >= 0) sum += expf(d);
        if (d != -INFINITY) ref = fmaxf(ref, at);
    }
    sum = row_reduce<G, false>(sum, scratch);
    ref = row_reduce<G, true>(ref, scratch);
    if (ref == -INFINITY) ref = 0.f;
    const float log_sum = logf(sum);
    if (G == 32) __syncwarp();
    else __syncthreads();
    float cross = 0.f;
    for (int k = lane; have && k < K; k += G) {
        int id = some ? ids[k] : -1;
        float own = 0.f;
        if (id >= 0) {
            const float lp = p[k] - log_sum;
            own = expf(lp);
            if (own != 0.f) cross += own * (lp - (z[k] - ref) / te.temperature);
            out_at[k] = z[k];
            // the first entry of an id stands for all of them; ids are hardly
            // ever given twice, so first only whether one is
            int equal = 0;
#pragma unroll 4
            for (int j = 0; j < K4; ++j) {
                const int4 o = ids4[j];
                equal += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
            }
            for (int j = 0; equal > 1 && j < K; ++j) {
                if (ids[j] != id || j == k) continue;
                if (j < k) {
                    id = -1;
                    break;
                }
                own += expf(p[j] - log_sum);
            }
        }
        out_ids[k] = id;
        out_prob[k] = own;
    }
    cross = row_reduce<G, false>(cross, scratch);
    return TeacherSums{cross, ref, some};
}

// A row's teacher as the kernels over the rows use it: from the workspace, or
// made by the block itself (INSIDE) where rows are few, to save a launch.
struct RowTeacher {
    const int32_t *ids;
    const float *prob, *at;
    float cross, ref;
    bool some;
};

// 16-byte vectors of shared memory per four entries that INSIDE needs
constexpr int INSIDE_VECTORS = 5;

template <typename T, int NT, bool INSIDE>
__device__ __forceinline__ RowTeacher row_teacher(const T *z_row, int64_t V, const Teacher &te, const TeacherRows &rows,
                                                  int64_t row, int4 *smem, float *scratch, int32_t *status) {
    if constexpr (INSIDE) {
        const int K4 = (te.K + 3) / 4;
        int32_t *ids = (int32_t *)(smem + 3 * K4);
        float *prob = (float *)(smem + 4 * K4), *at = (float *)(smem + 2 * K4);
        const TeacherSums t = reduce_teacher<T, NT>(z_row, V, te, row, true, threadIdx.x, smem, scratch, ids, prob, at,
                                                    status);
        __syncthreads();
        return RowTeacher{ids, prob, at, t.cross, t.ref, t.some};
    } else {
        wait_for_launch_before();
        return RowTeacher{rows.ids + row * te.K, rows.prob + row * te.K, rows.at + row * te.K, rows.cross[row],
                          rows.ref[row], rows.some[row] != 0};
    }
}

// Largest of a vector's elements and m (a NaN is passed over; the sum has it).
template <typename T, int VEC> __device__ __forceinline__ float max_of(const Raw<T, VEC> &r, float m) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, __uint_as_float(r.w[i]));
        return m;
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 h = *reinterpret_cast<const T2 *>(&r.w[0]);
#pragma unroll
        for (int i = 1; i < VEC / 2; ++i) h = __hmax2(h, *reinterpret_cast<const T2 *>(&r.w[i]));
        return fmaxf(m, fmaxf(to_f32(h.x), to_f32(h.y)));
    }
}

// The part of a row that is read as 16-byte vectors: [head, head + VEC*vectors).
template <typename T> struct RowSpan {
    int64_t head, vectors;
    __device__ __forceinline__ RowSpan(const T *row, int64_t n) {
        constexpr int VEC = 16 / (int)sizeof(T);
        head = ((16 - ((uintptr_t)row & 15)) & 15) / sizeof(T);
        if (head > n) head = n;
        vectors = (int64_t)((uint64_t)(n - head) / VEC);
    }
};

// ---- sums of exponentials
// exp((z - m) / c) = 2^(z scale - C) with one rounding of the exponent: C, the
// maximum times scale, is the same number in the sum and in the gradient, so
// that its own rounding (the residue) cancels.  Where the product is large the
// residue is too: 2^residue is beyond 32 bits from a product of about 2^31 on.
// From 2^20 on (a residue of 2^-5) the exponent is made of the difference z - m
// instead, at one instruction more per logit.
constexpr float FAR_AWAY = 1048576.f;

struct Exponent {
    float m, C, scale;
    bool far;
    __device__ __forceinline__ Exponent(float m_, float scale_) : scale(scale_) {
        m = m_ == -INFINITY ? 0.f : m_;
        C = m_ * scale;
        far = !(fabsf(C) < FAR_AWAY);
        if (far) C = 0.f;
    }
    template <bool FAR> __device__ __forceinline__ float of(float z) const {
        return exp2_approx(FAR ? (z - m) * scale : fmaf(z, scale, -C));
    }
    // VEC logits' exponentials, two at a time
    template <bool FAR, int VEC> __device__ __forceinline__ void of(float (&z)[VEC]) const {
        if constexpr (FAR || VEC == 1) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) z[i] = of<FAR>(z[i]);
        } else {
            const float2 s2 = make_float2(scale, scale), c2 = make_float2(-C, -C);
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 e = __ffma2_rn(make_float2(z[i], z[i + 1]), s2, c2);
                z[i] = exp2_approx(e.x);
                z[i + 1] = exp2_approx(e.y);
            }
        }
    }
    // what C differs from m scale by
    __device__ __forceinline__ float residue() const { return far ? 0.f : fmaf(m, scale, -C); }
    // a sum of this one's exponentials counts 2^to(whole) times in a sum of whole's
    __device__ __forceinline__ float to(const Exponent &whole) const {
        return far || whole.far ? (m - whole.m) * scale - residue() + whole.residue() : C - whole.C;
    }
};

// A part of a row: its maximum m and s = sum_j exp((z_j - m) / c) (m = 0 there
// for a part whose logits are all -inf).
struct Part {
    float m, s;
};

// The 32 lanes' parts as one.  A part of masked logits only keeps its sum: 0,
// or a NaN.
__device__ __forceinline__ Part join_parts(Part a, float scale) {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    if (a.m != -INFINITY) a.s *= exp2_approx(Exponent(a.m, scale).to(Exponent(m, scale)));
#pragma unroll
    for (int o = 16; o > 0; o /= 2) a.s += __shfl_xor_sync(FULL, a.s, o);
    a.m = m;
    return a;
}

// A thread's part of a row: every STEP-th of `count` vectors, and one element
// of the row's ends (-inf for none), with a running maximum and sum.  STREAM:
// the vectors are not read again.
template <typename T, int STEP, bool STREAM>
__device__ __forceinline__ Part add_part(const T *body, int64_t count, int lane, float edge, float scale) {
    constexpr int VEC = 16 / sizeof(T), B = 4;
    float m = -INFINITY, s = 0.f;
    // raises the running maximum and brings the sum to it
    auto raise = [&](float to) {
        if (!(to > m)) return;
        if (m != -INFINITY) s *= exp2_approx(Exponent(m, scale).to(Exponent(to, scale)));
        m = to;
    };
    for (int64_t i0 = 0; i0 < count; i0 += B * STEP) {
        Raw<T, VEC> r[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (i0 + b * STEP + lane < count) r[b] = load_raw<T, VEC, STREAM>(body + (i0 + b * STEP + lane) * VEC);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (i0 + b * STEP + lane >= count) break;
            raise(max_of<T, VEC>(r[b], -INFINITY));
            float f[VEC];
            widen<T, VEC>(r[b], f);
            const Exponent e(m, scale);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += e.far ? e.of<true>(f[j]) : e.of<false>(f[j]);
        }
    }
    raise(edge);
    const Exponent e(m, scale);
    s += e.far ? e.of<true>(edge) : e.of<false>(edge);
    return Part{m, s};
}

// Element `i` of the row's ends outside its span of vectors, -inf beyond them.
template <typename T> __device__ __forceinline__ float end_of(const T *row, int64_t n, const RowSpan<T> &span, int i) {
    const int64_t tail = span.head + span.vectors * (16 / (int)sizeof(T));
    return i < span.head + n - tail ? to_f32(row[i < span.head ? i : tail + i - span.head]) : -INFINITY;
}

// log of a part's sum, without the maximum
__device__ __forceinline__ float log_of(const Part &a, float scale) {
    return logf(a.s) - Exponent(a.m, scale).residue() * 0.693147180559945f;
}

// lse and loss of a row.
__device__ __forceinline__ void write_loss(const RowTeacher &t, int64_t row, float c, float scale, Part a,
                                           float *loss, float *lse) {
    const float log_total = log_of(a, scale);
    loss[row] = c * c * (t.cross - ((t.ref - a.m) / c - log_total));
    lse[row] = a.m / c + log_total;
}

// ---------------------------------------------------------------------------
// The teachers of all rows.  Bound by latency: an entry's id, then the logit
// there.  A block takes a row beyond K = 256.  The logits are gathered here and
// not by the kernels over the rows, where they lengthen every block's way to its
// sum.  2048 x 128 entries out of 537 MB of logits take 18 us, the time of as many
// reads at random places; 4096 x 64 12-17 us.
//
// For a gradient from a stored lse (LSE) it also says how to take differences
// with it.  A number of 32 bits holds an lse to 2^-24 of its size, and the
// gradient's exponentials are off by as much: below LSE_MOST by 2^-19 at most.
// Beyond (large logits, small temperatures) the row's maximum and sum are made
// again here, by the lanes that have the row, before anything overwrites its
// logits: one more read of such rows (a gradient of 1000 x 50,021 f16 takes 105 us
// then, 44 otherwise; 2048 x 50,257 bf16 148 and 113).
constexpr float LSE_MOST = 64.f;

template <typename T, int G, bool LSE>
__global__ void __launch_bounds__(256)
distill_teacher_kernel(const T *__restrict__ logits, int64_t stride, int64_t rows, int64_t V, Teacher te,
                       TeacherRows out, const float *__restrict__ lse, int32_t *status) {
    constexpr int ROWS = 256 / G;
    extern __shared__ int4 teacher_smem[];
    __shared__ float scratch[8];
    __shared__ Part parts[8];
    launch_dependents();
    const int group = threadIdx.x / G, lane = threadIdx.x % G, K = te.K, K4 = (K + 3) / 4;
    const int64_t row = (int64_t)blockIdx.x * ROWS + group;
    const T *z = logits + row * stride;
    const TeacherSums t = reduce_teacher<T, G>(z, V, te, row, row < rows, lane, teacher_smem + group * 3 * K4, scratch,
                                               out.ids + row * K, out.prob + row * K, out.at + row * K, status);
    if (row >= rows) return;
    if (lane == 0) {
        out.cross[row] = t.cross;
        out.ref[row] = t.ref;
        out.some[row] = t.some;
    }
    if constexpr (LSE) {
        float high = 0.f, log_sum = t.some ? lse[row] : 0.f;
        if (!(fabsf(log_sum) <= LSE_MOST)) {   // the lanes of a row agree
            const float scale = LOG2E / te.temperature;
            const RowSpan<T> span(z, V);
            Part a = join_parts(add_part<T, G, true>(z + span.head, span.vectors, lane, end_of(z, V, span, lane), scale), scale);
            if constexpr (G > 32) {
                if ((lane & 31) == 0) parts[lane >> 5] = a;
                __syncthreads();
                a = join_parts((lane & 31) < G / 32 ? parts[lane & 31] : Part{-INFINITY, 0.f}, scale);
            }
            high = a.m;
            log_sum = log_of(a, scale);
        }
        if (lane == 0) {
            out.high[row] = high;
            out.log_sum[row] = log_sum;
        }
    }
}

// ---------------------------------------------------------------------------
// Loss alone, for rows of any length: one block per row, a running maximum
// and sum per thread.  Bound by the one read of the logits: 2048 x 65,536 f32
// take 82 us, 6.5 TB/s.
constexpr int FWD_THREADS = 512;

template <typename T, bool INSIDE>
__global__ void __launch_bounds__(FWD_THREADS)
distill_forward_kernel(const T *__restrict__ logits, int64_t stride, int64_t V, Teacher te, TeacherRows rows,
                       float *__restrict__ loss, float *__restrict__ lse, int32_t *status) {
    extern __shared__ int4 teacher_smem[];
    __shared__ float scratch[FWD_THREADS / 32];
    constexpr int WARPS = FWD_THREADS / 32;
    __shared__ Part parts[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const float c = te.temperature;
    const RowTeacher t = row_teacher<T, FWD_THREADS, INSIDE>(logits + row * stride, V, te, rows, row, teacher_smem,
                                                             scratch, status);
    if (!t.some) {
        if (tid == 0) {
            loss[row] = 0.f;
            lse[row] = 0.f;
        }
        return;
    }
    const float scale = LOG2E / c;
    const T *z = logits + row * stride;
    const RowSpan<T> span(z, V);
    Part a = join_parts(add_part<T, FWD_THREADS, true>(z + span.head, span.vectors, tid, end_of(z, V, span, tid), scale), scale);
    if (lane == 0) parts[warp] = a;
    __syncthreads();
    if (warp != 0) return;
    a = join_parts(lane < WARPS ? parts[lane] : Part{-INFINITY, 0.f}, scale);
    if (lane == 0) {
        write_loss(t, row, c, scale, a, loss, lse);
        if (!INSIDE) {
            rows.high[row] = a.m;
            rows.log_sum[row] = log_of(a, scale);
        }
    }
}

// ---------------------------------------------------------------------------
// Loss and gradient at once: rows held in shared memory.  A CTA holds a slice
// of a row, brought in by one bulk copy, so that the row is read from memory
// once for its sum and its gradient; rows of more than a slice are spread over
// a cluster of CTAs, which send one (maximum, sum) each to the others' shared
// memory.  Bound by one read and one write of the logits: nothing waits for
// the copy but its own CTA, and several CTAs per SM are in different phases.
// 4096 x 131,072 bf16, one row in 20 without an entry (2.1 GB): 352 us, 6.0
// TB/s; 1000 x 50,021 f16: 35 us.  (In an earlier form, at 368 us, slices in
// registers took 415 us; clusters that stay and bring the next row's slice while
// they work on one 444: two slices a CTA leave three CTAs an SM, which wait for
// their exchanges.)

constexpr int MAX_CLUSTER = 8;

// The slice of a row that a CTA owns: `count` vectors from element `body` on,
// and the row's unaligned ends in the first and the last slice.
template <typename T> struct Slice {
    int64_t body, edge_at;   // edge_at: the end element of thread tid < edges
    int count, edges;
    int64_t lo, hi;          // all its elements
    __device__ __forceinline__ Slice(const T *row, int64_t V, int rank, int slices, int per_slice, int tid) {
        constexpr int VEC = 16 / sizeof(T);
        const RowSpan<T> span(row, V);
        const int64_t v0 = min(span.vectors, (int64_t)rank * per_slice), v1 = min(span.vectors, v0 + per_slice);
        const bool first = rank == 0, last = rank + 1 == slices;
        const int64_t tail = span.head + span.vectors * VEC;
        const int heads = first ? (int)span.head : 0;
        count = (int)(v1 - v0);
        body = span.head + v0 * VEC;
        edges = heads + (last ? (int)(V - tail) : 0);
        edge_at = tid < heads ? tid : tail + tid - heads;
        lo = first ? 0 : body;
        hi = last ? V : body + (int64_t)count * VEC;
    }
};

template <typename T>
__device__ __forceinline__ void write_zeros(T *dz, const Slice<T> &sl, int tid, int threads) {
    constexpr int VEC = 16 / sizeof(T);
    Raw<T, VEC> zero;
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::WORDS; ++i) zero.w[i] = 0;
    for (int i = tid; i < sl.count; i += threads) store_raw<T, VEC>(dz + sl.body + (int64_t)i * VEC, zero);
    if (tid < sl.edges) dz[sl.edge_at] = from_f32<T>(0.f);
}

// The warps' parts as the row's, through the cluster; called once or twice
// after a first cluster_arrive (where there is more than one slice).
template <int WARPS>
__device__ __forceinline__ Part join_row(Part a, bool first, float scale, Part *parts, Part (*cta_parts)[MAX_CLUSTER],
                                         int slices, int rank) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) parts[warp] = a;
    __syncthreads();
    a = join_parts(lane < WARPS ? parts[lane] : Part{-INFINITY, 0.f}, scale);
    if (slices > 1) {
        if (first) cluster_wait();   // every CTA of the cluster runs
        Part *to = cta_parts[first ? 0 : 1];
        if (warp == 0) {
            if (lane < slices) {
                cluster_store(&to[rank].m, lane, a.m);
                cluster_store(&to[rank].s, lane, a.s);
            }
            __syncwarp();
            cluster_arrive<true>();
        } else {
            cluster_arrive<false>();
        }
        cluster_wait();
        a = join_parts(lane < slices ? to[lane] : Part{-INFINITY, 0.f}, scale);
    }
    return a;
}

// A copy that is not there within the limit of waits leaves NaN in its row's
// loss, lse and gradient, flagged or not (status may be NULL); the CTA waits for
// it once more, as long, before it ends.  WITHHELD, for the self-test of that
// limit: the copies are waited for, but not issued.
template <typename T, int NT, bool INSIDE, bool WITHHELD = false>
__global__ void __launch_bounds__(NT, NT == 128 ? 7 : 1536 / NT)
distill_rows_kernel(const T *logits, int64_t stride, int64_t V, Teacher te, TeacherRows rows,
                    const float *__restrict__ grad_loss, float grad_scale, float *loss, float *lse, T *grad,
                    int64_t grad_stride, uint32_t slices, int per_slice, int32_t *status) {
    constexpr int VEC = 16 / sizeof(T), WARPS = NT / 32;
    extern __shared__ __align__(128) unsigned char held[];
    __shared__ Part parts[WARPS], cta_parts[2][MAX_CLUSTER];
    __shared__ float scratch[WARPS];
    __shared__ __align__(8) uint64_t arrived;
    const T *mine = reinterpret_cast<const T *>(held);
    const int tid = threadIdx.x;
    const uint32_t row = blockIdx.x / slices;
    const int rank = (int)(blockIdx.x - row * slices);   // of the slice in its row: the CTA's rank in the cluster
    const T *z = logits + row * stride;
    T *dz = grad + row * grad_stride;
    const Slice<T> sl(z, V, rank, (int)slices, per_slice, tid);
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&arrived);
    if (tid == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n\tfence.proxy.async.shared::cta;" ::"r"(bar) : "memory");
    }
    const float c = te.temperature;
    auto bring = [&]() {
        if (tid != 0 || sl.count == 0) return;
        const uint32_t bytes = (uint32_t)sl.count * 16;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
        if (WITHHELD) return;
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(held)),
                     "l"(z + sl.body), "r"(bytes), "r"(bar)
                     : "memory");
    };
    if (INSIDE) bring();   // beside the teacher, whether or not it has an entry
    const RowTeacher t = row_teacher<T, NT, INSIDE>(z, V, te, rows, row, (int4 *)(held + (size_t)per_slice * 16), scratch,
                                                    rank == 0 ? status : nullptr);
    if (!INSIDE && t.some) bring();
    if (!INSIDE) __syncthreads();   // the barrier is ready (row_teacher has waited for all otherwise)
    // waits for the slice; one that is late is flagged and waited for again
    auto wait_copy = [&]() {
        if (sl.count == 0 || mbar_wait_bounded(bar, 0)) return true;
        if (status != nullptr) atomicOr(status + 1, TBE_FLAG_COPY_TIMEOUT);
        mbar_wait_bounded(bar, 0);
        return false;
    };
    if (!t.some) {   // all CTAs of a row agree
        if (INSIDE) wait_copy();   // the copy must not outlive the CTA
        write_zeros(dz, sl, tid, NT);
        if (rank == 0 && tid == 0) {
            loss[row] = 0.f;
            lse[row] = 0.f;
        }
        return;
    }
    if (slices > 1) cluster_arrive<false>();   // waited for before the first store to another CTA
    float edge = -INFINITY;
    if (tid < sl.edges) edge = to_f32(z[sl.edge_at]);
    const float g = (grad_loss != nullptr ? __ldg(grad_loss + row) * grad_scale : grad_scale) * c;
    const float scale = LOG2E / c;
    const float late = wait_copy() ? 0.f : NAN;   // a thread's share of a late slice

    // sum of a thread's exponentials
    auto add = [&](const Exponent &e, auto far) {
        constexpr bool FAR = decltype(far)::value;
        float2 s = make_float2(e.of<FAR>(edge), 0.f);
#pragma unroll 4
        for (int i = tid; i < sl.count; i += NT) {
            float f[VEC];
            widen<T, VEC>(load_raw<T, VEC>(mine + i * VEC), f);
            e.of<FAR>(f);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) s = __fadd2_rn(s, make_float2(f[j], f[j + 1]));
        }
        float sum = s.x + s.y + late;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(FULL, sum, o);
        return sum;
    };
    auto join = [&](Part a, bool first) {
        return join_row<WARPS>(a, first, scale, parts, cta_parts, (int)slices, rank);
    };
    // The teacher's largest logit stands for the row's maximum: one pass over
    // the slice.  Where that is not near (the sum tells, to all CTAs alike), or
    // something is not finite, the maximum is looked for.
    const Exponent guess(t.ref, scale);
    Part a = join(Part{t.ref, guess.far ? INFINITY : add(guess, std::false_type())}, true);
    if (!(a.s >= 0.0625f && a.s <= 1048576.f)) {
        float wm = edge;
#pragma unroll 4
        for (int i = tid; i < sl.count; i += NT) wm = max_of<T, VEC>(load_raw<T, VEC>(mine + i * VEC), wm);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) wm = fmaxf(wm, __shfl_xor_sync(FULL, wm, o));
        const Exponent we(wm, scale);
        const float ws = we.far ? add(we, std::true_type()) : add(we, std::false_type());
        __syncthreads();   // `parts` have been read
        a = join(Part{wm, ws}, false);
    }
    const float factor = g / a.s;
    if (rank == 0 && tid == 0) write_loss(t, row, c, scale, a, loss, lse);

    const Exponent e(a.m, scale);
    auto write = [&](auto far) {
        constexpr bool FAR = decltype(far)::value;
#pragma unroll 2
        for (int i = tid; i < sl.count; i += NT) {
            float f[VEC];
            widen<T, VEC>(load_raw<T, VEC>(mine + i * VEC), f);
            e.of<FAR>(f);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {   // g q
                const float2 q = __fmul2_rn(make_float2(f[j], f[j + 1]), make_float2(factor, factor));
                f[j] = q.x;
                f[j + 1] = q.y;
            }
            store_raw<T, VEC>(dz + sl.body + (int64_t)i * VEC, narrow<T, VEC>(f));
        }
        if (tid < sl.edges) dz[sl.edge_at] = from_f32<T>(factor * e.of<FAR>(edge));
        __syncthreads();   // the entries' gradients replace what their vectors' owners wrote
        for (int k = tid; k < te.K; k += NT) {
            const int id = t.ids[k];
            if (id >= 0 && id >= sl.lo && id < sl.hi)
                dz[id] = from_f32<T>(factor * e.of<FAR>(t.at[k]) - g * t.prob[k]);
        }
    };
    if (e.far) write(std::true_type());
    else write(std::false_type());
}

// q = 2^(((z - high) / c - log_sum) log2 e), by a row's sum that another launch
// made: its maximum and log of the sum, or 0 and a stored lse.
struct KnownSum {
    float high, log_sum;
    Quotient per_c;
    __device__ __forceinline__ KnownSum(float high_, float log_sum_, float c) : high(high_), log_sum(log_sum_), per_c(c) {}
    __device__ __forceinline__ float probability(float z) const {
        return exp2_approx(per_c.minus(z - high, log_sum) * LOG2E);
    }
};

// Loss and gradient for rows longer than a cluster holds, and few rows whose
// gradient starts at another place within 16 bytes than the logits (together =
// false): slices are read twice, for the sum and for the gradient, the second
// time mostly from L2, and gradients of another place are written element by
// element.  40 x 900,001 bf16: 64 us (by a launch for the loss and one for the
// gradient 107), 512 x 500,000 f32: 435 (527); 7 x 32,003 f32 at another place 12
// (25).  Many rows at another place are faster by two launches: 1000 x 50,021 f16
// take 87 us, 117 this way.
//
// It is also the gradient of few rows from a stored lse (`loss` NULL), read
// once where the lse is precise enough: 16 x 131,072 bf16 12 us (16 where it is
// not).
//
// Every CTA reads and writes its own slice only (what it reads of the others'
// for the teacher stays unused), so the gradient may replace the logits.
constexpr int STREAM_THREADS = 512;

template <typename T, bool INSIDE>
__global__ void __launch_bounds__(STREAM_THREADS, 2)
distill_stream_kernel(const T *logits, int64_t stride, int64_t V, Teacher te, TeacherRows rows,
                      const float *__restrict__ grad_loss, float grad_scale, float *loss, float *lse, T *grad,
                      int64_t grad_stride, uint32_t slices, int per_slice, bool together, int32_t *status) {
    constexpr int VEC = 16 / sizeof(T), NT = STREAM_THREADS, WARPS = NT / 32, B = 8;
    extern __shared__ int4 teacher_smem[];
    __shared__ Part parts[WARPS], cta_parts[2][MAX_CLUSTER];
    __shared__ float scratch[WARPS];
    const int tid = threadIdx.x;
    const uint32_t row = blockIdx.x / slices;
    const int rank = (int)(blockIdx.x - row * slices);
    const T *z = logits + row * stride;
    T *dz = grad + row * grad_stride;
    const Slice<T> sl(z, V, rank, (int)slices, per_slice, tid);
    const float c = te.temperature;
    const RowTeacher t = row_teacher<T, NT, INSIDE>(z, V, te, rows, row, teacher_smem, scratch, rank == 0 ? status : nullptr);
    if (!t.some) {   // all CTAs of a row agree
        if (together) write_zeros(dz, sl, tid, NT);
        else for (int64_t j = sl.lo + tid; j < sl.hi; j += NT) dz[j] = from_f32<T>(0.f);
        if (rank == 0 && tid == 0 && loss != nullptr) {
            loss[row] = 0.f;
            lse[row] = 0.f;
        }
        return;
    }
    const float edge = tid < sl.edges ? to_f32(z[sl.edge_at]) : -INFINITY;
    const float g = (grad_loss != nullptr ? __ldg(grad_loss + row) * grad_scale : grad_scale) * c;
    const float scale = LOG2E / c;
    auto write = [&](auto weighted) {   // g q of a logit
        if (together) {
            for (int i0 = tid; i0 < sl.count; i0 += B * NT) {
                Raw<T, VEC> r[B];
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (i0 + b * NT < sl.count) r[b] = load_raw<T, VEC, true>(z + sl.body + (int64_t)(i0 + b * NT) * VEC);
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (i0 + b * NT >= sl.count) break;
                    float f[VEC];
                    widen<T, VEC>(r[b], f);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) f[j] = weighted(f[j]);
                    store_raw<T, VEC>(dz + sl.body + (int64_t)(i0 + b * NT) * VEC, narrow<T, VEC>(f));
                }
            }
            if (tid < sl.edges) dz[sl.edge_at] = from_f32<T>(weighted(edge));
        } else {
            for (int64_t j0 = sl.lo + tid; j0 < sl.hi; j0 += B * NT) {
                T x[B];
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (j0 + b * NT < sl.hi) x[b] = z[j0 + b * NT];
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (j0 + b * NT < sl.hi) dz[j0 + b * NT] = from_f32<T>(weighted(to_f32(x[b])));
            }
        }
        __syncthreads();   // the entries' gradients replace what others wrote
        for (int k = tid; k < te.K; k += NT) {
            const int id = t.ids[k];
            if (id >= 0 && id >= sl.lo && id < sl.hi) dz[id] = from_f32<T>(weighted(t.at[k]) - g * t.prob[k]);
        }
    };
    if (loss == nullptr && fabsf(lse[row]) <= LSE_MOST) {   // here too
        const KnownSum q(0.f, lse[row], c);
        write([&](float x) { return g * q.probability(x); });
        return;
    }
    if (slices > 1) cluster_arrive<false>();
    const Part a = join_row<WARPS>(join_parts(add_part<T, NT, false>(z + sl.body, sl.count, tid, edge, scale), scale), true,
                                   scale, parts, cta_parts, (int)slices, rank);
    const float factor = g / a.s;
    if (rank == 0 && tid == 0 && loss != nullptr) write_loss(t, row, c, scale, a, loss, lse);
    const Exponent e(a.m, scale);
    if (e.far) write([&](float x) { return factor * e.template of<true>(x); });
    else write([&](float x) { return factor * e.template of<false>(x); });
}

// ---------------------------------------------------------------------------
// Gradient of many rows by sums that another launch made: from a stored lse (the
// teachers' launch says how), or after the loss.
//
// The slices of a row are independent; R vectors per thread are on their way
// at once.  2048 x 65,536 f32 (1.05 GB read and written): 149 us, 7.0 TB/s.
template <typename T, int R>
__global__ void __launch_bounds__(256, 4)
distill_backward_kernel(const T *logits, int64_t stride, int64_t V, Teacher te, TeacherRows rows,
                        const float *__restrict__ grad_loss, float grad_scale, T *grad, int64_t grad_stride,
                        uint32_t slices, int per_slice) {
    constexpr int VEC = 16 / sizeof(T), NT = 256;
    const int tid = threadIdx.x;
    const uint32_t row = blockIdx.x / slices;
    const T *z = logits + row * stride;
    T *dz = grad + row * grad_stride;
    const Slice<T> sl(z, V, (int)(blockIdx.x - row * slices), (int)slices, per_slice, tid);
    const RowTeacher t = row_teacher<T, NT, false>(z, V, te, rows, row, nullptr, nullptr, nullptr);
    if (!t.some) {
        write_zeros(dz, sl, tid, NT);
        return;
    }
    Raw<T, VEC> r[R];
    float edge = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i * NT + tid < sl.count) r[i] = load_raw<T, VEC, true>(z + sl.body + (int64_t)(i * NT + tid) * VEC);
    if (tid < sl.edges) edge = to_f32(z[sl.edge_at]);
    const float g = (grad_loss != nullptr ? __ldg(grad_loss + row) * grad_scale : grad_scale) * te.temperature;
    const KnownSum q(rows.high[row], rows.log_sum[row], te.temperature);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i * NT + tid >= sl.count) break;
        float f[VEC];
        widen<T, VEC>(r[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = g * q.probability(f[j]);
        store_raw<T, VEC>(dz + sl.body + (int64_t)(i * NT + tid) * VEC, narrow<T, VEC>(f));
    }
    if (tid < sl.edges) dz[sl.edge_at] = from_f32<T>(g * q.probability(edge));
    __syncthreads();   // the entries' gradients replace what their vectors' owners wrote
    for (int k = tid; k < te.K; k += NT) {
        const int id = t.ids[k];
        if (id >= 0 && id >= sl.lo && id < sl.hi) dz[id] = from_f32<T>(g * q.probability(t.at[k]) - g * t.prob[k]);
    }
}

// Gradient rows that start at another place within 16 bytes than the logits'
// rows do, element by element.
constexpr int SCALAR_THREADS = 256;
constexpr int SCALAR_CHUNK = 8192;   // logits of a row per block

template <typename T>
__global__ void __launch_bounds__(SCALAR_THREADS)
distill_scalar_kernel(const T *__restrict__ logits, int64_t stride, int64_t V, Teacher te, TeacherRows rows,
                      const float *__restrict__ grad_loss, float grad_scale, T *__restrict__ grad, int64_t grad_stride,
                      uint32_t slices) {
    const uint32_t row = blockIdx.x / slices;
    const T *z = logits + row * stride;
    T *dz = grad + row * grad_stride;
    const int64_t lo = (int64_t)(blockIdx.x - row * slices) * SCALAR_CHUNK, hi = min(V, lo + SCALAR_CHUNK);
    const RowTeacher t = row_teacher<T, SCALAR_THREADS, false>(z, V, te, rows, row, nullptr, nullptr, nullptr);
    const float g = (grad_loss != nullptr ? __ldg(grad_loss + row) * grad_scale : grad_scale) * te.temperature;
    const KnownSum q(rows.high[row], rows.log_sum[row], te.temperature);
    for (int64_t j = lo + threadIdx.x; j < hi; j += SCALAR_THREADS)
        dz[j] = from_f32<T>(t.some ? g * q.probability(to_f32(z[j])) : 0.f);
    if (!t.some) return;
    __syncthreads();
    for (int k = threadIdx.x; k < te.K; k += SCALAR_THREADS) {
        const int id = t.ids[k];
        if (id >= 0 && id >= lo && id < hi) dz[id] = from_f32<T>(g * q.probability(t.at[k]) - g * t.prob[k]);
    }
}

// ---------------------------------------------------------------------------
// host

static bool same_buffer(const tbe_matrix *a, const tbe_matrix *b) {
    return a->data == b->data && a->stride == b->stride;
}

// Whether two matrices of one shape may share an element: where one's bytes lie
// apart from the other's, or the rows of both have one stride and lie in
// between one another, they do not.
static bool overlap(const tbe_matrix *a, const tbe_matrix *b) {
    const uintptr_t e = dtype_bytes(a->dtype), p = (uintptr_t)a->data, q = (uintptr_t)b->data;
    const uintptr_t row = a->cols * e, stride = a->stride * e;
    auto bytes = [&](const tbe_matrix *m) { return ((m->rows - 1) * m->stride + m->cols) * e; };
    if (p >= q + bytes(b) || q >= p + bytes(a)) return false;
    if (a->stride != b->stride || stride == 0) return true;
    const uintptr_t gap = p > q ? (stride - (p - q) % stride) % stride : (q - p) % stride;   // a row of b after one of a
    return gap < row || stride - gap < row;
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

// Rows are read as 16-byte vectors between their unaligned ends; the gradient
// with them when its rows start at the same place within 16 bytes.
static bool same_phase(const tbe_matrix *a, const tbe_matrix *b) {
    const int64_t e = dtype_bytes(a->dtype);
    return ((uintptr_t)a->data - (uintptr_t)b->data) % 16 == 0 &&
           (a->rows <= 1 || (a->stride - b->stride) * e % 16 == 0);
}

// Launch shape of distill_rows_kernel for rows of `vectors` 16-byte vectors:
// CTAs per row and threads per CTA; 0 slices: longer than a cluster holds.
// Bytes of a slice aimed at: six CTAs per SM.  Calls with their teachers' launch,
// in us, with slices of at most 24, 32, 48 and 64 KB: 4096 x 131,072 bf16 378, 377,
// 377, 391; 1000 x 50,021 f16 62 (eight CTAs a row), 48, 48, 50; 2048 x 32,000 bf16
// 70, 58, 58, 55; 2048 x 65,536 f32 188, 188, 188, 187.
constexpr int64_t SLICE_BYTES = 32768;
constexpr int64_t SLICE_MOST = 200 * 1024;            // one CTA per SM
constexpr int64_t SMEM_MOST = SLICE_MOST + 21 * 1024;  // and a teacher of 256 entries
struct RowShape {
    int slices, threads;
};

static int row_slices(int64_t vectors, int64_t rows, int sms) {
    int n = 1;
    while (n < MAX_CLUSTER && vectors * 16 > SLICE_BYTES * n) n *= 2;
    // few rows: more CTAs for each
    while (n < MAX_CLUSTER && rows * n * 2 <= sms && vectors >= 512 * n) n *= 2;
    return n;
}

static RowShape row_shape(int64_t vectors, int64_t rows, int sms) {
    RowShape s{row_slices(vectors, rows, sms), 128};
    const int64_t bytes = (vectors + s.slices - 1) / s.slices * 16;
    if (bytes > SLICE_MOST) s.slices = 0;
    // few threads with many vectors each: what a warp does once per slice
    // weighs less.  128, 256, 512 and 1024 threads, us: 32 KB, the 16-bit rows above,
    // 377 and 389, 48 and 52, 58 and 59; 64 KB, 2048 x 131,072 f32, 371, 377, 401,
    // 926; 100 KB, 512 x 200,000 f32, 156, 154, 162, 285; 200 KB, 256 x 400,000 f32,
    // 211, 203, 205, 215.
    s.threads = bytes <= 36 * 1024 ? 128 : bytes <= 72 * 1024 ? 256 : bytes <= 110 * 1024 ? 512 : 1024;
    return s;
}

constexpr int64_t MAX_GRID = ((int64_t)1 << 31) - 1;

// Few rows: every block makes its row's teacher itself.  Loss and gradient so, and
// with the teachers' launch, in us: 64 x 32,003 f32 12 and 15 (K = 10), 13 and 17
// (64), 17 and 42 (256); 64 x 131,072 bf16 16 and 18, 16 and 21, 23 and 44.  At 512
// rows it is slower for small K: 41 and 35, 41 and 38, 51 and 62; between, it
// depends on K.
static bool teacher_inside(int64_t rows, int K) { return rows <= 64 && K <= 256; }
static size_t inside_bytes(int K) { return (size_t)(K + 3) / 4 * INSIDE_VECTORS * 16; }

static size_t teacher_bytes(int64_t rows, int K) {
    return teacher_inside(rows, K) ? 0 : round_up((size_t)rows * (12 * (size_t)K + 20), 256);
}

// The teacher's entries of every row in the workspace; with `lse` also how the
// gradient takes differences with it.
template <typename T>
static TeacherRows run_teacher(Launch &L, const tbe_matrix *logits, const Teacher &te, void *ws, const float *lse,
                               int32_t *status) {
    const int64_t rows = logits->rows, n = rows * te.K;
    TeacherRows out;
    out.ids = (int32_t *)ws;
    out.prob = (float *)(out.ids + n);
    out.at = out.prob + n;
    out.cross = out.at + n;
    out.ref = out.cross + rows;
    out.some = (int32_t *)(out.ref + rows);
    out.high = (float *)(out.some + rows);
    out.log_sum = out.high + rows;
    const size_t smem = (size_t)((te.K + 3) / 4) * 48;   // of a row
    const bool warps = te.K <= 256;
    auto *fn = warps ? (lse != nullptr ? distill_teacher_kernel<T, 32, true> : distill_teacher_kernel<T, 32, false>)
                     : (lse != nullptr ? distill_teacher_kernel<T, 256, true> : distill_teacher_kernel<T, 256, false>);
    L.before("tbe_distill_teacher");
    fn<<<(unsigned)(warps ? (rows + 7) / 8 : rows), 256, warps ? 8 * smem : smem, L.stream>>>(
        (const T *)logits->data, logits->stride, rows, logits->cols, te, out, lse, status);
    L.after();
    return out;
}

template <typename T, bool INSIDE>
static void run_forward(Launch &L, const tbe_matrix *logits, const Teacher &te, const TeacherRows &rows, float *loss,
                        float *lse, int32_t *status) {
    launch_with(L, "tbe_distill_fwd", !INSIDE, 1, distill_forward_kernel<T, INSIDE>, dim3((unsigned)logits->rows),
                FWD_THREADS, INSIDE ? inside_bytes(te.K) : 0, (const T *)logits->data, logits->stride, logits->cols, te,
                rows, loss, lse, status);
}

template <typename T>
static tbe_status run_backward(Launch &L, const tbe_matrix *logits, const Teacher &te, const TeacherRows &rows,
                               const float *grad_loss, float grad_scale, const tbe_matrix *grad) {
    const int64_t N = logits->rows, V = logits->cols;
    const T *z = (const T *)logits->data;
    T *dz = (T *)grad->data;
    if (same_phase(logits, grad)) {
        const int64_t vectors = V / (16 / (int)sizeof(T));
        const int R = vectors <= 512 ? 2 : 8;
        const int64_t slices = vectors <= 256 * R ? 1 : (vectors + 256 * R - 1) / (256 * R);
        if (N > MAX_GRID / slices) return TBE_ERR_INVALID_ARGUMENT;
        launch_with(L, "tbe_distill_bwd", true, 1, R == 2 ? distill_backward_kernel<T, 2> : distill_backward_kernel<T, 8>,
                    dim3((unsigned)(N * slices)), 256, 0, z, logits->stride, V, te, rows, grad_loss, grad_scale, dz,
                    grad->stride, (uint32_t)slices, (int)((vectors + slices - 1) / slices));
        return TBE_OK;
    }
    const int64_t slices = (V + SCALAR_CHUNK - 1) / SCALAR_CHUNK;
    if (N > MAX_GRID / slices) return TBE_ERR_INVALID_ARGUMENT;
    launch_with(L, "tbe_distill_scalar", true, 1, distill_scalar_kernel<T>, dim3((unsigned)(N * slices)), SCALAR_THREADS, 0,
                z, logits->stride, V, te, rows, grad_loss, grad_scale, dz, grad->stride, (uint32_t)slices);
    return TBE_OK;
}

// Loss and gradient; or, with `loss` NULL, the gradient of few rows from their lse.
template <typename T, bool INSIDE>
static tbe_status run_loss_grad(Launch &L, const tbe_matrix *logits, const Teacher &te, const TeacherRows &rows,
                                const float *grad_loss, float grad_scale, float *loss, float *lse,
                                const tbe_matrix *grad, int32_t *status) {
    const int64_t vectors = logits->cols / (16 / (int)sizeof(T));
    const RowShape s = row_shape(vectors, logits->rows, L.num_sms);
    const int slices = s.slices > 0 ? s.slices : MAX_CLUSTER;
    if (logits->rows > MAX_GRID / slices) return TBE_ERR_INVALID_ARGUMENT;
    const int64_t per_slice = (vectors + slices - 1) / slices;
    const dim3 grid((unsigned)(logits->rows * slices));
    const size_t smem = INSIDE ? inside_bytes(te.K) : 0;
    const bool together = same_phase(logits, grad);
    if (loss != nullptr && s.slices > 0 && together) {
        auto *fn = s.threads == 128 ? distill_rows_kernel<T, 128, INSIDE>
                 : s.threads == 256 ? distill_rows_kernel<T, 256, INSIDE>
                 : s.threads == 512 ? distill_rows_kernel<T, 512, INSIDE> : distill_rows_kernel<T, 1024, INSIDE>;
        cached_smem_attr(L.dev, (const void *)fn, (size_t)SMEM_MOST);
        launch_with(L, "tbe_distill_rows", !INSIDE, slices, fn, grid, s.threads, (size_t)per_slice * 16 + smem,
                    (const T *)logits->data, logits->stride, logits->cols, te, rows, grad_loss, grad_scale, loss, lse,
                    (T *)grad->data, grad->stride, (uint32_t)slices, (int)per_slice, status);
        return TBE_OK;
    }
    if (!INSIDE && !together) {
        run_forward<T, INSIDE>(L, logits, te, rows, loss, lse, nullptr);
        return run_backward<T>(L, logits, te, rows, grad_loss, grad_scale, grad);
    }
    launch_with(L, "tbe_distill_stream", !INSIDE, slices, distill_stream_kernel<T, INSIDE>, grid, STREAM_THREADS, smem,
                (const T *)logits->data, logits->stride, logits->cols, te, rows, grad_loss, grad_scale, loss, lse,
                (T *)grad->data, grad->stride, (uint32_t)slices, (int)per_slice, together, status);
    return TBE_OK;
}

// What is to be computed of the rows: any of loss and gradient.
struct DistillCall {
    float *loss, *lse;   // lse without loss: a stored one
    const float *grad_loss;
    float grad_scale;
    const tbe_matrix *grad;
};

template <typename T>
static tbe_status run_distill(Launch &L, const tbe_matrix *logits, const tbe_teacher *teacher, const DistillCall &d,
                              void *ws, int32_t *status) {
    const Teacher te{teacher->ids, teacher->logits, teacher->index_type, teacher->dtype, teacher->K,
                     teacher->temperature};
    tbe_status st = TBE_OK;
    if (teacher_inside(logits->rows, te.K)) {
        if (d.grad == nullptr) run_forward<T, true>(L, logits, te, TeacherRows{}, d.loss, d.lse, status);
        else st = run_loss_grad<T, true>(L, logits, te, TeacherRows{}, d.grad_loss, d.grad_scale, d.loss, d.lse, d.grad, status);
    } else {
        const bool stored = d.loss == nullptr;
        const TeacherRows rows = run_teacher<T>(L, logits, te, ws, stored ? d.lse : nullptr, status);
        // the teachers' kernel has counted the ids
        if (d.grad == nullptr) run_forward<T, false>(L, logits, te, rows, d.loss, d.lse, nullptr);
        else if (stored) st = run_backward<T>(L, logits, te, rows, d.grad_loss, d.grad_scale, d.grad);
        else st = run_loss_grad<T, false>(L, logits, te, rows, d.grad_loss, d.grad_scale, d.loss, d.lse, d.grad, status);
    }
    if (st != TBE_OK) return st;
    return L.failed ? TBE_ERR_CUDA : TBE_OK;
}

static tbe_status enqueue(const tbe_matrix *logits, const tbe_teacher *teacher, const DistillCall &d, void *ws,
                          size_t ws_bytes, int32_t *status, const tbe_config *cfg, cudaStream_t stream) {
    if (logits->rows == 0) return TBE_OK;
    const size_t need = teacher_bytes(logits->rows, teacher->K);
    if (need > 0 && ws == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(ws, 256)) return TBE_ERR_MISALIGNED;
    if (ws_bytes < need) return TBE_ERR_BUFFER_TOO_SMALL;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        if (logits->dtype == TBE_F32) return run_distill<float>(L, logits, teacher, d, ws, status);
        if (logits->dtype == TBE_F16) return run_distill<__half>(L, logits, teacher, d, ws, status);
        return run_distill<__nv_bfloat16>(L, logits, teacher, d, ws, status);
    });
}

// Self-test of the slices' copy wait: two rows of SELFTEST_V logits, the second
// without an entry, whose copies are withheld.  `ws` as the header lays it out.
constexpr int SELFTEST_V = 64;
struct DistillSelftest {
    float loss[2], lse[2], grad[2][SELFTEST_V];
    alignas(16) float logits[2][SELFTEST_V];
    int32_t ids[2];
    float teacher[2];
};

size_t distill_selftest_bytes() { return round_up(sizeof(DistillSelftest), 256); }

__global__ void distill_selftest_init_kernel(DistillSelftest *w) {
    const int i = threadIdx.x;   // of 2 SELFTEST_V
    w->grad[0][i] = 1.f;
    w->logits[0][i] = 0.f;
    if (i < 2) {
        w->loss[i] = w->lse[i] = 1.f;
        w->ids[i] = i == 0 ? 5 : -1;
        w->teacher[i] = 0.f;
    }
}

tbe_status launch_distill_selftest(Launch &L, void *ws, int32_t *status) {
    auto *w = (DistillSelftest *)ws;
    L.before("tbe_selftest_init");
    distill_selftest_init_kernel<<<1, 2 * SELFTEST_V, 0, L.stream>>>(w);
    L.after();
    const Teacher te{w->ids, w->teacher, TBE_INDEX_I32, TBE_F32, 1, 1.f};
    constexpr int VECTORS = SELFTEST_V / 4;
    launch_with(L, "tbe_distill_rows", false, 1, distill_rows_kernel<float, 128, true, true>, dim3(2), 128,
                VECTORS * 16 + inside_bytes(1), w->logits[0], SELFTEST_V, SELFTEST_V, te, TeacherRows{},
                (const float *)nullptr, 1.f, w->loss, w->lse, w->grad[0], SELFTEST_V, 1u, VECTORS, status);
    return TBE_OK;
}

}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_distill_workspace_bytes(int64_t rows, int32_t K) {
    if (rows < 0 || rows >= TOKEN_MAX_ROWS || K < 1 || K > DISTILL_MAX_K) return 0;
    return teacher_bytes(rows, K);
}

tbe_status tbe_distill_forward(const tbe_matrix *logits, const tbe_teacher *teacher, float *loss, float *lse,
                               void *workspace, size_t workspace_bytes, int32_t *dev_status,
                               const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_floats(loss, logits->rows);
    if (st == TBE_OK) st = check_floats(lse, logits->rows);
    if (st == TBE_OK) st = check_floats(dev_status, 0);
    if (st != TBE_OK) return st;
    return enqueue(logits, teacher, DistillCall{loss, lse, nullptr, 0.f, nullptr}, workspace, workspace_bytes,
                   dev_status, cfg, stream);
}

tbe_status tbe_distill_backward(const tbe_matrix *logits, const tbe_teacher *teacher, const float *lse,
                                const float *grad_loss, float grad_scale, const tbe_matrix *grad_logits,
                                void *workspace, size_t workspace_bytes, const tbe_config *cfg,
                                cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_floats(lse, logits->rows);
    if (st == TBE_OK) st = check_gradient(logits, grad_logits, grad_loss);
    if (st != TBE_OK) return st;
    return enqueue(logits, teacher, DistillCall{nullptr, const_cast<float *>(lse), grad_loss, grad_scale, grad_logits},
                   workspace, workspace_bytes, nullptr, cfg, stream);
}

tbe_status tbe_distill_loss_grad(const tbe_matrix *logits, const tbe_teacher *teacher, const float *grad_loss,
                                 float grad_scale, float *loss, float *lse, const tbe_matrix *grad_logits,
                                 void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                 const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_distill(logits, teacher);
    if (st == TBE_OK) st = check_gradient(logits, grad_logits, grad_loss);
    if (st == TBE_OK) st = check_floats(loss, logits->rows);
    if (st == TBE_OK) st = check_floats(lse, logits->rows);
    if (st == TBE_OK) st = check_floats(dev_status, 0);
    if (st != TBE_OK) return st;
    return enqueue(logits, teacher, DistillCall{loss, lse, grad_loss, grad_scale, grad_logits}, workspace,
                   workspace_bytes, dev_status, cfg, stream);
}

}  // extern "C"
