// Token embedding: the lookup of one table row per token with a scale, and the
// gradient of the table by sorted tokens.
//
//   forward   out[n,:] = scale * W[id_n,:]          (zero row for an id outside the table)
//   backward  dW[v,:]  = scale * sum_{n: id_n = v} G[n,:]   for every row v of the table
//
// The pooled lookup of forward.cu sums bags and its backward updates the
// touched rows with Adagrad; here every token keeps its own row and the
// gradient is a dense matrix, as a table that is also the output layer of a
// model needs it (the two gradients are added before the update).
#include "token_internal.cuh"

namespace tbe {

// ---------------------------------------------------------------------------
// Lookup.  Bound by memory: one read of the different rows, one write of N
// rows.  A row is taken by 2^lg lanes (a warp for rows of 32 vectors or more,
// several rows per warp for shorter ones), a column chunk of U vectors per
// lane per blockIdx.y, so that no thread loops and all its loads are issued
// before the first is used; a single token of a long row still spreads over
// several warps.
template <typename WT, typename OT, int VEC, int U>
__global__ void __launch_bounds__(256)
token_fwd_kernel(const WT *__restrict__ table, int64_t table_stride, int64_t V,
                 const void *__restrict__ ids, int index_type, int64_t N, int vectors, int lg,
                 float scale, OT *__restrict__ out, int64_t out_stride, int32_t *status) {
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int c0 = (blockIdx.y << lg) * U + lane;
    int64_t id = -1;
    if (row < N) id = load_index(ids, index_type, row);
    const bool inside = id >= 0 && id < V;
    if (status != nullptr && blockIdx.y == 0) {
        const int bad = __syncthreads_count(row < N && lane == 0 && !inside);
        if (threadIdx.x == 0 && bad != 0) atomicAdd(status, bad);
    }
    if (row >= N) return;
    Raw<WT, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + (u << lg);
#pragma unroll
        for (int i = 0; i < Raw<WT, VEC>::WORDS; ++i) r[u].w[i] = 0;
        if (inside && c < vectors) r[u] = load_raw<WT, VEC>(table + id * table_stride + (int64_t)c * VEC);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + (u << lg);
        if (c >= vectors) break;
        float f[VEC];
        widen<WT, VEC>(r[u], f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = inside ? f[i] * scale : 0.f;
        store_raw<OT, VEC>(out + row * out_stride + (int64_t)c * VEC, narrow<OT, VEC>(f));
    }
}

template <typename WT, typename OT, int VEC>
static void launch_fwd(Launch &L, const tbe_matrix *table, const void *ids, int index_type, float scale,
                       const tbe_matrix *out, int32_t *status) {
    const int vectors = (int)(table->cols / VEC);
    const int lg = lane_shift(vectors);
    const int U = vectors <= (1 << lg) ? 1 : vectors <= (2 << lg) ? 2 : 4;
    const int64_t blocks = ((out->rows << lg) + 255) / 256;
    const dim3 grid((unsigned)blocks, (unsigned)((vectors + (U << lg) - 1) / (U << lg)));
    auto *fn = U == 1 ? token_fwd_kernel<WT, OT, VEC, 1>
                      : U == 2 ? token_fwd_kernel<WT, OT, VEC, 2> : token_fwd_kernel<WT, OT, VEC, 4>;
    L.before("tbe_token_fwd");
    fn<<<grid, 256, 0, L.stream>>>((const WT *)table->data, table->stride, table->rows, ids, index_type,
                                   out->rows, vectors, lg, scale, (OT *)out->data, out->stride, status);
    L.after();
}

template <typename WT, typename OT>
static void dispatch_fwd(Launch &L, const tbe_matrix *table, const void *ids, int index_type, float scale,
                         const tbe_matrix *out, int32_t *status) {
    constexpr int MOST = sizeof(WT) == 4 && sizeof(OT) == 4 ? 4 : 8;
    const tbe_matrix *ms[2] = {table, out};
    switch (vector_of(MOST, table->cols, ms, 2)) {
    case 8:
        if constexpr (MOST == 8) launch_fwd<WT, OT, 8>(L, table, ids, index_type, scale, out, status);
        break;
    case 4: launch_fwd<WT, OT, 4>(L, table, ids, index_type, scale, out, status); break;
    case 2: launch_fwd<WT, OT, 2>(L, table, ids, index_type, scale, out, status); break;
    default: launch_fwd<WT, OT, 1>(L, table, ids, index_type, scale, out, status); break;
    }
}

// ---------------------------------------------------------------------------
// Gradient.  1. keys: id, or V for a token without a gradient; 2. a stable
// sort by key (sort.cu), so the tokens of a row follow one another in the
// order of the batch; 3. sums of runs of equal keys, in that order: the result
// does not depend on the launch's timing.

__global__ void __launch_bounds__(256)
token_keys_kernel(const void *__restrict__ ids, int index_type, int64_t N, int64_t V, int64_t padding_id,
                  uint32_t *__restrict__ keys, uint32_t *__restrict__ vals, int32_t *long_count,
                  int32_t *sort_status, int32_t *status) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    bool bad = false;
    if (n < N) {
        const int64_t id = load_index(ids, index_type, n);
        bad = id < 0 || id >= V;
        keys[n] = bad || id == padding_id ? (uint32_t)V : (uint32_t)id;
        vals[n] = (uint32_t)n;
    }
    if (n < 4) sort_status[n] = 0;
    if (n == 0) *long_count = 0;
    if (status != nullptr) {
        const int count = __syncthreads_count(bad);
        if (threadIdx.x == 0 && count != 0) atomicAdd(status, count);
    }
}

// Every row of the gradient as zeros.
template <typename OT, int VEC>
__global__ void __launch_bounds__(256)
token_zero_kernel(OT *out, int64_t stride, int64_t rows, int vectors) {
    Raw<OT, VEC> zero;
#pragma unroll
    for (int i = 0; i < Raw<OT, VEC>::WORDS; ++i) zero.w[i] = 0;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * 8)
        for (int c = threadIdx.x & 31; c < vectors; c += 32)
            store_raw<OT, VEC>(out + r * stride + (int64_t)c * VEC, zero);
}

// Runs of more than LONG_RUN tokens are summed in pieces by several lane
// groups and joined by token_join_kernel; shorter ones by one group.
constexpr int LONG_RUN = 32;
constexpr int POSITIONS = 32;   // sorted positions per warp

// The runs near the 32 positions p0.. of a warp, from the keys of the 32
// before, its own and the 32 after: bit i of `cur` says that a run starts at
// p0+i, of `prev` at p0-32+i (bit 0 is not known), of `next` at p0+32+i.
// Positions from the first key V on (tokens without a gradient) count as the
// start of a run.
struct RunWindow {
    int64_t p0;
    uint32_t prev, cur, next;
    // first position of the run that holds p0+i, or -1: before p0-31, so the
    // run has more than LONG_RUN positions
    __device__ __forceinline__ int64_t start(int i) const {
        const uint32_t m = cur & (0xffffffffu >> (31 - i));
        if (m) return p0 + 31 - __clz(m);
        const uint32_t b = prev & ~1u;
        return b ? p0 - 32 + 31 - __clz(b) : -1;
    }
    // end of the run that holds p0+i, or -1: beyond p0+63
    __device__ __forceinline__ int64_t end(int i) const {
        const uint32_t m = i == 31 ? 0u : cur >> (i + 1);
        if (m) return p0 + i + __ffs(m);
        return next ? p0 + 31 + __ffs(next) : -1;
    }
    __device__ __forceinline__ bool is_long(int i) const {
        const int64_t s = start(i), e = end(i);
        return s < 0 || e < 0 || e - s > LONG_RUN;
    }
    __device__ __forceinline__ bool starts(int64_t p) const {   // p in [p0, p0+64)
        const int i = (int)(p - p0);
        return ((i < 32 ? cur >> i : next >> (i - 32)) & 1u) != 0;
    }
};

// Sum of runs.  Bound by memory: one read of the tokens' gradient rows, one
// write of the touched rows.  A warp holds 32 sorted positions; a group of
// 2^lg lanes takes as many of them and walks over its positions once, B rows
// loaded ahead of the sum whatever runs they belong to, and writes a row out
// where its run ends.  A short run belongs to the group of its first position,
// which walks on to the run's end; a long run's piece of each group goes to
// `partial` (slot 2q of group q: the run began before the group, 2q+1: within).
template <typename GT, typename OT, int VEC, int U>
__global__ void __launch_bounds__(256)
token_reduce_kernel(const GT *__restrict__ grad, int64_t grad_stride, const uint32_t *__restrict__ keys,
                    const uint32_t *__restrict__ vals, int64_t N, uint32_t V, int vectors, int lg,
                    float scale, OT *__restrict__ out, int64_t out_stride, int accumulate,
                    float *__restrict__ partial, int64_t partial_stride, int32_t *long_count,
                    int32_t *long_group, int max_long) {
    const int lane = threadIdx.x & 31;
    RunWindow w;
    w.p0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * POSITIONS;
    if (w.p0 >= N) return;
    auto key_at = [&](int64_t p) { return p < 0 || p >= N ? V : __ldg(keys + p); };
    const uint32_t kp = key_at(w.p0 - 32 + lane), kc = key_at(w.p0 + lane), kn = key_at(w.p0 + 32 + lane);
    uint32_t before = __shfl_up_sync(FULL, kp, 1);
    w.prev = __ballot_sync(FULL, lane > 0 && (kp != before || kp >= V));
    before = __shfl_up_sync(FULL, kc, 1);
    const uint32_t last_p = __shfl_sync(FULL, kp, 31), last_c = __shfl_sync(FULL, kc, 31);
    w.cur = __ballot_sync(FULL, kc >= V || kc != (lane ? before : last_p));
    before = __shfl_up_sync(FULL, kn, 1);
    w.next = __ballot_sync(FULL, kn >= V || kn != (lane ? before : last_c));
    if (w.p0 == 0) w.cur |= 1u;
    const int valid = __popc(__ballot_sync(FULL, kc < V));   // keys ascend: a prefix of the warp's

    const int group = lane >> lg, gl = lane & ((1 << lg) - 1);
    const int i0 = group << lg, i1 = min(valid, (group + 1) << lg);
    if (i0 >= i1) return;
    const int64_t x0 = w.p0 + i0, x1 = w.p0 + i1, q = x0 >> lg;
    // [a, b): the positions that this group sums
    int64_t a = x0, b = x1;
    bool head_long = false;
    if (!(w.cur >> i0 & 1u)) {
        head_long = w.is_long(i0);
        if (!head_long) a = w.end(i0);
    }
    if (a >= x1) return;
    const int64_t tail_start = w.start(i1 - 1);
    bool tail_long = false;
    if (w.end(i1 - 1) != x1) {
        tail_long = w.is_long(i1 - 1);
        if (!tail_long) b = w.end(i1 - 1);
    }
    const bool tail_is_head = head_long && tail_start < x0;   // one long run holds them all
    if (tail_long && !tail_is_head && blockIdx.y == 0 && gl == 0) {
        const int at = atomicAdd(long_count, 1);
        if (at < max_long) long_group[at] = (int32_t)q;
    }

    const int c0 = (blockIdx.y << lg) * U + gl;
    float acc[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[u][i] = 0.f;
    bool first = true;
    constexpr int B = 4;
    for (int64_t p = a; p < b; p += B) {
        Raw<GT, VEC> r[B][U];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (p + j < b) {
                const int64_t n = min((int64_t)__ldg(vals + p + j), N - 1);
                const GT *src = grad + n * grad_stride;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + (u << lg) < vectors)
                        r[j][u] = load_raw<GT, VEC, true>(src + (int64_t)(c0 + (u << lg)) * VEC);
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t pos = p + j;
            if (pos >= b) break;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (c0 + (u << lg) >= vectors) continue;
                float f[VEC];
                widen<GT, VEC>(r[j][u], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[u][i] += f[i];
            }
            const bool last = pos + 1 == b;
            if (!last && !w.starts(pos + 1)) continue;
            const bool in_head = first && head_long;
            if (in_head || (last && tail_long)) {
                float *dst = partial + (2 * q + (in_head ? 0 : 1)) * partial_stride;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + (u << lg) < vectors)
                        store_raw<float, VEC>(dst + (int64_t)(c0 + (u << lg)) * VEC, narrow<float, VEC>(acc[u]));
            } else {
                // (keys and positions out of range come only from a sort that gave up)
                const uint32_t key = __ldg(keys + pos);
                OT *dst = out + (int64_t)key * out_stride;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c0 + (u << lg) >= vectors || key >= V) continue;
                    OT *d = dst + (int64_t)(c0 + (u << lg)) * VEC;
                    float f[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] = 0.f;
                    if (accumulate) widen<OT, VEC>(load_raw<OT, VEC>(d), f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) f[i] += acc[u][i] * scale;
                    store_raw<OT, VEC>(d, narrow<OT, VEC>(f));
                }
            }
            first = false;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[u][i] = 0.f;
        }
    }
}

// Long runs: the pieces of a run added in the order of the sorted positions
// (eight warps take every eighth piece, then the eight sums are added in
// order).  blockIdx.y: 128 columns.
template <typename OT>
__global__ void __launch_bounds__(256)
token_join_kernel(const float *__restrict__ partial, int64_t partial_stride, int lg,
                  const uint32_t *__restrict__ keys, int64_t N, uint32_t V, const int32_t *long_count,
                  const int32_t *__restrict__ long_group, int max_long, int D, float scale, OT *__restrict__ out,
                  int64_t out_stride, int accumulate) {
    __shared__ float4 sums[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = (int64_t)blockIdx.y * 128 + lane * 4;
    const int count = min(*long_count, max_long);
    for (int item = blockIdx.x; item < count; item += gridDim.x) {
        const int64_t q = long_group[item];
        const int64_t last = min(N, (q + 1) << lg) - 1;
        const uint32_t key = __ldg(keys + last);
        // end of the run: 32-way search of the first position with another key
        int64_t lo = last, hi = N;   // key at lo; another key (or the end) at hi
        while (hi - lo > 1) {
            const int64_t step = (hi - lo + 32) / 33;
            const int64_t p = lo + (lane + 1) * step;
            const bool same = p < hi && __ldg(keys + p) == key;
            const int k = __popc(__ballot_sync(FULL, same));   // keys ascend: a prefix of the lanes
            const int64_t next_hi = lo + (k + 1) * step;
            lo += k * step;
            if (next_hi < hi) hi = next_hi;
        }
        const int64_t pieces = ((hi - 1) >> lg) - q + 1;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < D && key < V) {
#pragma unroll 4
            for (int64_t j = warp; j < pieces; j += 8) {
                const float *src = partial + (2 * (q + j) + (j == 0 ? 1 : 0)) * partial_stride + col;
                const float4 v = *reinterpret_cast<const float4 *>(src);
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
        }
        sums[warp][lane] = s;
        __syncthreads();
        if (threadIdx.x < 128 && (int64_t)blockIdx.y * 128 + threadIdx.x < D && key < V) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) t += reinterpret_cast<const float *>(sums[k])[threadIdx.x];
            OT *d = out + (int64_t)key * out_stride + (int64_t)blockIdx.y * 128 + threadIdx.x;
            *d = from_f32<OT>((accumulate ? to_f32(*d) : 0.f) + t * scale);
        }
        __syncthreads();
    }
}

// Workspace of the gradient: sorted pairs twice, the sort's scratch, pieces of
// long runs, the list of long runs.
struct TokenWs {
    size_t keys_a, vals_a, keys_b, vals_b, sort, partial, groups, counters, total;
    int64_t partial_stride;
};

static int token_key_bits(int64_t V) {
    int b = 0;
    while ((V >> b) != 0) ++b;
    return b;
}

static TokenWs token_ws(int64_t N, int64_t V, int64_t D) {
    TokenWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = round_up(off + bytes, 256);
        return at;
    };
    w.counters = take(256);
    w.keys_a = take((size_t)N * 4 + 16);
    w.vals_a = take((size_t)N * 4 + 16);
    w.keys_b = take((size_t)N * 4 + 16);
    w.vals_b = take((size_t)N * 4 + 16);
    w.sort = take(sort_workspace_bytes(N, token_key_bits(V)));
    w.partial_stride = (D + 3) / 4 * 4;
    // a group has as many positions as lanes; the widest vectors (8 elements)
    // give the shortest groups, so the most of them
    const int lg_min = lane_shift((D + 7) / 8);
    const int64_t groups = (N + (1 << lg_min) - 1) >> lg_min;
    w.partial = take((size_t)groups * 2 * w.partial_stride * 4);
    w.groups = take((size_t)(N / (LONG_RUN + 1) + 1) * 4);
    w.total = off;
    return w;
}

template <typename GT, typename OT, int VEC>
static void launch_reduce(Launch &L, const tbe_matrix *grad, const uint32_t *keys, const uint32_t *vals,
                          int64_t V, float scale, const tbe_matrix *out, int accumulate, float *partial,
                          int64_t partial_stride, int32_t *long_count, int32_t *long_group) {
    const int64_t N = grad->rows;
    const int vectors = (int)(grad->cols / VEC);
    const int lg = lane_shift(vectors);
    const int U = vectors <= (1 << lg) ? 1 : 2;
    const int64_t most = N / (LONG_RUN + 1);   // long runs at most
    const dim3 rgrid((unsigned)((N + 8 * POSITIONS - 1) / (8 * POSITIONS)),
                     (unsigned)((vectors + (U << lg) - 1) / (U << lg)));
    auto *fn = U == 1 ? token_reduce_kernel<GT, OT, VEC, 1> : token_reduce_kernel<GT, OT, VEC, 2>;
    L.before("tbe_token_reduce");
    fn<<<rgrid, 256, 0, L.stream>>>((const GT *)grad->data, grad->stride, keys, vals, N, (uint32_t)V,
                                    vectors, lg, scale, (OT *)out->data, out->stride, accumulate, partial,
                                    partial_stride, long_count, long_group, (int)most);
    L.after();
    if (most == 0) return;
    const dim3 jgrid((unsigned)(most < L.num_sms ? most : L.num_sms), (unsigned)((grad->cols + 127) / 128));
    L.before("tbe_token_join");
    token_join_kernel<OT><<<jgrid, 256, 0, L.stream>>>(partial, partial_stride, lg, keys, N, (uint32_t)V,
                                                       long_count, long_group, (int)most,
                                                       (int)grad->cols, scale,
                                                       (OT *)out->data, out->stride, accumulate);
    L.after();
}

template <typename GT, typename OT>
static tbe_status run_backward(Launch &L, const tbe_matrix *grad, const void *ids, int index_type,
                               int64_t padding_id, float scale, const tbe_matrix *out, int accumulate,
                               char *ws, int32_t *status) {
    const int64_t N = grad->rows, V = out->rows, D = out->cols;
    const TokenWs w = token_ws(N, V, D);
    uint32_t *keys_a = (uint32_t *)(ws + w.keys_a), *vals_a = (uint32_t *)(ws + w.vals_a);
    uint32_t *keys_b = (uint32_t *)(ws + w.keys_b), *vals_b = (uint32_t *)(ws + w.vals_b);
    int32_t *counters = (int32_t *)(ws + w.counters);   // [0] long runs, [4..8) the sort's status
    constexpr int MOST = sizeof(GT) == 4 && sizeof(OT) == 4 ? 4 : 8;
    const tbe_matrix *ms[2] = {grad, out};
    const int vec = vector_of(MOST, D, ms, 2);
    if (!accumulate) {
        const int zv = vector_of(16 / (int)sizeof(OT), D, ms + 1, 1);
        const unsigned zgrid = (unsigned)((V + 7) / 8 < 8 * L.num_sms ? (V + 7) / 8 : 8 * L.num_sms);
        L.before("tbe_token_zero");
        switch (zv) {
        case 8:
            if constexpr (sizeof(OT) == 2)
                token_zero_kernel<OT, 8><<<zgrid, 256, 0, L.stream>>>((OT *)out->data, out->stride, V, (int)(D / 8));
            break;
        case 4: token_zero_kernel<OT, 4><<<zgrid, 256, 0, L.stream>>>((OT *)out->data, out->stride, V, (int)(D / 4)); break;
        case 2: token_zero_kernel<OT, 2><<<zgrid, 256, 0, L.stream>>>((OT *)out->data, out->stride, V, (int)(D / 2)); break;
        default: token_zero_kernel<OT, 1><<<zgrid, 256, 0, L.stream>>>((OT *)out->data, out->stride, V, (int)D); break;
        }
        L.after();
    }
    if (N == 0) return TBE_OK;
    L.before("tbe_token_keys");
    token_keys_kernel<<<(unsigned)((N + 255) / 256), 256, 0, L.stream>>>(
        ids, index_type, N, V, padding_id, keys_a, vals_a, counters, counters + 4, status);
    L.after();
    bool in_b = false;
    const tbe_status st = launch_sort(L, keys_a, vals_a, keys_b, vals_b, N, token_key_bits(V), 4,
                                      ws + w.sort, status != nullptr ? status : counters + 4, &in_b);
    if (st != TBE_OK) return st;
    const uint32_t *keys = in_b ? keys_b : keys_a, *vals = in_b ? vals_b : vals_a;
    float *partial = (float *)(ws + w.partial);
    int32_t *groups = (int32_t *)(ws + w.groups);
    switch (vec) {
    case 8:
        if constexpr (MOST == 8)
            launch_reduce<GT, OT, 8>(L, grad, keys, vals, V, scale, out, accumulate, partial,
                                     w.partial_stride, counters, groups);
        break;
    case 4:
        launch_reduce<GT, OT, 4>(L, grad, keys, vals, V, scale, out, accumulate, partial,
                                 w.partial_stride, counters, groups);
        break;
    case 2:
        launch_reduce<GT, OT, 2>(L, grad, keys, vals, V, scale, out, accumulate, partial,
                                 w.partial_stride, counters, groups);
        break;
    default:
        launch_reduce<GT, OT, 1>(L, grad, keys, vals, V, scale, out, accumulate, partial,
                                 w.partial_stride, counters, groups);
        break;
    }
    return TBE_OK;
}

// A table (or its gradient) as the token operators take it.
static tbe_status check_table(const tbe_matrix *m, bool written) {
    const tbe_status st = check_matrix(m, written);
    if (st != TBE_OK) return st;
    // ids are sorted as 32-bit keys, with V for tokens without a gradient
    if (m->rows < 1 || m->rows >= ((int64_t)1 << 31) - 1 || m->cols > TOKEN_MAX_COLS)
        return TBE_ERR_INVALID_ARGUMENT;
    return TBE_OK;
}

static tbe_status check_ids(const void *ids, int index_type, int64_t N) {
    if (!known_index(index_type)) return TBE_ERR_INVALID_ARGUMENT;
    if (N > 0 && ids == nullptr) return TBE_ERR_NULL_POINTER;
    return is_aligned(ids, index_type == TBE_INDEX_I64 ? 8 : 4) ? TBE_OK : TBE_ERR_MISALIGNED;
}

}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_token_forward(const tbe_matrix *table, const void *ids, int32_t index_type, float scale,
                             const tbe_matrix *out, int32_t *dev_status, const tbe_config *cfg,
                             cudaStream_t stream) {
    tbe_status st = check_table(table, false);
    if (st == TBE_OK) st = check_matrix(out, true);
    if (st != TBE_OK) return st;
    if (out->cols != table->cols || out->rows >= TOKEN_MAX_ROWS) return TBE_ERR_INVALID_ARGUMENT;
    if (out->dtype != table->dtype && out->dtype != TBE_F32) return TBE_ERR_UNSUPPORTED_DTYPE;
    if ((st = check_ids(ids, index_type, out->rows)) != TBE_OK) return st;
    if (!is_aligned(dev_status, 4)) return TBE_ERR_MISALIGNED;
    if (out->rows == 0) return TBE_OK;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        if (table->dtype == TBE_F32)
            dispatch_fwd<float, float>(L, table, ids, index_type, scale, out, dev_status);
        else if (table->dtype == TBE_F16 && out->dtype == TBE_F16)
            dispatch_fwd<__half, __half>(L, table, ids, index_type, scale, out, dev_status);
        else if (table->dtype == TBE_F16)
            dispatch_fwd<__half, float>(L, table, ids, index_type, scale, out, dev_status);
        else if (out->dtype == TBE_BF16)
            dispatch_fwd<__nv_bfloat16, __nv_bfloat16>(L, table, ids, index_type, scale, out, dev_status);
        else
            dispatch_fwd<__nv_bfloat16, float>(L, table, ids, index_type, scale, out, dev_status);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

size_t tbe_token_workspace_bytes(int64_t N, int64_t V, int64_t D) {
    if (N < 0 || N >= TOKEN_MAX_ROWS || V < 1 || V >= ((int64_t)1 << 31) - 1 || D < 1 || D > TOKEN_MAX_COLS)
        return 0;
    return token_ws(N, V, D).total;
}

tbe_status tbe_token_backward(const tbe_matrix *grad_out, const void *ids, int32_t index_type,
                              int64_t padding_id, float scale, const tbe_matrix *grad_table,
                              int32_t accumulate, void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_table(grad_table, true);
    if (st == TBE_OK) st = check_matrix(grad_out, false);
    if (st != TBE_OK) return st;
    const int64_t N = grad_out->rows, V = grad_table->rows, D = grad_table->cols;
    if (grad_out->cols != D || N >= TOKEN_MAX_ROWS || (accumulate != 0 && accumulate != 1))
        return TBE_ERR_INVALID_ARGUMENT;
    if (grad_table->dtype != grad_out->dtype && grad_table->dtype != TBE_F32) return TBE_ERR_UNSUPPORTED_DTYPE;
    if ((st = check_ids(ids, index_type, N)) != TBE_OK) return st;
    if (workspace == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(workspace, 256) || !is_aligned(dev_status, 4)) return TBE_ERR_MISALIGNED;
    if (workspace_bytes < token_ws(N, V, D).total) return TBE_ERR_BUFFER_TOO_SMALL;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        char *ws = (char *)workspace;
        tbe_status s;
        const int g = grad_out->dtype, o = grad_table->dtype;
        if (g == TBE_F32)
            s = run_backward<float, float>(L, grad_out, ids, index_type, padding_id, scale, grad_table, accumulate, ws, dev_status);
        else if (g == TBE_F16 && o == TBE_F16)
            s = run_backward<__half, __half>(L, grad_out, ids, index_type, padding_id, scale, grad_table, accumulate, ws, dev_status);
        else if (g == TBE_F16)
            s = run_backward<__half, float>(L, grad_out, ids, index_type, padding_id, scale, grad_table, accumulate, ws, dev_status);
        else if (o == TBE_BF16)
            s = run_backward<__nv_bfloat16, __nv_bfloat16>(L, grad_out, ids, index_type, padding_id, scale, grad_table, accumulate, ws, dev_status);
        else
            s = run_backward<__nv_bfloat16, float>(L, grad_out, ids, index_type, padding_id, scale, grad_table, accumulate, ws, dev_status);
        if (s != TBE_OK) return s;
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
