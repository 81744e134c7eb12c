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
// sort by key, so the tokens of a row follow one another in the order of the
// batch; 3. sums of runs of equal keys, in that order: the result does not
// depend on the launch's timing.
//
// The sort is a radix sort of digits of up to ten bits, on (key, token) pairs
// of eight bytes.  A batch that fits one CTA is sorted by one launch; a larger
// one takes two per digit: every CTA counts the digits of its tile of tokens,
// then adds up the counts before its tile and places its tokens in order.
// These launches are bound by latency and leave most of the device idle, and
// most of a call's bytes are the zeros of rows without a token: the zeros are
// written by the other CTAs of the same launches, a share by each.  (A cluster
// of eight CTAs exchanging counts through shared memory, one launch for all
// digits, took 145 us for 262,144 tokens: its scattered writes alone go
// through eight SMs only.)
constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32;   // a thread has two digits
constexpr int DIGIT_BITS = 10, BINS = 1 << DIGIT_BITS;
constexpr int64_t ONE_CTA_MOST = 8192;    // tokens that one CTA sorts by itself
constexpr int64_t TILE_LEAST = 4096;

struct SortSmem {
    uint32_t count[SORT_WARPS][BINS];     // of a warp's tokens, then the place of its next one
    uint32_t warp_sum[SORT_WARPS];
};

struct SortSource {   // of a pass: the ids (first pass) or the pairs of the pass before
    const void *ids;
    const uint2 *pairs;
    int64_t N, V, padding_id;
    int index_type;
};

struct Zeros {        // a share of the gradient, written by the CTAs from `first` on
    uint4 *data;
    int64_t begin, end;
    unsigned first;
};

__device__ __forceinline__ void write_share(const Zeros &z) {
    const int64_t parts = gridDim.x - z.first, part = blockIdx.x - z.first;
    const int64_t per = (z.end - z.begin + parts - 1) / parts;
    const int64_t end = min(z.end, z.begin + (part + 1) * per);
    for (int64_t i = z.begin + part * per + threadIdx.x; i < end; i += SORT_THREADS) z.data[i] = make_uint4(0, 0, 0, 0);
}

// Pairs of the tokens p + 32 b + lane of a warp, b < B; nothing beyond `end`.
template <int B>
__device__ __forceinline__ void load_pairs(const SortSource &src, int64_t p, int64_t end, uint2 (&v)[B], int *bad) {
    const int lane = threadIdx.x & 31;
    if (src.pairs != nullptr) {
#pragma unroll
        for (int b = 0; b < B; ++b)
            v[b] = p + b * 32 + lane < end ? __ldcg(src.pairs + p + b * 32 + lane) : make_uint2(0, 0);
        return;
    }
    int64_t id[B];
#pragma unroll
    for (int b = 0; b < B; ++b)
        id[b] = p + b * 32 + lane < end ? load_index(src.ids, src.index_type, p + b * 32 + lane) : 0;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const bool outside = id[b] < 0 || id[b] >= src.V;
        if (bad != nullptr) *bad += outside;
        v[b] = make_uint2(outside || id[b] == src.padding_id ? (uint32_t)src.V : (uint32_t)id[b],
                          (uint32_t)(p + b * 32 + lane));
    }
}

// A CTA's tokens [t0, t1): warp w's share of them.
__device__ __forceinline__ void warp_share(int64_t t0, int64_t t1, int64_t &p0, int64_t &p1) {
    const int64_t share = ((t1 - t0 + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32;
    p0 = min(t1, t0 + (threadIdx.x >> 5) * share);
    p1 = min(t1, p0 + share);
}

// Digits of the CTA's tokens, counted per warp.
__device__ __forceinline__ void count_digits(SortSmem &S, const SortSource &src, int64_t t0, int64_t t1, int shift,
                                             int bits, int *bad) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    int64_t p0, p1;
    warp_share(t0, t1, p0, p1);
    for (int d = lane; d < bins; d += 32) S.count[warp][d] = 0;
    __syncwarp();
    constexpr int B = 4;
    for (int64_t p = p0; p < p1; p += 32 * B) {
        uint2 v[B];
        load_pairs<B>(src, p, p1, v, bad);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (p + b * 32 + lane < p1) atomicAdd(&S.count[warp][(v[b].x >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
}

// Sums of digits 2 tid and 2 tid + 1 over the warps, each warp's counts
// replaced by the sums of the warps before it.
__device__ __forceinline__ uint2 scan_warps(SortSmem &S, int bins) {
    uint2 sum = make_uint2(0, 0);
    if (2 * threadIdx.x < bins) {
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            uint2 *at = reinterpret_cast<uint2 *>(&S.count[w][2 * threadIdx.x]);
            const uint2 n = *at;
            *at = sum;
            sum.x += n.x;
            sum.y += n.y;
        }
    }
    return sum;
}

// The digits' first places (an exclusive sum over them) and `before` more to
// every warp's counts.
__device__ __forceinline__ void add_bases(SortSmem &S, int bins, uint2 all, uint2 before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t own = all.x + all.y;
    uint32_t scan = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(FULL, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) S.warp_sum[warp] = scan;
    __syncthreads();
    uint32_t add = lane < warp ? S.warp_sum[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) add += __shfl_xor_sync(FULL, add, o);
    const uint32_t first = add + scan - own;
    if (2 * threadIdx.x < bins) {
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            uint2 *at = reinterpret_cast<uint2 *>(&S.count[w][2 * threadIdx.x]);
            *at = make_uint2(at->x + first + before.x, at->y + first + all.x + before.y);
        }
    }
    __syncthreads();
}

// The CTA's tokens to their places, in order.  Lanes with the same digit are
// found bit by bit; count holds the places of the warps' next tokens.
__device__ __forceinline__ void place_tokens(SortSmem &S, const SortSource &src, int64_t t0, int64_t t1, int shift,
                                             int bits, uint2 *out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    int64_t p0, p1;
    warp_share(t0, t1, p0, p1);
    constexpr int B = 4;
    for (int64_t p = p0; p < p1; p += 32 * B) {
        uint2 v[B];
        load_pairs<B>(src, p, p1, v, nullptr);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (p + b * 32 >= p1) break;
            const bool in = p + b * 32 + lane < p1;
            const uint32_t d = (v[b].x >> shift) & (bins - 1);
            unsigned same = __ballot_sync(FULL, in);
            for (int i = 0; i < bits; ++i) {
                const unsigned set = __ballot_sync(FULL, (d >> i) & 1u);
                same &= (d >> i) & 1u ? set : ~set;
            }
            const int earlier = __popc(same & ((1u << lane) - 1));
            uint32_t at = 0;
            if (in) at = S.count[warp][d] + earlier;
            __syncwarp();
            if (in && earlier == 0) S.count[warp][d] += __popc(same);
            __syncwarp();
            if (in) out[at] = v[b];
        }
    }
}

// counts[tile][digit] of the tokens of each tile.
__global__ void __launch_bounds__(SORT_THREADS, 3)
token_count_kernel(SortSource src, int64_t tile, int shift, int bits, uint32_t *counts, int32_t *long_count,
                   int32_t *status, Zeros zeros) {
    __shared__ uint32_t count[BINS];
    launch_dependents();
    if (blockIdx.x >= zeros.first) return write_share(zeros);
    const int tid = threadIdx.x, bins = 1 << bits;
    for (int d = tid; d < bins; d += SORT_THREADS) count[d] = 0;
    wait_for_launch_before();
    if (blockIdx.x == 0 && tid == 0) *long_count = 0;
    __syncthreads();
    const int64_t t0 = min(src.N, blockIdx.x * tile), t1 = min(src.N, t0 + tile);
    int64_t p0, p1;
    warp_share(t0, t1, p0, p1);
    constexpr int B = 4;
    int bad = 0;
    for (int64_t p = p0; p < p1; p += 32 * B) {
        uint2 v[B];
        load_pairs<B>(src, p, p1, v, &bad);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (p + b * 32 + (tid & 31) < p1) atomicAdd(&count[(v[b].x >> shift) & (bins - 1)], 1u);
    }
    if (status != nullptr) {
        bad = __reduce_add_sync(FULL, bad);
        if ((tid & 31) == 0 && bad != 0) atomicAdd(status, bad);
    }
    __syncthreads();
    for (int d = tid; d < bins; d += SORT_THREADS) counts[(int64_t)blockIdx.x * bins + d] = count[d];
}

__global__ void __launch_bounds__(SORT_THREADS, 3)
token_place_kernel(SortSource src, int64_t tile, int shift, int bits, const uint32_t *counts, uint2 *out,
                   Zeros zeros) {
    launch_dependents();
    if (blockIdx.x >= zeros.first) return write_share(zeros);
    extern __shared__ __align__(16) unsigned char smem[];
    SortSmem &S = *reinterpret_cast<SortSmem *>(smem);
    const int tid = threadIdx.x, bins = 1 << bits, tiles = zeros.first;
    const int64_t t0 = min(src.N, blockIdx.x * tile), t1 = min(src.N, t0 + tile);
    wait_for_launch_before();
    count_digits(S, src, t0, t1, shift, bits, nullptr);
    scan_warps(S, bins);
    uint2 before = make_uint2(0, 0), all = before;
    if (2 * tid < bins) {
#pragma unroll 16
        for (int t = 0; t < tiles; ++t) {
            const uint2 n = __ldcg(reinterpret_cast<const uint2 *>(counts + (int64_t)t * bins) + tid);
            if (t < (int)blockIdx.x) {
                before.x += n.x;
                before.y += n.y;
            }
            all.x += n.x;
            all.y += n.y;
        }
    }
    add_bases(S, bins, all, before);
    place_tokens(S, src, t0, t1, shift, bits, out);
}

// All digits of at most ONE_CTA_MOST tokens; the result is in `a` after an odd
// number of passes, else in `b`.
__global__ void __launch_bounds__(SORT_THREADS, 3)
token_sort_kernel(SortSource src, int passes, int bits, uint2 *a, uint2 *b, int32_t *long_count, int32_t *status,
                  Zeros zeros) {
    launch_dependents();
    if (blockIdx.x >= zeros.first) return write_share(zeros);
    extern __shared__ __align__(16) unsigned char smem[];
    SortSmem &S = *reinterpret_cast<SortSmem *>(smem);
    const int tid = threadIdx.x, bins = 1 << bits;
    if (tid == 0) *long_count = 0;
    int bad = 0;
    for (int pass = 0; pass < passes; ++pass) {
        count_digits(S, src, 0, src.N, pass * bits, bits, pass == 0 ? &bad : nullptr);
        add_bases(S, bins, scan_warps(S, bins), make_uint2(0, 0));
        place_tokens(S, src, 0, src.N, pass * bits, bits, pass % 2 ? b : a);
        __syncthreads();   // the next pass reads what every warp has placed
        src.pairs = pass % 2 ? b : a;
    }
    if (status != nullptr) {
        bad = __reduce_add_sync(FULL, bad);
        if ((tid & 31) == 0 && bad != 0) atomicAdd(status, bad);
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
constexpr int POSITIONS = 32;   // sorted positions around a warp's

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
// write of the touched rows.  A group of 2^lg lanes takes 2^pg sorted positions
// (the groups of a warp lie among the same 32) and walks over them once, B
// rows loaded ahead of the sum whatever runs they belong to, and writes a row
// out where its run ends.  A short run belongs to the group of its first position,
// which walks on to the run's end; a long run's piece of each group goes to
// `partial` (slot 2q of group q: the run began before the group, 2q+1: within).
template <typename GT, typename OT, int VEC>
__global__ void __launch_bounds__(256)
token_reduce_kernel(const GT *__restrict__ grad, int64_t grad_stride, const uint2 *pairs,
                    int64_t N, uint32_t V, int vectors, int lg, int pg,
                    float scale, OT *__restrict__ out, int64_t out_stride, int accumulate,
                    float *__restrict__ partial, int64_t partial_stride, int32_t *long_count,
                    int32_t *long_group) {
    __shared__ uint32_t near_keys[8][2 * POSITIONS], near_vals[8][2 * POSITIONS];
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the warp's first position, and the 32 positions around it
    const int64_t first_p = ((int64_t)blockIdx.x * 8 + warp) << (5 - lg + pg);
    RunWindow w;
    w.p0 = first_p & ~(int64_t)(POSITIONS - 1);
    if (first_p >= N) return;
    wait_for_launch_before();
    auto pair_at = [&](int64_t p) { return p < 0 || p >= N ? make_uint2(V, 0) : pairs[p]; };
    const uint2 mine = pair_at(w.p0 + lane), next = pair_at(w.p0 + 32 + lane);
    const uint32_t kp = pair_at(w.p0 - 32 + lane).x, kc = mine.x, kn = next.x;
    near_keys[warp][lane] = kc;
    near_keys[warp][32 + lane] = kn;
    near_vals[warp][lane] = mine.y;
    near_vals[warp][32 + lane] = next.y;
    __syncwarp();
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
    const int i0 = (int)(first_p - w.p0) + (group << pg), i1 = min(valid, i0 + (1 << pg));
    if (i0 >= i1) return;
    const int64_t x0 = w.p0 + i0, x1 = w.p0 + i1, q = x0 >> pg;
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
        long_group[atomicAdd(long_count, 1)] = (int32_t)q;
    }

    const int c = (blockIdx.y << lg) + gl;
    if (c >= vectors) return;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    bool first = true;
    constexpr int B = 8;
    const GT *column = grad + (int64_t)c * VEC;
    for (int64_t p = a; p < b; p += B) {
        Raw<GT, VEC> r[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (p + j < b)
                r[j] = load_raw<GT, VEC, true>(column + (int64_t)near_vals[warp][p + j - w.p0] * grad_stride);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t pos = p + j;
            if (pos >= b) break;
            float f[VEC];
            widen<GT, VEC>(r[j], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += f[i];
            const bool last = pos + 1 == b;
            if (!last && !w.starts(pos + 1)) continue;
            const bool in_head = first && head_long;
            const uint32_t key = near_keys[warp][pos - w.p0];
            if (in_head || (last && tail_long)) {
                float *dst = partial + (2 * q + (in_head ? 0 : 1)) * partial_stride + (int64_t)c * VEC;
                store_raw<float, VEC>(dst, narrow<float, VEC>(acc));
            } else {
                OT *dst = out + (int64_t)key * out_stride + (int64_t)c * VEC;
                float old[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) old[i] = 0.f;
                if (accumulate) widen<OT, VEC>(load_raw<OT, VEC>(dst), old);
#pragma unroll
                for (int i = 0; i < VEC; ++i) old[i] += acc[i] * scale;
                store_raw<OT, VEC>(dst, narrow<OT, VEC>(old));
            }
            first = false;
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
        }
    }
}

// Long runs: the pieces of a run added in the order of the sorted positions
// (eight warps take every eighth piece, then the eight sums are added in
// order).  A CTA takes 32 columns of a run; narrow, so that the pieces of the
// longest run are read by many CTAs.
template <typename OT>
__global__ void __launch_bounds__(256)
token_join_kernel(const float *partial, int64_t partial_stride, int pg, const uint2 *pairs, int64_t N,
                  const int32_t *long_count, const int32_t *long_group, int D, float scale,
                  OT *__restrict__ out, int64_t out_stride, int accumulate) {
    __shared__ float sums[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strips = (D + 31) / 32;
    wait_for_launch_before();
    const int64_t work = (int64_t)*long_count * strips;
    for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
        const int item = (int)(i / strips);
        const int col = (int)(i - (int64_t)item * strips) * 32 + lane;
        const int64_t q = long_group[item];
        const uint32_t key = pairs[((q + 1) << pg) - 1].x;
        // groups that the run reaches into: 32 at a time by their first positions
        // (keys ascend: a prefix of the lanes), then 32 steps of a growing width
        int64_t g = q, step = 1;
        for (;;) {
            const int64_t p = (g + (lane + 1) * step) << pg;
            const int k = __popc(__ballot_sync(FULL, p < N && pairs[p].x == key));
            g += k * step;
            if (k == 32) step *= 32;
            else if (step > 1) step /= 32;
            else break;
        }
        const int64_t pieces = g - q + 1;
        float s = 0.f;
        if (col < D) {
#pragma unroll 16
            for (int64_t j = warp; j < pieces; j += 8)
                s += partial[(2 * (q + j) + (j == 0 ? 1 : 0)) * partial_stride + col];
        }
        sums[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && col < D) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) t += sums[k][lane];
            OT *d = out + (int64_t)key * out_stride + col;
            *d = from_f32<OT>((accumulate ? to_f32(*d) : 0.f) + t * scale);
        }
        __syncthreads();
    }
}

// Workspace of the gradient: sorted pairs twice, the tiles' digit counts,
// pieces of long runs, the list of long runs.
struct TokenWs {
    size_t pairs_a, pairs_b, counts, partial, groups, long_count, total;
    int64_t partial_stride;
};

static int token_key_bits(int64_t V) {
    int b = 0;
    while ((V >> b) != 0) ++b;
    return b;
}

// Positions of a lane group, as a shift: as many as the group has lanes (a
// warp's groups lie among 32 positions), fewer where that leaves SMs short of
// warps, 8 at least.
#ifndef TBE_TOKEN_WARPS
#define TBE_TOKEN_WARPS 32
#endif
static int position_shift(int64_t N, int lg, int64_t strips, int sms) {
    int pg = lg;
    while (pg > 3 && (N >> (5 - lg + pg)) * strips < (int64_t)TBE_TOKEN_WARPS * sms) --pg;
    return pg;
}

// Lane groups at most, for any vector width (one to eight elements) and device.
static int64_t token_groups(int64_t N, int64_t D) {
    int pg = lane_shift((D + 7) / 8);
    if (pg > 3) pg = 3;
    return (N + (1 << pg) - 1) >> pg;
}

// Tiles of the sort's CTAs: at most 128 of them, for the time that every CTA
// takes to add up the others' counts.
struct SortTiles {
    int64_t tile;
    int tiles;
};
static SortTiles token_tiles(int64_t N) {
    SortTiles t;
    t.tile = (N + 127) / 128;
    if (t.tile < TILE_LEAST) t.tile = TILE_LEAST;
    t.tiles = (int)((N + t.tile - 1) / t.tile);
    return t;
}

static TokenWs token_ws(int64_t N, int64_t V, int64_t D) {
    TokenWs w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = round_up(off + bytes, 256);
        return at;
    };
    w.long_count = take(256);
    w.pairs_a = take((size_t)N * 8);
    w.pairs_b = take((size_t)N * 8);
    w.counts = take(N > ONE_CTA_MOST ? (size_t)token_tiles(N).tiles * BINS * 4 : 0);
    w.partial_stride = (D + 3) / 4 * 4;
    w.partial = take((size_t)token_groups(N, D) * 2 * w.partial_stride * 4);
    w.groups = take((size_t)(N / (LONG_RUN + 1) + 1) * 4);
    w.total = off;
    return w;
}

template <typename GT, typename OT, int VEC>
static void launch_reduce(Launch &L, const tbe_matrix *grad, const uint2 *pairs, int64_t V, float scale, const tbe_matrix *out, int accumulate, float *partial,
                          int64_t partial_stride, int32_t *long_count, int32_t *long_group) {
    const int64_t N = grad->rows;
    const int vectors = (int)(grad->cols / VEC);
    const int lg = lane_shift(vectors);
    const int64_t most = N / (LONG_RUN + 1);   // long runs at most
    const int64_t strips = (vectors + (1 << lg) - 1) >> lg;
    const int pg = position_shift(N, lg, strips, L.num_sms);
    const int64_t warps = (N + (32 >> lg << pg) - 1) / (32 >> lg << pg);
    const dim3 rgrid((unsigned)((warps + 7) / 8), (unsigned)strips);
    launch_with(L, "tbe_token_reduce", true, 1, token_reduce_kernel<GT, OT, VEC>, rgrid, 256, 0, (const GT *)grad->data,
                grad->stride, pairs, N, (uint32_t)V, vectors, lg, pg, scale, (OT *)out->data, out->stride, accumulate,
                partial, partial_stride, long_count, long_group);
    if (most == 0) return;
    const int64_t jobs = most * ((grad->cols + 31) / 32), fit = 8 * L.num_sms;
    launch_with(L, "tbe_token_join", true, 1, token_join_kernel<OT>, dim3((unsigned)(jobs < fit ? jobs : fit)), 256, 0,
                partial, partial_stride, pg, pairs, N, long_count, long_group, (int)grad->cols, scale, (OT *)out->data,
                out->stride, accumulate);
}

template <typename GT, typename OT>
static tbe_status run_backward(Launch &L, const tbe_matrix *grad, const void *ids, int index_type,
                               int64_t padding_id, float scale, const tbe_matrix *out, int accumulate,
                               char *ws, int32_t *status) {
    const int64_t N = grad->rows, V = out->rows, D = out->cols;
    const TokenWs w = token_ws(N, V, D);
    uint2 *pairs_a = (uint2 *)(ws + w.pairs_a), *pairs_b = (uint2 *)(ws + w.pairs_b);
    int32_t *long_count = (int32_t *)(ws + w.long_count);
    constexpr int MOST = sizeof(GT) == 4 && sizeof(OT) == 4 ? 4 : 8;
    const tbe_matrix *ms[2] = {grad, out};
    const int vec = vector_of(MOST, D, ms, 2);
    const int key_bits = token_key_bits(V);
    // a gradient without gaps between its rows is zeroed by the sort's launches
    const bool by_sort = N > 0 && !accumulate && (out->stride == D || V == 1) && is_aligned(out->data, 16) &&
                         V * D * (int64_t)sizeof(OT) % 16 == 0;
    if (!accumulate && !by_sort) {
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
    const int passes = (key_bits + DIGIT_BITS - 1) / DIGIT_BITS, bits = (key_bits + passes - 1) / passes;
    const int64_t zero_vectors = by_sort ? V * D * (int64_t)sizeof(OT) / 16 : 0;
    SortSource src{ids, nullptr, N, V, padding_id, index_type};
    // launch i of n: its share of the zeros, written by as many CTAs as run at
    // once beside the sort's (`per_sm` an SM)
    auto share = [&](int i, int n, int sort_ctas) {
        return Zeros{(uint4 *)out->data, zero_vectors * i / n, zero_vectors * (i + 1) / n, (unsigned)sort_ctas};
    };
    auto grid = [&](const Zeros &z, int per_sm) {
        const int64_t most = (z.end - z.begin + 4095) / 4096;
        int64_t fit = (int64_t)per_sm * L.num_sms - z.first;
        if (fit < 1) fit = 1;
        return dim3((unsigned)(z.first + (most < fit ? most : fit)));
    };
    cached_smem_attr(L.dev, (const void *)token_sort_kernel, sizeof(SortSmem));
    cached_smem_attr(L.dev, (const void *)token_place_kernel, sizeof(SortSmem));
    if (N <= ONE_CTA_MOST) {
        const Zeros z = share(0, 1, 1);
        launch_with(L, "tbe_token_sort", false, 1, token_sort_kernel, grid(z, 3), SORT_THREADS, sizeof(SortSmem), src, passes,
                    bits, pairs_a, pairs_b, long_count, status, z);
    } else {
        const SortTiles t = token_tiles(N);
        uint32_t *counts = (uint32_t *)(ws + w.counts);
        for (int pass = 0; pass < passes; ++pass) {
            const Zeros zc = share(2 * pass, 2 * passes, t.tiles), zp = share(2 * pass + 1, 2 * passes, t.tiles);
            launch_with(L, "tbe_token_count", pass > 0, 1, token_count_kernel, grid(zc, 4), SORT_THREADS, 0, src, t.tile,
                        pass * bits, bits, counts, long_count, pass == 0 ? status : (int32_t *)nullptr, zc);
            uint2 *to = pass % 2 ? pairs_b : pairs_a;
            launch_with(L, "tbe_token_place", true, 1, token_place_kernel, grid(zp, 3), SORT_THREADS, sizeof(SortSmem), src,
                        t.tile, pass * bits, bits, counts, to, zp);
            src.pairs = to;
        }
    }
    const uint2 *pairs = passes % 2 ? pairs_a : pairs_b;
    float *partial = (float *)(ws + w.partial);
    int32_t *groups = (int32_t *)(ws + w.groups);
    switch (vec) {
    case 8:
        if constexpr (MOST == 8)
            launch_reduce<GT, OT, 8>(L, grad, pairs, V, scale, out, accumulate, partial, w.partial_stride,
                                 long_count, groups);
        break;
    case 4:
        launch_reduce<GT, OT, 4>(L, grad, pairs, V, scale, out, accumulate, partial, w.partial_stride,
                                 long_count, groups);
        break;
    case 2:
        launch_reduce<GT, OT, 2>(L, grad, pairs, V, scale, out, accumulate, partial, w.partial_stride,
                                 long_count, groups);
        break;
    default:
        launch_reduce<GT, OT, 1>(L, grad, pairs, V, scale, out, accumulate, partial, w.partial_stride,
                                 long_count, groups);
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
