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
// several warps.  Where there are many tokens, a group takes M of them.
// 131,072 rows of 512 f16 out of 1,000,000 (173 MB): 31 us, 5.6 TB/s.
template <typename WT, typename OT, int VEC, int U, int M>
__global__ void __launch_bounds__(256)
token_fwd_kernel(const WT *__restrict__ table, int64_t table_stride, int64_t V,
                 const void *__restrict__ ids, int index_type, int64_t N, int vectors, int lg,
                 float scale, OT *__restrict__ out, int64_t out_stride, int32_t *status) {
    const int64_t group = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg;
    const int lane = threadIdx.x & ((1 << lg) - 1);
    const int c0 = (blockIdx.y << lg) * U + lane;
    int64_t id[M];
#pragma unroll
    for (int m = 0; m < M; ++m) id[m] = group * M + m < N ? load_index(ids, index_type, group * M + m) : -1;
    Raw<WT, VEC> r[M][U];
    int bad = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const bool inside = id[m] >= 0 && id[m] < V;
        bad += !inside && lane == 0 && group * M + m < N;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + (u << lg);
#pragma unroll
            for (int i = 0; i < Raw<WT, VEC>::WORDS; ++i) r[m][u].w[i] = 0;
            if (inside && c < vectors) r[m][u] = load_raw<WT, VEC>(table + id[m] * table_stride + (int64_t)c * VEC);
        }
    }
    if (status != nullptr && blockIdx.y == 0) {
        bad = __reduce_add_sync(FULL, bad);
        if ((threadIdx.x & 31) == 0 && bad != 0) atomicAdd(status, bad);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (group * M + m >= N) break;
        const bool inside = id[m] >= 0 && id[m] < V;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + (u << lg);
            if (c >= vectors) break;
            float f[VEC];
            widen<WT, VEC>(r[m][u], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = inside ? f[i] * scale : 0.f;
            store_raw<OT, VEC>(out + (group * M + m) * out_stride + (int64_t)c * VEC, narrow<OT, VEC>(f));
        }
    }
}

template <typename WT, typename OT, int VEC>
static void launch_fwd(Launch &L, const tbe_matrix *table, const void *ids, int index_type, float scale,
                       const tbe_matrix *out, int32_t *status) {
    const int vectors = (int)(table->cols / VEC);
    const int lg = lane_shift(vectors);
    const int U = vectors <= (1 << lg) ? 1 : vectors <= (2 << lg) ? 2 : 4;
    // several tokens per group once that leaves every SM its fill of groups
    const bool many = ((out->rows / 4) << lg) >= (int64_t)L.num_sms * 2048;
    const int M = !many ? 1 : U == 1 ? 4 : U == 2 ? 2 : 1;
    const int64_t groups = (out->rows + M - 1) / M, blocks = ((groups << lg) + 255) / 256;
    const dim3 grid((unsigned)blocks, (unsigned)((vectors + (U << lg) - 1) / (U << lg)));
    auto *fn = U == 1 ? (M == 1 ? token_fwd_kernel<WT, OT, VEC, 1, 1> : token_fwd_kernel<WT, OT, VEC, 1, 4>)
             : U == 2 ? (M == 1 ? token_fwd_kernel<WT, OT, VEC, 2, 1> : token_fwd_kernel<WT, OT, VEC, 2, 2>)
                      : token_fwd_kernel<WT, OT, VEC, 4, 1>;
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
// written by the other CTAs of the same launches, a share by each.  262,144
// tokens of a table of 1,000,000 (two digits): 14 + 24 us a digit, beside 512 MB
// of zeros; the zeros alone take 70 us.  (A cluster
// of eight CTAs exchanging counts through shared memory, one launch for all
// digits, took 145 us for 262,144 tokens: its scattered writes alone go
// through eight SMs only.)
constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32;   // a thread has two digits
constexpr int DIGIT_BITS = 10, BINS = 1 << DIGIT_BITS;
// Tokens that one CTA sorts by itself.  A whole call this way and by tiles, in us,
// beside tables of 1000 x 64 and 20,000 x 256 bf16 and 131,072 x 1024 bf16 -> f32:
// 2100 tokens 19 and 22, 24 and 29, 87 and 86; 4096: 23 and 26, 25 and 33, 89 and
// 89; 8192: 28 and 26, 38 and 37, 93 and 94; 16,384: 40 and 28, 54 and 37, 115 and 105.
constexpr int64_t ONE_CTA_MOST = 8192;
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

struct Zeros {        // a share of the gradient, written by the CTAs from `first` on, a piece each
    uint4 *data;
    int64_t begin, end;
    unsigned first;
    int tail;         // two-byte words after `end`, fewer than a vector
};

// A CTA writes one piece and ends: pieces in the order in which the device
// starts CTAs are written at 7.3-7.5 TB/s, by CTAs that stay and take pieces in
// turn, with stores or with bulk copies, at 6.2-6.5.
constexpr int ZERO_PER = 4;
constexpr int ZERO_PIECE = SORT_THREADS * ZERO_PER;   // 16-byte vectors

__device__ __forceinline__ void write_share(const Zeros &z) {
    const int64_t first = z.begin + (int64_t)(blockIdx.x - z.first) * ZERO_PIECE + threadIdx.x;
#pragma unroll
    for (int u = 0; u < ZERO_PER; ++u)
        if (first + u * SORT_THREADS < z.end) z.data[first + u * SORT_THREADS] = make_uint4(0, 0, 0, 0);
    if (blockIdx.x == z.first && (int)threadIdx.x < z.tail) reinterpret_cast<uint16_t *>(z.data + z.end)[threadIdx.x] = 0;
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

constexpr int HELD = 8;   // 32-token steps of a warp's share that it keeps in registers

// Digits of the CTA's tokens, counted per warp.  The warp's first pairs stay
// in `held` for place_tokens.
__device__ __forceinline__ void count_digits(SortSmem &S, const SortSource &src, int64_t t0, int64_t t1, int shift,
                                             int bits, uint2 (&held)[HELD], int *bad) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    int64_t p0, p1;
    warp_share(t0, t1, p0, p1);
    load_pairs<HELD>(src, p0, p1, held, bad);
    for (int d = lane; d < bins; d += 32) S.count[warp][d] = 0;
    __syncwarp();
#pragma unroll
    for (int b = 0; b < HELD; ++b)
        if (p0 + b * 32 + lane < p1) atomicAdd(&S.count[warp][(held[b].x >> shift) & (bins - 1)], 1u);
    for (int64_t p = p0 + 32 * HELD; p < p1; p += 32 * HELD) {
        uint2 v[HELD];
        load_pairs<HELD>(src, p, p1, v, bad);
#pragma unroll
        for (int b = 0; b < HELD; ++b)
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
                                             int bits, const uint2 (&held)[HELD], uint2 *out) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
    int64_t p0, p1;
    warp_share(t0, t1, p0, p1);
    for (int64_t p = p0; p < p1; p += 32 * HELD) {
        uint2 v[HELD];
        if (p == p0) {
#pragma unroll
            for (int b = 0; b < HELD; ++b) v[b] = held[b];
        } else {
            load_pairs<HELD>(src, p, p1, v, nullptr);
        }
#pragma unroll
        for (int b = 0; b < HELD; ++b) {
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

__global__ void __launch_bounds__(SORT_THREADS, 2)
token_place_kernel(SortSource src, int64_t tile, int shift, int bits, const uint32_t *counts, uint2 *out,
                   Zeros zeros) {
    launch_dependents();
    if (blockIdx.x >= zeros.first) return write_share(zeros);
    extern __shared__ __align__(16) unsigned char smem[];
    SortSmem &S = *reinterpret_cast<SortSmem *>(smem);
    const int tid = threadIdx.x, bins = 1 << bits, tiles = zeros.first;
    const int64_t t0 = min(src.N, blockIdx.x * tile), t1 = min(src.N, t0 + tile);
    wait_for_launch_before();
    uint2 held[HELD];
    count_digits(S, src, t0, t1, shift, bits, held, nullptr);
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
    place_tokens(S, src, t0, t1, shift, bits, held, out);
}

// All digits of at most ONE_CTA_MOST tokens; the result is in `a` after an odd
// number of passes, else in `b`.
__global__ void __launch_bounds__(SORT_THREADS, 2)
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
        uint2 held[HELD];
        count_digits(S, src, 0, src.N, pass * bits, bits, held, pass == 0 ? &bad : nullptr);
        add_bases(S, bins, scan_warps(S, bins), make_uint2(0, 0));
        place_tokens(S, src, 0, src.N, pass * bits, bits, held, pass % 2 ? b : a);
        __syncthreads();   // the next pass reads what every warp has placed
        src.pairs = pass % 2 ? b : a;
    }
    if (status != nullptr) {
        bad = __reduce_add_sync(FULL, bad);
        if ((tid & 31) == 0 && bad != 0) atomicAdd(status, bad);
    }
}

// ---------------------------------------------------------------------------
// Few tokens: the whole gradient by one launch, bound by latency and by the
// zeros.  A block takes a strip of 32 vectors of the row of one token, if no
// token before it has the same id; its warps share the list of the row's tokens
// and add their sums in order.  The blocks from token_blocks on write the rows
// without a token, a piece each.  Every block looks at all ids, and a row of
// many tokens is one block's: beyond FEW_BLOCKS strips in all the sort is
// faster (512 tokens of 2048 bf16 over 20,000 rows: 22-33 us, with the sort
// 16-19; 512 of 1024: 10 and 11-13; 2000 of 256: 12-13 and 14-17).  300 tokens
// over 10,007 x 99 f32: 9 us (in four launches 20).
constexpr int FEW_TOKENS = 2048;
constexpr int FEW_BLOCKS = 2048;
constexpr int ZERO_ROWS = 8192;           // rows that a block of zeros knows of

static bool few_tokens(int64_t N, int64_t strips) { return N <= FEW_TOKENS && N * strips <= FEW_BLOCKS; }

template <typename GT, typename OT, int VEC>
__global__ void __launch_bounds__(256)
token_few_kernel(const GT *__restrict__ grad, int64_t grad_stride, const void *__restrict__ ids, int index_type,
                 int N, int64_t V, int64_t padding_id, int D, int vectors, int strips, int token_blocks, float scale,
                 OT *__restrict__ out, int64_t out_stride, int accumulate, int flat, int32_t *status) {
    __shared__ uint32_t keys[FEW_TOKENS];
    __shared__ uint32_t touched[ZERO_ROWS / 32];
    __shared__ uint16_t list[FEW_TOKENS];
    __shared__ int warp_count[8];
    __shared__ float sums[8][32 * VEC];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int bad = 0;
#pragma unroll 4
    for (int m = tid; m < N; m += 256) {
        const int64_t id = load_index(ids, index_type, m);
        const bool outside = id < 0 || id >= V;
        bad += outside;
        keys[m] = outside || id == padding_id ? (uint32_t)V : (uint32_t)id;
    }
    if (status != nullptr && blockIdx.x == 0) {
        bad = __reduce_add_sync(FULL, bad);
        if (lane == 0 && bad != 0) atomicAdd(status, bad);
    }
    __syncthreads();
    if ((int)blockIdx.x >= token_blocks) {
        const int64_t piece = blockIdx.x - token_blocks, pieces = gridDim.x - token_blocks;
        // rows [r0, r0 + rows) have a bit each
        auto mark = [&](int64_t r0, int rows) {
            __syncthreads();
            for (int i = tid; i < ZERO_ROWS / 32; i += 256) touched[i] = 0;
            __syncthreads();
            for (int m = tid; m < N; m += 256) {
                const int64_t r = (int64_t)keys[m] - r0;
                if (r >= 0 && r < rows) atomicOr(&touched[r >> 5], 1u << (r & 31));
            }
            __syncthreads();
        };
        auto is_touched = [&](int r) { return (touched[r >> 5] >> (r & 31) & 1u) != 0; };
        if (flat) {   // no gaps between the rows: vectors of 16 bytes, whatever rows they lie in
            constexpr int FV = 16 / (int)sizeof(OT);
            const int64_t total = V * D, all = (total + FV - 1) / FV;
            const int64_t share = (all + pieces - 1) / pieces, end = min(all, (piece + 1) * share);
            // as many vectors at a time as the bits reach
            const int64_t most = max((int64_t)256, min((int64_t)1 << 20, ((int64_t)ZERO_ROWS - 2) * D / FV));
            for (int64_t v0 = piece * share; v0 < end; v0 += most) {
                const int64_t v1 = min(end, v0 + most), r0 = v0 * FV / D;
                const int64_t last = min(total, v1 * FV) - 1;
                mark(r0, (int)(last / D - r0) + 1);
                const uint32_t base = (uint32_t)(v0 * FV - r0 * D);   // of the first element in row r0
                for (int i = tid; i < (int)(v1 - v0); i += 256) {
                    const uint32_t e = base + (uint32_t)i * FV;
                    int r = (int)(e / (uint32_t)D);
                    const int64_t at = (v0 + i) * FV;
                    if (e - (uint32_t)r * D + FV <= (uint32_t)D) {   // within a row
                        if (!is_touched(r)) *reinterpret_cast<uint4 *>(out + at) = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    int in_row = (int)(e - (uint32_t)r * D);
                    for (int j = 0; j < FV && at + j < total; ++j) {
                        if (!is_touched(r)) out[at + j] = from_f32<OT>(0.f);
                        if (++in_row == D) {
                            in_row = 0;
                            ++r;
                        }
                    }
                }
            }
            return;
        }
        Raw<OT, VEC> zero;
#pragma unroll
        for (int i = 0; i < Raw<OT, VEC>::WORDS; ++i) zero.w[i] = 0;
        const int64_t share = (V + pieces - 1) / pieces, end = min(V, (piece + 1) * share);
        const int lg = vectors >= 256 ? 8 : 32 - __clz(max(vectors - 1, 0));   // 2^lg threads a row
        for (int64_t r0 = piece * share; r0 < end; r0 += ZERO_ROWS) {
            const int rows = (int)min((int64_t)ZERO_ROWS, end - r0);
            mark(r0, rows);
            for (int r = tid >> lg; r < rows; r += 256 >> lg) {
                if (is_touched(r)) continue;
                OT *dst = out + (r0 + r) * out_stride;
                for (int c = tid & ((1 << lg) - 1); c < vectors; c += 1 << lg)
                    store_raw<OT, VEC>(dst + (int64_t)c * VEC, zero);
            }
        }
        return;
    }
    const int n = blockIdx.x / strips, c = (blockIdx.x - n * strips) * 32 + lane;
    const uint32_t key = keys[n];
    if (key >= V) return;
    // a warp looks at an eighth of the tokens
    constexpr int SHARE = FEW_TOKENS / 8;
    unsigned found[SHARE / 32];
    int count = 0;
    bool earlier = false;
#pragma unroll
    for (int i = 0; i < SHARE / 32; ++i) {
        const int m = warp * SHARE + i * 32 + lane;
        const bool same = m < N && keys[m] == key;
        earlier |= same && m < n;
        found[i] = __ballot_sync(FULL, same);
        count += __popc(found[i]);
    }
    if (lane == 0) warp_count[warp] = count;
    if (__syncthreads_or(earlier)) return;
    int at = 0, length = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) at += warp_count[w];
        length += warp_count[w];
    }
#pragma unroll
    for (int i = 0; i < SHARE / 32; ++i) {
        if (found[i] >> lane & 1u)
            list[at + __popc(found[i] & ((1u << lane) - 1))] = (uint16_t)(warp * SHARE + i * 32 + lane);
        at += __popc(found[i]);
    }
    __syncthreads();
    // warp w takes tokens [w * each, (w + 1) * each) of the list
    const int each = (length + 7) / 8, l0 = min(length, warp * each), l1 = min(length, l0 + each);
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    constexpr int B = 4;
    for (int l = l0; c < vectors && l < l1; l += B) {
        Raw<GT, VEC> r[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (l + j < l1) r[j] = load_raw<GT, VEC, true>(grad + (int64_t)list[l + j] * grad_stride + (int64_t)c * VEC);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (l + j >= l1) break;
            float f[VEC];
            widen<GT, VEC>(r[j], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += f[i];
        }
    }
    if (length > 1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[warp][i * 32 + lane] = acc[i];
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w * each < length; ++w)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += sums[w][i * 32 + lane];
    }
    if (warp != 0 || c >= vectors) return;
    OT *dst = out + (int64_t)key * out_stride + (int64_t)c * VEC;
    float old[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) old[i] = 0.f;
    if (accumulate) widen<OT, VEC>(load_raw<OT, VEC>(dst), old);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = acc[i] * scale + old[i];
    store_raw<OT, VEC>(dst, narrow<OT, VEC>(acc));
}

template <typename GT, typename OT, int VEC>
static void launch_few(Launch &L, const tbe_matrix *grad, const void *ids, int index_type, int64_t padding_id,
                       float scale, const tbe_matrix *out, int accumulate, int32_t *status) {
    const int N = (int)grad->rows, vectors = (int)(out->cols / VEC), strips = (vectors + 31) / 32;
    const int64_t V = out->rows, D = out->cols;
    const int flat = (out->stride == D || V == 1) && is_aligned(out->data, 16);
    // pieces of 16 KB while they run at once, then of up to 64 KB
    const int64_t bytes = V * D * (int64_t)sizeof(OT), fit = 8 * L.num_sms;
    int64_t pieces = (bytes + 16383) / 16384;
    if (pieces > fit) pieces = (bytes + 65535) / 65536 > fit ? (bytes + 65535) / 65536 : fit;
    if (pieces > 1 << 24) pieces = 1 << 24;
    if (accumulate) pieces = 0;
    L.before("tbe_token_few");
    token_few_kernel<GT, OT, VEC><<<(unsigned)(N * strips + pieces), 256, 0, L.stream>>>(
        (const GT *)grad->data, grad->stride, ids, index_type, N, V, padding_id, (int)D, vectors, strips, N * strips,
        scale, (OT *)out->data, out->stride, accumulate, flat, status);
    L.after();
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

// Sum of runs.  Bound by memory: one read of the tokens' gradient rows, one
// write of the touched rows.  A group of 2^lg lanes takes 2^pg sorted positions
// (the groups of a warp lie among the same 32) and walks over them once, B
// rows loaded ahead of the sum whatever runs they belong to, and writes a row
// out where its run ends.  A short run belongs to the group of its first
// position, which walks on to the run's end; a long run's piece of each group
// goes to `partial` (slot 2q of group q: the run began before the group, 2q+1:
// within).
//
// Which runs are short is read from the keys of 96 positions, the 32 before,
// the 32 around and the 32 after: a bit of prev, cur and next says that a run
// starts there (bit 0 of prev is not known, but a run from there on into cur
// has more than LONG_RUN positions anyway).  Positions without a gradient (key
// V, the last ones) count as starts.
//
// 262,144 rows of 256 f16 over 1,000,000: 30 us, 4.5 TB/s with the partials'
// traffic; 16,384 of 1024 bf16 over 131,072: 15 us, bound by latency.
template <typename GT, typename OT, int VEC>
__global__ void __launch_bounds__(256, 4)
token_reduce_kernel(const GT *__restrict__ grad, int64_t grad_stride, const uint2 *pairs,
                    int N, uint32_t V, int vectors, int lg, int pg,
                    float scale, OT *__restrict__ out, int64_t out_stride, int accumulate,
                    float *__restrict__ partial, int64_t partial_stride, int32_t *long_count,
                    int2 *long_runs) {
    __shared__ uint2 near_pairs[8][2 * POSITIONS];
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the warp's first position, and the 32 positions around it
    const int first_p = (blockIdx.x * 8 + warp) << (5 - lg + pg);
    const int p0 = first_p & ~(POSITIONS - 1);
    if (first_p >= N) return;
    wait_for_launch_before();
    auto pair_at = [&](int p) { return p < 0 || p >= N ? make_uint2(V, 0) : pairs[p]; };
    const uint2 mine = pair_at(p0 + lane), after = pair_at(p0 + 32 + lane);
    const uint32_t kp = pair_at(p0 - 32 + lane).x, kc = mine.x, kn = after.x;
    uint2 *pair = near_pairs[warp];
    pair[lane] = mine;
    pair[32 + lane] = after;
    uint32_t before = __shfl_up_sync(FULL, kp, 1);
    const uint32_t prev = __ballot_sync(FULL, lane > 0 && (kp != before || kp >= V));
    before = __shfl_up_sync(FULL, kc, 1);
    const uint32_t last_p = __shfl_sync(FULL, kp, 31), last_c = __shfl_sync(FULL, kc, 31);
    const uint32_t cur = __ballot_sync(FULL, kc >= V || kc != (lane ? before : last_p)) | (p0 == 0 ? 1u : 0u);
    before = __shfl_up_sync(FULL, kn, 1);
    const uint32_t next = __ballot_sync(FULL, kn >= V || kn != (lane ? before : last_c));
    const int valid = __popc(__ballot_sync(FULL, kc < V));   // keys ascend: a prefix of the positions
    __syncwarp();   // `pair`

    const int group = lane >> lg, gl = lane & ((1 << lg) - 1);
    const int i0 = first_p - p0 + (group << pg), i1 = min(valid, i0 + (1 << pg));
    const int c = (blockIdx.y << lg) + gl;
    if (i0 >= i1 || c >= vectors) return;
    const int q = (p0 + i0) >> pg;
    const uint64_t starts = (uint64_t)next << 32 | cur;
    constexpr int UNKNOWN = 99;   // far enough to make a run long
    // [a, b): the positions that this group sums, as offsets from p0
    int a = i0, b = i1;
    const uint32_t in_cur = cur & ((1u << i0) - 1);
    const int head_start = in_cur ? 31 - __clz(in_cur) : prev ? -1 - __clz(prev) : -UNKNOWN;
    bool head_long = false, tail_long = false, tail_is_head = false;
    if (!(cur >> i0 & 1u)) {
        const uint64_t rest = starts >> i0;
        const int e = rest ? i0 + __ffsll(rest) - 1 : UNKNOWN;
        head_long = e - head_start > LONG_RUN;
        if (!head_long) a = e;
    }
    if (a >= i1) return;
    if (!(i1 == 32 ? next & 1u : cur >> i1 & 1u)) {   // the last run goes on
        const uint64_t rest = starts >> i1;
        const int e = rest ? i1 + __ffsll(rest) - 1 : UNKNOWN;
        const uint32_t upto = cur & (0xffffffffu >> (32 - i1)) & ~((1u << i0) - 1);   // starts in the group
        const int s = upto ? 31 - __clz(upto) : head_start;
        tail_is_head = upto == 0;
        tail_long = e - s > LONG_RUN;
        if (!tail_long) b = e;
    }
    if (tail_long && !tail_is_head && blockIdx.y == 0 && gl == 0)
        long_runs[atomicAdd(long_count, 1)] = make_int2(q, (int)pair[i1 - 1].x);

    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
    constexpr int B = 8;
    const GT *column = grad + (int64_t)c * VEC;
    OT *out_column = out + (int64_t)c * VEC;
    float *piece = partial + (int64_t)q * 2 * partial_stride + (int64_t)c * VEC;
    // bit j: position a + j is the last of its run, or of the group
    uint64_t ends = (starts >> 1 >> a) | 1ull << (b - 1 - a);
    bool to_head = head_long;     // the next row to be finished is a long run's piece
    for (int p = a; p < b; p += B) {
        Raw<GT, VEC> r[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (p + j < b) r[j] = load_raw<GT, VEC, true>(column + (int64_t)pair[p + j].y * grad_stride);
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (p + j >= b) break;
            float f[VEC];
            widen<GT, VEC>(r[j], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += f[i];
            if (!(ends >> j & 1u)) continue;
            if (to_head || (tail_long && p + j + 1 == b)) {
                store_raw<float, VEC>(piece + (to_head ? 0 : partial_stride), narrow<float, VEC>(acc));
            } else {
                OT *dst = out_column + (int64_t)pair[p + j].x * out_stride;
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] *= scale;
                if (accumulate) {
                    float old[VEC];
                    widen<OT, VEC>(load_raw<OT, VEC>(dst), old);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[i] += old[i];
                }
                store_raw<OT, VEC>(dst, narrow<OT, VEC>(acc));
            }
            to_head = false;
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
        }
        ends >>= B;
    }
}

// Long runs: the pieces of a run added in the order of the sorted positions.
// A warp takes 32 columns of a run; runs of many pieces are left to the whole
// block, whose warps take every eighth piece and then add their sums in order.
// Bound by latency: the batch's few hundred long runs give a warp one each, and
// the longest run's pieces are read one after another (17 us for 570 runs of
// 262,144 tokens, the longest of 25,000).
constexpr int MANY_PIECES = 64;

template <typename OT>
__global__ void __launch_bounds__(256)
token_join_kernel(const float *partial, int64_t partial_stride, int pg, const uint2 *pairs, int64_t N,
                  const int32_t *long_count, const int2 *long_runs, int D, float scale,
                  OT *__restrict__ out, int64_t out_stride, int accumulate) {
    __shared__ float sums[8][32];
    __shared__ int64_t many_group[8], many_pieces[8];
    __shared__ uint32_t many_key[8];
    __shared__ int many_col[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int strips = (D + 31) / 32;
    wait_for_launch_before();
    const int64_t work = (int64_t)*long_count * strips;
    // sum of every step-th piece from `first` on of the run that begins in group q
    auto add_pieces = [&](int64_t q, int64_t pieces, int col, int first, int step) {
        float s = 0.f;
        if (col >= D) return s;
        constexpr int B = 8;
        const float *at = partial + 2 * q * partial_stride + col;
        for (int64_t j0 = first; j0 < pieces; j0 += B * step) {
            float v[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int64_t j = j0 + b * step;
                v[b] = j < pieces ? at[(2 * j + (j == 0 ? 1 : 0)) * partial_stride] : 0.f;
            }
#pragma unroll
            for (int b = 0; b < B; ++b) s += v[b];
        }
        return s;
    };
    auto write = [&](uint32_t key, int col, float sum) {
        if (col >= D) return;
        OT *d = out + (int64_t)key * out_stride + col;
        *d = from_f32<OT>((accumulate ? to_f32(*d) : 0.f) + sum * scale);
    };
    for (int64_t i0 = 0; i0 < work; i0 += 8 * gridDim.x) {
        const int64_t i = i0 + (int64_t)warp * gridDim.x + blockIdx.x;   // neighbours in different blocks
        int64_t pieces = 0;
        if (i < work) {
            const int item = (int)(i / strips);
            const int col = (int)(i - (int64_t)item * strips) * 32 + lane;
            const int2 run = long_runs[item];
            const int64_t q = run.x;
            const uint32_t key = (uint32_t)run.y;
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
            pieces = g - q + 1;
            if (pieces <= MANY_PIECES) {
                write(key, col, add_pieces(q, pieces, col, 0, 1));
            } else if (lane == 0) {
                many_group[warp] = q;
                many_pieces[warp] = pieces;
                many_key[warp] = key;
                many_col[warp] = col;
            }
        }
        unsigned many = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) many |= __syncthreads_or(warp == w && pieces > MANY_PIECES) ? 1u << w : 0u;
        for (; many != 0; many &= many - 1) {
            const int w = __ffs(many) - 1, col = many_col[w] + lane;
            sums[warp][lane] = add_pieces(many_group[w], many_pieces[w], col, warp, 8);
            __syncthreads();
            if (warp == 0) {
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) t += sums[k][lane];
                write(many_key[w], col, t);
            }
            __syncthreads();
        }
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
// warp's groups lie among 32 positions), fewer where that leaves an SM with
// less than 32 warps (16 and 64 measured within 5% of that), 8 at least.
static int position_shift(int64_t N, int lg, int64_t strips, int sms) {
    int pg = lg;
    while (pg > 3 && (N >> (5 - lg + pg)) * strips < (int64_t)32 * sms) --pg;
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

static TokenWs token_ws(int64_t N, int64_t D) {
    TokenWs w = {};
    if (few_tokens(N, (D + 31) / 32)) return w;   // for any vector width
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
    w.groups = take((size_t)(N / (LONG_RUN + 1) + 1) * 8);
    w.total = off;
    return w;
}

template <typename GT, typename OT, int VEC>
static void launch_reduce(Launch &L, const tbe_matrix *grad, const uint2 *pairs, int64_t V, float scale,
                          const tbe_matrix *out, int accumulate, float *partial, int64_t partial_stride,
                          int32_t *long_count, int2 *long_runs) {
    const int64_t N = grad->rows;
    const int vectors = (int)(grad->cols / VEC);
    const int lg = lane_shift(vectors);
    const int64_t most = N / (LONG_RUN + 1);   // long runs at most
    const int64_t strips = (vectors + (1 << lg) - 1) >> lg;
    const int pg = position_shift(N, lg, strips, L.num_sms);
    const int64_t warps = (N + (32 >> lg << pg) - 1) / (32 >> lg << pg);
    const dim3 rgrid((unsigned)((warps + 7) / 8), (unsigned)strips);
    launch_with(L, "tbe_token_reduce", true, 1, token_reduce_kernel<GT, OT, VEC>, rgrid, 256, 0, (const GT *)grad->data,
                grad->stride, pairs, (int)N, (uint32_t)V, vectors, lg, pg, scale, (OT *)out->data, out->stride, accumulate,
                partial, partial_stride, long_count, long_runs);
    if (most == 0) return;
    const int64_t jobs = (most * ((grad->cols + 31) / 32) + 7) / 8, fit = 8 * L.num_sms;
    launch_with(L, "tbe_token_join", true, 1, token_join_kernel<OT>, dim3((unsigned)(jobs < fit ? jobs : fit)), 256, 0,
                partial, partial_stride, pg, pairs, N, long_count, long_runs, (int)grad->cols, scale, (OT *)out->data,
                out->stride, accumulate);
}

template <typename GT, typename OT>
static tbe_status run_backward(Launch &L, const tbe_matrix *grad, const void *ids, int index_type,
                               int64_t padding_id, float scale, const tbe_matrix *out, int accumulate,
                               char *ws, int32_t *status) {
    const int64_t N = grad->rows, V = out->rows, D = out->cols;
    const TokenWs w = token_ws(N, D);
    uint2 *pairs_a = (uint2 *)(ws + w.pairs_a), *pairs_b = (uint2 *)(ws + w.pairs_b);
    int32_t *long_count = (int32_t *)(ws + w.long_count);
    constexpr int MOST = sizeof(GT) == 4 && sizeof(OT) == 4 ? 4 : 8;
    const tbe_matrix *ms[2] = {grad, out};
    const int vec = vector_of(MOST, D, ms, 2);
    if (N > 0 && few_tokens(N, (D / vec + 31) / 32)) {
        switch (vec) {
        case 8:
            if constexpr (MOST == 8)
                launch_few<GT, OT, 8>(L, grad, ids, index_type, padding_id, scale, out, accumulate, status);
            break;
        case 4: launch_few<GT, OT, 4>(L, grad, ids, index_type, padding_id, scale, out, accumulate, status); break;
        case 2: launch_few<GT, OT, 2>(L, grad, ids, index_type, padding_id, scale, out, accumulate, status); break;
        default: launch_few<GT, OT, 1>(L, grad, ids, index_type, padding_id, scale, out, accumulate, status); break;
        }
        return TBE_OK;
    }
    const int key_bits = token_key_bits(V);
    // a gradient without gaps between its rows is zeroed by the sort's launches
    const bool by_sort = N > 0 && !accumulate && (out->stride == D || V == 1) && is_aligned(out->data, 16);
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
    const int zero_tail = by_sort ? (int)(V * D * (int64_t)sizeof(OT) % 16 / 2) : 0;
    SortSource src{ids, nullptr, N, V, padding_id, index_type};
    // parts [i, j) of n of the zeros go with a launch
    auto share = [&](int i, int j, int n, int sort_ctas) {
        return Zeros{(uint4 *)out->data, zero_vectors * i / n, zero_vectors * j / n, (unsigned)sort_ctas,
                     j == n ? zero_tail : 0};
    };
    auto grid = [&](const Zeros &z) {
        const int64_t pieces = (z.end - z.begin + ZERO_PIECE - 1) / ZERO_PIECE;
        return dim3((unsigned)(z.first + (pieces == 0 && z.tail > 0 ? 1 : pieces)));
    };
    cached_smem_attr(L.dev, (const void *)token_sort_kernel, sizeof(SortSmem));
    cached_smem_attr(L.dev, (const void *)token_place_kernel, sizeof(SortSmem));
    if (N <= ONE_CTA_MOST) {
        const Zeros z = share(0, 1, 1, 1);
        launch_with(L, "tbe_token_sort", false, 1, token_sort_kernel, grid(z), SORT_THREADS, sizeof(SortSmem), src, passes,
                    bits, pairs_a, pairs_b, long_count, status, z);
    } else {
        const SortTiles t = token_tiles(N);
        uint32_t *counts = (uint32_t *)(ws + w.counts);
        for (int pass = 0; pass < passes; ++pass) {
            // placing takes longer than counting, so more of the zeros go with it
            const Zeros zc = share(8 * pass, 8 * pass + 3, 8 * passes, t.tiles);
            const Zeros zp = share(8 * pass + 3, 8 * pass + 8, 8 * passes, t.tiles);
            launch_with(L, "tbe_token_count", pass > 0, 1, token_count_kernel, grid(zc), SORT_THREADS, 0, src, t.tile,
                        pass * bits, bits, counts, long_count, pass == 0 ? status : (int32_t *)nullptr, zc);
            uint2 *to = pass % 2 ? pairs_b : pairs_a;
            launch_with(L, "tbe_token_place", true, 1, token_place_kernel, grid(zp), SORT_THREADS, sizeof(SortSmem), src,
                        t.tile, pass * bits, bits, counts, to, zp);
            src.pairs = to;
        }
    }
    const uint2 *pairs = passes % 2 ? pairs_a : pairs_b;
    float *partial = (float *)(ws + w.partial);
    int2 *groups = (int2 *)(ws + w.groups);
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
    return token_ws(N, D).total;
}

tbe_status tbe_token_backward(const tbe_matrix *grad_out, const void *ids, int32_t index_type,
                              int64_t padding_id, float scale, const tbe_matrix *grad_table,
                              int32_t accumulate, void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, const tbe_config *cfg, cudaStream_t stream) {
    tbe_status st = check_table(grad_table, true);
    if (st == TBE_OK) st = check_matrix(grad_out, false);
    if (st != TBE_OK) return st;
    const int64_t N = grad_out->rows, D = grad_table->cols;
    if (grad_out->cols != D || N >= TOKEN_MAX_ROWS || (accumulate != 0 && accumulate != 1))
        return TBE_ERR_INVALID_ARGUMENT;
    if (grad_table->dtype != grad_out->dtype && grad_table->dtype != TBE_F32) return TBE_ERR_UNSUPPORTED_DTYPE;
    if ((st = check_ids(ids, index_type, N)) != TBE_OK) return st;
    const size_t need = token_ws(N, D).total;
    if (need > 0 && workspace == nullptr) return TBE_ERR_NULL_POINTER;
    if (!is_aligned(workspace, 256) || !is_aligned(dev_status, 4)) return TBE_ERR_MISALIGNED;
    if (workspace_bytes < need) return TBE_ERR_BUFFER_TOO_SMALL;
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
