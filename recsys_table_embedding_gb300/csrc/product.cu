// The experts' products: rows sorted by expert times their expert's matrix, and
// the gradients of both.
//
//   forward    out[s,n] = sum_k x[s,k] W_e[n,k]
//   rows       dx[s,k]  = sum_n dy[s,n] W_e[n,k]
//   weights    dW_e[n,k] = sum_{s of e} dy[s,n] x[s,k]
//
// with the gated block's activation, or its gradient, where the sums end.
#include <limits.h>

#include "layer_checks.cuh"
#include "pairs.cuh"
#include "product_internal.cuh"
#include "tensor_core.cuh"

namespace tbe {

// ---- activations: a(g) and a'(g), of pairs: the epilogues that evaluate them are
// bound by their instructions.
// FP32 results: expf (2 units in the last place); 16-bit ones: the hardware's 2^x of
// a rounded product, off by 2^-22 (2 + |x|), far below their rounding.
template <typename T> __device__ __forceinline__ float exponential(float x) {
    if constexpr (sizeof(T) == 4) return expf(x);
    else return __expf(x);
}
__device__ __forceinline__ float reciprocal(float x) {      // 2^-23; 0 for infinity
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <typename T> __device__ __forceinline__ Pair sigmoid(Pair g) {
    const float2 m = unpair(mul(g, pair(-1.0f, -1.0f)));
    const float2 d = unpair(add(pair(exponential<T>(m.x), exponential<T>(m.y)), pair(1.0f, 1.0f)));
    return pair(reciprocal(d.x), reciprocal(d.y));
}
// Phi(x) = erfc(-x / sqrt 2) / 2, which keeps its relative precision for x << 0
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(-0.70710678118654752f * x); }
__device__ __forceinline__ Pair normal_cdf(Pair g) {
    const float2 f = unpair(g);
    return pair(normal_cdf(f.x), normal_cdf(f.y));
}

// The branch lies outside the loops, whose elements the compiler then interleaves.
// g becomes a(g) u
template <typename T, int N> __device__ __forceinline__ void gate_products(int kind, Pair (&g)[N], const Pair (&u)[N]) {
    if (kind == TBE_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = mul(mul(g[j], sigmoid<T>(g[j])), u[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] = mul(mul(g[j], normal_cdf(g[j])), u[j]);
    }
}
// g becomes dg = dh u a'(g), u becomes du = dh a(g)
template <typename T, int N> __device__ __forceinline__ void gate_gradients(int kind, const Pair (&dh)[N], Pair (&g)[N], Pair (&u)[N]) {
    const Pair one = pair(1.0f, 1.0f), minus = pair(-1.0f, -1.0f);
    if (kind == TBE_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const Pair s = sigmoid<T>(g[j]), value = mul(g[j], s);
            const Pair slope = mul(s, fma(g[j], fma(s, minus, one), one));
            g[j] = mul(mul(dh[j], u[j]), slope);
            u[j] = mul(dh[j], value);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const Pair c = normal_cdf(g[j]), value = mul(g[j], c);
            const float2 q = unpair(mul(mul(g[j], g[j]), pair(-0.5f, -0.5f)));
            const Pair slope = fma(mul(g[j], pair(0.3989422804014327f, 0.3989422804014327f)),
                                   pair(exponential<T>(q.x), exponential<T>(q.y)), c);
            g[j] = mul(mul(dh[j], u[j]), slope);
            u[j] = mul(dh[j], value);
        }
    }
}
// Arrays of floats as pairs, and back.
template <int N> __device__ __forceinline__ void to_pairs(const float (&f)[2 * N], Pair (&a)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = pair(f[2 * j], f[2 * j + 1]);
}
template <int N> __device__ __forceinline__ void from_pairs(const Pair (&a)[N], float (&f)[2 * N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float2 v = unpair(a[j]);
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
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

enum Epilogue { STORE = 0, GATED = 1, GATE_GRAD = 2 };

// ---------------------------------------------------------------------------
// Tensor cores: 256 x 256 tiles by pairs of CTAs.

// What a product multiplies: rows with the weight as it lies or transposed, or
// the rows' two matrices with one another.
enum Form { ROWS = 0, ROWS_GRAD = 1, WEIGHTS = 2 };

constexpr int TC_TILE = 256, TC_K = 64, TC_EPILOGUE = 8;
constexpr int TC_OPERAND = 128 * TC_K * 2, TC_STAGE = 2 * TC_OPERAND;      // bytes a CTA holds of a step
constexpr int TC_STAGED = 32 * 128;        // bytes of a warp's rows on their way out
// Steps under way: as many as shared memory takes beside the table of the groups.
constexpr int TC_STAGES = 6, TC_STAGES_MANY = 5, TC_FEW_EXPERTS = 400;
// Terms after which sums leave the tensor core: it cuts them off at 24 bits after each
// product of 16 instead of rounding, which makes a sum of terms of one sign too small
// by about 2^-27.3 of itself a term (FP16, measured: 5.0e-5 after 8192, 2.0e-4 after
// 32,768, 6.2e-3 after 2^20; of both signs 9.1e-6 after 8192).  What leaves is added up
// in registers.  The weights' sums leave after 512 rows for FP32 results (2.4e-7), after
// 2048 for 16-bit ones.  Sums of rows, whose results are of 16 bits, stay where they lose
// less than a fifth of the smallest half step: 8192 terms of FP16, 65,536 of BF16.
// Longer ones leave after 4096, in a kernel of its own: 8192 x 2048 results of 11,008
// FP16 terms take 273 us (in one piece 261), the gate's gradient 277 (279).  After 2048
// terms the gate's gradient takes 371 us: the products wait for the tile's end.
constexpr int TC_SEGMENT = 512, TC_SEGMENT_HALF = 2048;      // of FP32 results, of 16-bit ones
constexpr int TC_LONG_F16 = 8192, TC_LONG_BF16 = 65536, TC_LONG_SEGMENT = 4096;
// Warps: four that load, issue and clear, eight that finish the sums.  Of the 168
// registers a thread that a CTA of 384 is launched with the first give up what
// the others take: 128 * 56 + 256 * 216 <= 384 * 168.
constexpr int TC_CONTROL = 4, TC_THREADS = 32 * (TC_CONTROL + TC_EPILOGUE);
constexpr int TC_LAUNCH_REGS = 168, TC_CONTROL_REGS = 56, TC_EPILOGUE_REGS = 216;
static_assert(32 * (TC_CONTROL * TC_CONTROL_REGS + TC_EPILOGUE * TC_EPILOGUE_REGS) <= TC_THREADS * TC_LAUNCH_REGS,
              "an increase beyond the launch's registers never ends");
static_assert(TC_CONTROL_REGS <= TC_LAUNCH_REGS && TC_EPILOGUE_REGS >= TC_LAUNCH_REGS,
              "an increase to fewer registers, or a decrease to more, is an illegal instruction");

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
    int stages;                 // steps under way
    int segment;                // WEIGHTS, LONG: terms after which the sums leave the tensor core
    int withhold;               // the self-test: operands that never arrive
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
    uint32_t loaded;            // WEIGHTS: steps whose copies have been issued
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

// Twice 32 sums at once; without products: `fill`
__device__ __forceinline__ void load_sums(float (&v)[32], float (&u)[32], uint32_t from, uint32_t other, bool some, float fill) {
    if (some) {
        uint32_t a[32], b[32];
        __syncwarp();
        tc::tmem_ld32(from, a);
        tc::tmem_ld32(other, b);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            v[j] = __uint_as_float(a[j]);
            u[j] = __uint_as_float(b[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = u[j] = fill;
    }
}

// 64 columns of this lane's rows, staged and written.
template <typename T>
__device__ __forceinline__ void write_packed(unsigned char *staged, int lane, const uint32_t (&w)[2][16], T *out,
                                             int64_t stride, int rows, int cols, bool whole) {
    stage_columns(staged, lane, 0, w[0]);
    stage_columns(staged, lane, 1, w[1]);
    write_columns<T>(staged, lane, out, stride, rows, cols, whole);
}

// 32 columns of the gate's sums g and the other half's u: both and their product as T.
template <typename T>
__device__ __forceinline__ void pack_gated(const TensorProduct &p, float (&g)[32], const float (&u)[32], uint32_t (&gate)[16],
                                           uint32_t (&up)[16], uint32_t (&product)[16]) {
    if (p.gate_up != nullptr) {
        pack_columns<T>(g, gate);
        pack_columns<T>(u, up);
    }
    Pair a[16], b[16];
    to_pairs(g, a);
    to_pairs(u, b);
    gate_products<T>(p.activation, a, b);
    from_pairs(a, g);
    pack_columns<T>(g, product);
}
// 64 columns of hidden from `c` on, and of gate_up where it is wanted.
template <typename T>
__device__ __forceinline__ void write_gated(const TensorProduct &p, unsigned char *staged, int lane, const uint32_t (&gate)[2][16],
                                            const uint32_t (&up)[2][16], const uint32_t (&product)[2][16], int64_t row, int rows,
                                            int c) {
    const int cols = min(64, p.N - c);
    write_packed<T>(staged, lane, product, (T *)p.out + row * p.os + c, p.os, rows, cols, p.whole_out);
    if (p.gate_up != nullptr) {
        T *z = (T *)p.gate_up + row * p.gs + c;
        write_packed<T>(staged, lane, gate, z, p.gs, rows, cols, p.whole_gate);
        write_packed<T>(staged, lane, up, z + p.N, p.gs, rows, cols, p.whole_gate && p.N % 8 == 0);
    }
}

// What a warp writes of a tile of rows: 32 rows from `row`, `rows` of which exist,
// and its half of the tile's columns, from TMEM column `from` on.  `some`: there
// are sums, otherwise `fill` stands for them.  `release`: the sums have been read.
template <typename T, int EPI, typename Release>
__device__ __forceinline__ void finish_rows(const TensorProduct &p, unsigned char *staged, int lane, uint32_t from,
                                            bool some, float fill, int64_t row, int rows, int c, Release release) {
    if constexpr (EPI == STORE) {
        // (32 columns read at a time, in the middle of the writes: 64, or all before the
        // writes, are slower, 330 us against 289 for 262,144 x 1024 through 768)
#pragma unroll 1
        for (int i = 0; i < 2; ++i, c += 64, from += 64) {
            uint32_t w[2][16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[32];
                load_sums(v, from + h * 32, some, fill);
                pack_columns<T>(v, w[h]);
                stage_columns(staged, lane, h, w[h]);
            }
            write_columns<T>(staged, lane, (T *)p.out + row * p.os + c, p.os, rows, min(64, p.N - c), p.whole_out);
        }
        if (some) release();
    } else {
        // the gate's sums, the others 128 columns further, and the product
        uint32_t gate[2][16], up[2][16], product[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float g[32], u[32];
            load_sums(g, u, from + h * 32, from + 128 + h * 32, some, fill);
            if (h == 1 && some) release();
            pack_gated<T>(p, g, u, gate[h], up[h], product[h]);
        }
        write_gated<T>(p, staged, lane, gate, up, product, row, rows, c);
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
    // FULL: all 32 rows and columns exist, in aligned vectors.  (Rows behind the last
    // group are not read: they may hold anything.)
    template <bool FULL>
    __device__ __forceinline__ void load(const TensorProduct &p, int lane, bool some, int64_t row, int rows, int c) {
        const int j = c + (lane & 7) * 4, left = p.N - j;
        const T *z = (const T *)p.gate_up + (row + (lane >> 3)) * p.gs + j, *y = z + p.N;
        const int64_t step = 4 * p.gs;
#pragma unroll
        for (int i = 0; i < 8; ++i, z += step, y += step) {
            if constexpr (FULL) {
                g[i] = load_raw<T, 4>(z);
                u[i] = load_raw<T, 4>(y);
            } else {
                const bool here = some && i * 4 + (lane >> 3) < rows;
                if (here && p.whole_gate && left >= 4) {
                    g[i] = load_raw<T, 4>(z);
                    u[i] = load_raw<T, 4>(y);
                } else {
                    uint16_t h[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[k] = here && k < left ? *(const uint16_t *)(z + k) : 0;
                        h[4 + k] = here && k < left ? *(const uint16_t *)(y + k) : 0;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        g[i].w[k] = h[2 * k] | (uint32_t)h[2 * k + 1] << 16;
                        u[i].w[k] = h[4 + 2 * k] | (uint32_t)h[5 + 2 * k] << 16;
                    }
                }
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void store_four(T *out, const Raw<T, 4> &f, int left, bool whole) {
    if (whole && left >= 4) {
        store_raw<T, 4>(out, f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= left) continue;
            if constexpr (sizeof(T) == 4) *(uint32_t *)(out + k) = f.w[k];
            else *(uint16_t *)(out + k) = (uint16_t)(f.w[k >> 1] >> (16 * (k & 1)));
        }
    }
}
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

// The staged 32 rows x 32 sums to `out`, `rows` and `cols` of which exist.
template <typename T>
__device__ __forceinline__ void write_rows(const unsigned char *staged, int lane, T *out, int64_t stride, int rows, int cols,
                                           bool whole) {
    __syncwarp();
    const int left = cols - (lane & 7) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (lane >> 3);
        const float4 q = staged_sums(staged, lane, i);
        const float f[4] = {q.x, q.y, q.z, q.w};
        if (row < rows) store_four<T>(out + row * stride + (lane & 7) * 4, f, left, whole);
    }
    __syncwarp();
}

// Four elements of a row, `left` of which exist (the others are 0).
template <typename T> __device__ __forceinline__ void load_four(const T *p, float (&f)[4], int left, bool whole) {
    if (whole && left >= 4) {
        widen<T, 4>(load_raw<T, 4>(p), f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = k < left ? to_f32(p[k]) : 0.f;
    }
}

// The staged 32 rows x 32 columns of dh through the gate, read here: [dg | du].
// Rows without products (`some` false) get zeros, and their gate is not read.
template <typename T>
__device__ __forceinline__ void write_gate_grad(const TensorProduct &p, const unsigned char *staged, int lane, bool some,
                                                int64_t row, int rows, int c) {
    __syncwarp();
    const int j = c + (lane & 7) * 4, left = p.N - j;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        const float4 q = staged_sums(staged, lane, i);
        const float dh[4] = {q.x, q.y, q.z, q.w};
        float g[4], u[4];
        const int read = some && r < rows ? left : 0;
        const T *z = (const T *)p.gate_up + (row + r) * p.gs + j;
        load_four<T>(z, g, read, p.whole_gate);
        load_four<T>(z + p.N, u, read, p.whole_gate);
        Pair a[2], b[2], d[2];
        to_pairs(g, a);
        to_pairs(u, b);
        to_pairs(dh, d);
        gate_gradients<T>(p.activation, d, a, b);
        from_pairs(a, g);
        from_pairs(b, u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            g[k] = some ? g[k] : 0.f;
            u[k] = some ? u[k] : 0.f;
        }
        if (r < rows) {
            T *out = (T *)p.out + (row + r) * p.os + j;
            store_four<T>(out, g, left, p.whole_out);
            store_four<T>(out + p.N, u, left, p.whole_out);
        }
    }
    __syncwarp();
}

// The staged 32 rows x 32 columns of dh through the gate: [dg | du].
template <typename T, bool FULL>
__device__ __forceinline__ void write_gate_grad(const TensorProduct &p, const unsigned char *staged, const GateUp<T> &z,
                                                int lane, bool some, int64_t row, int rows, int c) {
    __syncwarp();
    const int j = c + (lane & 7) * 4, left = p.N - j;
    T *out = (T *)p.out + (row + (lane >> 3)) * p.os + j, *other = out + p.N;
    const int64_t step = 4 * p.os;
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 4) {
        Pair g[8], u[8], dh[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 q = staged_sums(staged, lane, i0 + i);
            dh[2 * i] = pair(q.x, q.y);
            dh[2 * i + 1] = pair(q.z, q.w);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                g[2 * i + k] = widen_pair<T, 4>(z.g[i0 + i], k);
                u[2 * i + k] = widen_pair<T, 4>(z.u[i0 + i], k);
            }
        }
        if (FULL || some) {
            gate_gradients<T>(p.activation, dh, g, u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = u[i] = pair(0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i, out += step, other += step) {
            Raw<T, 4> a, b;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                narrow_pair<T, 4>(a, k, g[2 * i + k]);
                narrow_pair<T, 4>(b, k, u[2 * i + k]);
            }
            if constexpr (FULL) {
                store_raw<T, 4>(out, a);
                store_raw<T, 4>(other, b);
            } else if ((i0 + i) * 4 + (lane >> 3) < rows) {
                store_four(out, a, left, p.whole_out);
                store_four(other, b, left, p.whole_out);
            }
        }
    }
    __syncwarp();
}

// What finish_rows and the gate's gradient do, from sums in registers (four times 32
// columns; GATED: the gate's first).
template <typename T, int EPI>
__device__ __forceinline__ void finish_sums(const TensorProduct &p, unsigned char *staged, int lane, float (&sum)[4][32],
                                            bool some, int64_t row, int rows, int c) {
    if constexpr (EPI == GATE_GRAD) {
        auto finish = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                GateUp<T> z;
                z.template load<FULL>(p, lane, some, row, rows, c + i * 32);
                stage_sums(staged, lane, sum[i]);
                write_gate_grad<T, FULL>(p, staged, z, lane, some, row, rows, c + i * 32);
            }
        };
        if (some && rows == 32 && p.N - c >= 128 && p.whole_out && p.whole_gate) finish(std::true_type());
        else finish(std::false_type());
    } else if constexpr (EPI == GATED) {
        uint32_t gate[2][16], up[2][16], product[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h) pack_gated<T>(p, sum[h], sum[2 + h], gate[h], up[h], product[h]);
        write_gated<T>(p, staged, lane, gate, up, product, row, rows, c);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[2][16];
            pack_columns<T>(sum[2 * i], w[0]);
            pack_columns<T>(sum[2 * i + 1], w[1]);
            const int at = c + 64 * i;
            write_packed<T>(staged, lane, w, (T *)p.out + row * p.os + at, p.os, rows, min(64, p.N - at), p.whole_out);
        }
    }
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
//
// 256 columns of a pair take each operand once from L2 for 256 products; at 8192 x
// 8192 x 8192 the tensor cores bound it: 1800 TFLOP/s in bf16 (WEIGHTS, whose sums
// leave TMEM in segments: 1660).  At 262,144 rows of 128 experts, 1024 through 768,
// the epilogues' writes and the experts' last, partly empty tiles add a fifth.
// LONG: products of rows whose sums leave TMEM in segments as well.
template <typename T, int FORM, int EPI, bool LONG = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TC_THREADS, 1)
product_tensor_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap amap_few,
                      const __grid_constant__ CUtensorMap bmap, const TensorProduct p) {
    extern __shared__ unsigned char dynamic[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    const int STAGES = p.stages;
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
        bars.loaded = 0;
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
    constexpr bool SEGMENTS = FORM == WEIGHTS || LONG;
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
        const int SEGMENT = p.segment;
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
            if (lane == 0) tc::bar_arrive_cluster_relaxed(taken0 + 8 * (turn & 1));
            ++turn;
        };
        const float given_up = __int_as_float(0x7FC00000);      // NaN where products are missing
        for (int64_t t = t0; t < total; t += step) {
            const TensorTile a = tile_at(t);
            const bool some = a.s1 > a.s0;
            const int row = a.r0 + (int)rank * 128 + quarter * 32, rows = min(32, a.r1 - row);
            if constexpr (SEGMENTS) {
                if (FORM == WEIGHTS && !some && p.accumulate) continue;
                float sum[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
                for (int begin = a.s0; begin < a.s1; begin = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1) {
                    wait_sums();
                    if (alive) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v[32];
                            const int column = EPI == GATED ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * 128 + i * 32;
                            load_sums(v, lanes + (turn & 1) * 256 + column, true, 0.f);
#pragma unroll
                            for (int j = 0; j < 32; ++j) sum[i][j] += v[j];
                        }
                        release_sums();
                    }
                }
                __syncwarp();
                if (some && !alive) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[i][j] = given_up;
                }
                if constexpr (FORM == WEIGHTS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = a.c + half * 128 + i * 32, cols = min(32, p.N - c);
                        stage_sums(staged, lane, sum[i]);
                        const int64_t slice = p.slices > 1 ? (int64_t)a.slice * p.groups.experts * p.oe : 0;
                        const int64_t at = slice + (int64_t)a.e * p.oe + (int64_t)row * p.os + c;
                        if (p.out_f32) write_weights((float *)p.out + at, p, staged, lane, rows, cols);
                        else write_weights((T *)p.out + at, p, staged, lane, rows, cols);
                    }
                } else {
                    finish_sums<T, EPI>(p, staged, lane, sum, some, row, rows, a.c + half * (WIDTH / 2));
                }
            } else {
                if constexpr (EPI == GATE_GRAD) {
                    // a chunk's gate is loaded while the one before it is finished
                    const int c = a.c + half * 128;
                    auto finish = [&](auto full) {
                        constexpr bool FULL = decltype(full)::value;
                        GateUp<T> z;
                        z.template load<FULL>(p, lane, some, row, rows, c);
                        if (some) wait_sums();
                        const uint32_t from = lanes + (turn & 1) * 256 + half * 128;
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            float v[32];
                            load_sums(v, from + i * 32, some && alive, some ? given_up : 0.f);
                            if (i == 3 && some && alive) release_sums();
                            stage_sums(staged, lane, v);
                            GateUp<T> now = z;
                            if (i < 3) z.template load<FULL>(p, lane, some, row, rows, c + (i + 1) * 32);
                            write_gate_grad<T, FULL>(p, staged, now, lane, some, row, rows, c + i * 32);
                        }
                    };
                    if (some && rows == 32 && p.N - c >= 128 && p.whole_out && p.whole_gate) finish(std::true_type());
                    else finish(std::false_type());
                    continue;
                }
                if constexpr (EPI != GATE_GRAD) {
                    if (some) wait_sums();
                    finish_rows<T, EPI>(p, staged, lane, lanes + (turn & 1) * 256 + half * (WIDTH / 2), some && alive,
                                        some ? given_up : 0.f, row, rows, a.c + half * (WIDTH / 2), release_sums);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TC_CONTROL_REGS));
        if (warp == 0) {
            if (lane == 0) {
                uint32_t stage = 0, phase = 0, steps = 0;
                const uint32_t full0 = tc::of_rank(full, 0);
                for (int64_t t = t0; t < total && alive; t += step) {
                    const TensorTile a = tile_at(t);
                    // Boxes of 32 rows that this CTA and both load: groups that end early leave
                    // the others' rows as they are (they reach only rows that are not written)
                    auto boxes_of = [&](int r) { return max(0, min(4, (a.r1 - a.r0 - r * 128 + 31) / 32)); };
                    const int boxes = FORM == WEIGHTS ? 4 : boxes_of((int)rank), all = FORM == WEIGHTS ? 8 : boxes_of(0) + boxes_of(1);
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
                            tc::bar_expect(full + 8 * stage, 2 * TC_OPERAND + all * (TC_OPERAND / 4));
                        }
                        if (p.withhold) {
                            // (nothing is loaded: the waits for it give up)
                        } else if constexpr (FORM == WEIGHTS) {
                            *(volatile uint32_t *)&bars.loaded = ++steps;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                tc::load_box(at + j * (TC_OPERAND / 2), &amap, bar, a.r0 + rank * 128 + j * 64, s, 0);
                                tc::load_box(bt + j * (TC_OPERAND / 2), &bmap, bar, a.c + rank * 128 + j * 64, s, 0);
                            }
                        } else {
                            if (boxes == 4) {
                                tc::load_box(at, &amap, bar, s, a.r0 + rank * 128, 0);
                            } else {
                                for (int j = 0; j < boxes; ++j)
                                    tc::load_box(at + j * (TC_OPERAND / 4), &amap_few, bar, s, a.r0 + rank * 128 + j * 32, 0);
                            }
                            if constexpr (FORM == ROWS) {
                                tc::load_box(bt, &bmap, bar, s, a.c + (EPI == GATED ? rank * p.N : rank * 128), a.e);
                            } else {
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    tc::load_box(bt + j * (TC_OPERAND / 2), &bmap, bar, a.c + rank * 128 + j * 64, s, a.e);
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
                const int SEGMENT = SEGMENTS ? p.segment : INT_MAX;
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
            // The next such step may lie any number of tiles ahead: the wait for it gives up
            // only when no step has been loaded for as long as a wait lasts.
            auto wait_tail = [&](uint32_t bar, uint32_t parity) {
                for (;;) {
                    const uint32_t before = *(volatile uint32_t *)&bars.loaded;
                    if (tc::bar_wait(bar, parity)) return true;
                    if (*(volatile uint32_t *)&bars.loaded == before) return false;
                }
            };
            for (int64_t t = t0; t < total && alive; t += step) {
                const TensorTile a = tile_at(t);
                chunks += (a.s1 - a.s0 + TC_K - 1) / TC_K;
                const int rows = (a.s1 - a.s0) % TC_K;
                if (rows == 0) continue;
                const uint32_t stage = (chunks - 1) % STAGES;
                alive = wait_tail(tail + 8 * stage, (turns >> stage) & 1);
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

// ---------------------------------------------------------------------------
// Any type, stride and place: 128 x 128 tiles by one CTA, whose warps load the
// operands.
//
// FP32 operands are cut into three BF16 pieces, x = x0 + x1 + x2 exactly (8 bits
// each, rounded to the nearest; below 2^-110 to within 2^-134, half of BF16's smallest
// number), and six of the nine products of pieces are summed: x0 y0 by itself, and
// x0 y1, x1 y0, x0 y2, x2 y0, x1 y1, which are 2^-7 of it at most; the three left out
// are below 2^-24.  The tensor core cuts sums off
// instead of rounding (2^-27.3 of a sum for each term), so x0 y0 leaves it after 128
// terms to be summed in registers, the others, which lose 2^-8 of that each, after
// 2048.
//
// The loading warps bound it: at 8192 x 2048 x 2048 it reaches 146 TFLOP/s in FP32
// (1.5e-7 of the result), six times as many on the tensor cores; at 8192 x 2047 x
// 2047, whose rows have no vectors, 117 and, in 16 bits, 246.

constexpr int GEN_TILE = 128, GEN_EPILOGUE = 8;
constexpr int GEN_PIECE = GEN_TILE * TC_K * 2;      // bytes of a piece of an operand's step
// Warps that load, four for control, eight that finish the sums, and how they
// divide the registers of the launch.  FP32: eight loading warps of many registers
// (16 of fewer are a tenth slower); 16 bits: 16, which have two steps under way (a
// third faster than 8).
template <bool F32> struct GenWarps {
    static constexpr int LOADERS = F32 ? 8 : 16, THREADS = 32 * (LOADERS + 4 + GEN_EPILOGUE);
    static constexpr int LAUNCH = F32 ? 96 : 72, LOAD = F32 ? 104 : 64, CONTROL = F32 ? 64 : 56, EPILOGUE = F32 ? 104 : 96;
    static_assert(32 * (LOADERS * LOAD + 4 * CONTROL + GEN_EPILOGUE * EPILOGUE) <= THREADS * LAUNCH,
                  "an increase beyond the launch's registers never ends");
    static_assert(CONTROL <= LAUNCH && EPILOGUE >= LAUNCH,
                  "an increase to fewer registers, or a decrease to more, is an illegal instruction");
};
template <typename T> constexpr int gen_pieces() { return sizeof(T) == 4 ? 3 : 1; }
template <typename T> constexpr int gen_stages() { return sizeof(T) == 4 ? 2 : 5; }
constexpr int GEN_SMALL = 2048;     // terms after which the small products' sums leave: whole segments
template <typename T> constexpr int gen_segment() { return sizeof(T) == 4 ? 128 : TC_SEGMENT; }
static_assert(GEN_SMALL % gen_segment<float>() == 0, "small sums end with a segment");

struct GeneralProduct {
    TensorProduct t;
    const void *a, *b;          // rows (WEIGHTS: grad_out), weight (WEIGHTS: rows)
    int64_t as, bs, be;         // strides of their rows, of the experts
    int whole_a, whole_b;       // rows of 16-byte vectors
};

struct GeneralBars {
    uint64_t full[5], empty[5], sums[2], taken[2], small_taken[2];
    uint32_t tmem;
};

// Eight consecutive elements of a row, as they were read.  FP32: one by one where
// the rows are not of 16-byte vectors.  16 bits: then from the two aligned vectors
// that hold them, where these lie in the row as well; they are moved into place
// when they are used, so that no load is waited for before the next is issued.
template <typename T> struct Cell {
    uint32_t w[8];
    uint32_t shift;     // 16 bits: elements before the first
};

// From column `col` of a row of `cols` on; elements that do not exist are 0.
template <typename T> __device__ __forceinline__ void load_cell(Cell<T> &r, const T *row, int col, int cols, bool whole) {
    const T *p = row + col;
    r.shift = 0;
    if (whole && col + 8 <= cols) {
        const Raw<T, 8> q = load_raw<T, 8>(p);
#pragma unroll
        for (int i = 0; i < Raw<T, 8>::WORDS; ++i) r.w[i] = q.w[i];
        return;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k] = col + k < cols ? *(const uint32_t *)(p + k) : 0u;
    } else {
        const int shift = (int)(((uintptr_t)p / 2) % 8);
        if (col >= shift && col - shift + 16 <= cols) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p - shift), b = *reinterpret_cast<const uint4 *>(p - shift + 8);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            r.shift = shift;
            return;
        }
        uint16_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = col + k < cols ? *(const uint16_t *)(p + k) : (uint16_t)0;
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = h[2 * k] | (uint32_t)h[2 * k + 1] << 16;
    }
}
// 16 bits: the eight elements.
template <typename T> __device__ __forceinline__ uint4 cell_words(const Cell<T> &r) {
    uint32_t w[7];
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = r.shift & 4 ? r.w[i + 2] : r.w[i];
    w[6] = r.w[6];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = r.shift & 2 ? w[i + 1] : w[i];
    const uint32_t bits = (r.shift & 1) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Tile number t: of the groups' rows and all columns, or (WEIGHTS) of the experts'
// slices and their matrices; e < 0 beyond the last.  By a whole warp.
template <int FORM>
__device__ __forceinline__ TensorTile general_tile(const TensorProduct &p, int64_t t, int lane) {
    TensorTile r;
    r.slice = 0;
    if constexpr (FORM == WEIGHTS) {
        const int64_t per = (int64_t)p.tiles_m * p.tiles_n, g = t / per;
        r.e = (int)(g / p.slices);
        if (r.e >= p.groups.experts) {
            r.e = -1;
            return r;
        }
        r.slice = (int)(g % p.slices);
        const int i = (int)(t - g * per);
        r.r0 = i / p.tiles_n * GEN_TILE;
        r.r1 = p.M;
        r.c = i % p.tiles_n;
        r.s0 = group_start(p.groups, r.e);
        r.s1 = max(r.s0, group_start(p.groups, r.e + 1));
        if (p.slices > 1) {
            const int each = ((r.s1 - r.s0 + p.slices - 1) / p.slices + TC_K - 1) / TC_K * TC_K;
            r.s0 = min(r.s1, r.s0 + r.slice * each);
            r.s1 = min(r.s1, r.s0 + each);
        }
    } else {
        const int64_t row_tile = t / p.tiles_n;
        if (row_tile > INT_MAX) {
            r.e = -1;
            return r;
        }
        const RowTile f = find_tile<GEN_TILE>(p.groups, (int)row_tile, lane);
        r.e = f.e;
        r.r0 = f.r0;
        r.r1 = f.r1;
        r.c = (int)(t - row_tile * p.tiles_n);
        r.s0 = 0;
        r.s1 = f.e < p.groups.experts ? p.K : 0;
    }
    return r;
}

template <typename T, int FORM, int EPI>
__global__ void __launch_bounds__(GenWarps<sizeof(T) == 4>::THREADS, 1) product_general_kernel(const __grid_constant__ GeneralProduct g) {
    using Warps = GenWarps<sizeof(T) == 4>;
    constexpr int GEN_LOADERS = Warps::LOADERS;
    constexpr int PIECES = gen_pieces<T>(), STAGES = gen_stages<T>(), SEGMENT = gen_segment<T>();
    constexpr int STAGE = 2 * PIECES * GEN_PIECE;
    constexpr int WIDTH = EPI == GATED ? GEN_TILE / 2 : GEN_TILE;       // columns of a tile
    constexpr bool A_ACROSS = FORM == WEIGHTS, B_ACROSS = FORM != ROWS;
    const TensorProduct &p = g.t;
    extern __shared__ unsigned char dynamic[];
    unsigned char *smem = (unsigned char *)(((uintptr_t)dynamic + 1023) & ~(uintptr_t)1023);
    unsigned char *staging = smem + STAGES * STAGE;
    GeneralBars &bars = *(GeneralBars *)(staging + GEN_EPILOGUE * TC_STAGED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tiles0 = tc::smem_u32(smem), full = tc::smem_u32(bars.full), empty = tc::smem_u32(bars.empty),
                   sums = tc::smem_u32(bars.sums), taken = tc::smem_u32(bars.taken), small_taken = tc::smem_u32(bars.small_taken);
    if (warp == GEN_LOADERS) {
        if (lane == 0) {
            for (int i = 0; i < STAGES; ++i) {
                tc::bar_init(full + 8 * i, GEN_LOADERS);
                tc::bar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                tc::bar_init(sums + 8 * i, 1);
                tc::bar_init(taken + 8 * i, GEN_EPILOGUE);
                tc::bar_init(small_taken + 8 * i, GEN_EPILOGUE);
            }
            tc::fence_bar_init();
        }
        __syncwarp();
        tc::tmem_alloc1(&bars.tmem, 512);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    launch_dependents();
    const uint32_t tmem = bars.tmem;
    bool alive = true;

    if (warp < GEN_LOADERS) {
        if constexpr (Warps::LOAD > Warps::LAUNCH) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Warps::LOAD));
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Warps::LOAD));
        // A step has 2048 cells of 8 elements, as many of each operand: of the first,
        // cell thread + i * threads lies in line (thread >> 3) + i * LINES, at place
        // thread & 7 of it.
        // Lines are rows of an operand that is contiguous along what is summed, and
        // otherwise what is summed, twice 64 of them for 128 columns.
        // The next step is under way while one is stored.
        constexpr int LINES = GEN_LOADERS * 4, EACH = GEN_TILE / LINES;
        const int unit = threadIdx.x & 7, line0 = threadIdx.x >> 3;
        uint32_t stage = 0, phase = 0;
        Cell<T> cells[2 * EACH];
        int64_t t = blockIdx.x;
        TensorTile tile = general_tile<FORM>(p, t, lane);
        auto skip = [&]() {     // to the next tile that has products
            while (tile.e >= 0 && tile.s1 <= tile.s0) {
                t += gridDim.x;
                tile = general_tile<FORM>(p, t, lane);
            }
        };
        skip();
        int s = tile.s0;        // next step to load
        // the step's cells, and on to the next step
        auto load = [&]() {
            const T *b = (const T *)g.b + (FORM == WEIGHTS ? 0 : tile.e * g.be);
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int line = line0 + LINES * i;
                int64_t row;
                int col, cols;
                bool here;
                if constexpr (A_ACROSS) {
                    row = s + (line & 63);
                    col = tile.r0 + (line & 64) + unit * 8;
                    cols = p.M;
                    here = row < tile.s1;
                } else {
                    row = tile.r0 + line;
                    col = s + unit * 8;
                    cols = p.K;
                    here = row < tile.r1;
                }
                load_cell<T>(cells[i], (const T *)g.a + row * g.as, col, here ? cols : 0, g.whole_a);
                if constexpr (B_ACROSS) {
                    row = s + (line & 63);
                    col = tile.c * WIDTH + (line & 64) + unit * 8;
                    cols = p.N;
                    here = row < tile.s1;
                } else {
                    const int n = tile.c * WIDTH + (EPI == GATED ? line & 63 : line);
                    row = n + (EPI == GATED && line >= 64 ? p.N : 0);
                    col = s + unit * 8;
                    cols = p.K;
                    here = n < p.N;
                }
                load_cell<T>(cells[EACH + i], b + row * g.bs, col, here ? cols : 0, g.whole_b);
            }
            s += TC_K;
            if (s >= tile.s1) {
                t += gridDim.x;
                tile = general_tile<FORM>(p, t, lane);
                skip();
                s = tile.s0;
            }
        };
        auto store = [&]() {
#pragma unroll
            for (int i = 0; i < 2 * EACH; ++i) {
                const int line = line0 + LINES * (i % EACH);
                uint4 *at = (uint4 *)(smem + stage * STAGE + i / EACH * PIECES * GEN_PIECE + line * 128 + ((unit ^ (line & 7)) << 4));
                if constexpr (PIECES == 1) {
                    *at = cell_words(cells[i]);
                } else {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(cells[i].w[k]);
#pragma unroll
                    for (int piece = 0; piece < 3; ++piece) {
                        const Raw<__nv_bfloat16, 8> q = narrow<__nv_bfloat16, 8>(f);
                        at[piece * (GEN_PIECE / 16)] = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
                        if (piece < 2) {
                            float w[8];
                            widen<__nv_bfloat16, 8>(q, w);
                            // (an infinite piece leaves nothing)
#pragma unroll
                            for (int k = 0; k < 8; ++k) f[k] = fabsf(w[k]) <= 3.402823466e38f ? f[k] - w[k] : 0.f;
                        }
                    }
                }
            }
        };
        bool some = tile.e >= 0;
        if (some) load();
        while (some) {
            alive = __all_sync(FULL, tc::bar_wait(empty + 8 * stage, phase ^ 1));
            if (!alive) break;
            store();
            some = tile.e >= 0;
            if (some) load();
            tc::fence_smem_writes();
            __syncwarp();
            if (lane == 0 && !p.withhold) tc::bar_arrive(full + 8 * stage);
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
    } else if (warp >= GEN_LOADERS + 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Warps::EPILOGUE));
        const int quarter = warp & 3, half = (warp - GEN_LOADERS - 4) >> 2;
        unsigned char *staged = staging + (warp - GEN_LOADERS - 4) * TC_STAGED;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        // GATED: the gate's columns and the same of the other half
        const int c0 = EPI == GATED ? half * 32 : half * 64, c1 = EPI == GATED ? 64 + half * 32 : half * 64 + 32;
        const float given_up = __int_as_float(0x7FC00000);      // NaN where products are missing
        int turn = 0, smalls = 0;
        for (int64_t t = blockIdx.x;; t += gridDim.x) {
            const TensorTile a = general_tile<FORM>(p, t, lane);
            if (a.e < 0) break;
            const bool some = a.s1 > a.s0;
            if (FORM == WEIGHTS && !some && p.accumulate) continue;
            float v[32], u[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = u[j] = 0.f;
            auto gather = [&](uint32_t from) {
                float more[32];
                load_sums(more, from + c0, true, 0.f);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += more[j];
                load_sums(more, from + c1, true, 0.f);
#pragma unroll
                for (int j = 0; j < 32; ++j) u[j] += more[j];
            };
            for (int begin = a.s0; begin < a.s1; begin = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1) {
                if (alive) alive = tc::bar_wait(sums + 8 * (turn & 1), (turn >> 1) & 1);
                alive = __all_sync(FULL, alive);
                tc::fence_after();
                if (!alive) continue;
                gather(lanes + (turn & 1) * GEN_TILE);
                tc::fence_before();
                if (lane == 0) tc::bar_arrive(taken + 8 * (turn & 1));
                ++turn;
                const int end = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1;
                if (PIECES > 1 && (end == a.s1 || (end - a.s0) % GEN_SMALL == 0)) {
                    // (the sums' arrival stands for these as well)
                    gather(lanes + 2 * GEN_TILE + (smalls & 1) * GEN_TILE);
                    tc::fence_before();
                    if (lane == 0) tc::bar_arrive(small_taken + 8 * (smalls & 1));
                    ++smalls;
                }
            }
            if (!alive) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = u[j] = given_up;
            }
            const int row = a.r0 + quarter * 32, rows = min(32, a.r1 - row), c = a.c * WIDTH + c0;
            if constexpr (FORM == WEIGHTS) {
                const int64_t slice = p.slices > 1 ? (int64_t)a.slice * p.groups.experts * p.oe : 0;
                const int64_t at = slice + (int64_t)a.e * p.oe + (int64_t)row * p.os + c;
                auto put = [&](const float (&f)[32], int64_t at, int cols) {
                    stage_sums(staged, lane, f);
                    if (p.out_f32) write_weights((float *)p.out + at, p, staged, lane, rows, cols);
                    else write_weights((T *)p.out + at, p, staged, lane, rows, cols);
                };
                put(v, at, min(32, p.N - c));
                put(u, at + 32, min(32, p.N - c - 32));
            } else if constexpr (EPI == GATED) {
                const int cols = min(32, p.N - c);
                if (p.gate_up != nullptr) {
                    T *z = (T *)p.gate_up + (int64_t)row * p.gs + c;
                    stage_sums(staged, lane, v);
                    write_rows<T>(staged, lane, z, p.gs, rows, cols, p.whole_gate);
                    stage_sums(staged, lane, u);
                    write_rows<T>(staged, lane, z + p.N, p.gs, rows, cols, p.whole_gate);
                }
                Pair pv[16], pu[16];
                to_pairs(v, pv);
                to_pairs(u, pu);
                gate_products<T>(p.activation, pv, pu);
                from_pairs(pv, v);
                stage_sums(staged, lane, v);
                write_rows<T>(staged, lane, (T *)p.out + (int64_t)row * p.os + c, p.os, rows, cols, p.whole_out);
            } else if constexpr (EPI == GATE_GRAD) {
                stage_sums(staged, lane, v);
                write_gate_grad<T>(p, staged, lane, some, row, rows, c);
                stage_sums(staged, lane, u);
                write_gate_grad<T>(p, staged, lane, some, row, rows, c + 32);
            } else {
                T *out = (T *)p.out + (int64_t)row * p.os + c;
                stage_sums(staged, lane, v);
                write_rows<T>(staged, lane, out, p.os, rows, min(32, p.N - c), p.whole_out);
                stage_sums(staged, lane, u);
                write_rows<T>(staged, lane, out + 32, p.os, rows, min(32, p.N - c - 32), p.whole_out);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Warps::CONTROL));
        if (warp == GEN_LOADERS) {
            using Piece = typename std::conditional<sizeof(T) == 4, __nv_bfloat16, T>::type;
            constexpr uint32_t idesc = tc::instruction<Piece, A_ACROSS, B_ACROSS>(GEN_TILE, GEN_TILE);
            uint32_t stage = 0, phase = 0;
            int turn = 0, smalls = -1;
            for (int64_t t = blockIdx.x; alive; t += gridDim.x) {
                const TensorTile a = general_tile<FORM>(p, t, lane);
                if (a.e < 0) break;
                if (a.s1 <= a.s0) continue;
                for (int begin = a.s0; begin < a.s1 && alive; begin = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1, ++turn) {
                    const uint32_t acc = tmem + (turn & 1) * GEN_TILE;
                    const int end = a.s1 - begin > SEGMENT ? begin + SEGMENT : a.s1;
                    alive = __all_sync(FULL, tc::bar_wait(taken + 8 * (turn & 1), ((turn >> 1) & 1) ^ 1));
                    const bool first = (begin - a.s0) % GEN_SMALL == 0;     // of the small sums
                    if (PIECES > 1 && first) {
                        ++smalls;
                        if (alive) alive = __all_sync(FULL, tc::bar_wait(small_taken + 8 * (smalls & 1), ((smalls >> 1) & 1) ^ 1));
                    }
                    const uint32_t small = tmem + 2 * GEN_TILE + (smalls & 1) * GEN_TILE;
                    for (int s = begin; s < end && alive; s += TC_K) {
                        alive = __all_sync(FULL, tc::bar_wait(full + 8 * stage, phase));
                        if (!alive) break;
                        tc::fence_after();
                        if (lane == 0) {
                            const uint32_t at = tiles0 + stage * STAGE, bt = at + PIECES * GEN_PIECE;
                            const int steps = min(TC_K, a.s1 - s);
                            for (int k = 0; k * 16 < steps; ++k) {
                                const uint32_t ak = at + k * (A_ACROSS ? 2048 : 32), bk = bt + k * (B_ACROSS ? 2048 : 32);
                                auto product = [&](uint32_t d, int i, int j, bool add) {
                                    tc::mma1(d, tc::operand<A_ACROSS>(ak + i * GEN_PIECE, GEN_PIECE / 2),
                                             tc::operand<B_ACROSS>(bk + j * GEN_PIECE, GEN_PIECE / 2), idesc, add);
                                };
                                product(acc, 0, 0, s > begin || k > 0);
                                if (PIECES > 1) {
                                    product(small, 0, 1, !first || s > begin || k > 0);
                                    product(small, 1, 0, true);
                                    product(small, 0, 2, true);
                                    product(small, 2, 0, true);
                                    product(small, 1, 1, true);
                                }
                            }
                            tc::commit1(empty + 8 * stage);
                            if (s + TC_K >= end) tc::commit1(sums + 8 * (turn & 1));
                        }
                        __syncwarp();
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
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
    }
    if (!alive) {
        if (p.status != nullptr) atomicOr(p.status + 1, TBE_FLAG_MMA_TIMEOUT);
        tc::wait_out();
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == GEN_LOADERS) tc::tmem_free1(tmem, 512);
}

// ---------------------------------------------------------------------------
// Few rows (the newest tokens of a few sequences): the weights are read by a warp two
// rows of theirs, against up to FEW_ROWS rows of a group at a time, and again for each
// FEW_ROWS more.  HBM bounds it: the tensor cores' tiles, of which there are too few to
// cover the latency of loads, take 36 us for one token through 8 experts of 2048 x 1024.

// Rows of a call that this serves: 16 by experts (1 token of 8 experts: 27 us
// against 36; 16 rows of as many experts 39 against 57, of one 35 against 38), 4 of
// a dense layer (4096 x 4096: 1 row 10 us against 27, 4 rows 21, 8 rows 29).
constexpr int FEW_ROWS = 4, FEW_WARPS = 4, FEW_MOST = 16, FEW_MOST_DENSE = 4;

template <typename T, int EPI, bool WHOLE>
__global__ void __launch_bounds__(32 * FEW_WARPS) product_few_kernel(const __grid_constant__ GeneralProduct g) {
    // two rows of the weight a warp: neighbours, or (GATED) of the gate and the other half
    constexpr int MATRICES = 2, VEC = WHOLE ? 16 / sizeof(T) : 1, U = WHOLE ? 4 : 8;
    const TensorProduct &p = g.t;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const RowTile tile = find_tile<FEW_ROWS>(p.groups, blockIdx.y, lane);
    const int n = (blockIdx.x * FEW_WARPS + warp) * (EPI == GATED ? 1 : 2);
    if (tile.e < 0 || n >= p.N) return;
    // from the first to the second (the last row of an odd number is taken twice)
    const int64_t second = (EPI == GATED ? p.N : n + 1 < p.N ? 1 : 0) * g.bs;
    const int rows = tile.r1 - tile.r0;
    float acc[MATRICES][FEW_ROWS] = {};
    if (tile.e < p.groups.experts) {
        const T *x = (const T *)g.a + tile.r0 * g.as, *w = (const T *)g.b + tile.e * g.be + n * g.bs;
        const int vectors = p.K / VEC;
        for (int v0 = lane; v0 < vectors; v0 += 32 * U) {
            Raw<T, VEC> q[MATRICES][U];
#pragma unroll
            for (int m = 0; m < MATRICES; ++m)
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (v0 + 32 * i < vectors)
                        q[m][i] = load_raw<T, VEC, true>(w + m * second + (int64_t)(v0 + 32 * i) * VEC);
#pragma unroll
            for (int r = 0; r < FEW_ROWS; ++r) {
                if (r >= rows) break;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (v0 + 32 * i < vectors) {
                        float a[VEC];
                        widen<T, VEC>(load_raw<T, VEC>(x + r * g.as + (int64_t)(v0 + 32 * i) * VEC), a);
#pragma unroll
                        for (int m = 0; m < MATRICES; ++m) {
                            float b[VEC];
                            widen<T, VEC>(q[m][i], b);
#pragma unroll
                            for (int k = 0; k < VEC; ++k) acc[m][r] = fmaf(a[k], b[k], acc[m][r]);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MATRICES; ++m)
#pragma unroll
        for (int r = 0; r < FEW_ROWS; ++r)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[m][r] += __shfl_xor_sync(FULL, acc[m][r], o);
#pragma unroll
    for (int r = 0; r < FEW_ROWS; ++r) {
        if (lane != r || r >= rows) continue;
        const int64_t row = tile.r0 + r;
        float h[1] = {acc[0][r]};
        if constexpr (EPI == GATED) {
            if (p.gate_up != nullptr) {
                T *z = (T *)p.gate_up + row * p.gs + n;
                z[0] = from_f32<T>(acc[0][r]);
                z[p.N] = from_f32<T>(acc[1][r]);
            }
            Pair a[1] = {pair(acc[0][r], 0.f)};
            const Pair u[1] = {pair(acc[1][r], 0.f)};
            gate_products<T>(p.activation, a, u);
            h[0] = unpair(a[0]).x;
        }
        T *out = (T *)p.out + row * p.os + n;
        out[0] = from_f32<T>(h[0]);
        if (EPI != GATED && n + 1 < p.N) out[1] = from_f32<T>(acc[1][r]);
    }
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

// The route's offsets and the status words, as the checks of shared memory take them.
static Span offsets_of(const tbe_route *route) {
    return span_of(route != nullptr ? route->offset : nullptr, route != nullptr ? (route->experts + (uintptr_t)1) * 4 : 0);
}
static Span words_of(const int32_t *dev_status) { return span_of(dev_status, 16); }

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

// Whether a kernel was compiled for the registers that its warps divide: with
// fewer, their increase would wait for ever.
template <typename Kernel> static bool has_registers(Kernel *fn, int registers) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, (const void *)fn) == cudaSuccess && a.numRegs == registers;
}

constexpr size_t TC_SMEM = 232448;      // the most of a CTA

template <typename T, int FORM, int EPI, bool LONG = false>
static void launch_tensor(Launch &L, const char *name, const CUtensorMap &a, const CUtensorMap &few, const CUtensorMap &b,
                          TensorProduct &p) {
    constexpr int WIDTH = EPI == GATED ? TC_TILE / 2 : TC_TILE;
    p.tiles_m = (p.M + TC_TILE - 1) / TC_TILE;
    p.tiles_n = (p.N + WIDTH - 1) / WIDTH;
    const int64_t groups = p.groups.experts + 1 < p.groups.rows ? p.groups.experts + 1 : p.groups.rows;
    const int64_t most = FORM == WEIGHTS ? (int64_t)p.groups.experts * p.slices * p.tiles_m * p.tiles_n
                                         : ((int64_t)p.groups.rows / TC_TILE + groups) * p.tiles_n;
    int64_t pairs = L.num_sms / 2 > 0 ? L.num_sms / 2 : 1;
    if (pairs > most) pairs = most;
    auto *fn = product_tensor_kernel<T, FORM, EPI, LONG>;
    static const bool ready = has_registers(fn, TC_LAUNCH_REGS);
    if (!ready) {
        L.failed = true;
        return;
    }
    p.stages = FORM == WEIGHTS || p.groups.experts <= TC_FEW_EXPERTS ? TC_STAGES : TC_STAGES_MANY;
    const size_t smem = 1024 + (size_t)p.stages * TC_STAGE + TC_EPILOGUE * TC_STAGED + sizeof(TensorBars) +
                        (FORM == WEIGHTS ? 0 : (size_t)(p.stages == TC_STAGES ? TC_FEW_EXPERTS + 2 : PRODUCT_MOST_EXPERTS + 2) * 4);
    static_assert(1024 + TC_STAGES * TC_STAGE + TC_EPILOGUE * TC_STAGED + sizeof(TensorBars) + (TC_FEW_EXPERTS + 2) * 4 <= TC_SMEM &&
                      1024 + TC_STAGES_MANY * TC_STAGE + TC_EPILOGUE * TC_STAGED + sizeof(TensorBars) +
                              (PRODUCT_MOST_EXPERTS + 2) * 4 <= TC_SMEM,
                  "shared memory");
    cached_smem_attr(L.dev, (const void *)fn, TC_SMEM);      // (one size a kernel: it is set once)
    L.before(name);
    fn<<<(unsigned)(2 * pairs), TC_THREADS, smem, L.stream>>>(a, few, b, p);
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
    CUtensorMap a, few, b;
    if (!tc::make_map(&a, x->data, x->dtype, x->cols, x->rows, 1, x->stride, 0, 128) ||
        !tc::make_map(&few, x->data, x->dtype, x->cols, x->rows, 1, x->stride, 0, 32) ||
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
    p.segment = TC_LONG_SEGMENT;
    if (p.K > (x->dtype == TBE_F16 ? TC_LONG_F16 : TC_LONG_BF16))
        TBE_HALF_SWITCH(x->dtype, (launch_tensor<T, FORM, EPI, true>(L, "tbe_product_tensor_long", a, few, b, p)));
    else
        TBE_HALF_SWITCH(x->dtype, (launch_tensor<T, FORM, EPI>(L, "tbe_product_tensor", a, few, b, p)));
    return true;
}

template <typename T, int FORM, int EPI> static void launch_general(Launch &L, const char *name, GeneralProduct &g) {
    constexpr int WIDTH = EPI == GATED ? GEN_TILE / 2 : GEN_TILE;
    TensorProduct &p = g.t;
    p.tiles_m = (p.M + GEN_TILE - 1) / GEN_TILE;
    p.tiles_n = (p.N + WIDTH - 1) / WIDTH;
    const int64_t groups = p.groups.experts + 1 < p.groups.rows ? p.groups.experts + 1 : p.groups.rows;
    const int64_t most = FORM == WEIGHTS ? (int64_t)p.groups.experts * p.slices * p.tiles_m * p.tiles_n
                                         : ((int64_t)p.groups.rows / GEN_TILE + groups) * p.tiles_n;
    auto *fn = product_general_kernel<T, FORM, EPI>;
    static const bool ready = has_registers(fn, GenWarps<sizeof(T) == 4>::LAUNCH);
    if (!ready) {
        L.failed = true;
        return;
    }
    const size_t smem = 1024 + (size_t)gen_stages<T>() * 2 * gen_pieces<T>() * GEN_PIECE + GEN_EPILOGUE * TC_STAGED + sizeof(GeneralBars);
    cached_smem_attr(L.dev, (const void *)fn, smem);
    L.before(name);
    fn<<<(unsigned)(L.num_sms < most ? L.num_sms : most), GenWarps<sizeof(T) == 4>::THREADS, smem, L.stream>>>(g);
    L.after();
}

// A product of rows: by TMA where it takes both operands.
template <int FORM, int EPI>
static void run_rows(Launch &L, const tbe_matrix *x, const tbe_experts *w, const tbe_matrix *out, const tbe_matrix *gate_up,
                     int activation, int32_t *status, const tbe_route *route) {
    const Groups groups = groups_of(route, x->rows, w->experts);
    const bool few = FORM == ROWS && x->rows <= (w->experts > 1 ? FEW_MOST : FEW_MOST_DENSE);
    if (!few && run_tensor<FORM, EPI>(L, x, w, out, gate_up, activation, status, groups)) return;
    GeneralProduct g = {};
    TensorProduct &p = g.t;
    p.out = out->data;
    p.os = out->stride;
    p.gate_up = gate_up != nullptr ? gate_up->data : nullptr;
    p.gs = gate_up != nullptr ? gate_up->stride : 0;
    p.N = (int)(FORM == ROWS ? (EPI == GATED ? w->rows / 2 : w->rows) : w->cols);
    p.K = (int)(FORM == ROWS ? w->cols : w->rows);
    p.activation = activation;
    // (results are written four elements at a time: 16 or 8 bytes)
    p.whole_out = whole_rows(out->data, out->stride, EPI == GATE_GRAD ? p.N : 0, 4);
    p.whole_gate = gate_up != nullptr && whole_rows(gate_up->data, gate_up->stride, p.N, 4);
    p.status = status;
    p.groups = groups;
    const int bytes = dtype_bytes(x->dtype);
    g.a = x->data;
    g.as = x->stride;
    g.whole_a = whole_rows(x->data, x->stride, 0, bytes);
    g.b = w->data;
    g.bs = w->stride;
    g.be = w->expert_stride;
    g.whole_b = whole_rows(w->data, w->stride, w->expert_stride, bytes);
    if constexpr (FORM == ROWS) {
        if (few) {
            const int64_t tiles = (x->rows + FEW_ROWS - 1) / FEW_ROWS + (w->experts + 1 < x->rows ? w->experts + 1 : x->rows);
            const int each = FEW_WARPS * (EPI == GATED ? 1 : 2);
            const dim3 grid((unsigned)((p.N + each - 1) / each), (unsigned)tiles);
            const bool whole = g.whole_a && g.whole_b && p.K % (16 / bytes) == 0;
            L.before("tbe_product_few");
            TBE_TYPE_SWITCH(x->dtype, {
                auto *fn = whole ? product_few_kernel<T, EPI, true> : product_few_kernel<T, EPI, false>;
                fn<<<grid, 32 * FEW_WARPS, 0, L.stream>>>(g);
            });
            L.after();
            return;
        }
    }
    TBE_TYPE_SWITCH(x->dtype, (launch_general<T, FORM, EPI>(L, "tbe_product_general", g)));
}

// The weights' gradient.
static void run_weights(Launch &L, const tbe_matrix *dy, const tbe_matrix *x, const tbe_experts *dw, int accumulate,
                        void *workspace, int32_t *status, const tbe_route *route) {
    TensorProduct p = {};
    p.out = dw->data;
    p.os = dw->stride;
    p.oe = dw->expert_stride;
    p.M = (int)dw->rows;
    p.N = (int)dw->cols;
    p.accumulate = accumulate;
    p.out_f32 = dw->dtype == TBE_F32;
    p.whole_out = whole_rows(dw->data, dw->stride, dw->experts > 1 ? dw->expert_stride : 0, 4);
    p.status = status;
    p.groups = groups_of(route, x->rows, dw->experts);
    p.slices = weight_slices(x->rows, dw->experts, p.M, p.N);
    p.segment = p.out_f32 || p.slices > 1 ? TC_SEGMENT : TC_SEGMENT_HALF;
    GeneralProduct part = {};
    part.t = p;
    if (p.slices > 1) {
        part.t.out = workspace;
        part.t.os = p.N;
        part.t.oe = (int64_t)p.M * p.N;
        part.t.accumulate = 0;
        part.t.out_f32 = 1;
        part.t.whole_out = p.N % 4 == 0;
    }
    CUtensorMap a, b;
    if (x->rows > 0 && tc::make_map(&a, dy->data, x->dtype, dy->cols, x->rows, 1, dy->stride, 0, 64) &&
        tc::make_map(&b, x->data, x->dtype, x->cols, x->rows, 1, x->stride, 0, 64)) {
        TBE_HALF_SWITCH(x->dtype, (launch_tensor<T, WEIGHTS, STORE>(L, "tbe_product_tensor_weights", a, a, b, part.t)));
    } else {
        const int bytes = dtype_bytes(x->dtype);
        part.a = dy->data;
        part.as = dy->stride;
        part.whole_a = whole_rows(dy->data, dy->stride, 0, bytes);
        part.b = x->data;
        part.bs = x->stride;
        part.whole_b = whole_rows(x->data, x->stride, 0, bytes);
        TBE_TYPE_SWITCH(x->dtype, (launch_general<T, WEIGHTS, STORE>(L, "tbe_product_general_weights", part)));
    }
    if (p.slices == 1 || L.failed) return;
    const bool whole = p.whole_out && p.N % 4 == 0;
    const dim3 grid((unsigned)(dw->experts * p.M), (unsigned)((p.N + (whole ? 1023 : 255)) / (whole ? 1024 : 256)));
    TBE_TYPE_SWITCH(dw->dtype, {
        auto *fn = whole ? product_join_kernel<T, 4> : product_join_kernel<T, 1>;
        launch_with(L, "tbe_product_join", true, 1, fn, grid, 256, 0, (const float *)workspace, p);
    });
}

// ---- self-test: both kernels' products of operands that never arrive
constexpr int SELFTEST_ROWS = 8;
struct ProductSelftest {
    __nv_bfloat16 out[2][SELFTEST_ROWS][64];        // first: the caller looks at it
    __nv_bfloat16 x[SELFTEST_ROWS][64], w[64][64];
};
size_t product_selftest_bytes() { return round_up(sizeof(ProductSelftest), 256); }

__global__ void product_selftest_init_kernel(ProductSelftest *w) {
    for (int i = threadIdx.x; i < (int)(sizeof(ProductSelftest) / 2); i += blockDim.x)
        ((__nv_bfloat16 *)w)[i] = __float2bfloat16_rn(1.f);
}

tbe_status launch_product_selftest(Launch &L, void *ws, int32_t *status) {
    auto *s = (ProductSelftest *)ws;
    L.before("tbe_selftest_init");
    product_selftest_init_kernel<<<1, 256, 0, L.stream>>>(s);
    L.after();
    GeneralProduct g = {};
    TensorProduct &p = g.t;
    p.os = 64;
    p.N = p.K = 64;
    p.whole_out = 1;
    p.withhold = 1;
    p.status = status;
    p.groups = Groups{nullptr, 1, SELFTEST_ROWS};
    CUtensorMap a, few, b;
    if (!tc::make_map(&a, s->x, TBE_BF16, 64, SELFTEST_ROWS, 1, 64, 0, 128) ||
        !tc::make_map(&few, s->x, TBE_BF16, 64, SELFTEST_ROWS, 1, 64, 0, 32) ||
        !tc::make_map(&b, s->w, TBE_BF16, 64, 64, 1, 64, 0, 128))
        return TBE_ERR_CUDA;
    TensorProduct first = p;
    first.out = s->out[0];
    launch_tensor<__nv_bfloat16, ROWS, STORE>(L, "tbe_product_tensor", a, few, b, first);
    p.out = s->out[1];
    g.a = s->x;
    g.b = s->w;
    g.as = g.bs = 64;
    g.whole_a = g.whole_b = 1;
    launch_general<__nv_bfloat16, ROWS, STORE>(L, "tbe_product_general", g);
    return TBE_OK;
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
    const Span offsets = offsets_of(route), words = words_of(dev_status);
    if (share(span_of(hidden), span_of(gate_up), span_of(rows), span_of(weight), offsets, words) ||
        share(span_of(gate_up), span_of(rows), span_of(weight), offsets, words))
        return TBE_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_rows<ROWS, GATED>(L, rows, weight, hidden, gate_up, activation, dev_status, route);
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
    if (share(span_of(out), span_of(rows), span_of(weight), offsets_of(route), words_of(dev_status))) return TBE_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_rows<ROWS, STORE>(L, rows, weight, out, nullptr, 0, dev_status, route);
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
    if (share(span_of(grad_rows), span_of(grad_out), span_of(weight), span_of(gate_up), offsets_of(route), words_of(dev_status)))
        return TBE_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        if (gate_up != nullptr)
            run_rows<ROWS_GRAD, GATE_GRAD>(L, grad_out, weight, grad_rows, gate_up, activation, dev_status, route);
        else
            run_rows<ROWS_GRAD, STORE>(L, grad_out, weight, grad_rows, nullptr, 0, dev_status, route);
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
    const Span ws = span_of(workspace, need), offsets = offsets_of(route), words = words_of(dev_status);
    if (share(span_of(grad_weight), span_of(grad_out), span_of(rows), ws, offsets, words) ||
        share(ws, span_of(grad_out), span_of(rows), offsets, words))
        return TBE_ERR_INVALID_ARGUMENT;
    return guarded([&]() -> tbe_status {
        Launch L(stream, cfg);
        run_weights(L, grad_out, rows, grad_weight, accumulate, workspace, dev_status, route);
        return L.failed ? TBE_ERR_CUDA : TBE_OK;
    });
}

}  // extern "C"
