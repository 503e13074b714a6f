// Layer norm and its gradients.
//
//   xh = (x - mean) r, r = 1 / sqrt(mean((x - mean)^2) + eps), y = xh w + b
//   g = dy w, dx = r (g - mean(g) - xh mean(g xh)), dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both directions are bound by memory: a row is read once and stays in registers while its moments are taken (the
// mean first, then the squares about it: no cancellation).  A row is spread over G lanes of a wave with U chunks of
// 16 bytes each, so a wave takes 64 / G rows at a time and a row's sums need log2 G exchanges; longer rows take a
// block, and rows past its registers are read again for each pass (they lie in L2 by then).  A row's last chunk is its
// last 16 bytes: what it shares with the chunk before it counts there, and is written by both, the same bits.  The
// backward's sums over the rows stay in the registers of the lane that has the columns; each block leaves one partial of
// them, which a second launch adds in a fixed order.
#include "linear_tile.h"

namespace gs {
namespace {

struct NormArgs {
    const void *x, *w, *b, *dy;
    void *y, *dx;
    float* part;  // [blocks][2][n]: dw and db
    void *dw, *db;  // one block: the results themselves
    int64_t rows, ld_x, ld_y, ld_dx;
    int32_t n;
    float eps;
};

constexpr int kMostChunks = 256;  // of a row that a wave holds: 4 a lane
constexpr int kBlockU = 8;        // chunks a lane of a block's row, at most
constexpr int kSumBlocks = 1024;  // partials of the backward at most

// sum / n: the product with inv = 1 / n, and what it leaves.  A row of one value has that value for its mean.
__device__ __forceinline__ float mean_of(float sum, float inv, int n) {
    const float mean = sum * inv;
    return fmaf(fmaf(-mean, (float)n, sum), inv, mean);
}

// Sum over the G lanes of a row, in all of them.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The same of K sums over the 256 threads of a block.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float (*s_sum)[K]) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = row_sum<64>(v[i]);
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < K; ++i) s_sum[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = (s_sum[0][i] + s_sum[1][i]) + (s_sum[2][i] + s_sum[3][i]);
}
__device__ __forceinline__ float block_sum(float v, float (*s_sum)[1]) {
    float one[1] = {v};
    block_sums(one, s_sum);
    return one[0];
}

template <int G, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*s_sum)[K]) {
    if constexpr (G == 256) {
        block_sums(v, s_sum);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = row_sum<G>(v[i]);
    }
}

// A lane's chunks of a row of n >= E elements: chunk u of lane `at` of G is that of number at + u G.  FULL: all lanes
// have all of their chunks whole.
template <typename T, int G, int U, bool FULL>
struct Lane {
    static constexpr int E = Tile<T>::E;
    typedef typename Tile<T>::Frag Frag;
    int from[U];  // where the chunk lies
    int skip[U];  // how many of its elements belong to the chunk before (E: all, there is no such chunk)
    __device__ __forceinline__ Lane(int at, int n) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (at + u * G) * E;
            from[u] = FULL ? k : min(k, n - E);
            skip[u] = FULL ? 0 : min(k - from[u], E);
        }
    }
    __device__ __forceinline__ void load(const T* row, Frag (&f)[U]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) f[u] = load16(row + from[u]);
    }
    __device__ __forceinline__ bool counts(int u, int j) const { return FULL || j >= skip[u]; }
    __device__ __forceinline__ void store(T* row, int u, Frag f) const {
        if (FULL || skip[u] < E) __builtin_memcpy(row + from[u], &f, 16);
    }
    // elements of a vector of n, or `missing` without one
    __device__ __forceinline__ void vector(const void* p, float missing, float (&v)[U][E]) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Frag f;
            if (p) f = load16(static_cast<const T*>(p) + from[u]);
#pragma unroll
            for (int j = 0; j < E; ++j) v[u][j] = p ? (float)f[j] : missing;
        }
    }
};

// Forward, G lanes a row (of a wave; G == 256: of a block), U chunks a lane; the next rows are in flight while the
// sums are taken.  1M rows of 128 bfloat16: 96 us, 5.35 TB/s, a copy's rate; one row of 512 float32 2.4, a launch.
template <typename T, int G, int U, bool FULL>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs p) {
    constexpr int E = Tile<T>::E, kRows = 256 / G;  // rows a block takes at a time
    __shared__ float s_sum[4][1];
    const Lane<T, G, U, FULL> lane(threadIdx.x % G, p.n);
    float w[U][E], b[U][E];
    lane.vector(p.w, 1.f, w);
    lane.vector(p.b, 0.f, b);
    const float inv = 1.f / (float)p.n;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    // rows of the same block end together: G == 256 meets at its barriers
    const int64_t sets = (p.rows + kRows - 1) / kRows;
    const T* x = static_cast<const T*>(p.x);
    typename Tile<T>::Frag next[U];
    if (blockIdx.x < sets) lane.load(x + (row < p.rows ? row : 0) * p.ld_x, next);
    for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
        float v[U][E], sum[1] = {0.f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                v[u][j] = (float)next[u][j];
                sum[0] += lane.counts(u, j) ? v[u][j] : 0.f;
            }
        if (set + gridDim.x < sets) lane.load(x + (row + step < p.rows ? row + step : 0) * p.ld_x, next);
        row_sums<G>(sum, s_sum);
        const float mean = mean_of(sum[0], inv, p.n);
        float squares[1] = {0.f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                v[u][j] -= mean;
                const float d = lane.counts(u, j) ? v[u][j] : 0.f;
                squares[0] = fmaf(d, d, squares[0]);
            }
        row_sums<G>(squares, s_sum);
        const float r = 1.f / sqrtf(squares[0] * inv + p.eps);
        if (row >= p.rows) continue;
        T* y = static_cast<T*>(p.y) + row * p.ld_y;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            typename Tile<T>::Frag f;
#pragma unroll
            for (int j = 0; j < E; ++j) f[j] = (T)fmaf(v[u][j] * r, w[u][j], b[u][j]);
            lane.store(y, u, f);
        }
    }
}

// Backward, the same way.  1M rows of 128 float16: 141 us and 5 of the join, 5.3 TB/s; 100k of 333 float32 76 and 5.
template <typename T, int G, int U, bool FULL>
__global__ __launch_bounds__(256) void k_norm_bwd(NormArgs p) {
    constexpr int E = Tile<T>::E, kRows = 256 / G;
    __shared__ float s_sum[4][1], s_sums[4][3];
    extern __shared__ float s_part[];  // [kRows][G * U * E], one of dw and db at a time
    const int at = threadIdx.x % G;
    const Lane<T, G, U, FULL> lane(at, p.n);
    float w[U][E], dw[U][E] = {}, db[U][E] = {};
    lane.vector(p.w, 1.f, w);
    const float inv = 1.f / (float)p.n;
    const int64_t step = (int64_t)gridDim.x * kRows, sets = (p.rows + kRows - 1) / kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    typename Tile<T>::Frag next_x[U], next_g[U];
    auto fetch = [&](int64_t to) {
        to = to < p.rows ? to : 0;
        lane.load(static_cast<const T*>(p.x) + to * p.ld_x, next_x);
        lane.load(static_cast<const T*>(p.dy) + to * p.ld_y, next_g);
    };
    if (blockIdx.x < sets) fetch(row);
    for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
        float x[U][E], g[U][E], sum[1] = {0.f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                x[u][j] = (float)next_x[u][j], g[u][j] = (float)next_g[u][j];
                sum[0] += lane.counts(u, j) ? x[u][j] : 0.f;
            }
        if (set + gridDim.x < sets) fetch(row + step);
        row_sums<G>(sum, s_sum);
        const float mean = mean_of(sum[0], inv, p.n);
        float sums[3] = {0.f, 0.f, 0.f};  // of squares, of g xh, of g
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                x[u][j] -= mean;
                const bool in = lane.counts(u, j);
                const float d = in ? x[u][j] : 0.f, gw = in ? g[u][j] * w[u][j] : 0.f;
                sums[0] = fmaf(d, d, sums[0]);
                sums[1] = fmaf(gw, d, sums[1]);
                sums[2] += gw;
            }
        row_sums<G>(sums, s_sums);
        const float r = 1.f / sqrtf(sums[0] * inv + p.eps);
        const float along = sums[1] * inv * r * r, flat = sums[2] * inv;
        if (row >= p.rows) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            typename Tile<T>::Frag f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                f[j] = (T)(r * (fmaf(g[u][j], w[u][j], -flat) - x[u][j] * along));
                dw[u][j] = fmaf(g[u][j], x[u][j] * r, dw[u][j]);
                db[u][j] += g[u][j];
            }
            if (p.dx) lane.store(static_cast<T*>(p.dx) + row * p.ld_dx, u, f);
        }
    }
    if (!p.part) return;
    // the block's rows join in LDS
    for (int which = 0; which < 2; ++which) {
        float* part = p.part + ((int64_t)blockIdx.x * 2 + which) * p.n;
        T* out = static_cast<T*>(which ? p.db : p.dw);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (lane.counts(u, j))
                    s_part[threadIdx.x / G * (G * U * E) + lane.from[u] + j] = which ? db[u][j] : dw[u][j];
        __syncthreads();
        for (int k = threadIdx.x; k < p.n; k += 256) {
            float sum = 0.f;
            for (int i = 0; i < kRows; ++i) sum += s_part[i * (G * U * E) + k];
            if (gridDim.x > 1) part[k] = sum;
            else if (out) out[k] = (T)sum;
        }
    }
}

// Rows shorter than a chunk: a thread each, whose element loads meet in the lines of its neighbours'.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_short(NormArgs p) {
    constexpr int E = Tile<T>::E;
    __shared__ float s_part[256][E];
    const float inv = 1.f / (float)p.n;
    float w[E], b[E], dw[E] = {}, db[E] = {};
#pragma unroll
    for (int j = 0; j < E; ++j) {
        w[j] = j < p.n ? p.w ? (float)static_cast<const T*>(p.w)[j] : 1.f : 0.f;
        b[j] = j < p.n && p.b ? (float)static_cast<const T*>(p.b)[j] : 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x; row < p.rows; row += (int64_t)gridDim.x * 256) {
        const T* from = static_cast<const T*>(p.x) + row * p.ld_x;
        float x[E], sum = 0.f, squares = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = j < p.n ? (float)from[j] : 0.f, sum += x[j];
        const float mean = mean_of(sum, inv, p.n);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            x[j] = j < p.n ? x[j] - mean : 0.f;
            squares = fmaf(x[j], x[j], squares);
        }
        const float r = 1.f / sqrtf(squares * inv + p.eps);
        if (p.y) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (j < p.n) static_cast<T*>(p.y)[row * p.ld_y + j] = (T)fmaf(x[j] * r, w[j], b[j]);
            continue;
        }
        const T* grad = static_cast<const T*>(p.dy) + row * p.ld_y;
        float g[E], along = 0.f, flat = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            g[j] = j < p.n ? (float)grad[j] : 0.f;
            along = fmaf(g[j] * w[j], x[j], along);
            flat = fmaf(g[j], w[j], flat);
            dw[j] = fmaf(g[j], x[j] * r, dw[j]);
            db[j] += g[j];
        }
        along *= inv * r * r, flat *= inv;
        if (p.dx)
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (j < p.n)
                    static_cast<T*>(p.dx)[row * p.ld_dx + j] = (T)(r * (fmaf(g[j], w[j], -flat) - x[j] * along));
    }
    if (!p.part) return;
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < E; ++j) s_part[threadIdx.x][j] = which ? db[j] : dw[j];
        for (int o = 128; o > 0; o >>= 1) {
            __syncthreads();
            if ((int)threadIdx.x < o)
#pragma unroll
                for (int j = 0; j < E; ++j) s_part[threadIdx.x][j] += s_part[threadIdx.x + o][j];
        }
        T* out = static_cast<T*>(which ? p.db : p.dw);
        if (threadIdx.x == 0)
            for (int j = 0; j < p.n; ++j) {
                if (gridDim.x > 1) p.part[((int64_t)blockIdx.x * 2 + which) * p.n + j] = s_part[0][j];
                else if (out) out[j] = (T)s_part[0][j];
            }
    }
}

// Rows longer than a block's registers: one block a row at a time, read again for each pass.  The sums over the rows
// add up in the block's partial in memory, each column by one thread.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_long(NormArgs p) {
    __shared__ float s_sum[4][1];
    const T *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    const float inv = 1.f / (float)p.n;
    float* part = p.part ? p.part + (int64_t)blockIdx.x * 2 * p.n : nullptr;
    if (part)
        for (int k = threadIdx.x; k < p.n; k += 256) part[k] = part[p.n + k] = 0.f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
        float sum = 0.f;
#pragma unroll 8
        for (int k = threadIdx.x; k < p.n; k += 256) sum += (float)x[k];
        const float mean = mean_of(block_sum(sum, s_sum), inv, p.n);
        float squares = 0.f, along = 0.f, flat = 0.f;
        const T* g = p.y ? nullptr : static_cast<const T*>(p.dy) + row * p.ld_y;
        for (int k = threadIdx.x; k < p.n; k += 256) {
            const float d = (float)x[k] - mean;
            squares = fmaf(d, d, squares);
            if (g) {
                const float gw = w ? (float)g[k] * (float)w[k] : (float)g[k];
                along = fmaf(gw, d, along);
                flat += gw;
            }
        }
        const float r = 1.f / sqrtf(block_sum(squares, s_sum) * inv + p.eps);
        if (p.y) {
            T* y = static_cast<T*>(p.y) + row * p.ld_y;
            for (int k = threadIdx.x; k < p.n; k += 256)
                y[k] = (T)fmaf(((float)x[k] - mean) * r, w ? (float)w[k] : 1.f, b ? (float)b[k] : 0.f);
            continue;
        }
        along = block_sum(along, s_sum) * inv * r * r, flat = block_sum(flat, s_sum) * inv;
        T* dx = p.dx ? static_cast<T*>(p.dx) + row * p.ld_dx : nullptr;
        for (int k = threadIdx.x; k < p.n; k += 256) {
            const float d = (float)x[k] - mean, dy = (float)g[k];
            if (part) {
                part[k] = fmaf(dy, d * r, part[k]);
                part[p.n + k] += dy;
            }
            if (dx) dx[k] = (T)(r * (fmaf(dy, w ? (float)w[k] : 1.f, -flat) - d * along));
        }
    }
}

// dw and db from the blocks' partials: 16 columns a block, 16 threads a column.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_join(const float* part, int parts, int32_t n, T* dw, T* db) {
    __shared__ float s_sum[16][17];
    const int col = threadIdx.x & 15, from = threadIdx.x >> 4;
    const int64_t k = (int64_t)blockIdx.x * 16 + col;  // of dw, then of db
    float sum = 0.f;
    if (k < 2 * (int64_t)n)
#pragma unroll 8
        for (int i = from; i < parts; i += 16) sum += part[(int64_t)i * 2 * n + k];
    s_sum[from][col] = sum;
    __syncthreads();
    if (from != 0 || k >= 2 * (int64_t)n) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += s_sum[i][col];
    T* to = k < n ? dw : db;
    if (to) to[k < n ? k : k - n] = (T)sum;
}

inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int size_of(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }

enum { NORM_SHORT, NORM_WAVE, NORM_LONG };

struct NormPlan {
    int kind, lanes, chunks;  // lanes a row and chunks a lane
    bool full;                // which the row fills
    int64_t sets;             // of rows that a block takes at a time
};

// Lanes of a row: the fewest that hold it a chunk each, up to a wave; then up to 4 chunks a lane, then a block.
// 400 MB of bfloat16 rows of 2100: by a wave of 8 chunks a lane forward 454 us, backward 521, by a block of 2 180 and
// 364; of 1500 by 4 chunks a lane 205 and 262, by 3 153 and 249.
NormPlan plan_of(const gs_layer_norm* d) {
    const int e = 16 / size_of(d->dtype);
    const int64_t chunks = cdiv64(d->n, e);
    NormPlan p{};
    if (d->n < e) {
        p.kind = NORM_SHORT, p.sets = cdiv64(d->rows, 256);
    } else if (chunks <= kMostChunks) {
        p.kind = NORM_WAVE, p.lanes = 1;
        while (p.lanes < 64 && p.lanes < chunks) p.lanes *= 2;
        p.chunks = (int)cdiv64(chunks, p.lanes);
        p.sets = cdiv64(d->rows, 256 / p.lanes);
    } else if (chunks <= 256 * kBlockU) {
        p.kind = NORM_WAVE, p.lanes = 256, p.chunks = (int)cdiv64(chunks, 256), p.sets = d->rows;
        if (p.chunks > 4) p.chunks = 8;
    } else {
        p.kind = NORM_LONG, p.sets = d->rows;
    }
    p.full = d->n == (int64_t)p.lanes * p.chunks * e;
    return p;
}

// Blocks of the backward: a partial of 8 n bytes each, so past 256 of them (or all sets, if those are fewer) no more than
// a tenth of the rows' bytes asks for.  256 go before the tenth: few long rows would leave most of the GPU idle.  300
// float16 rows of 5000 (a tenth: 7 blocks) 20.9 us, with 64 at least 20.3, 16 42, 1 83; 1000 rows 24, 39, 79, 79; 300 of
// 20000 253, 461, 1574, 3555.  A few sets of rows go to one block, which needs no second launch (but for rows that a block
// reads again).
int bwd_blocks(const gs_layer_norm* d, const NormPlan& plan) {
    if (plan.kind != NORM_LONG && plan.sets <= 4) return 1;
    const int64_t most = d->rows * size_of(d->dtype) / 80;
    int64_t blocks = plan.sets < kSumBlocks ? plan.sets : kSumBlocks;
    const int64_t least = plan.sets < 256 ? plan.sets : 256;
    if (blocks > most) blocks = most;
    if (blocks < least) blocks = least;
    return (int)blocks;
}

template <typename T, int G, int U, bool FULL>
void norm_launch(const NormArgs& p, int blocks, bool back, hipStream_t s) {
    if (back)
        hipLaunchKernelGGL((k_norm_bwd<T, G, U, FULL>), dim3(blocks), dim3(256),
                           p.part ? (256 / G) * G * U * Tile<T>::E * 4 : 0, s, p);
    else
        hipLaunchKernelGGL((k_norm_fwd<T, G, U, FULL>), dim3(blocks), dim3(256), 0, s, p);
}
template <typename T, int G, int U>
void norm_any(const NormArgs& p, const NormPlan& plan, int blocks, bool back, hipStream_t s) {
    if (plan.full) norm_launch<T, G, U, true>(p, blocks, back, s);
    else norm_launch<T, G, U, false>(p, blocks, back, s);
}

template <typename T>
void norm_run(const NormArgs& p, const NormPlan& plan, int blocks, bool back, hipStream_t s) {
    if (plan.kind == NORM_SHORT) {
        hipLaunchKernelGGL(k_norm_short<T>, dim3(blocks), dim3(256), 0, s, p);
    } else if (plan.kind == NORM_LONG) {
        hipLaunchKernelGGL(k_norm_long<T>, dim3(blocks), dim3(256), 0, s, p);
    } else {
        switch (plan.lanes < 64 ? plan.lanes : plan.lanes * 10 + plan.chunks) {
            case 1: norm_any<T, 1, 1>(p, plan, blocks, back, s); break;
            case 2: norm_any<T, 2, 1>(p, plan, blocks, back, s); break;
            case 4: norm_any<T, 4, 1>(p, plan, blocks, back, s); break;
            case 8: norm_any<T, 8, 1>(p, plan, blocks, back, s); break;
            case 16: norm_any<T, 16, 1>(p, plan, blocks, back, s); break;
            case 32: norm_any<T, 32, 1>(p, plan, blocks, back, s); break;
            case 641: norm_any<T, 64, 1>(p, plan, blocks, back, s); break;
            case 642: norm_any<T, 64, 2>(p, plan, blocks, back, s); break;
            case 643: norm_any<T, 64, 3>(p, plan, blocks, back, s); break;
            case 644: norm_any<T, 64, 4>(p, plan, blocks, back, s); break;
            case 2562: norm_any<T, 256, 2>(p, plan, blocks, back, s); break;
            case 2563: norm_any<T, 256, 3>(p, plan, blocks, back, s); break;
            case 2564: norm_any<T, 256, 4>(p, plan, blocks, back, s); break;
            default: norm_any<T, 256, 8>(p, plan, blocks, back, s); break;
        }
    }
}

int check_shape(const gs_layer_norm* d) {
    if (!d || d->rows < 0 || d->n < 1 || d->dtype < GS_F32 || d->dtype > GS_BF16 || !(d->eps >= 0.f)) return GS_EINVAL;
    if (d->rows > 0x7fffffff || d->n > (1 << 20)) return GS_ECAPACITY;
    return GS_OK;
}

inline bool element_aligned(const void* p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (size_of(dtype) - 1)) == 0;
}

size_t workspace_of(const gs_layer_norm* d) {
    if (d->rows == 0) return 256;
    return ((size_t)bwd_blocks(d, plan_of(d)) * 2 * d->n * 4 + 255) & ~(size_t)255;
}

template <typename T>
void fwd(const gs_layer_norm* d, NormArgs& p, hipStream_t s) {
    const NormPlan plan = plan_of(d);
    norm_run<T>(p, plan, (int)(plan.sets < 4096 ? plan.sets : 4096), false, s);
}

template <typename T>
void bwd(const gs_layer_norm* d, NormArgs& p, void* dw, void* db, hipStream_t s) {
    const NormPlan plan = plan_of(d);
    const int blocks = d->rows > 0 ? bwd_blocks(d, plan) : 0;
    if (blocks > 0) norm_run<T>(p, plan, blocks, true, s);
    if ((dw || db) && (blocks != 1 || plan.kind == NORM_LONG))
        hipLaunchKernelGGL(k_norm_join<T>, dim3((unsigned)cdiv64(2 * (int64_t)d->n, 16)), dim3(256), 0, s, p.part, blocks,
                           d->n, static_cast<T*>(dw), static_cast<T*>(db));
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_layer_norm_fwd(const gs_layer_norm* d, const void* x, const void* w, const void* b, void* y,
                                 void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (d->rows == 0) return GS_OK;
    if (!x || !y || d->ld_x < d->n || d->ld_y < d->n) return GS_EINVAL;
    for (const void* t : {x, w, b, (const void*)y})
        if (!element_aligned(t, d->dtype)) return GS_EALIGN;
    NormArgs p{x, w, b, nullptr, y, nullptr, nullptr, nullptr, nullptr, d->rows, d->ld_x, d->ld_y, 0, d->n, d->eps};
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        fwd<float>(d, p, s);
    else if (d->dtype == GS_F16)
        fwd<_Float16>(d, p, s);
    else
        fwd<__bf16>(d, p, s);
    return launch_status();
}

extern "C" int gs_layer_norm_bwd_workspace_size(const gs_layer_norm* d, size_t* bytes) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (!bytes) return GS_EINVAL;
    *bytes = workspace_of(d);
    return GS_OK;
}

extern "C" int gs_layer_norm_bwd(const gs_layer_norm* d, const void* x, const void* w, const void* dy, void* dx,
                                 void* dw, void* db, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (!dx && !dw && !db) return GS_OK;
    if (d->rows > 0 && (!x || !dy || d->ld_x < d->n || d->ld_y < d->n || (dx && d->ld_dx < d->n))) return GS_EINVAL;
    for (const void* t : {x, w, dy, (const void*)dx, (const void*)dw, (const void*)db})
        if (!element_aligned(t, d->dtype)) return GS_EALIGN;
    if ((dw || db) && !workspace) return GS_EINVAL;
    if ((dw || db) && workspace_bytes < workspace_of(d)) return GS_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GS_EALIGN;
    NormArgs p{x, w, nullptr, dy, nullptr, dx, dw || db ? static_cast<float*>(workspace) : nullptr, dw, db, d->rows,
               d->ld_x, d->ld_y, d->ld_dx, d->n, d->eps};
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        bwd<float>(d, p, dw, db, s);
    else if (d->dtype == GS_F16)
        bwd<_Float16>(d, p, dw, db, s);
    else
        bwd<__bf16>(d, p, dw, db, s);
    return launch_status();
}
