// Layer norm and its gradients.
//
//   xh = (x - mean) r, r = 1 / sqrt(mean((x - mean)^2) + eps), y = xh w + b
//   g = dy w, dx = r (g - mean(g) - xh mean(g xh)), dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both directions are bound by memory: a row is read once and stays in registers while its moments are taken (the
// mean first, then the squares about it: no cancellation).  A row is spread over G lanes of a wave with U chunks of
// 16 bytes each, so a wave takes 64 / G rows at a time and a row's sums need log2 G exchanges; longer rows take a
// block, and rows past its registers are read again for each pass (they lie in L2 by then).  The backward's sums
// over the rows stay in the registers of the lane that has the columns; each block leaves one partial of them, which
// a second launch adds in a fixed order.
#include "linear_tile.h"

namespace gs {
namespace {

struct NormArgs {
    const void *x, *w, *b, *dy;
    void *y, *dx;
    float* part;  // [blocks][2][n]: dw and db
    int64_t rows, ld_x, ld_y, ld_dx;
    int32_t n;
    float eps;
};

constexpr int kMostChunks = 512;  // of a row that a wave holds
constexpr int kBlockU = 8;        // chunks a lane of a block's row
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

// The same over the 256 threads of a block.
__device__ __forceinline__ float block_sum(float v, float* s_sum) {
    v = row_sum<64>(v);
    __syncthreads();  // the last sum has been read
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

// A lane's chunks of a row, whose c-th is chunk first + c * step, as float32.  Elements past the row are 0; `count`
// of each chunk's elements are the row's.
template <typename T, int U>
struct Chunks {
    static constexpr int E = Tile<T>::E;
    typename Tile<T>::Frag f[U];

    // n >= E
    __device__ __forceinline__ void load(const T* row, int first, int step, int n) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (first + u * step) * E;
            f[u] = load16(row + max(min(k0, n - E), 0));
        }
    }
    __device__ __forceinline__ void fix(int first, int step, int n, bool in) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (first + u * step) * E, drop = in ? min(max(k0 - (n - E), 0), E) * 8 * (int)sizeof(T) : 128;
            union {
                typename Tile<T>::Frag f;
                uint64_t q[2];
            } v;
            v.f = f[u];
            if (drop >= 64) {
                v.q[0] = drop >= 128 ? 0 : v.q[1] >> (drop - 64);
                v.q[1] = 0;
            } else if (drop > 0) {
                v.q[0] = (v.q[0] >> drop) | (v.q[1] << (64 - drop));
                v.q[1] >>= drop;
            }
            f[u] = v.f;
        }
    }
    __device__ __forceinline__ float at(int u, int j) const { return (float)f[u][j]; }
};

// Forward, G lanes a row (of a wave; G == 256: of a block), U chunks a lane.
template <typename T, int G, int U>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs p) {
    constexpr int E = Tile<T>::E, kRows = 256 / G;  // rows a block takes at a time
    __shared__ float s_sum[4];
    const int at = threadIdx.x % G;
    auto total = [&](float v) {
        if constexpr (G == 256) return block_sum(v, s_sum);
        else return row_sum<G>(v);
    };
    float w[U][E], b[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int k = min((at + u * G) * E + j, p.n - 1);
            w[u][j] = p.w ? (float)static_cast<const T*>(p.w)[k] : 1.f;
            b[u][j] = p.b ? (float)static_cast<const T*>(p.b)[k] : 0.f;
        }
    const float inv = 1.f / (float)p.n;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    // rows of the same block end together: G == 256 meets at its barriers
    const int64_t sets = (p.rows + kRows - 1) / kRows;
    Chunks<T, U> next;
    if (blockIdx.x < sets) next.load(static_cast<const T*>(p.x) + (row < p.rows ? row : 0) * p.ld_x, at, G, p.n);
    for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
        const bool in = row < p.rows;
        Chunks<T, U> x = next;
        if (set + gridDim.x < sets) {
            const int64_t to = row + step;
            next.load(static_cast<const T*>(p.x) + (to < p.rows ? to : 0) * p.ld_x, at, G, p.n);
        }
        x.fix(at, G, p.n, in);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) sum += x.at(u, j);
        const float mean = mean_of(total(sum), inv, p.n);
        float squares = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float d = (at + u * G) * E + j < p.n ? x.at(u, j) - mean : 0.f;
                squares = fmaf(d, d, squares);
            }
        const float r = 1.f / sqrtf(total(squares) * inv + p.eps);
        if (!in) continue;
        T* y = static_cast<T*>(p.y) + row * p.ld_y;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            typename Tile<T>::Frag f;
#pragma unroll
            for (int j = 0; j < E; ++j) f[j] = (T)fmaf((x.at(u, j) - mean) * r, w[u][j], b[u][j]);
            store_run(y, (at + u * G) * E, p.n, f);
        }
    }
}

// Backward, the same way.
template <typename T, int G, int U>
__global__ __launch_bounds__(256) void k_norm_bwd(NormArgs p) {
    constexpr int E = Tile<T>::E, kRows = 256 / G;
    __shared__ float s_sum[4];
    extern __shared__ float s_part[];  // [kRows][G * U * E], one of dw and db at a time
    const int at = threadIdx.x % G;
    auto total = [&](float v) {
        if constexpr (G == 256) return block_sum(v, s_sum);
        else return row_sum<G>(v);
    };
    float w[U][E], dw[U][E], db[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int k = (at + u * G) * E + j;
            w[u][j] = k >= p.n ? 0.f : p.w ? (float)static_cast<const T*>(p.w)[k] : 1.f;
            dw[u][j] = db[u][j] = 0.f;
        }
    const float inv = 1.f / (float)p.n;
    const int64_t step = (int64_t)gridDim.x * kRows, sets = (p.rows + kRows - 1) / kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    Chunks<T, U> next_x, next_g;
    auto fetch = [&](int64_t to) {
        to = to < p.rows ? to : 0;
        next_x.load(static_cast<const T*>(p.x) + to * p.ld_x, at, G, p.n);
        next_g.load(static_cast<const T*>(p.dy) + to * p.ld_y, at, G, p.n);
    };
    if (blockIdx.x < sets) fetch(row);
    for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
        const bool in = row < p.rows;
        Chunks<T, U> x = next_x, g = next_g;
        if (set + gridDim.x < sets) fetch(row + step);
        x.fix(at, G, p.n, in);
        g.fix(at, G, p.n, in);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) sum += x.at(u, j);
        const float mean = mean_of(total(sum), inv, p.n);
        float squares = 0.f, along = 0.f, flat = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float d = (at + u * G) * E + j < p.n ? x.at(u, j) - mean : 0.f, gw = g.at(u, j) * w[u][j];
                squares = fmaf(d, d, squares);
                along = fmaf(gw, d, along);
                flat += gw;
            }
        const float r = 1.f / sqrtf(total(squares) * inv + p.eps);
        along = total(along) * inv * r * r, flat = total(flat) * inv;
        if (in) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                typename Tile<T>::Frag f;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float d = x.at(u, j) - mean, dy = g.at(u, j);
                    f[j] = (T)(r * (fmaf(dy, w[u][j], -flat) - d * along));
                    dw[u][j] = fmaf(dy, d * r, dw[u][j]);
                    db[u][j] += dy;
                }
                if (p.dx) store_run(static_cast<T*>(p.dx) + row * p.ld_dx, (at + u * G) * E, p.n, f);
            }
        }
    }
    if (!p.part) return;
    // the block's rows join in LDS
    for (int which = 0; which < 2; ++which) {
        float* part = p.part + ((int64_t)blockIdx.x * 2 + which) * p.n;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j)
                s_part[threadIdx.x / G * (G * U * E) + (at + u * G) * E + j] = which ? db[u][j] : dw[u][j];
        __syncthreads();
        for (int k = threadIdx.x; k < p.n; k += 256) {
            float sum = 0.f;
            for (int i = 0; i < kRows; ++i) sum += s_part[i * (G * U * E) + k];
            part[k] = sum;
        }
    }
}

// Rows shorter than a chunk: a thread each.
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
        if (threadIdx.x == 0)
            for (int j = 0; j < p.n; ++j) p.part[((int64_t)blockIdx.x * 2 + which) * p.n + j] = s_part[0][j];
    }
}

// Rows longer than a block's registers: one block a row at a time, read again for each pass.  The sums over the rows
// add up in the block's partial in memory, each column by one thread.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_long(NormArgs p) {
    __shared__ float s_sum[4];
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

enum { NORM_SHORT, NORM_WAVE, NORM_BLOCK, NORM_LONG };

struct NormPlan {
    int kind, lanes, chunks;  // lanes a row and chunks a lane
    int64_t sets;             // of rows that a block takes at a time
};

// Lanes of a row: the fewest that hold it a chunk each, up to a wave; then more chunks a lane, then a block.
NormPlan plan_of(const gs_layer_norm* d) {
    const int e = 16 / size_of(d->dtype);
    const int64_t chunks = cdiv64(d->n, e);
    NormPlan p{};
    if (d->n < e) {
        p.kind = NORM_SHORT, p.sets = cdiv64(d->rows, 256);
    } else if (chunks <= kMostChunks) {
        p.kind = NORM_WAVE, p.lanes = 1, p.chunks = 1;
        while (p.lanes < 64 && p.lanes < chunks) p.lanes *= 2;
        while (p.lanes * p.chunks < chunks) p.chunks *= 2;
        p.sets = cdiv64(d->rows, 256 / p.lanes);
    } else if (chunks <= 256 * kBlockU) {
        p.kind = NORM_BLOCK, p.lanes = 256, p.chunks = chunks <= 256 * 4 ? 4 : 8, p.sets = d->rows;
    } else {
        p.kind = NORM_LONG, p.sets = d->rows;
    }
    return p;
}

// Blocks of the backward: a partial of 8 n bytes each, so no more than a tenth of the rows' bytes asks for.
int bwd_blocks(const gs_layer_norm* d, const NormPlan& plan) {
    const int64_t most = d->rows * size_of(d->dtype) / 80;
    int64_t blocks = plan.sets < kSumBlocks ? plan.sets : kSumBlocks;
    const int64_t least = plan.sets < 256 ? plan.sets : 256;
    if (blocks > most) blocks = most;
    if (blocks < least) blocks = least;
    return (int)blocks;
}

template <typename T, int G, int U>
void norm_launch(const NormArgs& p, int blocks, bool back, hipStream_t s) {
    if (back)
        hipLaunchKernelGGL((k_norm_bwd<T, G, U>), dim3(blocks), dim3(256),
                           p.part ? (256 / G) * G * U * Tile<T>::E * 4 : 0, s, p);
    else
        hipLaunchKernelGGL((k_norm_fwd<T, G, U>), dim3(blocks), dim3(256), 0, s, p);
}

template <typename T>
void norm_run(const NormArgs& p, const NormPlan& plan, int blocks, bool back, hipStream_t s) {
    if (plan.kind == NORM_SHORT) {
        hipLaunchKernelGGL(k_norm_short<T>, dim3(blocks), dim3(256), 0, s, p);
    } else if (plan.kind == NORM_LONG) {
        hipLaunchKernelGGL(k_norm_long<T>, dim3(blocks), dim3(256), 0, s, p);
    } else if (plan.kind == NORM_BLOCK) {
        if (plan.chunks == 4) norm_launch<T, 256, 4>(p, blocks, back, s);
        else norm_launch<T, 256, 8>(p, blocks, back, s);
    } else if (plan.lanes == 64) {
        switch (plan.chunks) {
            case 1: norm_launch<T, 64, 1>(p, blocks, back, s); break;
            case 2: norm_launch<T, 64, 2>(p, blocks, back, s); break;
            case 4: norm_launch<T, 64, 4>(p, blocks, back, s); break;
            default: norm_launch<T, 64, 8>(p, blocks, back, s); break;
        }
    } else {
        switch (plan.lanes) {
            case 1: norm_launch<T, 1, 1>(p, blocks, back, s); break;
            case 2: norm_launch<T, 2, 1>(p, blocks, back, s); break;
            case 4: norm_launch<T, 4, 1>(p, blocks, back, s); break;
            case 8: norm_launch<T, 8, 1>(p, blocks, back, s); break;
            case 16: norm_launch<T, 16, 1>(p, blocks, back, s); break;
            default: norm_launch<T, 32, 1>(p, blocks, back, s); break;
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
    int blocks = 0;
    if (d->rows > 0) {
        const NormPlan plan = plan_of(d);
        blocks = bwd_blocks(d, plan);
        norm_run<T>(p, plan, blocks, true, s);
    }
    if (dw || db)
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
    NormArgs p{x, w, b, nullptr, y, nullptr, nullptr, d->rows, d->ld_x, d->ld_y, 0, d->n, d->eps};
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
    NormArgs p{x, w, nullptr, dy, nullptr, dx, dw || db ? static_cast<float*>(workspace) : nullptr, d->rows, d->ld_x,
               d->ld_y, d->ld_dx, d->n, d->eps};
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        bwd<float>(d, p, dw, db, s);
    else if (d->dtype == GS_F16)
        bwd<_Float16>(d, p, dw, db, s);
    else
        bwd<__bf16>(d, p, dw, db, s);
    return launch_status();
}
