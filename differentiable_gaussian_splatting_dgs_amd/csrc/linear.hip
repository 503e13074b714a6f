// The fused linear layer of the networks beside the Gaussians, and its backward.
//
//   z = x w^T + bias      y = act(z) + residual
//   dz = dy act'(z)       dx = dz w       dw = dz^T x       db = sum over rows of dz
//
// Products are summed in float32, the activation runs in float32, and every
// result is rounded once.
#include "gs_internal.h"

namespace gs {
namespace {

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == GS_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays NaN
    if (ACT == GS_ACT_SILU) return z / (1.f + __expf(-z));
    if (ACT == GS_ACT_GELU) {
        const float u = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        return z / (1.f + __expf(-u));
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if (ACT == GS_ACT_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    if (ACT == GS_ACT_SILU) {
        const float s = 1.f / (1.f + __expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    if (ACT == GS_ACT_GELU) {
        const float u = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        const float s = 1.f / (1.f + __expf(-u));
        return s * (1.f + z * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z * z));
    }
    return 1.f;
}

// C(i, j) = sum_k A(i, k) B(k, j) with element strides, one 64 x 64 tile per block.
enum { EPI_FWD, EPI_DZ, EPI_PLAIN, EPI_PART };

struct TileArgs {
    const void* a;
    const void* b;
    const void* bias;   // FWD, DZ: [cols]
    const void* other;  // FWD: residual; DZ: dy
    void* c;
    int64_t rows, cols, depth;
    int64_t sa_i, sa_k, sb_k, sb_j;
    int64_t ld_other, ld_c;
    int64_t depth_per;  // PART: depth of one split (blockIdx.z)
};

template <typename T, int EPI, int ACT>
__global__ __launch_bounds__(256) void k_tile(TileArgs p) {
    __shared__ float s_a[16][65], s_b[16][65];
    const T* a = static_cast<const T*>(p.a);
    const T* b = static_cast<const T*>(p.b);
    const int64_t i0 = (int64_t)blockIdx.x * 64, j0 = (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    const int64_t k_begin = EPI == EPI_PART ? (int64_t)blockIdx.z * p.depth_per : 0;
    const int64_t k_end = EPI == EPI_PART ? min(p.depth, k_begin + p.depth_per) : p.depth;
    for (int64_t k0 = k_begin; k0 < k_end; k0 += 16) {
#pragma unroll
        for (int e = threadIdx.x; e < 1024; e += 256) {
            // neighbouring lanes along the contiguous index
            const int ai = p.sa_k == 1 ? e >> 4 : e & 63, ak = p.sa_k == 1 ? e & 15 : e >> 6;
            const int bj = p.sb_k == 1 ? e >> 4 : e & 63, bk = p.sb_k == 1 ? e & 15 : e >> 6;
            s_a[ak][ai] = (i0 + ai < p.rows && k0 + ak < k_end) ? (float)a[(i0 + ai) * p.sa_i + (k0 + ak) * p.sa_k]
                                                                : 0.f;
            s_b[bk][bj] = (j0 + bj < p.cols && k0 + bk < k_end) ? (float)b[(k0 + bk) * p.sb_k + (j0 + bj) * p.sb_j]
                                                                : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += s_a[k][ty + 16 * i] * s_b[k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
            if (r >= p.rows || c >= p.cols) continue;
            if (EPI == EPI_PART) {
                static_cast<float*>(p.c)[((int64_t)blockIdx.z * p.rows + r) * p.cols + c] = acc[i][j];
                continue;
            }
            float v = acc[i][j];
            if (EPI == EPI_FWD || EPI == EPI_DZ)
                if (p.bias) v += (float)static_cast<const T*>(p.bias)[c];
            if (EPI == EPI_FWD) {
                v = act_value<ACT>(v);
                if (p.other) v += (float)static_cast<const T*>(p.other)[r * p.ld_other + c];
            }
            if (EPI == EPI_DZ) v = (float)static_cast<const T*>(p.other)[r * p.ld_other + c] * act_slope<ACT>(v);
            static_cast<T*>(p.c)[r * p.ld_c + c] = (T)v;
        }
}

// out[e] = sum over splits of part[s][e], in order.
template <typename T>
__global__ __launch_bounds__(256) void k_join(const float* part, int splits, int64_t count, T* out) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= count) return;
    float acc = 0.f;
    for (int s = 0; s < splits; ++s) acc += part[(int64_t)s * count + e];
    out[e] = (T)acc;
}

// Column sums of dz over one split of the rows (blockIdx.y).
template <typename T>
__global__ __launch_bounds__(256) void k_colsum(const T* dz, int64_t ld, int64_t rows, int32_t cols, int64_t per,
                                                float* part) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(rows, r0 + per);
    float acc = 0.f;
    for (int64_t r = r0; r < r1; ++r) acc += (float)dz[r * ld + c];
    part[(int64_t)blockIdx.y * cols + c] = acc;
}

inline int size_of(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t pad256(size_t b) { return (b + 255) & ~(size_t)255; }

inline int check_shape(const gs_linear* d) {
    if (!d || d->rows < 0 || d->n_in < 0 || d->n_out < 0 || d->dtype < GS_F32 || d->dtype > GS_BF16 ||
        d->act < GS_ACT_NONE || d->act > GS_ACT_GELU)
        return GS_EINVAL;
    if (d->rows > 0x7fffffff || d->n_in > (1 << 20) || d->n_out > (1 << 20)) return GS_ECAPACITY;
    return GS_OK;
}

inline bool element_aligned(const void* p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (size_of(dtype) - 1)) == 0;
}

struct BwdPlan {
    size_t dz, dw_part, db_part, bytes;  // offsets in the workspace
    int splits;
    int64_t per;
};

inline BwdPlan bwd_plan(const gs_linear* d) {
    BwdPlan p{};
    p.splits = (int)(d->rows > 256 ? (d->rows + 255) / 256 : 1);
    if (p.splits > 64) p.splits = 64;
    p.per = cdiv(cdiv(d->rows, p.splits), 16) * 16;
    size_t at = 0;
    p.dz = at;
    if (d->act != GS_ACT_NONE) at += pad256((size_t)d->rows * d->n_out * size_of(d->dtype));
    p.dw_part = at;
    at += pad256((size_t)p.splits * d->n_out * d->n_in * 4);
    p.db_part = at;
    at += pad256((size_t)p.splits * d->n_out * 4);
    p.bytes = at;
    return p;
}

template <typename T, int EPI>
void launch_tile(const TileArgs& p, int act, int splits, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(p.rows, 64), (unsigned)cdiv(p.cols, 64), (unsigned)splits);
    switch (act) {
        case GS_ACT_RELU: hipLaunchKernelGGL((k_tile<T, EPI, GS_ACT_RELU>), grid, dim3(256), 0, s, p); break;
        case GS_ACT_SILU: hipLaunchKernelGGL((k_tile<T, EPI, GS_ACT_SILU>), grid, dim3(256), 0, s, p); break;
        case GS_ACT_GELU: hipLaunchKernelGGL((k_tile<T, EPI, GS_ACT_GELU>), grid, dim3(256), 0, s, p); break;
        default: hipLaunchKernelGGL((k_tile<T, EPI, GS_ACT_NONE>), grid, dim3(256), 0, s, p); break;
    }
}

template <typename T>
void fwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* residual, void* y,
         hipStream_t s) {
    TileArgs p{x, w, bias, residual, y, d->rows, d->n_out, d->n_in, d->ld_x, 1, 1, d->n_in, d->ld_res, d->ld_y, 0};
    launch_tile<T, EPI_FWD>(p, d->act, 1, s);
}

template <typename T>
void bwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* dy, void* dx, void* dw,
         void* db, char* ws, hipStream_t s) {
    const BwdPlan plan = bwd_plan(d);
    const void* dz = dy;
    int64_t ld_dz = d->ld_y;
    if (d->act != GS_ACT_NONE && d->rows > 0 && d->n_out > 0) {
        TileArgs p{x, w, bias, dy, ws + plan.dz, d->rows, d->n_out, d->n_in, d->ld_x, 1, 1, d->n_in, d->ld_y,
                   d->n_out, 0};
        launch_tile<T, EPI_DZ>(p, d->act, 1, s);
        dz = ws + plan.dz;
        ld_dz = d->n_out;
    }
    if (dx && d->rows > 0 && d->n_in > 0) {
        TileArgs p{dz, w, nullptr, nullptr, dx, d->rows, d->n_in, d->n_out, ld_dz, 1, d->n_in, 1, 0, d->ld_dx, 0};
        launch_tile<T, EPI_PLAIN>(p, GS_ACT_NONE, 1, s);
    }
    float* part = reinterpret_cast<float*>(ws + plan.dw_part);
    const int64_t n_w = (int64_t)d->n_out * d->n_in;
    if (dw && n_w > 0) {
        TileArgs p{dz, x, nullptr, nullptr, part, d->n_out, d->n_in, d->rows, 1, ld_dz, d->ld_x, 1, 0, 0, plan.per};
        launch_tile<T, EPI_PART>(p, GS_ACT_NONE, plan.splits, s);
        hipLaunchKernelGGL((k_join<T>), dim3((unsigned)cdiv(n_w, 256)), dim3(256), 0, s, part, plan.splits, n_w,
                           static_cast<T*>(dw));
    }
    if (db && d->n_out > 0) {
        float* dbp = reinterpret_cast<float*>(ws + plan.db_part);
        hipLaunchKernelGGL((k_colsum<T>), dim3((unsigned)cdiv(d->n_out, 256), plan.splits), dim3(256), 0, s,
                           static_cast<const T*>(dz), ld_dz, d->rows, d->n_out, plan.per, dbp);
        hipLaunchKernelGGL((k_join<T>), dim3((unsigned)cdiv(d->n_out, 256)), dim3(256), 0, s, dbp, plan.splits,
                           (int64_t)d->n_out, static_cast<T*>(db));
    }
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_linear_fwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* residual,
                             void* y, void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (d->rows == 0 || d->n_out == 0) return GS_OK;
    if (!y || (d->n_in > 0 && (!x || !w))) return GS_EINVAL;
    if (d->ld_x < d->n_in || d->ld_y < d->n_out || (residual && d->ld_res != 0 && d->ld_res < d->n_out))
        return GS_EINVAL;
    for (const void* p : {x, w, bias, residual, (const void*)y})
        if (!element_aligned(p, d->dtype)) return GS_EALIGN;
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        fwd<float>(d, x, w, bias, residual, y, s);
    else if (d->dtype == GS_F16)
        fwd<_Float16>(d, x, w, bias, residual, y, s);
    else
        fwd<__bf16>(d, x, w, bias, residual, y, s);
    return launch_status();
}

extern "C" int gs_linear_bwd_workspace_size(const gs_linear* d, size_t* bytes) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (!bytes) return GS_EINVAL;
    *bytes = bwd_plan(d).bytes;
    return GS_OK;
}

extern "C" int gs_linear_bwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* dy,
                             void* dx, void* dw, void* db, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (d->n_out == 0 && (!dx || d->rows == 0 || d->n_in == 0)) return GS_OK;
    if (d->rows > 0 && d->n_out > 0 && !dy) return GS_EINVAL;
    if (d->rows > 0 && d->n_in > 0 && d->n_out > 0 && (!x || !w)) return GS_EINVAL;
    if (d->rows > 0 && (d->ld_x < d->n_in || d->ld_y < d->n_out || (dx && d->ld_dx < d->n_in))) return GS_EINVAL;
    for (const void* p : {x, w, bias, dy, (const void*)dx, (const void*)dw, (const void*)db})
        if (!element_aligned(p, d->dtype)) return GS_EALIGN;
    const size_t need = bwd_plan(d).bytes;
    if (need > 0 && !workspace) return GS_EINVAL;
    if (workspace_bytes < need) return GS_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GS_EALIGN;
    hipStream_t s = as_stream(stream);
    char* ws = static_cast<char*>(workspace);
    if (d->dtype == GS_F32)
        bwd<float>(d, x, w, bias, dy, dx, dw, db, ws, s);
    else if (d->dtype == GS_F16)
        bwd<_Float16>(d, x, w, bias, dy, dx, dw, db, ws, s);
    else
        bwd<__bf16>(d, x, w, bias, dy, dx, dw, db, ws, s);
    return launch_status();
}
