// Gradient clipping by the global norm, and the Adam step that takes its coefficient.
//
// Method source: the forward/backward page (qqiyuan.cn, "3D Gaussian forward and
// backward, from derivation to efficient implementation") names gradient clipping
// among its numerical-stability measures; the 3DGS training notes (huajishe), C.2,
// Adam with per-parameter learning rates.
//
//   norm = sqrt(sum g^2) over every element of every tensor
//   coef = min(1, max_norm / (norm + 1e-6))
//
// The passes are bound by memory: the norm reads every gradient once, the clip
// reads it again and writes it, the Adam step reads gradient, parameter and
// moments and writes the last three.  A launch takes up to kTensors tensors in
// its arguments; their elements are cut into chunks of 16 KB and blocks walk the
// chunks of all tensors, so many small tensors cost one launch and a large one
// fills the GPU.
#include <math.h>

#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kTensors = 64;     // per launch: one ballot of a wave finds a chunk's tensor
constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // 16-byte loads in flight per lane
constexpr int kChunkBytes = kThreads * kUnroll * 16;
constexpr int kMaxBlocks = 1024;  // 4 blocks per CU: 8 read 177M float32 at 5.3 TB/s, 4 at 6.1

struct GradArgs {
    const void* grad[kTensors];
    void* out[kTensors];
    int64_t count[kTensors];
    int64_t first_chunk[kTensors + 1];
    int32_t dtype[kTensors];
    int32_t n;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec16 {  // 16 bytes of T
    static constexpr int kN = 16 / sizeof(T);
    T v __attribute__((ext_vector_type(16 / sizeof(T))));
};

// The tensor chunk c belongs to: the last one whose first chunk is <= c (empty
// tensors share their first chunk with the next one and are never the last).
__device__ __forceinline__ int tensor_of(const int64_t* first_chunk, int n, int64_t c) {
    const int lane = threadIdx.x & 63;
    const bool below = lane < n && first_chunk[lane] <= c;
    return __builtin_amdgcn_readfirstlane(__popcll(__ballot(below)) - 1);
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int64_t count, int64_t chunk) {
    constexpr int kN = Vec16<T>::kN;
    const int64_t e0 = chunk * (kChunkBytes / (int64_t)sizeof(T));
    double acc = 0.0;
    if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0 && e0 + kChunkBytes / (int64_t)sizeof(T) <= count) {
        const Vec16<T>* p = reinterpret_cast<const Vec16<T>*>(g + e0) + threadIdx.x;
        Vec16<T> x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = p[u * kThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const double d = (double)(float)x[u].v[j];
                acc = fma(d, d, acc);
            }
    } else {
        const int64_t e1 = min(count, e0 + kChunkBytes / (int64_t)sizeof(T));
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
            const double d = (double)(float)g[e];
            acc = fma(d, d, acc);
        }
    }
    return acc;
}

__device__ __forceinline__ double block_sum(double acc) {
    __shared__ double s_part[kThreads / 64];
    for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o, 64);
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = acc;
    __syncthreads();
    return (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
}

// Squares and sums in 64 bits: no magnitude of a gradient overflows them, and the
// arithmetic stays under the loads.  59M float32 43 to 46 us, 5.1 to 5.5 TB/s; 16 tensors of 64 or 4096
// bfloat16 4.7 us.
__global__ __launch_bounds__(kThreads) void k_norm(GradArgs a, double* partial) {
    double acc = 0.0;
    const int64_t chunks = a.first_chunk[a.n];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(a.first_chunk, a.n, c);
        const int64_t local = c - a.first_chunk[t];
        if (a.dtype[t] == GS_F32)
            acc += chunk_squares(static_cast<const float*>(a.grad[t]), a.count[t], local);
        else if (a.dtype[t] == GS_F16)
            acc += chunk_squares(static_cast<const _Float16*>(a.grad[t]), a.count[t], local);
        else
            acc += chunk_squares(static_cast<const __bf16*>(a.grad[t]), a.count[t], local);
    }
    acc = block_sum(acc);
    if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// The coefficient from the blocks' sums, added in a fixed order; `write`: this block
// also writes the clipping state.  A next launch does this (k_coef, or every block of
// k_scale): a counter by which the last block of k_norm would know itself costs each
// block a release at the scope of the GPU, 35 us more over 59M float32.
__device__ __forceinline__ float coefficient(const double* partial, int parts, float max_norm, float* clip,
                                             bool write) {
    double acc = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) acc += partial[i];
    acc = block_sum(acc);
    const double norm = sqrt(acc), c = (double)max_norm / (norm + 1e-6);
    const float coef = acc < INFINITY ? (float)(c < 1.0 ? c : 1.0) : NAN;
    if (write && threadIdx.x == 0) {
        clip[0] = (float)norm;
        clip[1] = coef;
    }
    return coef;
}

__global__ __launch_bounds__(kThreads) void k_coef(const double* partial, int parts, float max_norm, float* clip) {
    coefficient(partial, parts, max_norm, clip, true);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* out, int64_t count, int64_t chunk, float coef) {
    // non-temporal stores leave the last-level cache to the gradients that the norm has just read
    constexpr int kN = Vec16<T>::kN;
    const int64_t e0 = chunk * (kChunkBytes / (int64_t)sizeof(T));
    if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
        e0 + kChunkBytes / (int64_t)sizeof(T) <= count) {
        const Vec16<T>* p = reinterpret_cast<const Vec16<T>*>(g + e0) + threadIdx.x;
        Vec16<T>* q = reinterpret_cast<Vec16<T>*>(out + e0) + threadIdx.x;
        Vec16<T> x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = p[u * kThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int j = 0; j < kN; ++j) x[u].v[j] = (T)(coef * (float)x[u].v[j]);
            __builtin_nontemporal_store(x[u].v, &q[u * kThreads].v);
        }
    } else {
        const int64_t e1 = min(count, e0 + kChunkBytes / (int64_t)sizeof(T));
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) out[e] = (T)(coef * (float)g[e]);
    }
}

// back: chunks from the last to the first, which the norm has left in the last-level
// cache when all of them do not fit (177M float32: 363 against 395 us; 5.9M: 22 against 19).
// 59M float32 72 us, 6.6 TB/s, since part of the reads are hits there.
__global__ __launch_bounds__(kThreads) void k_scale(GradArgs a, const double* partial, int parts, float max_norm,
                                                    float* clip, bool write, bool back) {
    const float c0 = coefficient(partial, parts, max_norm, clip, write && blockIdx.x == 0);
    const bool same = !(c0 < 1.f);  // 1 or NaN: the values as they are
    const float coef = same ? 1.f : c0;
    const int64_t chunks = a.first_chunk[a.n];
    for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const int64_t c = back ? chunks - 1 - i : i;
        const int t = tensor_of(a.first_chunk, a.n, c);
        if (same && a.grad[t] == a.out[t]) continue;
        const int64_t local = c - a.first_chunk[t];
        if (a.dtype[t] == GS_F32)
            chunk_scale(static_cast<const float*>(a.grad[t]), static_cast<float*>(a.out[t]), a.count[t], local, coef);
        else if (a.dtype[t] == GS_F16)
            chunk_scale(static_cast<const _Float16*>(a.grad[t]), static_cast<_Float16*>(a.out[t]), a.count[t], local,
                        coef);
        else
            chunk_scale(static_cast<const __bf16*>(a.grad[t]), static_cast<__bf16*>(a.out[t]), a.count[t], local,
                        coef);
    }
}

constexpr int64_t kCacheBytes = 192 << 20;  // of the 256 MB last-level cache

constexpr int kAdamTensors = 32;  // per launch (the argument block holds up to 4 KB)
constexpr int kAdamPer = 4;       // elements of a lane, one 16-byte load of each array

struct ClipAdamArgs {
    gs_adam_tensor t[kAdamTensors];
    int64_t first_block[kAdamTensors + 1];
    int32_t n;
    float b1, b2, eps, inv_c1, inv_sqrt_c2;
    const float* clip;
};

__device__ __forceinline__ float load_as_float(const void* p, int32_t dtype, int64_t i) {
    if (dtype == GS_F32) return static_cast<const float*>(p)[i];
    if (dtype == GS_F16) return (float)static_cast<const _Float16*>(p)[i];
    return (float)static_cast<const __bf16*>(p)[i];
}

__device__ __forceinline__ void store_as(void* p, int32_t dtype, int64_t i, float v) {
    if (dtype == GS_F32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == GS_F16)
        static_cast<_Float16*>(p)[i] = (_Float16)v;
    else
        static_cast<__bf16*>(p)[i] = (__bf16)v;
}

template <typename T>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&g)[4]) {
    typedef T V __attribute__((ext_vector_type(4)));
    const V x = *reinterpret_cast<const V*>(static_cast<const T*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = (float)x[k];
}

template <typename T>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 v) {
    typedef T V __attribute__((ext_vector_type(4)));
    V x;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (T)v[k];
    *reinterpret_cast<V*>(static_cast<T*>(p) + i) = x;
}

// The update of gs_adam_step, with its hardware square root and reciprocal.
__device__ __forceinline__ void adam_update(float& p, float g, float& m, float& v, float lr, const ClipAdamArgs& a) {
    m = a.b1 * m + (1.f - a.b1) * g;
    v = a.b2 * v + (1.f - a.b2) * g * g;
    const float denom = __builtin_amdgcn_sqrtf(v) * a.inv_sqrt_c2 + a.eps;
    p -= lr * (m * a.inv_c1) * __builtin_amdgcn_rcpf(denom);
}

template <bool STREAM>
__device__ __forceinline__ f32x4 take4(const float* p) {
    const f32x4* q = reinterpret_cast<const f32x4*>(p);
    return STREAM ? __builtin_nontemporal_load(q) : *q;
}
template <bool STREAM>
__device__ __forceinline__ void give4(float* p, f32x4 v) {
    f32x4* q = reinterpret_cast<f32x4*>(p);
    if (STREAM)
        __builtin_nontemporal_store(v, q);
    else
        *q = v;
}

// STREAM: for more than the last-level cache holds, parameters and moments pass it by
// (non-temporal) and blocks run from the last tensor's end, where the norm left the
// gradients in it: 59M float32 parameters 261 against 314 us (6.4 TB/s); 5.9M, which
// the cache holds from step to step, 27.4 against 26.5.
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void k_adam_clipped(ClipAdamArgs a) {
    const float coef = a.clip ? a.clip[1] : 1.f;
    if (!(coef <= 1.f)) return;  // NaN: the norm is not finite
    const int64_t block = STREAM ? (int64_t)gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int ti = tensor_of(a.first_block, a.n, block);
    const gs_adam_tensor& G = a.t[ti];
    const int64_t local = block - a.first_block[ti];
    if (G.normalize_rows) {
        // one lane per row: update the row, then renormalise it
        const int64_t row = local * kThreads + threadIdx.x;
        if (row >= G.rows) return;
        const int64_t base = row * G.row_len;
        float ss = 0.f;
        for (int c = 0; c < G.row_len; ++c) {
            float p = G.param[base + c], m = G.exp_avg[base + c], v = G.exp_avg_sq[base + c];
            adam_update(p, coef * load_as_float(G.grad, G.grad_dtype, base + c), m, v, G.lr, a);
            G.exp_avg[base + c] = m;
            G.exp_avg_sq[base + c] = v;
            G.param[base + c] = p;
            ss += p * p;
        }
        const float inv = 1.f / sqrtf(ss);
        for (int c = 0; c < G.row_len; ++c) {
            const float p = G.param[base + c] * inv;
            G.param[base + c] = p;
            if (G.copy) store_as(G.copy, G.copy_dtype, base + c, p);
        }
        return;
    }
    const int ncol = G.col_end - G.col_begin;
    const int64_t total = G.rows * ncol, e0 = local * (kThreads * kAdamPer) + threadIdx.x * kAdamPer;
    if (e0 >= total) return;
    const bool whole = ncol == G.row_len;
    const uintptr_t at = reinterpret_cast<uintptr_t>(G.param) | reinterpret_cast<uintptr_t>(G.exp_avg) |
                         reinterpret_cast<uintptr_t>(G.exp_avg_sq) | reinterpret_cast<uintptr_t>(G.grad) |
                         reinterpret_cast<uintptr_t>(G.copy);
    if (whole && (at & 15u) == 0 && e0 + kAdamPer <= total) {
        f32x4 p = take4<STREAM>(G.param + e0), m = take4<STREAM>(G.exp_avg + e0), v = take4<STREAM>(G.exp_avg_sq + e0);
        float g[4];
        if (G.grad_dtype == GS_F32)
            load4<float>(G.grad, e0, g);
        else if (G.grad_dtype == GS_F16)
            load4<_Float16>(G.grad, e0, g);
        else
            load4<__bf16>(G.grad, e0, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float pk = p[k], mk = m[k], vk = v[k];
            adam_update(pk, coef * g[k], mk, vk, G.lr, a);
            p[k] = pk;
            m[k] = mk;
            v[k] = vk;
        }
        give4<STREAM>(G.param + e0, p);
        give4<STREAM>(G.exp_avg + e0, m);
        give4<STREAM>(G.exp_avg_sq + e0, v);
        if (G.copy) {
            if (G.copy_dtype == GS_F32)
                store4<float>(G.copy, e0, p);
            else if (G.copy_dtype == GS_F16)
                store4<_Float16>(G.copy, e0, p);
            else
                store4<__bf16>(G.copy, e0, p);
        }
        return;
    }
    for (int64_t e = e0; e < e0 + kAdamPer && e < total; ++e) {
        const int64_t row = whole ? 0 : e / ncol;
        const int64_t i = whole ? e : row * G.row_len + G.col_begin + (e - row * ncol);
        float p = G.param[i], m = G.exp_avg[i], v = G.exp_avg_sq[i];
        adam_update(p, coef * load_as_float(G.grad, G.grad_dtype, i), m, v, G.lr, a);
        G.param[i] = p;
        G.exp_avg[i] = m;
        G.exp_avg_sq[i] = v;
        if (G.copy) store_as(G.copy, G.copy_dtype, i, p);
    }
}

inline bool dtype_ok(int32_t t) { return t == GS_F32 || t == GS_F16 || t == GS_BF16; }
inline int dtype_size(int32_t t) { return t == GS_F32 ? 4 : 2; }
inline bool element_aligned(const void* p, int32_t t) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype_size(t) - 1)) == 0;
}

inline int grad_launches(int32_t n) { return (n + kTensors - 1) / kTensors; }

int check_grads(int32_t n, const gs_grad_tensor* t, float max_norm, const float* clip, const void* workspace,
                size_t workspace_bytes, bool need_out) {
    if (n < 0 || (n > 0 && !t) || !clip || !(max_norm >= 0.f)) return GS_EINVAL;
    for (int32_t i = 0; i < n; ++i) {
        if (!dtype_ok(t[i].dtype) || t[i].count < 0) return GS_EINVAL;
        if (t[i].count > 0 && (!t[i].grad || (need_out && !t[i].out))) return GS_EINVAL;
        if (t[i].count > ((int64_t)1 << 44)) return GS_ECAPACITY;
    }
    for (int32_t i = 0; i < n; ++i)
        if (!element_aligned(t[i].grad, t[i].dtype) || (need_out && !element_aligned(t[i].out, t[i].dtype)))
            return GS_EALIGN;
    if (!aligned16(clip)) return GS_EALIGN;
    size_t need = 0;
    gs_grad_workspace_size(n, &need);
    if (need > 0 && !workspace) return GS_EINVAL;
    if (workspace_bytes < need) return GS_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GS_EALIGN;
    return GS_OK;
}

// Fills the arguments of one launch with tensors [i0, i1); the number of chunks.
int64_t fill_args(GradArgs& a, const gs_grad_tensor* t, int32_t i0, int32_t i1) {
    int64_t chunks = 0;
    a.n = i1 - i0;
    for (int32_t i = i0; i < i1; ++i) {
        a.grad[i - i0] = t[i].grad;
        a.out[i - i0] = t[i].out;
        a.count[i - i0] = t[i].count;
        a.dtype[i - i0] = t[i].dtype;
        a.first_chunk[i - i0] = chunks;
        const int64_t per = kChunkBytes / dtype_size(t[i].dtype);
        chunks += (t[i].count + per - 1) / per;
    }
    a.first_chunk[a.n] = chunks;
    return chunks;
}

// The launches of the sums of squares; how many partial sums they leave.
int norm_launches(int32_t n, const gs_grad_tensor* t, double* partial, hipStream_t s) {
    int parts = 0;
    for (int32_t i0 = 0; i0 < n; i0 += kTensors) {
        GradArgs a;
        const int64_t chunks = fill_args(a, t, i0, i0 + kTensors < n ? i0 + kTensors : n);
        const int blocks = (int)(chunks < kMaxBlocks ? chunks : kMaxBlocks);
        if (blocks > 0) hipLaunchKernelGGL(k_norm, dim3(blocks), dim3(kThreads), 0, s, a, partial + parts);
        parts += blocks;
    }
    return parts;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_grad_workspace_size(int32_t n_tensors, size_t* bytes) {
    if (n_tensors < 0 || !bytes) return GS_EINVAL;
    *bytes = (size_t)grad_launches(n_tensors) * kMaxBlocks * sizeof(double);
    return GS_OK;
}

extern "C" int gs_grad_norm(int32_t n_tensors, const gs_grad_tensor* tensors, float max_norm, float* clip,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_grads(n_tensors, tensors, max_norm, clip, workspace, workspace_bytes, false);
    if (rc != GS_OK) return rc;
    hipStream_t s = as_stream(stream);
    double* partial = static_cast<double*>(workspace);
    const int parts = norm_launches(n_tensors, tensors, partial, s);
    hipLaunchKernelGGL(k_coef, dim3(1), dim3(kThreads), 0, s, partial, parts, max_norm, clip);
    return launch_status();
}

extern "C" int gs_grad_clip(int32_t n_tensors, const gs_grad_tensor* tensors, float max_norm, float* clip,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_grads(n_tensors, tensors, max_norm, clip, workspace, workspace_bytes, true);
    if (rc != GS_OK) return rc;
    hipStream_t s = as_stream(stream);
    double* partial = static_cast<double*>(workspace);
    const int parts = norm_launches(n_tensors, tensors, partial, s);
    int64_t bytes = 0;
    for (int32_t i = 0; i < n_tensors; ++i) bytes += tensors[i].count * dtype_size(tensors[i].dtype);
    bool write = true;  // the state, by the first launch
    for (int32_t i0 = 0; i0 < n_tensors; i0 += kTensors) {
        GradArgs a;
        const int64_t chunks = fill_args(a, tensors, i0, i0 + kTensors < n_tensors ? i0 + kTensors : n_tensors);
        if (chunks == 0) continue;
        hipLaunchKernelGGL(k_scale, dim3((unsigned)(chunks < kMaxBlocks ? chunks : kMaxBlocks)), dim3(kThreads), 0, s,
                           a, partial, parts, max_norm, clip, write, bytes > kCacheBytes);
        write = false;
    }
    if (write) hipLaunchKernelGGL(k_coef, dim3(1), dim3(kThreads), 0, s, partial, parts, max_norm, clip);
    return launch_status();
}

extern "C" int gs_adam_step_clipped(int32_t n_tensors, const gs_adam_tensor* tensors, float beta1, float beta2,
                                    float eps, int32_t step, const float* clip, void* stream) {
    if (n_tensors < 0 || step < 1 || (n_tensors > 0 && !tensors)) return GS_EINVAL;
    if (clip && !aligned16(clip)) return GS_EALIGN;
    int64_t most = 0, values = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const gs_adam_tensor& G = tensors[i];
        if (G.rows < 0 || G.row_len <= 0 || G.col_begin < 0 || G.col_end > G.row_len || G.col_begin >= G.col_end ||
            !dtype_ok(G.grad_dtype) || (G.copy && !dtype_ok(G.copy_dtype)))
            return GS_EINVAL;
        if (G.rows > 0 && (!G.param || !G.grad || !G.exp_avg || !G.exp_avg_sq)) return GS_EINVAL;
        if (G.normalize_rows && (G.col_begin != 0 || G.col_end != G.row_len)) return GS_EINVAL;
        if (!element_aligned(G.param, GS_F32) || !element_aligned(G.exp_avg, GS_F32) ||
            !element_aligned(G.exp_avg_sq, GS_F32) || !element_aligned(G.grad, G.grad_dtype) ||
            (G.copy && !element_aligned(G.copy, G.copy_dtype)))
            return GS_EALIGN;
        if (G.rows > ((int64_t)1 << 40) / G.row_len) return GS_ECAPACITY;
        const int64_t work = G.normalize_rows ? G.rows : G.rows * (G.col_end - G.col_begin);
        most += work / kThreads + 1;
        values += G.rows * (G.col_end - G.col_begin);
    }
    if (most > 0x7fffffff) return GS_ECAPACITY;
    hipStream_t s = as_stream(stream);
    bool launched = false;
    for (int32_t i0 = 0; i0 < n_tensors; i0 += kAdamTensors) {
        ClipAdamArgs a;
        a.n = i0 + kAdamTensors < n_tensors ? kAdamTensors : n_tensors - i0;
        a.b1 = beta1; a.b2 = beta2; a.eps = eps;
        a.inv_c1 = (float)(1.0 / (1.0 - pow((double)beta1, step)));
        a.inv_sqrt_c2 = (float)(1.0 / sqrt(1.0 - pow((double)beta2, step)));
        a.clip = clip;
        int64_t blocks = 0;
        for (int i = 0; i < a.n; ++i) {
            const gs_adam_tensor& G = tensors[i0 + i];
            a.t[i] = G;
            a.first_block[i] = blocks;
            const int64_t work = G.normalize_rows ? G.rows : G.rows * (G.col_end - G.col_begin);
            const int64_t per = G.normalize_rows ? kThreads : kThreads * kAdamPer;
            blocks += (work + per - 1) / per;
        }
        a.first_block[a.n] = blocks;
        if (blocks == 0) continue;
        if (12 * values > kCacheBytes)  // parameters and moments
            hipLaunchKernelGGL((k_adam_clipped<true>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
        else
            hipLaunchKernelGGL((k_adam_clipped<false>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
        launched = true;
    }
    return launched ? launch_status() : GS_OK;
}
