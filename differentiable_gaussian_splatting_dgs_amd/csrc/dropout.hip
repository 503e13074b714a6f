// Dropout from a counter: y = x keep / (1 - p) + residual, and its gradient, the same call on dy.
//
// The mask is a function of seed, offset, row and column (Philox4x32-10: Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011) and is never stored.  One evaluation gives 128 bits: 16 for each of 8
// columns, 16 bytes of a 16-bit type.  Bits of a column's own would be 32 with half the columns: the generator's
// twenty 32-bit products, at a quarter of the rate, would then take as long as the memory does.
#include <math.h>

#include "linear_tile.h"

namespace gs {
namespace {

struct DropArgs {
    const void *x, *residual;
    void* y;
    const uint64_t* state;
    int64_t rows, ld_x, ld_y, ld_res;
    int32_t n, blocks;  // groups of 8 columns in a row
    uint32_t least;     // of the half-words that keep
    float factor;
    uint64_t seed, offset;
};

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint64_t offset, uint64_t seed) {
    uint32_t x0 = c0, x1 = c1, x2 = (uint32_t)offset, x3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)b;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return Words{{x0, x1, x2, x3}};
}

// Every thread takes one group of 8 columns at a time.  1M rows of 128 bfloat16 with a residual: 138 us, 5.5 TB/s; 100k of
// 509 float32 88 us, 4.6 TB/s (odd rows: their loads and stores are not whole lines).
template <typename T, bool RES>
__global__ __launch_bounds__(256) void k_dropout(DropArgs p) {
    constexpr int E = Tile<T>::E, F = 8 / E;  // fragments of a group
    typedef typename Tile<T>::Frag Frag;
    const uint64_t seed = p.state ? p.state[0] : p.seed, offset = p.offset + (p.state ? p.state[1] : 0);
    const int64_t total = p.rows * p.blocks, step = (int64_t)gridDim.x * 256;
    int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t row = at / p.blocks;
    int32_t block = (int32_t)(at - row * p.blocks);
    const int64_t row_step = step / p.blocks;
    const int32_t block_step = (int32_t)(step - row_step * p.blocks);
    for (; at < total; at += step) {
        const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
        Frag f[F], r[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            f[i] = load_frag(x, block * 8 + i * E, p.n);
            if (RES) r[i] = load_frag(static_cast<const T*>(p.residual) + row * p.ld_res, block * 8 + i * E, p.n);
        }
        const Words w = philox((uint32_t)block, (uint32_t)row, offset, seed);
#pragma unroll
        for (int i = 0; i < F; ++i) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int k = i * E + j;
                const uint32_t half = w.w[k / 2] >> (16 * (k & 1)) & 0xffffu;
                const float v = half >= p.least ? (float)f[i][j] * p.factor : 0.f;
                f[i][j] = (T)(RES ? v + (float)r[i][j] : v);
            }
            store_part(static_cast<T*>(p.y) + row * p.ld_y, block * 8 + i * E, p.n, f[i]);
        }
        row += row_step, block += block_step;
        if (block >= p.blocks) block -= p.blocks, ++row;
    }
}

template <typename T>
void run(const DropArgs& p, hipStream_t s) {
    const int64_t blocks = (p.rows * p.blocks + 255) / 256;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    if (p.residual)
        hipLaunchKernelGGL((k_dropout<T, true>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_dropout<T, false>), grid, dim3(256), 0, s, p);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_dropout(const gs_dropout_args* d, const uint64_t* state, const void* x, const void* residual, void* y,
                          void* stream) {
    if (!d || d->rows < 0 || d->n < 0 || d->dtype < GS_F32 || d->dtype > GS_BF16 || !(d->p >= 0.0 && d->p <= 1.0))
        return GS_EINVAL;
    if (d->rows > 0x7fffffff || d->n > (1 << 20)) return GS_ECAPACITY;
    if (d->rows == 0 || d->n == 0) return GS_OK;
    if (!x || !y || d->ld_x < d->n || d->ld_y < d->n || (residual && d->ld_res != 0 && d->ld_res < d->n))
        return GS_EINVAL;
    const uintptr_t mask = d->dtype == GS_F32 ? 3 : 1;
    for (const void* t : {x, residual, (const void*)y})
        if (reinterpret_cast<uintptr_t>(t) & mask) return GS_EALIGN;
    if (reinterpret_cast<uintptr_t>(state) & 7u) return GS_EALIGN;
    const uint32_t least = (uint32_t)nearbyint(d->p * 65536.0);
    DropArgs p{x, residual, y, state, d->rows, d->ld_x, d->ld_y, d->ld_res, d->n, (d->n + 7) / 8, least,
               least < 65536 ? (float)(65536.0 / (65536.0 - least)) : 0.f, d->seed, d->offset};
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        run<float>(p, s);
    else if (d->dtype == GS_F16)
        run<_Float16>(p, s);
    else
        run<__bf16>(p, s);
    return launch_status();
}
