// The narrow layers' backward in one pass over the rows.
//
// A block holds the weights in LDS and walks tiles of 16 rows per wave.  Per tile a
// wave reads its rows' x and dy once, recomputes z^T = w x^T, turns the result
// registers into dz, which are at once the fragments of dx^T = w^T dz^T (see
// linear_tile.h), and writes dx; x and dz go to LDS in the layer's type, where
// the block's waves share out dw += dz^T x, each keeping its part of dw in registers
// for the life of the block.  db adds up in the registers of dz, before its rounding.
// Nothing else touches memory: x and dy are read once, dx is written once, and
// each block leaves one partial dw and db for the join.  A layer with few inputs and
// more outputs than a block holds goes through in parts of the outputs (PARTS): dy is
// still read once, and dx adds up in float32 from part to part.
//
// 1M rows 128 -> 128 float16 silu: 200 us and 13 for the join, where 770 MB take 147 at
// the rate of a copy, the matrix units are busy for 49 and the slope's arithmetic for
// some 90; two waves a SIMD (the weights and the tile fill LDS, dw the registers)
// overlap them only in part.  One block of eight waves 280 us against 257
// for two of four; each group's z before its own slope 255 against 209 for all z first.
// 100k rows 64 -> 64 float32 gelu: 42 us, of which 20 are float32 matrix instructions.
#pragma once

#include "linear_tile.h"

namespace gs {

struct BwdArgs {
    const void* x;
    const void* w;
    const void* bias;
    const void* dy;
    void* dx;     // NULL: not wanted
    float* part;  // [blocks][n_out * n_in of dw, then n_out of db], each if wanted
    int64_t rows, ld_x, ld_dy, ld_dx;
    int32_t n_in, n_out, act;
    int32_t want_dw, want_db;
    void* dw;  // one block: the results themselves instead of a partial
    void* db;
    // a layer with more outputs, some of them at a time: dx so far [rows][KP] float32, and whether these outputs
    // are the first and the last
    float* dx_sum;
    int32_t first, last;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBwdGroups = 4;  // groups of KS inputs and of KS outputs at most
constexpr int kPartInputs = 64;  // of a layer that goes through in parts of its outputs, at most

template <typename T, int SL, int NG>
struct BwdGeom {
    static constexpr int KS = Tile<T>::KS, TG = Tile<T>::TG;
    static constexpr int KP = SL * KS, NP = NG * KS;  // padded inputs and outputs
    static constexpr int kWaves = 4;
    static constexpr int kRows = 16 * kWaves;
    static constexpr int kW = KP * NP * (int)sizeof(T);
    static constexpr int kTiles = kRows * (KP + NP) * (int)sizeof(T);
    static constexpr int kLds = kW + kTiles + NP * 4 + NG * 64;
    // blocks per CU: three where the LDS and 168 registers hold them, else two; the grid counts on it
    static constexpr bool kManyRegs = sizeof(T) == 2 ? 30 + 40 * NG + 18 * SL > 168 : NG == kBwdGroups;  // by the builds
    static constexpr int kPerCu = kLds > 53 * 1024 || kManyRegs ? 2 : 3;
    static_assert(kLds <= 80 * 1024, "two blocks per CU");
    // dw's 16 x 16 tiles, NT by KT, dealt to the waves as TN x TK rectangles
    static constexpr int NT = NG * TG, KT = SL * TG;
    static constexpr int split() {
        int best = 1, cost = 1 << 30;
        for (int wn = 1; wn <= kWaves; wn *= 2) {
            const int tn = (NT + wn - 1) / wn, tk = (KT + kWaves / wn - 1) / (kWaves / wn);
            if (64 * tn * tk + tn + tk < cost) cost = 64 * tn * tk + tn + tk, best = wn;
        }
        return best;
    }
    static constexpr int WN = split(), WK = kWaves / WN;
    static constexpr int TN = (NT + WN - 1) / WN, TK = (KT + WK - 1) / WK;
};

// Slot of the fragment of lane (r, g) in LDS.  The rows of the four lane groups are
// rotated against each other so that the reads of w^T, which take one piece of 16
// (float32: 64) different fragments at a time, find them in different banks.
template <typename T>
__device__ __forceinline__ int w_slot(int r, int g) {
    return ((r + (sizeof(T) == 2 ? 4 * g : g)) & 15) + 16 * g;
}

// 16-bit: the pieces are 8 bytes, and two of the 32 that one cycle takes would meet in
// each 16; fragments of odd lane groups lie with their halves swapped.  The product
// with x then takes x with its halves swapped there too: the sum's order is free.
template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag swap_halves(typename Tile<T>::Frag f, bool swap) {
    union {
        typename Tile<T>::Frag f;
        uint64_t q[2];
    } u;
    u.f = f;
    const uint64_t lo = swap ? u.q[1] : u.q[0], hi = swap ? u.q[0] : u.q[1];
    u.q[0] = lo;
    u.q[1] = hi;
    return u.f;
}

template <typename T, int SL, int NG, bool PARTS>
__global__ __launch_bounds__((BwdGeom<T, SL, NG>::kWaves * 64), (BwdGeom<T, SL, NG>::kPerCu)) void k_bwd_narrow(BwdArgs p) {
    typedef BwdGeom<T, SL, NG> G;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    constexpr int kPair = sizeof(T) == 2 ? 2 : 1;  // groups of dx stored together: whole 128-byte lines
    typedef typename Tile<T>::Frag Frag;
    extern __shared__ __align__(16) char s_mem[];
    Frag* s_w = reinterpret_cast<Frag*>(s_mem);  // [NG][TG][SL][64]
    char* s_dz = s_mem + G::kW;
    char* s_x = s_dz + G::kRows * G::NP * (int)sizeof(T);
    float* s_bias = reinterpret_cast<float*>(s_x + G::kRows * G::KP * (int)sizeof(T));
    u32x4* s_live = reinterpret_cast<u32x4*>(s_bias + G::NP);  // [NG][4]: the bits of a fragment that are outputs
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tn0 = wave / G::WK * G::TN, tk0 = wave % G::WK * G::TK;
    const int64_t tiles = (p.rows + G::kRows - 1) / G::kRows;
    f32x4 dw[G::TN][G::TK] = {};
    float db[NG * E] = {};
    const Matrix<T> mx(p.x, p.rows, p.ld_x, p.n_in), my(p.dy, p.rows, p.ld_dy, p.n_out);
    const bool even = p.n_in == G::KP && p.n_out == G::NP;
    Frag x[SL], dy[NG];
    auto fetch = [&](int64_t tile) {  // past the end: the last row again
        const int64_t row = min(tile * G::kRows + wave * 16 + r, p.rows - 1);
#pragma unroll
        for (int s = 0; s < SL; ++s) x[s] = mx.raw(row, s * KS + E * g);
#pragma unroll
        for (int n = 0; n < NG; ++n) dy[n] = my.raw(row, n * KS + E * g);
    };
    fetch(blockIdx.x);
    auto place = [&](int f, int& n, int& k0) {  // output and first input of fragment f of this lane
        n = f / SL / TG * KS + out_row<T>(f / SL % TG, r);
        k0 = f % SL * KS + E * g;
    };
    if ((int64_t)p.n_out * p.n_in >= E) {
        const Matrix<T> mw(p.w, p.n_out, p.n_in, p.n_in);
        constexpr int kMine = (NG * TG * SL + G::kWaves - 1) / G::kWaves;
        Frag v[kMine];
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            int n, k0;
            place(min(wave + u * G::kWaves, NG * TG * SL - 1), n, k0);
            v[u] = mw.raw(min(n, p.n_out - 1), k0);
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int f = wave + u * G::kWaves;
            if (f >= NG * TG * SL) break;
            int n, k0;
            place(f, n, k0);
            const Frag w = mw.fixed(v[u], min(n, p.n_out - 1), k0, n < p.n_out);
            s_w[f * 64 + w_slot<T>(r, g)] = sizeof(T) == 2 ? swap_halves<T>(w, g & 1) : w;
        }
    } else {  // fewer weights than a fragment
        for (int f = wave; f < NG * TG * SL; f += G::kWaves) {
            int n, k0;
            place(f, n, k0);
            Frag w = zero_frag<T>();
            if (n < p.n_out) w = load_edge(static_cast<const T*>(p.w) + n * p.n_in, k0, p.n_in);
            s_w[f * 64 + w_slot<T>(r, g)] = sizeof(T) == 2 ? swap_halves<T>(w, g & 1) : w;
        }
    }
    for (int i = threadIdx.x; i < G::NP; i += blockDim.x)
        s_bias[i] = p.bias && i < p.n_out ? (float)static_cast<const T*>(p.bias)[i] : 0.f;
    if (threadIdx.x < NG * 4) {
        u32x4 live;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int left = (p.n_out - (int)threadIdx.x * E) * (int)sizeof(T) - 4 * q;  // bytes
            live[q] = left >= 4 ? 0xffffffffu : left == 2 ? 0xffffu : 0u;
        }
        s_live[threadIdx.x] = live;
    }
    __syncthreads();
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t row = tile * G::kRows + wave * 16 + r;
        const int m = wave * 16 + r;
        if ((tile + 1) * G::kRows > p.rows) {  // rows past the end add nothing: dz = 0, x = 0
            const int64_t rc = min(row, p.rows - 1);
#pragma unroll
            for (int s = 0; s < SL; ++s) x[s] = mx.fixed(x[s], rc, s * KS + E * g, row < p.rows);
#pragma unroll
            for (int n = 0; n < NG; ++n) dy[n] = my.fixed(dy[n], rc, n * KS + E * g, row < p.rows);
        } else if (!even) {  // only the last group of a row can reach past its end
            x[SL - 1] = mx.fixed(x[SL - 1], row, (SL - 1) * KS + E * g, true);
#pragma unroll
            for (int n = 0; n < NG; ++n)
                if (!PARTS && n < NG - 1)
                    continue;
                else
                    dy[n] = my.fixed(dy[n], row, n * KS + E * g, true);
        }
#pragma unroll
        for (int s = 0; s < SL; ++s) *reinterpret_cast<Frag*>(s_x + row_chunk<T, G::KP>(m, s * 4 + g)) = x[s];
        if (sizeof(T) == 2) {
#pragma unroll
            for (int s = 0; s < SL; ++s) x[s] = swap_halves<T>(x[s], g & 1);
        }
        // every group's z before the one switch over the activations: branches between the groups would
        // leave the matrix instructions waiting for each other's operands
        float v[NG * E], d[NG * E];
        if (p.act != GS_ACT_NONE) {
            f32x4 z[NG][TG];
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int t = 0; t < TG; ++t) z[n][t] = *reinterpret_cast<f32x4*>(s_bias + n * KS + E * g + 4 * t);
#pragma unroll
            for (int s = 0; s < SL; ++s)
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int t = 0; t < TG; ++t)
                        mma(z[n][t], s_w[((n * TG + t) * SL + s) * 64 + w_slot<T>(r, g)], x[s]);
#pragma unroll
            for (int j = 0; j < NG * E; ++j) v[j] = z[j / E][j % E / 4][j % 4];
        }
#pragma unroll
        for (int j = 0; j < NG * E; ++j) d[j] = (float)dy[j / E][j % E];
        slope_run<T>(p.act, v, d);
        if ((tile + 1) * G::kRows > p.rows && row >= p.rows) {  // the bias can be infinite or NaN there
#pragma unroll
            for (int j = 0; j < NG * E; ++j) v[j] = 0.f;
        }
        Frag dz[NG];
#pragma unroll
        for (int j = 0; j < NG * E; ++j) {
            db[j] += v[j];
            dz[j / E][j % E] = (T)v[j];
        }
        // Past the outputs z is 0 times x, so NaN where x is infinite, and dz with it.  Masks from LDS: 1M rows 128 -> 113
        // float16 279 us; 297 with them in registers, which then spill, and 300 with a comparison for each element.
        if (p.n_out < G::NP) {
#pragma unroll
            for (int n = PARTS ? 0 : NG - 1; n < NG; ++n) {
                union {
                    Frag f;
                    u32x4 q;
                } u;
                u.f = dz[n];
                u.q &= s_live[n * 4 + g];
                dz[n] = u.f;
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) *reinterpret_cast<Frag*>(s_dz + row_chunk<T, G::NP>(m, n * 4 + g)) = dz[n];
        if (p.dx) {
            T* out = static_cast<T*>(p.dx) + row * p.ld_dx;
#pragma unroll
            for (int k0 = 0; k0 < SL; k0 += kPair) {
                Frag f[kPair];
#pragma unroll
                for (int q = 0; q < kPair; ++q) {
                    const int k = k0 + q;
                    if (k >= SL) break;
                    f32x4 acc[TG] = {};
                    if (PARTS && !p.first) {
                        const float* sum = p.dx_sum + min(row, p.rows - 1) * G::KP + k * KS + E * g;
#pragma unroll
                        for (int t = 0; t < TG; ++t) acc[t] = *reinterpret_cast<const f32x4*>(sum + 4 * t);
                    }
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int t = 0; t < TG; ++t) {
                            if constexpr (sizeof(T) == 2) {
                                union {
                                    Frag f;
                                    s16x4 h[2];
                                } u;
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    u.h[h] = read_transposed(
                                        reinterpret_cast<const char*>(s_w + ((n * TG + h) * SL + k) * 64 +
                                                                      w_slot<T>(4 * g + (r >> 2), r & 3)) +
                                        8 * (t ^ (r & 1)));
                                mma(acc[t], u.f, dz[n]);
                            } else {
                                Frag a;  // input r of outputs 4 g .. 4 g + 3
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    a[j] = reinterpret_cast<const float*>(
                                        s_w + (n * SL + k) * 64 + w_slot<T>(4 * g + j, r >> 2))[r & 3];
                                mma(acc[t], a, dz[n]);
                            }
                        }
                    if (PARTS && !p.last) {
                        float* sum = p.dx_sum + row * G::KP + k * KS + E * g;
                        if (row < p.rows) {
#pragma unroll
                            for (int t = 0; t < TG; ++t) *reinterpret_cast<f32x4*>(sum + 4 * t) = acc[t];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < E; ++j) f[q][j] = (T)acc[j / 4][j % 4];
                }
                if ((!PARTS || p.last) && row < p.rows) {
#pragma unroll
                    for (int q = 0; q < kPair; ++q)
                        if (k0 + q < SL) store_run(out, (k0 + q) * KS + E * g, p.n_in, f[q]);
                }
            }
        }
        fetch(tile + gridDim.x);
        __syncthreads();
        if (p.want_dw) {
#pragma unroll
            for (int h = 0; h < G::kRows / KS; ++h) {
                // a rectangle that reaches past dw's edge repeats the last tiles, which are not stored
                Frag fz[G::TN], fx[G::TK];
#pragma unroll
                for (int i = 0; i < G::TN; ++i)
                    fz[i] = column_frag<T, G::NP>(s_dz, h * KS, min(tn0 + i, G::NT - 1) * 16, lane);
#pragma unroll
                for (int j = 0; j < G::TK; ++j)
                    fx[j] = column_frag<T, G::KP>(s_x, h * KS, min(tk0 + j, G::KT - 1) * 16, lane);
#pragma unroll
                for (int i = 0; i < G::TN; ++i)
#pragma unroll
                    for (int j = 0; j < G::TK; ++j) mma(dw[i][j], fz[i], fx[j]);
            }
        }
        __syncthreads();
    }
    const int64_t n_w = p.want_dw ? (int64_t)p.n_out * p.n_in : 0;
    float* part = p.part + blockIdx.x * (n_w + (p.want_db ? p.n_out : 0));
    if (p.want_dw) {
#pragma unroll
        for (int i = 0; i < G::TN; ++i)
#pragma unroll
            for (int j = 0; j < G::TK; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = (tn0 + i) * 16 + 4 * g + q, k = (tk0 + j) * 16 + r;
                    if (n >= p.n_out || k >= p.n_in) continue;
                    if (p.dw)
                        static_cast<T*>(p.dw)[(int64_t)n * p.n_in + k] = (T)dw[i][j][q];
                    else
                        part[(int64_t)n * p.n_in + k] = dw[i][j][q];
                }
    }
    if (p.want_db) {  // over the 16 rows of the lanes, then over the waves, in a fixed order
        float* s_db = reinterpret_cast<float*>(s_dz);  // [waves][NP]
#pragma unroll
        for (int j = 0; j < NG * E; ++j) {
            float v = db[j];
            for (int o = 1; o < 16; o <<= 1) v += __shfl_xor(v, o, 64);
            if (r == 0) s_db[wave * G::NP + j / E * KS + E * g + j % E] = v;
        }
        __syncthreads();
        for (int n = threadIdx.x; n < p.n_out; n += blockDim.x) {
            float v = 0.f;
            for (int i = 0; i < G::kWaves; ++i) v += s_db[i * G::NP + n];
            if (p.db)
                static_cast<T*>(p.db)[n] = (T)v;
            else
                part[n_w + n] = v;
        }
    }
}

// Whether a layer is narrow enough, the blocks its rows fill, and the launch.
template <typename T>
bool bwd_narrow_fits(int32_t n_in, int32_t n_out);
template <typename T>
int bwd_narrow_blocks(int64_t rows, int32_t n_in, int32_t n_out);
template <typename T>
void launch_bwd_narrow(const BwdArgs& p, int blocks, hipStream_t s);

// Their definitions for one type, for the source that compiles it.
template <typename T, int SL, int NG>
inline void bwd_narrow_one(const BwdArgs& p, int64_t rows, int* blocks, hipStream_t s, bool launch) {
    typedef BwdGeom<T, SL, NG> G;
    if (!launch) {
        const int64_t tiles = (rows + G::kRows - 1) / G::kRows, most = 256 * G::kPerCu;
        *blocks = (int)(tiles < most ? tiles : most);
        return;
    }
    if (!p.dx_sum)
        hipLaunchKernelGGL((k_bwd_narrow<T, SL, NG, false>), dim3(*blocks), dim3(G::kWaves * 64), G::kLds, s, p);
    else if constexpr (NG == kBwdGroups && SL * Tile<T>::KS <= kPartInputs)
        hipLaunchKernelGGL((k_bwd_narrow<T, SL, NG, true>), dim3(*blocks), dim3(G::kWaves * 64), G::kLds, s, p);
}

template <typename T, int SL>
inline void bwd_narrow_out(const BwdArgs& p, int64_t rows, int32_t ng, int* blocks, hipStream_t s, bool launch) {
    switch (ng) {
        case 1: bwd_narrow_one<T, SL, 1>(p, rows, blocks, s, launch); break;
        case 2: bwd_narrow_one<T, SL, 2>(p, rows, blocks, s, launch); break;
        case 3: bwd_narrow_one<T, SL, 3>(p, rows, blocks, s, launch); break;
        default: bwd_narrow_one<T, SL, 4>(p, rows, blocks, s, launch); break;
    }
}

template <typename T>
inline void bwd_narrow_any(const BwdArgs& p, int64_t rows, int32_t n_in, int32_t n_out, int* blocks, hipStream_t s,
                           bool launch) {
    const int sl = (n_in + Tile<T>::KS - 1) / Tile<T>::KS;
    const int ng = p.dx_sum ? kBwdGroups : (n_out + Tile<T>::KS - 1) / Tile<T>::KS;
    switch (sl) {
        case 1: bwd_narrow_out<T, 1>(p, rows, ng, blocks, s, launch); break;
        case 2: bwd_narrow_out<T, 2>(p, rows, ng, blocks, s, launch); break;
        case 3: bwd_narrow_out<T, 3>(p, rows, ng, blocks, s, launch); break;
        default: bwd_narrow_out<T, 4>(p, rows, ng, blocks, s, launch); break;
    }
}

#define GS_DEFINE_BWD_NARROW(T)                                                                 \
    template <>                                                                                 \
    bool bwd_narrow_fits<T>(int32_t n_in, int32_t n_out) {                                      \
        constexpr int kMost = kBwdGroups * Tile<T>::KS;                                         \
        return n_in > 0 && n_out > 0 && n_in <= kMost && n_out <= kMost;                        \
    }                                                                                           \
    template <>                                                                                 \
    int bwd_narrow_blocks<T>(int64_t rows, int32_t n_in, int32_t n_out) {                       \
        int blocks = 0;                                                                         \
        bwd_narrow_any<T>(BwdArgs{}, rows, n_in, n_out, &blocks, nullptr, false);               \
        return blocks;                                                                          \
    }                                                                                           \
    template <>                                                                                 \
    void launch_bwd_narrow<T>(const BwdArgs& p, int blocks, hipStream_t s) {                    \
        bwd_narrow_any<T>(p, p.rows, p.n_in, p.n_out, &blocks, s, true);                        \
    }

}  // namespace gs
