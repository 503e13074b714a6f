// Register tiles of the linear layer's kernels (gfx950 matrix instructions, wave64).
//
// A fragment is 16 bytes of a row per lane: lane l holds row l % 16 and, in the
// lane group g = l / 16, the E = 16 / sizeof(T) elements from E g on.  Sixteen
// rows and KS = 4 E elements of the summed index make one step: one 16x16x32
// instruction for the 16-bit types, four 16x16x4 ones for float32 (the j-th
// takes element j of every lane: the sum's order is free as long as both
// operands agree).  Both operands are loaded the same way, so rows that are
// contiguous along the summed index go from memory to the instruction with no
// transpose.
//
// The first operand's rows become the result's rows: lane l then holds rows 4 g
// .. 4 g + 3 of column l % 16.  The layer computes y^T = w x^T, so that a lane
// holds consecutive outputs of one row of y.  For the 16-bit types two tiles
// share a group of KS = 32 outputs with their rows interleaved in fours
// (out_row), so that a lane's 4 + 4 results are 8 consecutive outputs: a run of
// 16 bytes, which is also the fragment of that row that a next product over the
// outputs takes.
#pragma once

#include "gs_internal.h"

namespace gs {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Tile {
    static constexpr int E = 16 / (int)sizeof(T);  // elements of a fragment, and of a result run
    static constexpr int KS = 4 * E;               // elements of the summed index per step, outputs per group
    static constexpr int TG = E / 4;               // 16-row tiles per group of outputs
    typedef T Frag __attribute__((ext_vector_type(16 / sizeof(T))));
};

__device__ __forceinline__ void mma(f32x4& c, Tile<float>::Frag a, Tile<float>::Frag b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4& c, Tile<_Float16>::Frag a, Tile<_Float16>::Frag b) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4& c, Tile<__bf16>::Frag a, Tile<__bf16>::Frag b) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Output (within its group of KS) of row r of tile t.
template <typename T>
__device__ __forceinline__ int out_row(int t, int r) {
    return Tile<T>::E * (r >> 2) + 4 * t + (r & 3);
}

template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag zero_frag() {
    typename Tile<T>::Frag f;
#pragma unroll
    for (int j = 0; j < Tile<T>::E; ++j) f[j] = (T)0.f;
    return f;
}

// 16 bytes at any element alignment (the hardware takes them in one access).
template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag load16(const T* p) {
    typename Tile<T>::Frag f;
    __builtin_memcpy(&f, p, 16);
    return f;
}

// Elements [k0, k0 + E) of a row of `count` elements, zeros from `count` on;
// reads nothing outside the row.  A fragment that straddles the end is loaded
// from the row's last 16 bytes and shifted down.
template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag load_edge(const T* row, int k0, int count) {
    constexpr int E = Tile<T>::E;
    const int last = count - E;
    union {
        typename Tile<T>::Frag f;
        uint64_t q[2];
    } u;
    if (last < 0) {  // a row shorter than a fragment
        u.q[0] = u.q[1] = 0;
#pragma unroll 1
        for (int j = 0; k0 + j < count; ++j) {
            uint64_t b = 0;
            __builtin_memcpy(&b, row + k0 + j, sizeof(T));
            const int at = j * 8 * (int)sizeof(T);
            u.q[0] |= at < 64 ? b << (at & 63) : 0;
            u.q[1] |= at < 64 ? 0 : b << (at & 63);
        }
        return u.f;
    }
    u.f = load16(row + (k0 < last ? k0 : last));
    const int bits = k0 > last ? (k0 - last) * 8 * (int)sizeof(T) : 0;
    if (bits >= 64) {
        u.q[0] = bits >= 128 ? 0 : u.q[1] >> (bits - 64);
        u.q[1] = 0;
    } else if (bits > 0) {
        u.q[0] = (u.q[0] >> bits) | (u.q[1] << (64 - bits));
        u.q[1] >>= bits;
    }
    return u.f;
}

template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag load_frag(const T* row, int k0, int count) {
    if (k0 + Tile<T>::E <= count) return load16(row + k0);
    return load_edge(row, k0, count);
}

// The same in two steps, for loads that stay in flight while other work is done: a
// branch between the load and its use would make the compiler wait for the data at
// the branch's end.  raw() loads 16 bytes from where the fragment starts, or from
// the matrix's last 16 bytes if that is later (the bytes may belong to the next
// rows: nothing outside the matrix is read); fixed() then drops what is not the
// row's.  The matrix spans at least 16 bytes.
template <typename T>
struct Matrix {
    typedef typename Tile<T>::Frag Frag;
    const T* base;
    const T* last;  // start of the last 16 bytes
    int64_t ld;
    int count;      // elements of a row

    __device__ __forceinline__ Matrix(const void* p, int64_t rows, int64_t ld_, int count_)
        : base(static_cast<const T*>(p)), last(base + (rows - 1) * ld_ + count_ - Tile<T>::E), ld(ld_), count(count_) {}
    __device__ __forceinline__ const T* at(int64_t row, int k0) const { return base + row * ld + k0; }
    __device__ __forceinline__ Frag raw(int64_t row, int k0) const {
        const T* p = at(row, k0);
        return load16(p < last ? p : last);
    }
    // in: whether the row counts at all (else zeros)
    __device__ __forceinline__ Frag fixed(Frag f, int64_t row, int k0, bool in) const {
        constexpr int E = Tile<T>::E, kBits = 8 * (int)sizeof(T);
        const T* p = at(row, k0);
        const int64_t over = p - last;
        const int bits = over > 0 ? (over < E ? (int)over * kBits : 128) : 0;
        const int keep = !in || k0 >= count ? 0 : (count - k0 < E ? (count - k0) * kBits : 128);
        union {
            Frag f;
            uint64_t q[2];
        } u;
        u.f = f;
        if (bits >= 64) {
            u.q[0] = bits >= 128 ? 0 : u.q[1] >> (bits - 64);
            u.q[1] = 0;
        } else if (bits > 0) {
            u.q[0] = (u.q[0] >> bits) | (u.q[1] << (64 - bits));
            u.q[1] >>= bits;
        }
        u.q[0] &= keep >= 64 ? ~0ull : (1ull << (keep & 63)) - 1;
        u.q[1] &= keep >= 128 ? ~0ull : keep > 64 ? (1ull << (keep & 63)) - 1 : 0;
        return u.f;
    }
};

// Stores the run's elements that lie inside a row of `count`.
template <typename T>
__device__ __forceinline__ void store_run(T* row, int n0, int count, typename Tile<T>::Frag f) {
    constexpr int E = Tile<T>::E;
    if (n0 + E <= count) {
        __builtin_memcpy(row + n0, &f, 16);
        return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (n0 + j < count) row[n0 + j] = f[j];
}

// The same with at most three stores for the row's last elements, 8, 4 and 2 (float32: 8 and 4) bytes of them.
template <typename T>
__device__ __forceinline__ void store_part(T* row, int n0, int count, typename Tile<T>::Frag f) {
    constexpr int E = Tile<T>::E, kBits = 8 * (int)sizeof(T);
    if (n0 + E <= count) {
        __builtin_memcpy(row + n0, &f, 16);
        return;
    }
    uint64_t q[2];
    __builtin_memcpy(q, &f, 16);
    T* to = row + n0;
    const int left = count - n0;  // may be negative: nothing
    if (left <= 0) return;
    if (left & (E / 2)) {
        __builtin_memcpy(to, q, 8);
        to += E / 2;
        q[0] = q[1];
    }
    if constexpr (E == 8)
        if (left & 2) {
            __builtin_memcpy(to, q, 4);
            to += 2;
            q[0] >>= 2 * kBits;
        }
    if (left & 1) __builtin_memcpy(to, q, sizeof(T));
}

// 1 / (1 + exp(-u)).  float32 results take exp's argument to twice the width (the
// product with log2 e alone is off by |u| 2^-24, which exp multiplies up); the
// 16-bit types' rounding hides that.
template <typename T>
__device__ __forceinline__ float logistic(float u) {
    const float l2e = 1.44269504f;
    float t = -u * l2e, e;
    if (sizeof(T) == 4) {
        // log2 e = l2e + 1.925963033e-8; the low part of -u log2 e moves exp2 by a factor 1 + lo ln 2
        const float lo = fmaf(-u, 1.925963033e-8f, fmaf(-u, l2e, -t));
        const float x = __builtin_amdgcn_exp2f(t);
        e = x > 0.f && x < 3e38f ? fmaf(x, lo * 0.69314718f, x) : x;  // 0, infinity and NaN stay
    } else {
        e = __builtin_amdgcn_exp2f(t);
    }
    return __builtin_amdgcn_rcpf(1.f + e);
}

__device__ __forceinline__ float bounded(float z) {  // gelu's cubic; beyond 64 it is z or 0; NaN stays
    return z > 64.f ? 64.f : (z < -64.f ? -64.f : z);
}
constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act over a lane's run.
template <typename T, int N>
__device__ __forceinline__ void act_run(int act, float (&v)[N]) {
    if (act == GS_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];
    } else if (act == GS_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= logistic<T>(v[j]);
    } else if (act == GS_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float z = bounded(v[j]);
            v[j] *= logistic<T>(kGelu * fmaf(0.044715f * z * z, z, z));
        }
    }
}

// v <- g act'(v) over a lane's run.
template <typename T, int N>
__device__ __forceinline__ void slope_run(int act, float (&v)[N], const float (&g)[N]) {
    if (act == GS_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] > 0.f ? g[j] : (v[j] <= 0.f ? 0.f : v[j]);
    } else if (act == GS_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float z = v[j], s = logistic<T>(z);
            v[j] = g[j] * (s * fmaf(z, 1.f - s, 1.f));
        }
    } else if (act == GS_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float z = bounded(v[j]), q = z * z, s = logistic<T>(kGelu * fmaf(0.044715f * q, z, z));
            v[j] = g[j] * (s * fmaf(z * (1.f - s), kGelu * fmaf(0.134145f, q, 1.f), 1.f));
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = g[j];
    }
}

// v of another lane of the 16 of a lane group.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sums of a run's 8 columns over the rows of the 16 lanes r: columns pair_of(r) and the
// next, the same bits in the four lanes that share them.  Neighbours first halve what
// each of them has to add: 10 additions and 12 selections where every column's own
// sum in every lane would take 32 additions.
__device__ __forceinline__ int pair_of(int r) { return 4 * (r & 1) + (r & 2); }
__device__ __forceinline__ void run_sums(const float (&v)[8], int r, float (&sum)[2]) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = (r & 1 ? v[j + 4] : v[j]) + moved<0xb1>(r & 1 ? v[j] : v[j + 4]);  // lanes 1 0 3 2
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sum[j] = (r & 2 ? q[j + 2] : q[j]) + moved<0x4e>(r & 2 ? q[j] : q[j + 2]);  // lanes 2 3 0 1
        sum[j] += moved<0x128>(sum[j]);                                             // eight lanes on
        sum[j] += moved<0x124>(sum[j]);                                             // four lanes on
    }
}

// Fragments of the transposed operands of dw = dz^T x, whose sum runs down the
// rows: a step takes KS rows, and lane l needs, of column l % 16, E of them.  The
// tile lies in LDS in its own row order, COLS columns a row.  16-bit: two
// transposing reads, each of which hands a group of 16 lanes the 4 x 16 block that
// its lanes' 8-byte pieces of 4 rows make up (lane i: column i); float32: one
// 4-byte read for each of the instruction's four 4-row slices.  Chunks of 16 bytes
// are swapped within a row by a key of the row that serves both accesses: the eight
// rows that a 16-byte write fills at a time differ in it, and so do the pieces (32
// bytes of four rows, float32: 64 bytes of two) that one read takes together.
template <typename T, int COLS>
__device__ __forceinline__ int row_chunk(int m, int c) {  // byte offset of 16-byte chunk c of row m
    constexpr int kChunks = COLS * (int)sizeof(T) / 16;
    int key;
    if constexpr (sizeof(T) == 2) {
        if constexpr (kChunks % 16 == 0)
            key = ((m & 3) << 1) | ((m >> 2) & 1) | (m & 8);
        else if constexpr (kChunks == 8)
            key = ((m & 3) << 1) | ((m >> 2) & 1);
        else  // 4 or 12: rows alternate between the halves of 128 bytes by themselves
            key = (m & 2) | ((m >> 2) & 1);
    } else {
        if constexpr (kChunks % 16 == 0)
            key = ((m & 1) << 2) | ((m >> 1) & 3) | ((m & 2) << 2);
        else if constexpr (kChunks == 8)
            key = ((m & 1) << 2) | ((m >> 1) & 3);
        else
            key = (m >> 1) & 3;
    }
    return m * (COLS * (int)sizeof(T)) + ((c ^ key) << 4);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ s16x4 read_transposed(const char* lds) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<char*>(lds));
}

// Columns [c0, c0 + 16) of rows [m0, m0 + KS), transposed.
template <typename T, int COLS>
__device__ __forceinline__ typename Tile<T>::Frag column_frag(const char* tile, int m0, int c0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
        union {
            typename Tile<T>::Frag f;
            s16x4 h[2];
        } u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = m0 + 8 * g + 4 * h + (r >> 2), c = c0 + 4 * (r & 3);
            u.h[h] = read_transposed(tile + row_chunk<T, COLS>(m, c >> 3) + (c & 7) * 2);
        }
        return u.f;
    } else {
        typename Tile<T>::Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + 4 * j + g, c = c0 + r;
            f[j] = *reinterpret_cast<const float*>(tile + row_chunk<T, COLS>(m, c >> 2) + (c & 3) * 4);
        }
        return f;
    }
}

}  // namespace gs
