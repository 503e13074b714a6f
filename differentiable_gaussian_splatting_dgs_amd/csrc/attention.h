// Cross attention: softmax(scale q k^T) v of every batch item and head, and its gradients (gfx950 matrix
// instructions, wave64).
//
// A problem is a batch item and a head of keys.  The `group` heads of queries that share the keys are rows of one
// matrix, row = query * group + head in the group, so that every key is read once for all of them; queries past a
// batch item's length are the last rows.  Products are taken so that softmax's rows lie in lanes: s^T = k q^T gives
// a lane 4 (16-bit: 4 + 4) consecutive keys of one row (linear_tile.h's fragments and its order of rows within a
// group of tiles), which are, rounded, the fragment that the next product takes: o^T = v^T p^T.  A row's maximum and
// sum are numbers of its lane, the same in the four lane groups.  Fragments down the rows of a tile in LDS (v^T)
// come from transposing reads.
//
// exp is exp2 of scale log2 e s.  A row's reference m trails its maximum: it moves (and what is summed so far is
// scaled) only when a logit passes it by more than kSlack, which nothing that is summed in float32 notices.
// float16 weights are held times 2^kShift: the range from 2^-24 up would lose the small ones of a long row.
// A key that its length or mask takes out has weight 0 and is zero in LDS: 0 times infinity or NaN would
// otherwise reach every row.
#pragma once

#include "attention_args.h"
#include "linear_tile.h"

namespace gs {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t divided(uint32_t n, Div d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

template <typename T>
struct Softmax {  // base 2
    static constexpr float kShift = sizeof(T) == 2 ? 0.f : 0.f, kSlack = 8.f;
};
template <>
struct Softmax<_Float16> {
    static constexpr float kShift = 13.f, kSlack = 2.f;  // 2^15 < 65504
};

// Rows of a tile in LDS, for two buffers of two tiles at two blocks a CU.
template <typename T, int D>
struct AttnTile {
    static constexpr int kRows = 16384 / (D * (int)sizeof(T)) < 64 ? 16384 / (D * (int)sizeof(T)) : 64;
    static constexpr int kBytes = kRows * D * (int)sizeof(T);
    static constexpr int kChunks = D / Tile<T>::E;           // of 16 bytes, in a row
    static constexpr int kEach = kRows * kChunks / 256;      // that a thread moves
    static constexpr int kGroups = kRows / Tile<T>::KS;      // of KS rows: the steps of a sum over the rows
    static constexpr int kSteps = D / Tile<T>::KS;           // of a sum over a row
    static constexpr int kPairs = D / 16 / Tile<T>::TG;      // groups of TG result tiles over the columns
    static_assert(kEach >= 1 && kGroups >= 1 && 256 % kChunks == 0, "tile");
};

// 16-row tiles of queries, and of keys, that a wave holds: what its registers allow.
template <typename T, int D>
struct AttnShape {
    static constexpr bool kSmall = sizeof(T) == 2;
    static constexpr int kFwd = D <= 64 && kSmall ? 4 : D <= 128 ? 2 : 1;
    static constexpr int kDq = D <= 64 ? 2 : 1;
    static constexpr int kDkv = D <= 64 ? 2 : 1;
    static constexpr int kOcc = D * (int)sizeof(T) >= 256 && !(kSmall && D == 128) ? 1 : 2;  // waves a SIMD
};

// Byte offset of 16-byte chunk c of row m.  float32: reads of a row's chunks take sixteen rows at a time, reads
// down the columns four rows that lie four apart, and the key tells both apart.
template <typename T, int D>
__device__ __forceinline__ int tile_at(int m, int c) {
    if constexpr (sizeof(T) == 2) {
        return row_chunk<T, D>(m, c);
    } else {
        constexpr int kMask = D * 4 / 16 >= 16 ? 15 : 7;
        return m * (D * 4) + ((c ^ (m & kMask)) << 4);
    }
}

// Fragment of row m, step s: the first operand of a product over the columns.
template <typename T, int D>
__device__ __forceinline__ typename Tile<T>::Frag row_frag(const char* tile, int m, int s, int g) {
    return *reinterpret_cast<const typename Tile<T>::Frag*>(tile + tile_at<T, D>(m, 4 * s + g));
}

// Columns of result tile t of pair c over rows [m0, m0 + KS), transposed: lane (r, g) has column
// KS c + out_row(t, r), rows m0 + E g on.
template <typename T, int D>
__device__ __forceinline__ typename Tile<T>::Frag down_frag(const char* tile, int m0, int c, int t, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
        union {
            typename Tile<T>::Frag f;
            s16x4 h[2];
        } u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = m0 + 8 * g + 4 * h + (r >> 2);
            u.h[h] = read_transposed(tile + tile_at<T, D>(m, 4 * c + (r & 3)) + t * 8);
        }
        return u.f;
    } else {
        typename Tile<T>::Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = *reinterpret_cast<const float*>(tile + tile_at<T, D>(m0 + 4 * g + j, 4 * c + (r >> 2)) + (r & 3) * 4);
        return f;
    }
}

// A 16-byte chunk of a row of d elements, zeros from d on: the element where its load starts, and the bits of it
// that lie before the chunk.
template <typename T>
struct Chunk {
    int start, drop;
    __device__ __forceinline__ Chunk(int k0, int d) {
        constexpr int E = Tile<T>::E;
        start = max(min(k0, d - E), 0);
        drop = min(k0 - start, E) * 8 * (int)sizeof(T);
    }
};

// Rows shorter than a chunk are read element by element.  whole: the row has no end inside or before a chunk.
template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag chunk_load(const T* row, const Chunk<T>& c, int k0, int d) {
    if (d < Tile<T>::E) return load_edge(row, k0, d);
    return load16(row + c.start);
}
template <typename T>
__device__ __forceinline__ typename Tile<T>::Frag chunk_fixed(typename Tile<T>::Frag f, const Chunk<T>& c, int d,
                                                              bool whole, bool in) {
    union {
        typename Tile<T>::Frag f;
        uint64_t q[2];
    } u;
    u.f = f;
    if (!whole && d >= Tile<T>::E) {
        if (c.drop >= 64) {
            u.q[0] = c.drop >= 128 ? 0 : u.q[1] >> (c.drop - 64);
            u.q[1] = 0;
        } else if (c.drop > 0) {
            u.q[0] = (u.q[0] >> c.drop) | (u.q[1] << (64 - c.drop));
            u.q[1] >>= c.drop;
        }
    }
    u.q[0] = in ? u.q[0] : 0;
    u.q[1] = in ? u.q[1] : 0;
    return u.f;
}

// Rows of a matrix in memory on their way into a tile of LDS: each thread moves the same chunk of kEach rows.
template <typename T, int D>
struct Mover {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    Frag f[A::kEach];

    static __device__ __forceinline__ int row(int i) { return i * (256 / A::kChunks) + threadIdx.x / A::kChunks; }
    // at(row): where the tile's row starts in memory, some row inside the matrix for those that do not count
    template <typename At>
    __device__ __forceinline__ void load(At at, int d) {
        const int k0 = (int)(threadIdx.x % A::kChunks) * Tile<T>::E;
        const Chunk<T> c(k0, d);
#pragma unroll
        for (int i = 0; i < A::kEach; ++i) f[i] = chunk_load(at(row(i)), c, k0, d);
    }
    __device__ __forceinline__ void store(char* tile, uint64_t valid, int d, bool whole) const {
        const int ch = threadIdx.x % A::kChunks;
        const Chunk<T> c(ch * Tile<T>::E, d);
#pragma unroll
        for (int i = 0; i < A::kEach; ++i) {
            const int m = row(i);
            *reinterpret_cast<Frag*>(tile + tile_at<T, D>(m, ch)) = chunk_fixed<T>(f[i], c, d, whole, valid >> m & 1);
        }
    }
};

__device__ __forceinline__ int clamped(int n, int most) { return n < 0 ? 0 : n < most ? n : most; }

// The combination of a value over the four lane groups, in all of them.
template <typename F>
__device__ __forceinline__ float over_groups(float v, F f) {
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const unsigned p0 = p[0], p1 = p[1];
    const unsigned b = __builtin_bit_cast(unsigned, f(__builtin_bit_cast(float, p0), __builtin_bit_cast(float, p1)));
    const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const unsigned s0 = s[0], s1 = s[1];
    return f(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}

// A block's place: problem fastest, so that heads that share lines of memory run together, and each XCD a band.
struct Place {
    int b, hk, tile;
    bool none;
    __device__ __forceinline__ Place(const AttnArgs& p) {
        const uint32_t problems = (uint32_t)(p.batch * p.kv_heads);
        const uint64_t total = (uint64_t)problems * p.tiles;
        const uint32_t per = gridDim.x >> 3;
        const uint64_t id = (uint64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
        none = id >= total;
        tile = (int)((uint32_t)id / problems);
        const uint32_t at = (uint32_t)id - tile * problems;
        b = (int)divided(at, p.by_kv);
        hk = (int)(at - b * p.kv_heads);
    }
};

// Keys of a tile that count, as bits.
struct Keys {
    const uint8_t* mask;
    int count;  // keys below the length
    __device__ __forceinline__ Keys(const AttnArgs& p, int b)
        : mask(p.mask ? p.mask + b * p.mask_b : nullptr), count(p.k_lengths ? clamped(p.k_lengths[b], p.nk) : p.nk) {}
    // a lane's byte of the tile at k0; asked for before it is needed
    __device__ __forceinline__ int byte(int k0, int lane) const {
        const int key = k0 + lane;
        if (!mask) return key < count;
        return key < count ? mask[key] : 0;
    }
};

template <int KEYS>
__device__ __forceinline__ uint64_t key_bits(int byte) {
    const uint64_t all = __ballot(byte != 0);
    return all & (~0ull >> (64 - KEYS));
}

// Query and head of a row of a problem (of row 0 for those that do not count).
struct Row {
    int64_t query;
    int head;
    __device__ __forceinline__ Row(const AttnArgs& p, int hk, int row, bool in) {
        const int at = in ? row : 0, i = (int)divided((uint32_t)at, p.by_group);
        query = i;
        head = hk * p.group + at - i * p.group;
    }
    __device__ __forceinline__ int64_t whole(const AttnArgs& p, int b) const {  // row of a whole [batch, nq, heads, d]
        return ((int64_t)b * p.nq + query) * p.heads + head;
    }
    __device__ __forceinline__ int64_t stat(const AttnArgs& p, int b) const {  // element of [batch, heads, nq]
        return ((int64_t)b * p.heads + head) * p.nq + query;
    }
};

// Rows that count: of queries below the length.
__device__ __forceinline__ int live_rows(const AttnArgs& p, int b) {
    return (p.q_lengths ? clamped(p.q_lengths[b], p.nq) : p.nq) * p.group;
}

// A row's fragments over all of its columns, zeros if it does not count.
template <typename T, int D, typename Frag, int STEPS>
__device__ __forceinline__ void row_frags(Frag (&f)[STEPS], const T* base, int g, int d, bool in) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int k0 = s * Tile<T>::KS + Tile<T>::E * g;
        const Chunk<T> ch(k0, d);
        f[s] = chunk_fixed<T>(chunk_load(base, ch, k0, d), ch, d, d == D, in);
    }
}

// Forward over tiles of 64 QC rows and all keys.
template <typename T, int D, int QC>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOcc)) void k_attn_fwd(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, KT = A::kRows, NG = A::kGroups;
    __shared__ __align__(16) char s_k[2][A::kBytes], s_v[2][A::kBytes];
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Keys keys(p, at.b);
    const int rows = p.nq * p.group, live = live_rows(p, at.b);
    const int row0 = (at.tile * 4 + wave) * 16 * QC;
    const bool whole = p.d == D;
    const float c2 = fabsf(p.scale) * kLog2e;

    Frag q[QC][A::kSteps];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const bool in = row0 + 16 * c + r < live;
        const Row w(p, at.hk, row0 + 16 * c + r, in);
        row_frags<T, D>(q[c], static_cast<const T*>(p.q) + at.b * p.q_b + w.query * p.q_n + w.head * p.q_h, g, p.d, in);
        if (p.scale < 0.f)
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s) q[c][s] = -q[c][s];
    }

    f32x4 o[QC][A::kPairs][TG] = {};
    float m[QC], l[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) m[c] = -INFINITY, l[c] = 0.f;
    uint64_t any = 0;
    Mover<T, D> mk, mv;
    const T* k_base = static_cast<const T*>(p.k) + at.b * p.k_b + at.hk * p.k_h;
    const T* v_base = static_cast<const T*>(p.v) + at.b * p.v_b + at.hk * p.v_h;
    const int last = keys.count - 1;
    auto fetch = [&](int k0) {
        mk.load([&](int i) { return k_base + (int64_t)min(k0 + i, last) * p.k_n; }, p.d);
        mv.load([&](int i) { return v_base + (int64_t)min(k0 + i, last) * p.v_n; }, p.d);
    };
    const int tiles = live > at.tile * 64 * QC ? (keys.count + KT - 1) / KT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        const int byte = keys.byte(0, lane);
        fetch(0);
        valid = key_bits<KT>(byte);
        mk.store(s_k[0], valid, p.d, whole);
        mv.store(s_v[0], valid, p.d, whole);
    }
    for (int t = 0; t < tiles; ++t) {
        int byte = 0;
        if (t + 1 < tiles) {
            byte = keys.byte((t + 1) * KT, lane);
            fetch((t + 1) * KT);
        }
        __syncthreads();
        const char* tk = s_k[t & 1];
        const char* tv = s_v[t & 1];
        f32x4 s[QC][NG][TG] = {};
#pragma unroll
        for (int kg = 0; kg < NG; ++kg)
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) {
                    const Frag a = row_frag<T, D>(tk, kg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(s[c][kg][u], a, q[c][e]);
                }
        any |= valid;
        if (valid != ~0ull >> (64 - KT)) {
#pragma unroll
            for (int kg = 0; kg < NG; ++kg)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = valid >> (kg * KS + E * g + 4 * u + j) & 1;
#pragma unroll
                        for (int c = 0; c < QC; ++c) s[c][kg][u][j] = in ? s[c][kg][u][j] : -INFINITY;
                    }
        }
        Frag w[QC][NG];
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int kg = 0; kg < NG; ++kg)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = fmaxf(top, s[c][kg][u][j]);
            top = over_groups(top, [](float a, float b) { return fmaxf(a, b); }) * c2;
            if (__any(top > m[c] + Softmax<T>::kSlack || m[c] == -INFINITY)) {
                const float next = fmaxf(top, m[c]);
                const float by = __builtin_amdgcn_exp2f(next == -INFINITY ? 0.f : m[c] - next);
                m[c] = next;
                l[c] *= by;
#pragma unroll
                for (int dp = 0; dp < A::kPairs; ++dp)
#pragma unroll
                    for (int u = 0; u < TG; ++u) o[c][dp][u] *= by;
            }
            const float ref = (m[c] == -INFINITY ? 0.f : m[c]) - Softmax<T>::kShift;
#pragma unroll
            for (int kg = 0; kg < NG; ++kg)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e = __builtin_amdgcn_exp2f(fmaf(s[c][kg][u][j], c2, -ref));
                        l[c] += e;
                        w[c][kg][4 * u + j] = (T)e;
                    }
        }
#pragma unroll
        for (int kg = 0; kg < NG; ++kg)
#pragma unroll
            for (int dp = 0; dp < A::kPairs; ++dp)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const Frag a = down_frag<T, D>(tv, kg * KS, dp, u, lane);
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(o[c][dp][u], a, w[c][kg]);
                }
        if (t + 1 < tiles) {
            valid = key_bits<KT>(byte);
            mk.store(s_k[(t + 1) & 1], valid, p.d, whole);
            mv.store(s_v[(t + 1) & 1], valid, p.d, whole);
        }
    }
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = row0 + 16 * c + r;
        if (row >= rows) continue;
        const Row at_row(p, at.hk, row, true);
        const bool empty = any == 0 || row >= live;
        const float sum = over_groups(l[c], [](float a, float b) { return a + b; });
        const float inv = 1.f / sum;
        T* out = static_cast<T*>(p.out) + at_row.whole(p, at.b) * p.d;
#pragma unroll
        for (int dp = 0; dp < A::kPairs; ++dp) {
            Frag f;
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * u + j] = empty ? (T)0.f : (T)(o[c][dp][u][j] * inv);
            store_run(out, KS * dp + E * g, p.d, f);
        }
        if (p.lse && g == 0)
            p.lse[at_row.stat(p, at.b)] =
                empty ? -INFINITY : (m[c] + __builtin_amdgcn_logf(sum) - Softmax<T>::kShift) * kLn2;
    }
}

// Gradients.  With P = exp(s - lse) and ds = P (dout v^T - delta), delta the row's sum of dout * out:
// dq = scale ds k, dk = scale ds^T q, dv = P^T dout.  P and ds enter the products rounded to the type.  float16:
// both are held times 2^kShift and, should a ds not fit then, scaled down with what is summed so far (Shrink).
template <typename T>
struct Shrink {
    float shift = 0.f;
    template <typename Over>
    __device__ __forceinline__ void operator()(float, Over) {}
};
template <>
struct Shrink<_Float16> {
    float shift = Softmax<_Float16>::kShift;
    // most: the lane's largest |ds| of this step; over(f) scales what the wave holds by f
    template <typename Over>
    __device__ __forceinline__ void operator()(float most, Over over) {
        if (!__any(most > 32768.f)) return;
        most = most < INFINITY ? most : 0.f;  // infinities and NaN stay what they are
        for (int o = 1; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
        const int by = most > 16384.f ? ilogbf(most) - 13 : 0;
        over(ldexpf(1.f, -by));
        shift -= (float)by;
    }
};

// dq over tiles of 64 QC rows and all keys; leaves the rows' delta for the other gradients.
template <typename T, int D, int QC>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOcc)) void k_attn_dq(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, KT = A::kRows, NG = A::kGroups;
    __shared__ __align__(16) char s_k[2][A::kBytes], s_v[2][A::kBytes];
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Keys keys(p, at.b);
    const int rows = p.nq * p.group, live = live_rows(p, at.b);
    const int row0 = (at.tile * 4 + wave) * 16 * QC;
    const bool whole = p.d == D;
    const float c2 = fabsf(p.scale) * kLog2e;

    Frag q[QC][A::kSteps], dout[QC][A::kSteps];
    float lse[QC], delta[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const bool in = row0 + 16 * c + r < live;
        const Row w(p, at.hk, row0 + 16 * c + r, in);
        row_frags<T, D>(q[c], static_cast<const T*>(p.q) + at.b * p.q_b + w.query * p.q_n + w.head * p.q_h, g, p.d, in);
        row_frags<T, D>(dout[c], static_cast<const T*>(p.dout) + at.b * p.g_b + w.query * p.g_n + w.head * p.g_h, g,
                        p.d, in);
        Frag out[A::kSteps];
        row_frags<T, D>(out, static_cast<const T*>(p.out) + w.whole(p, at.b) * p.d, g, p.d, in);
        if (p.scale < 0.f)
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s) q[c][s] = -q[c][s];
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < A::kSteps; ++s)
#pragma unroll
            for (int j = 0; j < E; ++j) sum = fmaf((float)dout[c][s][j], (float)out[s][j], sum);
        delta[c] = over_groups(sum, [](float a, float b) { return a + b; });
        lse[c] = in ? p.lse[w.stat(p, at.b)] * kLog2e : 0.f;
        if (in && g == 0) p.delta[w.stat(p, at.b)] = delta[c];
    }

    f32x4 dq[QC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    Mover<T, D> mk, mv;
    const T* k_base = static_cast<const T*>(p.k) + at.b * p.k_b + at.hk * p.k_h;
    const T* v_base = static_cast<const T*>(p.v) + at.b * p.v_b + at.hk * p.v_h;
    const int last = keys.count - 1;
    auto fetch = [&](int k0) {
        mk.load([&](int i) { return k_base + (int64_t)min(k0 + i, last) * p.k_n; }, p.d);
        mv.load([&](int i) { return v_base + (int64_t)min(k0 + i, last) * p.v_n; }, p.d);
    };
    const int tiles = p.dq && live > at.tile * 64 * QC ? (keys.count + KT - 1) / KT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        const int byte = keys.byte(0, lane);
        fetch(0);
        valid = key_bits<KT>(byte);
        mk.store(s_k[0], valid, p.d, whole);
        mv.store(s_v[0], valid, p.d, whole);
    }
    for (int t = 0; t < tiles; ++t) {
        int byte = 0;
        if (t + 1 < tiles) {
            byte = keys.byte((t + 1) * KT, lane);
            fetch((t + 1) * KT);
        }
        __syncthreads();
        const char* tk = s_k[t & 1];
        const char* tv = s_v[t & 1];
#pragma unroll
        for (int kg = 0; kg < NG; ++kg) {
            f32x4 s[QC][TG] = {}, dp[QC][TG] = {};
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) {
                    const Frag a = row_frag<T, D>(tk, kg * KS + out_row<T>(u, r), e, g);
                    const Frag b = row_frag<T, D>(tv, kg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                    for (int c = 0; c < QC; ++c) {
                        mma(s[c][u], a, q[c][e]);
                        mma(dp[c][u], b, dout[c][e]);
                    }
                }
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < QC; ++c) {
                const float ref = lse[c] - shrink.shift;
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = valid >> (kg * KS + E * g + 4 * u + j) & 1;
                        const float w = __builtin_amdgcn_exp2f(fmaf(s[c][u][j], c2, -ref));
                        const float ds = in ? w * (dp[c][u][j] - delta[c]) : 0.f;
                        s[c][u][j] = ds;
                        most = fmaxf(most, fabsf(ds));
                    }
            }
            shrink(most, [&](float f) {
#pragma unroll
                for (int c = 0; c < QC; ++c) {
#pragma unroll
                    for (int u = 0; u < TG; ++u) s[c][u] *= f;
#pragma unroll
                    for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                        for (int u = 0; u < TG; ++u) dq[c][e][u] *= f;
                }
            });
            Frag ds[QC];
#pragma unroll
            for (int c = 0; c < QC; ++c)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) ds[c][4 * u + j] = (T)s[c][u][j];
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const Frag a = down_frag<T, D>(tk, kg * KS, e, u, lane);
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(dq[c][e][u], a, ds[c]);
                }
        }
        if (t + 1 < tiles) {
            valid = key_bits<KT>(byte);
            mk.store(s_k[(t + 1) & 1], valid, p.d, whole);
            mv.store(s_v[(t + 1) & 1], valid, p.d, whole);
        }
    }
    if (!p.dq) return;
    const float by = p.scale * __builtin_amdgcn_exp2f(-shrink.shift);
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = row0 + 16 * c + r;
        if (row >= rows) continue;
        T* to = static_cast<T*>(p.dq) + Row(p, at.hk, row, true).whole(p, at.b) * p.d;
#pragma unroll
        for (int e = 0; e < A::kPairs; ++e) {
            Frag f;
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * u + j] = row < live ? (T)(dq[c][e][u][j] * by) : (T)0.f;
            store_run(to, KS * e + E * g, p.d, f);
        }
    }
}

// dk and dv over tiles of 64 KC keys and all rows.  Here a lane holds consecutive rows of one key: s = q k^T.
template <typename T, int D, int KC>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOcc)) void k_attn_dkv(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, RT = A::kRows, NG = A::kGroups;
    __shared__ __align__(16) char s_q[2][A::kBytes], s_g[2][A::kBytes];
    __shared__ __align__(16) float s_lse[2][RT], s_delta[2][RT];
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Keys keys(p, at.b);
    const int live = live_rows(p, at.b);
    const int key0 = (at.tile * 4 + wave) * 16 * KC;
    const bool whole = p.d == D;
    const float c2 = fabsf(p.scale) * kLog2e;

    Frag k[KC][A::kSteps], v[KC][A::kSteps];
    bool counts[KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int key = key0 + 16 * c + r;
        counts[c] = key < keys.count && (!keys.mask || keys.mask[key]);
        const int64_t from = counts[c] ? key : 0;
        row_frags<T, D>(k[c], static_cast<const T*>(p.k) + at.b * p.k_b + from * p.k_n + at.hk * p.k_h, g, p.d, counts[c]);
        row_frags<T, D>(v[c], static_cast<const T*>(p.v) + at.b * p.v_b + from * p.v_n + at.hk * p.v_h, g, p.d, counts[c]);
        if (p.scale < 0.f)
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s) k[c][s] = -k[c][s];
    }

    f32x4 dk[KC][A::kPairs][TG] = {}, dv[KC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    Mover<T, D> mq, mg;
    const T* q_base = static_cast<const T*>(p.q) + at.b * p.q_b;
    const T* g_base = static_cast<const T*>(p.dout) + at.b * p.g_b;
    float next_lse = 0.f, next_delta = 0.f;
    auto fetch = [&](int row0) {
        mq.load([&](int i) {
            const Row w(p, at.hk, row0 + i, row0 + i < live);
            return q_base + w.query * p.q_n + w.head * p.q_h;
        }, p.d);
        mg.load([&](int i) {
            const Row w(p, at.hk, row0 + i, row0 + i < live);
            return g_base + w.query * p.g_n + w.head * p.g_h;
        }, p.d);
        if (threadIdx.x < RT) {
            const int row = row0 + (int)threadIdx.x;
            const int64_t stat = Row(p, at.hk, row, row < live).stat(p, at.b);
            next_lse = p.lse[stat] * kLog2e;
            next_delta = p.delta[stat];
        }
    };
    auto place = [&](int buffer, uint64_t valid) {
        mq.store(s_q[buffer], valid, p.d, whole);
        mg.store(s_g[buffer], valid, p.d, whole);
        if (threadIdx.x < RT) s_lse[buffer][threadIdx.x] = next_lse, s_delta[buffer][threadIdx.x] = next_delta;
    };
    // rows below the last: bits of the tile's rows that count
    auto bits = [&](int row0) { return live - row0 >= 64 ? ~0ull : (1ull << (live - row0)) - 1; };
    const int tiles = keys.count > at.tile * 64 * KC ? (live + RT - 1) / RT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        fetch(0);
        valid = bits(0);
        place(0, valid);
    }
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) fetch((t + 1) * RT);
        __syncthreads();
        const char* tq = s_q[t & 1];
        const char* tg = s_g[t & 1];
#pragma unroll
        for (int rg = 0; rg < NG; ++rg) {
            f32x4 s[KC][TG] = {}, dp[KC][TG] = {};
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) {
                    const Frag a = row_frag<T, D>(tq, rg * KS + out_row<T>(u, r), e, g);
                    const Frag b = row_frag<T, D>(tg, rg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        mma(s[c][u], a, k[c][e]);
                        mma(dp[c][u], b, v[c][e]);
                    }
                }
            float most[KC] = {};
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const f32x4 lse = *reinterpret_cast<const f32x4*>(&s_lse[t & 1][rg * KS + E * g + 4 * u]);
                const f32x4 delta = *reinterpret_cast<const f32x4*>(&s_delta[t & 1][rg * KS + E * g + 4 * u]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = valid >> (rg * KS + E * g + 4 * u + j) & 1;
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const float w = in ? __builtin_amdgcn_exp2f(fmaf(s[c][u][j], c2, shrink.shift - lse[j])) : 0.f;
                        const float ds = in ? w * (dp[c][u][j] - delta[j]) : 0.f;
                        s[c][u][j] = w;
                        dp[c][u][j] = ds;
                        most[c] = fmaxf(most[c], fabsf(ds));
                    }
                }
            }
            float any = 0.f;  // keys that do not count have weights that mean nothing
#pragma unroll
            for (int c = 0; c < KC; ++c) any = fmaxf(any, counts[c] ? most[c] : 0.f);
            shrink(any, [&](float f) {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
#pragma unroll
                    for (int u = 0; u < TG; ++u) s[c][u] *= f, dp[c][u] *= f;
#pragma unroll
                    for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                        for (int u = 0; u < TG; ++u) dk[c][e][u] *= f, dv[c][e][u] *= f;
                }
            });
            Frag w[KC], ds[KC];
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[c][4 * u + j] = (T)s[c][u][j], ds[c][4 * u + j] = (T)dp[c][u][j];
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const Frag a = down_frag<T, D>(tg, rg * KS, e, u, lane);
                    const Frag b = down_frag<T, D>(tq, rg * KS, e, u, lane);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        mma(dv[c][e][u], a, w[c]);
                        mma(dk[c][e][u], b, ds[c]);
                    }
                }
        }
        if (t + 1 < tiles) {
            valid = bits((t + 1) * RT);
            place((t + 1) & 1, valid);
        }
    }
    const float by = __builtin_amdgcn_exp2f(-shrink.shift);
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int key = key0 + 16 * c + r;
        if (key >= p.nk) continue;
        const int64_t row = (((int64_t)at.b * p.nk + key) * p.kv_heads + at.hk) * p.d;
#pragma unroll
        for (int e = 0; e < A::kPairs; ++e) {
            Frag a, b;
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[4 * u + j] = counts[c] ? (T)(dk[c][e][u][j] * (by * p.scale)) : (T)0.f;
                    b[4 * u + j] = counts[c] ? (T)(dv[c][e][u][j] * by) : (T)0.f;
                }
            if (p.dk) store_run(static_cast<T*>(p.dk) + row, KS * e + E * g, p.d, a);
            if (p.dv) store_run(static_cast<T*>(p.dv) + row, KS * e + E * g, p.d, b);
        }
    }
}

// Launches.

inline int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }
inline dim3 grid_of(const AttnArgs& p) {
    const int64_t blocks = (int64_t)p.batch * p.kv_heads * p.tiles;
    return dim3((unsigned)((blocks + 7) / 8 * 8));
}

template <typename T, int D>
void attn_fwd_at(AttnArgs p, hipStream_t s) {
    constexpr int QC = AttnShape<T, D>::kFwd;
    p.tiles = (int32_t)tiles_of((int64_t)p.nq * p.group, 64 * QC);
    hipLaunchKernelGGL((k_attn_fwd<T, D, QC>), grid_of(p), dim3(256), 0, s, p);
}

template <typename T, int D>
void attn_bwd_at(AttnArgs p, hipStream_t s) {
    constexpr int QC = AttnShape<T, D>::kDq, KC = AttnShape<T, D>::kDkv;
    if (p.nq > 0) {
        p.tiles = (int32_t)tiles_of((int64_t)p.nq * p.group, 64 * QC);
        hipLaunchKernelGGL((k_attn_dq<T, D, QC>), grid_of(p), dim3(256), 0, s, p);
    }
    if (p.nk > 0 && (p.dk || p.dv)) {
        p.tiles = (int32_t)tiles_of(p.nk, 64 * KC);
        hipLaunchKernelGGL((k_attn_dkv<T, D, KC>), grid_of(p), dim3(256), 0, s, p);
    }
}

template <typename T>
void attn_fwd(const AttnArgs& p, hipStream_t s) {
    if (p.d <= 32) attn_fwd_at<T, 32>(p, s);
    else if (p.d <= 64) attn_fwd_at<T, 64>(p, s);
    else if (p.d <= 128) attn_fwd_at<T, 128>(p, s);
    else attn_fwd_at<T, 256>(p, s);
}

template <typename T>
void attn_bwd(const AttnArgs& p, hipStream_t s) {
    if (p.d <= 32) attn_bwd_at<T, 32>(p, s);
    else if (p.d <= 64) attn_bwd_at<T, 64>(p, s);
    else if (p.d <= 128) attn_bwd_at<T, 128>(p, s);
    else attn_bwd_at<T, 256>(p, s);
}

}  // namespace gs
