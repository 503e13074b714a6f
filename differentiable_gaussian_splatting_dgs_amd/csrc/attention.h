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

// A block's place: problem fastest, so that heads that share lines of memory run together, then the split, and each
// XCD a band.
struct Place {
    int b, hk, tile, split;
    uint32_t problem;
    bool none;
    __device__ __forceinline__ Place(const AttnArgs& p) {
        const uint32_t problems = (uint32_t)(p.batch * p.kv_heads);
        const uint32_t id = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
        none = id >= problems * (uint32_t)(p.tiles * p.splits);
        const uint32_t at = id / problems;
        problem = id - at * problems;
        tile = (int)(at / (uint32_t)p.splits);
        split = (int)at - tile * p.splits;
        b = (int)divided(problem, p.by_kv);
        hk = (int)problem - b * p.kv_heads;
    }
    // first row of this split's partial results of `rows` rows
    __device__ __forceinline__ int64_t part(const AttnArgs& p, int rows) const {
        return ((int64_t)problem * p.splits + split) * rows;
    }
};

// Keys of a tile that count, as bits.
struct Keys {
    const uint8_t* mask;
    int count;  // keys below the length
    __device__ __forceinline__ Keys(const AttnArgs& p, int b)
        : mask(p.mask ? p.mask + b * p.mask_b : nullptr), count(p.k_lengths ? clamped(p.k_lengths[b], p.nk) : p.nk) {}
    // of the split's keys alone
    __device__ __forceinline__ void until(int end) { count = min(count, end); }
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

// A forward's rows: the results, or those of a split.  o is relative to the reference m.
template <typename T, int D, int QC>
__device__ __forceinline__ void forward_rows(const AttnArgs& p, const Place& at, int row0, int live, bool any,
                                             const float (&m)[QC], const float (&l)[QC],
                                             const f32x4 (&o)[QC][AttnTile<T, D>::kPairs][Tile<T>::TG], int lane) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    typedef typename Tile<T>::Frag Frag;
    const int r = lane & 15, g = lane >> 4, rows = p.nq * p.group;
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = row0 + 16 * c + r;
        if (row >= rows) continue;
        if (p.splits > 1) {
            const int64_t to = at.part(p, rows) + row;
#pragma unroll
            for (int e = 0; e < AttnTile<T, D>::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u)
                    *reinterpret_cast<f32x4*>(p.part + to * D + KS * e + E * g + 4 * u) = o[c][e][u];
            if (g == 0) {
                p.part_stat[2 * to] = m[c];
                p.part_stat[2 * to + 1] = any && m[c] == -INFINITY ? NAN : l[c];
            }
            continue;
        }
        const Row w(p, at.hk, row, true);
        const bool empty = !any || row >= live;
        const float inv = 1.f / l[c];
        T* out = static_cast<T*>(p.out) + w.whole(p, at.b) * p.d;
#pragma unroll
        for (int e = 0; e < AttnTile<T, D>::kPairs; ++e) {
            Frag f;
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[4 * u + j] = empty ? (T)0.f : (T)(o[c][e][u][j] * inv);
            store_run(out, KS * e + E * g, p.d, f);
        }
        if (p.lse && g == 0)
            p.lse[w.stat(p, at.b)] =
                empty || m[c] == -INFINITY ? -INFINITY
                                           : (m[c] + __builtin_amdgcn_logf(l[c]) - Softmax<T>::kShift) * kLn2;
    }
}

// The splits' results together: WIDE threads of 4 columns for a row, times SPLITS that share out its splits.
template <typename T, int D, int SHARE>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p) {
    constexpr int kWide = D / 4, kRows = 256 / (kWide * SHARE);
    __shared__ f32x4 s_sum[256];
    __shared__ float s_l[256];
    const int col = threadIdx.x % kWide, share = threadIdx.x / kWide % SHARE, in = threadIdx.x / (kWide * SHARE);
    const int rows = p.nq * p.group;
    const int64_t at = (int64_t)blockIdx.x * kRows + in, total = (int64_t)p.batch * p.kv_heads * rows;
    const int64_t problem = at < total ? at / rows : 0;
    const int row = at < total ? (int)(at - problem * rows) : 0;
    const float* stat = p.part_stat + 2 * (problem * p.splits * rows + row);
    const float* part = p.part + (problem * p.splits * rows + row) * D + 4 * col;
    float m = -INFINITY;
    for (int i = 0; i < p.splits; ++i) m = fmaxf(m, stat[(int64_t)2 * rows * i]);
    f32x4 sum = {};
    float l = 0.f;
#pragma unroll 4
    for (int i = share; i < p.splits; i += SHARE) {
        const float mi = stat[(int64_t)2 * rows * i], li = stat[(int64_t)2 * rows * i + 1];
        const float w = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mi - m);
        const f32x4 o = *reinterpret_cast<const f32x4*>(part + (int64_t)rows * D * i);
        if (mi != -INFINITY || m == -INFINITY) {
            l = fmaf(w, li, l);
            sum += o * w;
        }
    }
    s_sum[threadIdx.x] = sum;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (share > 0 || at >= total) return;
#pragma unroll
    for (int i = 1; i < SHARE; ++i) {
        sum += s_sum[threadIdx.x + i * kWide];
        l += s_l[threadIdx.x + i * kWide];
    }
    const int b = (int)(problem / p.kv_heads), hk = (int)(problem - (int64_t)b * p.kv_heads);
    const Row w(p, hk, row, true);
    const bool empty = row >= live_rows(p, b) || (m == -INFINITY && l == 0.f);  // NaN: logits of -infinity
    const float inv = 1.f / l;
    T* out = static_cast<T*>(p.out) + w.whole(p, b) * p.d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (4 * col + j < p.d) out[4 * col + j] = empty ? (T)0.f : (T)(sum[j] * inv);
    if (p.lse && col == 0)
        p.lse[w.stat(p, b)] = empty || m == -INFINITY ? -INFINITY : (m + __builtin_amdgcn_logf(l) - Softmax<T>::kShift) * kLn2;
}

// Sums of the splits' gradients, rows of dq (KEYS false) or of dk and dv.
template <typename T, int D, int SHARE, bool KEYS>
__global__ __launch_bounds__(256) void k_attn_sum(AttnArgs p) {
    constexpr int kWide = D / 4, kRows = 256 / (kWide * SHARE);
    __shared__ f32x4 s_sum[256];
    const int col = threadIdx.x % kWide, share = threadIdx.x / kWide % SHARE, in = threadIdx.x / (kWide * SHARE);
    const int rows = KEYS ? p.nk : p.nq * p.group;
    const int64_t at = (int64_t)blockIdx.x * kRows + in, problems = (int64_t)p.batch * p.kv_heads;
    const int64_t total = problems * rows * (KEYS ? 2 : 1);
    const int64_t block = at < total ? at / rows : 0;  // KEYS: dk's problems, then dv's
    const int row = at < total ? (int)(at - block * rows) : 0;
    const float* part = p.part + (block * p.splits * rows + row) * D + 4 * col;
    f32x4 sum = {};
#pragma unroll 4
    for (int i = share; i < p.splits; i += SHARE) sum += *reinterpret_cast<const f32x4*>(part + (int64_t)rows * D * i);
    s_sum[threadIdx.x] = sum;
    __syncthreads();
    if (share > 0 || at >= total) return;
#pragma unroll
    for (int i = 1; i < SHARE; ++i) sum += s_sum[threadIdx.x + i * kWide];
    const int64_t problem = block < problems ? block : block - problems;
    const int b = (int)(problem / p.kv_heads), hk = (int)(problem - (int64_t)b * p.kv_heads);
    void* to = !KEYS ? p.dq : block < problems ? p.dk : p.dv;
    if (!to) return;
    T* out = static_cast<T*>(to) +
             (KEYS ? ((int64_t)b * p.nk + row) * p.kv_heads + hk : Row(p, hk, row, true).whole(p, b)) * p.d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (4 * col + j < p.d) out[4 * col + j] = (T)sum[j];
}

// Forward of few rows: 16 QC of them with all keys of a split, which the four waves of a block share out in tiles of
// their own.  A wave reads keys and values from memory as fragments, values through LDS of its own to turn them, and
// nothing but the end waits for another wave: what bounds it is the stream of keys and values.
template <typename T, int D>
struct FewTile {
    static constexpr int kGroups = 32 / (AttnTile<T, D>::kSteps * Tile<T>::TG * 4) < 1
                                       ? 1
                                       : (AttnTile<T, D>::kSteps * Tile<T>::TG * 4 <= 16 ? 2 : 1);
    static constexpr int kKeys = kGroups * Tile<T>::KS;
    static constexpr int kBytes = kKeys * D * (int)sizeof(T);
};

// Fragments of KS rows of a matrix: loads alone, and what they become.
template <typename T, int D, typename Frag, int STEPS>
__device__ __forceinline__ void raw_frags(Frag (&f)[STEPS], const T* base, int g, int d) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int k0 = s * Tile<T>::KS + Tile<T>::E * g;
        f[s] = chunk_load(base, Chunk<T>(k0, d), k0, d);
    }
}
template <typename T, int D, typename Frag, int STEPS>
__device__ __forceinline__ void fix_frags(Frag (&f)[STEPS], int g, int d, bool in) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const Chunk<T> ch(s * Tile<T>::KS + Tile<T>::E * g, d);
        f[s] = chunk_fixed<T>(f[s], ch, d, d == D, in);
    }
}

// What a wave has written to LDS is what its other lanes read.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename T, int D, int QC>
__global__ __launch_bounds__(256, (D * (int)sizeof(T) >= 512 ? 1 : 2)) void k_attn_few(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef FewTile<T, D> F;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, KG = F::kGroups, KW = F::kKeys;
    constexpr int kJoin = 16 * QC * D * 4;
    __shared__ __align__(16) char s_mem[4 * F::kBytes > kJoin ? 4 * F::kBytes : kJoin];
    __shared__ float s_m[4][16 * QC], s_l[4][16 * QC];
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Keys keys(p, at.b);
    const int first = at.split * p.per, last = keys.count - 1;
    keys.until(first + p.per);
    const int live = live_rows(p, at.b);
    const float c2 = fabsf(p.scale) * kLog2e;
    char* tv = s_mem + wave * F::kBytes;

    Frag q[QC][A::kSteps];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const bool in = 16 * c + r < live;
        const Row w(p, at.hk, 16 * c + r, in);
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
    const T* k_base = static_cast<const T*>(p.k) + at.b * p.k_b + at.hk * p.k_h;
    const T* v_base = static_cast<const T*>(p.v) + at.b * p.v_b + at.hk * p.v_h;
    Frag k[KG][TG][A::kSteps], v[KG][TG][A::kSteps];
    int byte = 0;
    auto fetch = [&](int k0) {
        byte = lane < KW ? keys.byte(k0, lane) : 0;
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const int64_t key = min(k0 + kg * KS + out_row<T>(u, r), last);
                raw_frags<T, D>(k[kg][u], k_base + key * p.k_n, g, p.d);
                raw_frags<T, D>(v[kg][u], v_base + key * p.v_n, g, p.d);
            }
    };
    int k0 = first + wave * KW;
    if (k0 < keys.count && live > 0) fetch(k0);
    for (; k0 < keys.count && live > 0; k0 += 4 * KW) {
        const uint64_t valid = __ballot(byte != 0);
        any |= valid;
        f32x4 s[QC][KG][TG] = {};
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                fix_frags<T, D>(k[kg][u], g, p.d, true);
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e)
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(s[c][kg][u], k[kg][u][e], q[c][e]);
                const int row = kg * KS + out_row<T>(u, r);
                fix_frags<T, D>(v[kg][u], g, p.d, valid >> row & 1);
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e)
                    *reinterpret_cast<Frag*>(tv + tile_at<T, D>(row, 4 * e + g)) = v[kg][u][e];
            }
        if (k0 + 4 * KW < keys.count) fetch(k0 + 4 * KW);
        wave_sync();
        if (valid != ~0ull >> (64 - KW)) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = valid >> (kg * KS + E * g + 4 * u + j) & 1;
#pragma unroll
                        for (int c = 0; c < QC; ++c) s[c][kg][u][j] = in ? s[c][kg][u][j] : -INFINITY;
                    }
        }
        Frag w[QC][KG];
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
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
                for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                    for (int u = 0; u < TG; ++u) o[c][e][u] *= by;
            }
            const float ref = (m[c] == -INFINITY ? 0.f : m[c]) - Softmax<T>::kShift;
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
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
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const Frag a = down_frag<T, D>(tv, kg * KS, e, u, lane);
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(o[c][e][u], a, w[c][kg]);
                }
        wave_sync();
    }
    // the waves' results together, in their order
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        l[c] = over_groups(l[c], [](float a, float b) { return a + b; });
        if (g == 0) s_m[wave][16 * c + r] = m[c], s_l[wave][16 * c + r] = l[c];
    }
    const bool some = __syncthreads_or(any != 0);
    float* s_o = reinterpret_cast<float*>(s_mem);  // [16 QC][D]
    float top[QC], sum[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = 16 * c + r;
        top[c] = fmaxf(fmaxf(s_m[0][row], s_m[1][row]), fmaxf(s_m[2][row], s_m[3][row]));
        sum[c] = 0.f;
        for (int i = 0; i < 4; ++i)
            if (s_m[i][row] != -INFINITY) sum[c] = fmaf(__builtin_amdgcn_exp2f(s_m[i][row] - top[c]), s_l[i][row], sum[c]);
        const float by = m[c] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[c] - top[c]);
#pragma unroll
        for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
            for (int u = 0; u < TG; ++u) o[c][e][u] *= by;
    }
    for (int i = 0; i < 4; ++i) {
        if (wave == i) {
#pragma unroll
            for (int c = 0; c < QC; ++c)
#pragma unroll
                for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                    for (int u = 0; u < TG; ++u) {
                        f32x4* to = reinterpret_cast<f32x4*>(s_o + (16 * c + r) * D + KS * e + E * g + 4 * u);
                        if (i > 0) o[c][e][u] += *to;
                        if (i < 3) *to = o[c][e][u];
                    }
        }
        __syncthreads();
    }
    if (wave == 3) forward_rows<T, D, QC>(p, at, 0, live, some, top, sum, o, lane);
}

// Forward over tiles of 64 QC rows and the keys of a split.
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
    Keys keys(p, at.b);
    const int first = at.split * p.per, last = keys.count - 1;
    keys.until(first + p.per);
    const int live = live_rows(p, at.b);
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
    auto fetch = [&](int k0) {
        mk.load([&](int i) { return k_base + (int64_t)min(k0 + i, last) * p.k_n; }, p.d);
        mv.load([&](int i) { return v_base + (int64_t)min(k0 + i, last) * p.v_n; }, p.d);
    };
    const int tiles = live > at.tile * 64 * QC ? (keys.count - first + KT - 1) / KT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        const int byte = keys.byte(first, lane);
        fetch(first);
        valid = key_bits<KT>(byte);
        mk.store(s_k[0], valid, p.d, whole);
        mv.store(s_v[0], valid, p.d, whole);
    }
    for (int t = 0; t < tiles; ++t) {
        int byte = 0;
        if (t + 1 < tiles) {
            byte = keys.byte(first + (t + 1) * KT, lane);
            fetch(first + (t + 1) * KT);
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
    for (int c = 0; c < QC; ++c) l[c] = over_groups(l[c], [](float a, float b) { return a + b; });
    forward_rows<T, D, QC>(p, at, row0, live, any != 0, m, l, o, lane);
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

// dq over tiles of 64 QC rows and the keys of a split; leaves the rows' delta for the other gradients.
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
    Keys keys(p, at.b);
    const int first = at.split * p.per, last = keys.count - 1;
    keys.until(first + p.per);
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
        if (in && g == 0 && at.split == 0) p.delta[w.stat(p, at.b)] = delta[c];
    }

    f32x4 dq[QC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    Mover<T, D> mk, mv;
    const T* k_base = static_cast<const T*>(p.k) + at.b * p.k_b + at.hk * p.k_h;
    const T* v_base = static_cast<const T*>(p.v) + at.b * p.v_b + at.hk * p.v_h;
    auto fetch = [&](int k0) {
        mk.load([&](int i) { return k_base + (int64_t)min(k0 + i, last) * p.k_n; }, p.d);
        mv.load([&](int i) { return v_base + (int64_t)min(k0 + i, last) * p.v_n; }, p.d);
    };
    const int tiles = p.dq && live > at.tile * 64 * QC ? (keys.count - first + KT - 1) / KT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        const int byte = keys.byte(first, lane);
        fetch(first);
        valid = key_bits<KT>(byte);
        mk.store(s_k[0], valid, p.d, whole);
        mv.store(s_v[0], valid, p.d, whole);
    }
    for (int t = 0; t < tiles; ++t) {
        int byte = 0;
        if (t + 1 < tiles) {
            byte = keys.byte(first + (t + 1) * KT, lane);
            fetch(first + (t + 1) * KT);
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
        if (p.splits > 1) {
            float* to = p.part + (at.part(p, rows) + row) * D;
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u)
                    *reinterpret_cast<f32x4*>(to + KS * e + E * g + 4 * u) = row < live ? dq[c][e][u] * by : f32x4{};
            continue;
        }
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

// dk and dv over tiles of 64 KC keys and the rows of a split.  Here a lane holds consecutive rows of one key: s = q k^T.
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
    const int first = at.split * p.per, live = min(live_rows(p, at.b), first + p.per);
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
    const int tiles = keys.count > at.tile * 64 * KC ? (live - first + RT - 1) / RT : 0;
    uint64_t valid = 0;
    if (tiles > 0) {
        fetch(first);
        valid = bits(first);
        place(0, valid);
    }
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) fetch(first + (t + 1) * RT);
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
            valid = bits(first + (t + 1) * RT);
            place((t + 1) & 1, valid);
        }
    }
    const float by = __builtin_amdgcn_exp2f(-shrink.shift);
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int key = key0 + 16 * c + r;
        if (key >= p.nk) continue;
        if (p.splits > 1) {
            float* to = p.part + (at.part(p, p.nk) + key) * D;
            float* to_v = to + (int64_t)p.batch * p.kv_heads * p.splits * p.nk * D;
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const int k = KS * e + E * g + 4 * u;
                    *reinterpret_cast<f32x4*>(to + k) = counts[c] ? dk[c][e][u] * (by * p.scale) : f32x4{};
                    *reinterpret_cast<f32x4*>(to_v + k) = counts[c] ? dv[c][e][u] * by : f32x4{};
                }
            continue;
        }
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

inline int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }
inline size_t padded(size_t b) { return (b + 255) & ~(size_t)255; }
inline dim3 grid_of(const AttnArgs& p) {
    const int64_t blocks = (int64_t)p.batch * p.kv_heads * p.tiles * p.splits;
    return dim3((unsigned)((blocks + 7) / 8 * 8));
}

// Splits of n, each of a multiple of `step`, that bring `blocks` blocks to about `want`, none shorter than `least`.
inline void split(int64_t n, int64_t blocks, int64_t want, int64_t least, int64_t step, int& splits, int& per) {
    int64_t parts = blocks > 0 ? want / blocks : 1;
    parts = parts > n / least ? n / least : parts;
    parts = parts < 1 ? 1 : parts > 512 ? 512 : parts;
    const int64_t each = tiles_of(tiles_of(n, parts), step) * step;
    per = (int)(each < step ? step : each);
    splits = (int)(n > 0 ? tiles_of(n, per) : 1);
}

template <typename T, int D>
AttnPlan plan_at(const AttnArgs& p) {
    typedef AttnShape<T, D> S;
    AttnPlan a{};
    const int64_t problems = (int64_t)p.batch * p.kv_heads, rows = (int64_t)p.nq * p.group;
    const size_t row_part = (size_t)problems * rows * D * 4, key_part = (size_t)problems * p.nk * D * 4;
    a.few = rows <= 16 ? 1 : rows <= 32 ? 2 : 0;
    a.fwd_qc = rows <= 64 * S::kFwd / 2 ? 1 : S::kFwd;
    a.dq_qc = rows <= 64 * S::kDq / 2 ? 1 : S::kDq;
    a.dkv_kc = p.nk <= 64 * S::kDkv / 2 ? 1 : S::kDkv;
    if (a.few) split(p.nk, problems, 1024, 512, 4 * FewTile<T, D>::kKeys, a.fwd_splits, a.fwd_per);
    else split(p.nk, problems * tiles_of(rows, 64 * a.fwd_qc), 512, 512, AttnTile<T, D>::kRows, a.fwd_splits, a.fwd_per);
    split(p.nk, problems * tiles_of(rows, 64 * a.dq_qc), 512, 256, AttnTile<T, D>::kRows, a.dq_splits, a.dq_per);
    split(rows, problems * tiles_of(p.nk, 64 * a.dkv_kc), 512, 256, AttnTile<T, D>::kRows, a.dkv_splits, a.dkv_per);
    if (a.fwd_splits > 1) a.fwd_bytes = padded(row_part * a.fwd_splits) + padded(row_part / D * 2 * a.fwd_splits);
    a.delta_bytes = padded((size_t)problems * rows * 4);
    if (a.dq_splits > 1) a.dq_bytes = padded(row_part * a.dq_splits);
    // dq's partials are joined before those of dk and dv are made
    const size_t kv = a.dkv_splits > 1 ? padded(2 * key_part * a.dkv_splits) : 0;
    a.bwd_bytes = a.delta_bytes + (a.dq_bytes > kv ? a.dq_bytes : kv);
    return a;
}

// A kernel over rows of WIDE threads, with as many threads for a row's splits as there are, up to a block.
#define GS_ATTN_SHARED(KERNEL, ROWS, ...)                                                                       \
    do {                                                                                                        \
        constexpr int kMost = 1024 / D;                                                                         \
        const int64_t rows_ = (ROWS);                                                                           \
        if (p.splits <= 2 || kMost < 4)                                                                         \
            hipLaunchKernelGGL((KERNEL<T, D, 1 __VA_ARGS__>), dim3((unsigned)tiles_of(rows_, kMost)), dim3(256), 0, s, p); \
        else if (p.splits <= 16 || kMost < 16)                                                                  \
            hipLaunchKernelGGL((KERNEL<T, D, 4 __VA_ARGS__>), dim3((unsigned)tiles_of(rows_, kMost / 4)), dim3(256), 0, s, p); \
        else                                                                                                    \
            hipLaunchKernelGGL((KERNEL<T, D, (kMost < 16 ? kMost : 16) __VA_ARGS__>),                           \
                               dim3((unsigned)tiles_of(rows_, kMost < 16 ? 1 : kMost / 16)), dim3(256), 0, s, p); \
    } while (0)

template <typename T, int D>
void attn_fwd_at(AttnArgs p, void* workspace, hipStream_t s) {
    const AttnPlan a = plan_at<T, D>(p);
    const int64_t rows = (int64_t)p.nq * p.group, problems = (int64_t)p.batch * p.kv_heads;
    p.splits = a.fwd_splits, p.per = a.fwd_per;
    p.part = static_cast<float*>(workspace);
    if (p.splits > 1) p.part_stat = p.part + padded((size_t)problems * rows * D * 4 * p.splits) / 4;
    if (a.few) {
        p.tiles = 1;
        if (a.few == 1) hipLaunchKernelGGL((k_attn_few<T, D, 1>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_few<T, D, 2>), grid_of(p), dim3(256), 0, s, p);
    } else {
        p.tiles = (int32_t)tiles_of(rows, 64 * a.fwd_qc);
        if (a.fwd_qc == 1) hipLaunchKernelGGL((k_attn_fwd<T, D, 1>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_fwd<T, D, AttnShape<T, D>::kFwd>), grid_of(p), dim3(256), 0, s, p);
    }
    if (p.splits > 1) GS_ATTN_SHARED(k_attn_join, problems * rows);
}

template <typename T, int D>
void attn_bwd_at(AttnArgs p, void* workspace, hipStream_t s) {
    const AttnPlan a = plan_at<T, D>(p);
    const int64_t rows = (int64_t)p.nq * p.group, problems = (int64_t)p.batch * p.kv_heads;
    p.delta = static_cast<float*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + a.delta_bytes);
    if (p.nq > 0) {
        p.splits = p.dq ? a.dq_splits : 1, p.per = p.dq ? a.dq_per : 0;
        p.tiles = (int32_t)tiles_of(rows, 64 * a.dq_qc);
        if (a.dq_qc == 1) hipLaunchKernelGGL((k_attn_dq<T, D, 1>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_dq<T, D, AttnShape<T, D>::kDq>), grid_of(p), dim3(256), 0, s, p);
        if (p.splits > 1) GS_ATTN_SHARED(k_attn_sum, problems * rows, , false);
    }
    if (p.nk > 0 && (p.dk || p.dv)) {
        p.splits = a.dkv_splits, p.per = a.dkv_per;
        p.tiles = (int32_t)tiles_of(p.nk, 64 * a.dkv_kc);
        if (a.dkv_kc == 1) hipLaunchKernelGGL((k_attn_dkv<T, D, 1>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_dkv<T, D, AttnShape<T, D>::kDkv>), grid_of(p), dim3(256), 0, s, p);
        if (p.splits > 1) GS_ATTN_SHARED(k_attn_sum, 2 * problems * p.nk, , true);
    }
}

#define GS_ATTN_BY_HEAD(CALL)            \
    (p.d <= 32    ? CALL<T, 32>          \
     : p.d <= 64  ? CALL<T, 64>          \
     : p.d <= 128 ? CALL<T, 128>         \
                  : CALL<T, 256>)

template <typename T>
AttnPlan attn_plan(const AttnArgs& p) {
    return GS_ATTN_BY_HEAD(plan_at)(p);
}
template <typename T>
void attn_fwd(const AttnArgs& p, void* workspace, hipStream_t s) {
    GS_ATTN_BY_HEAD(attn_fwd_at)(p, workspace, s);
}
template <typename T>
void attn_bwd(const AttnArgs& p, void* workspace, hipStream_t s) {
    GS_ATTN_BY_HEAD(attn_bwd_at)(p, workspace, s);
}

}  // namespace gs
