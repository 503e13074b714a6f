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
// exp is exp2 of scale log2 e s.  A row's reference trails its maximum: it moves (and what is summed so far is scaled)
// only when weights grow past 2^8, which nothing that is summed in float32 notices.
// float16 weights are held times 2^kShift: its steps of 2^-24 would lose the small ones of a long row.
// A key that its length or mask takes out has weight 0 and is zero in LDS: 0 times infinity or NaN would
// otherwise reach every row.
#pragma once

#include <utility>

#include "attention_args.h"
#include "linear_tile.h"

namespace gs {

constexpr int kHeadsApart = 65536;     // keys from which few rows' heads go to the waves of a block
constexpr int kThinBlocks = 512;       // that keep their keys: two a CU
constexpr int kThinTiles = 16;         // tiles of keys that a block keeps in LDS, at most
constexpr int kThinBytes = 64 * 1024;  // and their bytes: two blocks a CU
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t divided(uint32_t n, Div d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// The forward's weights are relative to 2^(reference - kShift); past kMost, in the sum of a lane's, it moves.
template <typename T>
struct Softmax {
    static constexpr float kShift = 0.f, kMost = 256.f;
};
template <>
struct Softmax<_Float16> {
    static constexpr float kShift = 7.f, kMost = 32768.f;
};

// Rows of a tile in LDS, for two buffers of two tiles at two blocks a CU.  D columns take part in products, a multiple
// of KS; rows lie a power of two apart.
constexpr int pitch_of(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 128 ? 128 : 256; }
template <typename T, int D>
struct AttnTile {
    static constexpr int kPitch = pitch_of(D);
    static constexpr int kRows = 16384 / (kPitch * (int)sizeof(T)) < 64 ? 16384 / (kPitch * (int)sizeof(T)) : 64;
    static constexpr int kBytes = kRows * kPitch * (int)sizeof(T);
    static constexpr int kChunks = kPitch / Tile<T>::E;      // of 16 bytes, in a row
    static constexpr int kEach = kRows * kChunks / 256;      // that a thread moves
    static constexpr int kGroups = kRows / Tile<T>::KS;      // of KS rows: the steps of a sum over the rows
    static constexpr int kSteps = D / Tile<T>::KS;           // of a sum over a row
    static constexpr int kPairs = D / 16 / Tile<T>::TG;      // groups of TG result tiles over the columns
    static_assert(kEach >= 1 && kGroups >= 1 && 256 % kChunks == 0 && D % Tile<T>::KS == 0, "tile");
};

// 16-row tiles of queries, and of keys, that a wave holds: each more is one more use of what a wave reads from LDS,
// for as many registers as a wave has at kOcc* waves a SIMD (512 in all).  bfloat16, 64k rows on 1024 keys of 128: dq
// takes 326 us with one tile, which LDS bounds (a fragment of 1 KB a product), 240 with two, though 60 bytes a lane spill;
// float32 products take four times as long for a fragment and want the second wave more: 20k rows on 512 keys of 128,
// forward 262 us with two tiles at one wave, 232 at two, 205 with one tile at two.
template <typename T, int D>
struct AttnShape {
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int kFwd = kHalf ? (D <= 64 ? 4 : D <= 128 ? 2 : 1) : D <= 96 ? 2 : 1;
    static constexpr int kDq = kHalf ? (D <= 128 ? 2 : 1) : D <= 64 ? 2 : 1;
    static constexpr int kDkv = kHalf ? (D <= 128 ? 2 : 1) : D <= 64 ? 2 : 1;
    static constexpr int kThin = D <= 32 ? (kHalf ? 4 : 2) : D <= 128 ? (kHalf ? 2 : 1) : 1;
    static constexpr int kOccThin = D * (int)sizeof(T) >= 512 ? 1 : 2;
    static constexpr int kOccFwd = D * (int)sizeof(T) >= 1024 ? 1 : 2;
    static constexpr int kOccDq = D * (int)sizeof(T) >= 1024 ? 1 : 2;
    static constexpr int kHeld = D <= (kHalf ? 128 : 64) ? 2 : 1;
    // by the registers of keys, values, their gradients and a tile's logits; the rest takes some 130
    static constexpr int occ_held(int kc) { return kc * ((kHalf ? D / 2 + D / 4 : D) + 32) <= 112 ? 2 : 1; }
    // by the registers of keys, values and their gradients, and what may spill: bfloat16, 30k x 600 of 160 320 us at one
    // wave and 167 at two, 64k x 1024 of 128 (192 registers) 400 and 848
    static constexpr int kOccDkv = kDkv * D * (kHalf ? 3 : 4) <= 576 ? 2 : 1;
};

// Keys that a wave takes at a time where rows are few: what 32 registers hold of them.
template <typename T, int D>
struct FewTile {
    static constexpr int kGroups = AttnTile<T, D>::kSteps * Tile<T>::TG * 4 <= 16 ? 2 : 1;
    static constexpr int kKeys = kGroups * Tile<T>::KS;
    static constexpr int kBytes = kKeys * pitch_of(D) * (int)sizeof(T);
};

// Byte offset of 16-byte chunk c of row m.  LDS hands out 256 bytes a cycle: 16 chunks, which for a row fragment are
// two neighbouring ones of 8 rows, four and four of 16 (out_row).  So the key tells rows apart by bits 0, 1 and 3 and
// leaves a chunk's lowest bit alone.  16-bit reads down the columns take
// the same half of four neighbouring chunks of 8 rows at a time and meet every bank twice at best, which is what they do
// here: 4 cycles a fragment by rows, 8 down the columns.  Shorter rows share the 256 bytes and need less of the key.
template <typename T, int D>
__device__ __forceinline__ int tile_at(int m, int c) {
    constexpr int kBytes = D < 32 ? D * (int)sizeof(T) : pitch_of(D) * (int)sizeof(T), kChunks = kBytes / 16;
    int key;
    if constexpr (sizeof(T) == 2) {
        const int x = (m >> 3 ^ m >> 2) & 1;
        key = kChunks >= 16 ? (m & 3) << 1 | x << 3 : kChunks == 8 ? (m & 2) << 1 | x << 1 : x << 1;
    } else {
        key = m & (kChunks >= 16 ? 15 : kChunks - 1);
    }
    return m * kBytes + ((c ^ key) << 4);
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

// How a kernel reads rows.  WHOLE: d fills the padded row, a power of two.  EVEN: d is some chunks.  PART: a row's last
// chunk is loaded from its last 16 bytes and shifted.  These take 32-bit offsets from a tile's first row.  ANY: rows
// shorter than a chunk, read element by element, and offsets of 64 bits.
enum { WHOLE, EVEN, PART, ANY };
constexpr bool direct(int mode) { return mode <= EVEN; }  // tiles of rows that loads can write to LDS by themselves

template <typename T, int MODE>
__device__ __forceinline__ typename Tile<T>::Frag chunk_load(const T* row, const Chunk<T>& c, int k0, int d) {
    if constexpr (MODE == WHOLE) return load16(row + k0);
    if constexpr (MODE == ANY)
        if (d < Tile<T>::E) return load_edge(row, k0, d);
    return load16(row + c.start);
}
// What of a loaded chunk is the row's; in: whether the row counts (else zeros).
template <typename T, int MODE>
__device__ __forceinline__ typename Tile<T>::Frag chunk_fixed(typename Tile<T>::Frag f, const Chunk<T>& c, int d,
                                                              bool in) {
    union {
        typename Tile<T>::Frag f;
        uint64_t q[2];
    } u;
    u.f = f;
    if (MODE == EVEN) in = in && c.drop == 0;
    if (MODE == PART || (MODE == ANY && d >= Tile<T>::E)) {
        const int by = c.drop & 63;
        const uint64_t low = by ? (u.q[0] >> by) | (u.q[1] << (64 - by)) : u.q[0], high = u.q[1] >> by;
        u.q[0] = c.drop < 64 ? low : c.drop < 128 ? high : 0;
        u.q[1] = c.drop < 64 ? high : 0;
    }
    u.q[0] = in ? u.q[0] : 0;
    u.q[1] = in ? u.q[1] : 0;
    return u.f;
}

// Rows of a matrix in memory on their way into a tile of LDS: each thread moves a chunk of kEach rows.  at holds the
// offsets of its loads from the tile's first row (bytes).  DIRECT: the loads write LDS themselves, lane l of a wave
// the l-th 16 bytes of the wave's run, so that a lane reads the chunk that tile_at has there, and hold no registers on
// their way; chunks past d are left as blank() made them.  64k rows of 128 on 1024 keys, forward and backward: 782 us
// against 862 through registers.
template <typename T, int D, int MODE, bool DIRECT = false>
struct Mover {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    static_assert(!DIRECT || direct(MODE), "direct loads");
    Frag f[DIRECT ? 1 : A::kEach];
    uint32_t at[MODE == ANY ? 1 : A::kEach];

    static __device__ __forceinline__ int row(int i) { return i * (256 / A::kChunks) + threadIdx.x / A::kChunks; }
    static __device__ __forceinline__ int first() { return (int)(threadIdx.x % A::kChunks) * Tile<T>::E; }
    // the column that a direct load of row(i) takes
    static __device__ __forceinline__ int column(int i) {
        return ((tile_at<T, D>(row(i), threadIdx.x % A::kChunks) >> 4) - row(i) * A::kChunks) * Tile<T>::E;
    }
    // of(i): element offset of the tile's row i
    template <typename Of>
    __device__ __forceinline__ void aim(Of of, int d) {
        if constexpr (MODE != ANY) {
            const uint32_t start = MODE == WHOLE ? first() : Chunk<T>(first(), d).start;
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                at[i] = ((uint32_t)of(row(i)) + (DIRECT ? (uint32_t)column(i) : start)) * (uint32_t)sizeof(T);
        }
    }
    // DIRECT: zeros in the chunks of a tile past d
    static __device__ __forceinline__ void blank(char* tile, int d) {
        if (DIRECT && MODE != WHOLE)
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                if (column(i) >= d) *reinterpret_cast<Frag*>(tile + (i * 256 + (int)threadIdx.x) * 16) = Frag{};
    }
    // from: the tile's first row in memory, the same for all lanes; to (DIRECT): the tile in LDS, which nobody reads now
    __device__ __forceinline__ void load(const T* from, char* to, int d) {
        if constexpr (DIRECT) {
            const uint32_t run = __builtin_amdgcn_readfirstlane(
                (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to + (threadIdx.x >> 6) * 1024);
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                if (MODE == WHOLE || column(i) < d)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is nobody's to keep, but what the compiler does with it must know
                    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(run + i * 4096),
                                 "v"(at[i]), "s"(from)
                                 : "memory", "m0");
#pragma clang diagnostic pop
        } else {
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                f[i] = load16(reinterpret_cast<const T*>(reinterpret_cast<const char*>(from) + at[i]));
        }
    }
    // where(i): the tile's row i in memory
    template <typename Where>
    __device__ __forceinline__ void load_any(Where where, int d) {
        const Chunk<T> c(first(), d);
#pragma unroll
        for (int i = 0; i < A::kEach; ++i) f[i] = chunk_load<T, ANY>(where(row(i)), c, first(), d);
    }
    // the loaded tile in LDS, zeros in rows that do not count; DIRECT: what a wave has in flight is there from here on
    __device__ __forceinline__ void place(char* tile, uint64_t valid, int d) const {
        if constexpr (DIRECT) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (valid == ~0ull >> (64 - A::kRows)) return;
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                if (!(valid >> row(i) & 1)) *reinterpret_cast<Frag*>(tile + (i * 256 + (int)threadIdx.x) * 16) = Frag{};
            return;
        }
        const int ch = threadIdx.x % A::kChunks;
        const Chunk<T> c(first(), d);
        if (MODE == WHOLE && valid == ~0ull >> (64 - A::kRows)) {
#pragma unroll
            for (int i = 0; i < A::kEach; ++i)
                *reinterpret_cast<Frag*>(tile + tile_at<T, D>(row(i), ch)) = f[DIRECT ? 0 : i];
            return;
        }
#pragma unroll
        for (int i = 0; i < A::kEach; ++i)
            *reinterpret_cast<Frag*>(tile + tile_at<T, D>(row(i), ch)) =
                chunk_fixed<T, MODE>(f[DIRECT ? 0 : i], c, d, valid >> row(i) & 1);
    }
};

// Tiles of consecutive keys of one matrix.
template <typename T, int D, int MODE, bool DIRECT = false>
struct KeyTiles {
    Mover<T, D, MODE, DIRECT> move;
    const T* base;  // of key 0
    int64_t stride;
    int end;        // of the keys that may be read: past it, the last one is read again
    __device__ __forceinline__ KeyTiles(const void* p, int64_t from, int64_t stride_, int end_, int d)
        : base(static_cast<const T*>(p) + from), stride(stride_), end(end_) {
        move.aim([&](int i) { return (uint32_t)i * (uint32_t)stride; }, d);
    }
    __device__ __forceinline__ void load(int key, int d, char* to) {
        if constexpr (MODE == ANY) {
            move.load_any([&](int i) { return base + (int64_t)min(key + i, end - 1) * stride; }, d);
        } else {
            if (key + AttnTile<T, D>::kRows > end)
                move.aim([&](int i) { return (uint32_t)min(i, end - 1 - key) * (uint32_t)stride; }, d);
            move.load(base + key * stride, to, d);
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

// Sum over the 16 lanes of a group, in all of them (rotated by 8, 4, 2 and 1).
__device__ __forceinline__ float over_row(float v) {
    auto turned = [](float v, auto by) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                     0x120 + decltype(by)::value, 0xf, 0xf, true));
    };
    v += turned(v, std::integral_constant<int, 8>());
    v += turned(v, std::integral_constant<int, 4>());
    v += turned(v, std::integral_constant<int, 2>());
    v += turned(v, std::integral_constant<int, 1>());
    return v;
}

// A block's place: problem fastest, so that heads that share lines of memory run together, then the split, and each
// XCD a band.
struct Place {
    int b, hk, tile, split;
    uint32_t problem;
    bool none;
    // together: the log of how many heads of keys a block takes
    __device__ __forceinline__ explicit Place(const AttnArgs& p, int together = 0) {
        const uint32_t problems = (uint32_t)(p.batch * p.kv_heads) >> together;
        const uint32_t id = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
        none = id >= problems * (uint32_t)(p.tiles * p.splits);
        const uint32_t at = id / problems;
        problem = id - at * problems;
        tile = (int)(at / (uint32_t)p.splits);
        split = (int)at - tile * p.splits;
        b = (int)divided(problem << together, p.by_kv);
        hk = (int)(problem << together) - b * p.kv_heads;
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

// Whether a tile's group of KS rows holds any that count.
template <typename T>
__device__ __forceinline__ bool group_counts(uint64_t valid, int group) {
    return (valid >> (group * Tile<T>::KS) & ((1ull << Tile<T>::KS) - 1)) != 0;
}

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

// A row's fragments over all of its columns: loads alone, and what they become (zeros if the row does not count).
template <typename T, int MODE, typename Frag, int STEPS>
__device__ __forceinline__ void raw_frags(Frag (&f)[STEPS], const T* base, int g, int d) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int k0 = s * Tile<T>::KS + Tile<T>::E * g;
        f[s] = chunk_load<T, MODE>(base, Chunk<T>(k0, d), k0, d);
    }
}
template <typename T, int MODE, typename Frag, int STEPS>
__device__ __forceinline__ void fix_frags(Frag (&f)[STEPS], int g, int d, bool in) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        f[s] = chunk_fixed<T, MODE>(f[s], Chunk<T>(s * Tile<T>::KS + Tile<T>::E * g, d), d, in);
}

// What a wave has written to LDS is what its other lanes read.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float added(float v) {
    return over_groups(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float highest(float v) {
    return over_groups(v, [](float a, float b) { return fmaxf(a, b); });
}

// Fragments of QC tiles of 16 rows from `row0` on, as second operands; negative: for a scale below 0.
template <typename T, int MODE, typename Frag, int QC, int STEPS>
__device__ __forceinline__ void rows_held(const AttnArgs& p, int b, int hk, int row0, int live, const void* from,
                                          int64_t s_b, int64_t s_n, int64_t s_h, bool negative, int lane,
                                          Frag (&f)[QC][STEPS]) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const Row w(p, hk, row0 + 16 * c + r, row0 + 16 * c + r < live);
        raw_frags<T, MODE>(f[c], static_cast<const T*>(from) + b * s_b + w.query * s_n + w.head * s_h, g, p.d);
    }
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        fix_frags<T, MODE>(f[c], g, p.d, row0 + 16 * c + r < live);
        if (negative)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) f[c][s] = -f[c][s];
    }
}

// Tiles of consecutive rows of a problem, of q or dout.
template <typename T, int D, int MODE, bool DIRECT = false>
struct RowTiles {
    Mover<T, D, MODE, DIRECT> move;
    const T* base;  // of the problem's first head
    int64_t s_n, s_h;
    __device__ __forceinline__ RowTiles(const AttnArgs& p, int b, int hk, const void* from, int64_t s_b, int64_t s_n_,
                                        int64_t s_h_)
        : base(static_cast<const T*>(from) + b * s_b + (int64_t)hk * p.group * s_h_), s_n(s_n_), s_h(s_h_) {
        if (p.group == 1) move.aim([&](int i) { return (uint32_t)i * (uint32_t)s_n; }, p.d);
    }
    // rows from row0 on; past the last live one it is read again
    __device__ __forceinline__ void load(const AttnArgs& p, int row0, int live, char* to) {
        if constexpr (MODE == ANY) {
            move.load_any([&](int i) {
                const Row w(p, 0, min(row0 + i, live - 1), true);
                return base + w.query * s_n + w.head * s_h;
            }, p.d);
        } else if (p.group == 1) {
            if (row0 + AttnTile<T, D>::kRows > live)
                move.aim([&](int i) { return (uint32_t)min(i, live - 1 - row0) * (uint32_t)s_n; }, p.d);
            move.load(base + row0 * s_n, to, p.d);
        } else {
            const int first = (int)divided((uint32_t)row0, p.by_group), in = row0 - first * p.group;
            move.aim([&](int i) {
                const uint32_t row = in + min(i, live - 1 - row0), query = divided(row, p.by_group);
                return query * (uint32_t)s_n + (row - query * p.group) * (uint32_t)s_h;
            }, p.d);
            move.load(base + first * s_n, to, p.d);
        }
    }
};

// Launches.

inline int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }
inline size_t padded(size_t b) { return (b + 255) & ~(size_t)255; }
inline dim3 grid_of(const AttnArgs& p) {
    const int64_t blocks = ((int64_t)p.batch * p.kv_heads >> p.together) * p.tiles * p.splits;
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

// Whether rows need more than 32-bit offsets from a tile of 64 keys or rows and the heads of a group, or are short.
template <typename T>
bool attn_any(const AttnArgs& p) {
    const int64_t most = ((int64_t)1 << 31) / (int64_t)sizeof(T);
    int64_t far = 64 * (p.k_n > p.v_n ? p.k_n : p.v_n);
    const int64_t d = p.d;  // out's rows are whole, also where q is one head expanded
    for (const auto& s : {std::pair<int64_t, int64_t>{p.q_n, p.q_h}, {p.g_n, p.g_h}, {p.heads * d, d}}) {
        const int64_t reach = (64 / p.group + 2) * s.first + (p.group > 1 ? p.group * s.second : 0);
        far = reach > far ? reach : far;
    }
    return far >= most || p.d < Tile<T>::E;
}
template <typename T, int D>
int attn_mode(const AttnArgs& p) {
    return attn_any<T>(p) ? ANY : p.d == pitch_of(D) ? WHOLE : p.d % Tile<T>::E == 0 ? EVEN : PART;
}

template <typename T, int D>
AttnPlan plan_at(const AttnArgs& p) {
    typedef AttnShape<T, D> S;
    AttnPlan a{};
    const int64_t problems = (int64_t)p.batch * p.kv_heads, rows = (int64_t)p.nq * p.group;
    const size_t row_part = (size_t)problems * rows * pitch_of(D) * 4;
    const size_t key_part = (size_t)problems * p.nk * pitch_of(D) * 4;
    // Few rows: the waves share out the keys and meet at the end alone.  On one GPU, by this kernel and by that of blocks:
    // float32, 5 rows on 500k keys of 4 heads of 64 206 and 321 us, of 128 363 and 592; bfloat16, 8 rows on 1M keys of 8
    // heads of 32 234 and 248, 32 rows, where the rule ends, 241 and 248; 8 on 20k of 4 of 64 14.7 and 15.1, 32 on 20k
    // 16.0 and 15.5; 1 on 256 of 8 of 64 9.3 and 9.4.  Long bfloat16 keys of wider heads are slower by it: 8 on 1M of 4
    // of 64 210 and 180, on 500k of 4 of 128 210 and 190.
    a.few = rows <= 16 ? 1 : rows <= 32 ? 2 : 0;
    a.fwd_qc = rows <= 64 * S::kFwd / 2 ? 1 : S::kFwd;
    a.dq_qc = rows <= 64 * S::kDq / 2 ? 1 : S::kDq;
    a.dkv_kc = p.nk <= 64 * S::kDkv / 2 ? 1 : S::kDkv;
    if (a.few) split(p.nk, problems, 1024, 512, 4 * FewTile<T, D>::kKeys, a.fwd_splits, a.fwd_per);
    else split(p.nk, problems * tiles_of(rows, 64 * a.fwd_qc), 512, 512, AttnTile<T, D>::kRows, a.fwd_splits, a.fwd_per);
    // Few keys and rows for two tiles a wave: blocks that keep the keys.  1M rows (64M / keys if that is less) of 4 heads,
    // by this kernel and by blocks of a tile of rows each, us: bfloat16 of 32, 16 keys 127 and 187, 64 126 and 200, 128
    // 88 and 105, 256 72 and 82, 512, where LDS ends it, 65 and 71; of 64, 16 203 and 219, 64 199 and 232, 256 102 and
    // 106; of 128, 64 414 and 421, 128 241 and 274; float32 of 32, 16 198 and 222, 64 349 and 346, 128 327 and 318, 256
    // 310 and 298.  Twice the blocks: 16 keys of 32 120 for 127, 64 129 for 126, the others within 4%.
    const int64_t key_tiles = tiles_of(p.nk, AttnTile<T, D>::kRows);
    if (!a.few && a.fwd_splits == 1 && key_tiles <= kThinTiles && key_tiles * 2 * AttnTile<T, D>::kBytes <= kThinBytes) {
        while (a.together < 2 && p.kv_heads % (2 << a.together) == 0 &&
               (key_tiles * 4 * AttnTile<T, D>::kBytes << a.together) <= kThinBytes)
            ++a.together;
        const int64_t blocks = tiles_of(rows, 64 * S::kThin >> a.together);
        const int64_t each = tiles_of(kThinBlocks, problems >> a.together);
        if (blocks >= 2 * each) a.thin = (int)each;
    }
    split(p.nk, problems * tiles_of(rows, 64 * a.dq_qc), 512, 256, AttnTile<T, D>::kRows, a.dq_splits, a.dq_per);
    // 512 blocks are two a CU, what LDS and registers hold: more splits are more to join
    split(rows, problems * tiles_of(p.nk, 64 * a.dkv_kc), 512, 256, AttnTile<T, D>::kRows, a.dkv_splits, a.dkv_per);
    // The backward of few rows in one pass over the keys, with the forward: 8 rows on 1M keys of 8 heads of 32 bfloat16
    // 839 us, by dq's and dkv's kernels 1135; on 200k of 4 of 64 162 and 180, 32 rows 176 and 186, 20k keys 34 and 41
    // (8 rows) and 39 and 43 (32); of 32 float32 149 and 249.
    a.few_back = a.few == 2 && sizeof(T) == 4 && D > 128 ? 0 : a.few;  // their tiles fill LDS
    // Heads of at most a line of memory: a wave each.  The first of these 839 us against 887 with a block a head, 200k of
    // 4 of 64 162 against 169, of 32 float32 149 against 166, near the rule's end 70k of 32 bfloat16 40 against 36; of
    // 128 326 against 335, and its tiles in LDS leave room for less
    if (D * sizeof(T) <= 128 && p.nk >= kHeadsApart)
        while (a.few_heads < 2 && p.kv_heads % (2 << a.few_heads) == 0) ++a.few_heads;
    split(p.nk, problems >> a.few_heads, 1024, 64 * (4 >> a.few_heads), Tile<T>::KS * (4 >> a.few_heads),
          a.few_splits, a.few_per);
    // Few keys: both kernels' work in one pass over the rows.  With the forward, 4 heads, by this kernel and by dq's and
    // dkv's, us at 64, 96 and 128 keys: bfloat16, 1M rows of 32 444 and 596, 606 and 687, 590 and 715; 300k of 64 199
    // and 301, 375 and 347, 365 and 361; 100k of 128 171 and 233, 219 and 276, 223 and 277; float32, 500k of 32 627 and
    // 842, 1274 and 1236, 1367 and 1361; 200k of 64 479 and 670, 880 and 944, 952 and 1057.  100k on 256 of 64 bfloat16
    // 468 against 377, so it stops at 128 keys.  Twice the blocks: 64 keys of 32 433 for 444, of 128 195 for 171.
    a.held = p.nk < 1 || a.few_back ? 0 : p.nk <= 64 ? 1 : p.nk <= 128 ? 2 : 0;
    if (a.held > S::kHeld) a.held = 0;
    split(rows, problems, 512, 4 * AttnTile<T, D>::kRows, AttnTile<T, D>::kRows, a.held_splits, a.held_per);
    if (a.fwd_splits > 1)
        a.fwd_bytes = padded(row_part * a.fwd_splits) + padded(row_part / pitch_of(D) * 2 * a.fwd_splits);
    a.delta_bytes = padded((size_t)problems * rows * 4);
    // dq's partials are joined before those of dk and dv are made
    size_t most = a.dq_splits > 1 ? padded(row_part * a.dq_splits) : 0;
    const size_t kv = a.dkv_splits > 1 ? padded(2 * key_part * a.dkv_splits) : 0;
    most = kv > most ? kv : most;
    const size_t few = a.few_back && a.few_splits > 1 ? padded(row_part * a.few_splits) : 0;
    most = few > most ? few : most;
    const size_t held = a.held && a.held_splits > 1 ? padded(2 * key_part * a.held_splits) : 0;
    most = held > most ? held : most;
    a.bwd_bytes = a.delta_bytes + most;
    return a;
}

// A kernel with a thread for every 4 of a row's columns and, with many splits, more of them to share the splits out.
#define GS_ATTN_SHARED(KERNEL, ROWS, ...)                                                                              \
    do {                                                                                                               \
        constexpr int kP = pitch_of(D), kMost = 1024 / kP, kFull = kMost < 16 ? kMost : 16;                            \
        const int64_t rows_ = (ROWS);                                                                                  \
        if (p.splits <= 2)                                                                                             \
            hipLaunchKernelGGL((KERNEL<T, kP, 1 __VA_ARGS__>), dim3((unsigned)tiles_of(rows_, kMost)), dim3(256), 0,   \
                               s, p);                                                                                  \
        else if (p.splits <= 16)                                                                                       \
            hipLaunchKernelGGL((KERNEL<T, kP, 4 __VA_ARGS__>), dim3((unsigned)tiles_of(rows_, kMost / 4)), dim3(256),  \
                               0, s, p);                                                                               \
        else                                                                                                           \
            hipLaunchKernelGGL((KERNEL<T, kP, kFull __VA_ARGS__>), dim3((unsigned)tiles_of(rows_, kMost / kFull)),     \
                               dim3(256), 0, s, p);                                                                    \
    } while (0)

// CALL of the columns that products take: between the powers of two one more, and 48 for float32, whose products are
// what takes the time.  Rows read as WHOLE and ANY take powers of two.
#define GS_ATTN_BY_HEAD(CALL, D_, ANY_)                                                    \
    ((D_) <= 32                             ? CALL<T, 32>                                  \
     : (D_) <= 48 && sizeof(T) == 4 && !(ANY_) ? CALL<T, sizeof(T) == 4 ? 48 : 64>         \
     : (D_) <= 64                           ? CALL<T, 64>                                  \
     : (D_) <= 96 && !(ANY_)                ? CALL<T, 96>                                  \
     : (D_) <= 128                          ? CALL<T, 128>                                 \
     : (D_) <= 192 && !(ANY_)               ? CALL<T, 192>                                 \
                                            : CALL<T, 256>)

}  // namespace gs
