// Forward of cross attention (attention.h).
#pragma once

#include "attention.h"

namespace gs {

// A forward's rows: the results, or those of a split.  o is relative to the reference m, which stays -infinity where no
// logit is above it: no key counts (l = 0, of a split 0 too), all logits are -infinity (0, -1) or some NaN (NaN).
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
                    *reinterpret_cast<f32x4*>(p.part + to * pitch_of(D) + KS * e + E * g + 4 * u) = o[c][e][u];
            if (g == 0) {
                p.part_stat[2 * to] = m[c];
                p.part_stat[2 * to + 1] = any && m[c] == -INFINITY && l[c] == 0.f ? -1.f : l[c];
            }
            continue;
        }
        const Row w(p, at.hk, row, true);
        const bool empty = !any || row >= live;
        const float inv = __builtin_amdgcn_rcpf(l[c]);
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
                empty || (m[c] == -INFINITY && l[c] == 0.f)
                    ? -INFINITY
                    : (m[c] + __builtin_amdgcn_logf(l[c]) - Softmax<T>::kShift) * kLn2;
    }
}

// The splits' results together: threads of 4 columns for a row, times SHARE that share out its splits; each weighs its
// sums by the split's reference.  In a fixed order, so that results repeat.  Bound by the latency of two rounds of loads:
// 64 rows of 32 from 126 splits 7 us of the 236 of 8 rows on 1M keys.
template <typename T, int D, int SHARE>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p) {
    constexpr int kWide = D / 4, kRows = 256 / (kWide * SHARE);
    __shared__ f32x4 s_sum[256];
    __shared__ float s_l[256], s_m[256];
    const int col = threadIdx.x % kWide, share = threadIdx.x / kWide % SHARE, in = threadIdx.x / (kWide * SHARE);
    const int rows = p.nq * p.group;
    const int64_t at = (int64_t)blockIdx.x * kRows + in, total = (int64_t)p.batch * p.kv_heads * rows;
    const int64_t problem = at < total ? at / rows : 0;
    const int row = at < total ? (int)(at - problem * rows) : 0;
    const float* stat = p.part_stat + 2 * (problem * p.splits * rows + row);
    const float* part = p.part + (problem * p.splits * rows + row) * D + 4 * col;
    float m = -INFINITY;
#pragma unroll 4
    for (int i = threadIdx.x % (kWide * SHARE); i < p.splits; i += kWide * SHARE)
        m = fmaxf(m, stat[(int64_t)2 * rows * i]);
    s_m[threadIdx.x] = m;
    __syncthreads();
    for (int o = kWide * SHARE / 2; o > 0; o >>= 1) {
        if (threadIdx.x % (kWide * SHARE) < o) s_m[threadIdx.x] = fmaxf(s_m[threadIdx.x], s_m[threadIdx.x + o]);
        __syncthreads();
    }
    m = s_m[in * (kWide * SHARE)];
    f32x4 sum = {};
    float l = 0.f;
#pragma unroll 4
    for (int i = share; i < p.splits; i += SHARE) {
        const float mi = stat[(int64_t)2 * rows * i], li = stat[(int64_t)2 * rows * i + 1];
        const float w = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mi - m);
        const f32x4 o = *reinterpret_cast<const f32x4*>(part + (int64_t)rows * D * i);
        l = fmaf(w, li, l);
        sum += o * w;
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
    const bool empty = row >= live_rows(p, b) || (m == -INFINITY && l == 0.f);
    const float inv = m == -INFINITY ? NAN : __builtin_amdgcn_rcpf(l);
    T* out = static_cast<T*>(p.out) + w.whole(p, b) * p.d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (4 * col + j < p.d) out[4 * col + j] = empty ? (T)0.f : (T)(sum[j] * inv);
    if (p.lse && col == 0)
        p.lse[w.stat(p, b)] =
            empty || (m == -INFINITY && l < 0.f) ? -INFINITY
                                                 : (m + __builtin_amdgcn_logf(l) - Softmax<T>::kShift) * kLn2;
}

// What a wave's rows have come to: sums relative to a reference, which trails the maximum.  Whether it has to move is
// seen from the weights themselves: the lane's sum of a step's weights, which is needed anyway, passes a limit if one
// of them does (a maximum of the logits for every step would be a sixth of the arithmetic).  The sums are of the weights
// before they are rounded: lse is float32's.
template <typename T, int D, int QC>
struct RowState {
    static constexpr int TG = Tile<T>::TG, E = Tile<T>::E;
    typedef typename Tile<T>::Frag Frag;
    f32x4 o[QC][AttnTile<T, D>::kPairs][TG];
    float l[QC];    // the lane's part of the weights' sum, before they are rounded (a product with ones would sum after)
    float ref[QC];  // what logits are relative to, less kShift; 0 until a key counts
    float most[QC]; // of a step's weights, or -1 until a key counts
    float c2;

    __device__ __forceinline__ explicit RowState(float scale) : o{}, c2(fabsf(scale) * kLog2e) {
#pragma unroll
        for (int c = 0; c < QC; ++c) l[c] = 0.f, ref[c] = 0.f, most[c] = -1.f;
    }
    __device__ __forceinline__ float reference(int c) const {
        return most[c] < 0.f ? -INFINITY : ref[c] + Softmax<T>::kShift;
    }
    // takes the highest logit of a step for the reference, where that is higher
    __device__ __forceinline__ void move(const f32x4 (&s)[QC][TG]) {
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            float top = s[c][0][0];
#pragma unroll
            for (int j = 1; j < E; ++j) top = fmaxf(top, s[c][j >> 2][j & 3]);
            const float old = reference(c), next = fmaxf(highest(top) * c2, old);
            if (next == -INFINITY) continue;  // none above it yet
            const float by = __builtin_amdgcn_exp2f(old - next);
            ref[c] = next - Softmax<T>::kShift;
            most[c] = Softmax<T>::kMost;
            l[c] *= by;
#pragma unroll
            for (int p = 0; p < AttnTile<T, D>::kPairs; ++p)
#pragma unroll
                for (int u = 0; u < TG; ++u) o[c][p][u] *= by;
        }
    }
    // the weights of KS keys from their logits, as the next product's fragment; first: of the wave's first keys
    __device__ __forceinline__ void weigh(const f32x4 (&s)[QC][TG], Frag (&w)[QC], bool first) {
        float e[QC][E], sum[QC];
        auto weights = [&]() {
            bool over = false;
#pragma unroll
            for (int c = 0; c < QC; ++c) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    e[c][j] = __builtin_amdgcn_exp2f(fmaf(s[c][j >> 2][j & 3], c2, -ref[c]));
                    sum[c] = j == 0 ? e[c][0] : sum[c] + e[c][j];
                }
                over |= sum[c] > most[c];
            }
            return over;
        };
        if (first) move(s);
        if (__any(weights())) {
            move(s);
            weights();
        }
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            l[c] += sum[c];
#pragma unroll
            for (int j = 0; j < E; ++j) w[c][j] = (T)e[c][j];
        }
    }
    // o += w v, values in a tile of LDS from row m0 on
    __device__ __forceinline__ void add(const char* tile, int m0, const Frag (&w)[QC], int lane) {
#pragma unroll
        for (int e = 0; e < AttnTile<T, D>::kPairs; ++e)
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const Frag a = down_frag<T, D>(tile, m0, e, u, lane);
#pragma unroll
                for (int c = 0; c < QC; ++c) mma(o[c][e][u], a, w[c]);
            }
    }
    __device__ __forceinline__ float sum(int c) const { return added(l[c]); }
};

// Logits of keys that do not count.  bits: the group's, from its first key on.
template <typename T, int QC>
__device__ __forceinline__ void without(f32x4 (&s)[QC][Tile<T>::TG], uint64_t bits, int g) {
#pragma unroll
    for (int u = 0; u < Tile<T>::TG; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = bits >> (Tile<T>::E * g + 4 * u + j) & 1;
#pragma unroll
            for (int c = 0; c < QC; ++c) s[c][u][j] = in ? s[c][u][j] : -INFINITY;
        }
}

// Forward of few rows: 16 QC of them with all keys of a split, which the four waves of a block share out in tiles of
// their own.  A wave reads keys and values from memory as fragments, values through LDS of its own to turn them, and
// nothing but the end waits for another wave: what bounds it is the stream of keys and values.  8 rows on 1M keys of 8
// heads of 32 bfloat16: 230 us, 4.45 TB/s, of a copy's 5.24; one row on 256 keys of 8 heads of 64 7.4, of which a
// launch is 4.
template <typename T, int D, int QC, int MODE>
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
    char* tv = s_mem + wave * F::kBytes;

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
                const int in = min(kg * KS + out_row<T>(u, r), last - k0);
                if constexpr (MODE == ANY) {
                    raw_frags<T, MODE>(k[kg][u], k_base + (int64_t)(k0 + in) * p.k_n, g, p.d);
                    raw_frags<T, MODE>(v[kg][u], v_base + (int64_t)(k0 + in) * p.v_n, g, p.d);
                } else {
                    raw_frags<T, MODE>(k[kg][u], k_base + k0 * p.k_n + (uint32_t)in * (uint32_t)p.k_n, g, p.d);
                    raw_frags<T, MODE>(v[kg][u], v_base + k0 * p.v_n + (uint32_t)in * (uint32_t)p.v_n, g, p.d);
                }
            }
    };
    int k0 = first + wave * KW;
    if (live == 0) k0 = keys.count;
    if (k0 < keys.count) fetch(k0);
    Frag q[QC][A::kSteps];
    rows_held<T, MODE>(p, at.b, at.hk, 0, live, p.q, p.q_b, p.q_n, p.q_h, p.scale < 0.f, lane, q);
    RowState<T, D, QC> rows(p.scale);
    bool first_keys = true;
    uint64_t any = 0;
    for (; k0 < keys.count; k0 += 4 * KW) {
        const uint64_t valid = __ballot(byte != 0);
        any |= valid;
        f32x4 s[KG][QC][TG] = {};
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                fix_frags<T, MODE>(k[kg][u], g, p.d, true);
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e)
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(s[kg][c][u], k[kg][u][e], q[c][e]);
                const int row = kg * KS + out_row<T>(u, r);
                fix_frags<T, MODE>(v[kg][u], g, p.d, valid >> row & 1);
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e)
                    *reinterpret_cast<Frag*>(tv + tile_at<T, D>(row, 4 * e + g)) = v[kg][u][e];
            }
        if (k0 + 4 * KW < keys.count) fetch(k0 + 4 * KW);
        wave_sync();
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
            if (!group_counts<T>(valid, kg)) continue;
            if (valid != ~0ull >> (64 - KW)) without<T, QC>(s[kg], valid >> (kg * KS), g);
            Frag w[QC];
            rows.weigh(s[kg], w, first_keys);
            first_keys = false;
            rows.add(tv, kg * KS, w, lane);
        }
        wave_sync();
    }
    // the waves' results together, in their order
    float sum[QC], top[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const float own = rows.sum(c);
        if (g == 0) s_m[wave][16 * c + r] = rows.reference(c), s_l[wave][16 * c + r] = own;
    }
    const bool some = __syncthreads_or(any != 0);
    float* s_o = reinterpret_cast<float*>(s_mem);  // [16 QC][D]
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = 16 * c + r;
        const float m = rows.reference(c);
        top[c] = fmaxf(fmaxf(s_m[0][row], s_m[1][row]), fmaxf(s_m[2][row], s_m[3][row]));
        sum[c] = 0.f;
        for (int i = 0; i < 4; ++i)
            sum[c] = fmaf(top[c] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(s_m[i][row] - top[c]), s_l[i][row], sum[c]);
        const float by = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top[c]);
#pragma unroll
        for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
            for (int u = 0; u < TG; ++u) rows.o[c][e][u] *= by;
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
                        if (i > 0) rows.o[c][e][u] += *to;
                        if (i < 3) *to = rows.o[c][e][u];
                    }
        }
        __syncthreads();
    }
    if (wave == 3) forward_rows<T, D, QC>(p, at, 0, live, some, top, sum, rows.o, lane);
}

// Forward over tiles of 64 QC rows and the keys of a split: two buffers of keys and values in LDS, the next tile's loads
// in flight while a tile is worked on, one barrier a tile.  Bound by the issue of vector instructions at heads of 64 and
// less (exp, sums and roundings of the weights: 8 an element): 100k rows on 1024 keys, 8 heads of 64 to 2 of keys, bfloat16 249
// us, 840 TFLOP/s; by matrix instructions, LDS and vector instructions taking turns at two waves a SIMD above: 64k on
// 1024 of 4 of 128 172 us, 800 TFLOP/s.
template <typename T, int D, int QC, int MODE>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOccFwd)) void k_attn_fwd(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int KS = Tile<T>::KS, TG = Tile<T>::TG, KT = A::kRows, NG = A::kGroups;
    __shared__ __align__(16) char s_k[2][A::kBytes], s_v[2][A::kBytes];
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Keys keys(p, at.b);
    const int first = at.split * p.per;
    KeyTiles<T, D, MODE, direct(MODE)> tile_k(p.k, at.b * p.k_b + at.hk * p.k_h, p.k_n, keys.count, p.d);
    KeyTiles<T, D, MODE, direct(MODE)> tile_v(p.v, at.b * p.v_b + at.hk * p.v_h, p.v_n, keys.count, p.d);
    keys.until(first + p.per);
    const int live = live_rows(p, at.b);
    const int row0 = (at.tile * 4 + wave) * 16 * QC;
    const int tiles = live > at.tile * 64 * QC ? (keys.count - first + KT - 1) / KT : 0;
    uint64_t valid = 0, any = 0;
    int byte = 0;
    for (char* t : {s_k[0], s_k[1], s_v[0], s_v[1]}) tile_k.move.blank(t, p.d);
    if (tiles > 0) {
        byte = keys.byte(first, lane);
        tile_k.load(first, p.d, s_k[0]);
        tile_v.load(first, p.d, s_v[0]);
    }
    Frag q[QC][A::kSteps];
    rows_held<T, MODE>(p, at.b, at.hk, row0, live, p.q, p.q_b, p.q_n, p.q_h, p.scale < 0.f, lane, q);
    RowState<T, D, QC> rows(p.scale);
    bool first_keys = true;
    if (tiles > 0) {
        valid = key_bits<KT>(byte);
        tile_k.move.place(s_k[0], valid, p.d);
        tile_v.move.place(s_v[0], valid, p.d);
    }
    for (int t = 0; t < tiles; ++t) {
        __syncthreads();
        if (t + 1 < tiles) {
            const int next = first + (t + 1) * KT;
            byte = keys.byte(next, lane);
            tile_k.load(next, p.d, s_k[(t + 1) & 1]);
            tile_v.load(next, p.d, s_v[(t + 1) & 1]);
        }
        const char* tk = s_k[t & 1];
        const char* tv = s_v[t & 1];
        any |= valid;
#pragma unroll
        for (int kg = 0; kg < NG; ++kg) {
            if (!group_counts<T>(valid, kg)) continue;
            f32x4 s[QC][TG] = {};
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) {
                    const Frag a = row_frag<T, D>(tk, kg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                    for (int c = 0; c < QC; ++c) mma(s[c][u], a, q[c][e]);
                }
            if (valid != ~0ull >> (64 - KT)) without<T, QC>(s, valid >> (kg * KS), g);
            Frag w[QC];
            rows.weigh(s, w, first_keys);
            first_keys = false;
            rows.add(tv, kg * KS, w, lane);
        }
        if (t + 1 < tiles) {
            valid = key_bits<KT>(byte);
            tile_k.move.place(s_k[(t + 1) & 1], valid, p.d);
            tile_v.move.place(s_v[(t + 1) & 1], valid, p.d);
        }
    }
    float m[QC], l[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) m[c] = rows.reference(c), l[c] = rows.sum(c);
    forward_rows<T, D, QC>(p, at, row0, live, any != 0, m, l, rows.o, lane);
}

// Forward of many rows on few keys: the keys and values of a problem stay in LDS for the life of a block, and each
// wave walks tiles of 16 QC rows with the next tile's queries in flight and no barrier.  1M rows on 64 keys of 4 heads of
// 32 float16: 127 us, 4.05 TB/s of rows, beside 60 us of vector instructions.
template <typename T, int D, int QC, int MODE>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOccThin)) void k_attn_thin(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, KT = A::kRows, NG = A::kGroups;
    extern __shared__ __align__(16) char s_mem[];  // [tiles of keys][keys, values]
    __shared__ uint64_t s_valid[kThinTiles];
    Place at(p, p.together);  // tile: the block's share of the rows
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Keys keys(p, at.b);
    const int rows = p.nq * p.group, live = live_rows(p, at.b);
    // the waves of a block take the same rows of its heads, which are neighbours in memory
    const int heads = 1 << p.together, step = p.tiles * (64 * QC >> p.together);
    int row0 = (at.tile * (4 >> p.together) + (wave >> p.together)) * 16 * QC;
    const int own = wave & (heads - 1), first_head = at.hk;
    at.hk += own;
    const T* q_base = static_cast<const T*>(p.q) + at.b * p.q_b;
    // one head for each head of keys: a lane's places in a whole tile of rows are the same from tile to tile
    const uint32_t out_n = (uint32_t)(p.heads * p.d);
    uint32_t q_at[QC], out_at[QC];
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        q_at[c] = (uint32_t)(16 * c + r) * (uint32_t)p.q_n;
        out_at[c] = (uint32_t)(16 * c + r) * out_n;
    }
    Frag next[QC][A::kSteps];
    auto fetch = [&](int from) {
        if (p.group == 1 && from + 16 * QC <= live) {
            const T* tile = q_base + from * p.q_n + at.hk * p.q_h;
#pragma unroll
            for (int c = 0; c < QC; ++c) raw_frags<T, MODE>(next[c], tile + q_at[c], g, p.d);
            return;
        }
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            const Row w(p, at.hk, from + 16 * c + r, from + 16 * c + r < live);
            raw_frags<T, MODE>(next[c], q_base + w.query * p.q_n + w.head * p.q_h, g, p.d);
        }
    };
    fetch(row0);
    const int tiles = (keys.count + KT - 1) / KT;
    uint64_t any = 0;
    for (int h = 0; h < heads; ++h) {
        KeyTiles<T, D, MODE> tile_k(p.k, at.b * p.k_b + (first_head + h) * p.k_h, p.k_n, keys.count, p.d);
        KeyTiles<T, D, MODE> tile_v(p.v, at.b * p.v_b + (first_head + h) * p.v_h, p.v_n, keys.count, p.d);
        char* to = s_mem + 2 * h * tiles * A::kBytes;
        for (int t = 0; t < tiles; ++t) {
            const int byte = keys.byte(t * KT, lane);
            tile_k.load(t * KT, p.d, nullptr);
            tile_v.load(t * KT, p.d, nullptr);
            const uint64_t valid = key_bits<KT>(byte);
            any |= valid;
            tile_k.move.place(to + 2 * t * A::kBytes, valid, p.d);
            tile_v.move.place(to + (2 * t + 1) * A::kBytes, valid, p.d);
            if (threadIdx.x == 0) s_valid[t] = valid;
        }
    }
    __syncthreads();
    for (; row0 < rows; row0 += step) {
        Frag q[QC][A::kSteps];
#pragma unroll
        for (int c = 0; c < QC; ++c) {
#pragma unroll
            for (int e = 0; e < A::kSteps; ++e) q[c][e] = next[c][e];
            fix_frags<T, MODE>(q[c], g, p.d, row0 + 16 * c + r < live);
            if (p.scale < 0.f)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) q[c][e] = -q[c][e];
        }
        if (row0 + step < rows) fetch(row0 + step);
        RowState<T, D, QC> state(p.scale);
        bool first_keys = true;
        for (int t = 0; t < tiles; ++t) {
            const char* tk = s_mem + 2 * (own * tiles + t) * A::kBytes;
            const char* tv = tk + A::kBytes;
            const uint64_t valid = s_valid[t];
#pragma unroll
            for (int kg = 0; kg < NG; ++kg) {
                if (!group_counts<T>(valid, kg)) continue;
                f32x4 s[QC][TG] = {};
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int e = 0; e < A::kSteps; ++e) {
                        const Frag a = row_frag<T, D>(tk, kg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                        for (int c = 0; c < QC; ++c) mma(s[c][u], a, q[c][e]);
                    }
                if (valid != ~0ull >> (64 - KT)) without<T, QC>(s, valid >> (kg * KS), g);
                Frag w[QC];
                state.weigh(s, w, first_keys);
                first_keys = false;
                state.add(tv, kg * KS, w, lane);
            }
        }
        float m[QC], l[QC];
#pragma unroll
        for (int c = 0; c < QC; ++c) m[c] = state.reference(c), l[c] = state.sum(c);
        if (!(p.group == 1 && row0 + 16 * QC <= live && any) || p.lse) {
            forward_rows<T, D, QC>(p, at, row0, live, any != 0, m, l, state.o, lane);
            continue;
        }
        T* out = static_cast<T*>(p.out) + ((int64_t)at.b * p.nq + row0) * out_n + at.hk * p.d;
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            const float inv = __builtin_amdgcn_rcpf(l[c]);
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e) {
                Frag f;
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[4 * u + j] = (T)(state.o[c][e][u][j] * inv);
                store_run(out + out_at[c], KS * e + E * g, p.d, f);
            }
        }
    }
}

template <typename T, int D, int MODE>
void attn_fwd_in(AttnArgs p, void* workspace, hipStream_t s) {
    const AttnPlan a = plan_at<T, D>(p);
    constexpr int kFew = MODE == ANY ? 1 : 2, kQc = MODE == ANY ? 1 : AttnShape<T, D>::kFwd;
    const int64_t rows = (int64_t)p.nq * p.group, problems = (int64_t)p.batch * p.kv_heads;
    p.splits = a.fwd_splits, p.per = a.fwd_per;
    p.part = static_cast<float*>(workspace);
    if (p.splits > 1) p.part_stat = p.part + padded((size_t)problems * rows * pitch_of(D) * 4 * p.splits) / 4;
    if (a.few && a.few <= kFew) {
        p.tiles = 1;
        if (a.few == 1) hipLaunchKernelGGL((k_attn_few<T, D, 1, MODE>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_few<T, D, kFew, MODE>), grid_of(p), dim3(256), 0, s, p);
    } else if (a.thin && MODE != ANY) {
        constexpr int kThin = AttnShape<T, D>::kThin;
        p.tiles = a.thin, p.together = a.together;
        const int64_t lds = tiles_of(p.nk, AttnTile<T, D>::kRows) * 2 * AttnTile<T, D>::kBytes << a.together;
        hipLaunchKernelGGL((k_attn_thin<T, D, kThin, MODE == ANY ? PART : MODE>), grid_of(p), dim3(256), (unsigned)lds, s,
                           p);
    } else {
        const int qc = a.fwd_qc < kQc ? a.fwd_qc : kQc;
        p.tiles = (int32_t)tiles_of(rows, 64 * qc);
        if (qc == 1) hipLaunchKernelGGL((k_attn_fwd<T, D, 1, MODE>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_fwd<T, D, kQc, MODE>), grid_of(p), dim3(256), 0, s, p);
    }
    if (p.splits > 1) GS_ATTN_SHARED(k_attn_join, problems * rows);
}

template <typename T, int D>
void attn_fwd_at(const AttnArgs& p, void* workspace, hipStream_t s) {
    const int mode = attn_mode<T, D>(p);
    if constexpr (D == pitch_of(D)) {
        if (mode == WHOLE) attn_fwd_in<T, D, WHOLE>(p, workspace, s);
        else if (mode == ANY) attn_fwd_in<T, D, ANY>(p, workspace, s);
    }
    if (mode == EVEN) attn_fwd_in<T, D, EVEN>(p, workspace, s);
    else if (mode == PART) attn_fwd_in<T, D, PART>(p, workspace, s);
}

// Bytes of workspace, by sizes alone: what either way to read the rows asks for.
template <typename T>
AttnBytes attn_bytes(const AttnArgs& p) {
    const AttnPlan a = GS_ATTN_BY_HEAD(plan_at, p.d, false)(p), b = GS_ATTN_BY_HEAD(plan_at, p.d, true)(p);
    return AttnBytes{a.fwd_bytes > b.fwd_bytes ? a.fwd_bytes : b.fwd_bytes,
                     a.bwd_bytes > b.bwd_bytes ? a.bwd_bytes : b.bwd_bytes};
}
template <typename T>
void attn_fwd(const AttnArgs& p, void* workspace, hipStream_t s) {
    GS_ATTN_BY_HEAD(attn_fwd_at, p.d, attn_any<T>(p))(p, workspace, s);
}

}  // namespace gs
