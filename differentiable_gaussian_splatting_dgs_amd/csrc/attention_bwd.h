// Gradients of cross attention (attention.h).
#pragma once

#include "attention.h"

namespace gs {

// Sums of the splits' gradients, rows of dq (KEYS false) or of dk and dv, in a fixed order.  Bound by memory: 64 MB of
// partial results (4 splits of dk and dv of 1024 keys of 128) in 12 us.
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

// Gradients.  With P = exp(s - lse) and ds = P (dout v^T - delta), delta the row's sum of dout * out:
// dq = scale ds k, dk = scale ds^T q, dv = P^T dout.  P and ds enter the products rounded to the type: the matrix
// instructions take no mixed operands, and twice the products would be 4 more beside 7.  That makes a 16-bit gradient's
// error sqrt(2) of what rounding the result alone makes it (float16, 1000 keys: 0.00029 for 0.00021).  Where the result's
// rounding enters delta, it moves all of a row's ds alike and takes dq along the mean key: 1.5 roundings at 180 keys and
// more whose mean is 0, 2.8 where it is 4/3 of their spread; dk and dv do not notice.  So k_attn_held, and k_attn_few_bwd
// where its waves have a tile of keys each, which have all keys at hand, sum P dP instead (8 rows on 4 keys, whose out
// is nearly one value, 1.5 for 2.1, with the mean 2.1 for 2.8, bfloat16 2.0 for 3.9).
// float16: both are held times 2^13; should a ds not fit then, ds are scaled down with what is summed of them so far
// (Shrink), and P stays as it is.
template <typename T>
struct Shrink {
    static constexpr bool kNeeded = false;
    static constexpr float kWeights = 0.f, shift = 0.f;  // powers of two of P and of ds
    static __device__ __forceinline__ bool moved() { return false; }
    template <typename Each, typename Over>
    __device__ __forceinline__ void operator()(Each, Over) {}
};
template <>
struct Shrink<_Float16> {
    static constexpr bool kNeeded = true;
    static constexpr float kWeights = 13.f;
    float shift = kWeights;
    // whether ds have another scale than P, the same in all lanes
    __device__ __forceinline__ bool moved() const {
        return __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, shift)) != __builtin_bit_cast(int, kWeights);
    }
    // each(f) calls f with the lane's ds of this step that count; over(f) scales what the wave holds of ds by f.
    // Infinities and NaN stay what they are, and what is beside them in a lane, of another row, is scaled to fit.
    template <typename Each, typename Over>
    __device__ __forceinline__ void operator()(Each each, Over over) {
        float most = 0.f;
        each([&](float v) { most = fmaxf(most, fabsf(v)); });
        if (!__any(most > 32768.f)) return;
        most = 0.f;
        each([&](float v) { most = fabsf(v) < INFINITY ? fmaxf(most, fabsf(v)) : most; });
        for (int o = 1; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
        const int by = most > 16384.f ? ilogbf(most) - 13 : 0;
        over(ldexpf(1.f, -by));
        shift -= (float)by;
    }
};

// dq over tiles of 64 QC rows and the keys of a split; leaves the rows' delta for the other gradients.  Three products a
// tile (s, dP, dq) and the forward's loop.  64k rows on 1024 keys of 4 heads of 128 bfloat16: 227 us, 910 TFLOP/s with s
// made again, a wave's fragments from LDS used twice; float32, 4 x 5003 on 333 of 40: 64 us, 120 TFLOP/s of the 48 columns that it takes.
template <typename T, int D, int QC, int MODE>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOccDq)) void k_attn_dq(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, KT = A::kRows, NG = A::kGroups;
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
    const int rows = p.nq * p.group, live = live_rows(p, at.b);
    const int row0 = (at.tile * 4 + wave) * 16 * QC;
    const float c2 = fabsf(p.scale) * kLog2e;
    const int tiles = p.dq && live > at.tile * 64 * QC ? (keys.count - first + KT - 1) / KT : 0;
    int byte = 0;
    for (char* t : {s_k[0], s_k[1], s_v[0], s_v[1]}) tile_k.move.blank(t, p.d);
    if (tiles > 0) {
        byte = keys.byte(first, lane);
        tile_k.load(first, p.d, s_k[0]);
        tile_v.load(first, p.d, s_v[0]);
    }

    Frag q[QC][A::kSteps], dout[QC][A::kSteps];
    float lse[QC], delta[QC];
    {
        Frag out[QC][A::kSteps];
        const int64_t row = p.d, query = row * p.heads;
        rows_held<T, MODE>(p, at.b, at.hk, row0, live, p.out, query * p.nq, query, row, false, lane, out);
        rows_held<T, MODE>(p, at.b, at.hk, row0, live, p.dout, p.g_b, p.g_n, p.g_h, false, lane, dout);
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            const bool in = row0 + 16 * c + r < live;
            const int64_t stat = Row(p, at.hk, row0 + 16 * c + r, in).stat(p, at.b);
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < E; ++j) sum = fmaf((float)dout[c][s][j], (float)out[c][s][j], sum);
            delta[c] = added(sum);
            lse[c] = in ? p.lse[stat] * kLog2e : 0.f;
            if (in && g == 0 && at.split == 0) p.delta[stat] = delta[c];
        }
    }
    rows_held<T, MODE>(p, at.b, at.hk, row0, live, p.q, p.q_b, p.q_n, p.q_h, p.scale < 0.f, lane, q);

    f32x4 dq[QC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    uint64_t valid = 0;
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
#pragma unroll
        for (int kg = 0; kg < NG; ++kg) {
            if (!group_counts<T>(valid, kg)) continue;
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
#pragma unroll
            for (int c = 0; c < QC; ++c) {
                const float ref = lse[c] - shrink.shift;
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float w = __builtin_amdgcn_exp2f(fmaf(s[c][u][j], c2, -ref));
                        s[c][u][j] = w * (dp[c][u][j] - delta[c]);
                    }
            }
            if (valid != ~0ull >> (64 - KT))
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = valid >> (kg * KS + E * g + 4 * u + j) & 1;
#pragma unroll
                        for (int c = 0; c < QC; ++c) s[c][u][j] = in ? s[c][u][j] : 0.f;
                    }
            auto each = [&](auto f) {
#pragma unroll
                for (int c = 0; c < QC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f(s[c][u][j]);
            };
            shrink(each, [&](float f) {
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
            tile_k.move.place(s_k[(t + 1) & 1], valid, p.d);
            tile_v.move.place(s_v[(t + 1) & 1], valid, p.d);
        }
    }
    if (!p.dq) return;
    const float by = p.scale * __builtin_amdgcn_exp2f(-shrink.shift);
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        const int row = row0 + 16 * c + r;
        if (row >= rows) continue;
        if (p.splits > 1) {
            float* to = p.part + (at.part(p, rows) + row) * pitch_of(D);
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

// The gradients of a lane's key: the results, or those of a split.
template <typename T, int D>
__device__ __forceinline__ void keys_out(const AttnArgs& p, const Place& at, int key, bool counts, float shift,
                                         const f32x4 (&dk)[AttnTile<T, D>::kPairs][Tile<T>::TG],
                                         const f32x4 (&dv)[AttnTile<T, D>::kPairs][Tile<T>::TG], int lane) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    const int g = lane >> 4;
    if (key >= p.nk) return;
    const float by_k = p.scale * __builtin_amdgcn_exp2f(-shift), by_v = __builtin_amdgcn_exp2f(-Shrink<T>::kWeights);
    if (p.splits > 1) {
        float* to = p.part + (at.part(p, p.nk) + key) * pitch_of(D);
        float* to_v = to + (int64_t)p.batch * p.kv_heads * p.splits * p.nk * pitch_of(D);
#pragma unroll
        for (int e = 0; e < AttnTile<T, D>::kPairs; ++e)
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const int k = KS * e + E * g + 4 * u;
                *reinterpret_cast<f32x4*>(to + k) = counts ? dk[e][u] * by_k : f32x4{};
                *reinterpret_cast<f32x4*>(to_v + k) = counts ? dv[e][u] * by_v : f32x4{};
            }
        return;
    }
    const int64_t row = (((int64_t)at.b * p.nk + key) * p.kv_heads + at.hk) * p.d;
#pragma unroll
    for (int e = 0; e < AttnTile<T, D>::kPairs; ++e) {
        typename Tile<T>::Frag a, b;
#pragma unroll
        for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[4 * u + j] = counts ? (T)(dk[e][u][j] * by_k) : (T)0.f;
                b[4 * u + j] = counts ? (T)(dv[e][u][j] * by_v) : (T)0.f;
            }
        if (p.dk) store_run(static_cast<T*>(p.dk) + row, KS * e + E * g, p.d, a);
        if (p.dv) store_run(static_cast<T*>(p.dv) + row, KS * e + E * g, p.d, b);
    }
}

// dk and dv over tiles of 64 KC keys and the rows of a split.  Here a lane holds consecutive rows of one key: s = q k^T.
// Four products a tile (s, dP, dv, dk).  64k rows on 1024 keys of 4 heads of 128 bfloat16: 388 us, 710 TFLOP/s: one
// wave a SIMD, so that exp and roundings wait for products and products for them (at two waves and one tile of keys
// LDS bounds it: the same time); float32, 4 x 5003 on 333 of 40: 115 us, 89 TFLOP/s of 48 columns.
template <typename T, int D, int KC, int MODE>
__global__ __launch_bounds__(256, (AttnShape<T, D>::kOccDkv)) void k_attn_dkv(AttnArgs p) {
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
    const float c2 = fabsf(p.scale) * kLog2e;
    const int tiles = keys.count > at.tile * 64 * KC ? (live - first + RT - 1) / RT : 0;
    RowTiles<T, D, MODE, direct(MODE)> tile_q(p, at.b, at.hk, p.q, p.q_b, p.q_n, p.q_h);
    RowTiles<T, D, MODE, direct(MODE)> tile_g(p, at.b, at.hk, p.dout, p.g_b, p.g_n, p.g_h);
    float next_lse = 0.f, next_delta = 0.f;
    auto fetch = [&](int row0, int buffer) {
        tile_q.load(p, row0, live, s_q[buffer]);
        tile_g.load(p, row0, live, s_g[buffer]);
        if (threadIdx.x < RT) {
            const int row = row0 + (int)threadIdx.x;
            const int64_t stat = Row(p, at.hk, row, row < live).stat(p, at.b);
            next_lse = p.lse[stat];
            next_delta = p.delta[stat];
        }
    };
    auto place = [&](int buffer, uint64_t valid) {
        tile_q.move.place(s_q[buffer], valid, p.d);
        tile_g.move.place(s_g[buffer], valid, p.d);
        if (threadIdx.x < RT)
            s_lse[buffer][threadIdx.x] = next_lse * kLog2e, s_delta[buffer][threadIdx.x] = next_delta;
    };
    for (char* t : {s_q[0], s_q[1], s_g[0], s_g[1]}) tile_q.move.blank(t, p.d);
    // the tile's rows that count
    auto bits = [&](int row0) { return ~0ull >> (64 - min(RT, live - row0)); };
    if (tiles > 0) fetch(first, 0);

    Frag k[KC][A::kSteps], v[KC][A::kSteps];
    bool counts[KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int key = key0 + 16 * c + r;
        counts[c] = key < keys.count && (!keys.mask || keys.mask[key]);
        const int64_t from = counts[c] ? key : 0;
        {
            raw_frags<T, MODE>(k[c], static_cast<const T*>(p.k) + at.b * p.k_b + from * p.k_n + at.hk * p.k_h, g, p.d);
            raw_frags<T, MODE>(v[c], static_cast<const T*>(p.v) + at.b * p.v_b + from * p.v_n + at.hk * p.v_h, g, p.d);
        }
    }
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        fix_frags<T, MODE>(k[c], g, p.d, counts[c]);
        fix_frags<T, MODE>(v[c], g, p.d, counts[c]);
        if (p.scale < 0.f)
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s) k[c][s] = -k[c][s];
    }

    f32x4 dk[KC][A::kPairs][TG] = {}, dv[KC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    uint64_t valid = 0;
    if (tiles > 0) {
        valid = bits(first);
        place(0, valid);
    }
    for (int t = 0; t < tiles; ++t) {
        __syncthreads();
        if (t + 1 < tiles) fetch(first + (t + 1) * RT, (t + 1) & 1);
        const char* tq = s_q[t & 1];
        const char* tg = s_g[t & 1];
#pragma unroll
        for (int rg = 0; rg < NG; ++rg) {
            if (!group_counts<T>(valid, rg)) continue;
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
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const f32x4 lse = *reinterpret_cast<const f32x4*>(&s_lse[t & 1][rg * KS + E * g + 4 * u]);
                const f32x4 delta = *reinterpret_cast<const f32x4*>(&s_delta[t & 1][rg * KS + E * g + 4 * u]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const float w = __builtin_amdgcn_exp2f(fmaf(s[c][u][j], c2, Shrink<T>::kWeights - lse[j]));
                        s[c][u][j] = w;
                        dp[c][u][j] = w * (dp[c][u][j] - delta[j]);
                    }
            }
            if (shrink.moved()) {
                const float f = __builtin_amdgcn_exp2f(shrink.shift - Shrink<T>::kWeights);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u) dp[c][u] *= f;
            }
            if (valid != ~0ull >> (64 - RT))
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = valid >> (rg * KS + E * g + 4 * u + j) & 1;
#pragma unroll
                        for (int c = 0; c < KC; ++c) {
                            s[c][u][j] = in ? s[c][u][j] : 0.f;
                            dp[c][u][j] = in ? dp[c][u][j] : 0.f;
                        }
                    }
            auto each = [&](auto f) {  // keys that do not count have weights that mean nothing
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f(counts[c] ? dp[c][u][j] : 0.f);
            };
            shrink(each, [&](float f) {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
#pragma unroll
                    for (int u = 0; u < TG; ++u) dp[c][u] *= f;
#pragma unroll
                    for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                        for (int u = 0; u < TG; ++u) dk[c][e][u] *= f;
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
#pragma unroll
    for (int c = 0; c < KC; ++c) keys_out<T, D>(p, at, key0 + 16 * c + r, counts[c], shrink.shift, dk[c], dv[c], lane);
}

// Columns [c0, c0 + 16) of keys [m0, m0 + KS) of a tile of keys down and RT rows across: lane (r, g) has row c0 + r,
// keys m0 + E g on.
template <typename T, int RT>
__device__ __forceinline__ typename Tile<T>::Frag across_frag(const char* tile, int m0, int c0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
        union {
            typename Tile<T>::Frag f;
            s16x4 h[2];
        } u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = m0 + 8 * g + 4 * h + (r >> 2), c = c0 + 4 * (r & 3);
            u.h[h] = read_transposed(tile + tile_at<T, RT>(m, c >> 3) + (c & 7) * 2);
        }
        return u.f;
    } else {
        typename Tile<T>::Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = *reinterpret_cast<const float*>(tile + tile_at<T, RT>(m0 + 4 * g + j, (c0 + r) >> 2) + (r & 3) * 4);
        return f;
    }
}

// The gradients where a block holds all keys of a problem (64 KC of them at most), 16 KC a wave, and walks the rows of
// its split.  ds goes through LDS, keys down and rows across, and comes back as the fragments of dq: s, P and ds are
// made once, q and dout are read once and dq is written once.  delta is the sum of P dP over all keys, which the waves
// exchange in LDS: so out is not read, and its rounding is not in it.  1M rows on 64 keys of 4 heads of 32 bfloat16, with
// the forward: 446 us, where its rows alone ask for 195; bound by vector instructions and the barriers of a tile.
template <typename T, int D, int KC>
struct HeldTile {
    static constexpr int kRows = AttnTile<T, D>::kRows, kKeys = 64 * KC;
    static constexpr int kDs = kKeys * kRows * (int)sizeof(T), kKeyBytes = kKeys * pitch_of(D) * (int)sizeof(T);
    static constexpr int kBytes = 2 * AttnTile<T, D>::kBytes + kDs + kKeyBytes + 5 * kRows * 4;
};

template <typename T, int D, int KC, int MODE>
__global__ __launch_bounds__(256, (AttnShape<T, D>::occ_held(KC))) void k_attn_held(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef HeldTile<T, D, KC> H;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, RT = A::kRows, NG = A::kGroups;
    extern __shared__ __align__(16) char s_mem[];
    char *s_q = s_mem, *s_g = s_q + A::kBytes, *s_k = s_g + A::kBytes, *s_ds = s_k + H::kKeyBytes;
    float *s_lse = reinterpret_cast<float*>(s_ds + H::kDs), *s_sum = s_lse + RT;  // the waves' sums of P dP
    const Place at(p);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Keys keys(p, at.b);
    const int rows = p.nq * p.group, first = at.split * p.per, end = min(rows, first + p.per);
    const int live = min(live_rows(p, at.b), end);
    const float c2 = fabsf(p.scale) * kLog2e;
    const int64_t d = p.d;
    RowTiles<T, D, MODE> tile_q(p, at.b, at.hk, p.q, p.q_b, p.q_n, p.q_h);
    RowTiles<T, D, MODE> tile_g(p, at.b, at.hk, p.dout, p.g_b, p.g_n, p.g_h);
    float next_lse = 0.f;
    auto fetch = [&](int row0) {
        tile_q.load(p, row0, live, nullptr);
        tile_g.load(p, row0, live, nullptr);
        if (threadIdx.x < RT) {
            const int row = row0 + (int)threadIdx.x;
            next_lse = p.lse[Row(p, at.hk, row, row < live).stat(p, at.b)];
        }
    };
    const int tiles = keys.count > 0 ? (live - first + RT - 1) / RT : 0;
    if (tiles > 0) fetch(first);

    Frag k[KC][A::kSteps], v[KC][A::kSteps];
    bool counts[KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const int key = (wave * KC + c) * 16 + r;
        counts[c] = key < keys.count && (!keys.mask || keys.mask[key]);
        const int64_t from = counts[c] ? key : 0;
        raw_frags<T, MODE>(k[c], static_cast<const T*>(p.k) + at.b * p.k_b + from * p.k_n + at.hk * p.k_h, g, p.d);
        raw_frags<T, MODE>(v[c], static_cast<const T*>(p.v) + at.b * p.v_b + from * p.v_n + at.hk * p.v_h, g, p.d);
    }
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        fix_frags<T, MODE>(k[c], g, p.d, counts[c]);
        fix_frags<T, MODE>(v[c], g, p.d, counts[c]);
#pragma unroll
        for (int e = 0; e < A::kSteps; ++e)
            *reinterpret_cast<Frag*>(s_k + tile_at<T, D>((wave * KC + c) * 16 + r, 4 * e + g)) = k[c][e];
        if (p.scale < 0.f)
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s) k[c][s] = -k[c][s];
    }

    f32x4 dk[KC][A::kPairs][TG] = {}, dv[KC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    __shared__ float s_shift[4];
    // the lane's ds of the tile's first groups
    auto rescale = [&](float f, int groups) {
        for (int rg = 0; rg < groups; ++rg)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                Frag* at_ds = reinterpret_cast<Frag*>(s_ds + tile_at<T, RT>((wave * KC + c) * 16 + r, 4 * rg + g));
                Frag v = *at_ds;
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = (T)((float)v[j] * f);
                *at_ds = v;
            }
    };
    for (int t = 0; t < tiles; ++t) {
        const int row0 = first + t * RT;
        const uint64_t valid = ~0ull >> (64 - min(RT, live - row0));
        tile_q.move.place(s_q, valid, p.d);
        tile_g.move.place(s_g, valid, p.d);
        if (threadIdx.x < RT) s_lse[threadIdx.x] = next_lse * kLog2e;
        __syncthreads();
        if (t + 1 < tiles) fetch(row0 + RT);
        f32x4 s[NG][KC][TG] = {}, dp[NG][KC][TG] = {};
#pragma unroll
        for (int rg = 0; rg < NG; ++rg) {
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int e = 0; e < A::kSteps; ++e) {
                    const Frag a = row_frag<T, D>(s_q, rg * KS + out_row<T>(u, r), e, g);
                    const Frag b = row_frag<T, D>(s_g, rg * KS + out_row<T>(u, r), e, g);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        mma(s[rg][c][u], a, k[c][e]);
                        mma(dp[rg][c][u], b, v[c][e]);
                    }
                }
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const f32x4 lse = *reinterpret_cast<const f32x4*>(&s_lse[rg * KS + E * g + 4 * u]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        s[rg][c][u][j] =
                            __builtin_amdgcn_exp2f(fmaf(s[rg][c][u][j], c2, Shrink<T>::kWeights - lse[j]));
            }
            // rows and keys that do not count
#pragma unroll
            for (int c = 0; c < KC; ++c)
                if (__any(valid != ~0ull >> (64 - RT) || !counts[c]))
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const bool in = counts[c] && (valid >> (rg * KS + E * g + 4 * u + j) & 1);
                            s[rg][c][u][j] = in ? s[rg][c][u][j] : 0.f;
                            dp[rg][c][u][j] = in ? dp[rg][c][u][j] : 0.f;
                        }
            const float by = __builtin_amdgcn_exp2f(-Shrink<T>::kWeights);
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                f32x4 sum = s[rg][0][u] * dp[rg][0][u];
#pragma unroll
                for (int c = 1; c < KC; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = fmaf(s[rg][c][u][j], dp[rg][c][u][j], sum[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = over_row(sum[j]) * by;
                if (r == 0) *reinterpret_cast<f32x4*>(&s_sum[wave * RT + rg * KS + E * g + 4 * u]) = sum;
            }
        }
        __syncthreads();
#pragma unroll
        for (int rg = 0; rg < NG; ++rg) {
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const float* sums = s_sum + rg * KS + E * g + 4 * u;
                f32x4 delta = *reinterpret_cast<const f32x4*>(sums);
#pragma unroll
                for (int i = 1; i < 4; ++i) delta += *reinterpret_cast<const f32x4*>(sums + i * RT);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dp[rg][c][u][j] = s[rg][c][u][j] * (dp[rg][c][u][j] - delta[j]);
            }
            if (shrink.moved()) {
                const float f = __builtin_amdgcn_exp2f(shrink.shift - Shrink<T>::kWeights);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u) dp[rg][c][u] *= f;
            }
            auto each = [&](auto f) {
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f(dp[rg][c][u][j]);
            };
            shrink(each, [&](float f) {
#pragma unroll
                for (int c = 0; c < KC; ++c) {
#pragma unroll
                    for (int u = 0; u < TG; ++u) dp[rg][c][u] *= f;
#pragma unroll
                    for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                        for (int u = 0; u < TG; ++u) dk[c][e][u] *= f;
                }
                rescale(f, rg);  // what this tile's earlier groups have left for dq
            });
            Frag w[KC], ds[KC];
#pragma unroll
            for (int c = 0; c < KC; ++c) {
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[c][4 * u + j] = (T)s[rg][c][u][j], ds[c][4 * u + j] = (T)dp[rg][c][u][j];
                *reinterpret_cast<Frag*>(s_ds + tile_at<T, RT>((wave * KC + c) * 16 + r, 4 * rg + g)) = ds[c];
            }
#pragma unroll
            for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                for (int u = 0; u < TG; ++u) {
                    const Frag a = down_frag<T, D>(s_g, rg * KS, e, u, lane);
                    const Frag b = down_frag<T, D>(s_q, rg * KS, e, u, lane);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        mma(dv[c][e][u], a, w[c]);
                        mma(dk[c][e][u], b, ds[c]);
                    }
                }
        }
        if (Shrink<T>::kNeeded && lane == 0) s_shift[wave] = shrink.shift;
        __syncthreads();
        if constexpr (Shrink<T>::kNeeded) {  // all waves' ds to one scale
            const float low = fminf(fminf(s_shift[0], s_shift[1]), fminf(s_shift[2], s_shift[3]));
            if (low != s_shift[0] || low != s_shift[1] || low != s_shift[2] || low != s_shift[3]) {
                const float f = __builtin_amdgcn_exp2f(low - shrink.shift);
                if (f != 1.f) {
                    rescale(f, NG);
#pragma unroll
                    for (int c = 0; c < KC; ++c)
#pragma unroll
                        for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                            for (int u = 0; u < TG; ++u) dk[c][e][u] *= f;
                    shrink.shift = low;
                }
                __syncthreads();
            }
        }
        if (p.dq) {
            // 16 rows a wave, or fewer columns of them where a tile has fewer rows
            constexpr int kRowTiles = RT / 16, kShare = 4 / kRowTiles;
            constexpr int kParts = (A::kPairs + kShare - 1) / kShare;
            const int tile = wave % kRowTiles, e0 = wave / kRowTiles * kParts;
            f32x4 dq[kParts][TG] = {};
#pragma unroll
            for (int key0 = 0; key0 < H::kKeys; key0 += KS) {
                if (key0 >= keys.count) break;
                const Frag ds = across_frag<T, RT>(s_ds, key0, tile * 16, lane);
#pragma unroll
                for (int e = 0; e < kParts; ++e)
#pragma unroll
                    for (int u = 0; u < TG; ++u) mma(dq[e][u], down_frag<T, D>(s_k, key0, e0 + e, u, lane), ds);
            }
            const float by = p.scale * __builtin_amdgcn_exp2f(-shrink.shift);
            const int row = row0 + tile * 16 + r;
            if (row < live) {
                T* to = static_cast<T*>(p.dq) + Row(p, at.hk, row, true).whole(p, at.b) * d;
#pragma unroll
                for (int e = 0; e < kParts; ++e) {
                    Frag f;
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[4 * u + j] = (T)(dq[e][u][j] * by);
                    store_run(to, KS * (e0 + e) + E * g, p.d, f);
                }
            }
        }
    }
    if (p.dq) {  // rows that do not count, or have no key that does
        const int64_t none = keys.count > 0 ? max(live, first) : first;
        for (int64_t i = none * p.d + threadIdx.x; i < (int64_t)end * p.d; i += 256) {
            const int row = (int)(i / p.d);
            static_cast<T*>(p.dq)[Row(p, at.hk, row, true).whole(p, at.b) * d + (i - (int64_t)row * p.d)] = (T)0.f;
        }
    }
#pragma unroll
    for (int c = 0; c < KC; ++c)
        keys_out<T, D>(p, at, (wave * KC + c) * 16 + r, counts[c], shrink.shift, dk[c], dv[c], lane);
}

// The gradients of few rows: 16 QC of them, with all keys of a split, in tiles that the waves of a block share out.
// A wave reads its keys and values once, writes their gradients, which are whole since it has all rows, and adds up dq.
// Keys and ds go through LDS of the wave's own to come back as fragments down the keys.  8 rows on 1M keys of 8 heads of
// 32 bfloat16: 620 us, 3.3 TB/s of keys, values and their gradients, beside the vector instructions that fix, weigh
// and round them.
template <typename T, int D, int QC>
struct FewBack {
    static constexpr int kParts = sizeof(T) == 2 ? 1 : QC;  // steps of a sum over the rows
    static constexpr int kFixed = D / 16 * kParts * 1024;   // fragments down the rows of q, and of dout
    static constexpr int kPitch = 16 * QC * (int)sizeof(T);
    static constexpr int kWave = Tile<T>::KS * (pitch_of(D) * (int)sizeof(T) + kPitch);
    static constexpr int kJoin = 16 * QC * D * 4;
    static int bytes(int heads) {
        const int join = heads * kJoin;
        return 2 * heads * kFixed + (4 * kWave > join ? 4 * kWave : join);
    }
};

template <typename T, int D, int QC, int MODE>
__global__ __launch_bounds__(256, (D * (int)sizeof(T) >= 256 ? 1 : 2)) void k_attn_few_bwd(AttnArgs p) {
    typedef AttnTile<T, D> A;
    typedef FewBack<T, D, QC> F;
    typedef typename Tile<T>::Frag Frag;
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    extern __shared__ __align__(16) char s_mem[];
    __shared__ __align__(16) float s_lse[4][16 * QC], s_delta[4][16 * QC];
    Place at(p, p.together);
    if (at.none) return;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = 1 << p.together, own = wave & (heads - 1), part = wave >> p.together, parts = 4 >> p.together;
    const int first_head = at.hk;
    at.hk += own;
    at.problem = (at.problem << p.together) + own;
    Keys keys(p, at.b);
    const int first = at.split * p.per, last = keys.count - 1;
    keys.until(first + p.per);
    const int rows = p.nq * p.group, live = live_rows(p, at.b), whole_end = min(p.nk, first + p.per);
    const float c2 = fabsf(p.scale) * kLog2e;
    Frag* s_qt = reinterpret_cast<Frag*>(s_mem + 2 * own * F::kFixed);
    Frag* s_gt = reinterpret_cast<Frag*>(s_mem + (2 * own + 1) * F::kFixed);
    char* tk = s_mem + 2 * heads * F::kFixed + wave * F::kWave;
    char* tds = tk + KS * pitch_of(D) * (int)sizeof(T);

    const T* k_base = static_cast<const T*>(p.k) + at.b * p.k_b + at.hk * p.k_h;
    const T* v_base = static_cast<const T*>(p.v) + at.b * p.v_b + at.hk * p.v_h;
    Frag k[TG][A::kSteps], v[TG][A::kSteps];
    int byte = 0;
    auto fetch = [&](int k0) {
        byte = lane < KS ? keys.byte(k0, lane) : 0;
#pragma unroll
        for (int u = 0; u < TG; ++u) {
            const int in = min(16 * u + r, last - k0);
            if constexpr (MODE == ANY) {
                raw_frags<T, MODE>(k[u], k_base + (int64_t)(k0 + in) * p.k_n, g, p.d);
                raw_frags<T, MODE>(v[u], v_base + (int64_t)(k0 + in) * p.v_n, g, p.d);
            } else {
                raw_frags<T, MODE>(k[u], k_base + k0 * p.k_n + (uint32_t)in * (uint32_t)p.k_n, g, p.d);
                raw_frags<T, MODE>(v[u], v_base + k0 * p.v_n + (uint32_t)in * (uint32_t)p.v_n, g, p.d);
            }
        }
    };
    int k0 = first + part * KS;
    const int end = live > 0 ? keys.count : 0;
    if (k0 < end) fetch(k0);
    // all keys in one tile of each wave (and so one split, of one head a block): delta is summed from P dP
    const bool whole = p.nk <= 4 * KS;
    // fragments down the rows: element 4 c + j (float32: j of part c) is row 16 c + 4 g + j
    for (int i = threadIdx.x; i < heads * 2 * (D / 16) * F::kParts * 64; i += 256) {
        const int l = i & 63, step = (i >> 6) % F::kParts, tile = (i >> 6) / F::kParts % (D / 16);
        const int which = i / (D / 16 * F::kParts * 64), head = first_head + (which >> 1);
        const bool is_q = (which & 1) == 0;
        const int col = KS * (tile / TG) + out_row<T>(tile % TG, l & 15);
        Frag f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int row = 16 * (sizeof(T) == 2 ? e >> 2 : step) + 4 * (l >> 4) + (e & 3);
            const bool in = row < live && row < 16 * QC && col < p.d;
            const Row w(p, head, row, in);
            const T* from = is_q ? static_cast<const T*>(p.q) + at.b * p.q_b + w.query * p.q_n + w.head * p.q_h
                                 : static_cast<const T*>(p.dout) + at.b * p.g_b + w.query * p.g_n + w.head * p.g_h;
            f[e] = in ? from[col] : (T)0.f;
        }
        reinterpret_cast<Frag*>(s_mem + which * F::kFixed)[(tile * F::kParts + step) * 64 + l] = f;
    }
    Frag q[QC][A::kSteps], dout[QC][A::kSteps];
    rows_held<T, MODE>(p, at.b, at.hk, 0, live, p.q, p.q_b, p.q_n, p.q_h, p.scale < 0.f, lane, q);
    rows_held<T, MODE>(p, at.b, at.hk, 0, live, p.dout, p.g_b, p.g_n, p.g_h, false, lane, dout);
    if (part == 0 && g == 0)
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            const bool in = 16 * c + r < live;
            s_lse[own][16 * c + r] = in ? p.lse[Row(p, at.hk, 16 * c + r, in).stat(p, at.b)] * kLog2e : 0.f;
        }
    if (part == 0 && !whole) {
        Frag out[QC][A::kSteps];
        const int64_t row = p.d, query = row * p.heads;
        rows_held<T, MODE>(p, at.b, at.hk, 0, live, p.out, query * p.nq, query, row, false, lane, out);
#pragma unroll
        for (int c = 0; c < QC; ++c) {
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < A::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < E; ++j) sum = fmaf((float)dout[c][s][j], (float)out[c][s][j], sum);
            sum = added(sum);
            if (g == 0) s_delta[own][16 * c + r] = sum;
        }
    }
    __syncthreads();
    f32x4 lse[QC], delta[QC] = {};
#pragma unroll
    for (int c = 0; c < QC; ++c) {
        lse[c] = *reinterpret_cast<const f32x4*>(&s_lse[own][16 * c + 4 * g]);
        if (!whole) delta[c] = *reinterpret_cast<const f32x4*>(&s_delta[own][16 * c + 4 * g]);
    }
    f32x4 dq[QC][A::kPairs][TG] = {};
    Shrink<T> shrink;
    const int64_t out_n = (int64_t)p.kv_heads * p.d;
    T* dk_base = static_cast<T*>(p.dk) + (int64_t)at.b * p.nk * out_n + at.hk * p.d;
    T* dv_base = static_cast<T*>(p.dv) + (int64_t)at.b * p.nk * out_n + at.hk * p.d;
    // whole: every wave once, to meet the others; without keys its tile is zeros and nothing is stored
    for (const int stop = whole ? max(end, k0 + 1) : end; k0 < stop; k0 += parts * KS) {
        const uint64_t valid = __ballot(byte != 0);
        f32x4 s[TG][QC] = {}, dp[TG][QC] = {};
#pragma unroll
        for (int u = 0; u < TG; ++u) {
            const bool in = valid >> (16 * u + r) & 1;
            fix_frags<T, MODE>(k[u], g, p.d, in);
            fix_frags<T, MODE>(v[u], g, p.d, in);
#pragma unroll
            for (int e = 0; e < A::kSteps; ++e) {
                *reinterpret_cast<Frag*>(tk + tile_at<T, D>(16 * u + r, 4 * e + g)) = k[u][e];
#pragma unroll
                for (int c = 0; c < QC; ++c) {
                    mma(s[u][c], q[c][e], k[u][e]);
                    mma(dp[u][c], dout[c][e], v[u][e]);
                }
            }
        }
        if (k0 + parts * KS < end) fetch(k0 + parts * KS);
        auto counts = [&](int u, int c, int j) { return (valid >> (16 * u + r) & 1) && 16 * c + 4 * g + j < live; };
#pragma unroll
        for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int c = 0; c < QC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[u][c][j] = counts(u, c, j)
                                     ? __builtin_amdgcn_exp2f(fmaf(s[u][c][j], c2, Shrink<T>::kWeights - lse[c][j]))
                                     : 0.f;
        if (whole) {
            const float by = __builtin_amdgcn_exp2f(-Shrink<T>::kWeights);
#pragma unroll
            for (int c = 0; c < QC; ++c) {
                f32x4 sum = {};
#pragma unroll
                for (int u = 0; u < TG; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sum[j] = counts(u, c, j) ? fmaf(s[u][c][j], dp[u][c][j], sum[j]) : sum[j];
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = over_row(sum[j]) * by;
                if (r == 0) *reinterpret_cast<f32x4*>(&s_delta[wave][16 * c + 4 * g]) = sum;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < QC; ++c) {
                delta[c] = *reinterpret_cast<const f32x4*>(&s_delta[0][16 * c + 4 * g]);
#pragma unroll
                for (int i = 1; i < 4; ++i) delta[c] += *reinterpret_cast<const f32x4*>(&s_delta[i][16 * c + 4 * g]);
            }
        }
#pragma unroll
        for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int c = 0; c < QC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    dp[u][c][j] = counts(u, c, j) ? s[u][c][j] * (dp[u][c][j] - delta[c][j]) : 0.f;
        if (shrink.moved()) {
            const float f = __builtin_amdgcn_exp2f(shrink.shift - Shrink<T>::kWeights);
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int c = 0; c < QC; ++c) dp[u][c] *= f;
        }
        auto each = [&](auto f) {
#pragma unroll
            for (int u = 0; u < TG; ++u)
#pragma unroll
                for (int c = 0; c < QC; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) f(dp[u][c][j]);
        };
        shrink(each, [&](float f) {
#pragma unroll
            for (int c = 0; c < QC; ++c) {
#pragma unroll
                for (int u = 0; u < TG; ++u) dp[u][c] *= f;
#pragma unroll
                for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                    for (int u = 0; u < TG; ++u) dq[c][e][u] *= f;
            }
        });
        Frag w[TG][F::kParts], ds[TG][F::kParts];
#pragma unroll
        for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int i = 0; i < F::kParts; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int c = sizeof(T) == 2 ? e >> 2 : i;
                    w[u][i][e] = c < QC ? (T)s[u][c < QC ? c : 0][e & 3] : (T)0.f;
                    ds[u][i][e] = c < QC ? (T)dp[u][c < QC ? c : 0][e & 3] : (T)0.f;
                }
#pragma unroll
        for (int u = 0; u < TG; ++u)
#pragma unroll
            for (int c = 0; c < QC; ++c) {
                typedef T Quad __attribute__((ext_vector_type(4)));
                Quad quad;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    quad[j] = sizeof(T) == 2 ? ds[u][0][(4 * c + j) % E] : ds[u][c % F::kParts][j];
                *reinterpret_cast<Quad*>(tds + (16 * u + r) * F::kPitch + (16 * c + 4 * g) * (int)sizeof(T)) = quad;
            }
        wave_sync();
        const float by_k = p.scale * __builtin_amdgcn_exp2f(-shrink.shift);
        const float by_v = __builtin_amdgcn_exp2f(-Shrink<T>::kWeights);
#pragma unroll
        for (int e = 0; e < A::kPairs; ++e) {
            f32x4 gk[TG][TG] = {}, gv[TG][TG] = {};  // of key tile, column tile
#pragma unroll
            for (int t = 0; t < TG; ++t)
#pragma unroll
                for (int i = 0; i < F::kParts; ++i) {
                    const Frag a = s_qt[((TG * e + t) * F::kParts + i) * 64 + lane];
                    const Frag b = s_gt[((TG * e + t) * F::kParts + i) * 64 + lane];
#pragma unroll
                    for (int u = 0; u < TG; ++u) {
                        mma(gk[u][t], a, ds[u][i]);
                        mma(gv[u][t], b, w[u][i]);
                    }
                }
#pragma unroll
            for (int u = 0; u < TG; ++u) {
                const int key = k0 + 16 * u + r;
                Frag a, b;
#pragma unroll
                for (int t = 0; t < TG; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[4 * t + j] = (T)(gk[u][t][j] * by_k);
                        b[4 * t + j] = (T)(gv[u][t][j] * by_v);
                    }
                // a key that does not count: its weights of 0 times an infinite row are NaN
                if (valid != ~0ull >> (64 - KS) && !(valid >> (16 * u + r) & 1)) a = Frag{}, b = Frag{};
                if (key < end) {  // the others are cleared below, by other lanes
                    if (p.dk) store_run(dk_base + key * out_n, KS * e + E * g, p.d, a);
                    if (p.dv) store_run(dv_base + key * out_n, KS * e + E * g, p.d, b);
                }
            }
#pragma unroll
            for (int t = 0; t < TG; ++t) {
                const Frag a = down_frag<T, D>(tk, 0, e, t, lane);
#pragma unroll
                for (int c = 0; c < QC; ++c) {
                    union {
                        Frag f;
                        s16x4 h[2];
                    } b;
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            b.h[h] = read_transposed(tds + (8 * g + 4 * h + (r >> 2)) * F::kPitch +
                                                     (16 * c + 4 * (r & 3)) * 2);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            b.f[j] = *reinterpret_cast<const T*>(tds + (4 * g + j) * F::kPitch + (16 * c + r) * 4);
                    }
                    mma(dq[c][e][t], a, b.f);
                }
            }
        }
        wave_sync();
    }
    // keys of the split past the length
    for (int64_t i = (int64_t)max(end, first) * p.d + part * 64 + lane; i < (int64_t)whole_end * p.d; i += parts * 64) {
        const int64_t key = i / p.d, to = key * out_n + (i - key * p.d);
        if (p.dk) dk_base[to] = (T)0.f;
        if (p.dv) dv_base[to] = (T)0.f;
    }
    if (!p.dq) return;
    __syncthreads();
    // [16 QC][D] of each head, its waves in their order
    float* s_dq = reinterpret_cast<float*>(s_mem + 2 * heads * F::kFixed) + own * (16 * QC * D);
    const float by = p.scale * __builtin_amdgcn_exp2f(-shrink.shift);
    for (int i = 0; i < parts; ++i) {
        if (part == i)
#pragma unroll
            for (int c = 0; c < QC; ++c)
#pragma unroll
                for (int e = 0; e < A::kPairs; ++e)
#pragma unroll
                    for (int t = 0; t < TG; ++t) {
                        f32x4* to = reinterpret_cast<f32x4*>(s_dq + (16 * c + r) * D + KS * e + E * g + 4 * t);
                        const f32x4 own = dq[c][e][t] * by;
                        *to = i > 0 ? *to + own : own;
                    }
        __syncthreads();
    }
    for (int i = part * 64 + lane; i < min(rows, 16 * QC) * D; i += parts * 64) {
        const int row = i / D, col = i % D;
        if (p.splits > 1)
            p.part[(at.part(p, rows) + row) * pitch_of(D) + col] = row < live ? s_dq[i] : 0.f;
        else if (col < p.d)
            static_cast<T*>(p.dq)[Row(p, at.hk, row, true).whole(p, at.b) * p.d + col] =
                row < live ? (T)s_dq[i] : (T)0.f;
    }
}

template <typename T, int D, int MODE>
void attn_bwd_in(AttnArgs p, void* workspace, hipStream_t s) {
    const AttnPlan a = plan_at<T, D>(p);
    constexpr int kQc = MODE == ANY ? 1 : AttnShape<T, D>::kDq, kKc = MODE == ANY ? 1 : AttnShape<T, D>::kDkv;
    const int64_t rows = (int64_t)p.nq * p.group, problems = (int64_t)p.batch * p.kv_heads;
    p.delta = static_cast<float*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + a.delta_bytes);
    if (a.few_back && p.nq > 0 && p.nk > 0 && (a.few_back == 1 || MODE != ANY)) {
        constexpr int kFew = MODE == ANY || (sizeof(T) == 4 && D > 128) ? 1 : 2;
        p.splits = a.few_splits, p.per = a.few_per, p.tiles = 1, p.together = a.few_heads;
        const int heads = 1 << p.together;
        if (a.few_back == 1) {
            const unsigned lds = (unsigned)FewBack<T, D, 1>::bytes(heads);
            hipLaunchKernelGGL((k_attn_few_bwd<T, D, 1, MODE>), grid_of(p), dim3(256), lds, s, p);
        } else {
            const unsigned lds = (unsigned)FewBack<T, D, kFew>::bytes(heads);
            hipLaunchKernelGGL((k_attn_few_bwd<T, D, kFew, MODE>), grid_of(p), dim3(256), lds, s, p);
        }
        if (p.splits > 1 && p.dq) GS_ATTN_SHARED(k_attn_sum, problems * rows, , false);
        return;
    }
    if (a.held && p.nq > 0 && MODE != ANY) {
        constexpr int kMost = AttnShape<T, D>::kHeld, kMode = MODE == ANY ? PART : MODE;
        p.splits = a.held_splits, p.per = a.held_per, p.tiles = 1;
        const dim3 grid = grid_of(p);
        if (a.held == 1)
            hipLaunchKernelGGL((k_attn_held<T, D, 1, kMode>), grid, dim3(256), (HeldTile<T, D, 1>::kBytes), s, p);
        else
            hipLaunchKernelGGL((k_attn_held<T, D, kMost, kMode>), grid, dim3(256), (HeldTile<T, D, kMost>::kBytes), s, p);
        if (p.splits > 1 && (p.dk || p.dv)) GS_ATTN_SHARED(k_attn_sum, 2 * problems * p.nk, , true);
        return;
    }
    if (p.nq > 0) {
        const int qc = a.dq_qc < kQc ? a.dq_qc : kQc;
        p.splits = p.dq ? a.dq_splits : 1, p.per = p.dq ? a.dq_per : 0;
        p.tiles = (int32_t)tiles_of(rows, 64 * qc);
        if (qc == 1) hipLaunchKernelGGL((k_attn_dq<T, D, 1, MODE>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_dq<T, D, kQc, MODE>), grid_of(p), dim3(256), 0, s, p);
        if (p.splits > 1) GS_ATTN_SHARED(k_attn_sum, problems * rows, , false);
    }
    if (p.nk > 0 && (p.dk || p.dv)) {
        const int kc = a.dkv_kc < kKc ? a.dkv_kc : kKc;
        p.splits = a.dkv_splits, p.per = a.dkv_per;
        p.tiles = (int32_t)tiles_of(p.nk, 64 * kc);
        if (kc == 1) hipLaunchKernelGGL((k_attn_dkv<T, D, 1, MODE>), grid_of(p), dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_attn_dkv<T, D, kKc, MODE>), grid_of(p), dim3(256), 0, s, p);
        if (p.splits > 1) GS_ATTN_SHARED(k_attn_sum, 2 * problems * p.nk, , true);
    }
}

template <typename T, int D>
void attn_bwd_at(const AttnArgs& p, void* workspace, hipStream_t s) {
    const int mode = attn_mode<T, D>(p);
    if constexpr (D == pitch_of(D)) {
        if (mode == WHOLE) attn_bwd_in<T, D, WHOLE>(p, workspace, s);
        else if (mode == ANY) attn_bwd_in<T, D, ANY>(p, workspace, s);
    }
    if (mode == EVEN) attn_bwd_in<T, D, EVEN>(p, workspace, s);
    else if (mode == PART) attn_bwd_in<T, D, PART>(p, workspace, s);
}

template <typename T>
void attn_bwd(const AttnArgs& p, void* workspace, hipStream_t s) {
    GS_ATTN_BY_HEAD(attn_bwd_at, p.d, attn_any<T>(p))(p, workspace, s);
}

}  // namespace gs
