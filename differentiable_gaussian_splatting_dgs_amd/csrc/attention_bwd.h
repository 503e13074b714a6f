// Gradients of cross attention (attention.h).
#pragma once

#include "attention.h"

namespace gs {

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

// Gradients.  With P = exp(s - lse) and ds = P (dout v^T - delta), delta the row's sum of dout * out:
// dq = scale ds k, dk = scale ds^T q, dv = P^T dout.  P and ds enter the products rounded to the type.  float16:
// both are held times 2^13 and, should a ds not fit then, scaled down with what is summed so far (Shrink).
template <typename T>
struct Shrink {
    static constexpr bool kNeeded = false;
    static constexpr float shift = 0.f;
    template <typename Over>
    __device__ __forceinline__ void operator()(float, Over) {}
};
template <>
struct Shrink<_Float16> {
    static constexpr bool kNeeded = true;
    float shift = 13.f;
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
    KeyTiles<T, D, MODE> tile_k(p.k, at.b * p.k_b + at.hk * p.k_h, p.k_n, keys.count, p.d);
    KeyTiles<T, D, MODE> tile_v(p.v, at.b * p.v_b + at.hk * p.v_h, p.v_n, keys.count, p.d);
    keys.until(first + p.per);
    const int rows = p.nq * p.group, live = live_rows(p, at.b);
    const int row0 = (at.tile * 4 + wave) * 16 * QC;
    const float c2 = fabsf(p.scale) * kLog2e;
    const int tiles = p.dq && live > at.tile * 64 * QC ? (keys.count - first + KT - 1) / KT : 0;
    int byte = 0;
    if (tiles > 0) {
        byte = keys.byte(first, lane);
        tile_k.load(first, p.d);
        tile_v.load(first, p.d);
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
        tile_k.move.store(s_k[0], valid, p.d);
        tile_v.move.store(s_v[0], valid, p.d);
    }
    for (int t = 0; t < tiles; ++t) {
        if (t + 1 < tiles) {
            const int next = first + (t + 1) * KT;
            byte = keys.byte(next, lane);
            tile_k.load(next, p.d);
            tile_v.load(next, p.d);
        }
        __syncthreads();
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
            float most = 0.f;
            if constexpr (Shrink<T>::kNeeded)
#pragma unroll
                for (int c = 0; c < QC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) most = fmaxf(most, fabsf(s[c][u][j]));
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
            tile_k.move.store(s_k[(t + 1) & 1], valid, p.d);
            tile_v.move.store(s_v[(t + 1) & 1], valid, p.d);
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
    RowTiles<T, D, MODE> tile_q(p, at.b, at.hk, p.q, p.q_b, p.q_n, p.q_h);
    RowTiles<T, D, MODE> tile_g(p, at.b, at.hk, p.dout, p.g_b, p.g_n, p.g_h);
    float next_lse = 0.f, next_delta = 0.f;
    auto fetch = [&](int row0) {
        tile_q.load(p, row0, live);
        tile_g.load(p, row0, live);
        if (threadIdx.x < RT) {
            const int row = row0 + (int)threadIdx.x;
            const int64_t stat = Row(p, at.hk, row, row < live).stat(p, at.b);
            next_lse = p.lse[stat];
            next_delta = p.delta[stat];
        }
    };
    auto place = [&](int buffer, uint64_t valid) {
        tile_q.move.store(s_q[buffer], valid, p.d);
        tile_g.move.store(s_g[buffer], valid, p.d);
        if (threadIdx.x < RT)
            s_lse[buffer][threadIdx.x] = next_lse * kLog2e, s_delta[buffer][threadIdx.x] = next_delta;
    };
    // the tile's rows that count
    auto bits = [&](int row0) { return ~0ull >> (64 - min(RT, live - row0)); };
    if (tiles > 0) fetch(first);

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
        if (t + 1 < tiles) fetch(first + (t + 1) * RT);
        __syncthreads();
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
                        const float w = __builtin_amdgcn_exp2f(fmaf(s[c][u][j], c2, shrink.shift - lse[j]));
                        s[c][u][j] = w;
                        dp[c][u][j] = w * (dp[c][u][j] - delta[j]);
                    }
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
            float any = 0.f;  // keys that do not count have weights that mean nothing
            if constexpr (Shrink<T>::kNeeded)
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int u = 0; u < TG; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) any = fmaxf(any, counts[c] ? fabsf(dp[c][u][j]) : 0.f);
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

template <typename T, int D, int MODE>
void attn_bwd_in(AttnArgs p, void* workspace, hipStream_t s) {
    const AttnPlan a = plan_at<T, D>(p);
    constexpr int kQc = MODE == ANY ? 1 : AttnShape<T, D>::kDq, kKc = MODE == ANY ? 1 : AttnShape<T, D>::kDkv;
    const int64_t rows = (int64_t)p.nq * p.group, problems = (int64_t)p.batch * p.kv_heads;
    p.delta = static_cast<float*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + a.delta_bytes);
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
    if (mode == WHOLE) attn_bwd_in<T, D, WHOLE>(p, workspace, s);
    else if (mode == PART) attn_bwd_in<T, D, PART>(p, workspace, s);
    else attn_bwd_in<T, D, ANY>(p, workspace, s);
}

template <typename T>
void attn_bwd(const AttnArgs& p, void* workspace, hipStream_t s) {
    GS_ATTN_BY_HEAD(attn_bwd_at)(p, workspace, s);
}

}  // namespace gs
