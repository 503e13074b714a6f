// The fused linear layer of the networks beside the Gaussians, and its backward.
//
//   z = x w^T + bias      y = act(z) + residual
//   dz = dy act'(z)       dx = dz w       dw = dz^T x       db = sum over rows of dz
//
// Products are summed in float32, the activation runs in float32, and every
// result is rounded once.  dz enters the two products of the backward rounded to the
// layer's type: the matrix instructions take no mixed operands, and in float32 they
// would run at a ninth of the 16-bit rate.  db is summed from dz before that rounding,
// where it is made: sums that cancel would keep the roundings.
#include "linear_bwd.h"

namespace gs {
namespace {

inline int size_of(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t pad256(size_t b) { return (b + 255) & ~(size_t)255; }

// One product y = epilogue(a b^T): a [rows, depth] (x or dz), b [cols, depth]
// (the weights, or their transpose for dx).
enum { EPI_FWD, EPI_DZ, EPI_PLAIN };

struct ProdArgs {
    const void* a;
    const void* b;
    const void* bias;   // FWD, DZ: [cols] or NULL
    const void* other;  // FWD: residual or NULL; DZ: dy
    void* out;
    int64_t rows, ld_a, ld_b, ld_other, ld_out;
    int32_t cols, depth, epi, act;
    float* sums;  // DZ: [runs of rows][ld_sums(cols)], the sums of dz's rows before its rounding, or NULL
    int32_t block_runs;  // k_prod_narrow: a run is a block's rows, added up in LDS, else 16 rows
};

inline __host__ __device__ int64_t ld_sums(int32_t cols) { return ((int64_t)cols + 3) / 4 * 4; }

// The epilogue of N runs (E consecutive outputs of one row each), with the runs of
// the residual or dy already in `other`; one switch over the kinds for all of them.
template <typename T, int N>
__device__ __forceinline__ void finish_runs(const ProdArgs& p, float (&v)[N * Tile<T>::E],
                                            const typename Tile<T>::Frag (&other)[N], typename Tile<T>::Frag (&out)[N]) {
    constexpr int E = Tile<T>::E;
    if (p.epi == EPI_FWD) {
        act_run<T>(p.act, v);
        if (p.other) {
#pragma unroll
            for (int j = 0; j < N * E; ++j) v[j] += (float)other[j / E][j % E];
        }
    } else if (p.epi == EPI_DZ) {
        float g[N * E];
#pragma unroll
        for (int j = 0; j < N * E; ++j) g[j] = (float)other[j / E][j % E];
        slope_run<T>(p.act, v, g);
    }
#pragma unroll
    for (int j = 0; j < N * E; ++j) out[j / E][j % E] = (T)v[j];
}

// Stores the sums of columns c0 to c0 + 7 over the rows of the lanes at `to`, a row of ld_sums(count) floats.
__device__ __forceinline__ void store_sums(float* to, int c0, int count, const float (&v)[8], int r) {
    float sum[2];
    run_sums(v, r, sum);
    const int c = c0 + pair_of(r);
    if (r < 4 && c < count) *reinterpret_cast<float2*>(to + c) = make_float2(sum[0], sum[1]);
}

// Few outputs or few rows: a block makes one group of KS outputs of 16 rows, its
// four waves taking every fourth step of the sum and joining in LDS.  The weights
// go straight from memory to the instruction: with few rows nothing would reuse
// them from LDS, and the launch's latency is all there is: 1 row 256 -> 256 bfloat16
// 3.5 us, of a call's 8.
template <typename T>
__global__ __launch_bounds__(256) void k_prod_few(ProdArgs p) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    __shared__ f32x4 s_acc[4][TG][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * KS;
    const int64_t row = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 16 + r;
    if (row - r >= p.rows) return;
    const T* a = static_cast<const T*>(p.a) + (row < p.rows ? row : p.rows - 1) * p.ld_a;
    const T* b[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        const int n = n0 + out_row<T>(t, r);
        b[t] = static_cast<const T*>(p.b) + (int64_t)(n < p.cols ? n : p.cols - 1) * p.ld_b;
    }
    f32x4 acc[TG] = {};
    const int whole = p.depth / KS;
    int s = wave;
    for (; s + 4 < whole; s += 8) {  // two steps' loads in flight
        const int k0 = s * KS + E * g, k1 = k0 + 4 * KS;
        const auto a0 = load16(a + k0), a1 = load16(a + k1);
        typename Tile<T>::Frag b0[TG], b1[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            b0[t] = load16(b[t] + k0);
            b1[t] = load16(b[t] + k1);
        }
#pragma unroll
        for (int t = 0; t < TG; ++t) mma(acc[t], b0[t], a0);
#pragma unroll
        for (int t = 0; t < TG; ++t) mma(acc[t], b1[t], a1);
    }
    for (; s * KS < p.depth; s += 4) {
        const int k0 = s * KS + E * g;
        const auto a0 = load_frag(a, k0, p.depth);
#pragma unroll
        for (int t = 0; t < TG; ++t) mma(acc[t], load_frag(b[t], k0, p.depth), a0);
    }
#pragma unroll
    for (int t = 0; t < TG; ++t) s_acc[wave][t][lane] = acc[t];
    __syncthreads();
    const bool in = row < p.rows;
    if (wave != 0 || (!in && !p.sums)) return;
    const int c0 = n0 + E * g;
    float v[E];
#pragma unroll
    for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[4 * t + i] = (s_acc[0][t][lane][i] + s_acc[1][t][lane][i]) + (s_acc[2][t][lane][i] + s_acc[3][t][lane][i]);
    if (p.bias) {
        const auto bias = load_frag(static_cast<const T*>(p.bias), c0, p.cols);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] += (float)bias[j];
    }
    typename Tile<T>::Frag other[1] = {zero_frag<T>()}, f[1];
    if (p.other && in) other[0] = load_frag(static_cast<const T*>(p.other) + row * p.ld_other, c0, p.cols);
    finish_runs<T, 1>(p, v, other, f);
    if (in) store_run(static_cast<T*>(p.out) + row * p.ld_out, c0, p.cols, f[0]);
    if constexpr (sizeof(T) == 2) {
        if (p.sums) {  // a run of 16 rows
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = in ? v[j] : 0.f;
            store_sums(p.sums + (row - r) / 16 * ld_sums(p.cols), c0, p.cols, v, r);
        }
    }
}

// Narrow layers over many rows: the weights stay in LDS as fragments for the
// life of the block, and each wave walks tiles of 16 rows, reading a row's whole
// depth (SL steps) into registers once and making all its outputs: x is read once
// and y written once, with no barrier in the loop.  Outputs are made and stored in
// pairs of groups, 128 bytes of a row at a time: with 64 the lines leave the caches
// half written (4.0 against 4.5 TB/s).  The next tile's x is on its way meanwhile.
// Rows whose outputs are not whole 16-byte runs (PACK) are put together in LDS and
// stored as the one contiguous piece of memory that a tile's rows are.  16-bit layers
// are bound by memory: 1M rows 128 -> 128 bfloat16 with a residual 146 us, 5.25 TB/s;
// 3M rows 64 -> 59 float16 138 us, 5.3 TB/s.  Float32 ones by the matrix rate and, under
// it, the start: 1M rows 128 -> 128 390 us, 84 TFLOP/s beside 2.6 TB/s; 100k rows
// 63 -> 128 28 us, of which 11 are products.
// SUMS: dz for a wide layer's backward, whose rows are added up on their way (the
// backward of 300k rows 128 -> 256 bfloat16 202 us against 196 without db's sums).
constexpr int narrow_threads(int sl) { return sl <= 4 ? 1024 : 512; }  // at most: deep rows need 256 registers
template <typename T, int SL, bool PACK, bool SUMS>
__global__ __launch_bounds__(narrow_threads(SL), sizeof(T) == 4 ? 4 : 1) void k_prod_narrow(ProdArgs p) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG, P = 2;
    typedef typename Tile<T>::Frag Frag;
    extern __shared__ __align__(16) char s_mem[];
    const int groups = (p.cols + KS - 1) / KS;
    Frag* s_w = reinterpret_cast<Frag*>(s_mem);                                     // [groups][TG][SL][64]
    f32x4* s_bias = reinterpret_cast<f32x4*>(s_w + (size_t)groups * TG * SL * 64);  // [groups][KS / 4]
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    T* s_out = reinterpret_cast<T*>(s_bias + groups * KS / 4) + wave * 16 * p.cols;  // PACK: [waves][16][cols]
    float* s_sum = reinterpret_cast<float*>(s_bias + groups * KS / 4);               // SUMS: [waves][groups * KS]
    const int64_t tiles = (p.rows + 15) / 16, step = (int64_t)gridDim.x * waves;
    int64_t tile = (int64_t)blockIdx.x * waves + wave;
    auto row_of = [&](int64_t t) { return min(t * 16 + r, p.rows - 1); };
    const Matrix<T> ma(p.a, p.rows, p.ld_a, p.depth), mo(p.other, p.rows, p.ld_other, p.cols);
    const bool even_a = p.depth == SL * KS, even_o = p.cols == groups * KS && groups % P == 0;
    Frag x[SL], next[SL];
    auto fetch = [&](int64_t t) {  // past the end: the last row again
        const int64_t row = row_of(t);
#pragma unroll
        for (int s = 0; s < SL; ++s) next[s] = ma.raw(row, s * KS + E * g);
    };
    fetch(tile);
    const int frags = groups * TG * SL * 64;
    auto place = [&](int i, int& n, int& k0) {  // output and first input of fragment i
        const int l = i & 63, gt = (i >> 6) / SL;
        n = gt / TG * KS + out_row<T>(gt % TG, l & 15);
        k0 = (i >> 6) % SL * KS + E * (l >> 4);
    };
    if ((p.cols - 1) * p.ld_b + p.depth >= E) {
        const Matrix<T> mb(p.b, p.cols, p.ld_b, p.depth);
        for (int i0 = threadIdx.x; i0 < frags; i0 += 8 * blockDim.x) {
            Frag v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                int n, k0;
                place(i0 + u * blockDim.x, n, k0);
                v[u] = mb.raw(min(n, p.cols - 1), k0);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                int n, k0;
                place(i0 + u * blockDim.x, n, k0);
                if (i0 + u * (int)blockDim.x < frags)
                    s_w[i0 + u * blockDim.x] = mb.fixed(v[u], min(n, p.cols - 1), k0, n < p.cols);
            }
        }
    } else {  // fewer weights than a fragment
        for (int i = threadIdx.x; i < frags; i += blockDim.x) {
            int n, k0;
            place(i, n, k0);
            s_w[i] = n < p.cols ? load_edge(static_cast<const T*>(p.b) + n * p.ld_b, k0, p.depth) : zero_frag<T>();
        }
    }
    for (int i = threadIdx.x; i < groups * KS; i += blockDim.x)
        reinterpret_cast<float*>(s_bias)[i] =
            p.bias && i < p.cols ? (float)static_cast<const T*>(p.bias)[i] : 0.f;
    if (SUMS && p.block_runs)
        for (int i = threadIdx.x; i < waves * groups * KS; i += blockDim.x) s_sum[i] = 0.f;
    __syncthreads();
    for (; tile < tiles; tile += step) {
        const int64_t row = tile * 16 + r;
#pragma unroll
        for (int s = 0; s < SL; ++s) x[s] = next[s];
        if (!even_a) x[SL - 1] = ma.fixed(x[SL - 1], row_of(tile), (SL - 1) * KS + E * g, true);  // the others lie inside
        fetch(tile + step);
        T* out = PACK ? s_out + r * p.cols : static_cast<T*>(p.out) + row * p.ld_out;
        for (int n = 0; n < groups; n += P) {
            Frag other[P];
            if (p.other) {
#pragma unroll
                for (int h = 0; h < P; ++h) other[h] = mo.raw(row_of(tile), (n + h) * KS + E * g);
            }
            f32x4 acc[P][TG];
#pragma unroll
            for (int h = 0; h < P; ++h) {
                if (h > 0 && n + h >= groups) break;
#pragma unroll
                for (int t = 0; t < TG; ++t) acc[h][t] = s_bias[((n + h) * KS + E * g) / 4 + t];
#pragma unroll
                for (int s = 0; s < SL; ++s)
#pragma unroll
                    for (int t = 0; t < TG; ++t) mma(acc[h][t], s_w[(((n + h) * TG + t) * SL + s) * 64 + lane], x[s]);
            }
            if (p.other && !even_o && n + P >= groups) {
#pragma unroll
                for (int h = 0; h < P; ++h)
                    other[h] = mo.fixed(other[h], row_of(tile), (n + h) * KS + E * g, true);
            }
            Frag f[P];
#pragma unroll
            for (int h = 0; h < P; ++h) {  // one at a time: both together spill registers
                if (h > 0 && n + h >= groups) break;
                float v[E];
                Frag o[1] = {other[h]}, to[1];
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = acc[h][j / 4][j % 4];
                finish_runs<T, 1>(p, v, o, to);
                f[h] = to[0];
                if constexpr (SUMS) {
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = row < p.rows ? v[j] : 0.f;
                    if (p.block_runs) {
                        float sum[2];
                        run_sums(v, r, sum);
                        float* to = s_sum + (wave * groups + n + h) * KS + E * g + pair_of(r);
                        if (r < 4) to[0] += sum[0], to[1] += sum[1];
                    } else {
                        store_sums(p.sums + tile * ld_sums(p.cols), (n + h) * KS + E * g, p.cols, v, r);
                    }
                }
            }
            if (PACK || row < p.rows) {
#pragma unroll
                for (int h = 0; h < P; ++h) {
                    if (h > 0 && n + h >= groups) break;
                    store_run(out, (n + h) * KS + E * g, p.cols, f[h]);
                }
            }
        }
        if (PACK) {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            const int count = (int)min((int64_t)16, p.rows - tile * 16) * p.cols;
            T* to = static_cast<T*>(p.out) + tile * 16 * p.cols;
            for (int i = lane * E; i + E <= count; i += 64 * E)
                *reinterpret_cast<Frag*>(to + i) = *reinterpret_cast<const Frag*>(s_out + i);
            for (int i = count / E * E + lane; i < count; i += 64) to[i] = s_out[i];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        }
    }
    if (SUMS && p.block_runs) {
        __syncthreads();
        for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
            float t = 0.f;
            for (int i = 0; i < waves; ++i) t += s_sum[i * groups * KS + c];
            p.sums[blockIdx.x * ld_sums(p.cols) + c] = t;
        }
    }
}

// Deep or wide layers: 128 x 128 outputs per block, 64 x 64 per wave.  Both
// operands pass through LDS in rows of 128 bytes (2 steps), their 16-byte chunks
// rotated by the row so that the fragments' reads meet no bank twice; the next
// two stages are on their way in registers while one is multiplied: with one, a
// stage (0.4 us) is shorter than the memory's answer.  65536 rows 512 -> 512 bfloat16
// 64 us, 530 TFLOP/s, and 54 us, 640 TFLOP/s, without an activation; 1024 -> 1024 218
// us; float32 512 -> 512 316 us, 109 TFLOP/s.  The matrix units are busy for 40% of the
// 16-bit time, the fragments' reads take as many cycles of LDS, and each stage ends in
// a barrier, at two blocks a CU.  256 x 128
// outputs over eight waves take as long (72 us against 74, 213 against 218).
constexpr int kBig = 128;  // rows and outputs of a block
template <typename T, int NT, bool SUMS>  // NT: tiles of 16 outputs a wave has, 4 (128 outputs a block) or 2 (64)
__global__ __launch_bounds__(256, 2) void k_prod_big(ProdArgs p) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    typedef typename Tile<T>::Frag Frag;
    __shared__ Frag s_a[2][kBig * 8], s_b[2][32 * NT * 8];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 16 * NT;
    // blocks of one XCD take neighbouring tiles, outputs first: they share rows of a
    const int64_t tn = (p.cols + 32 * NT - 1) / (32 * NT), total = (int64_t)gridDim.x, per = (total + 7) / 8;
    const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    const int64_t tiles = tn * ((p.rows + kBig - 1) / kBig);
    if (id >= tiles) return;
    const int64_t m0 = id / tn * kBig;
    const int n0 = (int)(id % tn) * 32 * NT;
    // staging: thread i brings chunk i % 8 of rows i / 8, + 32, + 64, + 96; the weights' rows in the order
    // that interleaves a group's tiles
    const int ch = threadIdx.x & 7, sr = threadIdx.x >> 3;
    const Matrix<T> ma(p.a, p.rows, p.ld_a, p.depth), mb(p.b, p.cols, p.ld_b, p.depth);
    int64_t row_a[4];
    int row_b[NT];
    Frag ra[2][4], rb[2][NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pos = sr + 32 * i, n = n0 + pos / KS * KS + out_row<T>(pos % KS / 16, pos % 16);
        row_a[i] = min(m0 + pos, p.rows - 1);
        if (i < NT) row_b[i] = n < p.cols ? n : p.cols - 1;
    }
    const int steps = (p.depth + 2 * KS - 1) / (2 * KS);
    auto fetch = [&](int s, Frag (&a)[4], Frag (&b)[NT]) {  // past the end: the matrices' last bytes, not used
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = ma.raw(row_a[i], s * 2 * KS + E * ch);
            if (i < NT) b[i] = mb.raw(row_b[i], s * 2 * KS + E * ch);
        }
    };
    auto put = [&](int s, int buf, Frag (&a)[4], Frag (&b)[NT]) {
        if ((s + 1) * 2 * KS > p.depth) {
            const int k0 = s * 2 * KS + E * ch;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = ma.fixed(a[i], row_a[i], k0, true);
                if (i < NT) b[i] = mb.fixed(b[i], row_b[i], k0, true);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pos = sr + 32 * i, at = pos * 8 + (ch ^ (pos & 7));
            s_a[buf][at] = a[i];
            if (i < NT) s_b[buf][at] = b[i];
        }
    };
    f32x4 acc[4][NT] = {};  // [m tile][n tile]
    if (steps > 0) {
        fetch(0, ra[0], rb[0]);
        fetch(1, ra[1], rb[1]);
        put(0, 0, ra[0], rb[0]);
    }
    __syncthreads();
    // 16-bit: the residual or dy is on its way during the products (the backward of 65536 rows 512 -> 512 bfloat16
    // 195 us against 205 with it fetched after them); in float32 there are twice the registers of it (920 against 905)
    const Matrix<T> mo(p.other, p.rows, p.ld_other, p.cols);
    Frag others[NT / TG][4];
    auto fetch_others = [&]() {
        if (!p.other) return;
#pragma unroll
        for (int q = 0; q < NT / TG; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                others[q][i] = mo.raw(min(m0 + wm + 16 * i + r, p.rows - 1), n0 + wn + q * KS + E * g);
    };
    if (sizeof(T) == 2) fetch_others();
    for (int s0 = 0; s0 < steps; s0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // stage s0 + u lies in buffer u, the next one in registers
            const int s = s0 + u;
            if (s >= steps) break;
            fetch(s + 2, ra[u], rb[u]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Frag fa[4], fb[NT];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int am = wm + 16 * i + r, bn = wn + 16 * i + r;
                    fa[i] = s_a[u][am * 8 + ((4 * h + g) ^ (am & 7))];
                    if (i < NT) fb[i] = s_b[u][bn * 8 + ((4 * h + g) ^ (bn & 7))];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma(acc[i][j], fb[j], fa[i]);
            }
            if (s + 1 < steps) put(s + 1, u ^ 1, ra[u ^ 1], rb[u ^ 1]);
            __syncthreads();
        }
    }
    if (sizeof(T) == 4) fetch_others();
    const bool even = n0 + 32 * NT <= p.cols;
#pragma unroll
    for (int q = 0; q < NT / TG; ++q) {  // groups of KS outputs
        const int c0 = n0 + wn + q * KS + E * g;
        Frag(&other)[4] = others[q];
        float bias[E] = {};
        if (p.bias) {
            const auto f = load_frag(static_cast<const T*>(p.bias), c0, p.cols);
#pragma unroll
            for (int j = 0; j < E; ++j) bias[j] = (float)f[j];
        }
        if (p.other && !even) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                other[i] = mo.fixed(other[i], min(m0 + wm + 16 * i + r, p.rows - 1), c0, true);
        }
        float v[4 * E];
        Frag f[4];
#pragma unroll
        for (int j = 0; j < 4 * E; ++j) v[j] = acc[j / E][q * TG + j % E / 4][j % 4] + bias[j % E];
        finish_runs<T, 4>(p, v, other, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = m0 + wm + 16 * i + r;
            if (row < p.rows) store_run(static_cast<T*>(p.out) + row * p.ld_out, c0, p.cols, f[i]);
        }
        if constexpr (SUMS) {  // a run is a wave's 64 rows
            float sum[E] = {};
#pragma unroll
            for (int j = 0; j < 4 * E; ++j) sum[j % E] += m0 + wm + 16 * (j / E) + r < p.rows ? v[j] : 0.f;
            if (m0 + wm < p.rows) store_sums(p.sums + (m0 + wm) / 64 * ld_sums(p.cols), c0, p.cols, sum, r);
        }
    }
}

constexpr size_t kLdsBytes = 160 * 1024;

// The kernel that a product takes, and the block of k_prod_narrow.
struct Route {
    bool few, narrow;
    int groups, steps;
    int threads;
    size_t lds;
    bool block_runs;  // sums of dz's rows go through LDS
};

// Blocks of k_prod_narrow that a CU holds.
inline int per_cu(size_t lds, int threads) {
    const int n = (int)(kLdsBytes / lds);
    return n < 1024 / threads ? n : 1024 / threads;
}
inline int64_t narrow_blocks(int64_t rows, const Route& q) {
    const int64_t blocks = cdiv(cdiv(rows, 16), q.threads / 64), most = 256 * per_cu(q.lds, q.threads);
    return blocks < most ? blocks : most;
}

// sums: of dz's rows.  Each wave of k_prod_narrow adds them up in LDS unless the CU then holds fewer blocks, and leaves
// those of every 16 rows if it does (the backward of 300k rows 128 -> 256 bfloat16 202 us, 212 with every 16 rows;
// 64 -> 512 354 us, 370 with LDS and fewer blocks).

template <typename T>
Route route(int64_t rows, int32_t cols, int32_t depth, bool sums) {
    constexpr int KS = Tile<T>::KS;
    Route q{};
    q.groups = (int)cdiv(cols, KS), q.steps = (int)cdiv(depth, KS);
    const int64_t tiles16 = cdiv(rows, 16);
    q.lds = (size_t)q.groups * KS * (q.steps * KS * sizeof(T) + 4);
    q.narrow = q.lds <= kLdsBytes && q.steps <= 8;
    q.threads = q.lds <= 40960 ? 256 : q.lds <= 81920 || q.steps > 4 ? 512 : 1024;
    if (sums && q.narrow) {
        const size_t lds = q.lds + (size_t)q.threads / 64 * q.groups * KS * 4;
        q.block_runs = per_cu(lds, q.threads) == per_cu(q.lds, q.threads);
        if (q.block_runs) q.lds = lds;
    }
    // Few tiles: a call of ordinary length is its launch, until about 2048 blocks of k_prod_few (500 rows 512 -> 512
    // bfloat16 8.5 us against 11.2 by k_prod_big, 1000 rows 8.9 against 11.8, 2000 rows 13.8 against 11.9; 16000 rows
    // 128 -> 128 8.5 by k_prod_narrow against 10.3).  In float32 a wave of k_prod_narrow takes 128 cycles for each of a
    // tile's groups and steps, and until there are tiles for every wave that is what the call lasts (8000 rows
    // 128 -> 192 14.6 against 25.2, 63 -> 128 9.6 against 10.6; 16000 rows 128 -> 128 18.1 against 18.9, 128 -> 64
    // 11.8 against 9.4).
    // Deep float32 rows of one group: k_prod_big's outputs would mostly be multiplied for nothing (150k rows 417 -> 3
    // 65 us against 95, 417 -> 16 93 against 95, 417 -> 32 156 against 96; bfloat16, whose products are short,
    // 417 -> 3 56 against 52, 417 -> 32 105 against 60).
    q.few = tiles16 * q.groups <= 2048 || (sizeof(T) == 4 && q.narrow && q.groups > 4 && tiles16 <= 640) ||
            (sizeof(T) == 4 && !q.narrow && q.groups == 1) || depth == 0;
    return q;
}

template <typename T, int SL>
void launch_narrow(ProdArgs p, Route q, hipStream_t s) {
    constexpr int E = Tile<T>::E;
    const size_t packed = (size_t)q.threads / 4 * p.cols * sizeof(T);
    const bool pack = !p.sums && p.ld_out == p.cols && p.cols % E != 0 && aligned16(p.out) && q.lds + packed <= kLdsBytes;
    if (pack) q.lds += packed;
    p.block_runs = q.block_runs;
    const dim3 grid((unsigned)narrow_blocks(p.rows, q));
    if (pack)
        hipLaunchKernelGGL((k_prod_narrow<T, SL, true, false>), grid, dim3(q.threads), q.lds, s, p);
    else if (!p.sums)
        hipLaunchKernelGGL((k_prod_narrow<T, SL, false, false>), grid, dim3(q.threads), q.lds, s, p);
    else if constexpr (sizeof(T) == 2)
        hipLaunchKernelGGL((k_prod_narrow<T, SL, false, true>), grid, dim3(q.threads), q.lds, s, p);
}

template <typename T>
void product(const ProdArgs& p, hipStream_t s) {
    const Route q = route<T>(p.rows, p.cols, p.depth, p.sums != nullptr);
    // the streaming kernels read 16 bytes at a time: x and the residual have to span them
    const auto spans = [](int64_t rows, int64_t ld, int32_t count) { return (rows - 1) * ld + count >= Tile<T>::E; };
    if (q.few || !spans(p.rows, p.ld_a, p.depth) || (p.other && !spans(p.rows, p.ld_other, p.cols))) {
        const int64_t tiles16 = cdiv(p.rows, 16), y = tiles16 < 32768 ? tiles16 : 32768;
        hipLaunchKernelGGL((k_prod_few<T>), dim3(q.groups, (unsigned)y, (unsigned)cdiv(tiles16, y)), dim3(256), 0, s, p);
        return;
    }
    // 1M rows 128 -> 128 bfloat16 110 us against 167 by k_prod_big, 256 -> 192 204 against 343, 64 -> 64 float16 52
    // against 94; 100k rows 63 -> 128 float32 29 against 38
    if (q.narrow) {
        switch (q.steps) {
            case 1: launch_narrow<T, 1>(p, q, s); return;
            case 2: launch_narrow<T, 2>(p, q, s); return;
            case 3: launch_narrow<T, 3>(p, q, s); return;
            case 4: launch_narrow<T, 4>(p, q, s); return;
            case 5: launch_narrow<T, 5>(p, q, s); return;
            case 6: launch_narrow<T, 6>(p, q, s); return;
            case 7: launch_narrow<T, 7>(p, q, s); return;
            case 8: launch_narrow<T, 8>(p, q, s); return;
        }
    }
    if constexpr (sizeof(T) == 4) {
        // 150k rows 417 -> 64 106 us against 180 with 128 outputs a block, 150 -> 40 47 against 84
        if (p.cols <= 64) {
            const int64_t tiles = cdiv(p.rows, kBig);
            hipLaunchKernelGGL((k_prod_big<T, 2, false>), dim3((unsigned)(cdiv(tiles, 8) * 8)), dim3(256), 0, s, p);
            return;
        }
    }
    const int64_t tiles = cdiv(p.cols, kBig) * cdiv(p.rows, kBig);
    const dim3 grid((unsigned)(cdiv(tiles, 8) * 8));
    if constexpr (sizeof(T) == 2) {
        if (p.sums) {
            hipLaunchKernelGGL((k_prod_big<T, 4, true>), grid, dim3(256), 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((k_prod_big<T, 4, false>), grid, dim3(256), 0, s, p);
}

// Runs of rows whose sums a product for dz leaves.
template <typename T>
int64_t sum_runs(int64_t rows, int32_t cols, int32_t depth) {
    const Route q = route<T>(rows, cols, depth, true);
    return !q.few && q.block_runs ? narrow_blocks(rows, q) : cdiv(rows, q.few || q.narrow ? 16 : 64);
}

struct DwArgs {
    const void* dz;
    const void* x;
    float* part;  // [splits][n_out * n_in of dw, then n_out of db], each if wanted
    int64_t rows, ld_dz, ld_x, per;
    int32_t n_out, n_in;
    int32_t want_dw, want_db, splits;
    const float* z_sums;  // [runs][ld_sums(n_out)]: sums of dz's rows before its rounding; NULL: dz lost nothing by it
    int64_t runs;
};

// One split of the rows for a 128 x 128 tile of dw: 64 x 64 per wave, the next
// stage's rows on their way while this one's are multiplied.  The blocks of the
// first column of tiles add up dz's columns as they pass, or the sums that its kernel
// has left of them where dz was rounded.  65536 rows 512 -> 512 bfloat16
// 56 us, 610 TFLOP/s: the stages' barriers bound it, as in k_prod_big.  Float32 layers of
// few outputs have narrower tiles, or the products of nothing would bound them: dx, dw
// and db of 150k rows 162 -> 9 104 us against 157 with 128 outputs, 417 -> 64 304
// against 362.
template <typename T, int NT>  // NT: tiles of 16 outputs a wave has; 1 or 2: a float32 layer of at most 32 or 64
__global__ __launch_bounds__(256, 2) void k_dw(DwArgs p) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS;
    typedef typename Tile<T>::Frag Frag;
    __shared__ __align__(16) char s_dz[2][16384], s_x[2][16384];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wn = (wave & 1) * 16 * NT, wk = (wave >> 1) * 64;
    // the tiles of one split run on one XCD, whose L2 then serves the rows that they share
    const int tn = (p.n_out + 127) / 128, tiles = tn * ((p.n_in + 127) / 128);
    const int64_t id = (int64_t)(blockIdx.x & 7) * ((gridDim.x + 7) / 8) + (blockIdx.x >> 3);
    const int64_t split = id / tiles;
    if (split >= p.splits) return;
    const int n0 = (int)(id % tiles) % tn * 128, k0 = (int)(id % tiles) / tn * 128;
    const int64_t m_begin = split * p.per, m_end = min(p.rows, m_begin + p.per);
    constexpr int kRows = 16384 / (128 * (int)sizeof(T));  // of a stage: 64 or 32
    constexpr int kChunks = 128 / E;                       // 16-byte chunks of a row
    constexpr int kPass = 256 / kChunks;  // rows that the block's threads cover at a time
    const int ch = threadIdx.x % kChunks, mr = threadIdx.x / kChunks;
    const Matrix<T> mz(p.dz, p.rows, p.ld_dz, p.n_out), mx(p.x, p.rows, p.ld_x, p.n_in);
    const bool even_z = n0 + 128 <= p.n_out, even_x = k0 + 128 <= p.n_in;
    Frag rz[2][4], rx[2][4];
    auto fetch = [&](int64_t m0, Frag (&z)[4], Frag (&x)[4]) {  // past the end: the last row, not used
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = min(m0 + mr + i * kPass, p.rows - 1);
            z[i] = mz.raw(m, n0 + ch * E);
            x[i] = mx.raw(m, k0 + ch * E);
        }
    };
    float sum[E] = {};
    const bool sums = p.want_db && k0 == 0, add = sums && !p.z_sums;
    auto put = [&](int64_t m0, int buf, Frag (&z)[4], Frag (&x)[4]) {
        if (!even_z || m0 + kRows > m_end) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + mr + i * kPass;
                z[i] = mz.fixed(z[i], min(m, p.rows - 1), n0 + ch * E, m < m_end);
            }
        }
        if (!even_x || m0 + kRows > m_end) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + mr + i * kPass;
                x[i] = mx.fixed(x[i], min(m, p.rows - 1), k0 + ch * E, m < m_end);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = row_chunk<T, 128>(mr + i * kPass, ch);
            *reinterpret_cast<Frag*>(s_dz[buf] + at) = z[i];
            *reinterpret_cast<Frag*>(s_x[buf] + at) = x[i];
            if (add)
#pragma unroll
                for (int j = 0; j < E; ++j) sum[j] += (float)z[i][j];
        }
    };
    f32x4 acc[NT][4] = {};  // [n tile][k tile]
    if (m_begin < m_end) {
        fetch(m_begin, rz[0], rx[0]);
        fetch(m_begin + kRows, rz[1], rx[1]);
        put(m_begin, 0, rz[0], rx[0]);
    }
    __syncthreads();
    for (int64_t m2 = m_begin; m2 < m_end; m2 += 2 * kRows) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // this stage lies in buffer u, the next one in registers
            const int64_t m0 = m2 + u * kRows;
            if (m0 >= m_end) break;
            fetch(m0 + 2 * kRows, rz[u], rx[u]);
#pragma unroll
            for (int h = 0; h < kRows / KS; ++h) {
                Frag fz[NT], fx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < NT) fz[i] = column_frag<T, 128>(s_dz[u], h * KS, wn + 16 * i, lane);
                    fx[i] = column_frag<T, 128>(s_x[u], h * KS, wk + 16 * i, lane);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma(acc[i][j], fz[i], fx[j]);
            }
            if (m0 + kRows < m_end) put(m0 + kRows, u ^ 1, rz[u ^ 1], rx[u ^ 1]);
            __syncthreads();
        }
    }
    const int64_t n_w = p.want_dw ? (int64_t)p.n_out * p.n_in : 0;
    float* part = p.part + split * (n_w + (p.want_db ? p.n_out : 0));
    if (p.want_dw) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = n0 + wn + 16 * i + 4 * g + q;
                if (n >= p.n_out) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = k0 + wk + 16 * j + r;
                    if (k < p.n_in) part[(int64_t)n * p.n_in + k] = acc[i][j][q];
                }
            }
    }
    if (sums && p.z_sums) {  // every splits-th run, an eighth of them by 32 threads with four outputs each
        float* s_sum = reinterpret_cast<float*>(s_dz[0]);  // [8][128]
        const int c = (threadIdx.x & 31) * 4, part8 = threadIdx.x >> 5;
        f32x4 t = {};
        if (n0 + c < p.n_out) {
            const float* from = p.z_sums + n0 + c;
#pragma unroll 8
            for (int64_t i = split + (int64_t)part8 * p.splits; i < p.runs; i += 8 * (int64_t)p.splits)
                t += *reinterpret_cast<const f32x4*>(from + i * ld_sums(p.n_out));
        }
        *reinterpret_cast<f32x4*>(s_sum + part8 * 128 + c) = t;
        __syncthreads();
        if (threadIdx.x < 128 && n0 + (int)threadIdx.x < p.n_out) {
            float sum_of = 0.f;
            for (int i = 0; i < 8; ++i) sum_of += s_sum[i * 128 + threadIdx.x];
            part[n_w + n0 + threadIdx.x] = sum_of;
        }
    } else if (sums) {  // the threads of one chunk column, in order
        float* s_sum = reinterpret_cast<float*>(s_dz[0]);  // [kPass][128]
#pragma unroll
        for (int j = 0; j < E; ++j) s_sum[mr * 128 + ch * E + j] = sum[j];
        __syncthreads();
        if (threadIdx.x < 128 && n0 + (int)threadIdx.x < p.n_out) {
            float t = 0.f;
            for (int i = 0; i < kPass; ++i) t += s_sum[i * 128 + threadIdx.x];
            part[n_w + n0 + threadIdx.x] = t;
        }
    }
}

// out [cols, rows] = in [rows, cols]^T, 64 x 64 per block: the weights, so that dx is
// the same product as the forward.  512 x 512 bfloat16 5 us, all of it latency.
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T* in, T* out, int32_t rows, int32_t cols) {
    __shared__ T s[64][65];
    const int c0 = blockIdx.x * 64, r0 = blockIdx.y * 64, x = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int r = y; r < 64; r += 4)
        if (r0 + r < rows && c0 + x < cols) s[r][x] = in[(int64_t)(r0 + r) * cols + c0 + x];
    __syncthreads();
    for (int c = y; c < 64; c += 4)
        if (c0 + c < cols && r0 + x < rows) out[(int64_t)(c0 + c) * rows + r0 + x] = s[x][c];
}

// The backward of few rows (views, not Gaussians): one kernel and the join of dx.
// A block has one group of KS outputs and 256 inputs.  It makes the group's z
// as k_prod_few does, keeps dz in LDS unrounded, and then every thread has one
// input: x's column in registers for its column of dw (complete: all rows are
// here) and the partial dx that this group of outputs gives.  The weights are read
// twice, the second time from the caches; what bounds it is latency: 8 rows 512 -> 1021
// float32 11 us and 4 for the join.  Two launches in place of the general path's five,
// or of a grid that so few rows leave empty: 8 rows 512 -> 1021 float32 16 us a call
// against 28, 16 rows 256 -> 256 bfloat16 18 against 25, 128 -> 128 16.6 against 17.1 by
// one block of k_bwd_narrow; 64 -> 64 16 against 14, which would round dz.
constexpr int kFewRows = 16;
struct FewArgs {
    const void* x;
    const void* w;
    const void* bias;
    const void* dy;
    void* dw;       // NULL: not wanted
    void* db;       // NULL: not wanted
    float* dx_part;  // [groups][rows][n_in], NULL: dx not wanted
    int64_t ld_x, ld_dy;
    int32_t rows, n_in, n_out, act;
};

template <typename T, int M>  // M: rows, rounded up
__global__ __launch_bounds__(256) void k_bwd_few(FewArgs p) {
    constexpr int E = Tile<T>::E, KS = Tile<T>::KS, TG = Tile<T>::TG;
    __shared__ f32x4 s_acc[4][TG][64];
    __shared__ float s_dz[KS][16];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * KS, c0 = n0 + E * g;
    const T* x = static_cast<const T*>(p.x);
    const T* w = static_cast<const T*>(p.w);
    const int k = (int)blockIdx.y * 256 + threadIdx.x, kc = k < p.n_in ? k : p.n_in - 1;  // -1: no inputs
    float xk[M] = {};  // on its way during the first half
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (kc >= 0) xk[m] = (float)x[(int64_t)(m < p.rows ? m : p.rows - 1) * p.ld_x + kc];
    f32x4 acc[TG] = {};
    if (p.act != GS_ACT_NONE) {
        const T* a = x + (int64_t)(r < p.rows ? r : p.rows - 1) * p.ld_x;
        const T* b[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const int n = n0 + out_row<T>(t, r);
            b[t] = w + (int64_t)(n < p.n_out ? n : p.n_out - 1) * p.n_in;
        }
        const int whole = p.n_in / KS;
        int s = wave;
        for (; s + 12 < whole; s += 16) {  // four steps' loads in flight
            typename Tile<T>::Frag fa[4], fb[4][TG];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k0 = (s + 4 * u) * KS + E * g;
                fa[u] = load16(a + k0);
#pragma unroll
                for (int t = 0; t < TG; ++t) fb[u][t] = load16(b[t] + k0);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int t = 0; t < TG; ++t) mma(acc[t], fb[u][t], fa[u]);
        }
        for (; s * KS < p.n_in; s += 4) {
            const int k0 = s * KS + E * g;
            const auto a0 = load_frag(a, k0, p.n_in);
#pragma unroll
            for (int t = 0; t < TG; ++t) mma(acc[t], load_frag(b[t], k0, p.n_in), a0);
        }
    }
#pragma unroll
    for (int t = 0; t < TG; ++t) s_acc[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave == 0) {
        float v[E], d[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int t = j / 4, i = j % 4;
            v[j] = (s_acc[0][t][lane][i] + s_acc[1][t][lane][i]) + (s_acc[2][t][lane][i] + s_acc[3][t][lane][i]);
            d[j] = 0.f;
        }
        if (p.bias) {
            const auto bias = load_frag(static_cast<const T*>(p.bias), c0, p.n_out);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] += (float)bias[j];
        }
        if (r < p.rows) {
            const auto dy = load_frag(static_cast<const T*>(p.dy) + (int64_t)r * p.ld_dy, c0, p.n_out);
#pragma unroll
            for (int j = 0; j < E; ++j) d[j] = (float)dy[j];
        }
        slope_run<T>(p.act, v, d);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (r >= p.rows || c0 + j >= p.n_out) v[j] = 0.f;
            s_dz[E * g + j][r] = v[j];
        }
    }
    __syncthreads();
    if (p.db && blockIdx.y == 0 && threadIdx.x < KS && n0 + (int)threadIdx.x < p.n_out) {
        float t = 0.f;
        for (int m = 0; m < p.rows; ++m) t += s_dz[threadIdx.x][m];
        static_cast<T*>(p.db)[n0 + threadIdx.x] = (T)t;
    }
    if (k >= p.n_in) return;
    float dx[M] = {};
    const int last = p.n_out - n0 < KS ? p.n_out - n0 : KS;
#pragma unroll(M > 8 ? 4 : 8)
    for (int n = 0; n < last; ++n) {
        const float wk = p.dx_part ? (float)w[(int64_t)(n0 + n) * p.n_in + k] : 0.f;
        float t = 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const float dz = s_dz[n][m];
            // rows past the end have dz = 0, but x there is another row's and may be infinite
            if (m < p.rows) t = fmaf(dz, xk[m], t);
            dx[m] = fmaf(dz, wk, dx[m]);
        }
        if (p.dw) static_cast<T*>(p.dw)[(int64_t)(n0 + n) * p.n_in + k] = (T)t;
    }
    if (p.dx_part)
        for (int m = 0; m < M; ++m)
            if (m < p.rows) p.dx_part[((int64_t)blockIdx.x * p.rows + m) * p.n_in + k] = dx[m];
}

template <typename T>
void launch_few(const FewArgs& p, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(p.n_out, Tile<T>::KS), (unsigned)(p.n_in > 0 ? cdiv(p.n_in, 256) : 1));
    if (p.rows <= 1)
        hipLaunchKernelGGL((k_bwd_few<T, 1>), grid, dim3(256), 0, s, p);
    else if (p.rows <= 4)
        hipLaunchKernelGGL((k_bwd_few<T, 4>), grid, dim3(256), 0, s, p);
    else if (p.rows <= 8)
        hipLaunchKernelGGL((k_bwd_few<T, 8>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_bwd_few<T, 16>), grid, dim3(256), 0, s, p);
}

// The join of partial results: element e of [0, count) is the sum over splits of
// part[s][e], 256 / lanes elements per block, `lanes` threads taking every lanes-th
// split each and joining in order: the same bits each time, where atomics would not
// give them.  Elements [0, first) go to out0, rows of `cols` elements ld apart, the rest
// to out1.  512 partials of 128 x 129 (34 MB, mostly in the caches) 13 us.
struct JoinArgs {
    const float* part;
    void* out0;
    void* out1;
    int64_t count, first, ld;
    int32_t cols, splits, lanes;
};

template <typename T>
__global__ __launch_bounds__(256) void k_join(JoinArgs p) {
    __shared__ float s_sum[256];
    const int width = 256 / p.lanes, e_in = threadIdx.x % width, l = threadIdx.x / width;
    const int64_t e = (int64_t)blockIdx.x * width + e_in;
    float acc = 0.f;
    if (e < p.count) {
#pragma unroll 8
        for (int s = l; s < p.splits; s += p.lanes) acc += p.part[(int64_t)s * p.count + e];
    }
    s_sum[threadIdx.x] = acc;
    __syncthreads();
    if (l != 0 || e >= p.count) return;
    for (int i = 1; i < p.lanes; ++i) acc += s_sum[i * width + e_in];
    if (e >= p.first)
        static_cast<T*>(p.out1)[e - p.first] = (T)acc;
    else
        static_cast<T*>(p.out0)[p.ld == p.cols ? e : e / p.cols * p.ld + e % p.cols] = (T)acc;
}

template <typename T>
void join(JoinArgs p, hipStream_t s) {
    p.lanes = 1;
    while (p.lanes < 16 && p.lanes * 8 <= p.splits) p.lanes *= 2;
    hipLaunchKernelGGL((k_join<T>), dim3((unsigned)cdiv(p.count, 256 / p.lanes)), dim3(256), 0, s, p);
}

inline int check_shape(const gs_linear* d) {
    if (!d || d->rows < 0 || d->n_in < 0 || d->n_out < 0 || d->dtype < GS_F32 || d->dtype > GS_BF16 ||
        d->act < GS_ACT_NONE || d->act > GS_ACT_GELU)
        return GS_EINVAL;
    if (d->rows > 0x7fffffff || d->n_in > (1 << 20) || d->n_out > (1 << 20)) return GS_ECAPACITY;
    return GS_OK;
}

inline bool element_aligned(const void* p, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (size_of(dtype) - 1)) == 0;
}

struct BwdPlan {
    bool few, narrow;            // one kernel for few rows; one pass over the rows
    int32_t outs;                // outputs of a pass (narrow)
    size_t dz, sums, wt, part, bytes;  // offsets in the workspace
    int64_t runs;                      // of rows, whose sums of dz lie at `sums` (0: none)
    int64_t ld_dz;
    int splits;  // of the rows: partial dw and db
    int64_t per;
};

// Few inputs, an activation and more outputs than a pass holds: passes over parts of the
// outputs, so that dz, many times x, makes no trip through memory.  1.76M rows 10 -> 364
// bfloat16 691 us against 1836 by separate products, 375k rows 63 -> 708 float32 1580
// against 2123, 300k rows 64 -> 512 bfloat16 270 against 354.  Where there are few rows,
// or more inputs, the parts' dx in float32 and their launches weigh more: 20k rows
// 20 -> 512 80 against 57; of more than 32 16-bit inputs 100k rows take 0.80 to 1.12
// times as long, 131072 rows 0.79 to 1.08, 200k rows 0.70 to 0.88; 300k rows 90 -> 512
// 485 against 357.
template <typename T>
inline bool plan_narrow(const gs_linear* d, BwdPlan& p) {
    constexpr int kMost = kBwdGroups * Tile<T>::KS;
    if (d->rows <= kFewRows || d->n_out < 1) return false;
    p.outs = d->n_out;
    const int64_t least = sizeof(T) == 2 && d->n_in > Tile<T>::KS ? 131072 : 65536;
    if (d->n_out > kMost && d->rows >= least && d->act != GS_ACT_NONE && d->n_in <= kPartInputs) p.outs = kMost;
    if (!bwd_narrow_fits<T>(d->n_in, p.outs)) return false;
    p.splits = bwd_narrow_blocks<T>(d->rows, d->n_in, p.outs);
    return true;
}

inline BwdPlan bwd_plan(const gs_linear* d) {
    BwdPlan p{};
    size_t at = 0;
    p.few = d->rows >= 1 && d->rows <= kFewRows && d->n_out > 0;
    if (p.few) {  // a block per group of outputs leaves a partial dx
        p.splits = (int)cdiv(d->n_out, d->dtype == GS_F32 ? Tile<float>::KS : Tile<_Float16>::KS);
        p.bytes = pad256((size_t)p.splits * d->rows * d->n_in * 4);
        return p;
    }
    p.narrow = d->dtype == GS_F32   ? plan_narrow<float>(d, p)
               : d->dtype == GS_F16 ? plan_narrow<_Float16>(d, p)
                                    : plan_narrow<__bf16>(d, p);
    if (!p.narrow) {
        // two blocks per CU between the tiles and the splits of the rows, each split at least 256 rows
        const int64_t tiles = cdiv(d->n_out, 128) * cdiv(d->n_in > 0 ? d->n_in : 1, 128);
        int64_t splits = tiles > 0 ? cdiv(512, tiles) : 1;
        if (splits > cdiv(d->rows, 256)) splits = cdiv(d->rows, 256);
        if (splits < 1) splits = 1;
        p.per = cdiv(cdiv(d->rows, splits), 64) * 64;
        p.splits = (int)(d->rows > 0 ? cdiv(d->rows, p.per) : 1);
        const int e = 16 / size_of(d->dtype);
        p.ld_dz = cdiv(d->n_out, e) * e;
        p.dz = at;
        if (d->act != GS_ACT_NONE) at += pad256((size_t)d->rows * p.ld_dz * size_of(d->dtype));
        p.sums = at;
        // relu's dz is dy or 0, which no rounding changes
        if (d->act != GS_ACT_NONE && d->act != GS_ACT_RELU && d->dtype != GS_F32 && d->rows > 0 && d->n_out > 0) {
            p.runs = d->dtype == GS_F16 ? sum_runs<_Float16>(d->rows, d->n_out, d->n_in)
                                        : sum_runs<__bf16>(d->rows, d->n_out, d->n_in);
            at += pad256((size_t)p.runs * ld_sums(d->n_out) * 4);
        }
        p.wt = at;
        at += pad256((size_t)d->n_out * d->n_in * size_of(d->dtype));
        p.outs = d->n_out;
    } else if (p.outs < d->n_out) {  // dx so far
        const int64_t ks = d->dtype == GS_F32 ? Tile<float>::KS : Tile<_Float16>::KS;
        p.dz = at;
        at += pad256((size_t)d->rows * cdiv(d->n_in, ks) * ks * 4);
    }
    p.part = at;
    at += pad256((size_t)p.splits * p.outs * ((size_t)d->n_in + 1) * 4);
    p.bytes = at;
    return p;
}

template <typename T>
void fwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* residual, void* y,
         hipStream_t s) {
    ProdArgs p{x, w, bias, residual, y, d->rows, d->ld_x, d->n_in, d->ld_res, d->ld_y, d->n_out, d->n_in, EPI_FWD,
               d->act, nullptr, 0};
    product<T>(p, s);
}

template <typename T>
void bwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* dy, void* dx, void* dw,
         void* db, char* ws, hipStream_t s) {
    const BwdPlan plan = bwd_plan(d);
    float* part = reinterpret_cast<float*>(ws + plan.part);
    if (plan.few) {
        FewArgs q{x, w, bias, dy, dw, db, dx && d->n_in > 0 ? part : nullptr, d->ld_x, d->ld_y, (int32_t)d->rows, d->n_in, d->n_out,
                  d->act};
        launch_few<T>(q, s);
        if (q.dx_part) {
            const int64_t count = d->rows * d->n_in;
            join<T>(JoinArgs{part, dx, nullptr, count, count, d->ld_dx, d->n_in, plan.splits, 0}, s);
        }
        return;
    }
    const bool want_dw = dw && d->n_out > 0 && d->n_in > 0, want_db = db && d->n_out > 0;
    const int64_t n_w = want_dw ? (int64_t)d->n_out * d->n_in : 0, n_b = want_db ? d->n_out : 0;
    if (plan.narrow) {
        for (int32_t n0 = 0; n0 < d->n_out; n0 += plan.outs) {
            const int32_t outs = d->n_out - n0 < plan.outs ? d->n_out - n0 : plan.outs;
            BwdArgs q{};
            q.x = x;
            q.w = static_cast<const T*>(w) + (int64_t)n0 * d->n_in;
            q.bias = bias ? static_cast<const T*>(bias) + n0 : nullptr;
            q.dy = static_cast<const T*>(dy) + n0;
            q.dx = dx;
            q.part = part;
            q.rows = d->rows, q.ld_x = d->ld_x, q.ld_dy = d->ld_y, q.ld_dx = d->ld_dx;
            q.n_in = d->n_in, q.n_out = outs, q.act = d->act;
            q.want_dw = want_dw, q.want_db = want_db;
            T* dw_out = want_dw ? static_cast<T*>(dw) + (int64_t)n0 * d->n_in : nullptr;
            T* db_out = want_db ? static_cast<T*>(db) + n0 : nullptr;
            if (plan.splits == 1) q.dw = dw_out, q.db = db_out;
            if (plan.outs < d->n_out) {
                q.dx_sum = reinterpret_cast<float*>(ws + plan.dz);
                q.first = n0 == 0, q.last = n0 + outs == d->n_out;
            }
            launch_bwd_narrow<T>(q, plan.splits, s);
            const int64_t c_w = want_dw ? (int64_t)outs * d->n_in : 0, count = c_w + (want_db ? outs : 0);
            if (plan.splits > 1 && count > 0)
                join<T>(JoinArgs{part, dw_out, db_out, count, c_w, d->n_in, d->n_in, plan.splits, 0}, s);
        }
        return;
    }
    const JoinArgs sums{part, dw, db, n_w + n_b, n_w, d->n_in, d->n_in, plan.splits, 0};
    const void* dz = dy;
    int64_t ld_dz = d->ld_y;
    // made whether db is wanted or not: dz then has the same bits either way
    float* z_sums = plan.runs > 0 ? reinterpret_cast<float*>(ws + plan.sums) : nullptr;
    if (d->act != GS_ACT_NONE && d->rows > 0 && d->n_out > 0) {
        ProdArgs p{x, w, bias, dy, ws + plan.dz, d->rows, d->ld_x, d->n_in, d->ld_y, plan.ld_dz, d->n_out, d->n_in,
                   EPI_DZ, d->act, z_sums, 0};
        product<T>(p, s);
        dz = ws + plan.dz;
        ld_dz = plan.ld_dz;
    }
    if (dx && d->rows > 0 && d->n_in > 0) {
        T* wt = reinterpret_cast<T*>(ws + plan.wt);
        if (d->n_out > 0)
            hipLaunchKernelGGL((k_transpose<T>), dim3((unsigned)cdiv(d->n_in, 64), (unsigned)cdiv(d->n_out, 64)),
                               dim3(256), 0, s, static_cast<const T*>(w), wt, d->n_out, d->n_in);
        ProdArgs p{dz, wt, nullptr, nullptr, dx, d->rows, ld_dz, d->n_out, 0, d->ld_dx, d->n_in, d->n_out, EPI_PLAIN,
                   GS_ACT_NONE, nullptr, 0};
        product<T>(p, s);
    }
    if (!want_dw && !want_db) return;
    // without dw there is one column of tiles, and its x side reads dz (the product is not stored)
    DwArgs q{dz, want_dw ? x : dz, part, d->rows, ld_dz, want_dw ? d->ld_x : ld_dz, plan.per, d->n_out,
             want_dw ? d->n_in : 1, want_dw, want_db,
             plan.splits, z_sums, plan.runs};
    const int64_t blocks = cdiv(q.n_out, 128) * cdiv(q.n_in, 128) * plan.splits;
    const dim3 grid((unsigned)(cdiv(blocks, 8) * 8));
    if constexpr (sizeof(T) == 4) {
        if (q.n_out <= 32)
            hipLaunchKernelGGL((k_dw<T, 1>), grid, dim3(256), 0, s, q);
        else if (q.n_out <= 64)
            hipLaunchKernelGGL((k_dw<T, 2>), grid, dim3(256), 0, s, q);
        else
            hipLaunchKernelGGL((k_dw<T, 4>), grid, dim3(256), 0, s, q);
    } else {
        hipLaunchKernelGGL((k_dw<T, 4>), grid, dim3(256), 0, s, q);
    }
    join<T>(sums, s);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_linear_fwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* residual,
                             void* y, void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (d->rows == 0 || d->n_out == 0) return GS_OK;
    if (!y || (d->n_in > 0 && (!x || !w))) return GS_EINVAL;
    if (d->ld_x < d->n_in || d->ld_y < d->n_out || (residual && d->ld_res != 0 && d->ld_res < d->n_out))
        return GS_EINVAL;
    for (const void* p : {x, w, bias, residual, (const void*)y})
        if (!element_aligned(p, d->dtype)) return GS_EALIGN;
    hipStream_t s = as_stream(stream);
    if (d->dtype == GS_F32)
        fwd<float>(d, x, w, bias, residual, y, s);
    else if (d->dtype == GS_F16)
        fwd<_Float16>(d, x, w, bias, residual, y, s);
    else
        fwd<__bf16>(d, x, w, bias, residual, y, s);
    return launch_status();
}

extern "C" int gs_linear_bwd_workspace_size(const gs_linear* d, size_t* bytes) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (!bytes) return GS_EINVAL;
    *bytes = bwd_plan(d).bytes;
    return GS_OK;
}

extern "C" int gs_linear_bwd(const gs_linear* d, const void* x, const void* w, const void* bias, const void* dy,
                             void* dx, void* dw, void* db, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_shape(d);
    if (rc != GS_OK) return rc;
    if (d->n_out == 0 && (!dx || d->rows == 0 || d->n_in == 0)) return GS_OK;
    if (d->rows > 0 && d->n_out > 0 && !dy) return GS_EINVAL;
    if (d->rows > 0 && d->n_in > 0 && d->n_out > 0 && (!x || !w)) return GS_EINVAL;
    if (d->rows > 0 && (d->ld_x < d->n_in || d->ld_y < d->n_out || (dx && d->ld_dx < d->n_in))) return GS_EINVAL;
    for (const void* p : {x, w, bias, dy, (const void*)dx, (const void*)dw, (const void*)db})
        if (!element_aligned(p, d->dtype)) return GS_EALIGN;
    const size_t need = bwd_plan(d).bytes;
    if (need > 0 && !workspace) return GS_EINVAL;
    if (workspace_bytes < need) return GS_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GS_EALIGN;
    hipStream_t s = as_stream(stream);
    char* ws = static_cast<char*>(workspace);
    if (d->dtype == GS_F32)
        bwd<float>(d, x, w, bias, dy, dx, dw, db, ws, s);
    else if (d->dtype == GS_F16)
        bwd<_Float16>(d, x, w, bias, dy, dx, dw, db, ws, s);
    else
        bwd<__bf16>(d, x, w, bias, dy, dx, dw, db, ws, s);
    return launch_status();
}
