// What the entry points of cross attention hand to its kernels.
#pragma once

#include "gs_internal.h"

namespace gs {

struct Div {  // n / d for n < 2^31
    uint32_t mul, shift;
};

struct AttnArgs {
    const void *q, *k, *v, *dout;
    const uint8_t* mask;                   // [batch] rows of nk, or NULL
    const int32_t *q_lengths, *k_lengths;  // [batch], or NULL
    void* out;                             // read by the backward
    float* lse;                            // [batch, heads, nq]
    float* delta;                          // the backward's sums of dout * out, like lse
    void *dq, *dk, *dv;
    int64_t q_b, q_n, q_h, k_b, k_n, k_h, v_b, v_n, v_h, g_b, g_n, g_h, mask_b;  // strides (g: dout's)
    int32_t batch, nq, nk, heads, kv_heads, group, d;
    float scale;
    Div by_group, by_kv;
    int32_t tiles;   // of rows or keys of a problem
    int32_t splits;  // of the keys (forward, dq) or of the rows (dk, dv)
    int32_t per;     // keys or rows of a split
    int32_t together;  // log of the heads of keys that a block takes, where it keeps the keys
    // more than one split: [problem][split][row or key][padded d] sums of each, joined by a next launch; the forward's
    // are relative to the split's reference, which part_stat holds with the sum of the weights: [..][2]
    float *part, *part_stat;
};

// How a call shares out its work: the same from sizes alone for the workspace and the launches.
struct AttnPlan {
    int few;                   // tiles of 16 rows that a wave takes with all of the keys of its own (0: block tiles)
    int few_heads;             // log of the heads that a block of few rows takes in the backward
    int thin;                  // blocks that share out a problem's rows and keep its keys (0: not so)
    int together;              // log of the heads of keys that such a block takes
    int fwd_qc, dq_qc, dkv_kc; // 16-row tiles a wave
    int held;                  // 16-key tiles a wave where a block holds all keys in the backward (0: it does not)
    int few_back;              // few, where the backward has it
    int few_splits, few_per, held_splits, held_per;  // of the backward
    int fwd_splits, fwd_per, dq_splits, dq_per, dkv_splits, dkv_per;
    size_t fwd_bytes, delta_bytes, bwd_bytes;  // workspaces, and parts of the backward's
};

inline Div div_by(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return Div{(uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
}

struct AttnBytes {
    size_t fwd, bwd;
};

template <typename T>
AttnBytes attn_bytes(const AttnArgs& p);
template <typename T>
void attn_fwd(const AttnArgs& p, void* workspace, hipStream_t s);
template <typename T>
void attn_bwd(const AttnArgs& p, void* workspace, hipStream_t s);

}  // namespace gs
