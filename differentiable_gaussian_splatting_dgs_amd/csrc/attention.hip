// Entry points of cross attention: checks, workspace, choice of the type's kernels (attention.h).
#include <math.h>

#include "attention_args.h"

namespace gs {
namespace {

inline int size_of(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }

int check_shape(const gs_attention* a) {
    if (!a || a->batch < 0 || a->nq < 0 || a->nk < 0 || a->heads < 1 || a->kv_heads < 1 || a->d < 1 ||
        a->dtype < GS_F32 || a->dtype > GS_BF16 || a->heads % a->kv_heads != 0 || a->scale == 0.f ||
        !isfinite(a->scale * kLog2e))  // what the kernels multiply by
        return GS_EINVAL;
    // 64-row tiles of all problems are numbered in 24 bits, rows and keys in 31
    const int64_t most = (int64_t)1 << 30;
    if (a->d > GS_MAX_HEAD_DIM || a->batch > most || a->nq > most || a->nk > most || a->heads > most) return GS_ECAPACITY;
    const int64_t problems = (int64_t)a->batch * a->kv_heads, group = a->heads / a->kv_heads;
    const int64_t tiles = 16000000;
    if (problems > tiles || a->nq * group > most || problems * ((a->nq * group + 63) / 64) > tiles ||
        problems * ((a->nk + 63) / 64) > tiles)
        return GS_ECAPACITY;
    return GS_OK;
}

bool no_strides_below_zero(const gs_attention* a, bool back) {
    for (int i = 0; i < 3; ++i)
        if (a->q_stride[i] < 0 || a->k_stride[i] < 0 || a->v_stride[i] < 0 || (back && a->dout_stride[i] < 0)) return false;
    return a->mask_stride >= 0;
}

bool aligned_to(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }

AttnArgs args_of(const gs_attention* a, const void* q, const void* k, const void* v, const uint8_t* mask,
                 const int32_t* q_lengths, const int32_t* k_lengths) {
    AttnArgs p{};
    p.q = q, p.k = k, p.v = v, p.mask = mask, p.q_lengths = q_lengths, p.k_lengths = k_lengths;
    p.q_b = a->q_stride[0], p.q_n = a->q_stride[1], p.q_h = a->q_stride[2];
    p.k_b = a->k_stride[0], p.k_n = a->k_stride[1], p.k_h = a->k_stride[2];
    p.v_b = a->v_stride[0], p.v_n = a->v_stride[1], p.v_h = a->v_stride[2];
    p.g_b = a->dout_stride[0], p.g_n = a->dout_stride[1], p.g_h = a->dout_stride[2];
    p.mask_b = a->mask_stride;
    p.batch = (int32_t)a->batch, p.nq = (int32_t)a->nq, p.nk = (int32_t)a->nk;
    p.heads = a->heads, p.kv_heads = a->kv_heads, p.group = a->heads / a->kv_heads, p.d = a->d;
    p.scale = a->scale;
    p.by_group = div_by((uint32_t)p.group), p.by_kv = div_by((uint32_t)p.kv_heads);
    return p;
}

AttnBytes bytes_of(const AttnArgs& p, int32_t dtype) {
    return dtype == GS_F32 ? attn_bytes<float>(p) : dtype == GS_F16 ? attn_bytes<_Float16>(p) : attn_bytes<__bf16>(p);
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need > 0 && !workspace) return GS_EINVAL;
    if (bytes < need) return GS_EWORKSPACE;
    return aligned_to(workspace, 256) ? GS_OK : GS_EALIGN;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" int gs_attention_fwd(const gs_attention* a, const void* q, const void* k, const void* v,
                                const uint8_t* mask, const int32_t* q_lengths, const int32_t* k_lengths, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_shape(a);
    if (rc != GS_OK) return rc;
    if (a->batch == 0 || a->nq == 0) return GS_OK;
    if (!q || !out || (a->nk > 0 && (!k || !v)) || !no_strides_below_zero(a, false)) return GS_EINVAL;
    for (const void* t : {q, k, v, (const void*)out})
        if (!aligned_to(t, size_of(a->dtype))) return GS_EALIGN;
    for (const void* t : {(const void*)q_lengths, (const void*)k_lengths, (const void*)lse})
        if (!aligned_to(t, 4)) return GS_EALIGN;
    AttnArgs p = args_of(a, q, k, v, mask, q_lengths, k_lengths);
    p.out = out, p.lse = lse;
    rc = check_workspace(workspace, workspace_bytes, bytes_of(p, a->dtype).fwd);
    if (rc != GS_OK) return rc;
    hipStream_t s = as_stream(stream);
    if (a->dtype == GS_F32)
        attn_fwd<float>(p, workspace, s);
    else if (a->dtype == GS_F16)
        attn_fwd<_Float16>(p, workspace, s);
    else
        attn_fwd<__bf16>(p, workspace, s);
    return launch_status();
}

static int workspace_size(const gs_attention* a, size_t AttnBytes::*which, size_t* bytes) {
    const int rc = check_shape(a);
    if (rc != GS_OK) return rc;
    if (!bytes) return GS_EINVAL;
    *bytes = bytes_of(args_of(a, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), a->dtype).*which;
    return GS_OK;
}

extern "C" int gs_attention_fwd_workspace_size(const gs_attention* a, size_t* bytes) {
    return workspace_size(a, &AttnBytes::fwd, bytes);
}

extern "C" int gs_attention_bwd_workspace_size(const gs_attention* a, size_t* bytes) {
    return workspace_size(a, &AttnBytes::bwd, bytes);
}

extern "C" int gs_attention_bwd(const gs_attention* a, const void* q, const void* k, const void* v,
                                const uint8_t* mask, const int32_t* q_lengths, const int32_t* k_lengths,
                                const void* out, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_shape(a);
    if (rc != GS_OK) return rc;
    if (a->batch == 0 || (a->nq == 0 && a->nk == 0)) return GS_OK;
    if (a->nq > 0 && (!q || !out || !lse || !dout)) return GS_EINVAL;
    if ((a->nk > 0 && (!k || !v)) || !no_strides_below_zero(a, true)) return GS_EINVAL;
    for (const void* t : {q, k, v, out, dout, (const void*)dq, (const void*)dk, (const void*)dv})
        if (!aligned_to(t, size_of(a->dtype))) return GS_EALIGN;
    for (const void* t : {(const void*)q_lengths, (const void*)k_lengths, (const void*)lse})
        if (!aligned_to(t, 4)) return GS_EALIGN;
    AttnArgs p = args_of(a, q, k, v, mask, q_lengths, k_lengths);
    p.out = const_cast<void*>(out), p.lse = const_cast<float*>(lse), p.dout = dout;
    p.dq = dq, p.dk = dk, p.dv = dv;
    rc = check_workspace(workspace, workspace_bytes, bytes_of(p, a->dtype).bwd);
    if (rc != GS_OK) return rc;
    hipStream_t s = as_stream(stream);
    if (a->dtype == GS_F32)
        attn_bwd<float>(p, workspace, s);
    else if (a->dtype == GS_F16)
        attn_bwd<_Float16>(p, workspace, s);
    else
        attn_bwd<__bf16>(p, workspace, s);
    return launch_status();
}
