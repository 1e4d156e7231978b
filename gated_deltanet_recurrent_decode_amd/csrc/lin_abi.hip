// lin_abi.hip -- the extern "C" boundary of linear attention: host-side validation, then the launches on the
// caller's stream.  Nothing here allocates, synchronises or reads device memory.  Contracts: include/gdn.h.

#include <math.h>
#include <stdint.h>

#include "gdn.h"
#include "lin_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

gdn_status from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

gdn_status check_dims(const gdn_lin_dims &d)
{
    if (d.B < 0 || d.T < 0 || d.H_k < 1 || d.H_v < 1 || d.H_v % d.H_k != 0 || d.N < 1 || d.per_token < 0 ||
        d.per_token > 1)
        return GDN_ERR_SHAPE;
    if ((d.d_k != 64 && d.d_k != 128) || (d.d_v != 64 && d.d_v != 128))
        return GDN_ERR_UNSUPPORTED;
    // a launch counts its threads in 32 bits: up to 4096 for a sequence and head
    return (int64_t)d.B * d.H_v >= 1 << 20 || d.T >= 1 << 30 ? GDN_ERR_SHAPE : GDN_OK;
}

gdn_status check_heads(const gdn_heads &h)
{
    // a chunk's rows, and a few heads of them, are addressed in 32 bits
    if (h.row_stride < 0 || h.head_stride < 0 || h.row_stride > 1 << 24 || h.head_stride > 1 << 24)
        return GDN_ERR_SHAPE;
    return !aligned(h.data, 16) || h.row_stride % 8 != 0 || h.head_stride % 8 != 0 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn::Heads heads_of(const gdn_heads &h) { return gdn::Heads{h.data, h.row_stride, h.head_stride}; }

// What the calls share; `tokens`: there are some, so their arrays are needed.
gdn_status check_arrays(const gdn_heads *q, const gdn_heads *k, const gdn_heads *v, const gdn_heads *out,
                        const float *g, const float *state, float q_scale, bool tokens, bool per_token)
{
    if (!q || !k || !v || !out || !state || (!g && (tokens || !per_token)))
        return GDN_ERR_NULL;
    for (const gdn_heads *h : {q, k, v, out}) {
        if (tokens && !h->data)
            return GDN_ERR_NULL;
        const gdn_status st = check_heads(*h);
        if (st != GDN_OK)
            return st;
    }
    if (!isfinite(q_scale))
        return GDN_ERR_SHAPE;
    return !aligned(state, 16) || !aligned(g, 4) ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn_status step_impl(const gdn_lin_dims *dims, const gdn_heads *q, const gdn_heads *k, const gdn_heads *v,
                     const float *g, float *state, const int32_t *read_slot, const int32_t *write_slot,
                     const int32_t *token_slots, const gdn_heads *out, float q_scale, hipStream_t stream)
{
    const gdn_lin_dims d = *dims;
    gdn_status st = check_dims(d);
    if (st != GDN_OK)
        return st;
    if (d.T < 1 || (int64_t)d.B * d.T >= 1 << 30)
        return GDN_ERR_SHAPE;
    if (!read_slot)
        return GDN_ERR_NULL;
    if ((st = check_arrays(q, k, v, out, g, state, q_scale, true, d.per_token == 1)) != GDN_OK)
        return st;
    gdn::LinStepParams p{};
    p.q = heads_of(*q);
    p.k = heads_of(*k);
    p.v = heads_of(*v);
    p.out = heads_of(*out);
    p.g = g;
    p.state = state;
    p.read_slot = read_slot;
    p.write_slot = write_slot;
    p.token_slots = token_slots;
    p.q_scale = q_scale;
    p.B = d.B;
    p.T = d.T;
    p.H_k = d.H_k;
    p.H_v = d.H_v;
    p.N = d.N;
    p.per_token = d.per_token;
    return from_hip(gdn::launch_lin_step(p, d.d_k, d.d_v, stream));
}

} // namespace

extern "C" {

gdn_status lin_attn_step(const gdn_lin_dims *dims, const gdn_heads *q, const gdn_heads *k, const gdn_heads *v,
                         const float *g, float *state, const int32_t *read_slot, const int32_t *write_slot,
                         const gdn_heads *out, float q_scale, hipStream_t stream)
{
    if (!dims)
        return GDN_ERR_NULL;
    if (dims->B == 0)
        return GDN_OK;
    return step_impl(dims, q, k, v, g, state, read_slot, write_slot, nullptr, out, q_scale, stream);
}

gdn_status lin_attn_step_tokens(const gdn_lin_dims *dims, const gdn_heads *q, const gdn_heads *k, const gdn_heads *v,
                                const float *g, float *state, const int32_t *read_slot, const int32_t *token_slots,
                                const gdn_heads *out, float q_scale, hipStream_t stream)
{
    if (!dims)
        return GDN_ERR_NULL;
    if (dims->B == 0)
        return GDN_OK;
    if (!token_slots)
        return GDN_ERR_NULL;
    return step_impl(dims, q, k, v, g, state, read_slot, nullptr, token_slots, out, q_scale, stream);
}

size_t lin_attn_prefill_workspace_bytes(const gdn_lin_dims *dims)
{
    if (!dims || check_dims(*dims) != GDN_OK)
        return 0;
    return gdn::lin_prefill_layout(dims->B, dims->T, dims->H_k, dims->H_v, dims->d_k, dims->d_v, nullptr, nullptr);
}

gdn_status lin_attn_prefill(const gdn_lin_dims *dims, const gdn_heads *q, const gdn_heads *k, const gdn_heads *v,
                            const float *g, const int32_t *cu_seqlens, float *state, const int32_t *read_slot,
                            const int32_t *write_slot, const gdn_heads *out, float q_scale, void *workspace,
                            size_t workspace_bytes, hipStream_t stream)
{
    if (!dims)
        return GDN_ERR_NULL;
    const gdn_lin_dims d = *dims;
    if (d.B == 0)
        return GDN_OK;
    gdn_status st = check_dims(d);
    if (st != GDN_OK)
        return st;
    if (!cu_seqlens || !read_slot || !workspace)
        return GDN_ERR_NULL;
    if ((st = check_arrays(q, k, v, out, g, state, q_scale, d.T > 0, d.per_token == 1)) != GDN_OK)
        return st;
    if (!aligned(workspace, 256))
        return GDN_ERR_UNSUPPORTED;
    gdn::LinPrefillParams p{};
    if (workspace_bytes < gdn::lin_prefill_layout(d.B, d.T, d.H_k, d.H_v, d.d_k, d.d_v, workspace, &p) ||
        (int64_t)p.segments * d.H_v >= 1 << 23) // 256 threads each, rounded up, of 2^32
        return GDN_ERR_SHAPE;
    p.q = heads_of(*q);
    p.k = heads_of(*k);
    p.v = heads_of(*v);
    p.out = heads_of(*out);
    p.g = g;
    p.state = state;
    p.cu = cu_seqlens;
    p.read_slot = read_slot;
    p.write_slot = write_slot;
    p.q_scale = q_scale;
    p.B = d.B;
    p.T = d.T;
    p.H_k = d.H_k;
    p.H_v = d.H_v;
    p.N = d.N;
    p.per_token = d.per_token;
    return from_hip(gdn::launch_lin_prefill(p, d.d_k, d.d_v, stream));
}

} // extern "C"
