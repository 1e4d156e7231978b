// lin_internal.h -- parameter blocks and launchers of linear attention with decay.
#pragma once

#include "attn_internal.h"

namespace gdn {

struct LinStepParams {
    Heads q, k, v, out;        // token r*T + t
    const float *g;            // log decays [H_v] or [B][T][H_v]
    float *state;              // [N][H_v][d_k][d_v]
    const int32_t *read_slot, *write_slot, *token_slots;
    float q_scale;
    int B, T, H_k, H_v, N, per_token;
};

struct LinPrefillParams {
    Heads q, k, v, out;
    const float *g;            // [H_v] or [T][H_v]
    float *state;
    const int32_t *cu, *read_slot, *write_slot;
    float *entry;              // workspace [segments][H_v][d_k][d_v]: the state that a segment begins with
    float *decay;              // workspace [segments][H_v]: what is left of it at the segment's end
    float q_scale;
    int B, T, H_k, H_v, N, per_token;
    int segment;               // tokens of a segment, a multiple of a chunk
    int segments;              // the most that the call can have: T / segment + B
};

hipError_t launch_lin_step(const LinStepParams &p, int d_k, int d_v, hipStream_t stream);
hipError_t launch_lin_prefill(const LinPrefillParams &p, int d_k, int d_v, hipStream_t stream);
// device scratch in bytes; fills the parameter block's pointers and segment sizes when it is given
size_t lin_prefill_layout(int B, int T, int H_k, int H_v, int d_k, int d_v, void *base, LinPrefillParams *p);

} // namespace gdn
