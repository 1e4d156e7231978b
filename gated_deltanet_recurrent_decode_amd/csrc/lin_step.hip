// lin_step.hip -- linear attention with a decay for each head: one token a row, or a few (gfx950).
//
// S <- e^g S + k v^T, o = q_scale S^T q, for each (row, value head).  A workgroup takes one head's state: a
// wave 32 of its columns and all its rows, a thread d_k/8 consecutive rows of four columns, so that its
// values of q and k are 16-byte loads and the read-out's sum over the rows ends inside the wave (in the
// thread, then over lane bits 3 to 5).
//
// What bounds it: the state, read once and written once.  MI355X, calls back to back: 64 rows at 16 heads of 128 x 128
// 26.4 us (5.1 TB/s, as a large copy), 24 rows of 4 tokens at 32 heads of 128 x 64 with all states kept 24.0 (5.3
// TB/s); one row 4.5 us of a kernel, what a launch costs.

#include "attn_common.h"
#include "lin_internal.h"
#include "step_common.h"

namespace gdn {

template <int DK, int DV, bool TOKENS>
__global__ __launch_bounds__(2 * DV) void lin_step_kernel(LinStepParams p)
{
    constexpr int RPT = DK / 8; // rows of a thread
    constexpr uint32_t TILE = (uint32_t)DK * DV * 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int rg = lane >> 3, col = wave * 32 + (lane & 7) * 4;
    const int r = blockIdx.x / p.H_v, hv = blockIdx.x % p.H_v, hk = hv / (p.H_v / p.H_k);

    const int rs = p.read_slot[r];
    const int ws = TOKENS ? 0 : (p.write_slot ? p.write_slot[r] : rs);
    const uint32_t n = (uint32_t)p.N;
    // a slot out of range, a row that would write the null slot, or with token slots its own read slot
    bool bad = ((uint32_t)rs >= n) | ((uint32_t)ws >= n) | (!TOKENS & (rs != 0) & (ws == 0)) |
               (!TOKENS & (p.write_slot != nullptr) & (rs != 0) & (ws == rs));
    if constexpr (TOKENS)
        for (int t = 0; t < p.T; ++t) {
            const int ts = p.token_slots[(int64_t)r * p.T + t];
            bad |= ((uint32_t)ts >= n) | ((rs != 0) & (ts == rs));
        }
    const bool real = rs != 0 && !bad;

    // unusable rows read through an empty resource: the loads leave without waiting for a branch
    const __amdgpu_buffer_rsrc_t rd =
        tile_rsrc(p.state + ((size_t)(real ? rs : 0) * p.H_v + hv) * (DK * DV), real ? TILE : 0u);
    const uint32_t voff = (uint32_t)((rg * RPT * DV + col) * 4);
    float4 s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        s[m] = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(rd, voff, m * DV * 4, kLoadPolicy));

    const uint16_t *qp = p.q.p + (int64_t)r * p.T * p.q.row + (int64_t)hk * p.q.head + rg * RPT;
    const uint16_t *kp = p.k.p + (int64_t)r * p.T * p.k.row + (int64_t)hk * p.k.head + rg * RPT;
    const uint16_t *vp = p.v.p + (int64_t)r * p.T * p.v.row + (int64_t)hv * p.v.head + col;
    uint16_t *op = p.out.p + (int64_t)r * p.T * p.out.row + (int64_t)hv * p.out.head + col;
    for (int t = 0; t < p.T; ++t) {
        if (!real) {
            const uint32_t y = rs == 0 ? 0u : 0x7fc07fc0u;
            if (rg == 0)
                *reinterpret_cast<u32x2 *>(op) = u32x2{y, y};
            op += p.out.row;
            continue;
        }
        u32x4 kk[RPT / 8], qq[RPT / 8];
#pragma unroll
        for (int i = 0; i < RPT / 8; ++i) {
            kk[i] = reinterpret_cast<const u32x4 *>(kp)[i];
            qq[i] = reinterpret_cast<const u32x4 *>(qp)[i];
        }
        const u32x2 vv = *reinterpret_cast<const u32x2 *>(vp);
        const float decay = expf(p.g[p.per_token ? ((int64_t)r * p.T + t) * p.H_v + hv : hv]);
        const float v0 = __uint_as_float(vv[0] << 16), v1 = __uint_as_float(vv[0] & 0xffff0000u),
                    v2 = __uint_as_float(vv[1] << 16), v3 = __uint_as_float(vv[1] & 0xffff0000u);
        float4 o = f4_zero();
#pragma unroll
        for (int m = 0; m < RPT; ++m) {
            const uint32_t kw = kk[m / 8][m % 8 / 2], qw = qq[m / 8][m % 8 / 2];
            const float k = __uint_as_float(m & 1 ? kw & 0xffff0000u : kw << 16);
            const float q = __uint_as_float(m & 1 ? qw & 0xffff0000u : qw << 16);
            s[m].x = fmaf(k, v0, decay * s[m].x);
            s[m].y = fmaf(k, v1, decay * s[m].y);
            s[m].z = fmaf(k, v2, decay * s[m].z);
            s[m].w = fmaf(k, v3, decay * s[m].w);
            o.x = fmaf(q, s[m].x, o.x);
            o.y = fmaf(q, s[m].y, o.y);
            o.z = fmaf(q, s[m].z, o.z);
            o.w = fmaf(q, s[m].w, o.w);
        }
        o.x = xor_sum<8>(o.x);
        o.y = xor_sum<8>(o.y);
        o.z = xor_sum<8>(o.z);
        o.w = xor_sum<8>(o.w);
        if (rg == 0)
            *reinterpret_cast<u32x2 *>(op) = u32x2{pack_bf16(o.x * p.q_scale, o.y * p.q_scale),
                                                   pack_bf16(o.z * p.q_scale, o.w * p.q_scale)};
        qp += p.q.row;
        kp += p.k.row;
        vp += p.v.row;
        op += p.out.row;
        const int to = TOKENS ? p.token_slots[(int64_t)r * p.T + t] : (t + 1 == p.T ? ws : 0);
        if (to != 0) {
            const __amdgpu_buffer_rsrc_t wr = tile_rsrc(p.state + ((size_t)to * p.H_v + hv) * (DK * DV), TILE);
#pragma unroll
            for (int m = 0; m < RPT; ++m)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, s[m]), wr, voff, m * DV * 4,
                                                       kStorePolicy);
        }
    }
}

template <int DK, int DV>
static hipError_t launch_step(const LinStepParams &p, hipStream_t stream)
{
    LinStepParams q = p;
    void *args[] = {&q};
    const void *f = p.token_slots ? reinterpret_cast<const void *>(&lin_step_kernel<DK, DV, true>)
                                  : reinterpret_cast<const void *>(&lin_step_kernel<DK, DV, false>);
    return hipLaunchKernel(f, dim3((unsigned)(p.B * p.H_v)), dim3(2 * DV), args, 0, stream);
}

hipError_t launch_lin_step(const LinStepParams &p, int d_k, int d_v, hipStream_t stream)
{
    if (d_k == 64)
        return d_v == 64 ? launch_step<64, 64>(p, stream) : launch_step<64, 128>(p, stream);
    return d_v == 64 ? launch_step<128, 64>(p, stream) : launch_step<128, 128>(p, stream);
}

} // namespace gdn
