// attn_prologue.hip -- q/k RMS norm, rotary positions and the write of the new
// tokens' k and v into the pages of a KV cache (gfx950), in one launch.
//
// The packed attention prologue of the mstar pages ("q/k norm, rope, KV write
// in one kernel").  Per head of d values: y = x (add + w) / sqrt(mean x^2 +
// eps); the pair (u, v) at angle a = position * freq becomes s (u cos a - v sin
// a, v cos a + u sin a); the result is rounded once, to bf16 or to e4m3.
//
// The angle is formed in turns in fp64 and only its fraction, at most half a turn,
// goes on in fp32: that rounding is off by 2^-26 of a turn at most, 1e-7 rad, at any
// position (the fp64 part by 4e-10 rad at position 2^20, where an fp32 product would
// be off by 0.06).
//
// A workgroup owns one token (and, when there are few tokens, one slice of its
// heads): it forms the token's cos/sin table once in LDS, then every wave takes
// 512 / d heads at a time with 16-byte loads, d / 8 lanes a head.  All of them are
// loaded before the token's place is looked up and the table is made, so the
// memory's latency hides behind those.  A pair's partner sits in another lane at an offset that depends on
// rot and the layout, so the normed head goes through LDS: written and read by
// one wave, with no barrier.

#include "attn_common.h"

namespace gdn {

// NP: heads a group of lanes loads at a time.
template <int D, bool E4M3, int NP>
__global__ __launch_bounds__(256) void attn_prologue_kernel(AttnPrologueParams p)
{
    constexpr int LPH = D / 8;       // lanes a head
    constexpr int HPW = 64 / LPH;    // heads a wave at a time
    constexpr int HPB = 4 * HPW;     // heads a workgroup at a time
    __shared__ __align__(16) float2 turn[D / 2];
    __shared__ __align__(16) float stage[4][HPW][D + 4];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = blockIdx.x;
    const int lh = lane / LPH, c = lane % LPH;
    const int nq = p.q.p ? p.H_q : 0, nkv = p.k.p ? p.H_kv : 0;
    const int heads = nq + 2 * nkv;

    // the first heads' values, before anything that waits
    auto source = [&](int h) -> const uint16_t * {
        if (h < nq)
            return p.q.p + (int64_t)t * p.q.row + (int64_t)h * p.q.head;
        h -= nq;
        if (h < nkv)
            return p.k.p + (int64_t)t * p.k.row + (int64_t)h * p.k.head;
        return p.v.p + (int64_t)t * p.v.row + (int64_t)(h - nkv) * p.v.head;
    };
    const int wh = wave * HPW + lh;
    u32x4 raws[NP];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            raws[k] = u32x4{0u, 0u, 0u, 0u};
            if (base + k * HPB + wh < heads)
                raws[k] = *reinterpret_cast<const u32x4 *>(source(base + k * HPB + wh) + c * 8);
        }
    };
    const int base0 = blockIdx.y * (HPB * NP), stride = gridDim.y * (HPB * NP);
    load(base0);

    // the token's sequence: the last b with cu[b] <= t, 64 probes a round
    int lo = 0, hi = p.B; // cu[lo] <= t < cu[hi], if t is in any sequence
    const bool inside = p.cu[0] <= t && t < p.cu[p.B];
    if (!inside)
        return; // as it was
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && p.cu[at] <= t;
        const int n = __popcll(__ballot(le));
        lo += n * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    const int r = p.row[lo];
    // 0: fine, 1: padding (zeros), 2: unusable (NaN)
    int kind = r == 0 ? 1 : (r < 0 || r >= p.R ? 2 : 0);
    int pos = 0;
    int64_t cell = 0; // the token's place in a page of its own head 0
    if (kind == 0) {
        const int len = p.kv_len[r];
        pos = len - (p.cu[lo + 1] - t);
        if (len < 0 || pos < 0 || (nkv && pos >= (p.width << p.page_shift))) {
            kind = 2;
        } else if (nkv) {
            const int page = p.page_table[(int64_t)r * p.width + (pos >> p.page_shift)];
            if (page < 1 || page >= p.N)
                kind = 2;
            cell = (((int64_t)page * p.H_kv) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
    }
    const int half = p.rot >> 1;
    if (kind == 0) {
        const double at = (double)(p.positions ? p.positions[t] : pos);
        for (int j = tid; j < half; j += 256) {
            const double turns = at * (p.freqs[j] * 0.15915494309189533577);
            float sn, cs;
            sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
            turn[j] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
        }
    }
    __syncthreads();

    float *st = stage[wave][lh];
    for (int base = base0; base < heads; base += stride) {
        if (base != base0)
            load(base);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int h = base + k * HPB + wh;
            const bool on = h < heads;
            const u32x4 raw = raws[k];
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(raw[i] << 16);
                x[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
            }
            const bool is_q = h < nq, is_k = !is_q && h < nq + nkv;
            const uint16_t *w = is_q ? p.q_w : (is_k ? p.k_w : nullptr);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int m = 1; m < LPH; m <<= 1)
                sum += __shfl_xor(sum, m);
            if (on && w) {
                const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
                const u32x4 wr = *reinterpret_cast<const u32x4 *>(w + c * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = x[2 * i] * inv * (p.add + __uint_as_float(wr[i] << 16));
                    x[2 * i + 1] = x[2 * i + 1] * inv * (p.add + __uint_as_float(wr[i] & 0xffff0000u));
                }
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = x[i];
            const bool turns = on && (is_q || is_k) && kind == 0 && c * 8 < p.rot;
            if (p.interleaved) { // a pair's partner is in the lane
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 cs = turn[c * 4 + i];
                        if (c * 8 + 2 * i < p.rot) {
                            y[2 * i] = fmaf(-x[2 * i + 1], cs.y, x[2 * i] * cs.x);
                            y[2 * i + 1] = fmaf(x[2 * i], cs.y, x[2 * i + 1] * cs.x);
                        }
                    }
                }
            } else if (half) { // uniform; it is in another lane: through LDS, in this wave
                *reinterpret_cast<f32x4 *>(st + c * 8) = f32x4{x[0], x[1], x[2], x[3]};
                *reinterpret_cast<f32x4 *>(st + c * 8 + 4) = f32x4{x[4], x[5], x[6], x[7]};
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (turns) {
                    if ((half & 7) == 0) { // uniform; all eight partners stand side by side
                        const bool second = c * 8 >= half;
                        const int j = second ? c * 8 - half : c * 8;
                        const float *o = st + (second ? j : j + half);
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            const f32x4 z = *reinterpret_cast<const f32x4 *>(o + i);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float2 cs = turn[j + i + q];
                                y[i + q] = fmaf(second ? z[q] : -z[q], cs.y, x[i + q] * cs.x);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int e = c * 8 + i;
                            if (e < p.rot) {
                                const bool second = e >= half;
                                const int j = second ? e - half : e;
                                const float2 cs = turn[j];
                                const float o = st[second ? j : j + half];
                                y[i] = fmaf(second ? o : -o, cs.y, x[i] * cs.x);
                            }
                        }
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (!on)
                continue;
            if (is_q) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = kind == 0 ? pack_bf16(y[2 * i], y[2 * i + 1]) : (kind == 1 ? 0u : 0x7fc07fc0u);
                uint16_t *to = p.q_out.p + (int64_t)t * p.q_out.row + (int64_t)h * p.q_out.head + c * 8;
                *reinterpret_cast<u32x4 *>(to) = o;
            } else if (kind == 0) {
                const int hk = is_k ? h - nq : h - nq - nkv;
                const int64_t at = (cell + ((int64_t)hk << p.page_shift)) * D + c * 8;
                void *pages = is_k ? p.k_pages : p.v_pages;
                if constexpr (E4M3) {
                    const float s = (is_k ? p.k_scale : p.v_scale)[hk];
                    u32x2 o;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            z[k] = min_finite(y[4 * i + k] / s, 448.0f);
                        const int low = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
                        o[i] = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], low, true);
                    }
                    *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(pages) + at) = o;
                } else {
                    u32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_bf16(y[2 * i], y[2 * i + 1]);
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(pages) + at) = o;
                }
            }
        }
    }
}

template <int D, bool E4M3>
static hipError_t launch_de(const AttnPrologueParams &p, hipStream_t stream)
{
    const int heads = (p.q.p ? p.H_q : 0) + (p.k.p ? 2 * p.H_kv : 0);
    AttnPrologueParams q = p;
    void *args[] = {&q};
    // Few tokens: past the heads that one pass takes, more workgroups a token, so that every load
    // leaves at once.  Many: one a token, which forms the angles once and loads three passes ahead
    // (8570 tokens of 16 + 4 heads of 256: the kernel alone 48.2 us, a call 46.6 to 48.2, 3.7 TB/s, into an
    // e4m3 cache 56.5; a wave a token instead 50.5 alone against 48.5).  First way / second: 512 tokens of
    // 16 + 4 heads of 256 12.0 / 11.4 us a call (the host's time), 1024 tokens 11.9 / 12.1, 2048 tokens
    // 17.2 / 13.8, 4096 tokens 28.9 / 22.6.
    const int per = 4 * 512 / D;
    if (p.T < 1024)
        return hipLaunchKernel(reinterpret_cast<const void *>(&attn_prologue_kernel<D, E4M3, 1>),
                               dim3((unsigned)p.T, (unsigned)((heads + per - 1) / per)), dim3(256), args, 0, stream);
    return hipLaunchKernel(reinterpret_cast<const void *>(&attn_prologue_kernel<D, E4M3, 3>), dim3((unsigned)p.T),
                           dim3(256), args, 0, stream);
}

template <int D>
static hipError_t launch_d(const AttnPrologueParams &p, bool e4m3, hipStream_t stream)
{
    return e4m3 ? launch_de<D, true>(p, stream) : launch_de<D, false>(p, stream);
}

hipError_t launch_attn_prologue(const AttnPrologueParams &p, int d, bool e4m3, hipStream_t stream)
{
    return d == 64 ? launch_d<64>(p, e4m3, stream)
                   : (d == 128 ? launch_d<128>(p, e4m3, stream) : launch_d<256>(p, e4m3, stream));
}

} // namespace gdn
