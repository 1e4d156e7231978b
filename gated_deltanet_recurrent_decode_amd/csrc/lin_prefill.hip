// lin_prefill.hip -- linear attention with a decay for each head over packed prompts, chunked (gfx950).
//
// With G_i the sum of the log decays of a chunk's tokens up to i, the recurrence S <- e^g S + k v^T,
// o = S^T q becomes, for a chunk that begins with state S,
//   o_i = e^(G_i) S^T q_i + sum_(j <= i) e^(G_i - G_j) (q_i . k_j) v_j,
//   S'  = e^(G_end) S + sum_j k_j (e^(G_end - G_j) v_j)^T.
// A workgroup walks the chunks of one value head, a wave 32 columns of v with all rows of S in its
// accumulators, so that S never leaves the registers.  Everything is a 32 x 32 x 16 bf16 product.  An operand
// that fp32 work made goes there as several bf16 numbers: as two (off by at most 2^-15 of itself) where the
// result is a read-out, which is rounded to bf16, and as three (all of its bits) where it is a state, which
// stays in fp32: P^T = K Q^T, O^T = S^T Q^T, O^T += V^T P^T, S += K^T V'.  The layouts meet with no exchange
// between lanes: rows of an accumulator are the contraction's places of the next product.  For that the rows
// of S lie in the order that the transposing reads of K give them, which is chosen so that a lane's eight
// rows are eight consecutive d_k (one 16-byte read of q and k), and the columns of v likewise (16-byte stores
// of o).
//
// A long prompt has more tokens than one workgroup should walk: it is cut into segments.  A first kernel
// forms each segment's own part of the state, a second carries them on along the prompt, and the walk then
// begins every segment with its state.

#include <type_traits>

#include "attn_common.h"
#include "gdn_internal.h"
#include "lin_internal.h"

namespace gdn {

namespace {

constexpr int C = 32; // tokens of a chunk

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint8_t lds_byte;

// Weights below 2^-149 are zero in fp32: a log2 decay is cut here, so that sums of them stay finite.
constexpr float kLeast = -256.0f;

__device__ __forceinline__ float log2_decay(float g)
{
    const float x = g * 1.44269504088896340736f;
    return x < kLeast ? kLeast : x; // a NaN stays
}

// 16 bytes a lane from base + off into LDS, lane after lane from `to` on.  As inline assembly because
// the compiler, given the builtin, waits for it before any read of LDS.  Whoever reads `to` waits for
// vmcnt(0) and a barrier first.
__device__ __forceinline__ void load_to_lds(lds_byte *to, const uint8_t *base, int off)
{
    const uint32_t at = (uint32_t)(uintptr_t)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform((int)at)), "v"(off),
                 "s"(base)
                 : "memory"); // m0 is reserved: whatever of the compiler's own needs it sets it first
}

// A segment of a sequence.  Segment s of sequence b has place cu[b] / segment + b + s: no two the same, and
// all below T / segment + B.
struct Segment {
    int b;             // sequence, -1: none
    int first, n;      // its tokens
    int s, count;      // segment, segments of the sequence
    int read, write;   // slots
    bool pad, bad;     // a padding sequence, an unusable one
};

__device__ __forceinline__ Segment sequence_of(const LinPrefillParams &p, int b)
{
    Segment x;
    x.b = b;
    x.first = p.cu[b];
    const int e = p.cu[b + 1];
    x.n = e - x.first;
    x.s = 0;
    x.read = p.read_slot[b];
    x.write = p.write_slot ? p.write_slot[b] : x.read;
    if (x.first < 0 || e > p.T || e < x.first)
        x.b = -1;
    x.count = x.n > 0 ? (x.n + p.segment - 1) / p.segment : 1;
    x.pad = x.read == 0 && x.write == 0;
    x.bad = (uint32_t)x.read >= (uint32_t)p.N || (uint32_t)x.write >= (uint32_t)p.N || (x.read != 0 && x.write == 0);
    return x;
}

// The segment at a place: the last sequence whose first place is not behind it.
__device__ __forceinline__ Segment segment_at(const LinPrefillParams &p, int place)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = p.B; // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && p.cu[at] / p.segment + at <= place;
        const int n = __popcll(__ballot(le));
        lo += n * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    lo = uniform(lo);
    Segment x = sequence_of(p, lo);
    if (x.b < 0)
        return x;
    x.s = place - (x.first / p.segment + lo);
    if (x.s < 0 || x.s >= x.count) {
        x.b = -1;
        return x;
    }
    x.n = uniform(x.s + 1 < x.count ? p.segment : x.n - x.s * p.segment);
    x.first = uniform(x.first + x.s * p.segment);
    return x;
}

// Row of an accumulator's 16 to place among 16: blocks of four, the middle two exchanged, so that a lane's
// two blocks (rows 4h.. and 8 + 4h..) stand for eight consecutive values.
__device__ __forceinline__ int swapped(int m) { return (m & 19) | ((m & 4) << 1) | ((m & 8) >> 1); }

template <int D>
__device__ __forceinline__ int swizzle(int key) // place of a 16-byte chunk within its row of D values
{
    return D == 64 ? (((key >> 1) & 1) << 2) | ((key >> 2) & 3) : ((key & 3) << 2) | ((key >> 2) & 3);
}

// A value as two bf16 numbers, pairs packed: its upper half and what that leaves.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = __builtin_amdgcn_perm(y, x, 0x07060302u);
    lo = pack_bf16(a - __uint_as_float(x & 0xffff0000u), b - __uint_as_float(y & 0xffff0000u));
}

// And as three, which hold all of its 24 bits.
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = __builtin_amdgcn_perm(y, x, 0x07060302u);
    split2(a - __uint_as_float(x & 0xffff0000u), b - __uint_as_float(y & 0xffff0000u), mid, lo);
}

__device__ __forceinline__ bf16x8 operand(const uint32_t (&x)[4])
{
    return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], x[2], x[3]});
}

__device__ __forceinline__ bool not_finite(uint32_t pair)
{
    return (pair & 0x7f80u) == 0x7f80u || (pair & 0x7f800000u) == 0x7f800000u;
}

} // namespace

// OUT: the walk, with read-outs.  Otherwise a segment's own part of the state, for all but a
// sequence's last.
template <int DK, int DV, bool OUT>
__global__ __launch_bounds__(2 * DV, 2) void lin_prefill_kernel(LinPrefillParams p)
{
    constexpr int NW = DV / 32, NT = 64 * NW;
    constexpr int TK = DK / 32;             // 32-row tiles of S
    constexpr int KB = C * DK * 2, VB = C * DV * 2; // bytes of a chunk's k (and q), v
    constexpr int BUF = (OUT ? 2 : 1) * KB + VB;
    __shared__ __align__(16) uint8_t sm[2][BUF];
    __shared__ __align__(16) float sm_hi[NW][C], sm_lo[NW][C];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n_ = lane & 31, hh = lane >> 5;
    // consecutive items (heads fastest) on one XCD: heads that share q and k meet in its L2
    const int items = p.segments * p.H_v, per = (items + 7) >> 3;
    const int item = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (item >= items || (int)(blockIdx.x >> 3) >= per)
        return;
    const int place = item / p.H_v, hv = item % p.H_v, hk = hv / (p.H_v / p.H_k);
    const Segment sg = segment_at(p, place);
    if (sg.b < 0)
        return;
    if (sg.pad || sg.bad) {
        if constexpr (OUT) {
            const uint32_t y = sg.pad ? 0u : 0x7fc07fc0u;
            for (int x = tid; x < sg.n * (DV / 8); x += NT)
                *reinterpret_cast<u32x4 *>(p.out.p + (int64_t)(sg.first + x / (DV / 8)) * p.out.row +
                                           (int64_t)hv * p.out.head + x % (DV / 8) * 8) = u32x4{y, y, y, y};
        }
        return;
    }
    const bool last = sg.s + 1 == sg.count;
    if (!OUT && (last || place + 1 >= p.segments)) // the second: sequences that overlap
        return;

    // this lane's column of v, and the rows of S
    const int col = wave * 32 + swapped(n_);
    const int64_t tile = (int64_t)DK * DV;
    auto row_of = [&](int t, int i) { return 32 * t + 16 * (i >> 3) + 8 * hh + (i & 7); };
    f32x16 S[TK];
    const float *from = nullptr;
    if (OUT && sg.count > 1)
        from = p.entry + ((int64_t)place * p.H_v + hv) * tile;
    else if (sg.s == 0 && sg.read != 0)
        from = p.state + ((int64_t)sg.read * p.H_v + hv) * tile;
    if (from) {
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                S[t][i] = from[row_of(t, i) * DV + col];
    } else {
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                S[t][i] = 0.f;
    }
    auto store_state = [&](float *to) {
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                to[row_of(t, i) * DV + col] = S[t][i];
    };
    if (!OUT && sg.s == 0) // the walk may find the slot already written: it begins from this copy
        store_state(p.entry + ((int64_t)place * p.H_v + hv) * tile);

    // staging: 1 KiB an instruction, whole rows, chunks of 16 bytes in the order of their row
    auto stage = [&](auto width, const Heads &x, int head, lds_byte *to, int c0) {
        constexpr int D = decltype(width)::value, CH = D / 8, RP = 64 / CH;
        const int rows = sg.n - c0 < C ? sg.n - c0 : C;
        const uint64_t from =
            reinterpret_cast<uint64_t>(x.p + (int64_t)(sg.first + c0) * x.row + (int64_t)head * x.head);
        const uint8_t *base = reinterpret_cast<const uint8_t *>(
            (uint64_t)(uint32_t)uniform((int)(from >> 32)) << 32 | (uint32_t)uniform((int)from));
#pragma unroll
        for (int i = 0; i < C / RP / NW; ++i) {
            const int r0 = (i * NW + wave) * RP, r = r0 + lane / CH;
            const int rr = r < rows ? r : rows - 1; // rows past the last repeat it
            load_to_lds(to + r0 * D * 2, base, rr * (int)x.row * 2 + ((lane % CH) ^ swizzle<D>(r)) * 16);
        }
    };
    const std::integral_constant<int, DK> width_k;
    const std::integral_constant<int, DV> width_v;
    auto bring = [&](int buf, int c0) {
        lds_byte *to = (lds_byte *)sm + buf * BUF;
        stage(width_k, p.k, hk, to, c0);
        stage(width_v, p.v, hv, to + KB, c0);
        if constexpr (OUT)
            stage(width_k, p.q, hk, to + KB + VB, c0);
    };
    // a token's log decay, of this lane's token of a chunk
    auto decay_of = [&](int c0) {
        const int t = c0 + n_;
        return t < sg.n ? p.g[p.per_token ? (int64_t)(sg.first + t) * p.H_v + hv : hv] : 0.f;
    };

    // transposing reads: lane (hv, r, c) points at key 4 hv + r (+ 8 for the second), columns 4 c
    const int gr = lane >> 4, r_ = (lane & 15) >> 2, c_ = swapped((lane & 3) << 2) >> 2;
    int tk_at[2], tv_at[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int key = 8 * y + 4 * (gr >> 1) + r_, chunk = (gr & 1) * 2 + (c_ >> 1);
        tk_at[y] = key * DK * 2 + ((chunk ^ swizzle<DK>(key)) * 16) + (c_ & 1) * 8;
        tv_at[y] = key * DV * 2 + (((wave * 4 + chunk) ^ swizzle<DV>(key)) * 16) + (c_ & 1) * 8;
    }
    auto transposed = [&](const uint8_t *at0, const uint8_t *at1, uint32_t (&x)[4]) {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at0));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at1));
        x[0] = a[0];
        x[1] = a[1];
        x[2] = b[0];
        x[3] = b[1];
    };

    float total = 1.f; // what the segment leaves of the state that it begins with
    float g_next = decay_of(0);
    if (sg.n > 0)
        bring(0, 0);
    for (int c0 = 0, buf = 0; c0 < sg.n; c0 += C, buf ^= 1) {
        const float g = g_next;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // this wave's part of the chunk is in LDS
        __syncthreads();
        if (c0 + C < sg.n) {
            g_next = decay_of(c0 + C);
            bring(buf ^ 1, c0 + C);
        }
        const int rows = sg.n - c0 < C ? sg.n - c0 : C;
        const uint8_t *kb = sm[buf], *vb = kb + KB, *qb = vb + VB;

        // G_n of this lane's token, in 64 bits, as two fp32 numbers: differences of large sums keep their bits
        double G = n_ < rows ? (double)log2_decay(g) : 0.0;
#pragma unroll
        for (int m = 1; m < C; m <<= 1) {
            const double o = __shfl_up(G, m, 32);
            if (n_ >= m)
                G += o;
        }
        const float G_hi = (float)G, G_lo = (float)(G - (double)G_hi);
        if (hh == 0) {
            sm_hi[wave][n_] = G_hi;
            sm_lo[wave][n_] = G_lo;
        }
        const float E_hi = __shfl(G_hi, 31), E_lo = __shfl(G_lo, 31);
        const float keep = __builtin_amdgcn_exp2f(E_hi + E_lo);
        total *= keep;
        __builtin_amdgcn_wave_barrier();
        f32x4 K_hi[4], K_lo[4]; // of the keys of this lane's rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            K_hi[i] = *reinterpret_cast<const f32x4 *>(&sm_hi[wave][8 * i + 4 * hh]);
            K_lo[i] = *reinterpret_cast<const f32x4 *>(&sm_lo[wave][8 * i + 4 * hh]);
        }

        uint32_t vf[2][4]; // v: column `col`, 16 keys each
#pragma unroll
        for (int u = 0; u < 2; ++u)
            transposed(vb + u * 16 * DV * 2 + tv_at[0], vb + u * 16 * DV * 2 + tv_at[1], vf[u]);

        if constexpr (OUT) {
            f32x16 P, O;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                P[i] = O[i] = 0.f;
#pragma unroll
            for (int t = 0; t < TK; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int chunk = t * 4 + u * 2 + hh;
                    const int at = n_ * DK * 2 + ((chunk ^ swizzle<DK>(n_)) * 16);
                    const bf16x8 qf = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(qb + at));
                    const bf16x8 kf = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(kb + at));
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split2(S[t][8 * u + 2 * e], S[t][8 * u + 2 * e + 1], hi[e], lo[e]);
                    P = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf, P, 0, 0, 0);
                    O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(hi), qf, O, 0, 0, 0);
                    O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(lo), qf, O, 0, 0, 0);
                }
            settle(P);
            settle(O);
            const float begin = __builtin_amdgcn_exp2f(G_hi + G_lo);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                O[i] *= begin;
            // An infinity or NaN in v must not reach tokens before it (0 times it is NaN): it leaves this
            // product, and from its token on the column becomes NaN.
            bool odd = false;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    odd |= not_finite(vf[u][e]);
            uint32_t vc[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    vc[u][e] = vf[u][e];
            if (__ballot(odd)) {
                int since = C; // the first such key of this lane's column
#pragma unroll
                for (int u = 1; u >= 0; --u)
#pragma unroll
                    for (int e = 3; e >= 0; --e) {
                        const int key = 16 * u + (e >> 1) * 8 + 4 * hh + (e & 1) * 2;
                        if ((vc[u][e] & 0x7f800000u) == 0x7f800000u) {
                            vc[u][e] &= 0xffffu;
                            since = key + 1 < since ? key + 1 : since;
                        }
                        if ((vc[u][e] & 0x7f80u) == 0x7f80u) {
                            vc[u][e] &= 0xffff0000u;
                            since = key < since ? key : since;
                        }
                    }
                const int other = __shfl_xor(since, 32);
                since = other < since ? other : since;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n_ >= __shfl(since, 8 * (i >> 2) + 4 * hh + (i & 3)))
                        O[i] = quiet_nan();
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float w[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int i = 8 * u + 2 * e + y, key = 8 * (i >> 2) + 4 * hh + (i & 3);
                        const float d = (G_hi - K_hi[i >> 2][i & 3]) + (G_lo - K_lo[i >> 2][i & 3]);
                        w[y] = key <= n_ ? P[i] * __builtin_amdgcn_exp2f(d) : 0.f;
                    }
                    split2(w[0], w[1], hi[e], lo[e]);
                }
                O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(vc[u]), operand(hi), O, 0, 0, 0);
                O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(vc[u]), operand(lo), O, 0, 0, 0);
            }
            settle(O);
            if (n_ < rows) {
                uint16_t *o = p.out.p + (int64_t)(sg.first + c0 + n_) * p.out.row + (int64_t)hv * p.out.head +
                              wave * 32 + 8 * hh;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = pack_bf16(O[8 * u + 2 * e] * p.q_scale, O[8 * u + 2 * e + 1] * p.q_scale);
                    *reinterpret_cast<u32x4 *>(o + 16 * u) = u32x4{y[0], y[1], y[2], y[3]};
                }
            }
        }

        // the state behind the chunk
#pragma unroll
        for (int t = 0; t < TK; ++t)
            S[t] *= keep;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float w[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int i = 8 * u + 2 * e + y, key = 8 * (i >> 2) + 4 * hh + (i & 3);
                    const float d = (E_hi - K_hi[i >> 2][i & 3]) + (E_lo - K_lo[i >> 2][i & 3]);
                    const float v = __uint_as_float(y ? vf[u][e] & 0xffff0000u : vf[u][e] << 16);
                    w[y] = key < rows ? v * __builtin_amdgcn_exp2f(d) : 0.f;
                }
                split3(w[0], w[1], hi[e], mid[e], lo[e]);
            }
#pragma unroll
            for (int t = 0; t < TK; ++t) {
                uint32_t kt[4];
                const int o = u * 16 * DK * 2, x = t * 64;
                transposed(kb + o + (tk_at[0] ^ x), kb + o + (tk_at[1] ^ x), kt);
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt), operand(hi), S[t], 0, 0, 0);
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt), operand(mid), S[t], 0, 0, 0);
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt), operand(lo), S[t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < TK; ++t)
            settle(S[t]);
    }
    if constexpr (OUT) {
        if (last)
            store_state(p.state + ((int64_t)sg.write * p.H_v + hv) * tile);
    } else {
        store_state(p.entry + ((int64_t)(place + 1) * p.H_v + hv) * tile);
        if (tid == 0)
            p.decay[(int64_t)(place + 1) * p.H_v + hv] = total;
    }
}

// Along each sequence: what a segment begins with is what the one before left by itself, and what its decay
// left of its own beginning.
template <int DK, int DV>
__global__ __launch_bounds__(256) void lin_carry_kernel(LinPrefillParams p)
{
    constexpr int PARTS = DK * DV / 1024, BATCH = 4;
    const int b = blockIdx.x / (p.H_v * PARTS), rest = blockIdx.x % (p.H_v * PARTS);
    const int hv = rest / PARTS, part = rest % PARTS;
    const Segment sg = sequence_of(p, b);
    if (sg.b < 0 || sg.pad || sg.bad || sg.count < 3)
        return;
    const int place = sg.first / p.segment + b;
    const int count = sg.count < p.segments - place ? sg.count : p.segments - place;
    const int64_t step = (int64_t)p.H_v * DK * DV / 4;
    f32x4 *at = reinterpret_cast<f32x4 *>(p.entry) + ((int64_t)(place + 1) * p.H_v + hv) * (DK * DV / 4) +
                part * 256 + threadIdx.x;
    const float *decay = p.decay + (int64_t)(place + 1) * p.H_v + hv;
    f32x4 x = at[0];
    for (int s = 2; s < count; s += BATCH) {
        f32x4 u[BATCH];
        float d[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int si = s + i < count ? s + i : s;
            u[i] = at[(si - 1) * step];
            d[i] = decay[(int64_t)(si - 1) * p.H_v];
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (s + i < count) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = fmaf(d[i], x[e], u[i][e]);
                at[(s + i - 1) * step] = x;
            }
    }
}

size_t lin_prefill_layout(int B, int T, int H_v, int d_k, int d_v, void *base, LinPrefillParams *p)
{
    // tokens of a segment: two waves a SIMD where the call has them
    const int64_t waves = (int64_t)device_cus() * 8;
    int64_t segment = ((int64_t)T * H_v * (d_v / 32) + waves - 1) / waves;
    segment = segment < 128 ? 128 : (segment > 1024 ? 1024 : segment);
    segment = (segment + C - 1) / C * C;
    const int64_t segments = T / segment + B;
    const size_t entry = T > segment ? round256((size_t)segments * H_v * d_k * d_v * 4) : 0;
    const size_t decay = T > segment ? round256((size_t)segments * H_v * 4) : 0;
    if (p) {
        p->segment = (int)segment;
        p->segments = (int)segments;
        p->entry = static_cast<float *>(base);
        p->decay = reinterpret_cast<float *>(static_cast<char *>(base) + entry);
    }
    return entry + decay + 256;
}

template <int DK, int DV>
static hipError_t launch_prefill(const LinPrefillParams &p, hipStream_t stream)
{
    LinPrefillParams q = p;
    void *args[] = {&q};
    const unsigned grid = (unsigned)(((int64_t)p.segments * p.H_v + 7) / 8 * 8);
    hipError_t e = hipSuccess;
    if (p.T > p.segment) { // some sequence may have several
        e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_prefill_kernel<DK, DV, false>), dim3(grid),
                            dim3(2 * DV), args, 0, stream);
        if (e == hipSuccess)
            e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_carry_kernel<DK, DV>),
                                dim3((unsigned)(p.B * p.H_v * (DK * DV / 1024))), dim3(256), args, 0, stream);
    }
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_prefill_kernel<DK, DV, true>), dim3(grid),
                            dim3(2 * DV), args, 0, stream);
    return e;
}

hipError_t launch_lin_prefill(const LinPrefillParams &p, int d_k, int d_v, hipStream_t stream)
{
    if (d_k == 64)
        return d_v == 64 ? launch_prefill<64, 64>(p, stream) : launch_prefill<64, 128>(p, stream);
    return d_v == 64 ? launch_prefill<128, 64>(p, stream) : launch_prefill<128, 128>(p, stream);
}

} // namespace gdn
