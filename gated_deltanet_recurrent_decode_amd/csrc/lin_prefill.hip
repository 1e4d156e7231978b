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
//
// What bounds it: memory, with what the segments add to it.  8191 tokens at 16 heads of 128 x 128 have to move 135 MB
// (26 us at a large copy's 5.2 TB/s) and move 334, k and v twice and the segments' states four times; own parts 25 us,
// carry 12, walk 40 to 43, calls back to back 74 to 80; without any of its products the walk is 10% faster.  16 prompts
// of 100-1500 tokens 124 to 126 us, 4 of 5000-9000 with four value heads of 64 columns a key head 202 to 205, one of 77
// 10.5.
//
// Scores and scales are dealt out among a head's waves (each forming all for itself: 89 -> 81 us, the long
// prompt's call); two barriers a chunk with 48 KiB of LDS less (81 -> 76).  Two value heads of a key head in one
// workgroup where they have 64 columns: q and k are read once for both (4 prompts 243 -> 205).  Tried and not faster,
// the long prompt's call: 64 or 16 columns a wave, rings of three and four chunks, stores of o past the cache (76 ->
// 81), two accumulators of a read-out, three waves a SIMD, the state's second number left out of the read-outs (4 to
// 8% of the time for half of its bits).

#include <type_traits>

#include "attn_common.h"
#include "gdn_internal.h"
#include "lin_internal.h"

namespace gdn {

namespace {

constexpr int C = 32; // tokens of a chunk

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
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

// The logarithm range that a state and a chunk's weights may share one scale in: 2^-32 .. 2^32.  What fp32 holds of v,
// of a state and of a read-out's sums ends that much earlier.  Calls with 2^16, 2^32 and 2^64, us: a long prompt 80.2,
// 79.9, 79.1, ragged ones 126.4, 126.0, 125.8, grouped heads 204.6, 203.5, 201.5.
constexpr float kRange = 32.0f;

// 2^x of a 64-bit logarithm: its fraction keeps all bits of fp32.
__device__ __forceinline__ float exp2_of(double x)
{
    const double n = __builtin_rint(x);
    return ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v)
{
    const uint64_t x = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// Inclusive sums over each half of the wave, by moves within rows of 16 and one of a row's last value.
__device__ __forceinline__ double scan32(double v)
{
    v += dpp_or_zero<0x111, 0xF>(v);
    v += dpp_or_zero<0x112, 0xF>(v);
    v += dpp_or_zero<0x114, 0xF>(v);
    v += dpp_or_zero<0x118, 0xF>(v);
    return v + dpp_or_zero<0x142, 0xA>(v);
}

__device__ __forceinline__ double lane_value(double v, int lane)
{
    const uint64_t x = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)x, lane), hi = __builtin_amdgcn_readlane((int)(x >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
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

// The same of 4 bytes a lane.
__device__ __forceinline__ void load_dword_to_lds(lds_byte *to, const float *at)
{
    const uint32_t m = (uint32_t)(uintptr_t)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(uniform((int)m)), "v"(at)
                 : "memory");
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

} // namespace

// A workgroup takes HPW value heads of one key head, a wave 32 columns of one of them.
// OUT: the walk, with read-outs.  Otherwise a segment's own part of the state, for all but a
// sequence's last.
//
// What the waves of a head would all compute is dealt out among them and goes through LDS: the weighted
// scores w_ij = q_scale (q_i . k_j) 2^(G_i - G_j), as pairs of bf16 numbers, and the scales of the tokens.
template <int DK, int DV, int HPW, bool OUT>
__global__ __launch_bounds__(HPW *DV * 2, 2) void lin_prefill_kernel(LinPrefillParams p)
{
    constexpr int WPH = DV / 32, NW = WPH * HPW, NT = 64 * NW;
    constexpr int TK = DK / 32;                     // 32-row tiles of S
    constexpr int KB = C * DK * 2, VB = C * DV * 2; // bytes of a chunk's k (and q), of a head's v
    constexpr int QKB = (OUT ? 2 : 1) * KB;
    constexpr int IK = KB / (1024 * NW), IV = HPW * VB / (1024 * NW); // instructions a wave that bring them
    constexpr int PR = 64;                          // bytes of a row of scores
    __shared__ __align__(16) uint8_t sm_qk[2][QKB], sm_v[2][HPW * VB]; // a chunk, and the next on its way
    __shared__ __align__(16) float sm_g[HPW][64];
    __shared__ __align__(16) uint8_t sm_p[HPW][2][OUT ? C * PR : 16];
    __shared__ __align__(16) float sm_begin[HPW][C], sm_b[HPW][C];
    __shared__ float sm_f[HPW];
    __shared__ double sm_off[HPW], sm_total[HPW];
    static_assert(!OUT || HPW * VB >= NW * 2 * C * 4, "room for a wave's sums");

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n_ = lane & 31, hh = lane >> 5;
    // consecutive items (heads fastest) on one XCD: heads that share q and k meet in its L2
    const int groups = p.H_v / HPW, items = p.segments * groups, per = (items + 7) >> 3;
    const int item = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (item >= items || (int)(blockIdx.x >> 3) >= per)
        return;
    const int place = item / groups, h0 = item % groups * HPW, hk = h0 / (p.H_v / p.H_k);
    const int hw = wave / WPH, hv = h0 + hw, col0 = wave % WPH * 32;
    const Segment sg = segment_at(p, place);
    if (sg.b < 0)
        return;
    if (sg.pad || sg.bad) {
        if constexpr (OUT) {
            const uint32_t y = sg.pad ? 0u : 0x7fc07fc0u;
            constexpr int CH = HPW * DV / 8;
            for (int x = tid; x < sg.n * CH; x += NT) {
                const int h = h0 + x % CH / (DV / 8), c = x % (DV / 8) * 8;
                *reinterpret_cast<u32x4 *>(p.out.p + (int64_t)(sg.first + x / CH) * p.out.row +
                                           (int64_t)h * p.out.head + c) = u32x4{y, y, y, y};
            }
        }
        return;
    }
    const bool last = sg.s + 1 == sg.count;
    if (!OUT && (last || place + 1 >= p.segments)) // the second: sequences that overlap
        return;

    // this lane's column of v, and the rows of S
    const int64_t tile = (int64_t)DK * DV;
    const int cell = 8 * hh * DV + col0 + swapped(n_);
    auto cell_of = [&](int t, int i) { return cell + (32 * t + 16 * (i >> 3) + (i & 7)) * DV; };
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
                S[t][i] = from[cell_of(t, i)];
    } else {
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                S[t][i] = 0.f;
    }
    auto store_state = [&](float *to) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                to[cell_of(t, i)] = S[t][i];
    };

    if (!OUT && sg.s == 0) // the walk may find the slot already written: it begins from this copy
        store_state(p.entry + ((int64_t)place * p.H_v + hv) * tile);

    // staging: 1 KiB an instruction, whole rows, chunks of 16 bytes in the order of their row
    auto offset = [&](auto width, const Heads &x, int i, int last) { // this lane's; rows past the last repeat it
        constexpr int D = decltype(width)::value, CH = D / 8, RP = 64 / CH, PER = C / RP; // instructions a head
        const int at = i * NW + wave, r = at % PER * RP + lane / CH;
        return (r < last ? r : last) * (int)x.row * 2 + at / PER * (int)x.head * 2 +
               ((lane % CH) ^ swizzle<D>(r)) * 16;
    };
    const std::integral_constant<int, DK> width_k;
    const std::integral_constant<int, DV> width_v;
    int off_k[IK], off_v[IV], off_q[IK];
#pragma unroll
    for (int i = 0; i < IK; ++i) {
        off_k[i] = offset(width_k, p.k, i, C - 1);
        off_q[i] = offset(width_k, p.q, i, C - 1);
    }
#pragma unroll
    for (int i = 0; i < IV; ++i)
        off_v[i] = offset(width_v, p.v, i, C - 1);
    auto base_of = [&](const Heads &x, int head, int token) { // in scalar registers
        const uint64_t at =
            reinterpret_cast<uint64_t>(x.p + (int64_t)(sg.first + token) * x.row + (int64_t)head * x.head);
        return reinterpret_cast<const uint8_t *>((uint64_t)(uint32_t)uniform((int)(at >> 32)) << 32 |
                                                 (uint32_t)uniform((int)at));
    };
    auto bring = [&](int buf, int c0) {
        const int last = sg.n - c0 - 1;
        if (last < C - 1) {
#pragma unroll
            for (int i = 0; i < IK; ++i) {
                off_k[i] = offset(width_k, p.k, i, last);
                off_q[i] = offset(width_k, p.q, i, last);
            }
#pragma unroll
            for (int i = 0; i < IV; ++i)
                off_v[i] = offset(width_v, p.v, i, last);
        }
        lds_byte *to = (lds_byte *)sm_qk + buf * QKB + wave * 1024;
        const uint8_t *base_k = base_of(p.k, hk, c0), *base_v = base_of(p.v, h0, c0);
#pragma unroll
        for (int i = 0; i < IK; ++i)
            load_to_lds(to + i * NW * 1024, base_k, off_k[i]);
        if constexpr (OUT) {
            const uint8_t *base_q = base_of(p.q, hk, c0);
#pragma unroll
            for (int i = 0; i < IK; ++i)
                load_to_lds(to + KB + i * NW * 1024, base_q, off_q[i]);
        }
        to = (lds_byte *)sm_v + buf * (HPW * VB) + wave * 1024;
#pragma unroll
        for (int i = 0; i < IV; ++i)
            load_to_lds(to + i * NW * 1024, base_v, off_v[i]);
        if (wave < HPW) { // the decays, a wave a head
            const int t = c0 + (n_ < last ? n_ : last), h = h0 + wave;
            load_dword_to_lds((lds_byte *)sm_g + wave * 256,
                              p.g + (p.per_token ? (int64_t)(sg.first + t) * p.H_v + h : (int64_t)h));
        }
    };

    // transposing reads: lane (hv, r, c) points at key 4 hv + r (+ 8 for the second), columns 4 c
    const int gr = lane >> 4, r_ = (lane & 15) >> 2, c_ = swapped((lane & 3) << 2) >> 2;
    int tk_at[2], tv_at[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int key = 8 * y + 4 * (gr >> 1) + r_, chunk = (gr & 1) * 2 + (c_ >> 1);
        tk_at[y] = key * DK * 2 + ((chunk ^ swizzle<DK>(key)) * 16) + (c_ & 1) * 8;
        tv_at[y] = hw * VB + key * DV * 2 + (((col0 / 8 + chunk) ^ swizzle<DV>(key)) * 16) + (c_ & 1) * 8;
    }
    // row reads: this lane's row, its chunk without the step's
    const int row_at = n_ * DK * 2 + (hh ^ swizzle<DK>(n_)) * 16;
    auto transposed = [&](const uint8_t *at0, const uint8_t *at1, uint32_t (&x)[4]) {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at0));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at1));
        x[0] = a[0];
        x[1] = a[1];
        x[2] = b[0];
        x[3] = b[1];
    };

    // The state is held without its latest decays, S = 2^off S~: with L_i = off + G_i, o_i = 2^(L_i) S~^T q_i
    // + sum_j w_ij v_j and S~ += k_j (2^(-L_j) v_j)^T, with no decay of the whole state, until some |L_i| of
    // a chunk passes kRange.  There S~ takes the scale of the chunk's end, 2^(off + G_end), and off is -G_end
    // for its weights.
    auto sums = [&](int c0, int head) { // G of this lane's token
        const int rows = sg.n - c0 < C ? sg.n - c0 : C;
        return scan32(n_ < rows ? (double)log2_decay(sm_g[head][n_]) : 0.0);
    };
    auto scales = [&](int c0, int head) { // of the chunk at token c0
        const double G = sums(c0, head), end = lane_value(G, C - 1);
        const double off = c0 > 0 ? sm_off[head] : 0.0, total = c0 > 0 ? sm_total[head] : 0.0;
        const bool far = __ballot(fabs(off + G) > (double)kRange) != 0;
        const double base = far ? -end : off;
        if (hh == 0) {
            sm_begin[head][n_] = exp2_of(off + G) * p.q_scale;
            sm_b[head][n_] = c0 + n_ < sg.n ? exp2_of(-(base + G)) : 0.f;
        }
        if (lane == 0) {
            sm_f[head] = far ? exp2_of(off + end) : 1.f;
            sm_off[head] = base + end;
            sm_total[head] = total + end;
        }
    };
    // A row of scores: its 16-byte chunk x of 4, at another place every two rows (32 lanes read 32 rows).
    auto score_at = [](int row, int x) { return row * PR + ((x ^ (row >> 1 & 3)) * 16); };
    // the scores of keys 16 kt.. and tokens 16 tt.., 16 x 16 x 32 products: a lane has a token and four keys
    auto scores = [&](int c0, int buf, int head, int kt, int tt) {
        const double G = sums(c0, head);
        const float G_hi = (float)G, G_lo = (float)(G - (double)G_hi);
        float *own = reinterpret_cast<float *>(sm_v[buf ^ 1]) + wave * 2 * C; // nobody reads v there any more
        if (hh == 0) {
            own[n_] = G_hi;
            own[C + n_] = G_lo;
        }
        const int m = lane & 15, g4 = lane >> 4;
        const uint8_t *kb = sm_qk[buf], *qb = kb + KB;
        f32x4 P = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
            const int at = ((4 * x + g4) ^ swizzle<DK>(m)) * 16;
            const u32x4 kf = *reinterpret_cast<const u32x4 *>(kb + (16 * kt + m) * DK * 2 + at);
            const u32x4 qf = *reinterpret_cast<const u32x4 *>(qb + (16 * tt + m) * DK * 2 + at);
            P = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf), __builtin_bit_cast(bf16x8, qf),
                                                        P, 0, 0, 0);
        }
        settle(P);
        __builtin_amdgcn_wave_barrier();
        const float T_hi = own[16 * tt + m], T_lo = own[C + 16 * tt + m];
        const f32x4 K_hi = *reinterpret_cast<const f32x4 *>(&own[16 * kt + 4 * g4]);
        const f32x4 K_lo = *reinterpret_cast<const f32x4 *>(&own[C + 16 * kt + 4 * g4]);
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float d = (T_hi - K_hi[i]) + (T_lo - K_lo[i]);
            w[i] = kt < tt || 4 * g4 + i <= m ? P[i] * p.q_scale * __builtin_amdgcn_exp2f(d) : 0.f;
        }
        u32x2 hi, lo;
        uint32_t x, y;
        split2(w[0], w[1], x, y);
        hi[0] = x, lo[0] = y;
        split2(w[2], w[3], x, y);
        hi[1] = x, lo[1] = y;
        // keys in the order of the product with v: blocks of four, 0 2 1 3
        const int at = score_at(16 * tt + m, 2 * kt + (g4 & 1)) + (g4 >> 1) * 8;
        *reinterpret_cast<u32x2 *>(&sm_p[head][0][at]) = hi;
        *reinterpret_cast<u32x2 *>(&sm_p[head][1][at]) = lo;
        __builtin_amdgcn_wave_barrier();
    };

    if (sg.n > 0)
        bring(0, 0);
    if constexpr (OUT) // scores of later keys: stay 0
        for (int x = tid; x < HPW * 2 * 16 * 4; x += NT)
            *reinterpret_cast<u32x2 *>(
                &sm_p[x >> 7][x >> 6 & 1][score_at(x >> 2 & 15, 2 + (x >> 1 & 1)) + (x & 1) * 8]) = u32x2{0u, 0u};
    // S is there: left to the compiler, every chunk would wait for it, and with it for what is asked for meanwhile
#pragma unroll
    for (int t = 0; t < TK; ++t)
        settle(S[t]);
    for (int c0 = 0, buf = 0; c0 < sg.n; c0 += C, buf ^= 1) {
        // The chunk is in LDS; the stores of the read-outs before it, two instructions behind its loads, may
        // still be on their way.
        if (OUT && c0 > 0)
            asm volatile("s_waitcnt vmcnt(2)" ::: "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
        constexpr int JOBS = OUT ? 4 : 1; // a head
        for (int job = wave; job < JOBS * HPW; job += NW) {
            const int head = job / JOBS, x = job % JOBS;
            if (x == JOBS - 1)
                scales(c0, head);
            else if constexpr (OUT)
                scores(c0, buf, head, x == 2, x > 0);
        }
        lds_barrier();
        if (c0 + C < sg.n) // every wave is past the chunk before this one
            bring(buf ^ 1, c0 + C);
        const uint8_t *kb = sm_qk[buf], *qb = kb + KB, *vb = sm_v[buf];
        uint32_t vf[2][4]; // this lane's column, 16 keys each
#pragma unroll
        for (int u = 0; u < 2; ++u)
            transposed(vb + u * 16 * DV * 2 + tv_at[0], vb + u * 16 * DV * 2 + tv_at[1], vf[u]);

        if constexpr (OUT) {
            f32x16 O;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                O[i] = 0.f;
            const float begin = sm_begin[hw][n_];
            int r_at = row_at; // addresses are formed anew each chunk: kept, they cost 8 registers
            asm volatile("" : "+v"(r_at));
#pragma unroll
            for (int t = 0; t < TK; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bf16x8 qf = __builtin_bit_cast(
                        bf16x8, *reinterpret_cast<const u32x4 *>(qb + (r_at ^ (t * 64 + u * 32))));
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split2(S[t][8 * u + 2 * e], S[t][8 * u + 2 * e + 1], hi[e], lo[e]);
                    O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(hi), qf, O, 0, 0, 0);
                    O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(lo), qf, O, 0, 0, 0);
                }
            settle(O);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                O[i] *= begin;
            u16x2 most = {0, 0};
            uint32_t vc[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    vc[u][e] = vf[u][e];
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, vf[u][e] & 0x7fff7fffu));
                }
            // An infinity or NaN in v must not reach tokens before it (0 times it is NaN): it leaves this
            // product, and from its token on the column becomes NaN.
            if (__ballot(most[0] >= 0x7f80 || most[1] >= 0x7f80)) {
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
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(&sm_p[hw][0][score_at(n_, 2 * u + hh)]);
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(&sm_p[hw][1][score_at(n_, 2 * u + hh)]);
                O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(vc[u]), __builtin_bit_cast(bf16x8, hi), O, 0, 0, 0);
                O = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(vc[u]), __builtin_bit_cast(bf16x8, lo), O, 0, 0, 0);
            }
            settle(O);
            if (c0 + n_ < sg.n) {
                uint16_t *o = p.out.p + (int64_t)(sg.first + c0 + n_) * p.out.row + (int64_t)hv * p.out.head + col0 +
                              8 * hh;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = pack_bf16(O[8 * u + 2 * e], O[8 * u + 2 * e + 1]);
                    *reinterpret_cast<u32x4 *>(o + 16 * u) = u32x4{y[0], y[1], y[2], y[3]};
                }
            }
        }

        // the state behind the chunk
        const float f = sm_f[hw];
        if (__ballot(f != 1.f)) { // uniform
#pragma unroll
            for (int t = 0; t < TK; ++t)
                S[t] *= f;
        }
        int k_at[2] = {tk_at[0], tk_at[1]};
        asm volatile("" : "+v"(k_at[0]), "+v"(k_at[1]));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t hi[4], mid[4], lo[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const f32x4 w = *reinterpret_cast<const f32x4 *>(&sm_b[hw][16 * u + 8 * x + 4 * hh]);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int e = 2 * x + y;
                    split3(__uint_as_float(vf[u][e] << 16) * w[2 * y],
                           __uint_as_float(vf[u][e] & 0xffff0000u) * w[2 * y + 1], hi[e], mid[e], lo[e]);
                }
            }
            uint32_t kt[TK][4];
#pragma unroll
            for (int t = 0; t < TK; ++t) {
                const int o = u * 16 * DK * 2, x = t * 64;
                transposed(kb + o + (k_at[0] ^ x), kb + o + (k_at[1] ^ x), kt[t]);
            }
#pragma unroll
            for (int t = 0; t < TK; ++t)
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt[t]), operand(hi), S[t], 0, 0, 0);
#pragma unroll
            for (int t = 0; t < TK; ++t)
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt[t]), operand(mid), S[t], 0, 0, 0);
#pragma unroll
            for (int t = 0; t < TK; ++t)
                S[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(kt[t]), operand(lo), S[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < TK; ++t)
            settle(S[t]);
    }
    if (sg.n > 0) {
        const float scale = exp2_of(sm_off[hw]);
#pragma unroll
        for (int t = 0; t < TK; ++t)
            S[t] *= scale;
    }
    if constexpr (OUT) {
        if (last)
            store_state(p.state + ((int64_t)sg.write * p.H_v + hv) * tile);
    } else {
        store_state(p.entry + ((int64_t)(place + 1) * p.H_v + hv) * tile);
        if (wave % WPH == 0 && lane == 0)
            p.decay[(int64_t)(place + 1) * p.H_v + hv] = exp2_of(sm_total[hw]);
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

// Workgroups of the walk that a CU holds: by their LDS with d_k = 64, by registers or LDS with 128.
static int walks_a_cu(int d_k, int d_v, bool pair)
{
    if (d_k == 64)
        return d_v == 128 ? 4 : (pair ? 3 : 5);
    return d_v == 128 || pair ? 2 : 3;
}

size_t lin_prefill_layout(int B, int T, int H_k, int H_v, int d_k, int d_v, void *base, LinPrefillParams *p)
{
    // Tokens of a segment: the shortest ones that give at most `rounds` times the workgroups that the chip holds
    // at once, sequences' last ones counted as whole, with the rounds that cost least.  A workgroup's start and end
    // and its state's way through memory cost about as much as kFixed tokens: segments half as long take 77, 146 and
    // 223 us of the three cases above, twice as long 78, 123 and 335, these 76, 126 and 205.  kMost: where no rounds
    // fit, which is with more sequences than 8 slots / groups (64 at 64 heads of 128 x 128) and close to that, and none
    // longer, so that one long prompt among many does not outlast the rest.  With 512, 1024, 2048, 4096, 8192, us: 64
    // heads of 128 x 128, one prompt of 8000 among 79 of 100 1074, 1138, 1117, 1085, 909, four of 4000 among 76 of 100
    // 1239, 1568, 1848, 1552, 1562, 80 of 300-500 531, 533, 523, 529, 535; 16 heads, one of 8000 among 299 of 50 425,
    // 424, 428, 501, 621.  512 has four times the segments of long prompts in the workspace.
    constexpr int64_t kFixed = 160, kMost = 2048, kFewest = 4 * C;
    const bool pair = d_v == 64 && H_v / H_k % 2 == 0;
    const int64_t groups = pair ? H_v / 2 : H_v, slots = (int64_t)device_cus() * walks_a_cu(d_k, d_v, pair);
    int64_t segment = 0, least = 0, most = 0;
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
        most = rounds * slots / groups; // segments: (T + B (L - 1)) / L of them at most
        if (most < B)
            continue;
        if (T >= B) {
            int64_t L = (T - B) / (most - B + 1) + 1;
            L = ((L < kFewest ? kFewest : L) + C - 1) / C * C;
            if (least == 0 || rounds * (L + kFixed) < least) {
                least = rounds * (L + kFixed);
                segment = L;
            }
        }
        // Up to whole segments and rounds the cost is most (T / (most - B) + kFixed), least where this becomes equal.
        if ((most - B) * (most - B) * kFixed >= (int64_t)B * T)
            break;
    }
    if (segment == 0 || segment > kMost)
        segment = kMost;
    const int64_t segments = T / segment + B;
    // Fewer sequences or tokens may have shorter segments, and more of them.  So that one workspace serves all calls up
    // to the largest, it has room for what no such call passes: with T - B < L (most - B + 1) places T / L + B are at
    // most most + ceil(B / L), and `most` is the last that was looked at, which only grows with B and T.
    int64_t room = 0;
    if (T > kFewest) {
        room = most + (B + kFewest - 1) / kFewest;
        room = T / kFewest + B < room ? T / kFewest + B : room;
        if (T > kMost && T / kMost + B > room)
            room = T / kMost + B;
    }
    const size_t entry = round256((size_t)room * H_v * d_k * d_v * 4), decay = round256((size_t)room * H_v * 4);
    if (p) {
        p->segment = (int)segment;
        p->segments = (int)segments;
        p->entry = static_cast<float *>(base);
        p->decay = reinterpret_cast<float *>(static_cast<char *>(base) + entry);
    }
    return entry + decay + 256;
}

template <int DK, int DV, int HPW>
static hipError_t launch_walk(const LinPrefillParams &p, hipStream_t stream)
{
    LinPrefillParams q = p;
    void *args[] = {&q};
    const dim3 grid((unsigned)(((int64_t)p.segments * (p.H_v / HPW) + 7) / 8 * 8)), block(HPW * DV * 2);
    hipError_t e = hipSuccess;
    if (p.T > p.segment) { // some sequence may have several
        e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_prefill_kernel<DK, DV, HPW, false>), grid, block, args,
                            0, stream);
        if (e == hipSuccess)
            e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_carry_kernel<DK, DV>),
                                dim3((unsigned)(p.B * p.H_v * (DK * DV / 1024))), dim3(256), args, 0, stream);
    }
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&lin_prefill_kernel<DK, DV, HPW, true>), grid, block, args,
                            0, stream);
    return e;
}

template <int DK, int DV>
static hipError_t launch_prefill(const LinPrefillParams &p, hipStream_t stream)
{
    if constexpr (DV == 64)
        if (p.H_v / p.H_k % 2 == 0)
            return launch_walk<DK, DV, 2>(p, stream);
    return launch_walk<DK, DV, 1>(p, stream);
}

hipError_t launch_lin_prefill(const LinPrefillParams &p, int d_k, int d_v, hipStream_t stream)
{
    if (d_k == 64)
        return d_v == 64 ? launch_prefill<64, 64>(p, stream) : launch_prefill<64, 128>(p, stream);
    return d_v == 64 ? launch_prefill<128, 64>(p, stream) : launch_prefill<128, 128>(p, stream);
}

} // namespace gdn
