// attn_paged.hip -- attention of new tokens over a paged KV cache (gfx950).
//
// o = sum_j softmax_j(scale q.k_j) v_j, in one pass over the keys with a running
// maximum m and sum l: for each block of keys, m' = max(m, s), l = l e^(m - m')
// + sum e^(s - m'), o = o e^(m - m') + sum e^(s - m') v; at the end o / l.
//
// The query heads of a group share their kv head, so a sequence's (token, head
// of the group) pairs form the rows of a tile of 16 and each key is read once
// for all of them.  Both products run on the matrix cores transposed, S^T = K
// Q^T and O^T = V^T P^T (16 x 16 x 32 bf16), which makes the layouts meet with
// no exchange between lanes: lane (g, n) of S^T holds row n's scores of keys
// 4g..4g+3 of two 16-key tiles, which is a P^T operand as it stands once the
// contraction's 32 places are dealt out to the keys in that order, and the V^T
// operand wants, of those same eight keys, one column of v, which a lane makes
// from eight 16-byte pieces of their rows by one byte permute a dword.  So K and
// V go from memory to registers to the matrix cores: no LDS and no barrier on
// the way.
//
// Work is dealt out by the key, not by the sequence: the units of 128 keys of all
// (sequence, kv head) pairs, one tile each, lie on one line, cut into equal pieces,
// one a workgroup.  A workgroup finds its piece from the lengths on the device (a
// captured step follows its lengths) and finishes what lies whole in it; of a pair
// that is cut it leaves (o, m, l) in the workspace for the second kernel.
//
// What bounds it: reading the cache.  MI355X, calls back to back: 64 sequences of
// 0.2-8 thousand tokens at 16/4 heads of 256, 1.2 GB, 223 us (5.36 TB/s); 8 of 40-131
// thousand e4m3 tokens at 32/4 heads of 128, 0.6 GB, 113 us (5.25 TB/s), the join's
// kernel 6.3 of them; one of 777 tokens 13.0 us, kernels of 9.4 and 4.2, a chain of
// dependent reads (lengths, page numbers, keys).  What gave most after the layouts:
// page numbers read a block ahead by the scalar unit (the kernel alone, under the
// profiler, 239 -> 228 us at the first size), the search within a wave (11.6 -> 10.6
// for the one sequence).  At 256 columns one workgroup a CU at a time with more
// registers is faster than two (the first size 223 us a call, two 232), at 128 two are
// no slower (long contexts 114.1, one 114.7).

#include "attn_common.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int TM = 16;    // rows of a tile, the most that a sequence has here
constexpr int UNIT = 128; // keys of a unit: a block of 32 a wave
constexpr int NT = 256;

// A sequence, and the units of each of its kv heads: of keys, or where it cannot be used, and may
// have any number of rows, of rows to fill.
struct RowSeq : Seq {
    int units;
};

__device__ __forceinline__ RowSeq read_row_seq(const AttnParams &p, int b)
{
    RowSeq s;
    static_cast<Seq &>(s) = read_seq(p, b);
    const int span = s.kind == kNormal ? s.L - s.lo : (s.kind == kSkip ? 0 : s.n * p.G);
    s.units = s.kind == kSkip ? 0 : (span > UNIT ? (span + UNIT - 1) / UNIT : 1);
    return s;
}

__device__ __forceinline__ long long seq_units(const AttnParams &p, const RowSeq &s)
{
    return (long long)p.H_kv * s.units;
}

struct Place {
    int b;            // sequence, -1: nowhere
    long long before; // units before it
    long long total;  // units of the call
    RowSeq s;
};

__device__ __forceinline__ long long lane_of(long long v, int lane)
{
    const uint32_t lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
    return (long long)((uint64_t)hi << 32 | lo);
}

// Where the line of units holds what `hit` asks for (a predicate of a sequence,
// its first unit, its units and the units of the call).  TH threads; up to 64
// sequences each wave for itself, with no barrier.
template <int TH, class Hit>
__device__ __forceinline__ Place locate(const AttnParams &p, Hit hit)
{
    __shared__ long long wave_sum[TH / 64];
    __shared__ Place found;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (p.B <= 64) {
        RowSeq s{};
        long long u = 0;
        if (lane < p.B) {
            s = read_row_seq(p, lane);
            u = seq_units(p, s);
        }
        long long inc = u;
        for (int m = 1; m < p.B; m <<= 1) {
            const long long o = __shfl_up(inc, m);
            if (lane >= m)
                inc += o;
        }
        Place f;
        f.total = lane_of(inc, p.B - 1);
        const uint64_t where = __ballot(u > 0 && hit(s, inc - u, u, f.total));
        const int k = where ? __builtin_ctzll(where) : 0;
        f.b = where ? k : -1;
        f.before = lane_of(inc - u, k);
        f.s.kind = __builtin_amdgcn_readlane(s.kind, k);
        f.s.first = __builtin_amdgcn_readlane(s.first, k);
        f.s.n = __builtin_amdgcn_readlane(s.n, k);
        f.s.L = __builtin_amdgcn_readlane(s.L, k);
        f.s.lo = __builtin_amdgcn_readlane(s.lo, k);
        f.s.r = __builtin_amdgcn_readlane(s.r, k);
        f.s.units = __builtin_amdgcn_readlane(s.units, k);
        return f;
    }
    long long total = 0;
    if (tid == 0)
        found.b = -1;
    for (int pass = 0; pass < 2; ++pass) {
        long long run = 0;
        for (int b0 = 0; b0 < p.B; b0 += TH) {
            const int b = b0 + tid;
            RowSeq s;
            long long u = 0;
            if (b < p.B) {
                s = read_row_seq(p, b);
                u = seq_units(p, s);
            }
            long long inc = u;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const long long o = __shfl_up(inc, m);
                if (lane >= m)
                    inc += o;
            }
            __syncthreads();
            if (lane == 63)
                wave_sum[wave] = inc;
            __syncthreads();
            long long before = run;
#pragma unroll
            for (int w = 0; w < TH / 64; ++w) {
                if (w < wave)
                    before += wave_sum[w];
                run += wave_sum[w];
            }
            if (pass == 1 || p.B <= TH) {
                const long long all = p.B <= TH ? run : total;
                if (u > 0 && hit(s, before + inc - u, u, all))
                    found = Place{b, before + inc - u, all, s};
            }
        }
        if (pass == 0)
            total = run;
        if (p.B <= TH)
            break;
    }
    __syncthreads();
    return found;
}

} // namespace

// D = 64, 128 or 256.  A lane owns EV consecutive columns of v in each of NH
// 128-column parts (D = 64: four columns of one part).
template <int D, bool E4M3>
__global__ __launch_bounds__(NT, D == 256 ? 1 : 2) void attn_rows_kernel(AttnParams p)
{
    constexpr int EV = D == 64 ? 4 : 8, NH = D / (16 * EV), NS = D / 32;
    constexpr int LD = D + 4; // LDS row, padded against bank conflicts
    __shared__ __align__(16) float sm_o[4][TM][LD];
    __shared__ float sm_m[4][TM], sm_l[4][TM], sm_mm[TM], sm_ll[TM];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n_ = lane & 15, g = lane >> 4;
    const int w = blockIdx.x;

    const Place at = locate<NT>(p, [&](const RowSeq &, long long before, long long units, long long total) {
        const int pieces = pieces_of(p, total);
        const long long u0 = piece_begin(total, w, pieces);
        return w < pieces && before <= u0 && u0 < before + units;
    });
    if (tid == 0)
        write_cut(p, w, Cut{-1});
    if (at.b < 0)
        return;
    const int pieces = pieces_of(p, at.total);
    long long u = piece_begin(at.total, w, pieces);
    const long long u_end = piece_begin(at.total, w + 1, pieces);
    const long long u_begin = u;
    int b = at.b;
    long long before = at.before;
    RowSeq s = at.s;

    while (u < u_end) {
        const long long units = seq_units(p, s);
        if (u >= before + units) {
            before += units;
            s = read_row_seq(p, ++b);
            continue;
        }
        const long long v = u - before;
        const int h = uniform((int)quotient(v, s.units));
        if (s.kind != kNormal) { // zeros, or NaN
            const uint32_t y = s.kind == kZero ? 0u : 0x7fc07fc0u;
            const int r0 = (int)(v - (long long)h * s.units) * UNIT, n = s.n * p.G - r0;
            for (int x = tid; x < (n < UNIT ? n : UNIT) * (D / 8); x += NT) {
                const int r = r0 + x / (D / 8), hq = h * p.G + r % p.G, c = x % (D / 8) * 8;
                const int64_t tk = s.first + r / p.G;
                *reinterpret_cast<u32x4 *>(p.out.p + tk * p.out.row + (int64_t)hq * p.out.head + c) =
                    u32x4{y, y, y, y};
                if (c == 0 && p.lse)
                    p.lse[tk * p.H_q + hq] = s.kind == kZero ? neg_inf() : quiet_nan();
            }
            ++u;
            continue;
        }
        const long long t0 = before + (long long)h * s.units, t1 = t0 + s.units;
        const int unit0 = (int)(u - t0);
        const long long e = t1 < u_end ? t1 : u_end;
        const int unit1 = unit0 + (int)(e - u);
        const bool whole = u == t0 && e == t1;
        const int slot = u == u_begin ? 0 : 1;
        if (tid == 0 && u == t0 && e < t1)
            write_cut(p, w, Cut{owner_of(at.total, t1 - 1, pieces), slot, s.first, s.n * p.G, h, 0});
        u = e;

        // this lane's row: a token and a head of the group
        const int rows = s.n * p.G;
        const bool valid = n_ < rows;
        const int tok = n_ / p.G, head = h * p.G + n_ % p.G;
        const int pos = valid ? s.L - s.n + tok : -1;
        const int low = p.window > 0 ? pos - p.window + 1 : 0;
        const int min_pos = s.L - s.n; // the first token's

        bf16x8 qf[NS];
        const uint16_t *qp = p.q.p + (int64_t)(s.first + tok) * p.q.row + (int64_t)head * p.q.head;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            // the 8-bit cache is read 16 values at a time, two steps of the contraction
            const int d0 = E4M3 ? (i >> 1) * 64 + g * 16 + (i & 1) * 8 : i * 32 + g * 8;
            u32x4 x = {0u, 0u, 0u, 0u};
            if (valid)
                x = *reinterpret_cast<const u32x4 *>(qp + d0);
            qf[i] = __builtin_bit_cast(bf16x8, x);
        }

        float m = neg_inf(), l = 0.f;
        f32x4 acc[NH][EV];
#pragma unroll
        for (int a = 0; a < NH; ++a)
#pragma unroll
            for (int c = 0; c < EV; ++c)
                acc[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
        bool bad = false;
        const float scale = E4M3 ? p.scale * p.k_scale[h] : p.scale;

        const int k_end = uniform(s.lo + unit1 * UNIT < s.L ? s.lo + unit1 * UNIT : s.L);
        auto *tab = (__attribute__((address_space(4))) const int32_t *)(p.page_table + (int64_t)uniform(s.r) * p.width);
        auto page_of = [&](int key) { return key < k_end ? tab[key >> p.page_shift] : 0; };
        const int key_first = uniform(s.lo + unit0 * UNIT + wave * 32);
        int next[2] = {page_of(key_first), page_of(key_first + 16)};
        for (int key0 = key_first; key0 < k_end; key0 += UNIT) {
            int page[2] = {next[0], next[1]};
            // the next block's page numbers, while this one is worked on
            next[0] = page_of(key0 + UNIT);
            next[1] = page_of(key0 + UNIT + 16);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (page[t] < 1 || page[t] >= p.N) { // uniform
                    const int k0 = key0 + 16 * t;
                    bad |= k0 < s.L && pos >= k0 && low <= k0 + 15;
                    page[t] = 0;
                }
            }
            // cells of the two 16-key tiles
            int64_t cell[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
                cell[t] = ((((int64_t)page[t] * p.H_kv + h) << p.page_shift) +
                           ((key0 + 16 * t) & ((1 << p.page_shift) - 1))) * D;

            f32x4 sc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                if constexpr (E4M3) {
                    const uint8_t *kp = static_cast<const uint8_t *>(p.k_pages) + cell[t] + n_ * D + g * 16;
#pragma unroll
                    for (int i = 0; i < NS / 2; ++i) {
                        const u32x4 x = *reinterpret_cast<const u32x4 *>(kp + i * 64);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const u32x4 y = {e4m3_to_bf16<false>(x[2 * q]), e4m3_to_bf16<true>(x[2 * q]),
                                             e4m3_to_bf16<false>(x[2 * q + 1]), e4m3_to_bf16<true>(x[2 * q + 1])};
                            sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, y),
                                                                            qf[2 * i + q], sc[t], 0, 0, 0);
                        }
                    }
                } else {
                    const uint16_t *kp = static_cast<const uint16_t *>(p.k_pages) + cell[t] + n_ * D + g * 8;
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const u32x4 x = *reinterpret_cast<const u32x4 *>(kp + i * 32);
                        sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), qf[i], sc[t], 0,
                                                                        0, 0);
                    }
                }
            }

            // v: eight keys of this lane (4g.. of both tiles), EV columns of each part, as bf16 pairs
            uint32_t vr[NH][8][EV / 2];
#pragma unroll
            for (int a = 0; a < NH; ++a)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int64_t o = cell[j >> 2] + (g * 4 + (j & 3)) * D + a * 128 + n_ * EV;
                    if constexpr (E4M3) {
                        const uint8_t *vp = static_cast<const uint8_t *>(p.v_pages) + o;
#pragma unroll
                        for (int c = 0; c < EV / 4; ++c) {
                            const uint32_t x = reinterpret_cast<const uint32_t *>(vp)[c];
                            vr[a][j][2 * c] = e4m3_to_bf16<false>(x);
                            vr[a][j][2 * c + 1] = e4m3_to_bf16<true>(x);
                        }
                    } else {
                        const uint16_t *vp = static_cast<const uint16_t *>(p.v_pages) + o;
#pragma unroll
                        for (int c = 0; c < EV / 2; ++c)
                            vr[a][j][c] = reinterpret_cast<const uint32_t *>(vp)[c];
                    }
                }

            settle(sc[0]);
            settle(sc[1]);

            // masks, where some row of the tile does not see every key of the block
            const bool mixed = key0 + 31 > min_pos || (p.window > 0 && key0 < s.L - p.window);
            float pr[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                pr[j] = sc[j >> 2][j & 3] * scale;
            bool odd_any = false;
            if (mixed) {
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int key = key0 + (j >> 2) * 16 + g * 4 + (j & 3);
                    if (key > pos || key < low)
                        pr[j] = neg_inf();
                    const bool past = key >= s.L;
#pragma unroll
                    for (int a = 0; a < NH; ++a)
#pragma unroll
                        for (int c = 0; c < EV / 2; ++c) {
                            const uint32_t x = past ? 0u : vr[a][j][c];
                            vr[a][j][c] = x;
                            odd |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
                        }
                }
                // An infinity or NaN in v must not reach rows that do not see its key (0 times it is
                // NaN): such values leave the product here and are added to the rows that do below.
                odd_any = __ballot(odd) != 0;
                if (odd_any) {
#pragma unroll
                    for (int a = 0; a < NH; ++a)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int c = 0; c < EV / 2; ++c) {
                                uint32_t x = vr[a][j][c];
                                if ((x & 0x7f80u) == 0x7f80u)
                                    x &= 0xffff0000u;
                                if ((x & 0x7f800000u) == 0x7f800000u)
                                    x &= 0xffffu;
                                vr[a][j][c] = x;
                            }
                }
            }

            float top = pr[0];
#pragma unroll
            for (int j = 1; j < 8; ++j)
                top = fmaxf(top, pr[j]);
            top = max_xor32(max_xor16(top));
            const float m_new = fmaxf(m, top);
            const float m_safe = m_new == neg_inf() ? 0.f : m_new;
            const float keep = __builtin_amdgcn_exp2f(m - m_safe);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                pr[j] = __builtin_amdgcn_exp2f(pr[j] - m_safe);
                sum += pr[j];
            }
            l = fmaf(l, keep, sum); // this lane's keys only; joined at the end
            m = m_new;
            // The matrix cores take bf16: a weight goes as two of them, its upper half and what that leaves
            // (off by at most 2^-15 of the weight together).  With one alone o is 0.0018 of its norm off 64
            // bits in place of the 0.0017 of its own rounding, and the calls are 0.4 to 1% faster (64 rows
            // 223.2 us against 224.1, long contexts 113.1 against 114.0).  What is left is kept above 0 (by
            // 2^-20 of the weight), or an infinity in v that every row of the tile sees would become a NaN.
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t y0 = __float_as_uint(pr[2 * j]), y1 = __float_as_uint(pr[2 * j + 1]);
                hi[j] = __builtin_amdgcn_perm(y1, y0, 0x07060302u);
                lo[j] = pack_bf16(fmaf(pr[2 * j], 1.0f + 0x1p-20f, -__uint_as_float(y0 & 0xffff0000u)),
                                  fmaf(pr[2 * j + 1], 1.0f + 0x1p-20f, -__uint_as_float(y1 & 0xffff0000u)));
            }
            const bf16x8 ph = __builtin_bit_cast(bf16x8, u32x4{hi[0], hi[1], hi[2], hi[3]});
            const bf16x8 pl = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], lo[2], lo[3]});
#pragma unroll
            for (int a = 0; a < NH; ++a)
#pragma unroll
                for (int c = 0; c < EV; ++c) {
                    constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
                    const uint32_t sel = (c & 1) ? kHigh : kLow;
                    u32x4 x;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = __builtin_amdgcn_perm(vr[a][2 * j + 1][c >> 1], vr[a][2 * j][c >> 1], sel);
                    const bf16x8 vf = __builtin_bit_cast(bf16x8, x);
                    acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph, acc[a][c] * keep, 0, 0, 0);
                    acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl, acc[a][c], 0, 0, 0);
                }
            if (odd_any) {
                for (int key = key0; key < key0 + 32 && key < s.L; ++key) {
                    const bool sees = key <= pos && key >= low;
                    const int64_t o = cell[(key - key0) >> 4] + ((key - key0) & 15) * D;
#pragma unroll
                    for (int a = 0; a < NH; ++a)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < EV; ++c) {
                                const int64_t q = o + a * 128 + (g * 4 + i) * EV + c;
                                uint32_t x;
                                if constexpr (E4M3)
                                    x = e4m3_to_bf16<false>(static_cast<const uint8_t *>(p.v_pages)[q]) << 16;
                                else
                                    x = (uint32_t) static_cast<const uint16_t *>(p.v_pages)[q] << 16;
                                if (sees && (x & 0x7f800000u) == 0x7f800000u)
                                    acc[a][c][i] += __uint_as_float(x);
                            }
                }
            }
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        // a needed page outside the pool
        if (__shfl_xor((int)bad, 16) | (int)bad)
            bad = true;
        if (__shfl_xor((int)bad, 32) | (int)bad)
            bad = true;
        if (bad)
            l = quiet_nan();

        // the four waves' keys together
        __syncthreads(); // the LDS of the piece before is free
        if (g == 0) {
            sm_m[wave][n_] = m;
            sm_l[wave][n_] = l;
        }
        __syncthreads();
        float mm = neg_inf();
#pragma unroll
        for (int q = 0; q < 4; ++q)
            mm = fmaxf(mm, sm_m[q][n_]);
        const float mm_safe = mm == neg_inf() ? 0.f : mm;
        const float mine = __builtin_amdgcn_exp2f(m - mm_safe);
#pragma unroll
        for (int a = 0; a < NH; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < EV; c += 4)
                    *reinterpret_cast<f32x4 *>(&sm_o[wave][n_][a * 128 + (g * 4 + i) * EV + c]) =
                        f32x4{acc[a][c][i], acc[a][c + 1][i], acc[a][c + 2][i], acc[a][c + 3][i]} * mine;
        if (wave == 0 && g == 0) {
            float ll = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                ll += sm_l[q][n_] * __builtin_amdgcn_exp2f(sm_m[q][n_] - mm_safe);
            sm_mm[n_] = mm;
            sm_ll[n_] = ll;
        }
        __syncthreads();
        constexpr int C4 = D / 4;
        for (int x = tid; x < TM * C4; x += NT) {
            const int rr = x / C4, c = (x % C4) * 4;
            if (rr >= rows)
                break;
            f32x4 o = *reinterpret_cast<const f32x4 *>(&sm_o[0][rr][c]);
#pragma unroll
            for (int q = 1; q < 4; ++q)
                o += *reinterpret_cast<const f32x4 *>(&sm_o[q][rr][c]);
            const float ll = sm_ll[rr];
            const int64_t tk = s.first + rr / p.G;
            const int hq = h * p.G + rr % p.G;
            if (whole) {
                const float vs = E4M3 ? p.v_scale[h] : 1.0f;
                const float inv = ll == 0.f ? 0.f : vs / ll;
                const u32x2 y = {pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
                *reinterpret_cast<u32x2 *>(p.out.p + tk * p.out.row + (int64_t)hq * p.out.head + c) = y;
                if (c == 0 && p.lse)
                    p.lse[tk * p.H_q + hq] = lse_of(sm_mm[rr], ll);
            } else {
                const int64_t part = ((int64_t)w * 2 + slot) * TM + rr;
                *reinterpret_cast<f32x4 *>(p.part_o + part * D + c) = o;
                if (c == 0) {
                    p.part_ml[part * 2] = sm_mm[rr];
                    p.part_ml[part * 2 + 1] = ll;
                }
            }
        }
    }
}

// The rows whose keys were cut into pieces: their parts' (o, m, l) together, in a
// fixed order.  blockIdx = the piece they begin in and the row of the tile; eight
// waves take every eighth part, four at a time with their sums, and meet in LDS.
constexpr int JT = 512;
template <int D, bool E4M3>
__global__ __launch_bounds__(JT) void attn_join_kernel(AttnParams p)
{
    constexpr int E = D / 64, JW = JT / 64, BATCH = 4;
    __shared__ float sm_m[JW], sm_l[JW], sm_o[JW][D];
    const int w0 = blockIdx.x;
    const Cut c = read_cut(p, w0);
    if (c.last < 0)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int w1 = c.last < p.workgroups ? c.last : p.workgroups - 1, slot0 = c.slot, h = c.h;
    // few parts: a wave a row, eight rows a workgroup; many: eight waves a row
    const bool alone = w1 - w0 < BATCH;
    const int rr = alone ? blockIdx.y * JW + wave : blockIdx.y;
    const int step = alone ? 1 : JW;
    if (rr >= c.rows)
        return; // alone: each wave for itself, with no barrier behind
    const int64_t t = c.first + rr / p.G;
    const int hq = h * p.G + rr % p.G;
    float m = neg_inf(), l = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
        o[i] = 0.f;
    for (int w = alone ? w0 : w0 + wave; w <= w1; w += step * BATCH) {
        float pm[BATCH], pl[BATCH], po[BATCH][E];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int wk = w + k * step <= w1 ? w + k * step : w;
            const int64_t part = ((int64_t)wk * 2 + (wk == w0 ? slot0 : 0)) * TM + rr;
            pm[k] = p.part_ml[part * 2];
            pl[k] = p.part_ml[part * 2 + 1];
#pragma unroll
            for (int i = 0; i < E; ++i)
                po[k][i] = p.part_o[part * D + i * 64 + lane];
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            top = fmaxf(top, pm[k]);
        const float safe = top == neg_inf() ? 0.f : top;
        const float keep = __builtin_amdgcn_exp2f(m - safe);
        l *= keep;
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] *= keep;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (w + k * step <= w1) { // uniform
                const float f = __builtin_amdgcn_exp2f(pm[k] - safe);
                l = fmaf(pl[k], f, l);
#pragma unroll
                for (int i = 0; i < E; ++i)
                    o[i] = fmaf(po[k][i], f, o[i]);
            }
        }
        m = top;
    }
    const float vs = E4M3 ? p.v_scale[h] : 1.0f;
    if (alone) {
        const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll
        for (int i = 0; i < E; ++i)
            p.out.p[t * p.out.row + (int64_t)hq * p.out.head + i * 64 + lane] = f32_to_bf16_rne(o[i] * inv);
        if (lane == 0 && p.lse)
            p.lse[t * p.H_q + hq] = lse_of(m, l);
        return;
    }
    if (lane == 0) {
        sm_m[wave] = m;
        sm_l[wave] = l;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        sm_o[wave][i * 64 + lane] = o[i];
    __syncthreads();
    if (tid < D) {
        float top = neg_inf();
#pragma unroll
        for (int k = 0; k < JW; ++k)
            top = fmaxf(top, sm_m[k]);
        const float safe = top == neg_inf() ? 0.f : top;
        float sum = 0.f, x = 0.f;
#pragma unroll
        for (int k = 0; k < JW; ++k) {
            const float f = __builtin_amdgcn_exp2f(sm_m[k] - safe);
            sum = fmaf(sm_l[k], f, sum);
            x = fmaf(sm_o[k][tid], f, x);
        }
        const float inv = sum == 0.f ? 0.f : vs / sum;
        p.out.p[t * p.out.row + (int64_t)hq * p.out.head + tid] = f32_to_bf16_rne(x * inv);
        if (tid == 0 && p.lse)
            p.lse[t * p.H_q + hq] = lse_of(top, sum);
    }
}

size_t attn_rows_layout(int d, void *base, AttnParams *p)
{
    // Two a CU.  Us a call with one / two / three: 8 sequences of 40-131 thousand e4m3 tokens at 32/4
    // heads of 128 129 / 114 / 122; 32 sequences of 4 tokens over 0.05-3 thousand at 32/8 heads of 128,
    // window 1024, 38.7 / 34.4 / 36.6 (inputs that stay in the memory-side cache; 40 with others each
    // call); 64 sequences of 0.2-8 thousand at 16/4 heads of 256 219 / 224 / 230.
    const int workgroups = 2 * device_cus();
    const size_t o = round256((size_t)workgroups * 2 * TM * d * 4), ml = round256((size_t)workgroups * 2 * TM * 2 * 4),
                 cut = round256((size_t)workgroups * 8 * 4);
    if (p) {
        p->workgroups = workgroups;
        p->part_o = static_cast<float *>(base);
        p->part_ml = reinterpret_cast<float *>(static_cast<char *>(base) + o);
        p->cut = reinterpret_cast<int32_t *>(static_cast<char *>(base) + o + ml);
    }
    return o + ml + cut;
}

template <int D, bool E4M3>
static hipError_t launch_de(const AttnParams &p, hipStream_t stream)
{
    AttnParams q = p;
    void *args[] = {&q};
    const int most = p.max_new * p.G; // rows of a sequence that can be cut
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_rows_kernel<D, E4M3>),
                                   dim3((unsigned)p.workgroups), dim3(NT), args, 0, stream);
    if (e == hipSuccess && most > 0)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_join_kernel<D, E4M3>),
                            dim3((unsigned)p.workgroups, (unsigned)(most < TM ? most : TM)), dim3(JT), args, 0,
                            stream);
    return e;
}

hipError_t launch_attn_rows(const AttnParams &p, int d, bool e4m3, hipStream_t stream)
{
    if (d == 64)
        return e4m3 ? launch_de<64, true>(p, stream) : launch_de<64, false>(p, stream);
    if (d == 128)
        return e4m3 ? launch_de<128, true>(p, stream) : launch_de<128, false>(p, stream);
    return e4m3 ? launch_de<256, true>(p, stream) : launch_de<256, false>(p, stream);
}

// Up to one tile of rows a sequence this kernel is used: it reads a sequence's keys once per 16
// rows, the other (attn_tiles.hip) once for 256, but through LDS and with a third launch, and its
// weights are bf16.  Rows here / there in us a call, bf16: 64 sequences over 2-4 thousand tokens, 32/4
// heads of 128: 8 rows 80 / 88, 16 rows 87 / 92; 8 over 0.5-1 thousand, 32/8 heads of 64: 4 rows 12.5 /
// 21, 16 rows 16.6 / 21; 12 over 2-4 thousand, 16/2 heads of 256: 8 rows 33 / 37, 16 rows 41 / 36.5 (the
// one point where there is faster).  With a tile per 16 rows this kernel lost past them: 32 rows 128 / 96
// and 50 / 38 at the first and last of these, 64 rows 239 / 105.
constexpr int kFewRows = 16;

bool attn_few_rows(int max_new, int G) { return (int64_t)max_new * G <= kFewRows; }

size_t attn_paged_layout(int B, int T, int max_new, int H_kv, int G, int d, void *base, AttnParams *p)
{
    if (attn_few_rows(max_new, G))
        return attn_rows_layout(d, base, p);
    return attn_tiles_layout(B, T, H_kv, G, d, base, p);
}

hipError_t launch_attn_paged(const AttnParams &p, int d, bool e4m3, hipStream_t stream)
{
    return attn_few_rows(p.max_new, p.G) ? launch_attn_rows(p, d, e4m3, stream) : launch_attn_tiles(p, d, e4m3, stream);
}

} // namespace gdn
