// attn_tiles.hip -- paged attention of prompt chunks: tiles of 256 rows (gfx950).
//
// The same sums as attn_paged.hip (one pass over the keys with a running maximum
// and sum) where a sequence has many (token, head of the group) rows.  A workgroup
// of eight waves takes 256 rows of one kv head, 32 a wave, and walks the keys in
// blocks of 64; k and v of the next block come into LDS, straight from memory
// where the cache is bf16, while this one is worked on, so there is one barrier a
// block.  S^T = K Q^T and O^T = V^T P^T in 32 x 32 x 16 bf16 products: a lane's
// scores are eight consecutive-by-four keys of its own row, and they are the P^T
// operand as they stand when the contraction's places go to the keys in that
// order; V^T comes out of LDS by transposing reads.
//
// LDS rows are 16-byte chunks, chunk c of key j at c ^ f(j): the 16 keys of a K
// read fall on different banks, and so do the four keys of a transposing read.
//
// The running maximum is only raised when a row's scores pass it by 2^8: weights
// stay below 256, in fp32 and in bf16, and most blocks skip the rescaling of o.
//
// Work is dealt out by the key: a first kernel lists every (sequence, kv head,
// tile) with its blocks that the causal mask and the window leave; the line of
// all blocks is cut into one piece a workgroup, and what is cut is joined by a
// third kernel.

#include "attn_common.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int TR = 256;  // rows of a tile
// keys of a block: with 256 columns the queries take half of the LDS
constexpr int block_keys(int d) { return d == 256 ? 32 : 64; }
constexpr int PT = 1024; // the planning workgroup

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(1))) const uint32_t global_u32;

// What a tile of a sequence sees: keys lo .. hi - 1, in blocks from lo on.
struct Span {
    int lo, hi, blocks, min_pos, max_pos;
};

__device__ __forceinline__ Span span_of(const AttnParams &p, const Seq &s, int tile)
{
    Span x;
    const int rows = s.n * p.G;
    const int last = (rows < (tile + 1) * TR ? rows : (tile + 1) * TR) - 1;
    x.min_pos = s.L - s.n + tile * TR / p.G;
    x.max_pos = s.L - s.n + last / p.G;
    x.hi = s.kind == kNormal && x.max_pos >= 0 ? x.max_pos + 1 : 0;
    x.lo = 0;
    if (p.window > 0 && x.min_pos - p.window + 1 > 0)
        x.lo = (x.min_pos - p.window + 1) & ~(p.block - 1);
    x.lo = x.lo < x.hi ? x.lo : (x.hi > 0 ? (x.hi - 1) & ~(p.block - 1) : 0);
    x.blocks = x.hi > x.lo ? (x.hi - x.lo + p.block - 1) / p.block : 1;
    return x;
}

__device__ __forceinline__ int tiles_of(const AttnParams &p, const Seq &s)
{
    return s.kind == kSkip ? 0 : (int)(((int64_t)s.n * p.G + TR - 1) / TR);
}

// The entry that holds unit u (before[e] <= u < before[e + 1]): 64 probes a round.
__device__ __forceinline__ int entry_of(const long long *before, int count, long long u)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && before[at] <= u;
        const int n = __popcll(__ballot(le));
        lo += n * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

// Exclusive sum over the planning workgroup.
template <class T>
__device__ __forceinline__ T plan_scan(T v, T *total)
{
    __shared__ T wave_sum[PT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T inc = v;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const T o = __shfl_up(inc, m);
        if (lane >= m)
            inc += o;
    }
    __syncthreads();
    if (lane == 63)
        wave_sum[wave] = inc;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < PT / 64; ++w) {
        before += w < wave ? wave_sum[w] : 0;
        all += wave_sum[w];
    }
    *total = all;
    return before + inc - v;
}

} // namespace

// The list of entries (sequence, kv head, tile), tiles fastest: neighbouring
// pieces then walk the same keys.
__global__ __launch_bounds__(PT) void attn_plan_kernel(AttnParams p)
{
    __shared__ int first_entry[PT + 1];
    __shared__ Seq seqs[PT];
    int entries = 0;
    long long units = 0;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + threadIdx.x;
        int mine = 0;
        __syncthreads(); // the round before has read the tables
        if (b < p.B) {
            const Seq s = read_seq(p, b);
            seqs[threadIdx.x] = s;
            mine = tiles_of(p, s) * p.H_kv;
        }
        int all;
        first_entry[threadIdx.x] = plan_scan(mine, &all);
        if (threadIdx.x == 0)
            first_entry[PT] = all;
        __syncthreads();
        for (int e0 = 0; e0 < all; e0 += PT) {
            const int e = e0 + threadIdx.x;
            long long u = 0;
            int q = 0, h = 0, tile = 0;
            if (e < all) {
                int lo = 0, hi = PT; // the last sequence with first_entry <= e
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (first_entry[mid] <= e)
                        lo = mid;
                    else
                        hi = mid;
                }
                q = lo;
                const Seq s = seqs[q];
                const int tiles = tiles_of(p, s), x = e - first_entry[q];
                h = x / tiles;
                tile = x - h * tiles;
                u = span_of(p, s, tile).blocks;
            }
            long long sum;
            const long long at = units + plan_scan(u, &sum);
            if (e < all) {
                const int64_t o = entries + e;
                p.before[o] = at;
                p.entry[o * 3] = b0 + q;
                p.entry[o * 3 + 1] = h;
                p.entry[o * 3 + 2] = tile;
            }
            units += sum;
        }
        entries += all;
    }
    if (threadIdx.x == 0) {
        p.before[entries] = units;
        *p.count = entries;
    }
}

// NW waves of RS times 32 rows.
template <int D, bool E4M3, int NW, int RS>
__global__ __launch_bounds__(64 * NW, NW / 4) void attn_tiles_kernel(AttnParams p)
{
    static_assert(NW * RS * 32 == TR, "a workgroup's rows");
    constexpr int NT = 64 * NW;
    constexpr int CH = D / 8;                 // chunks of a row
    constexpr int ST = D / 16;                // steps of a score's contraction
    constexpr int DT = D / 32;                // 32-column tiles of o
    constexpr int ROWB = D * 2;               // bytes of an LDS row
    constexpr int KB = block_keys(D);
    constexpr int NS = KB / 32;
    // steps whose queries a lane keeps in LDS, each lane its own: all 16 of 256 columns in
    // registers, beside 128 of o, spill
    constexpr int QL = D == 256 ? 8 : 0;
    __shared__ __align__(16) uint8_t sm_k[2][KB * ROWB], sm_v[2][KB * ROWB];
    __shared__ int sm_odd[2];
    __shared__ u32x4 sm_q[QL ? NW * RS * QL * 64 : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n_ = lane & 31, hh = lane >> 5;
    const int count = *p.count;
    const long long total = p.before[count];
    // consecutive pieces on one XCD (workgroups go round the eight): they share keys in its L2
    const int per = p.workgroups / 8;
    const int w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tid == 0)
        write_cut(p, w, Cut{-1});
    const int pieces = pieces_of(p, total);
    if (w >= pieces)
        return;
    long long u = piece_begin(total, w, pieces);
    const long long u_begin = u, u_end = piece_begin(total, w + 1, pieces);
    int e = uniform(entry_of(p.before, count, u));

    // a 16-byte chunk's place within its row
    auto swizzle = [](int key) {
        return D == 64 ? (((key >> 1) & 1) << 2) | ((key >> 2) & 3) : ((key & 3) << 2) | ((key >> 2) & 3);
    };
    // K reads: this lane's key of a 32-key part, and its chunk without the step's
    const int k_row = n_ * ROWB, k_chunk = (hh ^ swizzle(n_)) * 16;
    // V reads: lane (hv, r, c) points at key 4 hv + r (+ 8 for the second), columns 4 c
    const int gr = lane >> 4, r_ = (lane & 15) >> 2, c_ = lane & 3;
    int v_base[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int key = 8 * q + 4 * (gr >> 1) + r_;
        v_base[q] = key * ROWB + ((((gr & 1) * 2 + (c_ >> 1)) ^ swizzle(key)) * 16) + (c_ & 1) * 8;
    }

    while (u < u_end) {
        const int b = uniform(p.entry[(int64_t)e * 3]), h = uniform(p.entry[(int64_t)e * 3 + 1]),
                  tile = uniform(p.entry[(int64_t)e * 3 + 2]);
        const long long t0 = p.before[e], t1 = p.before[e + 1];
        const Seq s = read_seq(p, b);
        const Span span = span_of(p, s, tile);
        const long long stop = t1 < u_end ? t1 : u_end;
        const int blk0 = (int)(u - t0), blk1 = (int)(stop - t0);
        const bool whole = u == t0 && stop == t1;
        const int slot = u == u_begin ? 0 : 1;
        if (tid == 0 && u == t0 && stop < t1)
            write_cut(p, w, Cut{owner_of(total, t1 - 1, pieces), slot, s.first, s.n * p.G, h, tile});
        u = stop;
        ++e;

        const int rows = s.n * p.G;
        const int row0 = tile * TR + wave * (32 * RS); // this wave's first
        const bool any = row0 < rows && s.kind == kNormal;
        int pos[RS]; // of this lane's rows
#pragma unroll
        for (int x = 0; x < RS; ++x) {
            const int row = row0 + 32 * x + n_;
            pos[x] = row < rows && s.kind == kNormal ? s.L - s.n + row / p.G : -1;
        }
        const int reach = p.window > 0 ? p.window - 1 : 0x3fffffff; // a row sees keys pos - reach .. pos
        const int row1 = (rows < row0 + 32 * RS ? rows : row0 + 32 * RS) - 1;
        const int min_pos = uniform(s.L - s.n + row0 / p.G), max_pos = uniform(any ? s.L - s.n + row1 / p.G : -1);

        // scores are masked before they are scaled, so the scale has to be positive: a negative
        // one moves its sign into q, zero makes q zero
        float scale = E4M3 ? p.scale * p.k_scale[h] : p.scale;
        const uint32_t flip = scale < 0.f ? 0x80008000u : 0u, wipe = scale == 0.f ? 0u : 0xffffffffu;
        scale = scale == 0.f ? 1.0f : fabsf(scale);
        bf16x8 qf[RS][ST - QL];
        float m[RS], l[RS];
        f32x16 acc[RS][DT];
        bool bad[RS];
#pragma unroll
        for (int x = 0; x < RS; ++x) {
            int r = row0 + 32 * x + n_;
            r = r < rows ? r : rows - 1; // rows past the last do as it does, unseen
            const uint16_t *qp = p.q.p + (int64_t)(s.first + r / p.G) * p.q.row +
                                 (int64_t)(h * p.G + r % p.G) * p.q.head + hh * 8;
#pragma unroll
            for (int i = 0; i < ST; ++i) {
                const u32x4 q = (*reinterpret_cast<const u32x4 *>(qp + i * 16) ^ flip) & wipe;
                if (i < QL)
                    sm_q[((wave * RS + x) * QL + i) * 64 + lane] = q;
                else
                    qf[x][i - QL] = __builtin_bit_cast(bf16x8, q);
            }
            m[x] = neg_inf();
            l[x] = 0.f;
            bad[x] = false;
#pragma unroll
            for (int a = 0; a < DT; ++a)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[x][a][i] = 0.f;
        }
        const int32_t *tab = p.page_table + (int64_t)s.r * p.width;
        const int inside = (1 << p.page_shift) - 1;

        // a key's page; 0 (the null page) where there is none
        auto page_of = [&](int key) {
            const int pg = key < s.L ? tab[key >> p.page_shift] : 0;
            return pg < 1 || pg >= p.N ? 0 : pg;
        };
        // which of a block's 16-key parts hold keys on a page outside the pool
        int missing = 0;
        auto find_missing = [&](int key0) {
            missing = 0;
#pragma unroll
            for (int q = 0; q < KB / 16; ++q)
                if (key0 + 16 * q < s.L && page_of(key0 + 16 * q) == 0)
                    missing |= 1 << q;
        };
        auto cell_of = [&](int key) {
            return (((int64_t)page_of(key) * p.H_kv + h) << p.page_shift) + (key & inside);
        };
        // bf16: k and v of a block into LDS, one 1 KiB instruction at a time
        constexpr int PER = KB * CH / 64 / NW; // of each array, a wave
        constexpr int RP = 64 / CH;            // rows of an instruction
        static_assert(PER * NW * RP == KB, "every row of a block is staged once");
        auto stage = [&](int key0, int buf) {
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                const int r0 = (wave * PER + q) * RP;
                const int64_t cell = cell_of(key0 + r0);
                const int rl = lane / CH;
                const int off = rl * ROWB + ((lane % CH) ^ swizzle(r0 + rl)) * 16;
                const uint8_t *kp = static_cast<const uint8_t *>(p.k_pages) + cell * ROWB;
                const uint8_t *vp = static_cast<const uint8_t *>(p.v_pages) + cell * ROWB;
                __builtin_amdgcn_global_load_lds((global_u32 *)(kp + off), (lds_u32 *)&sm_k[buf][r0 * ROWB], 16, 0, 0);
                __builtin_amdgcn_global_load_lds((global_u32 *)(vp + off), (lds_u32 *)&sm_v[buf][r0 * ROWB], 16, 0, 0);
            }
        };
        // e4m3: through registers, 16 values at a time, which become two chunks
        constexpr int PE = KB * D / 16 > NT ? KB * D / 16 / NT : 1;
        u32x4 ek[PE], ev[PE];
        auto fetch = [&](int key0) {
#pragma unroll
            for (int q = 0; q < PE; ++q) {
                const int x = tid + q * NT, r0 = x / (D / 16), c = x % (D / 16);
                if (r0 < KB) {
                    const int64_t cell = cell_of(key0 + r0);
                    ek[q] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(p.k_pages) + cell * D + c * 16);
                    ev[q] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(p.v_pages) + cell * D + c * 16);
                }
            }
        };
        auto put = [&](int buf) {
#pragma unroll
            for (int q = 0; q < PE; ++q) {
                const int x = tid + q * NT, r0 = x / (D / 16), c = x % (D / 16);
                if (r0 < KB) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int at = r0 * ROWB + ((2 * c + y) ^ swizzle(r0)) * 16;
                        *reinterpret_cast<u32x4 *>(&sm_k[buf][at]) =
                            u32x4{e4m3_to_bf16<false>(ek[q][2 * y]), e4m3_to_bf16<true>(ek[q][2 * y]),
                                  e4m3_to_bf16<false>(ek[q][2 * y + 1]), e4m3_to_bf16<true>(ek[q][2 * y + 1])};
                        *reinterpret_cast<u32x4 *>(&sm_v[buf][at]) =
                            u32x4{e4m3_to_bf16<false>(ev[q][2 * y]), e4m3_to_bf16<true>(ev[q][2 * y]),
                                  e4m3_to_bf16<false>(ev[q][2 * y + 1]), e4m3_to_bf16<true>(ev[q][2 * y + 1])};
                    }
                }
            }
        };

        const int end = span.hi > span.lo ? blk1 : blk0; // no keys: nothing to walk
        __syncthreads(); // the buffers of the piece before are read
        if (tid < 2)
            sm_odd[tid] = 0;
        if (blk0 < end) {
            find_missing(span.lo + blk0 * KB);
            if constexpr (E4M3) {
                fetch(span.lo + blk0 * KB);
                put(0);
            } else {
                stage(span.lo + blk0 * KB, 0);
            }
        }
        for (int blk = blk0; blk < end; ++blk) {
            const int buf = (blk - blk0) & 1, key0 = span.lo + blk * KB;
            const int lost = missing;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // this wave's part of the block is in LDS
            __syncthreads();
            if (blk + 1 < end) {
                find_missing(key0 + KB);
                if constexpr (E4M3)
                    fetch(key0 + KB);
                else
                    stage(key0 + KB, buf ^ 1);
            }
            // A block that some row does not see whole: v of keys past the sequence's last is cleared,
            // and so are infinities and NaN, which 0 times would carry into rows that do not see them.
            bool odd = false;
            if (key0 + KB - 1 > span.min_pos || (p.window > 0 && key0 <= span.max_pos - p.window)) {
                if (tid == 0)
                    sm_odd[buf ^ 1] = 0;
#pragma unroll
                for (int q = 0; q < KB * CH / NT; ++q) {
                    const int x = tid + q * NT, key = key0 + x / CH;
                    u32x4 *at = reinterpret_cast<u32x4 *>(&sm_v[buf][x * 16]);
                    u32x4 v = *at;
                    bool found = false;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const bool lo_odd = (v[y] & 0x7f80u) == 0x7f80u, hi_odd = (v[y] & 0x7f800000u) == 0x7f800000u;
                        found |= lo_odd | hi_odd;
                        v[y] &= (lo_odd ? 0xffff0000u : 0xffffffffu) & (hi_odd ? 0xffffu : 0xffffffffu);
                    }
                    if (key >= s.L)
                        *at = u32x4{0u, 0u, 0u, 0u};
                    else if (found) {
                        *at = v;
                        sm_odd[buf] = 1;
                    }
                }
                __syncthreads();
                odd = sm_odd[buf] != 0;
            }
            if (any && key0 <= max_pos && !(p.window > 0 && key0 + KB - 1 <= min_pos - p.window)) {
                if (lost) {
#pragma unroll
                    for (int q = 0; q < KB / 16; ++q)
#pragma unroll
                        for (int x = 0; x < RS; ++x)
                            bad[x] |= (lost >> q & 1) && pos[x] >= key0 + 16 * q && pos[x] - reach <= key0 + 16 * q + 15;
                }
                // the LDS addresses are formed anew each block: kept, they cost 16 registers
                int k_at = k_chunk, v_at[2] = {v_base[0], v_base[1]};
                asm volatile("" : "+v"(k_at), "+v"(v_at[0]), "+v"(v_at[1]));
                const bool mixed = key0 + KB - 1 > min_pos || (p.window > 0 && key0 <= max_pos - p.window);
                const uint8_t *kb = sm_k[buf], *vb = sm_v[buf];
                {
                    f32x16 sc[RS][NS];
#pragma unroll
                    for (int x = 0; x < RS; ++x)
#pragma unroll
                        for (int y = 0; y < NS; ++y)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                sc[x][y][i] = 0.f;
#pragma unroll
                    for (int i = 0; i < ST; ++i)
#pragma unroll
                        for (int y = 0; y < NS; ++y) {
                            const u32x4 kf = *reinterpret_cast<const u32x4 *>(
                                kb + y * 32 * ROWB + k_row + (k_at ^ ((i & 7) * 32)) + (i >> 3) * 256);
#pragma unroll
                            for (int x = 0; x < RS; ++x) {
                                bf16x8 q;
                                if (i < QL)
                                    q = __builtin_bit_cast(bf16x8, sm_q[((wave * RS + x) * QL + i) * 64 + lane]);
                                else
                                    q = qf[x][i - QL];
                                sc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf), q,
                                                                                   sc[x][y], 0, 0, 0);
                            }
                        }
#pragma unroll
                    for (int x = 0; x < RS; ++x)
#pragma unroll
                        for (int y = 0; y < NS; ++y)
                            settle(sc[x][y]);
                    if (mixed) {
#pragma unroll
                        for (int x = 0; x < RS; ++x)
#pragma unroll
                            for (int y = 0; y < NS; ++y)
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const int back =
                                        pos[x] - (key0 + y * 32 + 8 * (i >> 2) + 4 * hh + (i & 3));
                                    if (back < 0 || back > reach)
                                        sc[x][y][i] = neg_inf();
                                }
                    }
                    float top[RS];
                    bool raise = false;
#pragma unroll
                    for (int x = 0; x < RS; ++x) {
                        top[x] = sc[x][0][0];
#pragma unroll
                        for (int y = 0; y < NS; ++y)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                top[x] = fmaxf(top[x], sc[x][y][i]);
                        top[x] = fmaxf(top[x], __shfl_xor(top[x], 32)) * scale;
                        raise |= top[x] > m[x] + 8.0f;
                    }
                    if (__ballot(raise)) {
#pragma unroll
                        for (int x = 0; x < RS; ++x) {
                            const float m_new = fmaxf(m[x], top[x]);
                            const float keep = m_new == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m[x] - m_new);
                            l[x] *= keep;
#pragma unroll
                            for (int a = 0; a < DT; ++a)
                                acc[x][a] *= keep;
                            m[x] = m_new;
                        }
                    }
                    bf16x8 pf[RS][2 * NS];
#pragma unroll
                    for (int x = 0; x < RS; ++x) {
                        const float off = m[x] == neg_inf() ? 0.f : -m[x];
                        float sum = 0.f;
#pragma unroll
                        for (int q = 0; q < 2 * NS; ++q) {
                            float e[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                e[i] = __builtin_amdgcn_exp2f(fmaf(sc[x][q >> 1][8 * (q & 1) + i], scale, off));
                                sum += e[i];
                            }
                            // rounded to bf16 for the matrix cores: off by at most 2^-9 of itself, and
                            // o is rounded to bf16 in the end
                            pf[x][q] = __builtin_bit_cast(bf16x8,
                                                          u32x4{pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]),
                                                                pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7])});
                        }
                        l[x] += sum;
                    }
#pragma unroll
                    for (int q = 0; q < 2 * NS; ++q)
#pragma unroll
                        for (int a = 0; a < DT; ++a) {
                            u32x4 vf;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const u32x2 v2 = __builtin_bit_cast(
                                    u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                               (__attribute__((address_space(3))) s16x4 *)(vb + q * 16 * ROWB +
                                                                                           (v_at[y] ^ ((a & 3) * 64)) +
                                                                                           (a >> 2) * 256)));
                                vf[2 * y] = v2[0];
                                vf[2 * y + 1] = v2[1];
                            }
#pragma unroll
                            for (int x = 0; x < RS; ++x)
                                acc[x][a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf),
                                                                                    pf[x][q], acc[x][a], 0, 0, 0);
                        }
                    if (odd) { // uniform: what left the product goes to the rows that see it
                        for (int j = 0; j < KB && key0 + j < s.L; ++j) {
                            const int64_t cell = cell_of(key0 + j) * D;
#pragma unroll
                            for (int a = 0; a < DT; ++a)
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const int64_t at = cell + a * 32 + 8 * (i >> 2) + 4 * hh + (i & 3);
                                    uint32_t y;
                                    if constexpr (E4M3)
                                        y = e4m3_to_bf16<false>(static_cast<const uint8_t *>(p.v_pages)[at]) << 16;
                                    else
                                        y = (uint32_t) static_cast<const uint16_t *>(p.v_pages)[at] << 16;
#pragma unroll
                                    for (int x = 0; x < RS; ++x) {
                                        const int back = pos[x] - (key0 + j);
                                        if (back >= 0 && back <= reach && (y & 0x7f800000u) == 0x7f800000u)
                                            acc[x][a][i] += __uint_as_float(y);
                                    }
                                }
                        }
                    }
                }
            }
            if constexpr (E4M3) {
                if (blk + 1 < end)
                    put(buf ^ 1);
            }
        }
#pragma unroll
        for (int x = 0; x < RS; ++x) {
            const int row = row0 + 32 * x + n_;
            l[x] += __shfl_xor(l[x], 32);
            if (((int)bad[x] | __shfl_xor((int)bad[x], 32)) || s.kind == kNan)
                l[x] = quiet_nan();
            if (row >= rows)
                continue;
            const int64_t tk = s.first + row / p.G;
            const int head = h * p.G + row % p.G;
            if (whole) {
                const float vs = E4M3 ? p.v_scale[h] : 1.0f;
                const float inv = l[x] == 0.f ? 0.f : vs / l[x];
                uint16_t *o = p.out.p + tk * p.out.row + (int64_t)head * p.out.head + 4 * hh;
#pragma unroll
                for (int a = 0; a < DT; ++a)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<u32x2 *>(o + a * 32 + 2 * i) =
                            u32x2{pack_bf16(acc[x][a][i] * inv, acc[x][a][i + 1] * inv),
                                  pack_bf16(acc[x][a][i + 2] * inv, acc[x][a][i + 3] * inv)};
                if (hh == 0 && p.lse)
                    p.lse[tk * p.H_q + head] = lse_of(m[x], l[x]);
            } else {
                const int64_t part = ((int64_t)w * 2 + slot) * TR + (row - tile * TR);
                float *o = p.part_o + part * D + 4 * hh;
#pragma unroll
                for (int a = 0; a < DT; ++a)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<f32x4 *>(o + a * 32 + 2 * i) =
                            f32x4{acc[x][a][i], acc[x][a][i + 1], acc[x][a][i + 2], acc[x][a][i + 3]};
                if (hh == 0) {
                    p.part_ml[part * 2] = m[x];
                    p.part_ml[part * 2 + 1] = l[x];
                }
            }
        }
    }
}

// blockIdx.x = a piece: what begins in it and goes on in the next; a wave a row of it.
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void attn_tiles_join_kernel(AttnParams p)
{
    constexpr int E = D / 64, BATCH = 2;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int w0 = blockIdx.x;
    const Cut c = read_cut(p, w0);
    if (c.last < 0)
        return;
    const int w1 = c.last < p.workgroups ? c.last : p.workgroups - 1, slot0 = c.slot, h = c.h;
    for (int rr = blockIdx.y * 4 + wave; rr < TR; rr += gridDim.y * 4) {
        const int row = c.tile * TR + rr;
        if (row >= c.rows)
            break;
        auto part_of = [&](int w) { return ((int64_t)w * 2 + (w == w0 ? slot0 : 0)) * TR + rr; };
        float m = neg_inf(), l = 0.f, o[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] = 0.f;
        for (int w = w0; w <= w1; w += BATCH) {
            float pm[BATCH], pl[BATCH], po[BATCH][E];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int64_t part = part_of(w + k <= w1 ? w + k : w);
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
                if (w + k <= w1) {
                    const float f = __builtin_amdgcn_exp2f(pm[k] - safe);
                    l = fmaf(pl[k], f, l);
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        o[i] = fmaf(po[k][i], f, o[i]);
                }
            }
            m = top;
        }
        const int64_t t = c.first + row / p.G;
        const int hq = h * p.G + row % p.G;
        const float vs = E4M3 ? p.v_scale[h] : 1.0f;
        const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll
        for (int i = 0; i < E; ++i)
            p.out.p[t * p.out.row + (int64_t)hq * p.out.head + i * 64 + lane] = f32_to_bf16_rne(o[i] * inv);
        if (lane == 0 && p.lse)
            p.lse[t * p.H_q + hq] = lse_of(m, l);
    }
}

size_t attn_tiles_layout(int B, int T, int H_kv, int G, int d, void *base, AttnParams *p)
{
    const int workgroups = (device_cus() + 7) / 8 * 8;
    const size_t entries = ((size_t)T * G / TR + B) * H_kv;
    const size_t o = round256((size_t)workgroups * 2 * TR * d * 4), ml = round256((size_t)workgroups * 2 * TR * 2 * 4),
                 bf = round256((entries + 1) * 8), en = round256(entries * 3 * 4),
                 cut = round256((size_t)workgroups * 8 * 4);
    if (p) {
        char *at = static_cast<char *>(base);
        p->workgroups = workgroups;
        p->part_o = reinterpret_cast<float *>(at);
        p->part_ml = reinterpret_cast<float *>(at + o);
        p->before = reinterpret_cast<long long *>(at + o + ml);
        p->entry = reinterpret_cast<int32_t *>(at + o + ml + bf);
        p->cut = reinterpret_cast<int32_t *>(at + o + ml + bf + en);
        p->count = reinterpret_cast<int32_t *>(at + o + ml + bf + en + cut);
    }
    return o + ml + bf + en + cut + 256;
}

template <int D, bool E4M3>
static hipError_t launch_de(const AttnParams &p, hipStream_t stream)
{
    AttnParams q = p;
    q.block = block_keys(D);
    void *args[] = {&q};
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_plan_kernel), dim3(1), dim3(PT), args, 0,
                                   stream);
    constexpr int NW = 8;
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_tiles_kernel<D, E4M3, NW, 8 / NW>),
                            dim3((unsigned)p.workgroups), dim3(64 * NW), args, 0, stream);
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_tiles_join_kernel<D, E4M3>),
                            dim3((unsigned)p.workgroups, 32), dim3(256), args, 0, stream);
    return e;
}

hipError_t launch_attn_tiles(const AttnParams &p, int d, bool e4m3, hipStream_t stream)
{
    if (d == 64)
        return e4m3 ? launch_de<64, true>(p, stream) : launch_de<64, false>(p, stream);
    if (d == 128)
        return e4m3 ? launch_de<128, true>(p, stream) : launch_de<128, false>(p, stream);
    return e4m3 ? launch_de<256, true>(p, stream) : launch_de<256, false>(p, stream);
}

} // namespace gdn
