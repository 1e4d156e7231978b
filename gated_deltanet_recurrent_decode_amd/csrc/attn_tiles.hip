// attn_tiles.hip -- paged attention of prompt chunks: tiles of 256 rows (gfx950).
//
// The same sums as attn_paged.hip (one pass over the keys with a running maximum
// and sum) where a sequence has many (token, head of the group) rows.  A workgroup
// of eight waves takes 256 rows of one kv head, 32 a wave, and walks the keys in
// blocks of 128 (of 32 with 256 columns); k and v of the next block come into LDS,
// straight from memory where the cache is bf16, while this one is worked on, so
// there is one barrier a block.  S^T = K Q^T and O^T = V^T P^T in 32 x 32 x 16 bf16
// products, 64 keys (32) at a time: a lane's scores are eight keys, four and four,
// of its own row, and they are the P^T operand as they stand when the contraction's
// places go to the keys in that order; V^T comes out of LDS by transposing reads.
//
// LDS rows are 16-byte chunks, chunk c of key j at c ^ f(j): the 16 keys of a K
// read fall on different banks, and so do the four keys of a transposing read (no
// bank conflicts are counted).
//
// The running maximum is only raised when a row's scores pass it by 2^8: weights
// stay below 256, in fp32 and in bf16, and most blocks skip the rescaling of o
// (raising it at once: the two sizes below 4 and 9% slower).  The largest weight of a
// row is then not 1 but rounded like the others, which shows in o as one more bf16
// rounding of its terms: 0.0023 of its norm from 64 bits in place of 0.0019.
//
// Work is dealt out by the key: a first kernel lists every (sequence, kv head,
// tile) with its blocks that the causal mask and the window leave; the line of
// all blocks is cut into one piece a workgroup, and what is cut is joined by a
// third kernel (26 us alone at 111 MB of parts, in the mixed step below; they lie in
// the workspace as they lay in the registers: 1 KiB a store).
//
// What bounds it: the two waves of a SIMD get their products and their weights
// overlapped by 40% only (counters: matrix cores busy 54% of the cycles, weights and
// masks 48%, a quarter waiting), because a wave's own work is a chain: scores,
// maximum, weights, products; and the card's power, for the clock falls to 1.7 GHz.
// MI355X, calls back to back, by card and session: 4096 + 3001 tokens at 16/2 heads of
// 128 over 8-12 thousand others 653 to 700 us (1022 to 953 TFLOP/s; an e4m3 cache 683 to
// 690, 64 columns 415 to 423, with a window of 1024 99 to 102 and at 64 columns 68 to 71);
// a mixed step of 12 sequences at 16/2 heads of 256 210 to 223 us (702 to 661 TFLOP/s;
// e4m3 220 to 225).
//
// A wave that forms its maximum goes before one with products, and that before one that
// forms scores (s_setprio: the chunks 673 -> 663 us a call).  Tried and slower, calls on
// one card each: the halves of the workgroup entering a block at different places (686 ->
// 704 us), two workgroups of 128 rows a CU (1% fewer cycles, but 663 -> 701: k and v
// staged twice lower the clock), weights as two bf16 numbers (699 -> 941, the mixed step
// 222 -> 276).  The kernel alone under the profiler, from 785 us: the next block's scores
// formed beside these weights (903; 32 more registers copied a block), the halves one
// phase apart by two barriers a block (892), the next block's loads spread between the
// score products (844).  A step's first LDS reads before the step: the same.  64 rows a
// wave, and blocks of 64 keys at 256 columns: spills.

#include "attn_common.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int TR = 256;  // rows of a tile
// keys of a block: with 256 columns the queries take half of the LDS
constexpr int block_keys(int d) { return d == 256 ? 32 : 128; }
constexpr int NW = TR / 32; // waves
constexpr int NT = 64 * NW;
constexpr int PT = 1024; // the planning workgroup
// what the plan says of an entry: kv head, tile, and its sequence, so that nobody reads the lengths again
constexpr int kEntry = 8;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint8_t lds_byte;

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

// 16 bytes a lane from base + off into LDS, lane after lane from `to` on.  As inline assembly
// because the compiler, given the builtin, waits for it before any read of LDS: the loads of the
// next block would be waited for before this one is worked on.  Whoever reads `to` waits for
// vmcnt(0) and a barrier first.
__device__ __forceinline__ void load_to_lds(lds_byte *to, const uint8_t *base, int off)
{
    const uint32_t at = (uint32_t)(uintptr_t)to;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform((int)at)), "v"(off),
                 "s"(base)
                 : "memory"); // m0 is reserved: whatever of the compiler's own needs it sets it first
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
        // sequences that overlap have more tiles than the workspace was sized for (and than 32 bits
        // count: 512 of 2^22 in a round): what is past its end is left out
        long long sum_all;
        const long long mine_at = plan_scan((long long)mine, &sum_all);
        const int room = p.capacity - entries, all = sum_all < room ? (int)sum_all : room;
        first_entry[threadIdx.x] = mine_at < all ? (int)mine_at : all;
        if (threadIdx.x == 0)
            first_entry[PT] = all;
        __syncthreads();
        for (int e0 = 0; e0 < all; e0 += PT) {
            const int e = e0 + threadIdx.x;
            long long u = 0;
            int q = 0, h = 0, tile = 0;
            Seq s{};
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
                s = seqs[q];
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
                i32x4 *to = reinterpret_cast<i32x4 *>(p.entry + o * kEntry);
                to[0] = i32x4{h, tile, s.kind, s.first};
                to[1] = i32x4{s.n, s.L, s.r, 0};
            }
            units += sum;
        }
        entries += all;
    }
    if (threadIdx.x == 0) {
        p.before[entries] = units;
        *p.count = entries;
        *reinterpret_cast<long long *>(p.count + 2) = units;
    }
}

template <int D, bool E4M3>
__global__ __launch_bounds__(NT, 2) void attn_tiles_kernel(AttnParams p)
{
    constexpr int CH = D / 8;                 // chunks of a row
    constexpr int ST = D / 16;                // steps of a score's contraction
    constexpr int DT = D / 32;                // 32-column tiles of o
    constexpr int ROWB = D * 2;               // bytes of an LDS row
    constexpr int KB = block_keys(D);
    constexpr int SB = D == 256 ? 32 : 64;    // keys of a softmax step
    constexpr int NS = SB / 32;
    constexpr int KA = D == 256 ? 2 : 4; // products whose LDS reads go ahead together
    // steps whose queries a lane keeps in LDS, each lane its own: all 16 of 256 columns in
    // registers, beside 128 of o, spill
    constexpr int QL = D == 256 ? (E4M3 ? 11 : 8) : 0;
    __shared__ __align__(16) uint8_t sm_k[2][KB * ROWB], sm_v[2][KB * ROWB];
    __shared__ int sm_odd[2];
    __shared__ __align__(8) uint8_t sm_lost[2][8]; // a block's 16-key parts whose page is outside the pool
    __shared__ u32x4 sm_q[QL ? NW * QL * 64 : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n_ = lane & 31, hh = lane >> 5;
    const int count = *p.count;
    const long long total = *reinterpret_cast<const long long *>(p.count + 2);
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
        const int32_t *entry = p.entry + (int64_t)e * kEntry;
        const int h = uniform(entry[0]), tile = uniform(entry[1]);
        const Seq s{uniform(entry[2]), uniform(entry[3]), uniform(entry[4]), uniform(entry[5]), 0, uniform(entry[6])};
        const long long t0 = p.before[e], t1 = p.before[e + 1];
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
        const int row0 = tile * TR + wave * 32; // this wave's first
        const bool any = row0 < rows && s.kind == kNormal;
        const int row = row0 + n_; // this lane's
        const int pos = row < rows && s.kind == kNormal ? s.L - s.n + row / p.G : -1;
        const int reach = p.window > 0 ? p.window - 1 : 0x3fffffff; // a row sees keys pos - reach .. pos
        const int row1 = (rows < row0 + 32 ? rows : row0 + 32) - 1;
        const int min_pos = uniform(s.L - s.n + row0 / p.G), max_pos = uniform(any ? s.L - s.n + row1 / p.G : -1);

        // scores are masked before they are scaled, so the scale has to be positive: a negative
        // one moves its sign into q, zero makes q zero
        float scale = E4M3 ? p.scale * p.k_scale[h] : p.scale;
        const uint32_t flip = scale < 0.f ? 0x80008000u : 0u, wipe = scale == 0.f ? 0u : 0xffffffffu;
        scale = scale == 0.f ? 1.0f : fabsf(scale);
        bf16x8 qf[ST - QL];
        float m = neg_inf(), l = 0.f;
        f32x16 acc[DT];
        int bad = 0;
        const int r = row < rows ? row : rows - 1; // rows past the last do as it does, unseen
        const uint16_t *qp = p.q.p + (int64_t)(s.first + r / p.G) * p.q.row +
                             (int64_t)(h * p.G + r % p.G) * p.q.head + hh * 8;
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            const u32x4 q = (*reinterpret_cast<const u32x4 *>(qp + i * 16) ^ flip) & wipe;
            if (i < QL)
                sm_q[(wave * QL + i) * 64 + lane] = q;
            else
                qf[i - QL] = __builtin_bit_cast(bf16x8, q);
        }
#pragma unroll
        for (int a = 0; a < DT; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[a][i] = 0.f;
        const int32_t *tab = p.page_table + (int64_t)s.r * p.width;
        const int inside = (1 << p.page_shift) - 1;

        // a key's page; 0 (the null page) where there is none
        auto page_of = [&](int key) {
            const int pg = key < s.L ? tab[key >> p.page_shift] : 0;
            return pg < 1 || pg >= p.N ? 0 : pg;
        };
        auto cell_of = [&](int key) {
            return (((int64_t)page_of(key) * p.H_kv + h) << p.page_shift) + (key & inside);
        };
        // Staging: a wave brings the same few rows of every block, all of them on one page.  Its
        // number is read a block ahead, by the scalar unit.
        constexpr int WR = KB / NW; // rows of a wave
        static_assert(WR <= 16, "on one page");
        const int my_row = wave * WR;
        auto *table = (__attribute__((address_space(4))) const int32_t *)tab;
        auto next_page = [&](int key0) {
            const int key = uniform(key0 + my_row);
            return key < s.L ? table[key >> p.page_shift] : 0;
        };
        auto first_cell = [&](int key0, int id) { // of the wave's rows
            return ((((int64_t)(id > 0 && id < p.N ? id : 0)) * p.H_kv + h) << p.page_shift) +
                   ((key0 + my_row) & inside);
        };
        // bf16: k or v of a block into LDS, 1 KiB an instruction
        auto stage = [&](const void *pages, lds_byte *to, int key0, int id) {
            constexpr int RP = 64 / CH; // rows of an instruction
            const uint8_t *from = static_cast<const uint8_t *>(pages) + first_cell(key0, id) * ROWB;
#pragma unroll
            for (int q = 0; q < WR / RP; ++q) {
                const int r0 = my_row + q * RP, rl = lane / CH;
                load_to_lds(to + r0 * ROWB, from, (q * RP + rl) * ROWB + ((lane % CH) ^ swizzle(r0 + rl)) * 16);
            }
        };
        // e4m3: through registers, 16 values a lane, which become two chunks
        constexpr int ER = 1024 / D, PE = WR / ER > 0 ? WR / ER : 1; // rows of a load, loads
        u32x4 ek[PE], ev[PE];
        const int er = my_row + lane / (D / 16), ec = lane % (D / 16);
        auto fetch = [&](const void *pages, u32x4(&x)[PE], int key0, int id) {
            const uint8_t *from = static_cast<const uint8_t *>(pages) + first_cell(key0, id) * D + lane * 16;
#pragma unroll
            for (int q = 0; q < PE; ++q)
                x[q] = *reinterpret_cast<const u32x4 *>(from + q * 1024);
        };
        auto put = [&](uint8_t *to, const u32x4(&x)[PE]) {
#pragma unroll
            for (int q = 0; q < PE; ++q)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = er + q * ER;
                    *reinterpret_cast<u32x4 *>(to + r * ROWB + ((2 * ec + y) ^ swizzle(r)) * 16) =
                        u32x4{e4m3_to_bf16<false>(x[q][2 * y]), e4m3_to_bf16<true>(x[q][2 * y]),
                              e4m3_to_bf16<false>(x[q][2 * y + 1]), e4m3_to_bf16<true>(x[q][2 * y + 1])};
                }
        };

        const int end = span.hi > span.lo ? blk1 : blk0; // no keys: nothing to walk
        auto note = [&](int key0, int slot, int id) { // whether the wave's keys have a usable page
            if (lane == 0 && my_row % 16 == 0) // of a part's waves the first: its keys are there if any are
                sm_lost[slot][my_row >> 4] = !(id > 0 && id < p.N) && key0 + my_row < s.L;
        };
        __syncthreads(); // the buffers of the piece before are read
        if (tid < 2) {
            sm_odd[tid] = 0;
            *reinterpret_cast<uint64_t *>(sm_lost[tid]) = 0;
        }
        __syncthreads();
        const int first_key = span.lo + blk0 * KB;
        int id = 0; // page of the block that is staged next
        auto bring = [&](int key0, int buf) {
            note(key0, buf, id);
            stage(p.k_pages, (lds_byte *)sm_k + buf * (KB * ROWB), key0, id);
            stage(p.v_pages, (lds_byte *)sm_v + buf * (KB * ROWB), key0, id);
            id = next_page(key0 + KB);
        };
        auto bring_e4m3 = [&](int key0, int buf) {
            note(key0, buf, id);
            fetch(p.k_pages, ek, key0, id);
            fetch(p.v_pages, ev, key0, id);
            id = next_page(key0 + KB);
        };
        if (blk0 < end) {
            id = next_page(first_key);
            if constexpr (E4M3) {
                bring_e4m3(first_key, 0);
                put(sm_k[0], ek);
                put(sm_v[0], ev);
            } else {
                bring(first_key, 0);
            }
        }
        auto read_k = [&](const uint8_t *kb, int at, int j) { // k of product j: step j / NS, part j % NS
            return *reinterpret_cast<const u32x4 *>(kb + (j % NS) * 32 * ROWB + k_row + (at ^ ((j / NS & 7) * 32)) +
                                                    (j / NS >> 3) * 256);
        };
        auto step_q = [&](int i) {
            return i < QL ? __builtin_bit_cast(bf16x8, sm_q[(wave * QL + i) * 64 + lane]) : qf[i < QL ? 0 : i - QL];
        };
        // all scores of a block
        auto score = [&](const uint8_t *kb, f32x16(&sc)[NS]) {
            // the LDS addresses are formed anew each block: kept, they cost 8 registers
            int k_at = k_chunk;
            asm volatile("" : "+v"(k_at));
#pragma unroll
            for (int y = 0; y < NS; ++y)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sc[y][i] = 0.f;
            // The LDS reads of the next few products leave before these: left to itself the
            // compiler reads, waits and multiplies one by one.
            u32x4 kf[2][KA];
            bf16x8 ql[2][KA];
#pragma unroll
            for (int g = -1; g < ST * NS / KA; ++g) {
                if (g + 1 < ST * NS / KA)
#pragma unroll
                    for (int k = 0; k < KA; ++k) {
                        kf[(g + 1) & 1][k] = read_k(kb, k_at, (g + 1) * KA + k);
                        ql[(g + 1) & 1][k] = step_q(((g + 1) * KA + k) / NS);
                    }
                __builtin_amdgcn_sched_barrier(0);
                if (g >= 0)
#pragma unroll
                    for (int k = 0; k < KA; ++k) {
                        f32x16 &o = sc[(g * KA + k) % NS];
                        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[g & 1][k]),
                                                                    ql[g & 1][k], o, 0, 0, 0);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto sees = [&](int key0) { // some row of the wave sees some key of the block
            return any && key0 <= max_pos && !(p.window > 0 && key0 + SB - 1 <= min_pos - p.window);
        };
        for (int blk = blk0; blk < end; ++blk) {
            const int buf = (blk - blk0) & 1, block0 = span.lo + blk * KB;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // this wave's part of the block is in LDS
            __syncthreads();
            if (blk + 1 < end) {
                if constexpr (E4M3)
                    bring_e4m3(block0 + KB, buf ^ 1);
                else
                    bring(block0 + KB, buf ^ 1);
            }
            // A block that some row does not see whole: v of keys past the sequence's last is cleared,
            // and so are infinities and NaN, which 0 times would carry into rows that do not see them.
            bool odd = false;
            if (block0 + KB - 1 > span.min_pos || (p.window > 0 && block0 <= span.max_pos - p.window)) {
                if (tid == 0)
                    sm_odd[buf ^ 1] = 0;
#pragma unroll
                for (int q = 0; q < KB * CH / NT; ++q) {
                    const int x = tid + q * NT, key = block0 + x / CH;
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
            // scores, weights and products of SB keys at a time: registers allow no more
#pragma unroll 1
            for (int sub = 0; sub < KB / SB; ++sub) {
                const int key0 = block0 + sub * SB;
                if (sees(key0)) {
                    uint32_t lost = *reinterpret_cast<const uint32_t *>(&sm_lost[buf][sub * (SB / 16)]);
                    __builtin_amdgcn_s_setprio(0);
                    int v_at[2] = {v_base[0], v_base[1]};
                    asm volatile("" : "+v"(v_at[0]), "+v"(v_at[1]));
                    const bool mixed = key0 + SB - 1 > min_pos || (p.window > 0 && key0 <= max_pos - p.window);
                    const uint8_t *vb = sm_v[buf] + sub * SB * ROWB;
                    f32x16 sc[NS];
                    score(sm_k[buf] + sub * SB * ROWB, sc);
                    constexpr int VA = DT < 4 ? DT : 4, VG = DT / VA; // products at a time
                    constexpr int GROUPS = 2 * NS * VG;
                    u32x4 vf[2][VA];
                    auto read_ahead = [&](int g) {
#pragma unroll
                        for (int k = 0; k < VA; ++k) {
                            const int q = g / VG, a = (g % VG) * VA + k;
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint8_t *from =
                                    vb + q * 16 * ROWB + (v_at[y] ^ ((a & 3) * 64)) + (a >> 2) * 256;
                                const u32x2 v2 = __builtin_bit_cast(
                                    u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)from));
                                vf[g & 1][k][2 * y] = v2[0];
                                vf[g & 1][k][2 * y + 1] = v2[1];
                            }
                        }
                    };
                    if (D == 256)
                        read_ahead(0); // arrives while the maximum is formed
#pragma unroll
                    for (int y = 0; y < NS; ++y)
                        settle(sc[y]);
                    asm volatile("" : "+v"(lost)); // waited for here, not before the scores
                    if (__ballot(lost != 0)) {
#pragma unroll
                        for (int q = 0; q < SB / 16; ++q)
                            bad |= (lost >> (8 * q) & 1) && pos >= key0 + 16 * q &&
                                           pos - reach <= key0 + 16 * q + 15
                                       ? 1
                                       : 0;
                    }
                    if (mixed) {
#pragma unroll
                        for (int y = 0; y < NS; ++y)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int back =
                                    pos - (key0 + y * 32 + 8 * (i >> 2) + 4 * hh + (i & 3));
                                if (back < 0 || back > reach)
                                    sc[y][i] = neg_inf();
                            }
                    }
                    __builtin_amdgcn_s_setprio(2);
                    float tops[NS]; // a chain each
#pragma unroll
                    for (int y = 0; y < NS; ++y) {
                        tops[y] = sc[y][0];
#pragma unroll
                        for (int i = 1; i < 16; ++i)
                            tops[y] = fmaxf(tops[y], sc[y][i]);
                    }
                    float top = NS == 2 ? fmaxf(tops[0], tops[NS - 1]) : tops[0];
                    top = max_xor32(top) * scale;
                    if (__ballot(top > m + 8.0f)) {
                        const float m_new = fmaxf(m, top);
                        const float keep = m_new == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - m_new);
                        l *= keep;
#pragma unroll
                        for (int a = 0; a < DT; ++a)
                            acc[a] *= keep;
                        m = m_new;
                    }
                    if (odd) { // uniform: what left v goes to the rows that see it
#pragma unroll 1
                        for (int j = 0; j < SB && key0 + j < s.L; ++j) {
                            const uint8_t *v = static_cast<const uint8_t *>(p.v_pages) +
                                               cell_of(key0 + j) * (E4M3 ? D : ROWB) + hh * (E4M3 ? 4 : 8);
                            const int back = pos - (key0 + j);
                            const bool seen = back >= 0 && back <= reach;
#pragma unroll
                            for (int c = 0; c < DT * 4; ++c) { // four columns of this lane's
                                u32x2 y;
                                if constexpr (E4M3) {
                                    const uint32_t z = *reinterpret_cast<const uint32_t *>(v + c * 8);
                                    y = u32x2{e4m3_to_bf16<false>(z), e4m3_to_bf16<true>(z)};
                                } else {
                                    y = *reinterpret_cast<const u32x2 *>(v + c * 16);
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t z = (i & 1) ? y[i >> 1] & 0xffff0000u : y[i >> 1] << 16;
                                    if (seen && (z & 0x7f800000u) == 0x7f800000u)
                                        acc[c >> 2][(c & 3) * 4 + i] += __uint_as_float(z);
                                }
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                    }
                    // weights of 16 keys at a time, and the products with their v beside the next ones
                    uint32_t pw[2][4]; // two groups of weights, bf16 pairs
                    const float off = m == neg_inf() ? 0.f : -m;
                    auto weigh = [&](int q, int i0, int i1) { // values i0 .. i1 - 1 of 16 keys' eight
#pragma unroll
                        for (int i = i0; i < i1; i += 2) {
                            const int at = 8 * (q & 1) + i;
                            const float e0 = __builtin_amdgcn_exp2f(fmaf(sc[q >> 1][at], scale, off));
                            const float e1 = __builtin_amdgcn_exp2f(fmaf(sc[q >> 1][at + 1], scale, off));
                            l += e0 + e1;
                            // rounded to bf16 for the matrix cores: off by at most 2^-8 of itself, as o is
                            // in the end; two numbers for each take half of the products again (above)
                            pw[q & 1][i >> 1] = pack_bf16(e0, e1);
                        }
                    };
                    if (D != 256)
                        read_ahead(0);
                    weigh(0, 0, 8);
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        const int q = g / VG, part = g % VG;
                        __builtin_amdgcn_sched_barrier(0);
                        if (g + 1 < GROUPS)
                            read_ahead(g + 1);
                        if (q + 1 < 2 * NS)
                            weigh(q + 1, part * 8 / VG, (part + 1) * 8 / VG);
                        const bf16x8 pf = __builtin_bit_cast(
                            bf16x8, u32x4{pw[q & 1][0], pw[q & 1][1], pw[q & 1][2], pw[q & 1][3]});
#pragma unroll
                        for (int k = 0; k < VA; ++k) {
                            f32x16 &o = acc[part * VA + k];
                            o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[g & 1][k]),
                                                                        pf, o, 0, 0, 0);
                        }
                    }
                }
            }
            if constexpr (E4M3) {
                if (blk + 1 < end) {
                    put(sm_k[buf ^ 1], ek);
                    put(sm_v[buf ^ 1], ev);
                }
            }
        }
        l += __shfl_xor(l, 32);
        if ((bad | __shfl_xor(bad, 32)) || s.kind == kNan)
            l = quiet_nan();
        if (row < rows) {
            const int64_t tk = s.first + row / p.G;
            const int head = h * p.G + row % p.G;
            if (whole) {
                const float vs = E4M3 ? p.v_scale[h] : 1.0f;
                const float inv = l == 0.f ? 0.f : vs / l;
                uint16_t *o = p.out.p + tk * p.out.row + (int64_t)head * p.out.head + 4 * hh;
#pragma unroll
                for (int a = 0; a < DT; ++a)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<u32x2 *>(o + a * 32 + 2 * i) =
                            u32x2{pack_bf16(acc[a][i] * inv, acc[a][i + 1] * inv),
                                  pack_bf16(acc[a][i + 2] * inv, acc[a][i + 3] * inv)};
                if (hh == 0 && p.lse)
                    p.lse[tk * p.H_q + head] = lse_of(m, l);
            } else {
                // as it lies in the registers, 1 KiB a store; the join reads it so
                const int64_t part = ((int64_t)w * 2 + slot) * NW + wave;
                float *o = p.part_o + part * 32 * D + lane * 4;
#pragma unroll
                for (int a = 0; a < DT; ++a)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<f32x4 *>(o + a * 1024 + i * 64) =
                            f32x4{acc[a][i], acc[a][i + 1], acc[a][i + 2], acc[a][i + 3]};
                if (hh == 0) {
                    p.part_ml[(part * 32 + n_) * 2] = m;
                    p.part_ml[(part * 32 + n_) * 2 + 1] = l;
                }
            }
        }
    }
}

// blockIdx.x = a piece: what begins in it and goes on in the next; a wave 32 rows by 32 columns
// of it, a lane the 16 values of its row that it had in the registers.
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void attn_tiles_join_kernel(AttnParams p)
{
    constexpr int DT = D / 32, BATCH = 2;
    const int lane = threadIdx.x & 63, n_ = lane & 31, hh = lane >> 5;
    const int item = uniform(blockIdx.y * 4 + (threadIdx.x >> 6)), wave = item / DT, a = item % DT;
    // on the XCD that wrote it: some of it is still in its L2
    const int w0 = (blockIdx.x & 7) * (p.workgroups / 8) + (blockIdx.x >> 3);
    const Cut c = read_cut(p, w0);
    if (c.last < 0)
        return;
    const int w1 = c.last < p.workgroups ? c.last : p.workgroups - 1, slot0 = c.slot, h = c.h;
    const int row = c.tile * TR + wave * 32 + n_;
    if (row >= c.rows)
        return;
    float m = neg_inf(), l = 0.f;
    f32x4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int w = w0; w <= w1; w += BATCH) {
        f32x2 ml[BATCH];
        f32x4 po[BATCH][4];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int at = w + k <= w1 ? w + k : w;
            const int64_t part = ((int64_t)at * 2 + (at == w0 ? slot0 : 0)) * NW + wave;
            ml[k] = *reinterpret_cast<const f32x2 *>(p.part_ml + (part * 32 + n_) * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                po[k][i] = *reinterpret_cast<const f32x4 *>(p.part_o + part * 32 * D + a * 1024 + i * 256 + lane * 4);
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            top = fmaxf(top, ml[k][0]);
        const float safe = top == neg_inf() ? 0.f : top;
        const float keep = __builtin_amdgcn_exp2f(m - safe);
        l *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] *= keep;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (w + k <= w1) {
                const float f = __builtin_amdgcn_exp2f(ml[k][0] - safe);
                l = fmaf(ml[k][1], f, l);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i >> 2][i & 3] = fmaf(po[k][i >> 2][i & 3], f, o[i >> 2][i & 3]);
            }
        }
        m = top;
    }
    const int64_t t = c.first + row / p.G;
    const int hq = h * p.G + row % p.G;
    const float vs = E4M3 ? p.v_scale[h] : 1.0f;
    const float inv = l == 0.f ? 0.f : vs / l;
    uint16_t *out = p.out.p + t * p.out.row + (int64_t)hq * p.out.head + a * 32 + 4 * hh;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<u32x2 *>(out + 8 * i) =
            u32x2{pack_bf16(o[i][0] * inv, o[i][1] * inv), pack_bf16(o[i][2] * inv, o[i][3] * inv)};
    if (a == 0 && hh == 0 && p.lse)
        p.lse[t * p.H_q + hq] = lse_of(m, l);
}

size_t attn_tiles_layout(int B, int T, int H_kv, int G, int d, void *base, AttnParams *p)
{
    const int workgroups = (device_cus() + 7) / 8 * 8;
    const size_t entries = ((size_t)T * G / TR + B) * H_kv;
    const size_t o = round256((size_t)workgroups * 2 * TR * d * 4), ml = round256((size_t)workgroups * 2 * TR * 2 * 4),
                 bf = round256((entries + 1) * 8), en = round256(entries * kEntry * 4),
                 cut = round256((size_t)workgroups * 8 * 4);
    if (p) {
        char *at = static_cast<char *>(base);
        p->workgroups = workgroups;
        p->capacity = (int)entries;
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
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_tiles_kernel<D, E4M3>),
                            dim3((unsigned)p.workgroups), dim3(64 * NW), args, 0, stream);
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_tiles_join_kernel<D, E4M3>),
                            dim3((unsigned)p.workgroups, NW * (D / 32) / 4), dim3(256), args, 0, stream);
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
