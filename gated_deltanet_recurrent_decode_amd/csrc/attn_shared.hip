// attn_shared.hip -- paged attention for a batch whose rows share long prefixes (gfx950).
//
// The keys of a row fall into those that its group has in common and its own.  A softmax over both is joined
// from its parts: with (o, m, l) of each, weights relative to its maximum m and their sum l,
//   m = max(m_a, m_b),  l = l_a e^(m_a - m) + l_b e^(m_b - m),  o = (o_a e^(m_a - m) + o_b e^(m_b - m)) / l.
// The rows of a group lie behind each other, so for the common keys they are one sequence: tiles of 256 (token,
// head of the group) rows that read each key once, where the rows by themselves would read it once each.  The
// tiles of attn_tiles.hip do both kinds of entries in one launch, dealt out by the key over all workgroups: a
// first kernel lists the sequences' own entries and then the groups', a last one joins each row's parts.
//
// What a group has in common is found on the device: the length that the call gives, cut to what every usable
// member has before its new tokens, and to whole 16 keys (a block's staging rows lie on one page so).  Longer or
// shorter, the result is the same; only what is read once changes.
//
// What bounds it, with few rows: a wave's own chain through a block (scores, maximum, weights, products: 1.05 us for
// 64 keys, which take the matrix cores 0.4, before weights of two numbers added 0.2), hidden by one other wave of its
// SIMD at most, for a tile's registers allow two; an entry's beginning (its record, its page numbers and its first
// block behind each other, 2.5 us); the plan and the join, 8.5 and 5 to 11 us of a call.  With many rows a sequence:
// the matrix cores, as in attn_tiles.hip.
// MI355X, calls back to back, and attn_paged's of the same rows: 64 rows at 32/4 heads of 128 over a prefix of 8000 and
// 50-800 own keys 51 to 52 us (attn_paged 88); 48 rows in 3 groups at 32/8 heads of 128, e4m3, 4000-30000 and 100-1000
// 99 us (270); 32 rows of 4 tokens at 16/4 heads of 256 over 6001 and 10-500 67 us (117); 8 chunks of 100-600 tokens at
// 32/4 heads of 128 over 12000 484 to 515 us (481; 983 to 924 TFLOP/s), where the rule below takes nothing together.
// The plan, the join and tiles that few rows leave idle cost more than sharing saves where little is shared: at 16/2
// heads of 128 with 10-500 own keys 8 rows over 4000 28.5 us (20.0), 64 over 1024 30.4 (23.2), 64 in 16 groups over
// 2048 33.4 (30.1), 64 in 32 groups over 8192 74.6 (77.3).
//
// Up to 16 rows a sequence keep 15 bits of their weights, as they do in attn_paged: with weights rounded to bf16 o is
// 0.0023 of its norm off 64 bits in place of 0.0017, and the first three of these calls take 45, 86 and 59 us.
//
// Tried, calls, with weights rounded to bf16: a tile's keys dealt out among its idle waves (the same); the waves' page
// numbers a block of 64 ahead in a register (the same); own keys by a kernel of 16-row tiles beside the groups' tiles,
// one more launch (8 rows 30 -> 36 us, 64 rows 62 -> 66, 3 groups 123 -> 111, all before the tiles of 128 rows); a
// block's weight on the line by the waves that have rows (3 groups 86.6 -> 85.1, 64 rows 47.0 -> 49.8, chunks 503 ->
// 535).

#include <algorithm>

#include "attn_tiles.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

// Which groups are taken together where the call does not say.  Members with tiles of their own read a key once a
// tile; together they are fewer tiles.  For that the rows' second parts have to be written and joined, about 512
// keys' time for a tile of a member, and the group's own tiles begun, 1024 each.  16/2 heads of 128, 512 rows with
// 10-2000 own keys, by tiles of their own / together, us: 256 groups of about 2 at a prefix of 1024 184 / 183, of 2048
// 248 / 227, of 8192 653 / 502; 64 groups of about 8 at 512 142 / 152, of 1024 155 / 155, of 4096 317 / 197.  Chunks
// of 100-600 tokens fill their own tiles: 499 / 509 with 12000 common keys.
constexpr int kPerMember = 512, kPerTile = 1024;
// And the call as a whole saves at least so many blocks a workgroup: below, a step of few rows is bound by how long a
// workgroup takes at all (the same with 64 rows in 16 groups at 1024, 3 blocks: 35.5 / 36.0; at 2048, 6: 43.1 / 40.1;
// 64 rows of one at 1024, 4: 36.7 / 36.8; 16 rows in 2 groups at 4096, 4: 31.7 / 32.7).
constexpr int kLeastBlocks = 5;

// The last x of n with first[x] <= v, the first at least.
__device__ __forceinline__ int last_at(const int *first, int n, int v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

} // namespace

// One workgroup, as what it finds is one line; it waits for memory and for its own sums most of the time, so the first
// PT sequences' numbers are read once, and a round's entries and the groups' are numbered together.
__global__ __launch_bounds__(PT) void attn_shared_plan_kernel(AttnParams p, int own_capacity, int shared_capacity)
{
    __shared__ int g_begin[PT + 1], g_len[PT], g_low[PT], g_row[PT], g_members[PT], g_entry[PT], g_tiles[PT],
        g_first[PT], g_tokens[PT], g_own_tiles[PT];
    __shared__ int first_entry[PT], sm_cu[PT + 1];
    __shared__ unsigned long long sm_saved; // blocks
    __shared__ Seq seqs[PT];
    const int tid = threadIdx.x;
    Seq own{kSkip};
    if (tid < p.B)
        own = read_seq(p, tid);
    for (int x = tid; x <= PT && x <= p.B; x += PT)
        sm_cu[x] = p.cu[x];
    for (int x = tid; x <= p.K; x += PT) {
        const int at = p.K > 0 ? p.cu_groups[x] : 0;
        g_begin[x] = at < 0 ? 0 : (at > p.B ? p.B : at);
        if (x < p.K) {
            g_len[x] = p.shared_len[x];
            g_low[x] = g_row[x] = 0x7fffffff;
            g_members[x] = g_own_tiles[x] = 0;
        }
    }
    seqs[tid] = own;
    if (tid == 0)
        sm_saved = 0;
    __syncthreads();
    auto group_of = [&](int b) { // or -1
        if (p.K == 0)
            return -1;
        const int g = last_at(g_begin, p.K, b);
        return b >= g_begin[g] && b < g_begin[g + 1] ? g : -1;
    };
    int own_group = -1;
    for (int b = tid; b < p.B; b += PT) {
        const Seq s = b == tid ? own : read_seq(p, b);
        const int g = s.kind == kNormal ? group_of(b) : -1;
        if (b == tid)
            own_group = g;
        if (g >= 0) {
            atomicMin(&g_len[g], s.L - s.n);
            atomicMin(&g_low[g], p.window > 0 ? s.L - s.n - p.window + 1 : 0);
            atomicMin(&g_row[g], b); // read through its first usable member
            atomicAdd(&g_members[g], 1);
            atomicAdd(&g_own_tiles[g], tiles_of(p, s, p.tile_rows));
        }
    }
    __syncthreads();
    int group_entries = 0, len = 0, low = 0, tokens = 0, first = 0, tiles = 0;
    bool ok = false;
    if (tid < p.K) {
        const int x0 = g_begin[tid], x1 = g_begin[tid + 1];
        first = x0 <= PT ? sm_cu[x0] : p.cu[x0];
        tokens = (x1 <= PT ? sm_cu[x1] : p.cu[x1]) - first;
        len = g_len[tid] > 0 ? g_len[tid] & ~15 : 0;
        low = g_low[tid] > 0 ? g_low[tid] & ~15 : 0;
        tiles = (int)(((int64_t)tokens * p.G + p.tile_rows - 1) / p.tile_rows);
        ok = g_members[tid] > 1 && x0 < x1 && len > low && first >= 0 && tokens > 0 && first + tokens <= p.T;
        if (p.least >= 0) {
            ok = ok && len - low >= p.least;
        } else if (ok) {
            const int64_t saved = (int64_t)(g_own_tiles[tid] - tiles) * (len - low);
            ok = saved >= (int64_t)kPerMember * g_own_tiles[tid] + (int64_t)kPerTile * tiles;
            if (ok)
                atomicAdd(&sm_saved, (unsigned long long)(saved / p.block * p.H_kv));
        }
    }
    __syncthreads();
    if (tid < p.K) {
        const int member = g_row[tid];
        ok = ok && (p.least >= 0 || sm_saved >= (unsigned long long)kLeastBlocks * p.workgroups);
        g_len[tid] = ok ? len : 0;
        g_low[tid] = low;
        g_row[tid] = ok ? (member < PT ? seqs[member].r : p.row[member]) : 0;
        g_first[tid] = first;
        g_tokens[tid] = tokens;
        g_tiles[tid] = ok ? tiles : 0;
        group_entries = g_tiles[tid] * p.H_kv;
    }
    int shared_entries = 0, entries = 0, own_entries = 0;
    long long units = 0;
    for (int b0 = 0; b0 < p.B; b0 += PT) {
        const int b = b0 + tid;
        int mine = 0;
        __syncthreads(); // the round before has read the tables, and the groups are written
        if (b < p.B) {
            Seq s = b0 == 0 ? own : read_seq(p, b);
            mine = tiles_of(p, s, p.tile_rows) * p.H_kv;
            const int g = b0 == 0 ? own_group : (s.kind == kNormal ? group_of(b) : -1);
            // For now its group.  Its tokens are among the group's if cu_seqlens does not decrease; the join relies on it.
            s.lo = g >= 0 && g_len[g] > 0 && s.first >= g_first[g] && s.first + s.n <= g_first[g] + g_tokens[g] ? g + 1
                                                                                                               : 0;
            seqs[tid] = s;
        }
        // Sequences or groups that overlap have more tiles than the workspace was sized for (and than 32 bits
        // count): what is past its end is left out.
        long long sum_all, sum_groups;
        long long group_at = group_entries; // of the first round
        const long long mine_at = plan_scan2((long long)mine, &sum_all, &group_at, &sum_groups);
        if (b0 == 0) {
            shared_entries = sum_groups < shared_capacity ? (int)sum_groups : shared_capacity;
            if (tid < p.K)
                g_entry[tid] = group_at < shared_entries ? (int)group_at : shared_entries;
        }
        const int room = own_capacity - entries, all = sum_all < room ? (int)sum_all : room;
        first_entry[tid] = mine_at < all ? (int)mine_at : all;
        __syncthreads();
        const int seqs_here = p.B - b0 < PT ? p.B - b0 : PT;
        const bool last_round = p.B - b0 <= PT;
        own_entries = entries + all;
        const int count = all + (last_round ? shared_entries : 0); // then the groups' common keys
        for (int e0 = 0; e0 < count; e0 += PT) {
            const int e = e0 + tid;
            long long u = 0;
            i32x4 x0{0, 0, 0, 0}, x1 = x0, x2 = x0;
            if (e < all) {
                const int q = last_at(first_entry, seqs_here, e);
                Seq s = seqs[q];
                const int g = s.lo - 1;
                s.lo = g >= 0 ? g_len[g] : 0;
                const int tiles = tiles_of(p, s, p.tile_rows), x = e - first_entry[q], h = x / tiles,
                          tile = x - h * tiles;
                u = p.pad + span_of<true>(p, s, tile, p.tile_rows).blocks;
                x0 = i32x4{h, tile, s.kind, s.first};
                x1 = i32x4{s.n, s.L, s.r, s.lo};
                if (g >= 0)
                    x2 = i32x4{g_first[g], g_entry[g], g_tiles[g], 0};
            } else if (e < count) {
                const int g = last_at(g_entry, p.K, e - all);
                const int x = e - all - g_entry[g], tiles = g_tiles[g] > 0 ? g_tiles[g] : 1, h = x / tiles;
                u = p.pad + (g_len[g] - g_low[g] + p.block - 1) / p.block;
                x0 = i32x4{h, x - h * tiles, kShared, g_first[g]};
                x1 = i32x4{g_tokens[g], g_len[g], g_row[g], g_low[g]};
            }
            long long sum;
            const long long at = units + plan_scan(u, &sum);
            if (e < count) {
                const int64_t o = entries + e;
                p.before[o] = at;
                i32x4 *to = reinterpret_cast<i32x4 *>(p.entry + o * kSharedEntry);
                to[0] = x0;
                to[1] = x1;
                to[2] = x2;
            }
            units += sum;
        }
        entries += count;
    }
    if (tid == 0) {
        p.before[entries] = units;
        p.count[0] = entries;
        p.count[1] = own_entries;
        *reinterpret_cast<long long *>(p.count + 2) = units;
    }
}

// blockIdx.x = an entry of a sequence's own keys, blockIdx.y 32 rows by 32 columns of it: a lane has 16 values of a row
// as the tiles had them in their registers.  Four waves take every fourth part and meet in LDS.
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void attn_shared_join_kernel(AttnParams p)
{
    constexpr int DT = D / 32, JW = 4;
    __shared__ f32x2 sm_ml[JW][64];
    __shared__ f32x4 sm_o[JW][4][64];
    const int lane = threadIdx.x & 63, n_ = lane & 31, hh = lane >> 5, wave = uniform(threadIdx.x >> 6);
    const int blk = blockIdx.y / DT, a = blockIdx.y % DT;
    const int e = blockIdx.x, own_entries = p.count[1];
    if (e >= own_entries)
        return;
    const int32_t *entry = p.entry + (int64_t)e * kSharedEntry;
    const int h = entry[0], tile = entry[1], kind = entry[2], first = entry[3], rows = entry[4] * p.G, lo = entry[7];
    const int tr = p.tile_rows;
    if (kind != kNormal || tile * tr + blk * 32 >= rows)
        return;
    const long long total = *reinterpret_cast<const long long *>(p.count + 2);
    const int pieces = pieces_of(p, total);
    const int w0 = owner_of(total, p.before[e] + p.pad, pieces), w1 = owner_of(total, p.before[e + 1] - 1, pieces);
    if (lo == 0 && w0 == w1)
        return; // whole, and it shares nothing: written by the tiles
    const int row = tile * tr + blk * 32 + n_;
    const bool valid = row < rows;
    float m = neg_inf(), l = 0.f;
    f32x4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](f32x2 ml, const f32x4(&x)[4]) {
        const float top = fmaxf(m, ml[0]), safe = top == neg_inf() ? 0.f : top;
        const float keep = __builtin_amdgcn_exp2f(m - safe), f = __builtin_amdgcn_exp2f(ml[0] - safe);
        l = fmaf(ml[1], f, l * keep);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i >> 2][i & 3] = fmaf(x[i >> 2][i & 3], f, o[i >> 2][i & 3] * keep);
        m = top;
    };
    // this wave's of the parts w_a .. w_b of a row: at(w) their 32-row block, r the row in it
    auto join = [&](int w_a, int w_b, int r, auto at) {
        constexpr int BATCH = 2;
        for (int w = w_a + wave; w <= w_b; w += JW * BATCH) {
            f32x2 ml[BATCH];
            f32x4 po[BATCH][4];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int64_t part = at(w + k * JW <= w_b ? w + k * JW : w);
                ml[k] = *reinterpret_cast<const f32x2 *>(p.part_ml + (part * 32 + r) * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    po[k][i] = *reinterpret_cast<const f32x4 *>(p.part_o + part * 32 * D + a * 1024 + i * 256 +
                                                                (hh * 32 + r) * 4);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (w + k * JW <= w_b)
                    add(ml[k], po[k]);
        }
    };
    if (lo > 0 && valid) { // the row's place among its group's
        const int64_t at = (int64_t)(first - entry[8]) * p.G + row;
        const int es = own_entries + entry[9] + h * entry[10] + (int)(at / tr);
        if (es < p.count[0])
            join(owner_of(total, p.before[es] + p.pad, pieces), owner_of(total, p.before[es + 1] - 1, pieces),
                 (int)(at % 32), [&](int w) { return shared_part(p, es, own_entries, w) + at % tr / 32; });
    }
    if (valid)
        join(w0, w1, n_, [&](int w) { return own_part(p, e, w) + blk; });
    sm_ml[wave][lane] = f32x2{m, l};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sm_o[wave][i][lane] = o[i];
    __syncthreads();
    if (wave != 0 || !valid)
        return;
#pragma unroll
    for (int q = 1; q < JW; ++q) {
        f32x4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = sm_o[q][i][lane];
        add(sm_ml[q][lane], x);
    }
    const int64_t t = first + row / p.G;
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

namespace {

struct Sizes {
    int tile_rows;
    size_t own, shared; // entries
    int own_blocks;     // 32-row blocks of an own part
};

Sizes sizes_of(int T, int B, int K, int max_new, int H_kv, int G, int d)
{
    const int64_t rows = (int64_t)max_new * G;
    // Few rows a sequence leave most waves of a 256-row tile idle: then tiles of 128 with blocks of 64 keys, so that a
    // CU holds two workgroups and one's waits are the other's work (with weights rounded to bf16, as in all figures
    // here: 64 rows 57.5 -> 47.5 us, 3 groups 118 -> 89).  By
    // the rows of a sequence, 32 of them in 2 groups at 16/2 heads of 128, tiles of 256 / 128: 64 rows 44.1 / 42.7 us,
    // 128 53.7 / 51.1, 256 71.8 / 72.9, 2048 380 / 403.  Tiles of 64, four a CU, read a group's keys twice as often and
    // leave twice the parts (64 rows 57 -> 59, 3 groups 99 -> 93, before an entry's beginning was counted).  With 256
    // columns the LDS has no room for two.
    const int tr = d < 256 && rows <= kSmallTile ? kSmallTile : TR;
    return Sizes{tr, ((size_t)T * G / tr + B) * H_kv, ((size_t)T * G / tr + K) * H_kv,
                 rows >= tr ? tr / 32 : (rows > 32 ? (int)((rows + 31) / 32) : 1)};
}

} // namespace

size_t attn_shared_layout(int B, int T, int K, int max_new, int H_kv, int G, int d, void *base, AttnParams *p)
{
    const Sizes s = sizes_of(T, B, K, max_new, H_kv, G, d);
    const int workgroups = (device_cus() + 7) / 8 * 8 * (TR / s.tile_rows);
    const size_t own = (s.own + workgroups) * s.own_blocks, blocks = own + (s.shared + workgroups) * (s.tile_rows / 32);
    const size_t o = round256(blocks * 32 * d * 4), ml = round256(blocks * 32 * 2 * 4),
                 bf = round256((s.own + s.shared + 1) * 8), en = round256((s.own + s.shared) * kSharedEntry * 4);
    if (p) {
        char *at = static_cast<char *>(base);
        p->workgroups = workgroups;
        p->tile_rows = s.tile_rows;
        p->own_blocks = s.own_blocks;
        p->shared_parts = (int64_t)own;
        p->part_o = reinterpret_cast<float *>(at);
        p->part_ml = reinterpret_cast<float *>(at + o);
        p->before = reinterpret_cast<long long *>(at + o + ml);
        p->entry = reinterpret_cast<int32_t *>(at + o + ml + bf);
        p->count = reinterpret_cast<int32_t *>(at + o + ml + bf + en);
    }
    // A workspace for some max_new serves calls with less, whose tiles may be smaller and more, or attn_paged's.
    size_t all = o + ml + bf + en + 256;
    const int fewer = kSmallTile / G;
    if (fewer > 0 && s.tile_rows != kSmallTile && d < 256 && max_new > fewer)
        all = std::max(all, attn_shared_layout(B, T, K, fewer, H_kv, G, d, nullptr, nullptr));
    return attn_few_rows(1, G) ? std::max(all, attn_paged_layout(B, T, 1, H_kv, G, d, nullptr, nullptr)) : all;
}

template <int D, bool E4M3>
static hipError_t launch_de(const AttnParams &p, hipStream_t stream)
{
    const Sizes s = sizes_of(p.T, p.B, p.K, p.max_new, p.H_kv, p.G, D);
    AttnParams q = p;
    q.block = block_keys(D, p.tile_rows == kSmallTile);
    // An entry's beginning in blocks' time.  With 0, 1, 2, 3, 5 (weights rounded to bf16): 64 rows 57, 44, 45, 46, 47
    // us, 3 groups 99, 90, 86, 87, 91, chunks that are taken together 722, 538, 505, 513, 523; 4 tokens a row (256
    // columns) 67, 64, 62, 60, 60.
    q.pad = D == 256 ? 3 : 2;
    int own = (int)s.own, shared = (int)s.shared;
    void *plan[] = {&q, &own, &shared}, *args[] = {&q};
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_shared_plan_kernel), dim3(1), dim3(PT), plan, 0,
                                   stream);
    if (e == hipSuccess)
        e = launch_attn_tiles_shared(q, D, E4M3, stream);
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void *>(&attn_shared_join_kernel<D, E4M3>),
                            dim3((unsigned)s.own, (unsigned)(s.own_blocks * (D / 32))), dim3(256), args, 0,
                            stream);
    return e;
}

// Whether the call's sizes alone say that no group will be taken together: every key that the table has room for,
// read by every tile but one, is less than the plan's rule asks for.
static bool nothing_to_share(const AttnParams &p, int d)
{
    if (p.K == 0 || p.least >= 0)
        return p.K == 0;
    const Sizes s = sizes_of(p.T, p.B, p.K, p.max_new, p.H_kv, p.G, d);
    const double blocks = (double)p.width * (1 << p.page_shift) / block_keys(d, s.tile_rows == kSmallTile);
    return (double)(s.own - p.H_kv) * blocks < (double)kLeastBlocks * p.workgroups;
}

hipError_t launch_attn_shared(const AttnParams &p, int d, bool e4m3, hipStream_t stream)
{
    // Then rows by themselves in tiles of 16, which need no plan: 8 rows at 16/2 heads of 256 over 500 + 1-40 keys 15.1
    // us a call, and 23.2 with a table of 4096 positions or more, where the rule would have room to hold: only the
    // device knows the lengths.
    if (attn_few_rows(p.max_new, p.G) && nothing_to_share(p, d)) {
        AttnParams q = p;
        attn_paged_layout(p.B, p.T, p.max_new, p.H_kv, p.G, d, p.part_o, &q); // the workspace's beginning
        return launch_attn_paged(q, d, e4m3, stream);
    }
    if (d == 64)
        return e4m3 ? launch_de<64, true>(p, stream) : launch_de<64, false>(p, stream);
    if (d == 128)
        return e4m3 ? launch_de<128, true>(p, stream) : launch_de<128, false>(p, stream);
    return e4m3 ? launch_de<256, true>(p, stream) : launch_de<256, false>(p, stream);
}

} // namespace gdn
