// attn_tiles.h -- what the kernels around the prompt-chunk tiles share (gfx950): sizes, the plan's entries, the
// planning workgroup's sums.
#pragma once

#include "attn_common.h"

namespace gdn {

// rows of a tile, and of one of a call with few rows a sequence (attn_shared.hip)
constexpr int TR = 256, kSmallTile = 128;
// keys of a block: with 256 columns the queries take half of the LDS
constexpr int block_keys(int d, bool few = false) { return d == 256 ? 32 : (few ? 64 : 128); }
constexpr int PT = 1024; // the planning workgroup
// what the plan says of an entry: kv head, tile, and its sequence, so that nobody reads the lengths again
constexpr int kEntry = 8;
// Where sequences share a prefix: kv head, tile, kind, first token, tokens, keys, row, first key; of a sequence's
// entry also the group's first token, its first shared entry and its tiles (0: it shares nothing).
constexpr int kSharedEntry = 12;
// a group's tokens as one sequence that sees all of its L keys
constexpr int kShared = 3;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int tiles_of(const AttnParams &p, const Seq &s, int tr = TR)
{
    return s.kind == kSkip ? 0 : (int)(((int64_t)s.n * p.G + tr - 1) / tr);
}

// What a tile of a sequence sees: keys lo .. hi - 1, in blocks from lo on.
struct Span {
    int lo, hi, blocks, min_pos, max_pos;
};

template <bool SHARED>
__device__ __forceinline__ Span span_of(const AttnParams &p, const Seq &s, int tile, int tr = TR)
{
    Span x;
    const int rows = s.n * p.G;
    const int last = (rows < (tile + 1) * tr ? rows : (tile + 1) * tr) - 1;
    x.min_pos = s.L - s.n + tile * tr / p.G;
    x.max_pos = s.L - s.n + last / p.G;
    x.hi = s.kind == kNormal && x.max_pos >= 0 ? x.max_pos + 1 : 0;
    x.lo = 0;
    if (p.window > 0 && x.min_pos - p.window + 1 > 0)
        x.lo = (x.min_pos - p.window + 1) & ~(p.block - 1);
    if constexpr (SHARED) {
        if (s.kind == kShared)
            x = Span{s.lo, s.L, 0, s.L - 1, s.L - 1};
        else if (x.lo < s.lo) // a multiple of 16, as pages are
            x.lo = s.lo;
    }
    x.lo = x.lo < x.hi ? x.lo : (x.hi > 0 ? (x.hi - 1) & ~(p.block - 1) : 0);
    x.blocks = x.hi > x.lo ? (x.hi - x.lo + p.block - 1) / p.block : 1;
    return x;
}

// The place of a part of entry e of a plan with shared prefixes, in 32-row blocks: walking along the line, every
// new (entry, piece) is another entry or another piece, so their sum numbers them.
__device__ __forceinline__ int64_t own_part(const AttnParams &p, int e, int w)
{
    return (int64_t)(e + w) * p.own_blocks;
}
__device__ __forceinline__ int64_t shared_part(const AttnParams &p, int e, int own_entries, int w)
{
    return p.shared_parts + (int64_t)(e - own_entries + w) * (p.tile_rows / 32);
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

// Two of them at once; *b is its value and becomes its sum.
__device__ __forceinline__ long long plan_scan2(long long a, long long *all_a, long long *b, long long *all_b)
{
    __shared__ long long wave_sum[2][PT / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    long long x = a, y = *b;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const long long o = __shfl_up(x, m), q = __shfl_up(y, m);
        if (lane >= m) {
            x += o;
            y += q;
        }
    }
    __syncthreads();
    if (lane == 63) {
        wave_sum[0][wave] = x;
        wave_sum[1][wave] = y;
    }
    __syncthreads();
    long long before_a = 0, before_b = 0;
    *all_a = *all_b = 0;
#pragma unroll
    for (int w = 0; w < PT / 64; ++w) {
        const long long o = wave_sum[0][w], q = wave_sum[1][w];
        before_a += w < wave ? o : 0;
        before_b += w < wave ? q : 0;
        *all_a += o;
        *all_b += q;
    }
    const long long at = before_a + x - a;
    *b = before_b + y - *b;
    return at;
}

} // namespace gdn
