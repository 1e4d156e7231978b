// attn_common.h -- device helpers shared by the paged-attention kernels (gfx950).
#pragma once

#include "attn_internal.h"
#include "device_common.h"

namespace gdn {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7fc00000u); }

// Two fp32 values as a bf16 pair, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Two of a dword's four e4m3 values (the low or the high pair) as a bf16 pair: exact.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_to_bf16(uint32_t v)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, HI));
}

__device__ __forceinline__ float min_finite(float x, float top) { return x > top ? top : (x < -top ? -top : x); }

// Ends a chain of matrix products: the result is in vector registers, read behind the waits
// that the matrix cores need, before any branch.  Without it the compiler has put the reads
// behind a branch with too few waits on its taken side (wrong scores, every time).
template <class T>
__device__ __forceinline__ void settle(T &x)
{
    asm volatile("" : "+v"(x));
}

// The larger of lane i's value and lane i ^ 16's or 32's, by gfx950's row swaps: in the vector
// unit, where a shuffle goes through LDS.
__device__ __forceinline__ float max_xor16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float max_xor32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

enum { kSkip = -1, kNormal = 0, kZero = 1, kNan = 2 };

// A sequence of the call as the arrays on the device give it.
struct Seq {
    int kind, first, n, L, lo; // first token, tokens, keys, first key in reach of the window
    int r;                     // row of the table
};

__device__ __forceinline__ Seq read_seq(const AttnParams &p, int b)
{
    Seq s;
    s.first = p.cu[b];
    const int e = p.cu[b + 1];
    s.n = e - s.first;
    s.kind = kNormal;
    s.r = p.row[b];
    s.L = s.lo = 0;
    if (s.first < 0 || e > p.T || e <= s.first) {
        s.kind = kSkip;
        return s;
    }
    if (s.r == 0) {
        s.kind = kZero;
    } else if (s.r < 0 || s.r >= p.R || s.n > p.max_new) {
        s.kind = kNan;
    } else {
        s.L = p.kv_len[s.r];
        if (s.L < 0 || s.L > (p.width << p.page_shift)) {
            s.kind = kNan;
            s.L = 0;
        } else if (p.window > 0 && s.L - s.n - p.window + 1 > 0) {
            s.lo = (s.L - s.n - p.window + 1) & ~31;
        }
    }
    return s;
}

// a / b for a >= 0, b > 0, in 32 bits where they suffice (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    if (((unsigned long long)a | (unsigned long long)b) >> 32)
        return (long long)((unsigned long long)a / (unsigned long long)b);
    return (uint32_t)a / (uint32_t)b;
}

// Work in units on one line, cut into pieces, one a workgroup, none of them empty; piece w
// begins at unit piece_begin(w).
__device__ __forceinline__ int pieces_of(const AttnParams &p, long long total)
{
    return total < p.workgroups ? (int)total : p.workgroups;
}

__device__ __forceinline__ long long piece_begin(long long total, int w, int pieces)
{
    return total == pieces ? w : quotient(total * w, pieces);
}

// The piece that holds unit u: the last w with piece_begin(w) <= u.
__device__ __forceinline__ int owner_of(long long total, long long u, int pieces)
{
    return total == pieces ? (int)u : (int)quotient((u + 1) * pieces - 1, total);
}

// A (sequence, kv head, tile) that begins in a workgroup's piece and goes on behind it: what
// the join needs of it, left in the workspace by that workgroup.
struct Cut {
    int last;  // piece of its last unit; -1: there is none
    int slot;  // its part in this workgroup's piece, 0 or 1 (0 in the pieces behind)
    int first; // its sequence's first token
    int rows;  // its sequence's rows
    int h, tile;
};

__device__ __forceinline__ void write_cut(const AttnParams &p, int w, const Cut &c)
{
    int32_t *o = p.cut + (int64_t)w * 8;
    o[0] = c.last;
    o[1] = c.slot;
    o[2] = c.first;
    o[3] = c.rows;
    o[4] = c.h;
    o[5] = c.tile;
}

__device__ __forceinline__ Cut read_cut(const AttnParams &p, int w)
{
    const int32_t *o = p.cut + (int64_t)w * 8;
    return Cut{o[0], o[1], o[2], o[3], o[4], o[5]};
}

// log2 of a sum relative to a maximum, as a natural logarithm
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? neg_inf() : (m + log2f(l)) * 0.69314718055994530942f;
}

} // namespace gdn
