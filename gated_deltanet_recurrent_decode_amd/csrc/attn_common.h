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

// log2 of a sum relative to a maximum, as a natural logarithm
__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? neg_inf() : (m + log2f(l)) * 0.69314718055994530942f;
}

} // namespace gdn
