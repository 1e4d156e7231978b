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

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

} // namespace gdn
