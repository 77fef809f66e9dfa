// Device helpers of the MXFP4 kernels.
#pragma once
#include "gq_common.h"

namespace gq {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// 2^(s - 127) of a scale byte as the conversion instructions take it: they read the
// exponent field alone, so 0 stands for 2^-127 and 255 for NaN
__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(s << 23); }

// the two values of byte B of q, scaled, as a bfloat16 pair
template <int B>
__device__ __forceinline__ uint32_t mx_bf16(uint32_t q, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, B);
    return __builtin_bit_cast(uint32_t, r);
}

// a / b for a, b >= 0: 64-bit division is some hundred instructions, and few sizes need it
__device__ __forceinline__ int64_t mx_div(int64_t a, int64_t b) {
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

}  // namespace gq
