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

// a code's value (scale 1)
__device__ __forceinline__ float mx_value(uint32_t q) {
    const float m = (q & 4u) ? (float)(2u + (q & 1u)) * ((q & 2u) ? 2.f : 1.f) : 0.5f * (float)(q & 3u);
    return (q & 8u) ? -m : m;
}

}  // namespace gq
