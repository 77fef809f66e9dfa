// Device helpers of the MXFP4 kernels.
#pragma once
#include "gq_common.h"

namespace gq {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// vectors at any element's address: a row of odd length starts anywhere, and the memory
// instructions take that
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// 8 values of a row of d from element i < d of it (row0: the row's first element); past the row: 0
template <bool BF16>
__device__ __forceinline__ void mx_load8(const void* p, int64_t row0, int64_t i, int64_t d,
                                         float (&v)[8]) {
    if (i + 8 <= d) {
        if constexpr (BF16) {
            const u32x4 w = *(const u32x4_any*)((const uint16_t*)p + row0 + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        } else {
            const f32x4 a = *(const f32x4_any*)((const float*)p + row0 + i);
            const f32x4 b = *(const f32x4_any*)((const float*)p + row0 + i + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) { v[k] = a[k]; v[4 + k] = b[k]; }
        }
    } else {
        // (loaded without a condition: past the row, its element i)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = load_elem<BF16>(p, row0 + (i + k < d ? i + k : i));
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < d ? v[k] : 0.f;
    }
}

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
