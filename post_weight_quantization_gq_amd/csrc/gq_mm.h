// Products in 8-bit floating point with block scales, and the gated feed-forward block: what the
// entry points call.
#pragma once
#include "gq_common.h"
#include "gq_internal.h"
#include "gq_mx.h"

namespace gq {

// timer stages, behind the MXFP4 ones (gq_product_stage of gq.h)
constexpr Stage ST_FP8_PACK = (Stage)(ST_COUNT + 2), ST_FP8_GEMM = (Stage)(ST_COUNT + 3),
                ST_FFN_GATE = (Stage)(ST_COUNT + 4), ST_FFN_BACK = (Stage)(ST_COUNT + 5);

// ---- packed rows and weights: codes of a row in whole blocks of 128, a row's scales in fours
__host__ __device__ inline int64_t fp8_blocks(int64_t d) { return (d + 127) / 128; }
__host__ __device__ inline int64_t fp8_bytes(int64_t d) { return 128 * fp8_blocks(d); }
__host__ __device__ inline int64_t fp8_scales(int64_t d) { return (fp8_blocks(d) + 3) / 4 * 4; }

hipError_t fp8_quantize_run(const void* x, bool x_bf16, int64_t rows, int64_t d, uint8_t* Q, void* S,
                            bool s_f32, hipStream_t st);
hipError_t fp8_dequantize_run(const uint8_t* Q, const void* S, bool s_f32, int64_t rows, int64_t d,
                              void* y, bool y_bf16, hipStream_t st);
hipError_t fp8_quantize_weight_run(const void* W, bool w_bf16, int experts, int64_t d_out, int64_t d_in,
                                   uint8_t* Q, void* S, bool s_f32, hipStream_t st);
hipError_t fp8_dequantize_weight_run(const uint8_t* Q, const void* S, bool s_f32, int experts,
                                     int64_t d_out, int64_t d_in, void* y, bool y_bf16, hipStream_t st);

// ---- products
enum MmForm {
    MM_NT = 0,                    // y = a W^T
    MM_GATE = 1,                  // h = act(a G^T) (a U^T)
    MM_NN = 2,                    // y = a W, or a[0] W[0] + a[1] W[1]
    MM_TN = 3                     // y[i] = a[i]^T w, for two a
};
// bfloat16; e4m3 with scales 2^(s - 127), or float32 ones.  The matrix cores add the products of 8 codes
// to 14 bits of their largest (a second product 2^-13 as large counts, one of 2^-14 is lost; between eights, and with
// the accumulator, all 24 bits count).  That leaves 4e-5 of a result, 4e-4 where one activation in 200 is 30 times the
// others: a quarter of a bfloat16 output's rounding or less, so such outputs take it.  The W types are for
// float32 outputs, and for packed ones, whose rounding a sum next to a border would take to the other side
// (a block of gate and down projection, against float64: 0.0033 off so, 0.0017 by W): codes converted
// to bfloat16 in registers, whose products are added in float32, at half the rate (4096 rows, 8192 -> 4096:
// 105 us, and 225 by W).
enum MmElt { MM_BF16 = 0, MM_E8 = 1, MM_FS = 2, MM_E8W = 3, MM_FSW = 4 };
constexpr bool mm_bytes(int elt) { return elt == MM_E8 || elt == MM_E8W; }     // scales are bytes
constexpr bool mm_wide(int elt) { return elt == MM_E8W || elt == MM_FSW; }

struct MmCall {
    MmForm form;
    MmElt elt;
    const void* a[2];             // rows of activations, n of them (MM_GATE: one; MM_NN: as many as weights)
    bool a_padded;                // bfloat16 rows that start at multiples of 8 values, zeros between
    const void* as;               // their scales
    int64_t n, d_in, d_out;
    const void* w[2];             // weights [experts][d_out][d_in] (MM_TN: x [n][d_in])
    const void* ws[2];            // their scales
    int experts;
    const int64_t* offsets;       // null: one weight for all rows
    void* y[2];                   // (MM_TN: two)
    bool y_bf16;
    float* z[2];                  // MM_GATE: both products, or null
    uint8_t* hq;                  // MM_GATE: h in packed rows instead of y, or null
    void* hs;
    int act;
};
size_t mm_workspace(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed, bool a_padded = false);
bool mm_fits(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets, bool packed);
// plan: wide, streamed, rows, columns, waves, parts
void mm_describe(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed, int32_t plan[6]);
hipError_t mm_run(const MmCall& c, void* ws, hipStream_t st);

// dzg = dh zu act'(zg), dzu = dh act(zg), `rows` rows of f values; those of dzg and dzu start `pitch` values
// (f, or f rounded up to a multiple of 8: zeros between) apart
hipError_t ffn_dz_run(const void* dh, bool dh_bf16, const float* zg, const float* zu, int64_t rows, int64_t f, int64_t pitch,
                      int act, uint16_t* dzg, uint16_t* dzu, hipStream_t st);

// ---- activations (gq_activation of gq.h)
enum Act { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

// 1 / (1 + e^-z) by the exponential and reciprocal instructions (an ulp each; the exponential's argument, rounded
// once more, adds |z| 2^-24): a gate's epilogue evaluates one for two products of the whole contraction, and the
// library's exponential and division took four times the instructions (8-bit gate of 4096 rows, 8192 -> 2048 packed:
// 118 us, 114 so).  The reciprocal's results below 2^-126 are zero.
__device__ __forceinline__ float logistic(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// act(z); *slope = act'(z).  Written so that neither tail cancels: 1 + tanh(u) = 2 / (1 + e^-2u), and
// the normal distribution's lower tail by erfc.
template <bool SLOPE>
__device__ __forceinline__ float act_of(float z, int act, float* slope) {
    if (act == ACT_GELU) {
        const float c = 0.5f * erfcf(z * -0.70710678118654752f);
        if (SLOPE) *slope = c + z * (0.39894228040143268f * expf(-0.5f * z * z));
        return z * c;
    }
    if (act == ACT_GELU_TANH) {
        const float k = 0.79788456080286536f, z2 = z * z;
        const float s = logistic(2.f * k * z * (1.f + 0.044715f * z2));
        // (where z z is over the largest number, s (1 - s) is zero)
        if (SLOPE) *slope = s + 2.f * z * s * (1.f - s) * (k * (1.f + 0.134145f * fminf(z2, 1e30f)));
        return z * s;
    }
    const float s = logistic(z);
    if (SLOPE) *slope = s * (1.f + z * (1.f - s));
    return z * s;
}

// ---- 8-bit conversions
// The scale byte of a block whose largest magnitude has the bits `top` (sign cleared): the smallest s
// with top <= 448 2^(s - 127), 448 = 1.75 2^8; 255 for NaN and infinity.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top) {
    const uint32_t s = (top >> 23) + ((top & 0x7fffffu) > 0x600000u ? 1u : 0u);
    return top >= 0x7f800000u ? 255u : (s > 8u ? s - 8u : 0u);
}
// 2^(s - 127), NaN for 255
__device__ __forceinline__ float fp8_scale_value(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7fc00000u : s << 23));
}
// 2^(127 - s), by which values are multiplied before they are rounded; 0 for 255
__device__ __forceinline__ float fp8_scale_inverse(uint32_t s) {
    return __uint_as_float(s == 255u ? 0u : (254u - s) << 23);
}
// four values (none over 448) rounded to e4m3, ties to even
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}
__device__ __forceinline__ void fp8_unpack4(uint32_t q, float (&v)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}
// scale i of an array in either type
template <bool F32>
__device__ __forceinline__ float fp8_load_scale(const void* S, int64_t i) {
    if constexpr (F32) return ((const float*)S)[i];
    else return fp8_scale_value(((const uint8_t*)S)[i]);
}

}  // namespace gq
