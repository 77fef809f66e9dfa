// MXFP4 rows and products: what the entry points call, and device helpers of the kernels.
#pragma once
#include "gq_common.h"
#include "gq_internal.h"

namespace gq {

// timer stages, behind those of the other entry points (gq_mxfp4_stage of gq.h)
constexpr Stage ST_MXFP4_PACK = (Stage)(ST_COUNT + 0), ST_MXFP4_GEMM = (Stage)(ST_COUNT + 1);

constexpr int64_t MX_MAX_D = (int64_t)1 << 20;      // widest row
constexpr int MX_MAX_EXPERTS = 4096;
__host__ __device__ inline int64_t mx_groups(int64_t d) { return (d + 127) / 128; }
__host__ __device__ inline int64_t mx_row_bytes(int64_t d) { return 64 * mx_groups(d); }
__host__ __device__ inline int64_t mx_row_scales(int64_t d) { return 4 * mx_groups(d); }
hipError_t mx_quantize_run(const void* x, bool x_bf16, int64_t rows, int64_t d, uint8_t* Q,
                           uint8_t* S, hipStream_t st);
hipError_t mx_dequantize_run(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t d, void* y,
                             bool y_bf16, hipStream_t st);

enum MxOp { MX_GEMM = 0, MX_GEMM_MX = 1, MX_GEMM_DX = 2 };
// One product: a [n][k] (bfloat16, float32, or MXFP4 with as) by W [experts][d_out][d_in].
struct MxCall {
    MxOp op;
    const void* a;
    const uint8_t* as;            // scales of a (MX_GEMM_MX)
    bool a_bf16;
    int64_t n, d_in, d_out;
    const uint8_t *Q, *S;
    int experts;
    const int64_t* offsets;       // null: one weight for all rows
    void* y;
    bool y_bf16;
};
size_t mx_gemm_workspace(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts);
bool mx_gemm_fits(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets);
// planes, streamed, rows and columns of a tile, waves, split; returns the rows that the first product takes
int64_t mx_gemm_plan(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets, int32_t (&plan)[6]);
hipError_t mx_gemm_run(const MxCall& c, void* ws, hipStream_t st);

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
