// Rows and weights in 8-bit floating point (e4m3) with a scale for each block of 128, or of 128 x 128,
// on gfx950: quantisation and reading back.
//
// A block of values x_i has the scale 2^e, e the smallest in -127.. with max|x_i| <= 448 2^e, and the
// codes are x_i 2^-e rounded to the nearest e4m3 value (ties to even).  The scale being a power of two,
// x_i 2^-e is exact and each value is rounded once; a scale max|x| / 448 would use at most one binade more of
// the codes' fifteen, and would round twice.  Both directions are one pass over the data, bound by HBM.
//
// A lane takes 8 consecutive values: 16 lanes are a row's block, its maximum four exchanges.  A weight's
// block is 256 lanes that keep their 64 values in registers between the maximum and the rounding.
//
// 8192 x 28672 bfloat16 values: rows packed in 122 to 125 us (5.7 TB/s), a weight in 145 to 160 (4.4 to 4.9), read back in
// 118 to 128 (5.5 to 6.0); one row of 4096 in 1.8 us.
#include "gq_mm.h"

namespace gq {

__device__ __forceinline__ uint32_t fp8_top8(const float (&v)[8]) {
    // the maximum by magnitude as its bits: they order like the values, NaN above infinity
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
        top = top > b ? top : b;
    }
    return top;
}

__device__ __forceinline__ u32x2 fp8_codes8(const float (&v)[8], uint32_t s) {
    const float f = fp8_scale_inverse(s);
    const u32x2 q{fp8_pack4(v[0] * f, v[1] * f, v[2] * f, v[3] * f), fp8_pack4(v[4] * f, v[5] * f, v[6] * f, v[7] * f)};
    return s == 255u ? u32x2{0u, 0u} : q;
}

template <bool F32>
__device__ __forceinline__ void fp8_store_scale(void* S, int64_t i, uint32_t s) {
    if constexpr (F32) ((float*)S)[i] = fp8_scale_value(s);
    else ((uint8_t*)S)[i] = (uint8_t)s;
}

// Lane t takes piece t of the padded rows (16 pieces a block).
template <bool BF16, bool F32>
__global__ __launch_bounds__(256) void k_fp8_quantize(const void* __restrict__ x, int64_t pieces, int64_t d,
                                                     int ppr, int spr, u32x2* __restrict__ Q, void* __restrict__ S) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= pieces) return;             // pieces is a multiple of 16: blocks stay whole
    const int64_t r = mx_div(t, ppr);
    const int p = (int)(t - r * ppr);
    const int64_t i = (int64_t)p * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < d) mx_load8<BF16>(x, r * d, i, d, v);
    uint32_t top = fp8_top8(v);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)top, o, 64);
        top = top > b ? top : b;
    }
    const uint32_t s = fp8_scale_byte(top);
    Q[t] = fp8_codes8(v, s);
    if ((p & 15) == 0) {
        fp8_store_scale<F32>(S, r * spr + p / 16, s);
        if (p + 16 >= ppr)               // the row's last block: what fills its scales up, 1
            for (int b = ppr / 16; b < spr; ++b) fp8_store_scale<F32>(S, r * spr + b, 127u);
    }
}

template <bool BF16>
__device__ __forceinline__ void fp8_store8(void* y, int64_t at, int64_t left, u32x2 q, float scale) {
    float v[8], lo[4], hi[4];
    fp8_unpack4(q[0], lo);
    fp8_unpack4(q[1], hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = lo[k] * scale;
        v[4 + k] = hi[k] * scale;
    }
    if constexpr (BF16) {
        const u32x4 w{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        uint16_t* o = (uint16_t*)y + at;
        if (left >= 8) {
            *(u32x4_any*)o = w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) o[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    } else {
        float* o = (float*)y + at;
        if (left >= 8) {
            *(f32x4_any*)o = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4_any*)(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) o[k] = v[k];
        }
    }
}

// WEIGHT: `spr` scales serve 128 rows, the rows counted within a weight of d_out from row `row0` of it on.
template <bool BF16, bool F32, bool WEIGHT>
__global__ __launch_bounds__(256) void k_fp8_dequantize(const u32x2* __restrict__ Q, const void* __restrict__ S,
                                                       int64_t pieces, int64_t d, int ppr, int spr, int64_t row0,
                                                       int64_t d_out, void* __restrict__ y) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= pieces) return;
    const int64_t r = mx_div(t, ppr);
    const int p = (int)(t - r * ppr);
    const int64_t i = (int64_t)p * 8;
    if (i >= d) return;
    int64_t at = r * spr + p / 16;
    if constexpr (WEIGHT) {
        const int64_t row = row0 + r, e = mx_div(row, d_out), in = row - e * d_out;
        at = (e * ((d_out + 127) / 128) + in / 128) * spr + p / 16;
    }
    fp8_store8<BF16>(y, r * d + i, d - i, Q[t], fp8_load_scale<F32>(S, at));
}

// A block of 128 x 128 values of one weight.
template <bool BF16, bool F32>
__global__ __launch_bounds__(256) void k_fp8_quantize_weight(const void* __restrict__ W, int64_t first, int64_t d_out,
                                                            int64_t d_in, int64_t rb, int64_t cb,
                                                            u32x2* __restrict__ Q, void* __restrict__ S) {
    __shared__ uint32_t tops[4];
    const int64_t block = first + blockIdx.x, row = mx_div(block, cb), c = block - row * cb;
    const int64_t e = mx_div(row, rb), r0 = (row - e * rb) * 128;
    const int tid = threadIdx.x, pr = tid >> 4;
    const int64_t i = c * 128 + (tid & 15) * 8;
    float v[8][8];
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
        const int64_t r = r0 + 16 * k + pr;
        if (r < d_out && i < d_in) mx_load8<BF16>(W, (e * d_out + r) * d_in, i, d_in, v[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = fp8_top8(v[k]);
        top = top > b ? top : b;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)top, o, 64);
        top = top > b ? top : b;
    }
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = top > tops[w] ? top : tops[w];
    const uint32_t s = fp8_scale_byte(top);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = r0 + 16 * k + pr;
        if (r < d_out) Q[((e * d_out + r) * cb + c) * 16 + (tid & 15)] = fp8_codes8(v[k], s);
    }
    if (tid == 0) fp8_store_scale<F32>(S, block, s);
}

// f(first row, rows) for parts of the rows, each one launch: a launch has fewer than 2^32 lanes.
template <class F>
static hipError_t fp8_rows_each(int64_t rows, int ppr, F f) {
    const int64_t most = ((int64_t)1 << 31) / ppr;
    for (int64_t r = 0; r < rows; r += most) {
        f(r, rows - r < most ? rows - r : most);
        GQ_LAUNCH_CHECK();
    }
    return hipSuccess;
}

hipError_t fp8_quantize_run(const void* x, bool x_bf16, int64_t rows, int64_t d, uint8_t* Q, void* S,
                            bool s_f32, hipStream_t st) {
    StageTimer tm(ST_FP8_PACK, st);
    const int ppr = (int)(16 * fp8_blocks(d)), spr = (int)fp8_scales(d);
    return fp8_rows_each(rows, ppr, [&](int64_t r, int64_t n) {
        const int64_t pieces = n * ppr;
        const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
        const void* v = (const char*)x + r * d * (x_bf16 ? 2 : 4);
        u32x2* q = (u32x2*)(Q + r * fp8_bytes(d));
        void* s = (char*)S + r * spr * (s_f32 ? 4 : 1);
        const auto k = x_bf16 ? (s_f32 ? k_fp8_quantize<true, true> : k_fp8_quantize<true, false>)
                              : (s_f32 ? k_fp8_quantize<false, true> : k_fp8_quantize<false, false>);
        hipLaunchKernelGGL(k, grid, block, 0, st, v, pieces, d, ppr, spr, q, s);
    });
}

template <bool WEIGHT>
static hipError_t fp8_back_run(const uint8_t* Q, const void* S, bool s_f32, int64_t rows, int64_t d, int spr,
                               int64_t d_out, void* y, bool y_bf16, hipStream_t st) {
    StageTimer tm(ST_FP8_PACK, st);
    const int ppr = (int)(16 * fp8_blocks(d));
    return fp8_rows_each(rows, ppr, [&](int64_t r, int64_t n) {
        const int64_t pieces = n * ppr;
        const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
        const u32x2* q = (const u32x2*)(Q + r * fp8_bytes(d));
        const void* s = WEIGHT ? S : (const void*)((const char*)S + r * spr * (s_f32 ? 4 : 1));
        void* v = (char*)y + r * d * (y_bf16 ? 2 : 4);
        const auto k = y_bf16 ? (s_f32 ? k_fp8_dequantize<true, true, WEIGHT> : k_fp8_dequantize<true, false, WEIGHT>)
                              : (s_f32 ? k_fp8_dequantize<false, true, WEIGHT> : k_fp8_dequantize<false, false, WEIGHT>);
        hipLaunchKernelGGL(k, grid, block, 0, st, q, s, pieces, d, ppr, spr, r, d_out, v);
    });
}

hipError_t fp8_dequantize_run(const uint8_t* Q, const void* S, bool s_f32, int64_t rows, int64_t d,
                              void* y, bool y_bf16, hipStream_t st) {
    return fp8_back_run<false>(Q, S, s_f32, rows, d, (int)fp8_scales(d), 1, y, y_bf16, st);
}

hipError_t fp8_dequantize_weight_run(const uint8_t* Q, const void* S, bool s_f32, int experts,
                                     int64_t d_out, int64_t d_in, void* y, bool y_bf16, hipStream_t st) {
    return fp8_back_run<true>(Q, S, s_f32, experts * d_out, d_in, (int)fp8_blocks(d_in), d_out, y, y_bf16, st);
}

hipError_t fp8_quantize_weight_run(const void* W, bool w_bf16, int experts, int64_t d_out, int64_t d_in,
                                   uint8_t* Q, void* S, bool s_f32, hipStream_t st) {
    StageTimer tm(ST_FP8_PACK, st);
    const int64_t rb = (d_out + 127) / 128, cb = fp8_blocks(d_in), blocks = experts * rb * cb, most = 1 << 23;
    const auto k = w_bf16 ? (s_f32 ? k_fp8_quantize_weight<true, true> : k_fp8_quantize_weight<true, false>)
                          : (s_f32 ? k_fp8_quantize_weight<false, true> : k_fp8_quantize_weight<false, false>);
    for (int64_t b = 0; b < blocks; b += most) {
        const dim3 grid((unsigned)(blocks - b < most ? blocks - b : most));
        hipLaunchKernelGGL(k, grid, dim3(256), 0, st, W, b, d_out, d_in, rb, cb, (u32x2*)Q, S);
        GQ_LAUNCH_CHECK();
    }
    return hipSuccess;
}

}  // namespace gq
