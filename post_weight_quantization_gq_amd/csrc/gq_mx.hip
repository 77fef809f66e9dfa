// MXFP4 rows on gfx950: quantisation and reading back.
//
// A block of 32 values x_i has the scale 2^e, e = clamp(floor(log2 max|x_i|) - 2, -127, 125),
// so its maximum lies in [4, 8) units of the scale; code_i is x_i 2^-e rounded to the nearest
// of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even index, 6 above it) with the sign of x_i.
// Both directions are one pass over the data, bound by HBM: a row of d values moves
// d (2 or 4) + 68 ceil(d / 128) bytes each way.
//
// A lane takes 8 consecutive values (a 16-byte load of bfloat16), so a block is 4 lanes and
// its maximum two exchanges between neighbours; the codes are a 4-byte store a lane.
//
// 8192 x 28672 bfloat16 values to MXFP4 and back: 220 to 224 us for 1.19 GB read and written (the
// packed rows both ways), 5.3 to 5.4 TB/s (a large copy on this card: 5.0 to 5.1); one row of 4096:
// 1.8 us each way, the launch.
#include "gq_mx.h"

namespace gq {

// Lane t of the grid takes the 8-value piece t of the padded rows (16 pieces a group of 128).
template <bool BF16>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ x, int64_t pieces,
                                                    int64_t d, int ppr, uint32_t* __restrict__ Q,
                                                    uint8_t* __restrict__ S) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= pieces) return;             // pieces is a multiple of 16: blocks stay whole
    const int64_t r = mx_div(t, ppr);
    const int64_t i = (t - r * ppr) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < d) mx_load8<BF16>(x, r * d, i, d, v);
    // the maximum by magnitude as its bits: they order like the values, NaN above infinity
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
        top = top > b ? top : b;
    }
    uint32_t o = (uint32_t)__shfl_xor((int)top, 1, 64);
    top = top > o ? top : o;
    o = (uint32_t)__shfl_xor((int)top, 2, 64);
    top = top > o ? top : o;
    // exponent field of the maximum minus 2 is the scale byte; below 2 (maximum under
    // 2^-125, subnormals and zero) it is 0
    const uint32_t ef = top >> 23;
    const bool bad = ef == 255u;
    const uint32_t s = bad ? 255u : (ef > 2u ? ef - 2u : 0u);
    const float scale = mx_scale(s);
    uint32_t q = 0u;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
    Q[t] = bad ? 0u : q;
    if ((t & 3) == 0) S[t >> 2] = (uint8_t)(i < d ? s : 127u);
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint32_t* __restrict__ Q,
                                                      const uint8_t* __restrict__ S,
                                                      int64_t pieces, int64_t d, int ppr,
                                                      void* __restrict__ y) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= pieces) return;
    const int64_t r = mx_div(t, ppr);
    const int64_t i = (t - r * ppr) * 8;
    if (i >= d) return;
    const uint32_t q = Q[t];
    const float scale = mx_scale(S[t >> 2]);
    const int64_t at = r * d + i;
    if constexpr (BF16) {
        const u32x4 w{mx_bf16<0>(q, scale), mx_bf16<1>(q, scale), mx_bf16<2>(q, scale),
                      mx_bf16<3>(q, scale)};
        uint16_t* o = (uint16_t*)y + at;
        if (i + 8 <= d) {
            *(u32x4_any*)o = w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < d) o[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    } else {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1);
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2);
        const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3);
        const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
        float* o = (float*)y + at;
        if (i + 8 <= d) {
            *(f32x4_any*)o = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4_any*)(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < d) o[k] = v[k];
        }
    }
}

// f(first row, rows) for parts of the rows, each one launch: a launch has fewer than 2^32 lanes,
// which 2^28 rows of up to 128 values would take (a loop in the kernels instead costs them 4 %
// at any size: 8192 x 28672 there and back 233 us, 224 without).
template <class F>
static hipError_t mx_rows_each(int64_t rows, int ppr, F f) {
    const int64_t most = ((int64_t)1 << 31) / ppr;
    for (int64_t r = 0; r < rows; r += most) {
        f(r, rows - r < most ? rows - r : most);
        GQ_LAUNCH_CHECK();
    }
    return hipSuccess;
}

hipError_t mx_quantize_run(const void* x, bool x_bf16, int64_t rows, int64_t d, uint8_t* Q,
                           uint8_t* S, hipStream_t st) {
    StageTimer tm(ST_MXFP4_PACK, st);
    const int ppr = (int)(16 * mx_groups(d));
    return mx_rows_each(rows, ppr, [&](int64_t r, int64_t n) {
        const int64_t pieces = n * ppr;
        const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
        const void* v = (const char*)x + r * d * (x_bf16 ? 2 : 4);
        uint32_t* q = (uint32_t*)(Q + r * mx_row_bytes(d));
        uint8_t* s = S + r * mx_row_scales(d);
        if (x_bf16) hipLaunchKernelGGL(k_mx_quantize<true>, grid, block, 0, st, v, pieces, d, ppr, q, s);
        else hipLaunchKernelGGL(k_mx_quantize<false>, grid, block, 0, st, v, pieces, d, ppr, q, s);
    });
}

hipError_t mx_dequantize_run(const uint8_t* Q, const uint8_t* S, int64_t rows, int64_t d, void* y,
                             bool y_bf16, hipStream_t st) {
    StageTimer tm(ST_MXFP4_PACK, st);
    const int ppr = (int)(16 * mx_groups(d));
    return mx_rows_each(rows, ppr, [&](int64_t r, int64_t n) {
        const int64_t pieces = n * ppr;
        const dim3 grid((unsigned)((pieces + 255) / 256)), block(256);
        const uint32_t* q = (const uint32_t*)(Q + r * mx_row_bytes(d));
        const uint8_t* s = S + r * mx_row_scales(d);
        void* v = (char*)y + r * d * (y_bf16 ? 2 : 4);
        if (y_bf16) hipLaunchKernelGGL(k_mx_dequantize<true>, grid, block, 0, st, q, s, pieces, d, ppr, v);
        else hipLaunchKernelGGL(k_mx_dequantize<false>, grid, block, 0, st, q, s, pieces, d, ppr, v);
    });
}

}  // namespace gq
