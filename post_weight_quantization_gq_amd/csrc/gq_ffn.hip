// The gated feed-forward block's backward pass, element by element, on gfx950.
//
//   h = act(zg) zu:   dzg = dh zu act'(zg),   dzu = dh act(zg)
//
// zg and zu are the forward pass's float32 products: rounded to bfloat16 they would add its half step to
// every gradient a second time, and their bytes are a twentieth of a training step's time.  dzg and dzu are
// rounded once, to the bfloat16 that the products after them multiply (and that the Fisher takes), also for float32
// gradients: 0.00166 of a gradient's norm, as much as rounding the gradient itself takes, 0.00235 together.  A
// second bfloat16 for what the first leaves would double the products after it, 1.1 of a training step's 1.9 ms.
// One pass, bound by HBM: 14 bytes a value with a bfloat16 dh (4096 x 11008: 125 us, 5.0 TB/s).
#include "gq_mm.h"

namespace gq {

// A lane takes 8 values of a row.
template <bool BF16>
__global__ __launch_bounds__(256) void k_ffn_dz(const void* __restrict__ dh, const float* __restrict__ zg,
                                               const float* __restrict__ zu, int64_t rows, int64_t f, int64_t pitch, int act,
                                               uint16_t* __restrict__ dzg, uint16_t* __restrict__ dzu) {
    const int64_t ppr = (f + 7) / 8, pieces = rows * ppr, stride = (int64_t)gridDim.x * 256;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < pieces; t += stride) {
        const int64_t r = mx_div(t, ppr), i = (t - r * ppr) * 8, at = r * pitch + i;
        float d[8], g[8], u[8];
        mx_load8<BF16>(dh, r * f, i, f, d);
        mx_load8<false>(zg, r * f, i, f, g);
        mx_load8<false>(zu, r * f, i, f, u);
        uint32_t a[4], b[4];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float s0, s1;
            const float v0 = act_of<true>(g[k], act, &s0), v1 = act_of<true>(g[k + 1], act, &s1);
            a[k / 2] = pack_bf16x2(d[k] * u[k] * s0, d[k + 1] * u[k + 1] * s1);
            b[k / 2] = pack_bf16x2(d[k] * v0, d[k + 1] * v1);
        }
        if (i + 8 <= pitch) {
            *(u32x4_any*)(dzg + at) = u32x4{a[0], a[1], a[2], a[3]};
            *(u32x4_any*)(dzu + at) = u32x4{b[0], b[1], b[2], b[3]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k < f) {
                    dzg[at + k] = (uint16_t)(a[k / 2] >> (16 * (k & 1)));
                    dzu[at + k] = (uint16_t)(b[k / 2] >> (16 * (k & 1)));
                }
        }
    }
}

hipError_t ffn_dz_run(const void* dh, bool dh_bf16, const float* zg, const float* zu, int64_t rows, int64_t f, int64_t pitch,
                      int act, uint16_t* dzg, uint16_t* dzu, hipStream_t st) {
    StageTimer tm(ST_FFN_BACK, st);
    const int64_t blocks = (rows * ((f + 7) / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    if (dh_bf16) hipLaunchKernelGGL(k_ffn_dz<true>, grid, dim3(256), 0, st, dh, zg, zu, rows, f, pitch, act, dzg, dzu);
    else hipLaunchKernelGGL(k_ffn_dz<false>, grid, dim3(256), 0, st, dh, zg, zu, rows, f, pitch, act, dzg, dzu);
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

}  // namespace gq
