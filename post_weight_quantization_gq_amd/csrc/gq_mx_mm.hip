// Products with MXFP4 weights on gfx950.
#include "gq_common.h"
#include "gq_internal.h"
#include "gq_mx.h"

namespace gq {

// Rows of expert e, clamped to [0, n].
__device__ __forceinline__ void mx_expert_rows(const int64_t* offsets, int e, int64_t n, int64_t& lo,
                                               int64_t& hi) {
    lo = 0;
    hi = n;
    if (!offsets) return;
    lo = offsets[e];
    hi = offsets[e + 1];
    lo = lo < 0 ? 0 : (lo > n ? n : lo);
    hi = hi < 0 ? 0 : (hi > n ? n : hi);
}

// One output a thread: the definition as it stands.
template <int OP>
__global__ __launch_bounds__(256) void k_mx_plain(MxCall c) {
    const int64_t m = OP == MX_GEMM_DX ? c.d_in : c.d_out, k = OP == MX_GEMM_DX ? c.d_out : c.d_in;
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int e = blockIdx.z;
    int64_t lo, hi;
    mx_expert_rows(c.offsets, e, c.n, lo, hi);
    const int64_t t = lo + blockIdx.y;
    if (j >= m || t >= hi) return;
    const int64_t qb = mx_row_bytes(c.d_in), sb = mx_row_scales(c.d_in);
    const uint8_t* Q = c.Q + (int64_t)e * c.d_out * qb;
    const uint8_t* S = c.S + (int64_t)e * c.d_out * sb;
    auto get = [](const uint8_t* q, const uint8_t* s, int64_t row, int64_t i, int64_t qb, int64_t sb) {
        const uint32_t b = q[row * qb + (i >> 1)], sc = s[row * sb + (i >> 5)];
        const float v = mx_value((i & 1) ? b >> 4 : b & 15u);
        return sc == 255u ? __uint_as_float(0x7fc00000u) : ldexpf(v, (int)sc - 127);
    };
    float acc = 0.f;
    for (int64_t i = 0; i < k; ++i) {
        float a;
        if (OP == MX_GEMM_MX) a = get((const uint8_t*)c.a, c.as, t, i, qb, sb);
        else a = c.a_bf16 ? load_elem<true>(c.a, t * k + i) : load_elem<false>(c.a, t * k + i);
        acc = fmaf(a, OP == MX_GEMM_DX ? get(Q, S, i, j, qb, sb) : get(Q, S, j, i, qb, sb), acc);
    }
    if (c.y_bf16) ((uint16_t*)c.y)[t * m + j] = (uint16_t)f32_to_bf16_bits(acc);
    else ((float*)c.y)[t * m + j] = acc;
}

size_t mx_gemm_workspace(MxOp, bool, int64_t, int64_t, int64_t, int) { return 0; }

hipError_t mx_gemm_run(const MxCall& c, void*, hipStream_t st) {
    StageTimer tm(ST_LUT_GEMV, st);
    const int64_t m = c.op == MX_GEMM_DX ? c.d_in : c.d_out;
    const dim3 grid((unsigned)((m + 255) / 256), (unsigned)c.n, (unsigned)c.experts);
    switch (c.op) {
        case MX_GEMM: hipLaunchKernelGGL(k_mx_plain<MX_GEMM>, grid, dim3(256), 0, st, c); break;
        case MX_GEMM_MX: hipLaunchKernelGGL(k_mx_plain<MX_GEMM_MX>, grid, dim3(256), 0, st, c); break;
        default: hipLaunchKernelGGL(k_mx_plain<MX_GEMM_DX>, grid, dim3(256), 0, st, c); break;
    }
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

}  // namespace gq
