// Products in 8-bit floating point with block scales, and with bfloat16 weights those of the gated
// feed-forward block, on gfx950.
//
//   MM_NT    y[t][j] = sum_i a[t][i] w[j][i]
//   MM_GATE  h[t][j] = act(zg) zu, zg[t][j] = sum_i a[t][i] g[j][i], zu alike
//   MM_NN    y[t][i] = sum_j a[t][j] w[j][i], of two pairs (a, w) added
//   MM_TN    y[j][i] = sum_t a[t][j] x[t][i], for two a
#include "gq_mm.h"

namespace gq {

// ---------------------------------------------------------------------------
// Every product in its plainest form: blocks of 64 x 64 outputs, 16 of the contraction at a time
// through LDS as float32.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float mm_value(MmElt elt, const void* p, int64_t row_bytes, int64_t row, int64_t i) {
    if (elt == MM_BF16) return bf16_bits_to_f32(*(const uint16_t*)((const char*)p + row * row_bytes + 2 * i));
    return __builtin_amdgcn_cvt_f32_fp8((int)*((const uint8_t*)p + row * row_bytes + i), 0);
}

__device__ __forceinline__ float mm_scale(MmElt elt, const void* S, int64_t i) {
    if (elt == MM_BF16) return 1.f;
    return elt == MM_E8 ? fp8_load_scale<false>(S, i) : fp8_load_scale<true>(S, i);
}

__global__ __launch_bounds__(256) void k_mm_plain(MmCall c, int64_t a_row, int64_t w_row) {
    __shared__ float xs[16][65], wsh[2][16][65];
    __shared__ int64_t place[4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const bool tn = c.form == MM_TN, nn = c.form == MM_NN, gate = c.form == MM_GATE;
    const int64_t m = nn || tn ? c.d_in : c.d_out, j0 = (int64_t)blockIdx.x * 64;
    int64_t e = 0, lo = 0, hi = c.n, t0 = (int64_t)blockIdx.y * 64;
    const int which = tn ? blockIdx.z & 1 : 0;
    if (tn && !c.y[which]) return;
    if (tn) {
        e = blockIdx.z >> 1;
        if (c.offsets) {
            lo = c.offsets[e];
            hi = c.offsets[e + 1];
            lo = lo < 0 ? 0 : (lo > c.n ? c.n : lo);
            hi = hi < lo ? lo : (hi > c.n ? c.n : hi);
        }
    } else if (c.offsets) {
        if (tid == 0) {
            int64_t left = blockIdx.y, found = -1, a = 0, b = 0;
            for (int x = 0; x < c.experts && found < 0; ++x) {
                a = c.offsets[x];
                b = c.offsets[x + 1];
                a = a < 0 ? 0 : (a > c.n ? c.n : a);
                b = b < a ? a : (b > c.n ? c.n : b);
                const int64_t tiles = (b - a + 63) / 64;
                if (left < tiles) found = x;
                else left -= tiles;
            }
            place[0] = found;
            place[1] = a + 64 * left;
            place[2] = b;
        }
        __syncthreads();
        e = place[0];
        if (e < 0) return;
        t0 = place[1];
        hi = place[2];
    }
    const int64_t rows_end = tn ? c.d_out : hi;
    if (t0 >= rows_end) return;
    const int64_t k_one = tn ? hi - lo : (nn ? c.d_out : c.d_in), k_all = nn && c.a[1] ? 2 * k_one : k_one;
    const int64_t wblocks = fp8_blocks(c.d_in), sbase = e * ((c.d_out + 127) / 128) * wblocks;
    const int64_t aspr = fp8_scales(nn ? c.d_out : c.d_in);
    float acc[2][4][4] = {};
    for (int64_t k0 = 0; k0 < k_all; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            const int kk = i & 15, r = i >> 4;
            const int64_t k = k0 + kk, src = nn && k >= k_one ? 1 : 0, kl = k - src * k_one;
            float x = 0.f, w[2] = {0.f, 0.f};
            if (k < k_all) {
                if (t0 + r < rows_end) {
                    if (tn) x = mm_value(c.elt, c.a[which], a_row, lo + kl, t0 + r);
                    else x = mm_value(c.elt, c.a[src], a_row, t0 + r, kl) * mm_scale(c.elt, c.as, (t0 + r) * aspr + kl / 128);
                }
                if (j0 + r < m) {
                    if (tn) w[0] = mm_value(c.elt, c.w[0], w_row, lo + kl, j0 + r);
                    else if (nn) w[0] = mm_value(c.elt, c.w[src], w_row, e * c.d_out + kl, j0 + r) * mm_scale(c.elt, c.ws[src], sbase + kl / 128 * wblocks + (j0 + r) / 128);
                    else
                        for (int q = 0; q <= gate; ++q)
                            w[q] = mm_value(c.elt, c.w[q], w_row, e * c.d_out + j0 + r, kl) * mm_scale(c.elt, c.ws[q], sbase + (j0 + r) / 128 * wblocks + kl / 128);
                }
            }
            xs[kk][r] = x;
            wsh[0][kk][r] = w[0];
            wsh[1][kk][r] = w[1];
        }
        __syncthreads();
        for (int kk = 0; kk < 16; ++kk)
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b) {
                    acc[0][a][b] += xs[kk][ty + 16 * a] * wsh[0][kk][tx + 16 * b];
                    if (gate) acc[1][a][b] += xs[kk][ty + 16 * a] * wsh[1][kk][tx + 16 * b];
                }
        __syncthreads();
    }
    void* y = tn ? (char*)c.y[which] + e * c.d_out * m * (c.y_bf16 ? 2 : 4) : c.y[0];
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int64_t t = t0 + ty + 16 * a, j = j0 + tx + 16 * b;
            if (t >= rows_end || j >= m) continue;
            float v = acc[0][a][b];
            if (gate) {
                if (c.z[0]) {
                    c.z[0][t * m + j] = v;
                    c.z[1][t * m + j] = acc[1][a][b];
                }
                v = act_of<false>(v, c.act, nullptr) * acc[1][a][b];
            }
            if (c.y_bf16) ((uint16_t*)y)[t * m + j] = (uint16_t)f32_to_bf16_bits(v);
            else ((float*)y)[t * m + j] = v;
        }
}

// h [n][m] of float32 into packed rows, those of an expert alone
template <bool F32>
__global__ __launch_bounds__(256) void k_mm_pack(const float* __restrict__ h, int64_t n, int64_t m,
                                                const int64_t* __restrict__ offsets, int experts, u32x2* __restrict__ Q,
                                                void* __restrict__ S) {
    const int64_t ppr = 16 * fp8_blocks(m), spr = fp8_scales(m), pieces = n * ppr;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= pieces) return;
    const int64_t r = mx_div(t, ppr), p = t - r * ppr, i = p * 8;
    if (offsets && (r < offsets[0] || r >= offsets[experts])) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < m) mx_load8<false>(h, r * m, i, m, v);
    uint32_t top = 0u;
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
        top = top > b ? top : b;
    }
    for (int o = 1; o < 16; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)top, o, 64);
        top = top > b ? top : b;
    }
    const uint32_t s = fp8_scale_byte(top);
    const float f = fp8_scale_inverse(s);
    const u32x2 q{fp8_pack4(v[0] * f, v[1] * f, v[2] * f, v[3] * f), fp8_pack4(v[4] * f, v[5] * f, v[6] * f, v[7] * f)};
    Q[t] = s == 255u ? u32x2{0u, 0u} : q;
    if (p % 16 == 0)
        for (int64_t b = p / 16; b < (p + 16 >= ppr ? spr : p / 16 + 1); ++b) {
            const uint32_t byte = b == p / 16 ? s : 127u;
            if (F32) ((float*)S)[r * spr + b] = fp8_scale_value(byte);
            else ((uint8_t*)S)[r * spr + b] = (uint8_t)byte;
        }
}

size_t mm_workspace(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed) {
    return packed ? ((size_t)n * d_out * 4 + 255) / 256 * 256 : 0;
}

bool mm_fits(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets, bool packed) {
    const int64_t rows = form == MM_TN ? d_out : n + 64 * (offsets ? experts : 0);
    return rows <= 65535 * 64 && ((form == MM_NN || form == MM_TN ? d_in : d_out) + 63) / 64 <= 1 << 23;
}

hipError_t mm_run(const MmCall& call, void* ws, hipStream_t st) {
    MmCall c = call;
    StageTimer tm(c.form == MM_GATE ? ST_FFN_GATE : (c.elt == MM_BF16 ? ST_FFN_BACK : ST_FP8_GEMM), st);
    if (c.hq) c.y[0] = ws;
    const bool fp8 = c.elt != MM_BF16;
    const int64_t ak = c.form == MM_NT || c.form == MM_GATE ? c.d_in : c.d_out;
    const int64_t m = c.form == MM_NN || c.form == MM_TN ? c.d_in : c.d_out;
    const int64_t rows = c.form == MM_TN ? (c.d_out + 63) / 64 : (c.n + 63) / 64 + (c.offsets ? c.experts : 0);
    const dim3 grid((unsigned)((m + 63) / 64), (unsigned)rows, c.form == MM_TN ? 2 * c.experts : 1);
    hipLaunchKernelGGL(k_mm_plain, grid, dim3(256), 0, st, c, fp8 ? fp8_bytes(ak) : 2 * ak, fp8 ? fp8_bytes(c.d_in) : 2 * c.d_in);
    GQ_LAUNCH_CHECK();
    if (c.hq) {
        const int64_t pieces = c.n * 16 * fp8_blocks(m);
        const auto k = c.elt == MM_FS ? k_mm_pack<true> : k_mm_pack<false>;
        hipLaunchKernelGGL(k, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, st, (const float*)ws, c.n, m, c.offsets, c.experts, (u32x2*)c.hq, c.hs);
        GQ_LAUNCH_CHECK();
    }
    return hipSuccess;
}

}  // namespace gq
