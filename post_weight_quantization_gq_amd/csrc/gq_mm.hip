// Products in 8-bit floating point with block scales, and with bfloat16 weights those of the gated
// feed-forward block, on gfx950.
//
//   MM_NT    y[t][j] = sum_i a[t][i] w[j][i]
//   MM_GATE  h[t][j] = act(zg) zu, zg[t][j] = sum_i a[t][i] g[j][i], zu alike
//   MM_NN    y[t][i] = sum_j a[t][j] w[j][i], of two pairs (a, w) added
//   MM_TN    y[j][i] = sum_t a[t][j] x[t][i], for two a
//
// This file plans a call and runs what is not a product: copies of rows whose length the
// asynchronous loads cannot take, and the outputs of contractions that are split over blocks.
#include "gq_mm_plan.h"
#include "gq_tile.h"
#include <math.h>

namespace gq {

// Rows of k bfloat16 values as rows of a multiple of 8, zeros behind: up to four arrays of them, `ends` the
// pieces of 8 up to each one's end.  One launch: a call of few rows is mostly launches (196 rows, gate of 1967 -> 585: 24.2 us by
// three launches, 20.3 so).
struct MmPadded {
    const void* x[4];
    int64_t k[4], ends[4];
    u32x4* out[4];
};
__global__ __launch_bounds__(256) void k_mm_pad(MmPadded a, int arrays) {
    const int64_t total = a.ends[arrays - 1], stride = (int64_t)gridDim.x * 256;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += stride) {
        const void* x = a.x[0];
        int64_t k = a.k[0], at = t;
        u32x4* out = a.out[0];
#pragma unroll
        for (int n = 1; n < 4; ++n)
            if (n < arrays && t >= a.ends[n - 1]) {
                x = a.x[n];
                k = a.k[n];
                at = t - a.ends[n - 1];
                out = a.out[n];
            }
        const int64_t pieces = (k + 7) / 8, r = mx_div(at, pieces), i = (at - r * pieces) * 8;
        float v[8];
        mx_load8<true>(x, r * k, i, k, v);
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xffff0000u);
        out[at] = w;
    }
}

// The rows of the experts' (all without offsets).
__device__ __forceinline__ void mm_rows(const int64_t* offsets, int experts, int64_t n, int64_t& lo, int64_t& hi) {
    lo = 0;
    hi = n;
    if (offsets) {
        int64_t a, b;
        tile_expert_rows(offsets, 0, n, lo, a);
        tile_expert_rows(offsets, experts - 1, n, b, hi);
    }
}

// The sum of `split` parts `all` values apart, V values of it, in their order.
template <class V>
__device__ __forceinline__ V mm_sum(const float* part, int split, int64_t all) {
    V s = *(const V*)part;
    int k = 1;
    for (; k + 4 <= split; k += 4) {               // four loads in flight, added in their order
        V v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *(const V*)(part + (k + i) * all);
#pragma unroll
        for (int i = 0; i < 4; ++i) s += v[i];
    }
    for (; k < split; ++k) s += *(const V*)(part + k * all);
    return s;
}

// y = the sum of a split contraction's parts, or of MM_GATE's two products h = act(zg) zu.
template <bool GATE>
__global__ __launch_bounds__(256) void k_mm_join(const float* __restrict__ part, int split, int64_t all, int64_t n, int64_t m,
                                                const int64_t* __restrict__ offsets, int experts, void* __restrict__ y, int y_bf16,
                                                int act, float* __restrict__ zg, float* __restrict__ zu) {
    int64_t lo, hi;
    mm_rows(offsets, experts, n, lo, hi);
    const int64_t first = lo * m, end = hi * m, stride = (int64_t)gridDim.x * 256;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, step = GATE ? 2 * all : all;
    auto value = [&](auto a, auto b) {
        if constexpr (!GATE) return a;
        else {
            auto v = a;
            if constexpr (sizeof(a) == 4) v = act_of<false>(a, act, nullptr) * b;
            else
                for (int i = 0; i < 4; ++i) v[i] = act_of<false>(a[i], act, nullptr) * b[i];
            return v;
        }
    };
    if (all % 4 == 0 && m % 4 == 0 && (((uintptr_t)y & (y_bf16 ? 7u : 15u)) | (((uintptr_t)zg | (uintptr_t)zu) & 15u)) == 0) {
        for (int64_t t = first + 4 * id; t < end; t += 4 * stride) {
            const f32x4 a = mm_sum<f32x4>(part + t, split, step), b = GATE ? mm_sum<f32x4>(part + all + t, split, step) : a;
            if (GATE && zg) {
                *(f32x4*)(zg + t) = a;
                *(f32x4*)(zu + t) = b;
            }
            const f32x4 s = value(a, b);
            if (y_bf16) *(u32x2*)((uint16_t*)y + t) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
            else *(f32x4*)((float*)y + t) = s;
        }
        return;
    }
    for (int64_t t = first + id; t < end; t += stride) {
        const float a = mm_sum<float>(part + t, split, step), b = GATE ? mm_sum<float>(part + all + t, split, step) : a;
        if (GATE && zg) {
            zg[t] = a;
            zu[t] = b;
        }
        const float s = value(a, b);
        if (y_bf16) ((uint16_t*)y)[t] = (uint16_t)f32_to_bf16_bits(s);
        else ((float*)y)[t] = s;
    }
}

// MM_GATE's h of a split contraction, or of tiles narrower than a block, into packed rows.  A lane takes
// 8 values, 16 lanes a block.
template <bool F32>
__global__ __launch_bounds__(256) void k_mm_join_pack(const float* __restrict__ part, int split, int64_t n, int64_t m,
                                                     const int64_t* __restrict__ offsets, int experts, int act,
                                                     u32x2* __restrict__ Q, void* __restrict__ S) {
    int64_t lo, hi;
    mm_rows(offsets, experts, n, lo, hi);
    const int64_t ppr = 16 * fp8_blocks(m), spr = fp8_scales(m), end = hi * ppr, all = n * m;
    for (int64_t t = lo * ppr + (int64_t)blockIdx.x * 256 + threadIdx.x; t < end; t += (int64_t)gridDim.x * 256) {
        const int64_t r = mx_div(t, ppr), p = t - r * ppr, i = p * 8;
        float v[8];
        if (m % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 a{0.f, 0.f, 0.f, 0.f}, b = a;
                if (i + 4 * h < m) {
                    const float* const from = part + r * m + i + 4 * h;
                    a = mm_sum<f32x4>(from, split, 2 * all);
                    b = mm_sum<f32x4>(from + all, split, 2 * all);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * h + k] = act_of<false>(a[k], act, nullptr) * b[k];
            }
        } else {
            for (int k = 0; k < 8; ++k) {
                v[k] = 0.f;
                if (i + k < m) {
                    const float* const from = part + r * m + i + k;
                    v[k] = act_of<false>(mm_sum<float>(from, split, 2 * all), act, nullptr) * mm_sum<float>(from + all, split, 2 * all);
                }
            }
        }
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
            top = top > b ? top : b;
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            const uint32_t b = (uint32_t)__shfl_xor((int)top, o, 64);
            top = top > b ? top : b;
        }
        const uint32_t s = fp8_scale_byte(top);
        const float f = fp8_scale_inverse(s);
        const u32x2 q{fp8_pack4(v[0] * f, v[1] * f, v[2] * f, v[3] * f), fp8_pack4(v[4] * f, v[5] * f, v[6] * f, v[7] * f)};
        Q[t] = s == 255u ? u32x2{0u, 0u} : q;
        if (p % 16 == 0)                           // with the row's last block, what fills its scales up: 1
            for (int64_t b = p / 16; b < (p + 16 >= ppr ? spr : p / 16 + 1); ++b) {
                const uint32_t byte = b == p / 16 ? s : 127u;
                if constexpr (F32) ((float*)S)[r * spr + b] = fp8_scale_value(byte);
                else ((uint8_t*)S)[r * spr + b] = (uint8_t)byte;
            }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static size_t mm_al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int64_t mm_al8(int64_t x) { return (x + 7) / 8 * 8; }

// Bytes of the padded copies of a call's activations and weights (each of them).
struct MmPads {
    size_t a, w;
    int as, ws;                   // how many
};
static MmPads mm_pads(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool a_padded) {
    MmPads p{};
    if (elt != MM_BF16) return p;
    const int64_t ak = form == MM_GATE ? d_in : d_out;
    p.as = form == MM_GATE ? 1 : 2;
    p.ws = form == MM_TN ? 1 : 2;
    if (ak % 8 && !a_padded) p.a = mm_al256((size_t)n * mm_al8(ak) * 2);
    if (d_in % 8) p.w = mm_al256((size_t)(form == MM_TN ? n : experts * d_out) * mm_al8(d_in) * 2);
    return p;
}

// What a launch of tiles takes, in microseconds, as the tile and the split are chosen by: with L tiles on the fullest
// compute unit and S stages each, fixed L^0.5 + stage S L^0.85, and of a split contraction the joining launch
// with its float32 sums (thousands of them a microsecond, written and read).  Fitted to launches of 16 to 4096 rows,
// contractions of 1024 to 11008 and as many columns, every tile by splits of 1 to 16: in 257 such products
// the chosen pair takes 4 percent longer than the best one (geometric mean, on another card).  A rule of "the largest
// tile that leaves 192 blocks, split to 256" took 7 percent longer, and up to twice as long (200 rows, 1024 x 1024:
// 13.3 us, 7.4 by tiles of 32 rows with no split; 400 rows, gradient of 1024 -> 4096: 22.3 and 13.3).
struct MmCost {
    float fixed[4], stage[4];     // by tiles of 32, 64, 128 and 256 rows; 0: no such tile
    float join, sums;
};
static const MmCost& mm_cost(MmForm form, MmElt elt) {
    static const MmCost rows8{{4.5f, 5.4f, 6.1f, 11.f}, {.38f, .42f, .63f, 1.23f}, 3.1f, 890.f};
    static const MmCost rowsw{{5.7f, 6.4f, 9.6f, 0.f}, {.66f, .63f, 1.49f, 0.f}, 2.6f, 830.f};
    static const MmCost gate{{3.6f, 5.3f, 6.1f, 8.9f}, {.35f, .4f, .63f, 1.37f}, 3.8f, 850.f};
    static const MmCost back8{{0.f, 6.8f, 6.6f, 9.4f}, {0.f, .79f, 1.13f, 1.25f}, 3.5f, 700.f};
    static const MmCost backw{{0.f, 8.3f, 9.1f, 0.f}, {0.f, 1.35f, 1.59f, 0.f}, 1.7f, 580.f};
    static const MmCost back{{0.f, 9.6f, 9.1f, 11.3f}, {0.f, .72f, .98f, 1.24f}, 1.f, 650.f};
    static const MmCost turned{{0.f, 0.f, 8.6f, 14.5f}, {0.f, 0.f, .57f, 1.45f}, 1.7f, 800.f};
    if (form == MM_TN) return turned;
    if (form == MM_NN) return elt == MM_BF16 ? back : (mm_wide(elt) ? backw : back8);
    return elt == MM_BF16 ? gate : (mm_wide(elt) ? rowsw : rows8);
}

static MmPlan mm_plan(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed, bool a_padded = false) {
    MmPlan P{};
    const bool tn = form == MM_TN, gate = form == MM_GATE, nn = form == MM_NN, fp8 = elt != MM_BF16, wide = mm_wide(elt);
    const int64_t k = tn ? n : (nn ? d_out : d_in), m = tn || nn ? d_in : d_out, ke = fp8 ? 128 : 64;
    const int64_t one = (k + ke - 1) / ke, per = (n + experts - 1) / experts;
    const int64_t live = experts > 1 ? (experts < n ? experts : n) : 1;           // experts with rows, at most
    const int64_t outputs = tn ? 2 * (int64_t)experts * d_out * m : (gate ? 2 : 1) * n * m;
    const MmPads pads = mm_pads(form, elt, n, d_in, d_out, experts, a_padded);
    P.pad_bytes = pads.a * pads.as + pads.w * pads.ws;
    P.stages = (int)(nn && !fp8 ? 2 * one : one);
    P.unit = fp8 ? 4 : 1;
    P.split = 1;
    const int64_t wcols = gate ? 2 * m : m;                                       // rows of weights that outputs need
    // Streamed: up to 16 rows of one weight, 8 an expert on average.  Its activations come from the L2 again for
    // each block, so not for the longest rows (16 rows with float32 scales, 28672 -> 8192: 47.0 us streamed, 40.6 by
    // tiles; 1 row 36.4 and 40.3), and 8-bit sums of one weight so wide that tiles fill the card go by tiles (1 row,
    // 8192 -> 28672: 39.7 and 36.2; in bfloat16 sums 38.7 and 49.9).  16 rows, 128 experts of 4096 -> 1536: 20.2 us streamed,
    // 23.9 by tiles, their packed gate 40.7 and 64.6; 512 rows, 64 experts of 2048 -> 1408 35.3 and 34.5, 700 rows 41.3 and 34.9.
    P.stream = (form == MM_NT || gate) && per <= (experts > 1 ? 8 : 16) && per * k <= 1 << 18 &&
               (experts > 1 || !fp8 || wide || (wcols + 127) / 128 < 192);
    if (P.stream) {
        P.bm = 16;
        P.bn = gate || live * ((m + 31) / 32) >= 256 ? 32 : 16;
        const int64_t blocks = live * ((wcols + P.bn - 1) / P.bn);
        // eight waves, of at least two lines each, where all blocks fit the card at once: of 32 columns two a compute unit
        // (16 rows, float32 scales, 4096 -> 8192: 10.3 us by four waves, 8.7 by eight; 8-bit gate 4096 -> 11008, 688 blocks:
        // 21.7 and 23.4)
        P.waves = one >= 16 && (P.bn == 16 || blocks <= 512) ? 8 : 4;
        const int64_t units = one / (2 * P.waves);
        // a block to each compute unit (16 rows, 8192 -> 1024: 9.6 us whole, 7.7 split by 4, 8.4 by 8), but for
        // fewer than eight lines a wave (4096 -> 1024: 6.6 us whole, 7.1 split by 2)
        int64_t s = units < 4 || blocks >= 256 ? 1 : 256 / blocks;
        s = s < units ? s : units;
        s = s < 1 ? 1 : (s > 16 ? 16 : s);
        if (s > 1) {
            const int64_t some = (units + s - 1) / s, parts = (units + some - 1) / some;
            // no part without a line, as the kernel shares them among all parts' waves (1 row, gate of 11008 -> 130: 172
            // lines, three a wave: 8 parts, of 10 two would write and add zeros)
            const int64_t each = (one + P.waves * parts - 1) / (P.waves * parts);
            P.split = (int)((one + each * P.waves - 1) / (each * P.waves));
        }
        P.join = P.split > 1 || packed;
    } else {
        const MmCost& cost = mm_cost(form, elt);
        const int64_t stages = tn ? (per + ke - 1) / ke : P.stages, units = tn && experts > 1 ? 1 : (stages + P.unit - 1) / P.unit;
        float best = 0.f;
        for (int i = 0; i < 4; ++i) {
            if (cost.stage[i] == 0.f) continue;
            const int bm = 32 << i, bn = tn ? bm : (bm == 256 || nn || (bm == 128 && wide) ? 256 : 128);
            // (an expert's last tile is half empty)
            const int64_t rows = tn ? 2 * experts * ((d_out + bm - 1) / bm) : (experts > 1 ? n / bm + (live + 1) / 2 : (n + bm - 1) / bm);
            const int64_t blocks = rows * ((wcols + bn - 1) / bn);
            int last = 0;
            for (int want = 1; want <= 16; want *= 2) {
                const int64_t each = units > 0 ? (units + want - 1) / want : 1;
                const int split = units > 0 ? (int)((units + each - 1) / each) : 1;
                if (split == last) continue;
                last = split;
                const int64_t some = stages < each * P.unit ? stages : each * P.unit;
                float load = (float)(blocks * split) / 256.f;
                load = load < 1.f ? 1.f : (load < 8.f ? ceilf(load) : load);
                const bool join = split > 1 || (packed && bn != 256);
                const float each_tile = load > 1.f ? powf(load, .85f) : 1.f;
                const float t = cost.fixed[i] * sqrtf(load) + cost.stage[i] * (float)(split > 1 ? some : stages) * each_tile +
                                (join ? cost.join + (float)split * (float)outputs / (1000.f * cost.sums) : 0.f);
                if (best == 0.f || t < best) {
                    best = t;
                    P.bm = bm;
                    P.bn = bn;
                    P.split = split;
                    P.join = join;
                }
                if (blocks >= 512) break;          // the card is full: parts would only cost
            }
        }
        P.waves = P.bm >= 128 && P.bn == 256 ? 8 : (P.bm == 32 && wide ? 2 : 4);
    }
    P.part_bytes = P.join ? mm_al256((size_t)P.split * outputs * 4) : 0;
    return P;
}

size_t mm_workspace(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed, bool a_padded) {
    const MmPlan P = mm_plan(form, elt, n, d_in, d_out, experts, packed, a_padded);
    return P.pad_bytes + P.part_bytes;
}

bool mm_fits(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets, bool packed) {
    const MmPlan P = mm_plan(form, elt, n, d_in, d_out, experts, packed);
    const int64_t m = form == MM_TN || form == MM_NN ? d_in : d_out;
    return P.stream || mm_blocks(form, n, m, d_out, experts, offsets, 2, P) * 64 * P.waves <= MM_MAX_LANES;
}

void mm_describe(MmForm form, MmElt elt, int64_t n, int64_t d_in, int64_t d_out, int experts, bool packed, int32_t plan[6]) {
    const MmPlan P = mm_plan(form, elt, n, d_in, d_out, experts, packed);
    const int32_t v[6] = {elt == MM_BF16 || mm_wide(elt), P.stream, P.bm, P.bn, P.waves, P.split};
    for (int i = 0; i < 6; ++i) plan[i] = v[i];
}

hipError_t mm_run(const MmCall& c, void* ws, hipStream_t st) {
    StageTimer tm(c.form == MM_GATE ? ST_FFN_GATE : (c.elt == MM_BF16 ? ST_FFN_BACK : ST_FP8_GEMM), st);
    const bool packed = c.hq != nullptr, fp8 = c.elt != MM_BF16, tn = c.form == MM_TN, nn = c.form == MM_NN;
    const MmPlan P = mm_plan(c.form, c.elt, c.n, c.d_in, c.d_out, c.experts, packed, c.a_padded);
    const MmPads pads = mm_pads(c.form, c.elt, c.n, c.d_in, c.d_out, c.experts, c.a_padded);
    const int64_t ak = nn || tn ? c.d_out : c.d_in, m = nn || tn ? c.d_in : c.d_out;
    char* at = (char*)ws;
    // rows of k values, copied to a multiple of 8 where they are none
    MmPadded copies{};
    int arrays = 0;
    auto padded = [&](const void* x, int64_t rows, int64_t k, size_t bytes) -> const uint8_t* {
        if (!bytes || !x) return (const uint8_t*)x;
        const uint8_t* const out = (const uint8_t*)at;
        const int64_t pieces = rows * (mm_al8(k) / 8);
        if (pieces > 0) {
            copies.x[arrays] = x;
            copies.k[arrays] = k;
            copies.ends[arrays] = pieces + (arrays ? copies.ends[arrays - 1] : 0);
            copies.out[arrays++] = (u32x4*)at;
        }
        at += bytes;
        return out;
    };
    MmTile t{};
    hipError_t e;
    for (int i = 0; i < 2; ++i) {
        t.A[i] = padded(c.a[i], c.n, ak, pads.a);
        t.W[i] = padded(c.w[i], tn ? c.n : c.experts * c.d_out, c.d_in, pads.w);
        t.WS[i] = c.ws[i];
        t.y[i] = c.y[i];
        t.z[i] = c.z[i];
    }
    if (arrays) {
        const int64_t blocks = (copies.ends[arrays - 1] + 255) / 256;
        hipLaunchKernelGGL(k_mm_pad, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, copies, arrays);
        GQ_LAUNCH_CHECK();
    }
    t.a_row = t.a_bytes = fp8 ? fp8_bytes(ak) : 2 * mm_al8(ak);
    t.w_row = t.w_bytes = fp8 ? fp8_bytes(c.d_in) : 2 * mm_al8(c.d_in);
    t.AS = c.as;
    t.as_row = fp8_scales(ak) * (mm_bytes(c.elt) ? 1 : 4);
    t.ws_row = fp8_blocks(c.d_in);
    t.ws_rows = fp8_blocks(c.d_out);
    t.ws_k = fp8_blocks(ak);
    t.offsets = c.offsets;
    t.experts = c.experts;
    t.n = c.n;
    t.m = m;
    t.d_out = c.d_out;
    t.stages = P.stages;
    t.stages_one = nn && !fp8 ? P.stages / 2 : P.stages;
    t.unit = P.unit;
    t.y_bf16 = c.y_bf16;
    t.outs = 1;
    if (tn) {                                      // the outputs that are wanted, in front
        t.outs = (c.y[0] != nullptr) + (c.y[1] != nullptr);
        if (!c.y[0]) {
            t.y[0] = t.y[1];
            t.A[0] = t.A[1];
        }
    }
    t.hq = c.hq;
    t.hs = c.hs;
    t.hq_row = fp8_bytes(m);
    t.hs_row = fp8_scales(m);
    t.act = c.act;
    t.part = P.join ? (float*)((char*)ws + P.pad_bytes) : nullptr;
    // Large outputs that the caches would not hold until they are read, or only in place of the operands, are stored past
    // the caches' order; others, and parts that the join reads at once, as usual.  With the product that reads h in bfloat16 (gate and
    // down projection, us as usual and past): 1024 rows, 2048 -> 5632 (12 MB) 81 and 86; 2048 rows 142 and 143 (23 MB), 4096 rows 228 and
    // 232 (46 MB), 8192 rows 423 and 427 (92 MB), 16384 rows 854 and 820 (185 MB); 4096 -> 11008: 512 rows 169 and 169, 3000
    // rows 656 and 655 (66 MB), 4096 rows 829 and 826 (90 MB; the gate alone 581 and 553), 6000 rows 1280 and 1246.  With an update that
    // reads both weights' gradients: 512 rows, 2048 -> 4096 (34 MB) 51 and 52, 4096 -> 4096 (67 MB) 93 and 99, 4096 -> 8192 (134 MB) 219
    // and 211; 4096 rows, 8192 -> 8192 1062 and 1035.  Parts: 16384 rows, 1024 -> 1024 in 8 81 and 85.
    if (c.form == MM_GATE) t.past = c.y_bf16 && (size_t)c.n * m * 2 >= (size_t)64 << 20;
    if (tn) t.past = !P.join && (size_t)t.outs * c.experts * c.d_out * m * (c.y_bf16 ? 2 : 4) >= (size_t)128 << 20;
    switch (c.elt) {
        case MM_BF16: e = mm_launch_bf16(c.form, t, P, st); break;
        case MM_E8: e = mm_launch_e8(c.form, t, P, st); break;
        case MM_FS: e = mm_launch_fs(c.form, t, P, st); break;
        case MM_E8W: e = mm_launch_e8w(c.form, t, P, st); break;
        default: e = mm_launch_fsw(c.form, t, P, st); break;
    }
    if (e != hipSuccess || !P.join) return e;
    if (packed) {
        const int64_t blocks = (c.n * 16 * fp8_blocks(m) + 255) / 256;
        const auto k = mm_bytes(c.elt) ? k_mm_join_pack<false> : k_mm_join_pack<true>;
        hipLaunchKernelGGL(k, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, t.part, P.split, c.n, m, c.offsets, c.experts, c.act,
                           (u32x2*)c.hq, c.hs);
        GQ_LAUNCH_CHECK();
        return hipSuccess;
    }
    const int64_t rows = tn ? c.experts * c.d_out : c.n, each = rows * m;
    const int64_t blocks = (each + 255) / 256 / (m % 4 == 0 ? 4 : 1) + 1;                    // four outputs a lane, or one
    const auto k = c.form == MM_GATE ? k_mm_join<true> : k_mm_join<false>;
    for (int i = 0; i < t.outs; ++i) {
        hipLaunchKernelGGL(k, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, t.part + i * each, P.split, t.outs * each, rows, m,
                           tn ? nullptr : c.offsets, c.experts, t.y[i], (int)c.y_bf16, c.act, t.z[0], t.z[1]);
        GQ_LAUNCH_CHECK();
    }
    return hipSuccess;
}

}  // namespace gq
