// Tiled products of one element type on gfx950: the kernels that gq_mm.hip plans and launches, included
// by the one file of each type (gq_mm_bf16.hip, gq_mm_e8.hip, gq_mm_fs.hip, gq_mm_e8w.hip, gq_mm_fsw.hip).
#pragma once
#include "gq_mm.h"
#include "gq_mm_plan.h"
#include "gq_tile.h"

namespace gq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A stage's line of 128 bytes is 8 chunks of 16.  Operands whose contraction runs along their rows lie
// in LDS as lines of a row, chunk c of row r in place c ^ mm_swz(r), so that the 16 rows of a fragment's read
// spread over the banks.  Operands whose contraction runs over their rows ("turned": the weights of
// MM_NN, both operands of MM_TN) lie as rows of the contraction, and are turned by the reads:
// ds_read_b64_tr_b16 and _b8 hand 16 lanes a block of 4 x 16 or 8 x 16 values, lane i the i-th column.
// mm_tswz spreads the rows of such a block, and those of a half-wave's other one, over the banks.
__device__ __forceinline__ int mm_swz(int row) { return (row >> 1) & 7; }
template <int ES>
__device__ __forceinline__ int mm_tswz(int row) {
    return ES == 2 ? (4 * (row & 1)) ^ (10 * ((row >> 1) & 1)) ^ (2 * ((row >> 3) & 1))
                   : (2 * (row & 3)) ^ (9 * ((row >> 2) & 1)) ^ ((row >> 4) & 1);
}

// tile_dma.  Kernels with turned reads take it as inline assembly: the compiler
// does not see then that it writes LDS, and would otherwise have every such read wait for all copies in flight (plain
// reads it leaves alone; 4096 rows, gradient of 11008 -> 4096 in bfloat16: 869 us, 618 so).  It has no
// outputs, and the kernels count its arrival themselves as they do the builtin's.  Five wait states lie between a
// scalar written by the vector unit and its use.
template <bool TURNED>
__device__ __forceinline__ void mm_dma(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff, uint32_t soff) {
    if constexpr (TURNED) {
        const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(tile_lds_t)dst);
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :: "s"(at), "v"(voff), "s"(r), "s"(soff) : "m0", "memory");
    } else {
        tile_dma(r, (u32x4*)dst, voff, soff);
    }
}

// The first LANES lanes' copies of SIZE bytes each, the others idle: by the execution mask, in place of a branch that
// would cut the loop in two (the compiler then moves products from one side to the other).  All lanes are
// active before and after.
template <int LANES, int SIZE>
__device__ __forceinline__ void mm_dma_first(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff) {
    static_assert(LANES < 64 && (SIZE == 4 || SIZE == 16), "a part of a wave, words or four of them");
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(tile_lds_t)dst);
    uint64_t all;
    if constexpr (SIZE == 16)
        asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, exec\n\ts_mov_b64 exec, %2\n\ts_nop 1\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds\n\ts_mov_b64 exec, %0"
                     : "=&s"(all) : "s"(at), "s"((uint64_t(1) << LANES) - 1), "v"(voff), "s"(r) : "m0", "memory");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, exec\n\ts_mov_b64 exec, %2\n\ts_nop 1\n\tbuffer_load_dword %3, %4, 0 offen lds\n\ts_mov_b64 exec, %0"
                     : "=&s"(all) : "s"(at), "s"((uint64_t(1) << LANES) - 1), "v"(voff), "s"(r) : "m0", "memory");
}

// Past the caches' order.  (The empty statements keep the compiler from making one ordinary store of this one and that of
// the other branch, before or behind both.)
__device__ __forceinline__ void mm_store_past(u32x4_any v, u32x4_any* to) {
    asm volatile("" ::: "memory");
    __builtin_nontemporal_store(v, to);
    asm volatile("" ::: "memory");
}

template <int ELT, int FORM, int BM, int BN, int WM, int NW, int R>
struct MmGeo {
    static constexpr int ES = ELT == MM_BF16 ? 2 : 1, KE = 128 / ES;    // bytes of a value, values of a stage
    static constexpr bool XT = FORM == MM_TN, WT = FORM == MM_NN || FORM == MM_TN;
    static constexpr int WN = NW / WM, TM = BM / WM, TN = BN / WN;      // waves, and a wave's tile
    static constexpr int FM = TM / 16, FN = TN / 16;                    // its fragments
    static constexpr int X = BM * 8, W = BN * 8, STAGE = X + W;         // 16-byte slots
    static constexpr bool SC = ELT != MM_BF16;
    static constexpr int SB = mm_bytes(ELT) ? 4 : 16;                   // bytes of four stages' scales of a row
    static constexpr int SCB = SC ? BM * SB : 0;                        // one of three buffers of them
    static constexpr size_t IN = (size_t)R * STAGE * 16 + 3 * SCB;
    static constexpr int HC = FORM == MM_GATE ? TN / 2 : TN;            // output columns of a wave
    static constexpr int PITCH = (FORM == MM_GATE ? 2 : 1) * HC * 4 + 16;  // bytes of a row on its way out
    static constexpr size_t OUT = (size_t)NW * 16 * PITCH + (FORM == MM_GATE ? 4 * WN * BM : 0);
    static constexpr size_t BYTES = IN > OUT ? IN : OUT;
    static_assert(BYTES <= 160 * 1024, "LDS of a compute unit");
    static_assert(FN % 2 == 0 && TM % 16 == 0 && TN % 32 == 0, "fragments go in pairs");
};

// Which tile a block of MM_TN has: weight gradient z / E of expert z % E.
struct MmTurned {
    int e, which;
    int64_t t0, lo, hi;           // first row of the output, rows of the contraction
    int col;
    bool ok;
};
__device__ __forceinline__ MmTurned mm_place_turned(const MmTile& p, int bm, int ncol) {
    MmTurned r;
    const int64_t nrow = (p.d_out + bm - 1) / bm, each = nrow * ncol, total = each * p.experts * p.outs;
    const int64_t eighth = (total + 7) / 8, in = blockIdx.x >> 3, lin = (int64_t)(blockIdx.x & 7) * eighth + in;
    r.ok = in < eighth && lin < total;
    const int64_t z = lin / each, rest = lin - z * each;
    r.e = (int)(z / p.outs);
    r.which = (int)(z - (int64_t)r.e * p.outs);
    constexpr int H = 8;
    const int64_t g = rest / (H * ncol), q = rest - g * (H * ncol), left = nrow - g * H, h = left < H ? left : H;
    r.t0 = (g * H + q % h) * bm;
    r.col = (int)(q / h);
    r.lo = 0;
    r.hi = p.n;
    if (p.offsets && r.ok) tile_expert_rows(p.offsets, r.e, p.n, r.lo, r.hi);
    if (r.hi < r.lo) r.hi = r.lo;
    return r;
}

// 8 codes (words i and i + 1 of q) times the power of two that the exponent of `scale` is, as bfloat16: exact (but
// below bfloat16's smallest number, 2^-133, and over its largest)
__device__ __forceinline__ u32x4 mm_widen8(u32x4 q, int i, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    u32x4 to;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i + k], scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i + k], scale, true);
        to[2 * k] = __builtin_bit_cast(uint32_t, a);
        to[2 * k + 1] = __builtin_bit_cast(uint32_t, b);
    }
    return to;
}

// 16 codes as bfloat16, 8 and 8: exact
__device__ __forceinline__ void mm_widen(u32x4 q, u32x4& lo, u32x4& hi) {
    lo = mm_widen8(q, 0, 1.f);
    hi = mm_widen8(q, 2, 1.f);
}

__device__ __forceinline__ i32x8 mm_pair(u32x4 a, u32x4 b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// ---------------------------------------------------------------------------
// A wave holds its rows' fragments of a stage (x) and takes its columns' one after another (w): while
// the products of one column fragment run, the next is read, and the loads of a later stage go out one
// beside each product or two.  One barrier a stage, before its last part: by then every wave has read
// all of the stage, so its slot is refilled from there on, and the last part's products run while the
// next stage's rows and first columns are read.  Half of those loads go out with the last part, half with the next
// stage's first one: all at once they hold the waves up (bfloat16 gate of 4096 x 4096 -> 2048: 112 us, 108 so).
//
// The products are the 16 x 16 ones.  On random data power holds the clock down, and for the same work they take less of
// it than the 32 x 32 ones: loops of either alone reach 2.08 and 1.80 PFLOP/s in bfloat16, 4.2 and 3.8 in 8 bits
// (gate of 4096 rows, 4096 -> 2048: 104 us, 111 by 32 x 32; dx 106 and 115).
//
// Tiles of 256 x 256 have eight waves of 64 x 128, two to a SIMD.  Four of 128 x 128 read each value from LDS two
// thirds as often, but have nothing beside their waits and epilogues: 4096 rows, 8192 -> 4096 124 us, 121 by eight;
// 2048 -> 4096 packed gate 47 and 39; with float32 scales, whose sums go through the vector unit, 153 and 118.
//
// Rates of full rounds (4096 rows, 4096 columns of weights, contraction 8192 in bfloat16 and 16384 in 8 bits): gate 1.41
// PFLOP/s, dx 1.38, dW 1.36; 8-bit products with byte scales 2.8, with float32 scales 2.5, gate 2.8; with float32 sums 1.3.
// (The library's 8192 x 8192 x 8192 products: 1.60 and, with one scale, 3.2.)  Matrix cores are busy 50 to 67 % of the
// cycles at 1.6 to 2.1 GHz, clocks that power sets; LDS 17 to 27 %.
// ---------------------------------------------------------------------------
template <int ELT, int FORM, int BM, int BN, int WM, int NW, int R>
__global__ __launch_bounds__(64 * NW) void k_mm_tile(MmTile p) {
    typedef MmGeo<ELT, FORM, BM, BN, WM, NW, R> G;
    constexpr int ES = G::ES, KE = G::KE, FM = G::FM, FN = G::FN, TM = G::TM, TN = G::TN;
    constexpr bool XT = G::XT, WT = G::WT, SC = G::SC, GATE = FORM == MM_GATE;
    constexpr int BC = GATE ? BN / 2 : BN;                       // output columns of a tile
    extern __shared__ u32x4 mm_lds[];
    uint8_t* const lds = (uint8_t*)mm_lds;

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave % WM, wn = wave / WM;
    const int ncol = (int)((p.m + BC - 1) / BC);
    int e, rows, col, which = 0, stages = p.stages;
    int64_t t0, k_lo = 0, k_rows = 0;
    if constexpr (FORM == MM_TN) {
        const MmTurned at = mm_place_turned(p, BM, ncol);
        if (!at.ok) return;
        e = __builtin_amdgcn_readfirstlane(at.e);
        which = __builtin_amdgcn_readfirstlane(at.which);
        col = __builtin_amdgcn_readfirstlane(at.col);
        t0 = (int64_t)__builtin_amdgcn_readfirstlane((int)at.t0);
        rows = (int)(p.d_out - t0 < BM ? p.d_out - t0 : BM);
        k_lo = (int64_t)__builtin_amdgcn_readfirstlane((int)at.lo);
        k_rows = (int64_t)__builtin_amdgcn_readfirstlane((int)at.hi) - k_lo;
        stages = (int)((k_rows + KE - 1) / KE);
    } else {
        TilePlace at = tile_place(p, BM, ncol);
        if (!at.ok) return;
        // (the same in every lane; said so, or the descriptors built from it are looped over lanes)
        e = __builtin_amdgcn_readfirstlane(at.e);
        col = __builtin_amdgcn_readfirstlane(at.col);
        rows = __builtin_amdgcn_readfirstlane(at.rows);
        t0 = (int64_t)__builtin_amdgcn_readfirstlane((int)at.t0);              // below 2^31
    }
    const int64_t j0 = (int64_t)col * BC;

    // this split's stages
    int s_lo = 0, s_hi = stages;
    if (gridDim.y > 1) {
        const int units = (stages + p.unit - 1) / p.unit;
        const int per = (units + (int)gridDim.y - 1) / (int)gridDim.y;
        s_lo = (int)blockIdx.y * per * p.unit;
        s_hi = s_lo + per * p.unit;
        s_lo = s_lo < stages ? s_lo : stages;
        s_hi = s_hi < stages ? s_hi : stages;
    }

    // ---- what is copied into LDS: a wave's slots of both operands
    constexpr int XPW = G::X / NW, WPW = G::W / NW, XI = XPW / 64, WI = WPW / 64, LOADS = XI + WI + (SC ? 1 : 0);
    static_assert(XPW % 64 == 0 && WPW % 64 == 0, "whole copies");
    const int wcols = (int)(p.m - j0 < BC ? p.m - j0 : BC);
    uint32_t xv[XI], wv[WI];
    // bfloat16 rows end within a stage: the first of this lane's stages past the row
    constexpr bool EDGE = ELT == MM_BF16;
    int xe[EDGE && !XT ? XI : 1], we[EDGE && !WT ? WI : 1];
    auto first_past = [&](int64_t bytes, int chunk) {
        const int64_t n = (bytes - 16 * chunk + 127) / 128;
        return (int)(n < 0 ? 0 : (n < 0x7fffffff ? n : 0x7fffffff));
    };
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int slot = wave * XPW + i * 64 + lane;
        if constexpr (XT) {
            constexpr int PR = BM * ES / 16;                     // slots of a row of the contraction
            const int row = slot / PR, c = slot % PR;
            xv[i] = (uint32_t)(row * p.a_row) + 16u * (c ^ mm_tswz<ES>(row));
        } else {
            const int row = slot / 8, c = (slot % 8) ^ mm_swz(row);
            xv[i] = (uint32_t)(row * p.a_row) + 16u * c;
            if constexpr (EDGE) xe[i] = first_past(p.a_bytes, c);
        }
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int slot = wave * WPW + i * 64 + lane;
        if constexpr (WT) {
            constexpr int PR = BN * ES / 16;
            const int row = slot / PR, c = slot % PR;
            wv[i] = (uint32_t)(row * p.w_row) + 16u * (c ^ mm_tswz<ES>(row));
        } else {
            const int row = slot / 8, c = (slot % 8) ^ mm_swz(row);
            // MM_GATE: 16 rows of one weight, then the same 16 of the other
            const int from = GATE ? row / 32 * 16 + row % 16 : row;
            wv[i] = (uint32_t)(from * p.w_row) + 16u * c;
            if constexpr (EDGE) we[i] = first_past(p.w_bytes, c);
        }
    }
    const int64_t e_rows = (int64_t)e * p.d_out;
    // load i of stage s (XI + WI of them).  Past the split's last stage they read nothing and clear a
    // slot that is not read, so that the counts of loads in flight stay what they are.
    auto issue_one = [&](int s, int i) {
        u32x4* const base = mm_lds + (s % R) * G::STAGE;
        const bool on = s < s_hi;
        // MM_NN with two pairs: the stages of the first, then those of the second
        const int src = FORM == MM_NN && s >= p.stages_one ? 1 : 0, sl = FORM == MM_NN ? s - src * p.stages_one : s;
        if (i < XI) {
            u32x4* const to = base + wave * XPW + i * 64;
            if constexpr (XT) {
                const int64_t k0 = (int64_t)s * KE, left = k_rows - k0 < KE ? k_rows - k0 : KE;
                mm_dma<WT>(tile_rsrc(p.A[which] + (k_lo + k0) * p.a_row + t0 * ES, (int)left, p.a_row, on, (int)(t0 * ES)), to, xv[i], 0);
            } else {
                const __amdgpu_buffer_rsrc_t xr = tile_rsrc(p.A[src] + t0 * p.a_row, rows, p.a_row, on);
                uint32_t v = xv[i];
                if constexpr (EDGE) v = sl < xe[i] ? v : 0xC0000000u;                 // past the row: zeros
                mm_dma<WT>(xr, to, v, (uint32_t)sl * 128u);
            }
        } else {
            i -= XI;
            u32x4* const to = base + G::X + wave * WPW + i * 64;
            if constexpr (WT) {
                const int64_t k0 = (int64_t)sl * KE, all = FORM == MM_TN ? k_rows : p.d_out, left = all - k0 < KE ? all - k0 : KE;
                const uint8_t* const from = p.W[src] + ((FORM == MM_TN ? k_lo : e_rows) + k0) * p.w_row + j0 * ES;
                mm_dma<WT>(tile_rsrc(from, (int)left, p.w_row, on, (int)(j0 * ES)), to, wv[i], 0);
            } else {
                const int half = GATE ? ((wave * WPW + i * 64) / 128) & 1 : 0;       // 8 rows a copy
                const __amdgpu_buffer_rsrc_t q = tile_rsrc(p.W[half] + (e_rows + j0) * p.w_row, wcols, p.w_row, on);
                uint32_t v = wv[i];
                if constexpr (EDGE) v = s < we[i] ? v : 0xC0000000u;
                mm_dma<WT>(q, to, v, (uint32_t)s * 128u);
            }
        }
    };
    // The rows' scales: four stages' of a row at a time, a quarter of the next four's rows with each stage.
    uint8_t* const sc_lds = lds + R * G::STAGE * 16;
    constexpr int SW = SC ? (BM / 4 / NW > 0 ? BM / 4 / NW : 1) : 1;            // rows of a wave's copy
    static_assert(!SC || SW * NW * 4 == BM, "every wave copies scales");
    auto scale_copy = [&](int span, int row, bool on) {
        if constexpr (SC) {
            const __amdgpu_buffer_rsrc_t z = tile_rsrc((const uint8_t*)p.AS + t0 * p.as_row, rows, p.as_row, on);
            uint8_t* const to = sc_lds + (span % 3) * G::SCB + row * G::SB;
            const uint32_t v = (uint32_t)((row + lane) * p.as_row) + (uint32_t)(G::SB * span);
            mm_dma_first<SW, G::SB>(z, to, v);
        }
    };
    auto issue_scales = [&](int s) { scale_copy(s / 4 + 1, (s % 4) * (BM / 4) + wave * SW, s < s_hi); };
    auto issue = [&](int s) {
        issue_scales(s);
#pragma unroll
        for (int i = 0; i < XI + WI; ++i) issue_one(s, i);
    };
    if constexpr (SC) {                           // the first four stages' whole
#pragma unroll
        for (int q = 0; q < 4; ++q) scale_copy(s_lo / 4, q * (BM / 4) + wave * SW, true);
    }

    // ---- the weight's scales: one for a wave's columns and a stage, 64 stages in a register
    float wsc[2] = {1.f, 1.f};                     // (MM_E8, MM_E8W: the byte)
    const int64_t wblocks = p.ws_row, sbase = (int64_t)e * ((p.d_out + 127) / 128) * wblocks;
    auto load_weight_scales = [&](int s) {
        if constexpr (SC) {
            const int k = s + lane < p.ws_k ? s + lane : (int)p.ws_k - 1;
            const int64_t jb = GATE ? j0 / 128 : (j0 + wn * TN) / 128;
            // (columns past the last block: any scale, they are not stored)
            const int64_t at = FORM == MM_NN ? (int64_t)k * wblocks + (jb < wblocks ? jb : wblocks - 1)
                                             : (jb < p.ws_rows ? jb : p.ws_rows - 1) * wblocks + k;
#pragma unroll
            for (int h = 0; h < (GATE ? 2 : 1); ++h) {
                if constexpr (mm_bytes(ELT)) wsc[h] = __uint_as_float(((const uint8_t*)p.WS[h])[sbase + at]);
                else wsc[h] = ((const float*)p.WS[h])[sbase + at];
                asm volatile("" : "+v"(wsc[h]));   // it has arrived
            }
        }
    };
    // ---- fragments.  A lane has two chunks of its line, 4 j + g.
    constexpr int CH = 2;
    f32x4 acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int q = 0; q < FM; ++q) acc[f][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int RPC = 16 / ES;                   // values of the contraction in a chunk
    constexpr int RPR = RPC / 2;                   // and in a turned read
    constexpr int LPR = 16 / RPR;                  // lanes that read one row of it
    // where a turned operand's column fragment starts: row g of chunks, row and part of a block
    auto turned = [&](int column, int pitch) {
        const int row = g * RPC + r / LPR, byte = (r % LPR) * 8, c = column * ES / 16 + byte / 16;
        return row * pitch + 16 * (c ^ mm_tswz<ES>(row)) + byte % 16;
    };
    int lx[XT ? FM : CH], lw[WT ? FN : CH];
    if constexpr (XT) {
#pragma unroll
        for (int q = 0; q < FM; ++q) lx[q] = turned(wm * TM + 16 * q, BM * ES);
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j) lx[j] = (wm * TM + r) * 128 + 16 * ((4 * j + g) ^ mm_swz(r));
    }
    if constexpr (WT) {
#pragma unroll
        for (int f = 0; f < FN; ++f) lw[f] = turned(wn * TN + 16 * f, BN * ES);
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j) lw[j] = (wn * TN + r) * 128 + 16 * ((4 * j + g) ^ mm_swz(r));
    }
    // chunk `chunk` of a lane's: two blocks of RPR rows
    auto turned_read = [&](int at, int pitch) {
        u32x4 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x2 d;
            if constexpr (ES == 2) {
                typedef short s16x4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s16x4* ptr;
                d = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + at + h * RPR * pitch)));
            } else {
                typedef int i32x2 __attribute__((ext_vector_type(2)));
                typedef __attribute__((address_space(3))) i32x2* ptr;
                d = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((ptr)(lds + at + h * RPR * pitch)));
            }
            v[2 * h] = d[0];
            v[2 * h + 1] = d[1];
        }
        return v;
    };
    u32x4 x[FM][CH], w[2][CH];
    float sx[FM];                                  // scales of the rows (MM_E8, MM_E8W: the byte)
    auto read_x = [&](int s, int q, int j) {
        const int base = (s % R) * G::STAGE * 16;
        if constexpr (XT) x[q][j] = turned_read(base + lx[q] + j * 4 * RPC * BM * ES, BM * ES);
        else x[q][j] = *(const u32x4*)(lds + base + lx[j] + q * 16 * 128);
    };
    auto read_sx = [&](int s, int q) {
        if constexpr (SC) {
            const int at = R * G::STAGE * 16 + ((s / 4) % 3) * G::SCB + (wm * TM + 16 * q + r) * G::SB + (s % 4) * (G::SB / 4);
            if constexpr (mm_bytes(ELT)) sx[q] = __uint_as_float((uint32_t)lds[at]);
            else sx[q] = *(const float*)(lds + at);
        }
    };
    auto read_w = [&](int s, int f, u32x4 (&to)[CH], int j) {
        const int base = (s % R) * G::STAGE * 16 + G::X * 16;
        if constexpr (WT) to[j] = turned_read(base + lw[f] + j * 4 * RPC * BN * ES, BN * ES);
        else to[j] = *(const u32x4*)(lds + base + lw[j] + f * 16 * 128);
    };

    // ---- products.  MM_FS, MM_FSW: a line's sum, of its 16 x 16 products alone, times its scales is
    // added LAG products later, so that the matrix cores' result has arrived and their next products run beside.
    constexpr int LAG = 3, RING = LAG + 1, ALL = FN * FM;
    constexpr bool E8W = ELT == MM_E8W, WIDE = mm_wide(ELT), FS = ELT == MM_FS || ELT == MM_FSW;
    static_assert(!FS || ALL % RING == 0, "sums of a line need a place that is known");
    f32x4 sum[FS ? RING : 1];
    float fac[2][FS ? FM : 1];
    uint32_t wbyte = 0u;                           // MM_E8, MM_E8W: the weight's scale (MM_GATE: both, whose fragments take turns)
    u32x4 xb[WIDE ? FM : 1][2 * CH], wb[E8W ? 2 : 2 * CH];       // WIDE: fragments in bfloat16
    auto take_scales = [&](int s) {                // of stage s, before its products
        if constexpr (mm_bytes(ELT)) {
            const int at = (s - s_lo) & 63;
            wbyte = (uint32_t)__builtin_amdgcn_readlane(__float_as_int(wsc[0]), at);
            if constexpr (GATE) wbyte |= (uint32_t)__builtin_amdgcn_readlane(__float_as_int(wsc[1]), at) << 8;
        } else if constexpr (FS) {
            const int at = (s - s_lo) & 63;
#pragma unroll
            for (int h = 0; h < (GATE ? 2 : 1); ++h) {
                const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wsc[h]), at));
#pragma unroll
                for (int q = 0; q < FM; ++q) {
                    fac[h][q] = v * sx[q];
                }
            }
        }
    };
    // adds the sum of product k (none for k < 0)
    auto add_sum = [&](auto index) {
        constexpr int k = decltype(index)::value;
        if constexpr (FS && k >= 0) {
            constexpr int f = k / FM, q = k % FM, h = GATE ? f & 1 : 0;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[f][q][v] = __builtin_fmaf(sum[k % RING][v], fac[h][q], acc[f][q][v]);
        }
    };
    // products of two fragments (MM_FSW: four, one after the other); MM_E8W goes through the columns' eights first and
    // converts each once, the others through the rows
    constexpr int KS = E8W ? 2 * CH : (ELT == MM_BF16 ? CH : CH / 2);
    // MM_E8W: eight j of the columns, and with the first fragment of the rows, as the products before it run
    auto widen = [&](auto fragment, const u32x4 (&wf)[CH], auto eight) {
        constexpr int j = decltype(eight)::value;
        constexpr int up = GATE ? 8 * (decltype(fragment)::value & 1) : 0;
        wb[j % 2] = mm_widen8(wf[j / 2], 2 * (j % 2), mx_scale((wbyte >> up) & 255u));
        if constexpr (decltype(fragment)::value == 0) {
#pragma unroll
            for (int q = 0; q < FM; ++q) xb[q][j] = mm_widen8(x[q][j / 2], 2 * (j % 2), mx_scale(__float_as_uint(sx[q])));
        }
    };
    auto product = [&](auto fragment, const u32x4 (&wf)[CH], auto index) {
        constexpr int f = decltype(fragment)::value, i = decltype(index)::value, q = i % FM, j = i / FM;
        if constexpr (E8W) {
            acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wb[j % 2]), as_bf16x8(xb[q][j]), acc[f][q], 0, 0, 0);
            if constexpr (q == 0 && j + 1 < 2 * CH) widen(fragment, wf, std::integral_constant<int, j + 1>{});
        } else if constexpr (ELT == MM_BF16) {
            acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wf[j]), as_bf16x8(x[q][j]), acc[f][q], 0, 0, 0);
        } else {
            const i32x8 a = mm_pair(wf[2 * j], wf[2 * j + 1]), b = mm_pair(x[q][2 * j], x[q][2 * j + 1]);
            (void)a, (void)b;
            if constexpr (ELT == MM_E8) {
                const int sw = (int)wbyte, sr = __float_as_int(sx[q]);
                acc[f][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[f][q], 0, 0, GATE ? f & 1 : 0, sw, 0, sr);
            } else if constexpr (WIDE) {
                constexpr int k = f * FM + q;
                f32x4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2 * CH; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wb[h]), as_bf16x8(xb[q][h]), d, 0, 0, 0);
                sum[k % RING] = d;
                add_sum(std::integral_constant<int, k - LAG>{});
            } else {
                constexpr int k = f * FM + q;
                sum[k % RING] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
                add_sum(std::integral_constant<int, k - LAG>{});
            }
        }
    };

    constexpr int LOADS_ALL = XI + WI, LATE = LOADS_ALL / 2, SOON = LOADS_ALL - LATE, PR = FM * KS;
    // Column fragment f of stage s, beside its products: the next fragment's reads, of the loads l0 .. l1 - 1 of stage sl
    // one after every so many products, and with the last fragment the next stage's rows as each is done with.
    auto part = [&](auto fragment, int s, int sl, auto l0, auto l1) {
        constexpr int f = decltype(fragment)::value, L0 = decltype(l0)::value, LN = decltype(l1)::value - L0;
        constexpr bool last = f == FN - 1;
        constexpr int RP = (2 * CH + PR - 1) / PR;               // reads beside a product
        if constexpr (E8W) {
            widen(fragment, w[f % 2], std::integral_constant<int, 0>{});
        } else if constexpr (WIDE) {
            if constexpr (f == 0) {
#pragma unroll
                for (int q = 0; q < FM; ++q)
#pragma unroll
                    for (int j = 0; j < CH; ++j) mm_widen(x[q][j], xb[q][2 * j], xb[q][2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) mm_widen(w[f % 2][j], wb[2 * j], wb[2 * j + 1]);
        }
        tile_each<PR>([&](auto index) {
            constexpr int i = decltype(index)::value;
#pragma unroll
            for (int k = RP * i; k < RP * (i + 1); ++k)
                if (k < CH) read_w(last ? s + 1 : s, last ? 0 : f + 1, w[(f + 1) % 2], k);
            product(fragment, w[f % 2], index);
            if constexpr (last && E8W) {               // (its rows have been converted)
#pragma unroll
                for (int k = i * FM * CH / PR; k < (i + 1) * FM * CH / PR; ++k) read_x(s + 1, k / CH, k % CH);
            } else if constexpr (last) {               // each where its last product has been
                constexpr int q = i % FM, j = i / FM;
#pragma unroll
                for (int k = j * CH / KS; k < (j + 1) * CH / KS; ++k) read_x(s + 1, q, k);
            }
#pragma unroll
            for (int l = i * LN / PR; l < (i + 1) * LN / PR; ++l) issue_one(sl, L0 + l);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    const std::integral_constant<int, 0> zero{};
    const std::integral_constant<int, SOON> soon{};
    const std::integral_constant<int, LOADS_ALL> all{};
    if (s_lo < s_hi) {
#pragma unroll
        for (int i = 0; i < R - 1; ++i) issue(s_lo + i);
        issue_scales(s_lo + R - 1);
#pragma unroll
        for (int i = 0; i < SOON; ++i) issue_one(s_lo + R - 1, i);
        tile_wait_vmcnt<LOADS * (R - 2) + LOADS - LATE>();
        tile_barrier();
        // a wave whose rows all lie past the tile's own only copies
        const bool idle = wm * TM >= rows;
        for (int s = s_lo; idle && s < s_hi; ++s) {
#pragma unroll
            for (int i = SOON; i < LOADS_ALL; ++i) issue_one(s + R - 1, i);
            tile_wait_vmcnt<LOADS * (R - 2)>();
            tile_barrier();
            issue_scales(s + R);
#pragma unroll
            for (int i = 0; i < SOON; ++i) issue_one(s + R, i);
        }
        if (!idle) {
#pragma unroll
            for (int q = 0; q < FM; ++q) {
#pragma unroll
                for (int j = 0; j < CH; ++j) read_x(s_lo, q, j);
                read_sx(s_lo, q);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) read_w(s_lo, 0, w[0], j);
        }
        for (int s = s_lo; !idle && s < s_hi; ++s) {
            if (SC && ((s - s_lo) & 63) == 0) load_weight_scales(s);
            take_scales(s);
            // the rest of the last stage's loads go out with the first part
            part(zero, s, s + R - 1, soon, all);
            tile_each<FN - 2>([&](auto i) { part(std::integral_constant<int, decltype(i)::value + 1>{}, s, 0, zero, zero); });
            tile_wait_vmcnt<LOADS * (R - 2)>();    // stage s + 1 has landed
            tile_barrier();                        // and this one's slot has been read by every wave
            issue_scales(s + R);
            part(std::integral_constant<int, FN - 1>{}, s, s + R, zero, soon);  // past the last stage: read and not used
            // the stage's last sums, while the next one's rows are read
            tile_each<LAG>([&](auto i) { add_sum(std::integral_constant<int, ALL - LAG + decltype(i)::value>{}); });
#pragma unroll
            for (int q = 0; q < FM; ++q) read_sx(s + 1, q);
        }
    }
    tile_wait_vmcnt<0>();          // no load may land in the LDS later
    __syncthreads();

    // ---- outputs, 16 rows of a wave's tile at a time, by way of LDS of its own: in the accumulators a
    // lane's neighbours are other rows, in memory they are a row's columns.  Lane (r, g) holds row r and columns
    // 4 g .. of each fragment.
    constexpr int HC = G::HC, HF = HC / 16;                      // output columns of a wave, in sixteens
    uint8_t* const own = lds + wave * (16 * G::PITCH);
    const int64_t jw = j0 + wn * HC;
    const int cols = (int)(p.m - jw < HC ? p.m - jw : HC);       // can be negative
    const int64_t at = t0 * p.m + jw;
    if constexpr (GATE) {
        const int64_t all_rows = p.n * p.m;
        float* const z0 = p.part ? p.part + 2 * blockIdx.y * all_rows : p.z[0];
        float* const z1 = p.part ? z0 + all_rows : p.z[1];
        constexpr bool PACKS = BN == 256 && mm_wide(ELT);        // (a block of 128 columns)
        const bool packs = PACKS && p.hq && !p.part;
        float* const tops = (float*)(lds + NW * 16 * G::PITCH);   // [WN][BM]
        constexpr int LANES = HC / 8;                            // a lane takes 8 columns of a row
        // (one copy of what follows for all q: with the activations in it, one for each would not fit the
        // instruction cache; 8-bit gate of 4096 rows, 8192 -> 2048: 139 us, 114 so)
#pragma unroll 1
        for (int q = 0; q < FM; ++q) {
            tile_each<FM>([&](auto index) {
                constexpr int Q = decltype(index)::value;
                if (q == Q) {
#pragma unroll
                    for (int c = 0; c < HF; ++c) {
                        uint8_t* const to = own + r * G::PITCH + (16 * c + 4 * g) * 4;
                        *(f32x4*)to = acc[2 * c][Q];
                        *(f32x4*)(to + HC * 4) = acc[2 * c + 1][Q];
                    }
                }
            });
            const int row0 = wm * TM + 16 * q, left = rows - row0;
            // products out, whole lines at a time (past the caches' order 4 rounds of 25 stages in bfloat16 take 209 us and 214
            // so, but the backward pass that reads them next is slower by as much)
            if (z0) {
                constexpr int FOURS = HC / 4;
#pragma unroll 1
                for (int i = lane; i < 16 * FOURS; i += 64) {
                    const int row = i / FOURS, c4 = 4 * (i % FOURS), some = cols - c4;
                    if (row >= left || some <= 0) continue;
                    const uint8_t* const from = own + row * G::PITCH + c4 * 4;
                    const f32x4 a = *(const f32x4*)from, b = *(const f32x4*)(from + HC * 4);
                    const int64_t to = at + (int64_t)(row0 + row) * p.m + c4;
                    if (some >= 4) {
                        *(f32x4_any*)(z0 + to) = a;
                        *(f32x4_any*)(z1 + to) = b;
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            if (k < some) {
                                z0[to + k] = a[k];
                                z1[to + k] = b[k];
                            }
                    }
                }
                if (p.part) continue;
            }
#pragma unroll 1
            for (int i = lane; i < 16 * LANES; i += 64) {         // h out or back in its place
                const int row = i / LANES, c8 = 8 * (i % LANES), some = cols - c8;
                uint8_t* const from = own + row * G::PITCH + c8 * 4;
                f32x4 a[2], b[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    a[k] = *(const f32x4*)(from + 16 * k);
                    b[k] = *(const f32x4*)(from + HC * 4 + 16 * k);
                }
                const bool stored = row < left && some > 0;
                const int64_t to = at + (int64_t)(row0 + row) * p.m + c8;
                auto values = [&](float* y, const f32x4 (&x)[2]) {
                    if (some >= 8) {
                        *(f32x4_any*)(y + to) = x[0];
                        *(f32x4_any*)(y + to + 4) = x[1];
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k < some) y[to + k] = x[k / 4][k % 4];
                    }
                };
                f32x4 h[2];
                if (p.act == ACT_SILU) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k / 4][k % 4] = act_of<false>(a[k / 4][k % 4], ACT_SILU, nullptr) * b[k / 4][k % 4];
                } else if (p.act == ACT_GELU) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k / 4][k % 4] = act_of<false>(a[k / 4][k % 4], ACT_GELU, nullptr) * b[k / 4][k % 4];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k / 4][k % 4] = act_of<false>(a[k / 4][k % 4], ACT_GELU_TANH, nullptr) * b[k / 4][k % 4];
                }
                if (packs) {
                    // a row's largest magnitude over this wave's columns
                    uint32_t top = 0u;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t v = __float_as_uint(h[k / 4][k % 4]) & 0x7fffffffu;
                        top = top > v ? top : v;
                    }
#pragma unroll
                    for (int o = 1; o < LANES; o <<= 1) {
                        const uint32_t v = (uint32_t)__shfl_xor((int)top, o, 64);
                        top = top > v ? top : v;
                    }
                    if (i % LANES == 0) tops[wn * BM + row0 + row] = __uint_as_float(top);
                    *(f32x4*)from = h[0];
                    *(f32x4*)(from + 16) = h[1];
                    continue;
                }
                if (!stored) continue;
                if (!p.y_bf16) {
                    values((float*)p.y[0], h);
                } else if (some >= 8) {
                    const u32x4_any v = u32x4{pack_bf16x2(h[0][0], h[0][1]), pack_bf16x2(h[0][2], h[0][3]),
                                              pack_bf16x2(h[1][0], h[1][1]), pack_bf16x2(h[1][2], h[1][3])};
                    u32x4_any* const at16 = (u32x4_any*)((uint16_t*)p.y[0] + to);
                    if (p.past) mm_store_past(v, at16);
                    else *at16 = v;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < some) ((uint16_t*)p.y[0])[to + k] = (uint16_t)f32_to_bf16_bits(h[k / 4][k % 4]);
                }
            }
            if constexpr (PACKS) {
                if (!packs) continue;
                __syncthreads();                                 // all waves of a row
#pragma unroll 1
                for (int i = lane; i < 16 * LANES; i += 64) {
                    const int row = i / LANES, c8 = 8 * (i % LANES);
                    uint32_t top = 0u;
#pragma unroll
                    for (int n = 0; n < G::WN; ++n) {
                        const uint32_t a = __float_as_uint(tops[n * BM + row0 + row]);
                        top = top > a ? top : a;
                    }
                    const uint32_t s = fp8_scale_byte(top);
                    const float f = fp8_scale_inverse(s);
                    const uint8_t* const from = own + row * G::PITCH + c8 * 4;
                    const f32x4 u = *(const f32x4*)from, v = *(const f32x4*)(from + 16);
                    const u32x2 codes{fp8_pack4(u[0] * f, u[1] * f, u[2] * f, u[3] * f), fp8_pack4(v[0] * f, v[1] * f, v[2] * f, v[3] * f)};
                    if (row >= left) continue;
                    *(u32x2*)(p.hq + (t0 + row0 + row) * p.hq_row + jw + c8) = s == 255u ? u32x2{0u, 0u} : codes;
                    if (wn == 0 && c8 == 0) {
                        // with the last block, what fills the row's scales up: 1
                        const int64_t at0 = (t0 + row0 + row) * p.hs_row + col, n = col == ncol - 1 ? p.hs_row - col : 1;
                        for (int64_t k = 0; k < n; ++k) {
                            const uint32_t byte = k == 0 ? s : 127u;
                            if constexpr (mm_bytes(ELT)) ((uint8_t*)p.hs)[at0 + k] = (uint8_t)byte;
                            else ((float*)p.hs)[at0 + k] = fp8_scale_value(byte);
                        }
                    }
                }
            }
        }
    } else {
        int64_t from = at;
        if constexpr (FORM == MM_TN) from += ((p.part ? (int64_t)which * p.experts : 0) + e) * p.d_out * p.m;
        const int64_t planes = FORM == MM_TN ? (int64_t)p.outs * p.experts * p.d_out * p.m : p.n * p.m;
        const int wide = p.part || !p.y_bf16 ? 4 : 2, pitch = HC * wide + 16;
        uint8_t* const out = p.part ? (uint8_t*)(p.part + blockIdx.y * planes + from) : (uint8_t*)p.y[which] + from * wide;
#pragma unroll 1
        for (int q = 0; q < FM; ++q) {
            tile_each<FM>([&](auto index) {
                constexpr int Q = decltype(index)::value;
                if (q == Q) {
#pragma unroll
                    for (int c = 0; c < HF; ++c) {
                        const f32x4 v = acc[c][Q];
                        uint8_t* const to = own + r * pitch + (16 * c + 4 * g) * wide;
                        if (wide == 4) *(f32x4*)to = v;
                        else *(u32x2*)to = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    }
                }
            });
            const int row0 = wm * TM + 16 * q, left = rows - row0;
            const int lanes = HC * wide / 16;                    // of a row: a power of two
            auto store = [&](auto ends) {                        // ends: rows may end inside 16 bytes
                for (int i = lane; i < 16 * lanes; i += 64) {
                    const int row = i / lanes, at16 = 16 * (i - row * lanes), some = cols * wide - at16;
                    const u32x4 v = *(const u32x4*)(own + row * pitch + at16);
                    if (row >= left || some <= 0) continue;
                    uint8_t* const to = out + (int64_t)(row0 + row) * p.m * wide + at16;
                    if (!decltype(ends)::value || some >= 16) {
                        if (FORM == MM_TN && p.past) mm_store_past(v, (u32x4_any*)to);
                        else *(u32x4_any*)to = v;
                    } else {
                        for (int b = 0; b < some; b += wide) {
                            if (wide == 4) *(uint32_t*)(to + b) = v[b / 4];
                            else *(uint16_t*)(to + b) = (uint16_t)(v[b / 4] >> (8 * (b & 2)));
                        }
                    }
                }
            };
            if (cols * wide % 16 == 0) store(std::false_type{});
            else store(std::true_type{});
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows: the weight is streamed once, each wave on its own, without a barrier before the end.  A block
// takes 16 MT rows of the weight (MM_GATE: 16 of each) and 16 rows of activations at a time; its
// waves share out the contraction and their sums are added in the waves' order.  A wave copies a line of each of
// its weight rows into LDS of its own, one line ahead.  Lane (r, b) holds chunks b and 4 + b of a line of
// weight row r, and the same of row r of the activations.  (8-bit gate of 16 rows, 4096 -> 11008: 21.7 us at 4.2 TB/s;
// 25.7 by two lines at a time, of which fewer waves fit a compute unit; 24.0 and 25.4 with two and three lines ahead.)
//
// An expert's block takes its first MM_FIRST groups of 16 rows, and what experts have beyond those is spread over
// blocks of its own that find their groups from the offsets: the plan knows the mean of the experts' rows alone.
// ---------------------------------------------------------------------------
template <int ELT, bool GATE, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mm_stream(MmTile p) {
    constexpr int LINE = 16 * MT * 8, LOADS = LINE / 64;        // slots of a line of each row, copies
    constexpr bool SC = ELT != MM_BF16;
    static_assert(!GATE || MT == 2, "16 rows of each weight");
    extern __shared__ u32x4 mm_lds[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, b = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    u32x4* const ring = mm_lds + wave * 2 * LINE;
    auto sums = [&](int w, int t) { return (float*)(mm_lds + w * 2 * LINE) + 256 * t; };    // over the rings at the end
    constexpr int BC = GATE ? 16 : 16 * MT;
    const int64_t j0 = (int64_t)blockIdx.x * BC;
    const int lines = (int)((p.w_bytes + 127) / 128);
    const int shares = WAVES * (int)gridDim.z, per = (lines + shares - 1) / shares;
    const int c0 = ((int)blockIdx.z * WAVES + wave) * per;
    const int c1 = c0 + per < lines ? c0 + per : lines;

    const int wrows = (int)(p.m - j0 < BC ? p.m - j0 : BC);
    uint32_t wv[LOADS];
    int wc[LOADS];                                 // the chunk's byte within a line
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int slot = i * 64 + lane, row = slot / 8;
        wc[i] = 16 * ((slot % 8) ^ mm_swz(row));
        wv[i] = (uint32_t)((GATE ? row % 16 : row) * p.w_row) + wc[i];
    }
    const int beyond = (int)blockIdx.y - p.experts, step = (int)gridDim.y - p.experts;
    int64_t lo = 0, hi = p.n;
    if (p.offsets && beyond < 0) tile_expert_rows(p.offsets, blockIdx.y, p.n, lo, hi);
    for (int turn = 0;; ++turn) {
        TilePlace place;
        if (beyond < 0) {
            place.e = blockIdx.y;
            place.t0 = lo + 16 * turn;
            place.rows = (int)(hi - place.t0 < 16 ? hi - place.t0 : 16);
            place.ok = turn < MM_FIRST && place.rows > 0;
        } else {
            tile_of_row(p, 16, beyond + turn * step, place, MM_FIRST);
        }
        if (!place.ok) return;
        if (turn > 0) __syncthreads();             // the sums of the rows before have been read
        const int rows = place.rows;
        const int64_t t0 = place.t0, row0 = (int64_t)place.e * p.d_out + j0;
        auto copy = [&](int c) {                   // past the last line: clears, reads nothing
            u32x4* const to = ring + (c & 1) * LINE;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const __amdgpu_buffer_rsrc_t wr = tile_rsrc(p.W[GATE ? i / (LOADS / 2) : 0] + row0 * p.w_row, wrows, p.w_row, c < c1);
                const int64_t byte = (int64_t)c * 128 + wc[i];
                tile_dma(wr, to + 64 * i, byte < p.w_bytes ? wv[i] : 0xC0000000u, (uint32_t)c * 128u);
            }
        };
        const int64_t xrow = t0 + (r < rows ? r : rows - 1);
        const uint8_t* const xp = p.A[0] + xrow * p.a_row;
        const int64_t sbase = ((int64_t)place.e * p.ws_rows + j0 / 128) * p.ws_row;
        f32x4 acc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (c0 < c1) copy(c0);
        for (int c = c0; c < c1; ++c) {
            // this line's activations and scales, then the next line's copies: once those alone are in
            // flight, both this line's copies and its activations have arrived
            u32x4 x[2];
            uint32_t xs, ws[GATE ? 2 : 1];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t byte = 128 * (int64_t)c + 64 * j + 16 * b;
                const u32x4 v = *(const u32x4*)(xp + (byte < p.a_bytes ? byte : 0));
                x[j] = byte < p.a_bytes ? v : u32x4{0u, 0u, 0u, 0u};
            }
            if constexpr (SC) {
                const uint8_t* const s = (const uint8_t*)p.AS + xrow * p.as_row;
                xs = mm_bytes(ELT) ? (uint32_t)s[c] : ((const uint32_t*)s)[c];
#pragma unroll
                for (int h = 0; h < (GATE ? 2 : 1); ++h)
                    ws[h] = mm_bytes(ELT) ? (uint32_t)((const uint8_t*)p.WS[h])[sbase + c] : ((const uint32_t*)p.WS[h])[sbase + c];
            }
            __builtin_amdgcn_sched_barrier(0);
            copy(c + 1);
            tile_wait_vmcnt<LOADS>();
            __builtin_amdgcn_sched_barrier(0);
            const uint8_t* const at = (const uint8_t*)(ring + (c & 1) * LINE);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                u32x4 w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j] = *(const u32x4*)(at + 16 * ((16 * t + r) * 8 + ((4 * j + b) ^ mm_swz(r))));
                if constexpr (ELT == MM_BF16) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w[j]), as_bf16x8(x[j]), acc[t], 0, 0, 0);
                } else if constexpr (ELT == MM_E8) {
                    acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mm_pair(w[0], w[1]), mm_pair(x[0], x[1]), acc[t], 0, 0, 0, (int)ws[GATE ? t : 0], 0, (int)xs);
                } else {
                    f32x4 d{0.f, 0.f, 0.f, 0.f};
                    if constexpr (mm_wide(ELT)) {
                        u32x4 a[4], v[4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            mm_widen(w[j], a[2 * j], a[2 * j + 1]);
                            mm_widen(x[j], v[2 * j], v[2 * j + 1]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[j]), as_bf16x8(v[j]), d, 0, 0, 0);
                    } else {
                        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mm_pair(w[0], w[1]), mm_pair(x[0], x[1]), d, 0, 0, 0, 127, 0, 127);
                    }
                    const uint32_t wk = ws[GATE ? t : 0];
                    if constexpr (mm_bytes(ELT)) {
                        // by the sum of the exponents: their powers' product need not be a float32 number where
                        // the result is one (2^100 by 2^100 would make NaN of a zero sum)
                        const int by = (int)(wk + xs) - 254;
                        const bool nan = wk == 255u || xs == 255u;
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[t][v] += nan ? __uint_as_float(0x7fc00000u) : __builtin_amdgcn_ldexpf(d[v], by);
                    } else {
                        const float by = __uint_as_float(wk) * __uint_as_float(xs);
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(d[v], by, acc[t][v]);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            tile_wait_lds();                       // read, before its half of the ring is copied into
        }
        tile_wait_vmcnt<0>();                      // no copy into the ring may land later
#pragma unroll
        for (int t = 0; t < MT; ++t) *(f32x4*)(sums(wave, t) + 4 * lane) = acc[t];
        __syncthreads();
        // output (row i / BC, column i % BC) is in lane 16 (column / 4) + row, element column % 4
        for (int i = tid; i < 16 * BC; i += 64 * WAVES) {
            const int row = i / BC, c = i - row * BC, t = c >> 4, from = 4 * (16 * ((c & 15) >> 2) + row) + (c & 3);
            if (row >= rows || j0 + c >= p.m) continue;
            float v[GATE ? 2 : 1];
#pragma unroll
            for (int h = 0; h < (GATE ? 2 : 1); ++h) {
                v[h] = sums(0, GATE ? h : t)[from];
#pragma unroll
                for (int w = 1; w < WAVES; ++w) v[h] += sums(w, GATE ? h : t)[from];
            }
            const int64_t all = p.n * p.m, at = (t0 + row) * p.m + j0 + c;
            float y = v[0];
            if constexpr (GATE) {
                if (p.part) {
                    p.part[2 * (int64_t)blockIdx.z * all + at] = v[0];
                    p.part[(2 * (int64_t)blockIdx.z + 1) * all + at] = v[1];
                    continue;
                }
                if (p.z[0]) {
                    p.z[0][at] = v[0];
                    p.z[1][at] = v[1];
                }
                y = act_of<false>(v[0], p.act, nullptr) * v[1];
            } else if (p.part) {
                p.part[(int64_t)blockIdx.z * all + at] = y;
                continue;
            }
            if (p.y_bf16) ((uint16_t*)p.y[0])[at] = (uint16_t)f32_to_bf16_bits(y);
            else ((float*)p.y[0])[at] = y;
        }
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int ELT, int FORM, int BM, int BN, int WM, int NW, int R>
static hipError_t mm_launch_tile(const MmTile& t, const MmPlan& P, hipStream_t st) {
    const auto k = k_mm_tile<ELT, FORM, BM, BN, WM, NW, R>;
    constexpr size_t lds = MmGeo<ELT, FORM, BM, BN, WM, NW, R>::BYTES;
    if (P.bm != BM || P.bn != BN || P.waves != NW) return hipErrorInvalidValue;      // (the plan's are these)
    const hipError_t e = ensure_dynamic_lds((const void*)k, lds);
    if (e != hipSuccess) return e;
    const int64_t grid = mm_blocks((MmForm)FORM, t.n, t.m, t.d_out, t.experts, t.offsets != nullptr, t.outs, P);
    if (grid * (64 * NW) > MM_MAX_LANES) return hipErrorInvalidValue;                // (refused before)
    hipLaunchKernelGGL(k, dim3((unsigned)grid, (unsigned)P.split), dim3(64 * NW), lds, st, t);
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

template <int ELT, bool GATE, int MT, int WAVES>
static hipError_t mm_launch_stream(const MmTile& t, const MmPlan& P, hipStream_t st) {
    const auto k = k_mm_stream<ELT, GATE, MT, WAVES>;
    const size_t lds = (size_t)WAVES * 2 * 16 * MT * 8 * 16;
    const hipError_t e = ensure_dynamic_lds((const void*)k, lds);
    if (e != hipSuccess) return e;
    // a block for each expert, and for the groups beyond its own those of a compute unit each
    const int64_t bc = GATE ? 16 : 16 * MT, cols = (t.m + bc - 1) / bc, far = (t.n + 15) / 16 - MM_FIRST, room = 256 / (cols * P.split);
    const int64_t more = !t.offsets || far < 1 ? 0 : (room < 1 ? 1 : (room < far ? room : far));
    hipLaunchKernelGGL(k, dim3((unsigned)cols, (unsigned)(t.experts + more), (unsigned)P.split), dim3(64 * WAVES), lds, st, t);
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

// NT and GATE
template <int ELT, int FORM>
static hipError_t mm_launch_rows(const MmTile& t, const MmPlan& P, hipStream_t st) {
    constexpr bool GATE = FORM == MM_GATE, WIDE = mm_wide(ELT);
    if (P.stream) {
        if constexpr (GATE) return P.waves == 8 ? mm_launch_stream<ELT, true, 2, 8>(t, P, st) : mm_launch_stream<ELT, true, 2, 4>(t, P, st);
        else if (P.bn == 32) return P.waves == 8 ? mm_launch_stream<ELT, false, 2, 8>(t, P, st) : mm_launch_stream<ELT, false, 2, 4>(t, P, st);
        else return P.waves == 8 ? mm_launch_stream<ELT, false, 1, 8>(t, P, st) : mm_launch_stream<ELT, false, 1, 4>(t, P, st);
    }
    if constexpr (WIDE) {
        if (P.bm == 128) return mm_launch_tile<ELT, FORM, 128, 256, 2, 8, 3>(t, P, st);
    } else {
        if (P.bm == 256) return mm_launch_tile<ELT, FORM, 256, 256, 4, 8, 2>(t, P, st);
        if (P.bm == 128) return mm_launch_tile<ELT, FORM, 128, 128, 2, 4, 2>(t, P, st);
    }
    if (P.bm == 64) return mm_launch_tile<ELT, FORM, 64, 128, 2, 4, 3>(t, P, st);
    return mm_launch_tile<ELT, FORM, 32, 128, 1, WIDE ? 2 : 4, 3>(t, P, st);
}

template <int ELT>
static hipError_t mm_launch_back(const MmTile& t, const MmPlan& P, hipStream_t st) {
    if constexpr (!mm_wide(ELT)) {
        if (P.bm == 256) return mm_launch_tile<ELT, MM_NN, 256, 256, 4, 8, 2>(t, P, st);
    }
    if (P.bm == 128) return mm_launch_tile<ELT, MM_NN, 128, 256, 2, 8, mm_wide(ELT) ? 3 : 2>(t, P, st);
    return mm_launch_tile<ELT, MM_NN, 64, 256, 2, 4, 3>(t, P, st);
}

}  // namespace gq
