// Products with MXFP4 weights on gfx950.
//
//   MX_GEMM     y[t][j]  = sum_i x[t][i] w[j][i]     x bfloat16, or float32 in three planes
//   MX_GEMM_MX  the same, x in MXFP4 too
//   MX_GEMM_DX  dx[t][i] = sum_j g[t][j] w[j][i]     g as x
//
// w = 2^(s - 127) c with c of two significant bits is exact in bfloat16 (down to its subnormal
// range, which the matrix cores keep), so the first and last are bfloat16 products of weights
// converted in registers, one instruction for two values; the second is the matrix cores' own
// scaled product.  All sums are float32; every order of summation depends on sizes alone.
//
// Three ways, chosen by mx_plan:
//   k_mx_tile    tiles of activations' rows by output columns, both operands copied by
//                asynchronous loads into a ring of LDS stages.  Bound by the matrix cores for
//                many rows, by the weight's bytes for few.
//   k_mx_stream  up to 16 rows of a small weight: waves that stream it each on its own.
//   k_mx_join    the sum of a contraction split over blocks, where tiles are too few.
// Several weights ("experts") are tiles of one launch; their row counts stay on the device.
//
// MI355X, calls among others of their kind; large ones vary from card to card by their clock:
//   4096 rows, 11008 -> 4096, bfloat16      282 to 295 us   1.25 to 1.31 PFLOP/s (the library's
//                                           bfloat16 matrix product reaches 1.20 to 1.33)
//   8192 rows, 28672 -> 8192, both MXFP4    840 to 885 us   4.3 to 4.6 PFLOP/s (the rows packed
//                                           before; a loop of the instruction alone: 7.3)
//   gradient, 4096 rows, 11008 -> 4096      307 to 320 us   1.15 to 1.20 PFLOP/s
//   1 row, 4096 -> 4096                     9 us, 5.1 of them on the GPU (9 MB)
//   8 rows, 28672 -> 8192, both MXFP4       27 to 29 us on the GPU, 4.3 to 4.6 TB/s (a large copy: 5.0)
//   96 rows over 64 experts, 2048 -> 1408   16 us           4.4 TB/s
#include "gq_mx.h"
#include "gq_tile.h"

namespace gq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Staged activations.  Float32 rows, and bfloat16 rows of no multiple of 8, are first written
// as rows of bfloat16 pieces of 64 values, P pieces (planes) for each 64 values of the row,
// zero past its end: value i of plane p is element (i / 64 * P + p) * 64 + i % 64.  The
// three planes of a float32 are its bits cut after 8, 16 and 24 significant ones (each
// difference is exact), so their sum is the value; a NaN or infinity is in the first alone.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(256) void k_mx_stage(const void* __restrict__ x, int64_t n, int64_t k,
                                                 int64_t pieces, uint16_t* __restrict__ out) {
    constexpr int P = BF16 ? 1 : 3;
    // a lane takes 8 values; 8 lanes a piece
    const int64_t total = n * pieces * 8;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t piece = t >> 3, r = mx_div(piece, pieces);
        const int64_t i = (piece - r * pieces) * 64 + (t & 7) * 8;
        u32x4* o = (u32x4*)(out + piece * P * 64 + (t & 7) * 8);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < k) mx_load8<BF16>(x, r * k, i, k, v);
        if constexpr (BF16) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xffff0000u);
            o[0] = w;
        } else {
            uint32_t w[3][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __float_as_uint(v[e]);
                uint32_t h = b & 0xffff0000u;
                float rest = 0.f;
                if ((b & 0x7f800000u) != 0x7f800000u) rest = v[e] - __uint_as_float(h);
                else if (b & 0x007fffffu) h |= 0x00400000u;            // a NaN stays one
                const uint32_t m = __float_as_uint(rest) & 0xffff0000u;
                w[0][e] = h >> 16;
                w[1][e] = m >> 16;
                w[2][e] = __float_as_uint(rest - __uint_as_float(m)) >> 16;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q)
                o[8 * q] = u32x4{w[q][0] | (w[q][1] << 16), w[q][2] | (w[q][3] << 16),
                                 w[q][4] | (w[q][5] << 16), w[q][6] | (w[q][7] << 16)};
        }
    }
}

// ---------------------------------------------------------------------------
// The tiled product.
//
// Tile and wave.  A wave's products need (rows + columns) fragments from LDS for rows x columns
// products, so waves are as large as the accumulators allow: 256 x 256 tiles of 4 waves of
// 128 x 128 (MX_GEMM_MX, 256 accumulator registers) or 8 waves of 64 x 128 (two to a SIMD; the
// bfloat16 products take four times the cycles for the same LDS bytes, and two waves hide each
// other's waits: 712 -> 336 us when they came).  A stage is 64 values of the contraction for the
// bfloat16 products (a 128-byte line of each row of x) and 256 for the fp4 one (a line of codes;
// with 128 the half lines were fetched twice: 1176 -> 1087 us).
//
// Loop.  A stage is used in parts; while a part's products run, the next part's fragments are
// read, and the loads of a later stage go out one beside each product or two: issued together
// they hold the wave up for longer than the part lasts (1031 -> 986 us).  One barrier a stage:
// after it the stage's slot is refilled.  Loads past the end read nothing, so the waits count
// the same number of loads throughout.
//
// Scales.  They stay where the caller has them, a row's bytes in a row: 16 bytes of each row are
// fetched at a time (512 values), each stage bringing its share of the next such span, into one
// of three buffers.  The fp4 products take a row's eight scales of a stage by one read and select
// bytes in the instruction (1011 -> 940 us against a read for each).
//
// Gradient.  The contraction runs over the weight's rows, but its codes lie along the columns: a
// lane reads 8 columns (4 bytes) of 8 rows, converts pairs along the columns and exchanges halves
// of two rows' words, which gives 8 fragments of 8 rows each.  Conversions and exchanges are one
// instruction each a product; with the addresses three vector instructions stand beside each product,
// 38 per cent of a prompt's cycles next to the matrix cores' 49, and the waves wait for a quarter.
//
// Outputs leave by way of LDS as whole lines; stored from the accumulators, each store touched 32
// rows (fp4 prompt 1006 -> 918 us, 32 experts 155 -> 128 us).
//
// The large tiles of a prompt run at 1.6 to 1.75 GHz (fp4) and 1.8 to 1.87 GHz (bfloat16) of 2.4, with
// the matrix cores busy 57 to 63 and 63 to 66 per cent of the cycles.  Power alone does not bound
// them: loops of the instructions alone keep the matrix cores busy throughout at 1.75 and 2.0 GHz.  Nor
// does LDS (20 and 34 per cent).  The waves wait 18 to 20 and 26 per cent of their cycles for loads, LDS
// and the barrier; which of these leaves the matrix cores idle has not been separated.
// ---------------------------------------------------------------------------
struct MxTile {
    const uint8_t* A;             // rows of the activations (bfloat16, or codes)
    int64_t a_row;                // bytes from one row to the next
    int64_t a_bytes;              // bytes of a row that the product reads (zeros follow)
    const uint8_t* AS;            // scales of the codes
    const uint8_t *Q, *S;
    int64_t qb, sb;               // bytes of a weight row's codes and scales
    const int64_t* offsets;
    int experts;
    int64_t n, m, d_out;          // rows, output columns, rows of one weight
    int stages;                   // stages of the whole contraction
    int kpad;                     // its length padded to whole groups (MX_GEMM, MX_GEMM_MX)
    int unit;                     // a split's range is a multiple of this many stages
    void* y;
    int y_bf16;
    float* part;                  // partial sums [split][n][m], or null
};

// Geometry of a stage in 16-byte LDS slots.  KS (MX_GEMM): pieces of 64 values a stage.  With
// one, the planes of float32 activations are stages of their own (and the weight is read for
// each); with more, a stage holds them all.
template <int MODE, int P, int BM, int BN, int KS>
struct MxGeo {
    // 128 x 128 tiles: three, so that a compute unit holds two blocks (2048 rows 4096 -> 4096: 69
    // us, 81 with four; 6000 rows over 64 experts 2048 -> 1408: 68 and 94; two: 69 and 70, but
    // 1024 rows 11008 -> 4096 121 and 102)
    static constexpr int RING = MODE == MX_GEMM_MX ? (BM >= 128 ? 2 : 3) : (KS > 1 ? 2 : (MODE == MX_GEMM_DX && BM == 64 ? 4 : 3));
    static constexpr int PS = KS > 1 ? P : 1;                      // planes within a stage
    static constexpr int PA = KS > 1 ? 1 : P;                      // stages for one piece of the weight
    static constexpr int XSPR = MODE == MX_GEMM ? 8 * KS * PS : 8; // slots a row of activations
    static constexpr int WROWS = MODE == MX_GEMM_DX ? 64 : BN;
    static constexpr int WSPR = MODE == MX_GEMM ? 2 * KS : (MODE == MX_GEMM_MX ? 8 : BN / 32);
    static constexpr int X = BM * XSPR, W = WROWS * WSPR;
    static constexpr int SRING = MODE == MX_GEMM_DX ? 64 : 0;      // scales that travel in the ring
    static constexpr int STAGE = X + W + SRING;
    // stages that one 16-byte piece of a row's scales serves, and its three buffers
    static constexpr int SPAN = MODE == MX_GEMM ? 8 / KS : 2;
    static constexpr int SROWS = MODE == MX_GEMM_DX ? 0 : (MODE == MX_GEMM ? BN : BN + BM);
    static constexpr int PARTS = MODE == MX_GEMM ? 2 * KS * PS : (MODE == MX_GEMM_MX ? 4 : 2);
    static constexpr size_t BYTES = (size_t)(RING * STAGE + 3 * SROWS) * 16;
    // a row's chunks are moved about so that the 16 rows of a fragment read spread over the banks
    static __device__ __forceinline__ int xswz(int row) { return KS > 1 ? row & 15 : (row >> 1) & 7; }
    static __device__ __forceinline__ int wswz(int row) {          // (of MX_GEMM)
        return KS == 4 ? (row >> 1) & 7 : (KS == 2 ? (row >> 2) & 3 : (row >> 3) & 1);
    }
};

// The fragments of a part of a stage, and an accumulator.
template <int MODE, int FM, int FN> struct MxHalf;
template <int FM, int FN> struct MxHalf<MX_GEMM, FM, FN> {
    typedef f32x16 Acc;
    static constexpr int T = 32, V = 16, STEPS = 2 * FM + FN, PRODUCTS = 2 * FM * FN;
    u32x4 x[FM][2];
    u32x2 w[FN];
    uint32_t ws[FN];
};
template <int FM, int FN> struct MxHalf<MX_GEMM_MX, FM, FN> {
    typedef f32x16 Acc;
    static constexpr int T = 32, V = 16, STEPS = FM + FN, PRODUCTS = FM * FN;
    u32x4 x[FM], w[FN];
};
template <int FM, int FN> struct MxHalf<MX_GEMM_DX, FM, FN> {
    typedef f32x4 Acc;
    static constexpr int T = 16, V = 4, STEPS = FM + 8, PRODUCTS = FM * FN;
    u32x4 x[FM];
    uint32_t w[8], ws[8];
};

template <int MODE, int P, int BM, int BN, int WM, int NW, int KS>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(1, BM == 256 && NW == 4 ? 1 : 8))) void k_mx_tile(MxTile p) {
    typedef MxGeo<MODE, P, BM, BN, KS> G;
    constexpr int WN = NW / WM, TM = BM / WM, TN = BN / WN;
    constexpr int T = MODE == MX_GEMM_DX ? 16 : 32, FM = TM / T, FN = TN / T;
    constexpr int R = G::RING, SPAN = G::SPAN, PA = G::PA;
    static_assert(MODE != MX_GEMM_DX || (TN == 128 && BN == 256), "a wave of the gradient takes 128 columns");
    extern __shared__ u32x4 mx_lds[];
    u32x4* const sc_lds = mx_lds + R * G::STAGE;

    TilePlace at = tile_place(p, BM, (int)((p.m + BN - 1) / BN));
    if (!at.ok) return;
    // (the same in every lane; said so, or the descriptors built from it are looped over lanes)
    at.e = __builtin_amdgcn_readfirstlane(at.e);
    at.col = __builtin_amdgcn_readfirstlane(at.col);
    at.rows = __builtin_amdgcn_readfirstlane(at.rows);
    at.t0 = (int64_t)__builtin_amdgcn_readfirstlane((int)at.t0);            // below 2^31
    const int tid = threadIdx.x, lane = tid & 63, r = lane & (T - 1), g = lane / T;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int64_t j0 = (int64_t)at.col * BN;

    // this split's stages
    int s_lo = 0, s_hi = p.stages;
    if (gridDim.y > 1) {
        const int units = (p.stages + p.unit - 1) / p.unit;
        const int per = (units + (int)gridDim.y - 1) / (int)gridDim.y;
        s_lo = (int)blockIdx.y * per * p.unit;
        s_hi = s_lo + per * p.unit;
        s_lo = s_lo < p.stages ? s_lo : p.stages;
        s_hi = s_hi < p.stages ? s_hi : p.stages;
    }

    // ---- sources
    const __amdgpu_buffer_rsrc_t xr = tile_rsrc(p.A + at.t0 * p.a_row, at.rows, p.a_row);
    const uint8_t* const Qe = p.Q + (int64_t)at.e * p.d_out * p.qb;
    const uint8_t* const Se = p.S + (int64_t)at.e * p.d_out * p.sb;
    const int wrows = (int)(p.m - j0 < BN ? p.m - j0 : BN);
    const __amdgpu_buffer_rsrc_t sr = tile_rsrc(Se + j0 * p.sb, wrows, p.sb);
    const __amdgpu_buffer_rsrc_t xsr =
        MODE == MX_GEMM_MX ? tile_rsrc(p.AS + at.t0 * p.sb, at.rows, p.sb) : sr;

    constexpr int XPW = G::X / NW, WPW = G::W / NW;          // slots a wave copies
    constexpr int XI = (XPW + 63) / 64, WI = (WPW + 63) / 64;
    constexpr int LOADS = XI + WI + (MODE == MX_GEMM_MX ? 2 : 1);
    uint32_t xv[XI], wv[WI];
    constexpr int XE = KS > 1 ? XI : (XI < 2 ? XI : 2);    // (chunks repeat every other load otherwise)
    int xe[XE];                                            // a chunk's first stage past the row
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int slot = wave * XPW + i * 64 + lane, row = slot / G::XSPR, c = slot % G::XSPR;
        const int chunk = c ^ G::xswz(row);
        if (i < XE) {
            const int64_t e = (p.a_bytes - 16 * chunk + 16 * G::XSPR - 1) / (16 * G::XSPR);
            xe[i] = e < s_hi ? (int)e : s_hi;
        }
        xv[i] = (uint32_t)(row * p.a_row) + 16u * chunk;
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
        const int slot = wave * WPW + i * 64 + lane;
        int row = slot / G::WSPR, c = slot % G::WSPR;
        if constexpr (MODE == MX_GEMM) c ^= G::wswz(row);
        if constexpr (MODE == MX_GEMM_MX) c ^= (row >> 1) & 7;
        if constexpr (MODE == MX_GEMM_DX) {
            row ^= (row >> 5) & 1;
            c ^= 4 * ((row >> 4) & 1);
        }
        wv[i] = (uint32_t)(row * p.qb) + 16u * c;
    }

    constexpr int SR = 64 / NW;                            // MX_GEMM_DX: rows whose scales a wave copies
    const uint32_t sv = (uint32_t)(wave * SR + lane) * (uint32_t)p.sb;
    // The loads of stage s, in two parts: a few scales (by some of the lanes), and the codes and
    // activations, one load at a time.  Past this split's last stage they read nothing and clear
    // a slot that is not read, so that the counts of loads in flight stay what they are.
    auto issue_scales = [&](int s) {
        const int ks = s / PA;
        if constexpr (MODE == MX_GEMM_DX) {
            const int o0 = ks * 64, left = (int)p.d_out - o0 < 64 ? (int)p.d_out - o0 : 64;
            const __amdgpu_buffer_rsrc_t z = tile_rsrc(Se + o0 * p.sb + j0 / 32, left, p.sb, s < s_hi, (int)(j0 / 32));
            u32x4* wb = mx_lds + (s % R) * G::STAGE + G::X;
            if (lane < SR) tile_dma(z, wb + G::W + wave * SR, sv, 0);
        } else {
            // a share of the next span's
            const int span = ks / SPAN + 1, part = ks % SPAN;
            u32x4* sb = sc_lds + (span % 3) * G::SROWS;
            const __amdgpu_buffer_rsrc_t z = tile_rsrc(Se + j0 * p.sb, wrows, p.sb, s < s_hi);
            constexpr int WR = BN / SPAN / NW;
            const int row = part * (BN / SPAN) + wave * WR;
            if (lane < WR) tile_dma(z, sb + row, (uint32_t)((row + lane) * p.sb) + 16u * span, 0);
            if constexpr (MODE == MX_GEMM_MX) {
                const __amdgpu_buffer_rsrc_t xz = tile_rsrc(p.AS + at.t0 * p.sb, at.rows, p.sb, s < s_hi);
                constexpr int XR = BM / SPAN / NW;
                const int xrow = part * (BM / SPAN) + wave * XR;
                if (lane < XR) tile_dma(xz, sb + BN + xrow, (uint32_t)((xrow + lane) * p.sb) + 16u * span, 0);
            }
        }
    };
    auto issue_one = [&](int s, int i) {         // load i of XI + WI
        u32x4* base = mx_lds + (s % R) * G::STAGE;
        if (i < XI) {
            const uint32_t v = s < xe[i % XE] ? xv[i] : 0xC0000000u;          // past the row: zeros
            if (XPW % 64 == 0 || lane < XPW % 64) tile_dma(xr, base + wave * XPW + i * 64, v, (uint32_t)s * (16u * G::XSPR));
        } else {
            i -= XI;
            u32x4* wb = base + G::X + wave * WPW + i * 64;
            const int ks = s / PA;
            if constexpr (MODE == MX_GEMM_DX) {
                const int o0 = ks * 64, left = (int)p.d_out - o0 < 64 ? (int)p.d_out - o0 : 64;
                const __amdgpu_buffer_rsrc_t q = tile_rsrc(Qe + o0 * p.qb + j0 / 2, left, p.qb, s < s_hi, (int)(j0 / 2));
                if (WPW % 64 == 0 || lane < WPW % 64) tile_dma(q, wb, wv[i], 0);
            } else {
                const __amdgpu_buffer_rsrc_t q = tile_rsrc(Qe + j0 * p.qb, wrows, p.qb, s < s_hi);
                if (WPW % 64 == 0 || lane < WPW % 64) tile_dma(q, wb, wv[i], (uint32_t)ks * (16u * G::WSPR));
            }
        }
    };
    auto issue = [&](int s) {
        issue_scales(s);
#pragma unroll
        for (int i = 0; i < XI + WI; ++i) issue_one(s, i);
    };

    if constexpr (MODE != MX_GEMM_DX) {
        // the first span's scales whole
        const int span = s_lo / PA / SPAN;
        u32x4* sb = sc_lds + (span % 3) * G::SROWS;
        constexpr int WR = BN / NW;
        if (lane < WR) tile_dma(sr, sb + wave * WR, (uint32_t)((wave * WR + lane) * p.sb) + 16u * span, 0);
        if constexpr (MODE == MX_GEMM_MX) {
            constexpr int XR = BM / NW;
            if (lane < XR) tile_dma(xsr, sb + BN + wave * XR, (uint32_t)((wave * XR + lane) * p.sb) + 16u * span, 0);
        }
    }

    // ---- the contraction, a part of a stage at a time: while one part's products run, the next
    // part's fragments are read, so the loop holds two parts and the accumulators
    typedef MxHalf<MODE, FM, FN> Half;
    typename Half::Acc acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int q = 0; q < FM; ++q)
#pragma unroll
            for (int v = 0; v < Half::V; ++v) acc[f][q][v] = 0.f;
    const uint8_t* const lds = (const uint8_t*)mx_lds;
    // MX_GEMM_MX: a row's eight scale bytes of a stage, and the two words that this lane's four
    // are bytes 0 and 2 of (block 2 h + g: word h / 2, byte 2 (h % 2)), which the products select
    u32x2 raw[MODE == MX_GEMM_MX ? FM + FN : 1];
    uint32_t scale[MODE == MX_GEMM_MX ? FM + FN : 1][2];
    auto take_scales = [&](int s) {
        if constexpr (MODE == MX_GEMM_MX) {
            // a contraction of an odd number of 128s ends in half a stage: its other half has
            // zeros of x against the next row's weights, whose scales must not be NaN
            const bool past = 256 * s + 128 >= p.kpad;
#pragma unroll
            for (int k = 0; k < FM + FN; ++k) {
                scale[k][0] = __builtin_amdgcn_alignbit(raw[k][1], raw[k][0], 8 * g);
                scale[k][1] = past ? 0x7f7f7f7fu : raw[k][1] >> (8 * g);
            }
        }
    };
    // Where this lane reads within a stage: what depends on the lane, once; the rest of an address
    // is the stage's start and a constant, which the instruction holds.
    constexpr int XV = MODE == MX_GEMM ? (KS > 1 ? 8 : 4) : (MODE == MX_GEMM_MX ? 4 : 2);
    constexpr int WV = MODE == MX_GEMM ? KS : (MODE == MX_GEMM_MX ? 4 : 2);
    int lx[XV], lw[WV], ls;
#pragma unroll
    for (int v = 0; v < XV; ++v) {
        // the chunk (its low four bits where a row has more than 8): values of part h
        const int chunk = MODE == MX_GEMM ? 8 * (v >> 2) + 4 * g + (v & 3) : (MODE == MX_GEMM_MX ? 2 * v + g : 2 * g + v);
        lx[v] = (wm * TM + r) * (16 * G::XSPR) + 16 * (chunk ^ G::xswz(r));
    }
#pragma unroll
    for (int v = 0; v < WV; ++v) {
        if constexpr (MODE == MX_GEMM) lw[v] = (wn * TN + r) * (16 * G::WSPR) + 16 * ((2 * v + g) ^ G::wswz(r));
        else if constexpr (MODE == MX_GEMM_MX) lw[v] = (wn * TN + r) * 128 + 16 * ((2 * v + g) ^ ((r >> 1) & 7));
        else lw[v] = (16 * g + (v ^ (g >> 1))) * 128 + 16 * ((wn * 4 + (r >> 2)) ^ (4 * (g & 1))) + 4 * (r & 3);
    }
    if constexpr (MODE == MX_GEMM) ls = (wn * TN + r) * 16 + g;
    else if constexpr (MODE == MX_GEMM_MX) ls = r * 16;
    else ls = 16 * g * 16 + wn * 4 + (r >> 2);
    // read k (of Half::STEPS) of part h of stage s: one fragment, with its scale
    auto read_one = [&](int s, auto part, Half& o, int k) {
        constexpr int h = decltype(part)::value;
        const int xb = (s % R) * G::STAGE * 16, wb = xb + G::X * 16, ks = s / PA;
        const int sb = (R * G::STAGE + ((ks / SPAN) % 3) * G::SROWS) * 16;
        if constexpr (MODE == MX_GEMM) {
            // part h: values 16 hh .. of the 32 that lane (r, g) has of piece kk, in plane q0
            constexpr int kk = h / (2 * G::PS), q0 = h / 2 % G::PS, hh = h % 2, at = kk * G::PS + q0;
            // an odd number of 128s ends in half a stage: its other half has zeros of x against
            // the next row's weights, whose scales must not be NaN
            const bool past = KS == 4 && kk >= 2 && 256 * ks + 128 >= p.kpad;
            if (k < FN) {
                o.w[k] = *(const u32x2*)(lds + (wb + lw[kk]) + (k * 32 * 16 * G::WSPR + 8 * hh));
                const uint32_t sc = *(lds + (sb + 2 * KS * (ks % SPAN) + ls) + (k * 32 * 16 + 2 * kk));
                o.ws[k] = past ? 127u : sc;
            } else {
                const int q = (k - FN) / 2, u = (k - FN) % 2;
                o.x[q][u] = *(const u32x4*)(lds + (xb + lx[4 * (at % 2) + 2 * hh + u]) + (q * 32 * 16 * G::XSPR + at / 2 * 256));
            }
        } else if constexpr (MODE == MX_GEMM_MX) {
            // lane (r, g): block 2 h + g of the stage's eight; with the first part, all eight scales
            if (k < FM) o.x[k] = *(const u32x4*)(lds + (xb + lx[h]) + k * 32 * 128);
            else o.w[k - FM] = *(const u32x4*)(lds + (wb + lw[h]) + (k - FM) * 32 * 128);
            if constexpr (h == 0) {
                const int row0 = k < FM ? BN + wm * TM : wn * TN;
                raw[k] = *(const u32x2*)(lds + (sb + 8 * (ks % SPAN) + row0 * 16 + ls) + (k < FM ? k : k - FM) * 32 * 16);
            }
        } else {
            // lane (r, g): rows 16 g + 8 h .. + 7 of the stage's 64, columns 8 r .. of the wave's 128
            if (k < 8) {
                o.w[k] = *(const uint32_t*)(lds + (wb + lw[k % 2]) + (8 * h + (k & ~1)) * 128);
                o.ws[k] = *(lds + (wb + ls) + (G::W * 16 + (8 * h + k) * 16));
            } else {
                o.x[k - 8] = *(const u32x4*)(lds + (xb + lx[h]) + (k - 8) * 16 * 128);
            }
        }
    };
    auto read = [&](int s, auto part, Half& o) {
#pragma unroll
        for (int k = 0; k < Half::STEPS; ++k) read_one(s, part, o, k);
    };
    // product i (of Half::PRODUCTS) of a part; `a`: the dequantised weights of the last ones
    u32x4 a[2];
    auto product = [&](const Half& o, auto part, auto index) {
        constexpr int i = decltype(index)::value;
        if constexpr (MODE == MX_GEMM) {
            constexpr int u = i / (FM * FN), f = i / FM % FN, q = i % FM;
            if constexpr (q == 0) {
                const uint32_t w = o.w[f][u];
                const float sc = mx_scale(o.ws[f]);
                a[0] = u32x4{mx_bf16<0>(w, sc), mx_bf16<1>(w, sc), mx_bf16<2>(w, sc), mx_bf16<3>(w, sc)};
            }
            acc[f][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a[0]), as_bf16x8(o.x[q][u]), acc[f][q], 0, 0, 0);
        } else if constexpr (MODE == MX_GEMM_MX) {
            constexpr int f = i / FM, q = i % FM;
            const i32x8 w{(int)o.w[f][0], (int)o.w[f][1], (int)o.w[f][2], (int)o.w[f][3], 0, 0, 0, 0};
            const i32x8 x{(int)o.x[q][0], (int)o.x[q][1], (int)o.x[q][2], (int)o.x[q][3], 0, 0, 0, 0};
            constexpr int h = decltype(part)::value, byte = 2 * (h % 2);
            acc[f][q] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc[f][q], 4, 4, byte, (int)scale[FM + f][h / 2], byte, (int)scale[q][h / 2]);
        } else {
            // byte b of the words: columns 8 r + 2 b and 8 r + 2 b + 1
            constexpr int b = i / (2 * FM), q = i / 2 % FM, odd = i % 2;
            if constexpr (i % (2 * FM) == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = mx_bf16<b>(o.w[2 * k], mx_scale(o.ws[2 * k]));
                    const uint32_t v = mx_bf16<b>(o.w[2 * k + 1], mx_scale(o.ws[2 * k + 1]));
                    a[0][k] = __builtin_amdgcn_perm(v, u, 0x05040100u);
                    a[1][k] = __builtin_amdgcn_perm(v, u, 0x07060302u);
                }
            }
            acc[2 * b + odd][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a[odd]), as_bf16x8(o.x[q]), acc[2 * b + odd][q], 0, 0, 0);
        }
    };
    // Products of `cur` (part `own`) while part `part` of stage s is read into `nxt` and loads l0 .. l1 - 1 of
    // stage sl are issued: the reads beside the first products, so that they have arrived when
    // the part ends, and the loads evenly, at the rate at which they are taken.
    auto run = [&](const Half& cur, auto own, int s, auto part, Half& nxt, int sl, auto l0, auto l1) {
        constexpr int MM = Half::PRODUCTS, L0 = decltype(l0)::value, LN = decltype(l1)::value - L0;
        constexpr int RP = (2 * Half::STEPS + MM - 1) / MM;                   // reads beside a product
        tile_each<MM>([&](auto index) {
            constexpr int i = decltype(index)::value;
#pragma unroll
            for (int k = RP * i; k < RP * (i + 1); ++k)
                if (k < Half::STEPS) read_one(s, part, nxt, k);
            product(cur, own, index);
#pragma unroll
            for (int l = i * LN / MM; l < (i + 1) * LN / MM; ++l) issue_one(sl, L0 + l);
            if constexpr (MODE != MX_GEMM_DX) __builtin_amdgcn_sched_barrier(0);
        });
    };

    constexpr int ALL = XI + WI, LATE = MODE == MX_GEMM_MX ? ALL / 2 : 0, SOON = ALL - LATE;
    const std::integral_constant<int, 0> zero{};
    const std::integral_constant<int, SOON> soon{};
    const std::integral_constant<int, ALL> all{};
    if (s_lo < s_hi) {
#pragma unroll
        for (int i = 0; i < R - 1; ++i) issue(s_lo + i);
        issue_scales(s_lo + R - 1);
#pragma unroll
        for (int i = 0; i < SOON; ++i) issue_one(s_lo + R - 1, i);
        tile_wait_vmcnt<LOADS * (R - 2) + LOADS - LATE>();
        tile_barrier();
        // a wave whose rows all lie past the tile's own only copies
        const bool idle = wm * TM >= at.rows;
        for (int s = s_lo; idle && s < s_hi; ++s) {
#pragma unroll
            for (int i = SOON; i < ALL; ++i) issue_one(s + R - 1, i);
            tile_wait_vmcnt<LOADS * (R - 2)>();
            tile_barrier();
            issue_scales(s + R);
#pragma unroll
            for (int i = 0; i < SOON; ++i) issue_one(s + R, i);
        }
        Half A, B;
        if (!idle) {
            read(s_lo, zero, A);
            take_scales(s_lo);
        }
        for (int s = s_lo; !idle && s < s_hi; ++s) {
            // the rest of the last stage's loads go out with the first part
            run(A, zero, s, std::integral_constant<int, 1>{}, B, s + R - 1, soon, all);
            tile_each<G::PARTS / 2 - 1>([&](auto i) {
                constexpr int h = 2 * decltype(i)::value;
                run(B, std::integral_constant<int, h + 1>{}, s, std::integral_constant<int, h + 2>{}, A, 0, zero, zero);
                run(A, std::integral_constant<int, h + 2>{}, s, std::integral_constant<int, h + 3>{}, B, 0, zero, zero);
            });
            tile_wait_vmcnt<LOADS * (R - 2)>();    // stage s + 1 has landed
            tile_barrier();                        // and this one's slot has been read by every wave
            issue_scales(s + R);
            run(B, std::integral_constant<int, G::PARTS - 1>{}, s + 1, zero, A, s + R, zero, soon);  // past the last stage: read and not used
            take_scales(s + 1);
        }
    }
    tile_wait_vmcnt<0>();          // no load may land in the LDS later
    __syncthreads();

    // ---- store, T rows of a wave's tile at a time, by way of LDS of its own: in the
    // accumulators a lane's neighbours are other rows, in memory they are a row's columns.
    // 16 x 16 products: lane (r, g) holds row r and columns 4 g + v (the gradient's fragment f:
    // column 8 c + f); 32 x 32: row r and columns 8 (v / 4) + 4 g + v % 4.
    float* const part = p.part ? p.part + (int64_t)blockIdx.y * p.n * p.m : nullptr;
    const int wide = part || !p.y_bf16 ? 4 : 2, pitch = TN * wide + 16;
    uint8_t* const own = (uint8_t*)mx_lds + wave * (T * (TN * 4 + 16));
    uint8_t* const out = part ? (uint8_t*)part : (uint8_t*)p.y;
    auto put = [&](int col, f32x4 v) {           // four columns of row r
        if (wide == 4) *(f32x4*)(own + r * pitch + 4 * col) = v;
        else *(u32x2*)(own + r * pitch + 2 * col) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    const int64_t jw = j0 + wn * TN;
    const int cols = (int)(p.m - jw < TN ? p.m - jw : TN);        // can be negative
#pragma unroll
    for (int q = 0; q < FM; ++q) {
        if constexpr (MODE == MX_GEMM_DX) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int f = 0; f < 8; f += 4)
                    put(8 * (4 * g + v) + f, f32x4{acc[f][q][v], acc[f + 1][q][v], acc[f + 2][q][v], acc[f + 3][q][v]});
        } else {
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int v = 0; v < 16; v += 4)
                    put(32 * f + 2 * v + 4 * g, f32x4{acc[f][q][v], acc[f][q][v + 1], acc[f][q][v + 2], acc[f][q][v + 3]});
        }
        const int row0 = wm * TM + T * q, left = at.rows - row0;
        const int lanes = TN * wide / 16;                        // of a row: a power of two
        auto store = [&](auto ends) {                            // ends: rows may end inside 16 bytes
            for (int i = lane; i < T * lanes; i += 64) {
                const int row = i / lanes, at16 = 16 * (i - row * lanes), some = cols * wide - at16;
                const u32x4 v = *(const u32x4*)(own + row * pitch + at16);
                if (row >= left || some <= 0) continue;
                uint8_t* const to = out + ((at.t0 + row0 + row) * p.m + jw) * wide + at16;
                if (!decltype(ends)::value || some >= 16) {
                    *(u32x4_any*)to = v;
                } else {
                    for (int c = 0; c < some; c += wide) {
                        if (wide == 4) *(uint32_t*)(to + c) = v[c / 4];
                        else *(uint16_t*)(to + c) = (uint16_t)(v[c / 4] >> (8 * (c & 2)));
                    }
                }
            }
        };
        if (cols * wide % 16 == 0) store(std::false_type{});
        else store(std::true_type{});
    }
}

// ---------------------------------------------------------------------------
// Few rows: the weight is streamed once, each wave on its own, without a barrier before the end
// (one row 4096 -> 4096: 5.1 us; by tiles 8.0 and 4.0 for the sum of the split).  A block takes 16 MT output
// columns of one weight and 16 rows of activations at a time; its waves share out the contraction and
// their sums are added in the waves' order at the end.  A wave copies pieces of
// KU groups of 128 values of its 16 MT weight rows into LDS of its own, one piece ahead: read
// straight into registers, 16 consecutive lanes would touch 16 rows and take four times the
// address cycles.  Lane (r, b) then holds block b of a group of column r's weight (16 bytes),
// dequantised in place to the products' left operand, and the same 32 values of row r of the
// activations; the order of the values within a product is free.
//
// The plan knows the mean of the experts' rows alone.  An expert's block takes its first two groups of
// 16 rows, and what experts have beyond those is spread over blocks of its own, up to one a compute
// unit, that find their groups from the offsets.  3040 rows, 190 experts of 8192 -> 128: evenly
// routed 52 us, by a lognormal of 0.7 63, all to one expert 63; with every group left to its
// expert's block 52, 92 and 1930.  Where no expert has more than 32 of over 32 rows those blocks end at
// once, which takes 0 to 1 us (128 rows, 8 of 4096 -> 1024: 10.9 us, 10.1 without).  With one group
// or four a block: 63 and 76 us by the lognormal, but 128 rows, 8 of 4096 -> 1024 14.7 and 13.4 (two: 13.4).
// ---------------------------------------------------------------------------
constexpr int MX_FIRST = 2;

template <int MODE, int P, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_stream(MxTile p) {
    constexpr int KU = P == 3 ? 2 : 4;           // (three planes of x fill the registers sooner)
    constexpr int SPR = 4 * KU, WS = 16 * MT * SPR, PIECE = WS + 64, LOADS = WS / 64 + 1;
    extern __shared__ u32x4 mx_lds[];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, b = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    u32x4* const ring = mx_lds + wave * 2 * PIECE;
    auto sums = [&](int w, int t) { return (float*)(mx_lds + w * 2 * PIECE) + 256 * t; };    // over the rings at the end
    const int64_t j0 = (int64_t)blockIdx.x * (16 * MT);
    const int groups = (int)(p.qb / 64), pieces = (groups + KU - 1) / KU;
    const int shares = WAVES * (int)gridDim.z, per = (pieces + shares - 1) / shares;
    const int c0 = ((int)blockIdx.z * WAVES + wave) * per;
    const int c1 = c0 + per < pieces ? c0 + per : pieces;

    const int wrows = (int)(p.m - j0 < 16 * MT ? p.m - j0 : 16 * MT);
    auto swizzle = [](int row) { return KU == 4 ? row & 15 : (row >> 1) & 7; };
    uint32_t wv[WS / 64];
#pragma unroll
    for (int i = 0; i < WS / 64; ++i) {
        const int slot = i * 64 + lane, row = slot / SPR;
        wv[i] = (uint32_t)(row * p.qb) + 16u * ((slot % SPR) ^ swizzle(row));
    }
    // This block's rows, 16 at a time: its expert's first MX_FIRST groups of them, or every step-th of
    // the groups that experts have beyond those.
    const int beyond = (int)blockIdx.y - p.experts, step = (int)gridDim.y - p.experts;
    int64_t lo = 0, hi = p.n;
    if (p.offsets && beyond < 0) tile_expert_rows(p.offsets, blockIdx.y, p.n, lo, hi);
    for (int turn = 0;; ++turn) {
        TilePlace place;
        if (beyond < 0) {
            place.e = blockIdx.y;
            place.t0 = lo + 16 * turn;
            place.rows = (int)(hi - place.t0 < 16 ? hi - place.t0 : 16);
            place.ok = turn < MX_FIRST && place.rows > 0;
        } else {
            tile_of_row(p, 16, beyond + turn * step, place, MX_FIRST);
        }
        if (!place.ok) return;
        if (turn > 0) __syncthreads();           // the sums of the rows before have been read
        const int rows = place.rows;
        const int64_t t0 = place.t0, row0 = (int64_t)place.e * p.d_out + j0;
        auto copy = [&](int c) {                     // past the last piece: clears, reads nothing
            u32x4* to = ring + (c & 1) * PIECE;
            const __amdgpu_buffer_rsrc_t wr = tile_rsrc(p.Q + row0 * p.qb, wrows, p.qb, c < c1);
            const __amdgpu_buffer_rsrc_t sr = tile_rsrc(p.S + row0 * p.sb, wrows, p.sb, c < c1);
#pragma unroll
            for (int i = 0; i < WS / 64; ++i) tile_dma(wr, to + 64 * i, wv[i], (uint32_t)c * (16u * SPR));
            tile_dma(sr, to + WS, lane < 16 * MT ? (uint32_t)(lane * p.sb) : 0xC0000000u, (uint32_t)c * (4u * KU));
        };

        const int64_t xrow = t0 + (r < rows ? r : rows - 1);
        const uint8_t* const xp = p.A + xrow * p.a_row;
        const uint8_t* const xsp = MODE == MX_GEMM_MX ? p.AS + xrow * p.sb : nullptr;
        f32x4 acc[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (c0 < c1) copy(c0);
        for (int c = c0; c < c1; ++c) {
            // this piece's activations, then the next piece's copies: once those alone are in
            // flight, both this piece's copies and its activations have arrived
            u32x4 x[KU][MODE == MX_GEMM_MX ? 1 : 4 * P];
            uint32_t xs[KU];
#pragma unroll
            for (int h = 0; h < KU; ++h) {
                const int g = KU * c + h;                     // (past the last: zeros)
                if constexpr (MODE == MX_GEMM_MX) {
                    const u32x4 v = *(const u32x4*)(xp + (g < groups ? 64 * g : 0) + 16 * b);
                    x[h][0] = g < groups ? v : u32x4{0u, 0u, 0u, 0u};
                    xs[h] = *(const uint32_t*)(xsp + (g < groups ? 4 * g : 0));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < P; ++q) {
                            // values 128 g + 32 b + 8 j .. of plane q
                            const int at = ((2 * g + (b >> 1)) * P + q) * 128 + 64 * (b & 1) + 16 * j;
                            const u32x4 v = *(const u32x4*)(xp + (at < p.a_bytes ? at : 0));
                            x[h][j * P + q] = at < p.a_bytes ? v : u32x4{0u, 0u, 0u, 0u};
                        }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            copy(c + 1);
            tile_wait_vmcnt<LOADS>();
            __builtin_amdgcn_sched_barrier(0);
            const uint8_t* const at = (const uint8_t*)(ring + (c & 1) * PIECE);
#pragma unroll
            for (int h = 0; h < KU; ++h) {
                const bool has = KU * c + h < groups;         // else codes and scales of the next row
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int row = 16 * t + r;
                    const u32x4 w = *(const u32x4*)(at + 16 * (row * SPR + ((4 * h + b) ^ swizzle(row))));
                    const uint32_t sb = at[16 * (WS + row) + 4 * h + b], sc = has ? sb : 127u;
                    if constexpr (MODE == MX_GEMM_MX) {
                        const i32x8 wa{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                        const i32x8 xa{(int)x[h][0][0], (int)x[h][0][1], (int)x[h][0][2], (int)x[h][0][3], 0, 0, 0, 0};
                        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xa, acc[t], 4, 4, 0, (int)sc, 0, (int)((xs[h] >> (8 * b)) & 255u));
                    } else {
                        const float f = mx_scale(sc);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x4 wa{mx_bf16<0>(w[j], f), mx_bf16<1>(w[j], f), mx_bf16<2>(w[j], f), mx_bf16<3>(w[j], f)};
#pragma unroll
                            for (int q = 0; q < P; ++q)
                                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wa), as_bf16x8(x[h][j * P + q]), acc[t], 0, 0, 0);
                        }
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
        // output (row i / (16 MT), column i % (16 MT)) is in lane 16 (column / 4) + row, element column % 4
        for (int i = tid; i < 256 * MT; i += 64 * WAVES) {
            const int row = i / (16 * MT), c = i - row * (16 * MT), t = c >> 4;
            const int from = 4 * (16 * ((c & 15) >> 2) + row) + (c & 3);
            if (row >= rows || j0 + c >= p.m) continue;
            float v = sums(0, t)[from];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += sums(w, t)[from];
            const int64_t at = (t0 + row) * p.m + j0 + c;
            if (p.part) p.part[(int64_t)blockIdx.z * p.n * p.m + at] = v;
            else if (p.y_bf16) ((uint16_t*)p.y)[at] = (uint16_t)f32_to_bf16_bits(v);
            else ((float*)p.y)[at] = v;
        }
    }
}

// y = the sum of a split contraction's parts, in their order; rows that belong to an expert
// (all of them without offsets).  2 to 4 us, most of it the launch, for up to 16 parts of a few
// hundred kilobytes.
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int split, int64_t n,
                                                int64_t m, const int64_t* __restrict__ offsets,
                                                int experts, void* __restrict__ y, int y_bf16) {
    int64_t lo = 0, hi = n;
    if (offsets) {
        int64_t a, b;
        tile_expert_rows(offsets, 0, n, lo, a);
        tile_expert_rows(offsets, experts - 1, n, b, hi);
    }
    const int64_t first = lo * m, end = hi * m, all = n * m, stride = (int64_t)gridDim.x * 256;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (all % 4 == 0 && m % 4 == 0 && ((uintptr_t)y & (y_bf16 ? 7u : 15u)) == 0) {
        for (int64_t t = first + 4 * id; t < end; t += 4 * stride) {
            f32x4 s = *(const f32x4*)(part + t);
            int k = 1;
            for (; k + 4 <= split; k += 4) {     // four loads in flight, added in their order
                f32x4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = *(const f32x4*)(part + (k + i) * all + t);
#pragma unroll
                for (int i = 0; i < 4; ++i) s += v[i];
            }
            for (; k < split; ++k) s += *(const f32x4*)(part + k * all + t);
            if (y_bf16) *(u32x2*)((uint16_t*)y + t) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
            else *(f32x4*)((float*)y + t) = s;
        }
        return;
    }
    for (int64_t t = first + id; t < end; t += stride) {
        float s = part[t];
        for (int k = 1; k < split; ++k) s += part[k * all + t];
        if (y_bf16) ((uint16_t*)y)[t] = (uint16_t)f32_to_bf16_bits(s);
        else ((float*)y)[t] = s;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static size_t mx_al256(size_t x) { return (x + 255) & ~(size_t)255; }

// What a call does, from its sizes and types alone.
struct MxPlan {
    bool staged;                  // activations are copied into planes first
    int planes;
    bool stream;                  // few rows a weight
    int bm, bn, split, waves;
    int stages, unit;
    size_t stage_bytes, part_bytes;
};

static MxPlan mx_plan(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts) {
    MxPlan P;
    const int64_t k = op == MX_GEMM_DX ? d_out : d_in, m = op == MX_GEMM_DX ? d_in : d_out;
    P.planes = a_bf16 ? 1 : 3;
    P.staged = op != MX_GEMM_MX && (!a_bf16 || k % 8 != 0);
    const int64_t k64 = op == MX_GEMM_DX ? (k + 63) / 64 : 2 * mx_groups(k);
    P.stage_bytes = P.staged ? mx_al256((size_t)n * k64 * 64 * P.planes * 2) : 0;
    const int64_t per = (n + experts - 1) / experts;
    // Streaming saves the tiles' split and its sum (one token 4096 -> 4096: 9.7 us a call, 13.7 by
    // tiles); where tiles need no split they are as fast or faster (8192 -> 28672: 31 and 29), and
    // with more activations than a wave's registers take in passing too (16 rows of 14336: 18 and
    // 14 us; 16 of 4096 in float32: 19 and 17; packed 16 of 28672: 25 and 24).
    const int64_t live = experts > 1 ? (experts < n ? experts : n) : 1;          // experts with rows, at most
    const int64_t room = op == MX_GEMM_MX ? 1 << 18 : (a_bf16 ? 1 << 17 : 3 << 14);
    P.stream = op != MX_GEMM_DX && per <= 16 && per * k <= room && live * ((m + 127) / 128) < 192;
    P.split = 1;
    P.stages = P.unit = 0;
    int64_t blocks, units, pieces = 0;
    if (P.stream) {
        P.bm = 16;
        P.bn = live * ((m + 31) / 32) >= 256 ? 32 : 16;
        const int ku = P.planes == 3 ? 2 : 4;
        pieces = (mx_groups(k) + ku - 1) / ku;
        P.waves = pieces >= 8 ? 8 : 4;
        blocks = live * ((m + P.bn - 1) / P.bn);
        units = pieces / P.waves;
    } else {
        // The largest tile that the rows of a weight fill and that gives most compute units
        // one, else the smallest: 1024 rows 4096 -> 4096 take 40 us by 128 x 128 and 54 by
        // 256 x 256 split in four, 2048 rows 69 and 79; fp4 17 and 41, 26 and 44.  In float32
        // (three times the products, so the split's sum weighs less) large tiles pay from 64
        // on: 1024 rows 104 us and 126 by 128 x 128, 512 rows 79 and 59 by 64 x 128.  The
        // gradient's smaller tiles convert the same weights for fewer products: it takes the
        // largest from 48 on (512 rows of 4096 x 4096: 45 us, 60 by 128 x 256).
        // Experts in fp4 have last tiles that are part empty, and after a short contraction a
        // compute unit's one large tile has its start and its stores to itself: up to 1024 rows
        // an expert and 2048 values take tiles of at most 128 x 128 (24000 rows over 64 experts
        // 2048 -> 1408: 84 us, 105 by 256 x 256; 16384 rows: 66 and 80; but 8 experts 2048 ->
        // 4096 of 2048 rows each 141 and 144, 16 experts 1024 -> 4096 of 1875 rows 197 and 186, one
        // weight 2048 -> 2048 with 8192 rows 32 and 30, 16 of 8192 -> 8192 with 137 rows 220 and 190).
        const bool small = op == MX_GEMM_MX && experts > 1 && per <= 1024 && k <= 2048;
        P.bm = per > 128 && !small ? 256 : (per > 64 ? 128 : (per > 32 || op == MX_GEMM_DX ? 64 : 32));
        for (;; P.bm /= 2) {
            P.bn = P.bm == 256 || op == MX_GEMM_DX ? 256 : 128;
            const int64_t rows = experts > 1 ? n / P.bm + (experts < n ? experts : n) : (n + P.bm - 1) / P.bm;
            blocks = rows * ((m + P.bn - 1) / P.bn);
            if (P.bm <= 64 || blocks >= (op == MX_GEMM_DX ? 48 : (P.planes == 3 && P.bm == 256 ? 64 : 192))) break;
        }
        // Few rows of x: stages of 256 (128: three planes of them) values, so that a weight row
        // is read by whole lines (24 rows 14336 -> 4096: 15.6 -> 12.9 us).
        const int deep = op != MX_GEMM || P.bm > 64 ? 1 : (P.bm == 64 && P.planes == 3 ? 2 : 4);
        P.stages = (int)(op == MX_GEMM_MX ? (mx_groups(k) + 1) / 2 : (deep == 1 ? k64 * P.planes : (k64 + deep - 1) / deep));
        P.unit = op == MX_GEMM_DX ? P.planes : (op == MX_GEMM_MX ? 2 : (deep == 1 ? 8 * P.planes : 8 / deep));
        units = (P.stages + P.unit - 1) / P.unit;
    }
    if (units < 1) units = 1;
    if (blocks < 256) {
        int64_t s = (P.stream ? 512 : 256) / blocks;
        // 129 to 170 large tiles of the gradient in thirds take two rounds of three: worth the sum
        // from 96 stages on (8192 -> 2048, 5060 rows: 198 us, 224 whole; float32, 2500 rows of
        // 4096 -> 4096: 295 and 356; but 4096 -> 2048 in bfloat16 123 and 118; the product itself,
        // 4096 -> 2048 in float32, 312 and 298).
        if (op == MX_GEMM_DX && P.bm == 256 && experts == 1 && P.stages >= 96 && blocks > 128 && blocks <= 170) s = 3;
        s = s < units ? s : units;
        s = s < 1 ? 1 : (s > 16 ? 16 : s);
        // A part's sums are written and read at about 4 TB/s; a stage of a tile takes 0.6 to 1.7 us:
        // no part that costs more than it saves (gradient of 1024 -> 256, 4000 rows: 32 -> 16 us)
        const int64_t t = P.bm == 256 ? 17 : (P.bm == 128 ? (op == MX_GEMM_DX ? 11 : 7) : 6);
        while (!P.stream && s > 1 && s * s * n * m * 20 > P.stages * (s - 1) * t * 1000000) --s;
        const int64_t each = (units + s - 1) / s;        // no part without work
        P.split = (int)((units + each - 1) / each);
        if (P.stream) {                                  // (nor one without a piece, as the kernel shares them out)
            const int64_t some = (pieces + P.waves * P.split - 1) / (P.waves * P.split);
            P.split = (int)((pieces + some * P.waves - 1) / (some * P.waves));
        }
    }
    P.part_bytes = P.split > 1 ? mx_al256((size_t)P.split * n * m * 4) : 0;
    return P;
}

// Rows that a product of one weight by plan P takes first, by full rounds of large tiles (one for
// each compute unit), where the others would be up to half a round more: those are then a product
// of their own, by smaller tiles or a split (4352 rows 4096 -> 4096: 130 us, 184 at once; float32
// 343 and 546, fp4 57 and 69, gradient 158 and 225).  Half a round at once takes the same or less
// from there on (6144 rows, half: 186 and 186; 6656: 221 and 191; gradient 231 and 226).
static int64_t mx_head(const MxPlan& P, MxOp op, int64_t n, int64_t d_in, int64_t d_out) {
    if (P.stream || P.bm < 256) return n;
    const int64_t cols = ((op == MX_GEMM_DX ? d_in : d_out) + 255) / 256, tiles = (n + 255) / 256 * cols;
    const int64_t head = (tiles - 1) / 256 * 256 / cols;          // row tiles
    return head * cols >= 192 && tiles - head * cols <= 128 ? head * 256 : n;
}

size_t mx_gemm_workspace(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts) {
    const MxPlan P = mx_plan(op, a_bf16, n, d_in, d_out, experts);
    size_t part = P.part_bytes;
    const int64_t head = experts == 1 ? mx_head(P, op, n, d_in, d_out) : n;
    if (head < n) {              // (a call with offsets takes all rows at once)
        const size_t rest = mx_plan(op, a_bf16, n - head, d_in, d_out, 1).part_bytes;
        part = part > rest ? part : rest;
    }
    return P.stage_bytes + part;
}

// Blocks of a launch of tiles of bm x bn: with offsets every expert can have a part-empty one
static int64_t mx_blocks(int64_t n, int64_t m, int bm, int bn, int64_t part_empty) {
    return (((n + bm - 1) / bm + part_empty) * ((m + bn - 1) / bn) + 7) / 8 * 8;
}

// A launch has fewer than 2^32 lanes: close to 2^31 rows of few columns, or thousands of experts with
// 2^18 columns each, would take more.
constexpr int64_t MX_MAX_LANES = ((int64_t)1 << 32) - 1;

static int mx_waves(const MxPlan& P, MxOp op) {
    return P.stream ? P.waves : ((P.bm == 256 && op != MX_GEMM_MX) || (P.bm == 128 && op == MX_GEMM_DX) ? 8 : 4);
}

int64_t mx_gemm_plan(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets, int32_t (&plan)[6]) {
    MxPlan P = mx_plan(op, a_bf16, n, d_in, d_out, experts);
    const int64_t head = offsets ? n : mx_head(P, op, n, d_in, d_out);
    if (head < n) P = mx_plan(op, a_bf16, head, d_in, d_out, 1);
    const int32_t v[6] = {P.planes, P.stream, P.bm, P.bn, mx_waves(P, op), P.split};
    for (int i = 0; i < 6; ++i) plan[i] = v[i];
    return head;
}

bool mx_gemm_fits(MxOp op, bool a_bf16, int64_t n, int64_t d_in, int64_t d_out, int experts, bool offsets) {
    const int64_t m = op == MX_GEMM_DX ? d_in : d_out;
    if ((n / 32 + 1 + experts) * ((m + 127) / 128) < (int64_t)1 << 22) return true;   // by any tiles
    const MxPlan whole = mx_plan(op, a_bf16, n, d_in, d_out, experts);
    const int64_t head = offsets ? n : mx_head(whole, op, n, d_in, d_out);
    for (int64_t rows : {head, n - head}) {
        if (rows == 0) continue;
        const MxPlan P = rows == n ? whole : mx_plan(op, a_bf16, rows, d_in, d_out, 1);
        if (!P.stream && mx_blocks(rows, m, P.bm, P.bn, offsets ? experts : 0) * 64 * mx_waves(P, op) > MX_MAX_LANES) return false;
    }
    return true;
}

template <int MODE, int P, int BM, int BN, int WM, int NW = 4, int KS = 1>
static hipError_t mx_launch(const MxTile& t, int split, hipStream_t st) {
    const void* k = (const void*)k_mx_tile<MODE, P, BM, BN, WM, NW, KS>;
    // the stages and scales, later the outputs on their way
    constexpr int T = MODE == MX_GEMM_DX ? 16 : 32, TN = BN / (NW / WM);
    constexpr size_t OUT = (size_t)NW * T * (TN * 4 + 16), IN = MxGeo<MODE, P, BM, BN, KS>::BYTES;
    constexpr size_t lds = IN > OUT ? IN : OUT;
    static_assert(lds <= 160 * 1024, "LDS of a compute unit");
    hipError_t e = ensure_dynamic_lds(k, lds);
    if (e != hipSuccess) return e;
    const int64_t grid = mx_blocks(t.n, t.m, BM, BN, t.offsets ? t.experts : 0);
    if (grid * (64 * NW) > MX_MAX_LANES) return hipErrorInvalidValue;     // (refused before)
    hipLaunchKernelGGL((k_mx_tile<MODE, P, BM, BN, WM, NW, KS>), dim3((unsigned)grid, (unsigned)split), dim3(64 * NW), lds, st, t);
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

template <int MODE, int P, int MT, int WAVES>
static hipError_t mx_launch_stream(const MxTile& t, const MxPlan& pl, hipStream_t st) {
    constexpr int KU = P == 3 ? 2 : 4;
    const size_t lds = (size_t)WAVES * 2 * (16 * MT * 4 * KU + 64) * 16;
    const hipError_t e = ensure_dynamic_lds((const void*)k_mx_stream<MODE, P, MT, WAVES>, lds);
    if (e != hipSuccess) return e;
    // a block for each expert, and for the groups beyond its own those of a compute unit each
    const int64_t cols = (t.m + 16 * MT - 1) / (16 * MT), far = (t.n + 15) / 16 - MX_FIRST, room = 256 / (cols * pl.split);
    const int64_t more = !t.offsets || far < 1 ? 0 : (room < 1 ? 1 : (room < far ? room : far));
    const dim3 grid((unsigned)cols, (unsigned)(t.experts + more), (unsigned)pl.split);
    hipLaunchKernelGGL((k_mx_stream<MODE, P, MT, WAVES>), grid, dim3(64 * WAVES), lds, st, t);
    GQ_LAUNCH_CHECK();
    return hipSuccess;
}

template <int MODE, int P>
static hipError_t mx_launch_size(const MxTile& t, const MxPlan& pl, hipStream_t st) {
    if constexpr (MODE != MX_GEMM_DX) {
        if (pl.stream && pl.waves == 8)
            return pl.bn == 32 ? mx_launch_stream<MODE, P, 2, 8>(t, pl, st) : mx_launch_stream<MODE, P, 1, 8>(t, pl, st);
        if (pl.stream)
            return pl.bn == 32 ? mx_launch_stream<MODE, P, 2, 4>(t, pl, st) : mx_launch_stream<MODE, P, 1, 4>(t, pl, st);
    }
    if constexpr (MODE == MX_GEMM_DX) {
        switch (pl.bm) {
            case 256: return mx_launch<MODE, P, 256, 256, 4, 8>(t, pl.split, st);
            case 128: return mx_launch<MODE, P, 128, 256, 4, 8>(t, pl.split, st);
            default: return mx_launch<MODE, P, 64, 256, 2>(t, pl.split, st);
        }
    } else {
        switch (pl.bm) {
            case 256:
                if constexpr (MODE == MX_GEMM_MX) return mx_launch<MODE, P, 256, 256, 2>(t, pl.split, st);
                else return mx_launch<MODE, P, 256, 256, 4, 8>(t, pl.split, st);
            case 128: return mx_launch<MODE, P, 128, 128, 2>(t, pl.split, st);
            case 64: return mx_launch<MODE, P, 64, 128, 1, 4, MODE == MX_GEMM ? (P == 1 ? 4 : 2) : 1>(t, pl.split, st);
            default: return mx_launch<MODE, P, 32, 128, 1, 4, MODE == MX_GEMM ? 4 : 1>(t, pl.split, st);
        }
    }
}

hipError_t mx_gemm_run(const MxCall& c, void* ws, hipStream_t st) {
    StageTimer tm(ST_MXFP4_GEMM, st);
    const MxPlan whole = mx_plan(c.op, c.a_bf16, c.n, c.d_in, c.d_out, c.experts);
    const int64_t k = c.op == MX_GEMM_DX ? c.d_out : c.d_in, m = c.op == MX_GEMM_DX ? c.d_in : c.d_out;
    MxTile t{};
    t.A = (const uint8_t*)c.a;
    t.AS = c.as;
    t.a_row = t.a_bytes = c.op == MX_GEMM_MX ? mx_row_bytes(k) : 2 * k;
    if (whole.staged) {
        const int64_t pieces = c.op == MX_GEMM_DX ? (k + 63) / 64 : 2 * mx_groups(k);
        t.A = (const uint8_t*)ws;
        t.a_row = t.a_bytes = pieces * whole.planes * 128;
        const int64_t blocks = (c.n * pieces * 8 + 255) / 256;
        const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096));
        if (c.a_bf16) hipLaunchKernelGGL(k_mx_stage<true>, grid, dim3(256), 0, st, c.a, c.n, k, pieces, (uint16_t*)ws);
        else hipLaunchKernelGGL(k_mx_stage<false>, grid, dim3(256), 0, st, c.a, c.n, k, pieces, (uint16_t*)ws);
        GQ_LAUNCH_CHECK();
    }
    t.Q = c.Q;
    t.S = c.S;
    t.qb = mx_row_bytes(c.d_in);
    t.sb = mx_row_scales(c.d_in);
    t.offsets = c.offsets;
    t.experts = c.experts;
    t.m = m;
    t.d_out = c.d_out;
    t.kpad = (int)(128 * mx_groups(k));
    t.y = c.y;
    t.y_bf16 = c.y_bf16;
    // the next `rows` rows of t
    auto product = [&](int64_t rows) -> hipError_t {
        const MxPlan pl = rows == c.n ? whole : mx_plan(c.op, c.a_bf16, rows, c.d_in, c.d_out, 1);
        t.n = rows;
        t.stages = pl.stages;
        t.unit = pl.unit;
        t.part = pl.split > 1 ? (float*)((char*)ws + whole.stage_bytes) : nullptr;
        hipError_t e;
        switch (c.op) {
            case MX_GEMM: e = pl.planes == 1 ? mx_launch_size<MX_GEMM, 1>(t, pl, st) : mx_launch_size<MX_GEMM, 3>(t, pl, st); break;
            case MX_GEMM_MX: e = mx_launch_size<MX_GEMM_MX, 1>(t, pl, st); break;
            default: e = pl.planes == 1 ? mx_launch_size<MX_GEMM_DX, 1>(t, pl, st) : mx_launch_size<MX_GEMM_DX, 3>(t, pl, st); break;
        }
        if (e != hipSuccess) return e;
        if (t.part) {
            const int64_t blocks = (rows * m + 255) / 256 / (m % 4 == 0 ? 4 : 1) + 1;  // four outputs a lane, or one
            hipLaunchKernelGGL(k_mx_join, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, t.part, pl.split,
                               rows, m, c.offsets, c.experts, t.y, (int)c.y_bf16);
            GQ_LAUNCH_CHECK();
        }
        t.A += rows * t.a_row;
        if (t.AS) t.AS += rows * t.sb;
        t.y = (char*)t.y + rows * m * (c.y_bf16 ? 2 : 4);
        return hipSuccess;
    };
    const int64_t head = c.offsets ? c.n : mx_head(whole, c.op, c.n, c.d_in, c.d_out);
    const hipError_t e = product(head);
    return e != hipSuccess || head == c.n ? e : product(c.n - head);
}

}  // namespace gq
