// How a product is done (gq_mm.hip), as the kernels of each element type take it (gq_mm_tile.h).
#pragma once
#include "gq_mm.h"

namespace gq {

// From sizes and types alone.
struct MmPlan {
    bool stream;                  // few rows a weight: waves that stream it
    int bm, bn, split, waves;     // rows and columns (of weights' rows: both of MM_GATE's) of a tile
    int stages, unit;
    bool join;                    // float32 sums first, outputs from them
    size_t pad_bytes, part_bytes; // copies of operands whose rows are no multiple of 8; sums
};

struct MmTile {
    const uint8_t* A[2];          // rows of the activations
    int64_t a_row, a_bytes;       // bytes from one to the next, and of one that count
    const void* AS;               // their scales, as_row bytes a row
    int64_t as_row;
    const uint8_t* W[2];
    int64_t w_row, w_bytes;
    const void* WS[2];            // ws_rows x ws_row scales a weight
    int64_t ws_row, ws_rows, ws_k;  // (and how many blocks the contraction has)
    const int64_t* offsets;
    int experts;
    int64_t n, m, d_out;          // rows, output columns, rows of one weight
    int stages, stages_one;       // stages of the contraction, and of the first of two pairs
    int unit;                     // a split's range is a multiple of this many stages
    void* y[2];
    int y_bf16, outs;             // (MM_TN: outputs wanted)
    float* z[2];
    uint8_t* hq;
    void* hs;
    int64_t hq_row, hs_row;       // bytes of a packed row, its scales
    int act;
    int past;                     // MM_GATE's h in bfloat16, MM_TN's outputs: stored past the caches' order
    float* part;                  // sums [split][n][m] (MM_GATE: [split][2][n][m], MM_TN:
                                  // [split][outs][experts][d_out][m]), or null
};

constexpr int MM_FIRST = 2;       // groups of 16 rows that an expert's own streaming blocks take

// A launch has fewer than 2^32 lanes.
constexpr int64_t MM_MAX_LANES = ((int64_t)1 << 32) - 1;

// Blocks of a launch of tiles, a multiple of the XCDs: with offsets every expert can have a part-empty one
inline int64_t mm_blocks(MmForm form, int64_t n, int64_t m, int64_t d_out, int experts, bool offsets, int outs, const MmPlan& P) {
    const int64_t cols = form == MM_GATE ? (m + P.bn / 2 - 1) / (P.bn / 2) : (m + P.bn - 1) / P.bn;
    const int64_t rows = form == MM_TN ? (d_out + P.bm - 1) / P.bm * experts * outs : (n + P.bm - 1) / P.bm + (offsets ? experts : 0);
    return (rows * cols + 7) / 8 * 8;
}

hipError_t mm_launch_bf16(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st);
hipError_t mm_launch_e8(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st);
hipError_t mm_launch_fs(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st);
hipError_t mm_launch_e8w(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st);
hipError_t mm_launch_fsw(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st);

}  // namespace gq
