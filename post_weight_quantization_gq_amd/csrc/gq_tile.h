// What tiled kernels share: asynchronous copies into LDS with their waits, and which tile a block has.
#pragma once
#include "gq_common.h"

#include <type_traits>

namespace gq {

typedef __attribute__((address_space(3))) void* tile_lds_t;

// At most N loads in flight, and this wave's LDS accesses done.  The copies into LDS are loads
// whose arrival only this counter tells, so no access moves across the wait.
template <int N>
__device__ __forceinline__ void tile_wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "a 6-bit counter");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
    asm volatile("" ::: "memory");
}

// lgkmcnt(0) alone
__device__ __forceinline__ void tile_wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ void tile_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// One wave copies 64 x 16 bytes into LDS from `dst` on; lane l's come from r at voff + soff
// (zeros out of r's range).
__device__ __forceinline__ void tile_dma(__amdgpu_buffer_rsrc_t r, u32x4* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (tile_lds_t)dst, 16, voff, soff, 0, 0);
}

// `rows` rows of `row` bytes from p on, the first `skip` bytes left out (none where `on` is
// false: every load reads zeros).  A tile's rows come to less than 2^31 bytes (256 of 2^20
// values in three planes), so 32 bits hold it, which the scalar unit compares and selects.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const uint8_t* p, int rows, int64_t row, bool on = true, int skip = 0) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, on ? rows * (int)row - skip : 0, 0x00020000);
}

// Rows of expert e, clamped to [0, n].
__device__ __forceinline__ void tile_expert_rows(const int64_t* offsets, int e, int64_t n, int64_t& lo,
                                               int64_t& hi) {
    lo = offsets[e];
    hi = offsets[e + 1];
    lo = lo < 0 ? 0 : (lo > n ? n : lo);
    hi = hi < 0 ? 0 : (hi > n ? n : hi);
}

struct TilePlace {
    int e;
    int64_t t0;                   // first row of the tile
    int rows;                     // rows of it
    int col;                      // column tile
    bool ok;
};

// Tiles of bm rows that expert e's rows make, the first `skip` left out.
template <class P>
__device__ __forceinline__ int tile_row_tiles(const P& p, int bm, int e, int skip = 0) {
    if (e >= p.experts) return 0;
    int64_t lo, hi;
    tile_expert_rows(p.offsets, e, p.n, lo, hi);
    lo += (int64_t)skip * bm;
    return hi > lo ? (int)((hi - lo + bm - 1) / bm) : 0;
}

// Row tile `row` of the experts' (without the first `skip` of each) in their order, counted from
// the offsets by each wave for itself, 64 experts at a time; not ok past the last one.
template <class P>
__device__ __forceinline__ void tile_of_row(const P& p, int bm, int row, TilePlace& r, int skip = 0) {
    const int lane = threadIdx.x & 63;
    r.ok = false;
    int first = 0;
    for (int b = 0; b < p.experts; b += 64) {
        const int c = tile_row_tiles(p, bm, b + lane, skip);
        if (skip && !__ballot(c > 0)) continue;
        int s = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(s, o, 64);
            if (lane >= o) s += v;
        }
        const unsigned long long hit = __ballot(first + s > row);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            r.e = __builtin_amdgcn_readfirstlane(b + l);
            const int before = __builtin_amdgcn_readfirstlane(first + __shfl(s - c, l, 64));
            int64_t lo, hi;
            tile_expert_rows(p.offsets, r.e, p.n, lo, hi);
            r.t0 = lo + (int64_t)(skip + row - before) * bm;
            r.rows = (int)(hi - r.t0 < bm ? hi - r.t0 : bm);
            r.ok = row >= before && r.rows > 0;     // (offsets out of order could count wrongly)
            return;
        }
        first += __builtin_amdgcn_readfirstlane(__shfl(s, 63, 64));
    }
}

// Block hw -> its tile.  XCD x (= hw % 8) takes a contiguous eighth of the tiles, which run
// row-tile fastest within groups of 8 row tiles, so the blocks that one L2 serves at a time
// share both operands.
template <class P>
__device__ __forceinline__ TilePlace tile_place(const P& p, int bm, int ncol) {
    TilePlace r;
    r.ok = false;
    int64_t nrow;
    if (p.offsets) {
        int c = 0;
        for (int b = 0; b < p.experts; b += 64) c += tile_row_tiles(p, bm, b + (threadIdx.x & 63));
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) c += __shfl_xor(c, o, 64);
        nrow = __builtin_amdgcn_readfirstlane(c);
    } else {
        nrow = (p.n + bm - 1) / bm;
    }
    const int64_t total = nrow * ncol, eighth = (total + 7) / 8;
    const int64_t in = blockIdx.x >> 3, lin = (int64_t)(blockIdx.x & 7) * eighth + in;
    if (in >= eighth || lin >= total) return r;
    constexpr int H = 8;
    const int64_t g = lin / (H * ncol), rest = lin - g * (H * ncol);
    const int64_t left = nrow - g * H;
    const int64_t h = left < H ? left : H;
    const int64_t row = g * H + rest % h;
    r.col = (int)(rest / h);
    if (p.offsets) {
        tile_of_row(p, bm, (int)row, r);
        return r;
    }
    r.e = 0;
    r.t0 = row * bm;
    r.rows = (int)(p.n - r.t0 < bm ? p.n - r.t0 : bm);
    r.ok = true;
    return r;
}

// f(integral_constant 0) .. f(integral_constant N - 1)
template <int N, class F>
__device__ __forceinline__ void tile_each(F f) {
    if constexpr (N > 0) {
        tile_each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

}  // namespace gq
