// q4_tile.hpp -- what the two products over many tokens (the layer and its
// input gradient) share: the order of output tiles, waits on staged chunks
// and the store of a wave's results (gfx950).
#pragma once

#include "q4.hpp"

namespace bk {

constexpr int kStoreBytes = 32 * 72 * 2;   // LDS of a wave in tile_store

// The LDS of a workgroup whose tile bodies need BYTES at most: one array,
// however many bodies a kernel chooses from.
template <int BYTES>
__shared__ __align__(16) char tile_lds[BYTES];

// Waits until at most `left` loads of this wave are in flight (they complete
// in order), then for the other waves.
template <int LEFT>
__device__ __forceinline__ void tile_wait()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// Which part of a tile's depth a workgroup takes: part k of `of`.  More than one of
// them write float32 partial sums instead of results, token t and column j at
// part[t ld + j].
struct TileShare {
    int k, of;
    float* part;
    int64_t ld;
};

// Workgroups are dealt to the eight XCDs round-robin; each XCD gets a
// contiguous run of the tile order below, so that its L2 sees few tokens and
// rows at a time: runs of 4 token blocks share their rows of W.
__device__ __forceinline__ void tile_at(unsigned b, int nt, int nr, int& bt, int& br)
{
    const unsigned total = (unsigned)nt * nr;
    const unsigned per = total / 8, rest = total % 8, xcd = b % 8;
    const unsigned p = xcd * per + min(xcd, rest) + b / 8;
    const unsigned band = 4u * nr, g = p / band;
    const unsigned h = min(4u, (unsigned)nt - 4 * g);
    bt = (int)(4 * g + (p - g * band) % h);
    br = (int)((p - g * band) / h);
}
__device__ __forceinline__ void tile_of(int nt, int nr, int& bt, int& br) { tile_at(blockIdx.x, nt, nr, bt, br); }

// Results through LDS, 32 tokens x 64 columns of a wave at a time, so that
// they leave as 16-byte stores (to any address); cut rows leave one by one.  acc:
// 32-token x 32-column MFMA tiles, times f.  `lds`: 4608 bytes of the wave's
// own, which no one else may touch any more.
template <class X, int TA>
__device__ __forceinline__ void tile_store(const f32x16 (&acc)[TA][2], float f, char* lds, int t0, int T, int col0,
                                           int cols, uint16_t* __restrict__ y, int64_t ldy)
{
    const int lane = threadIdx.x & 63, h = lane >> 5, ml = lane & 31;
    uint16_t* out = reinterpret_cast<uint16_t*>(lds);   // pitch 72: spread banks
#pragma unroll
    for (int a = 0; a < TA; ++a) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                out[(8 * (r >> 2) + 4 * h + (r & 3)) * 72 + 32 * b + ml] = X::down(f * acc[a][b][r]);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tl = 8 * i + (lane >> 3), c = 8 * (lane & 7);
            const u32x4 v = *reinterpret_cast<const u32x4*>(out + tl * 72 + c);
            const int t = t0 + 32 * a + tl, col = col0 + c;
            if (t >= T) continue;
            uint16_t* dst = y + (int64_t)t * ldy + col;
            if (col + 8 <= cols) {
                *reinterpret_cast<u32x4_any*>(dst) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (col + e < cols) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Host: which of the tile shapes a product over `depth` terms takes, and over
// how many workgroups each tile's terms are shared out: the choice that leaves
// the busiest CU the least time.  That is the tiles it gets times a tile's cost,
// and for shared tiles a launch that joins them and their partial sums' way
// through memory (at 4 TB/s, there and back).
struct TileShape {
    int tokens, cols;
    double us;   // 4096 terms of a tile, the chip full of them
};
struct TileChoice {
    int shape, splits;
};
template <int N>
inline TileChoice tile_choose(const TileShape (&shapes)[N], int64_t T, int64_t cols, int64_t depth, int64_t most)
{
    TileChoice best = {0, 1};
    double least = 0.0;
    for (int i = 0; i < N; ++i) {
        const int64_t tiles = ceil_div(T, shapes[i].tokens) * ceil_div(cols, shapes[i].cols);
        for (int s = 1; s == 1 || (s <= most && tiles * s <= 1024); ++s) {
            const double us = ceil_div(tiles * s, 256) * shapes[i].us * depth / (4096.0 * s) +
                              (s > 1 ? 2.0 + 8.0e-6 / 4 * s * T * cols : 0.0);
            if (least == 0.0 || us < least) least = us, best = {i, s};
        }
    }
    return best;
}

// A padded copy of x (T x n, n rounded up to 64 columns, zeros beyond n).
template <class X>
void copy_enqueue(const uint16_t* x, int64_t ldx, int64_t T, int n, uint16_t* copy, int64_t ldc, hipStream_t s);

// y (T x m) = the sum of `splits` float32 results part[split][t][m], in order.
template <class X>
void join_enqueue(const float* part, int splits, int64_t T, int m, uint16_t* y, int64_t ldy, hipStream_t s);

}  // namespace bk
