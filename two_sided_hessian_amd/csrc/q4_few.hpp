// q4_few.hpp -- the inner product of packed rows with a few tokens, shared by
// the linear layer and the expert layer (gfx950).
//
// Tokens are the rows of v_mfma_f32_16x16x32 and rows of W its columns, so the
// four results of a lane share one (s, z), and NT MFMA tiles of 16 tokens use
// each expanded code: with one token or sixteen the work is that of reading
// and expanding the codes.  A second product, with ones, gives the sums of x
// in the same layout.  What bounds it is HBM, and before that the latency of
// its loads: a wave issues the loads of U column blocks (codes, grids, x)
// together, and a workgroup's waves take the blocks of one row tile in turn,
// so that a row tile is finished in a few round trips.  U is small: more waves
// hide more than more loads of a wave, whose registers cost waves (the expert
// layer, 16 tokens, 6 of 64 experts of 2048 x 1024: 76 us, and 87 with twice
// the blocks in flight).
#pragma once

#include "q4.hpp"

namespace bk {

// x reaches the MFMA by way of LDS: read from memory as the fragment wants it,
// consecutive lanes would be different tokens, each its own cache line (11
// bytes a clock and CU measured); read along the rows, 16 lanes take a
// token's 256 bytes of a block and the four tokens of an instruction four
// runs.  The LDS rows are a wave's own, so no barrier is involved.

// Columns k .. k + 7 of a row of n, zeros beyond n; every load is made (of the
// last column where there is none), so that all are in flight together.
__device__ __forceinline__ u32x4 few_x_cut(const uint16_t* __restrict__ row, int k, int n)
{
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[min(k + i, n - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = k + i < n ? e[i] : 0u;
    return u32x4{e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
}

constexpr int kFewPitch = 272;   // bytes of a token's block in LDS: 256 + 16, spreads the banks
constexpr int few_lds(int TQ) { return (TQ < 4 ? 4 * TQ : 16) * kFewPitch; }   // bytes a wave needs

// acc[j][i][e] += sum over column blocks of row tile rt + j: s (u x - (16 + z) x)
// for token 16 i + 4 (lane >> 4) + e.  TQ: quads of tokens (1, 2, 4, 8 or 16).
// R row tiles share each fragment of x.  HALF: grids change within a block
// (groups of an odd multiple of 64).  Tiles beyond RT repeat the last; tokens
// beyond the wanted ones may be any valid row: those results are the caller's
// to drop.
template <class X, int TQ, int R, int U, bool HALF>
struct FewSpan {
    typedef typename X::vec vec;
    static constexpr int NT = TQ < 4 ? 1 : TQ / 4;
    static constexpr int NG = HALF ? 2 : 1;
    static constexpr int PER = TQ < 4 ? TQ : 4;   // quads of an MFMA tile
    const uint16_t* xr[TQ];   // the lane's row of quad t, token 4 t + (lane >> 4)
    const char* codes[R];     // uniform: the row tile's first block
    const char* grid[R];
    f32x4 acc[R][NT];
    int n, KB, G;
    uint32_t gm;
    char* lds;

    __device__ __forceinline__ FewSpan(char* wave_lds) : lds(wave_lds) {}
    // row tiles rt, rt + 1, ... of each of N layers of one shape, R = N times
    // so many
    template <int N>
    __device__ __forceinline__ void rows(const Q4Layer (&w)[N], int rt)
    {
        n = w[0].n, KB = w[0].KB, G = w[0].G, gm = w[0].gm;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t tile = min(rt + j % (R / N), w[0].RT - 1);
            codes[j] = reinterpret_cast<const char*>(w[j / (R / N)].codes + tile * KB * 64);
            grid[j] = reinterpret_cast<const char*>(w[j / (R / N)].grid + tile * G * 16);
        }
    }
    // the lane's token rows; clears the sums
    __device__ __forceinline__ void tokens(const uint16_t* const (&xs)[TQ])
    {
#pragma unroll
        for (int t = 0; t < TQ; ++t) xr[t] = xs[t];
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    struct Block {
        u32x4 c[R];
        f32x2 sz[R][NG];
        u32x4 x[TQ];
    };
    __device__ __forceinline__ void load_w(Block& b, int kb) const
    {
        const uint32_t lane = threadIdx.x & 63;
        uint32_t g[NG];
#pragma unroll
        for (int h = 0; h < NG; ++h) g[h] = 128u * (uint32_t)group_of(2 * kb + h, gm, G) + 8u * (lane & 15);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            b.c[j] = *reinterpret_cast<const u32x4*>(codes[j] + (1024u * (uint32_t)kb + 16u * lane));
#pragma unroll
            for (int h = 0; h < NG; ++h) b.sz[j][h] = *reinterpret_cast<const f32x2*>(grid[j] + g[h]);
        }
    }
    // a block of 128 columns that all exist
    __device__ __forceinline__ void load(Block& b, int kb) const
    {
        const int k = kb * 128 + 8 * (threadIdx.x & 15);
#pragma unroll
        for (int t = 0; t < TQ; ++t) b.x[t] = *reinterpret_cast<const u32x4_any*>(xr[t] + k);
        load_w(b, kb);
    }
    __device__ __forceinline__ void load_cut(Block& b, int kb) const
    {
        load_w(b, kb);
        const int k = kb * 128 + 8 * (threadIdx.x & 15);
#pragma unroll
        for (int t = 0; t < TQ; ++t) b.x[t] = few_x_cut(xr[t], k, n);
    }
    // on: 1, or 0 for a block that is not to count
    __device__ __forceinline__ void add(const Block& b, float on)
    {
        const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
        vec xf[NT][4];
        // (a wave's LDS operations complete in order: the next tile's writes
        // come after this one's reads)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int t = 0; t < PER; ++t)
                *reinterpret_cast<u32x4*>(lds + (4 * t + q) * kFewPitch + 16 * r) = b.x[PER * i + t];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int d = 0; d < 4; ++d)
                xf[i][d] = *reinterpret_cast<const vec*>(lds + min(r, 4 * PER - 1) * kFewPitch + 128 * (d >> 1) + 32 * q +
                                                         16 * (d & 1));
            __builtin_amdgcn_wave_barrier();
        }
        const vec ones = q4_ones<X>();
        f32x4 s[NT][NG];   // sums of x, per half block or block
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int h = HALF ? d >> 1 : 0;
                const bool fresh = HALF ? d % 2 == 0 : d == 0;
                s[i][h] = X::mfma16(xf[i][d], ones, fresh ? f32x4{0.f, 0.f, 0.f, 0.f} : s[i][h]);
            }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            vec wf[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) wf[d] = X::codes(b.c[j][d]);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < NG; ++h) {
                    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int d = 4 / NG * h; d < 4 / NG * (h + 1); ++d) t = X::mfma16(xf[i][d], wf[d], t);
                    const f32x2 g = b.sz[j][h];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[j][i][e] = fmaf(g.x * on, fmaf(-(g.y + kQ4Offset), s[i][h][e], t[e]), acc[j][i][e]);
                }
        }
    }
    // blocks first, first + by, ... below end
    __device__ __forceinline__ void run(int first, int by, int end)
    {
        const int whole = min(n / kQ4Cols, end), count = whole > first ? (whole - first + by - 1) / by : 0;
        for (int i = 0; i < count; i += U) {
            Block b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) load(b[u], first + by * min(i + u, count - 1));
            // every load before the first wait, and the blocks in the order of
            // their loads: left to itself the compiler waits for single ones
            // (32 tokens x 4096 x 4096: 8.5 us, so 7.1)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                add(b[u], i + u < count ? 1.f : 0.f);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (whole < end && whole >= first && (whole - first) % by == 0) {
            Block b;
            load_cut(b, whole);
            add(b, 1.f);
        }
    }
};

}  // namespace bk
