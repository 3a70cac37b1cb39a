// q4_grad.hpp -- the product of gradients with packed rows, shared by the linear
// layer's gradient and the experts' (gfx950).  The mathematics and what was
// measured stand in q4_grad.hip.
#pragma once

#include "q4_tile.hpp"

namespace bk {

template <int TA, int WJ = 4>
struct Grad {
    static constexpr int BT = 64 * TA;              // tokens of a workgroup
    static constexpr int BJ = 64 * WJ;              // columns of a workgroup of 2 WJ waves
    static constexpr int XBUF = BT * 128;           // bytes of a 64-row chunk of dy
    static constexpr int PITCH = 144;               // bytes of a column's 64 rows in LDS: 9 x 16, spreads the banks
    static constexpr int WBUF = BJ * PITCH;
    // Small tiles: a chunk is shorter than a load's latency, so codes and grids
    // come by direct loads too, some chunks ahead.  TA = 4: a chunk outlasts a
    // load, and LDS is what bounds it; codes and grids come to registers.  WJ = 2:
    // one chunk less ahead leaves room for two workgroups of a CU.
    static constexpr bool RAW = TA < 4;
    static constexpr int AHEAD = TA == 4 ? 1 : (TA == 2 ? 2 : 3) - (WJ == 2);
    static constexpr int NX = AHEAD + 1;
    static constexpr int XLOADS = BT / 8 / (2 * WJ);
    static constexpr int LOADS = XLOADS + (RAW ? 2 : 0);
    static constexpr int TILE = 1040;               // bytes of a code block in LDS: 65 x 16, spreads the banks
    static constexpr int GRIDS = 2 * WJ * TILE;     // codes [128 columns][row tile], then grids [row tile][64 columns][16]
    static constexpr int RAWBUF = RAW ? GRIDS + 512 * WJ : 0;   // of a chunk
    static constexpr int WEIGHTS = NX * XBUF, RAWS = WEIGHTS + 2 * WBUF, LDS = RAWS + NX * RAWBUF;
};

// Eight bytes to LDS byte address at + OFFSET.  Written out because the
// compiler would have every direct load in flight land before a store to LDS,
// whose target here is never theirs; tile_wait orders it before the barrier.
template <int OFFSET>
__device__ __forceinline__ void write64(uint32_t at, uint32_t lo, uint32_t hi)
{
    const uint64_t v = (uint64_t)hi << 32 | lo;
    asm volatile("ds_write_b64 %0, %1 offset:%2" ::"v"(at), "v"(v), "n"(OFFSET));
}

// What a thread of a chunk expands: 4 rows x 8 columns, as loaded.
struct GradRaw {
    uint32_t c[4];
    f32x4 g[2];   // (s, z) of rows 0, 1 and 2, 3
};

// One output tile: tokens t0 .. min(t0 + 64 TA, T) - 1 by columns 64 WJ bj ...
template <class X, int TA, int WJ = 4, int BYTES = Grad<TA, WJ>::LDS>
__device__ __forceinline__ void grad_tile(const uint16_t* __restrict__ dy, int64_t lddy, int t0, int T,
                                          const Q4Layer& w, uint16_t* __restrict__ dx, int64_t lddx, int bj,
                                          const TileShare& share)
{
    typedef Grad<TA, WJ> P;
    typedef typename X::vec vec;
    constexpr int BLOCKS = WJ / 2;   // of 128 columns
    static_assert(BYTES >= P::LDS);
    char(&lds)[BYTES] = tile_lds<BYTES>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, ml = lane & 31;
    const int wt = wave / WJ, wj = wave % WJ;
    const int j0 = bj * P::BJ;
    const int all = (w.m + 63) / 64;
    const int c0 = all * share.k / share.of, c1 = all * (share.k + 1) / share.of;   // this workgroup's chunks
    // what the weights of group g's columns are divided by; 1 where all are 0
    auto unit_of = [&](int g) {
        const float unit = w.unit[g];
        return unit > 0.f ? unit * X::kUnit : 1.f;
    };
    const int jw = j0 + wj * 64;   // the wave's columns, of one group
    const float unit = unit_of(min((WJ * bj + wj) / w.gb, w.G - 1));

    // staging of dy
    const Rsrc x = buffer_of(dy + (int64_t)t0 * lddy, 0x7FFFFFFFu);
    uint32_t x_at[P::XLOADS];
#pragma unroll
    for (int i = 0; i < P::XLOADS; ++i) {
        const int r = 8 * (wave * P::XLOADS + i) + (lane >> 3);
        x_at[i] = (uint32_t)(min(r, T - 1 - t0) * lddy * 2) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
    // load i of chunk c of dy, or (i = XLOADS, XLOADS + 1) of the codes and grids
    // of chunk c + 1, which is expanded a chunk before its products; row tiles
    // beyond RT repeat the last (dy is zero there)
    const uint32_t g_at = 128 * min((WJ * bj + 2 * (wave % BLOCKS) + (lane >> 5)) / w.gb, w.G - 1) + 4 * (lane & 31);
    auto stage = [&](int i, int c, int buf) {
        if (i < P::XLOADS) {
            load_lds16(x, x_at[i], 128 * min(c, c1 - 1), lds + buf * P::XBUF + (wave * P::XLOADS + i) * 1024);
        } else if (i == P::XLOADS) {
            const int64_t rt = min(4 * (c + 1) + (wave & 3), w.RT - 1);
            load_lds16(buffer_of(w.codes + (rt * w.KB + min(BLOCKS * bj + (wave >> 2), w.KB - 1)) * 64, 1024), 16 * lane, 0,
                       lds + P::RAWS + buf * P::RAWBUF + wave * P::TILE);
        } else {
            const int64_t rt = min(4 * (c + 1) + wave / BLOCKS, w.RT - 1);
            load_lds4(buffer_of(w.grid + rt * w.G * 16, 0x7FFFFFFFu), g_at, 0,
                      lds + P::RAWS + buf * P::RAWBUF + P::GRIDS + 256 * wave);
        }
    };

    // expansion: rows 4 a .. 4 a + 3 of the chunk, the eight columns of dword d
    // of unit column q of block kb
    const int a4 = lane & 15, d = lane >> 4, q = wave & 3;
    const int kb = min(BLOCKS * bj + (wave >> 2), w.KB - 1);
    const int g = min((2 * kb + (d >> 1)) / w.gb, w.G - 1);
    const float down = 1.f / unit_of(g);
    const int col = 128 * (wave >> 2) + 64 * (d >> 1) + 16 * q + 8 * (d & 1);
    const char* code_base = reinterpret_cast<const char*>(w.codes + (int64_t)kb * 64 + 16 * q);
    const char* grid_base = reinterpret_cast<const char*>(w.grid);
    const uint32_t code_lane = 64 * (a4 & 3) + 4 * d, grid_lane = 128 * g + 32 * (a4 & 3);
    const uint32_t w_at = (uint32_t)(uintptr_t)(lds_ptr)lds + P::WEIGHTS + col * P::PITCH + 8 * a4;
    auto fetch = [&](int c, GradRaw& v) {
        const int rt = min(4 * min(c, c1 - 1) + (a4 >> 2), w.RT - 1);
        const char* codes = code_base + ((int64_t)rt * w.KB * 1024 + code_lane);
        const char* grid = grid_base + ((int64_t)rt * w.G * 128 + grid_lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.c[i] = *reinterpret_cast<const uint32_t*>(codes + 16 * i);
        v.g[0] = *reinterpret_cast<const f32x4*>(grid);
        v.g[1] = *reinterpret_cast<const f32x4*>(grid + 16);
    };
    const uint32_t raw_code = P::RAWS + (4 * (wave >> 2) + (a4 >> 2)) * P::TILE + 256 * q + 64 * (a4 & 3) + 4 * d;
    const uint32_t raw_grid = P::RAWS + P::GRIDS + 128 * WJ * (a4 >> 2) + 128 * (2 * (wave >> 2) + (d >> 1)) + 32 * (a4 & 3);
    auto take = [&](int buf, GradRaw& v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.c[i] = *reinterpret_cast<const uint32_t*>(lds + raw_code + buf * P::RAWBUF + 16 * i);
        v.g[0] = *reinterpret_cast<const f32x4*>(lds + raw_grid + buf * P::RAWBUF);
        v.g[1] = *reinterpret_cast<const f32x4*>(lds + raw_grid + buf * P::RAWBUF + 16);
    };
    // column pair p of the four rows
    auto expand = [&](const GradRaw& v, int p, uint32_t s) {
        float f[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float step = v.g[i >> 1][2 * (i & 1)] * down, b = -step * v.g[i >> 1][2 * (i & 1) + 1];
            // two codes in bytes 0 and 2, which convert in one instruction each
            // (the empty statement hides that they are nibbles)
            uint32_t two = __builtin_rotateright32(v.c[i], 3 + 4 * p) & 0x000F000Fu;
            asm("" : "+v"(two));
            f[i][0] = fmaf(step, (float)(two & 0xFFu), b);
            f[i][1] = fmaf(step, (float)(two >> 16 & 0xFFu), b);
        }
        write64<0>(s + 2 * p * P::PITCH, X::down2(f[0][0], f[1][0]), X::down2(f[2][0], f[3][0]));
        write64<P::PITCH>(s + 2 * p * P::PITCH, X::down2(f[0][1], f[1][1]), X::down2(f[2][1], f[3][1]));
    };

    f32x16 acc[TA][2];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

    uint32_t x_lane[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) x_lane[v] = 128 * (32 * wt * TA + ml) + 16 * ((2 * v + h) ^ ((ml >> 1) & 7));
    const uint32_t b_lane = P::WEIGHTS + (64 * wj + ml) * P::PITCH + 16 * h;
    int bx = 0, px = P::AHEAD % P::NX;
    // Chunk c: its products, and the expansion of chunk c + 1 (from raw) between
    // them, while chunk c + 2 is fetched or further ones staged.
    auto chunk = [&](int c, int buf, GradRaw& raw, GradRaw& next) {
        // chunk c of dy and the weights of chunk c are in LDS for every wave,
        // and every wave is done with chunk c - 1
        tile_wait<(P::AHEAD - 1) * P::LOADS>();
        if (P::RAW) take(bx, raw);
        else fetch(c + 2, next);
        const char* xs = lds + bx * P::XBUF;
        const char* ws = lds + b_lane + buf * P::WBUF;
        const uint32_t to = w_at + (buf ^ 1) * P::WBUF;
        vec wf[2][2], xf[2][TA];
        auto read = [&](int v) {
#pragma unroll
            for (int b = 0; b < 2; ++b) wf[v & 1][b] = *reinterpret_cast<const vec*>(ws + 32 * v + 32 * b * P::PITCH);
#pragma unroll
            for (int a = 0; a < TA; ++a) xf[v & 1][a] = *reinterpret_cast<const vec*>(xs + x_lane[v] + 4096 * a);
        };
        read(0);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (v < 3) read(v + 1);
#pragma unroll
            for (int i = v; i < P::LOADS; i += 4) stage(i, c + P::AHEAD, px);
            expand(raw, v, to);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[a][b] = X::mfma32(xf[v & 1][a], wf[v & 1][b], acc[a][b]);
        }
        px = px + 1 == P::NX ? 0 : px + 1;
        bx = bx + 1 == P::NX ? 0 : bx + 1;
    };

    GradRaw raw[2];
    fetch(c0, raw[0]);
    if (!P::RAW) fetch(c0 + 1, raw[1]);
#pragma unroll
    for (int c = 0; c < P::AHEAD; ++c)
#pragma unroll
        for (int i = 0; i < P::LOADS; ++i) stage(i, c0 + c, c);
#pragma unroll
    for (int p = 0; p < 4; ++p) expand(raw[0], p, w_at);
    for (int c = c0; c < c1; c += 2) {
        chunk(c, 0, raw[1], raw[0]);
        if (c + 1 < c1) chunk(c + 1, 1, raw[0], raw[1]);
    }
    wait_direct_loads();
    const int tw = t0 + 32 * wt * TA;
    if (share.of > 1) {
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int t = tw + 32 * a + 8 * (r >> 2) + 4 * h + (r & 3), j = jw + 32 * b + ml;
                    if (t < T && j < w.n) share.part[t * share.ld + j] = unit * acc[a][b][r];
                }
        return;
    }
    __syncthreads();
    tile_store<X, TA>(acc, unit, lds + wave * kStoreBytes, tw, T, jw, w.n, dx, lddx);
}

}  // namespace bk
