// q4_prompt.hpp -- the product of many tokens with packed rows, shared by the
// linear layer and the experts' products (gfx950).  The mathematics and what was
// measured stand in q4_prompt.hip.
#pragma once

#include "q4_few.hpp"
#include "q4_tile.hpp"

namespace bk {

// ---------------------------------------------------------------- group sums
//
// One wave per token: lanes sum 8 columns, 8 lanes a 64-column half (the loads
// of four spans of 512 columns together), and the halves of a piece are added
// in order.  COPY: the row goes to `copy` too, columns n .. 64 ceil(n / 64) - 1
// zero.  HBM bounds it: 33 us for 8192 x 8192 (4.1 TB/s), 5 for 2048 x 4096.
constexpr int kSumsHalves = BAKRON_MAX_DIM / 64;

// Pieces of the columns, in halves of 64: a group's first, second, ... kPiece,
// the last of them cut where the group ends.
constexpr int kPiece = 8;
__host__ __device__ __forceinline__ int pieces_of(int gb) { return (gb + kPiece - 1) / kPiece; }
__host__ __device__ __forceinline__ int piece_at(int half, int gb)   // the piece of a half
{
    return half / gb * pieces_of(gb) + half % gb / kPiece;
}

template <class X, bool COPY>
__global__ __launch_bounds__(256) void k_q4_sums(const uint16_t* __restrict__ x, int64_t ldx, int T, int n, int gb, int P,
                                                 float* __restrict__ sums, int64_t lds_, uint16_t* __restrict__ copy,
                                                 int64_t ldc)
{
    __shared__ float half[4][kSumsHalves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    const int halves = (n + 63) / 64;
    if (t >= T) return;
    const uint16_t* row = x + t * ldx;
    constexpr int U = 4;
    for (int c0 = 8 * lane; c0 < 64 * halves; c0 += 512 * U) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 512 * u;
            v[u] = u32x4{0u, 0u, 0u, 0u};
            if (c + 8 <= n) v[u] = *reinterpret_cast<const u32x4_any*>(row + c);
            else if (COPY && c < n) v[u] = few_x_cut(row, c, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 512 * u;
            if (COPY && c < 64 * halves) *reinterpret_cast<u32x4*>(copy + t * ldc + c) = v[u];
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) s += X::up((uint16_t)v[u][i]) + X::up((uint16_t)(v[u][i] >> 16));
            s += __shfl_xor(s, 1);
            s += __shfl_xor(s, 2);
            s += __shfl_xor(s, 4);
            if ((lane & 7) == 0 && c < 64 * halves) half[wave][c >> 6] = s;
        }
    }
    __builtin_amdgcn_wave_barrier();   // (a wave's own LDS row)
    const int per = pieces_of(gb);
    for (int p = lane; p < P; p += 64) {
        const int g = p / per, h0 = g * gb + (p - g * per) * kPiece;
        const int h1 = min(min(h0 + kPiece, (g + 1) * gb), halves);
        float s = 0.f;
        for (int h = h0; h < h1; ++h) s += half[wave][h];
        sums[(int64_t)p * lds_ + t] = s;
    }
}

// ------------------------------------------------------------------ product

template <int TA, int WR>
struct Prompt {
    static constexpr int BT = 64 * TA;                // tokens of a workgroup
    static constexpr int BR = 64 * WR;                // rows of W of a workgroup
    static constexpr int XBUF = BT * 128;             // bytes of a 64-column chunk of x
    static constexpr int WBUF = BR * 64;              // bytes of a 128-column block of codes
    // chunks in flight: LDS has no room for 3 of TA = 4, nor of two workgroups of
    // TA = WR = 2
    static constexpr int AHEAD = TA == 4 || (TA == 2 && WR == 2) ? 2 : 3;
    static constexpr int NX = AHEAD + 1, NW = (AHEAD + 1) / 2 + 2;
    static constexpr int XLOADS = BT / 8 / (2 * WR);  // direct loads of a wave per chunk of x (8 tokens each)
    static constexpr int LOADS = XLOADS + 2;          // one of the grid and one of codes
    static constexpr int GBUF = BR * 8;               // bytes of the grid entries of a chunk
    static constexpr int CODES = NX * XBUF, GRID = CODES + NW * WBUF, LDS = GRID + NX * GBUF;
    static_assert(XLOADS >= 1, "a wave stages at least eight tokens");
};

// The direct loads of a workgroup, chunk by chunk: tokens [t0, t0 + BT) x
// columns [64 c, 64 c + 64) of x (token r's 16-byte slot v holds columns
// 8 (v ^ ((r >> 1) & 7))), the grid entries of the rows for that chunk, and
// half of the codes of column block c / 2 + 1, which is needed two chunks on.
// Tokens beyond T and row tiles beyond RT read the last ones (their results
// are not stored); past the last chunk the last one is loaded again, into a
// buffer that no one reads, so that every chunk counts the same loads.
template <int TA, int WR>
struct PromptStage {
    typedef Prompt<TA, WR> P;
    Rsrc x, codes, grid;
    uint32_t x_at[P::XLOADS], code_at[2], grid_at;
    int chunks, blocks, G, gb, wave;   // the first chunk and block past this workgroup's
    int group, in_group;               // of the next chunk staged, and chunks of that group before it
    char* lds;

    __device__ __forceinline__ PromptStage(const uint16_t* xp, int64_t ldx, int t0, int T, const Q4Layer& w, int rt0,
                                           int kb0, int kb1, char* lds_)
        : x(buffer_of(xp + t0 * ldx, 0x7FFFFFFFu)),
          codes(buffer_of(w.codes + (int64_t)rt0 * w.KB * 64, 0x7FFFFFFFu)),
          grid(buffer_of(w.grid + (int64_t)rt0 * w.G * 16, 0x7FFFFFFFu)),
          chunks(min((w.n + 63) / 64, 2 * kb1)), blocks(kb1), G(w.G), gb(w.gb),
          wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), group(min(2 * kb0 / w.gb, w.G - 1)),
          in_group(2 * kb0 % w.gb), lds(lds_)
    {
        const int lane = threadIdx.x & 63;
        const int rts = w.RT - 1 - rt0;
#pragma unroll
        for (int i = 0; i < P::XLOADS; ++i) {
            const int r = 8 * (wave * P::XLOADS + i) + (lane >> 3);
            x_at[i] = (uint32_t)(min(r, T - 1 - t0) * ldx * 2) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) code_at[p] = (uint32_t)min(p * 2 * WR + wave, rts) * w.KB * 1024 + 16 * lane;
        grid_at = (uint32_t)min(2 * wave + (lane >> 5), rts) * w.G * 128 + 4 * (lane & 31);
    }
    // Quarter v of the loads of chunk c, called for c = 2 kb0, 2 kb0 + 1, ... in
    // turn; bx, bw: the buffers of chunk c and of column block c / 2 + 1; part =
    // c & 1.
    __device__ __forceinline__ void quarter(int v, int c, int bx, int bw, int part)
    {
        constexpr int PER = (P::XLOADS + 3) / 4;
        char* s = lds + bx * P::XBUF + wave * P::XLOADS * 1024;
#pragma unroll
        for (int i = v * PER; i < (v + 1) * PER; ++i)
            if (i < P::XLOADS) load_lds16(x, x_at[i], 128 * min(c, chunks - 1), s + 1024 * i);
        if (v == 2) {
            load_lds4(grid, grid_at, 128 * group, lds + P::GRID + bx * P::GBUF + 256 * wave);
            if (++in_group == gb) in_group = 0, group = min(group + 1, G - 1);
        }
        if (v == 3)
            load_lds16(codes, code_at[part], 1024 * min((c >> 1) + 1, blocks - 1),
                       lds + P::CODES + bw * P::WBUF + 1024 * (part * 2 * WR + wave));
    }
    // the codes of block kb0
    __device__ __forceinline__ void first(int kb0) const
    {
#pragma unroll
        for (int p = 0; p < 2; ++p)
            load_lds16(codes, code_at[p], 1024 * kb0, lds + P::CODES + 1024 * (p * 2 * WR + wave));
    }
};

// The three-term split of a float32 value into bfloat16, v = a + b + c.
__device__ __forceinline__ void split3(float v, uint32_t& a, uint32_t& b, uint32_t& c)
{
    a = Bf16::down(v);
    const float r = v - Bf16::up((uint16_t)a);
    b = Bf16::down(r);
    c = Bf16::down(r - Bf16::up((uint16_t)b));
}

// acc += z X for the wave's tiles and two pieces: lane half h of the MFMAs takes
// one of them, its lanes X of their tokens and z of their rows, slots X1 Z1,
// X1 Z2, X2 Z1, X1 Z3, X2 Z2, X3 Z1.
template <int TA>
__device__ __forceinline__ void zero_points(f32x16 (&acc)[TA][2], const float (&xs)[TA], const float (&z)[2])
{
    bf16x8 zf[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        uint32_t z1, z2, z3;
        split3(z[b], z1, z2, z3);
        const u32x4 v = {z1 | (z2 << 16), z1 | (z3 << 16), z2 | (z1 << 16), 0u};
        zf[b] = __builtin_bit_cast(bf16x8, v);
    }
#pragma unroll
    for (int a = 0; a < TA; ++a) {
        uint32_t x1, x2, x3;
        split3(xs[a], x1, x2, x3);
        const u32x4 v = {x1 | (x1 << 16), x2 | (x1 << 16), x2 | (x3 << 16), 0u};
        const bf16x8 xf = __builtin_bit_cast(bf16x8, v);
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[a][b] = Bf16::mfma32(xf, zf[b], acc[a][b]);
    }
}

// One output tile: tokens t0 .. min(t0 + 64 TA, T) - 1 by rows 64 WR br .. of W.
// OWN: the sums of x come from a product with ones.
template <class X, int TA, int WR, bool OWN, int BYTES = Prompt<TA, WR>::LDS>
__device__ __forceinline__ void prompt_tile(const uint16_t* __restrict__ x, int64_t ldx, int t0, int T,
                                            const Q4Layer& w, const float* __restrict__ sums, int64_t lds_,
                                            uint16_t* __restrict__ y, int64_t ldy, int br, const TileShare& share)
{
    typedef Prompt<TA, WR> P;
    typedef typename X::vec vec;
    static_assert(BYTES >= P::LDS);
    char(&lds)[BYTES] = tile_lds<BYTES>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, ml = lane & 31;
    const int wt = wave / WR, wr = wave % WR;
    const int rt0 = br * (P::BR / 16);
    const int kb0 = w.KB * share.k / share.of, kb1 = w.KB * (share.k + 1) / share.of;
    PromptStage<TA, WR> stage(x, ldx, t0, T, w, rt0, kb0, kb1, lds);
    stage.first(kb0);
#pragma unroll
    for (int c = 0; c < P::AHEAD; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) stage.quarter(v, 2 * kb0 + c, c, ((c >> 1) + 1) % P::NW, c & 1);

    f32x16 acc[TA][2];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
    f32x16 sx[OWN ? TA : 1];   // sums of x over the piece so far, in every column of the tile
    const vec ones = q4_ones<X>();
    if (OWN) {
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int r = 0; r < 16; ++r) sx[a][r] = 0.f;
    }

    u32x4 codes[2][2];   // [row tile pair][unit h, h + 2]
    f32x2 sz[2] = {f32x2{1.f, 0.f}, f32x2{1.f, 0.f}};   // of the group whose steps the accumulators count in
    int in_group = 2 * kb0 % w.gb;   // chunks of that group up to the end of the present piece
    int left = 0;                    // and chunks left of the piece
    // Two pieces' zero points come off together: `open` says that the first of
    // them has ended, z_open is its -(16 + z) in units of the present step, xs
    // the X of both (lane half h's of piece `pair` + h), loaded when the first
    // begins.  A piece belongs to the split that it ends in.
    bool open = false;
    float z_open[2] = {0.f, 0.f}, xs[TA];
    int pair = piece_at(2 * kb0, w.gb);
    const int pieces = piece_at((w.n - 1) / 64, w.gb) + 1;
    const float* x_sums = sums + t0 + 32 * wt * TA + ml;
    auto load_sums = [&]() {
#pragma unroll
        for (int a = 0; a < TA; ++a) xs[a] = x_sums[min(pair + h, pieces - 1) * lds_ + 32 * a];
    };
    if (!OWN) load_sums();
    int bx = 0, bw = 0;                                  // buffers of chunk c and block kb
    int px = P::AHEAD, pw = (P::AHEAD / 2 + 1) % P::NW;   // and of the ones staged beside them
    // the lane's parts of the LDS addresses
    uint32_t x_lane[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
        x_lane[v] = 128 * (32 * wt * TA + ml) + 16 * ((4 * (v >> 1) + 2 * h + (v & 1)) ^ ((ml >> 1) & 7));
    const uint32_t w_lane = P::CODES + 1024 * (4 * wr + (ml >> 4)) + 256 * h + 16 * (ml & 15);
    const uint32_t g_lane = P::GRID + 8 * (64 * wr + ml);
    for (int kb = kb0; kb < kb1; ++kb) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c = 2 * kb + half;
            if (c < stage.chunks) {
                tile_wait<(P::AHEAD - 1) * P::LOADS>();
                if (half == 0) {
                    const char* s = lds + w_lane + bw * P::WBUF;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            codes[b][u] = *reinterpret_cast<const u32x4*>(s + 2048 * b + 512 * u);
                }
                // fragments of x PRE steps before their products: an LDS read
                // takes longer than a step of a small TA
                constexpr int PRE = TA == 4 ? 1 : 3;
                const char* s = lds + bx * P::XBUF;
                vec xf[PRE + 1][TA];
#pragma unroll
                for (int v = 0; v < PRE; ++v)
#pragma unroll
                    for (int a = 0; a < TA; ++a) xf[v][a] = *reinterpret_cast<const vec*>(s + x_lane[v] + 4096 * a);
                if (left == 0) {
                    // the end of a piece (or the start): its zero points, and
                    // where its group ends too, the next one's steps
                    const bool first = c == 2 * kb0, change = first || in_group == w.gb;
                    f32x2 s1[2];
                    float z[2], ratio[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        s1[b] = *reinterpret_cast<const f32x2*>(lds + g_lane + bx * P::GBUF + 256 * b);
                        z[b] = -(sz[b].y + kQ4Offset);
                    }
                    if (!OWN && !first) {
                        if (open) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) z[b] = h ? z[b] : z_open[b];
                            zero_points<TA>(acc, xs, z);
                            pair += 2;
                            load_sums();
                        } else {
#pragma unroll
                            for (int b = 0; b < 2; ++b) z_open[b] = z[b];
                        }
                        open = !open;
                    }
                    if (change && !first) in_group = 0;
                    if (OWN || change) {   // (OWN: one body for both; its code is read anew by every short launch)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            ratio[b] = change ? sz[b].x * __builtin_amdgcn_rcpf(s1[b].x) : 1.f;
                            sz[b] = s1[b];   // (unchanged within a group)
                            z_open[b] *= ratio[b];
#pragma unroll
                            for (int a = 0; a < TA; ++a)
#pragma unroll
                                for (int r = 0; r < 16; ++r)
                                    acc[a][b][r] = (OWN ? fmaf(z[b], sx[a][r], acc[a][b][r]) : acc[a][b][r]) * ratio[b];
                        }
                    }
                    if (OWN) {
#pragma unroll
                        for (int a = 0; a < TA; ++a)
#pragma unroll
                            for (int r = 0; r < 16; ++r) sx[a][r] = 0.f;
                    }
                    left = min(kPiece - in_group % kPiece, w.gb - in_group);
                    in_group += left;
                }
                --left;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (v + PRE < 4) {
#pragma unroll
                        for (int a = 0; a < TA; ++a)
                            xf[(v + PRE) % (PRE + 1)][a] =
                                *reinterpret_cast<const vec*>(s + x_lane[(v + PRE) % 4] + 4096 * a);
                    }
                    vec wf[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) wf[b] = X::codes(codes[b][v >> 1][2 * half + (v & 1)]);
                    // a quarter of the next loads, and then the products as one
                    // run: 4 % over all loads first and the compiler's order
                    stage.quarter(v, c + P::AHEAD, px, pw, (half + P::AHEAD) & 1);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int a = 0; a < TA; ++a) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) acc[a][b] = X::mfma32(xf[v % (PRE + 1)][a], wf[b], acc[a][b]);
                        if (OWN) sx[a] = X::mfma32(xf[v % (PRE + 1)][a], ones, sx[a]);
                    }
                }
                px = px + 1 == P::NX ? 0 : px + 1;
                if ((half + P::AHEAD) & 1) pw = pw + 1 == P::NW ? 0 : pw + 1;
                bx = bx + 1 == P::NX ? 0 : bx + 1;
            }
        }
        bw = bw + 1 == P::NW ? 0 : bw + 1;
    }
    const bool ended = left == 0 || kb1 == w.KB;   // the last piece
    if (!OWN && (open || ended)) {
        float z[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float last = ended ? -(sz[b].y + kQ4Offset) : 0.f;
            z[b] = open ? (h ? last : z_open[b]) : (h ? 0.f : last);
        }
        zero_points<TA>(acc, xs, z);
    }
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[a][b][r] = (OWN ? fmaf(-(sz[b].y + kQ4Offset), sx[a][r], acc[a][b][r]) : acc[a][b][r]) * sz[b].x;
    wait_direct_loads();
    const int tw = t0 + 32 * wt * TA, rw = br * P::BR + wr * 64;
    if (share.of > 1) {
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int t = tw + 32 * a + 8 * (r >> 2) + 4 * h + (r & 3), row = rw + 32 * b + ml;
                    if (t < T && row < w.m) share.part[t * share.ld + row] = acc[a][b][r];
                }
        return;
    }
    __syncthreads();
    tile_store<X, TA>(acc, 1.f, lds + wave * kStoreBytes, tw, T, rw, w.m, y, ldy);
}

}  // namespace bk
