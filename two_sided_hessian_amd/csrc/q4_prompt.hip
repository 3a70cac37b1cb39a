// q4_prompt.hip -- y = x W^T on 4-bit codes for many tokens (gfx950).
//
// Mathematics (q4.hpp): with u = 16 + c,
//     y_ti = sum_g s_ig sum_{j in g} u_ij x_tj  -  sum_g s_ig (16 + z_ig) X_tg,   X_tg = sum_{j in g} x_tj.
// The first sum runs on 16-bit MFMAs with exact operands.  Its accumulators
// are kept in units of the current group's step: on entering group g they are
// multiplied by s_{g-1} / s_g, one float32 multiplication each, so a group
// needs no second set of accumulators.  The zero points come off piece by
// piece, a piece being a group or 512 columns of a longer one: sums of (16 + c) x
// grow with the mean of x where the result does not, and every float32
// rounding, those of the steps' ratios among them, is one of the sum not yet
// taken off (x of a mean of two deviations, 2048 x 8192 x 16384 in groups of
// 128: an error of 5e-6 of the rms result, and 4e-4 with all zero points at
// the end; one grid per row: 4e-6 and 5e-5).  They enter in one of two ways:
//   * large tiles: X and 16 + z are split into three bfloat16 terms each and the
//     six leading products of a piece are six K slots of the same MFMAs (error
//     2^-24 of a term), two pieces at a time.  k_q4_sums makes X in a pass over
//     x of its own.
//   * small tiles, which do not fill the matrix cores: X comes from a product
//     with ones beside the others.
// Where x's rows are not 16-byte aligned or n is not a multiple of 64, the pass
// over x also makes a padded copy that the product can stage directly.
//
// k_q4_prompt: a workgroup of 2 x WR waves computes 64 TA tokens x 64 WR rows
// of W; a wave owns 32 TA tokens x 64 rows as TA x 2 MFMA tiles of 32 x 32
// (v_mfma_f32_32x32x16, tokens are its rows).  x goes through LDS in chunks
// of 64 columns by direct loads, 16-byte slots permuted so that fragment
// reads spread over the banks.  Codes come through LDS as they are (a quarter
// of the bytes of 16-bit weights); each wave expands its fragments in
// registers, 7 operations per 8 codes.  Two or three chunks are in flight at
// any time: a chunk's products take less than a load's latency.  Few tiles
// share out their columns over several workgroups, joined by k_q4_join.
//
// Measured, in the rate of 2 T m n (a large 16-bit product of the vendor's
// library reaches 1240 TFLOP/s): 8192 tokens x 8192 x 8192, one grid per row,
// 777 - 830 us, 1320 - 1410 TFLOP/s; in groups of 128, 910 - 935 us, 1180 - 1210;
// 2048 x 4096 x 4096, groups of 128, 72 - 78 us, 880 - 950; 777 x 4099 x 2050,
// groups of 64, unaligned, 34.6 - 36 us, 360 - 380.  MFMAs bound it, and the power
// limit their clock (1.9 GHz): of the cycles in which a CU has work they take
// 0.75 in the 8192 case and 0.52 in the 2048 one (TA = 2), where vector
// instructions (expansion, MFMA issue) take 0.52 too.  Groups of 64 change the
// accumulators' step at every chunk, 128 at every other: 12 % of the 8192 case.
#include <algorithm>

#include "../../include/bakron_q4.h"
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

// OWN: the sums of x come from a product with ones.  blockIdx.y of gridDim.y
// shares the columns; more than one of them writes float32 partial sums to
// part[blockIdx.y][token][row] instead of y.
template <class X, int TA, int WR, bool OWN>
__global__ __launch_bounds__(128 * WR, 2) void k_q4_prompt(const uint16_t* __restrict__ x, int64_t ldx, int T, Q4Layer w,
                                                           const float* __restrict__ sums, int64_t lds_,
                                                           uint16_t* __restrict__ y, int64_t ldy, int nt, int nr,
                                                           float* __restrict__ part)
{
    typedef Prompt<TA, WR> P;
    typedef typename X::vec vec;
    __shared__ __align__(16) char lds[P::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, ml = lane & 31;
    const int wt = wave / WR, wr = wave % WR;
    int bt, br;
    tile_of(nt, nr, bt, br);
    const int t0 = bt * P::BT, rt0 = br * (P::BR / 16);
    const int kb0 = w.KB * blockIdx.y / gridDim.y, kb1 = w.KB * (blockIdx.y + 1) / gridDim.y;
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
    if (gridDim.y > 1) {
        float* p = part + (int64_t)blockIdx.y * T * w.m;
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int t = tw + 32 * a + 8 * (r >> 2) + 4 * h + (r & 3), row = rw + 32 * b + ml;
                    if (t < T && row < w.m) p[(int64_t)t * w.m + row] = acc[a][b][r];
                }
        return;
    }
    __syncthreads();
    tile_store<X, TA>(acc, 1.f, lds + wave * kStoreBytes, tw, T, rw, w.m, y, ldy);
}

// y = the sum of `splits` partial results, in order; blockIdx.x is the token,
// eight loads are in flight.
template <class X>
__global__ __launch_bounds__(256) void k_q4_join(const float* __restrict__ part, int splits, int T, int m,
                                                 uint16_t* __restrict__ y, int64_t ldy)
{
    const int col = blockIdx.y * 256 + threadIdx.x;
    if (col >= m) return;
    const int64_t all = (int64_t)T * m;
    const float* p = part + (int64_t)blockIdx.x * m + col;
    constexpr int U = 8;
    float v = 0.f;
    for (int u0 = 0; u0 < splits; u0 += U) {
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = p[min(u0 + u, splits - 1) * all];
#pragma unroll
        for (int u = 0; u < U; ++u) v += u0 + u < splits ? a[u] : 0.f;
    }
    y[blockIdx.x * ldy + col] = X::down(v);
}

template <class X>
void join_enqueue(const float* part, int splits, int64_t T, int m, uint16_t* y, int64_t ldy, hipStream_t s)
{
    launch(nullptr, KK_Q4_JOIN, 0.0, 4.0 * splits * T * m, k_q4_join<X>, dim3((unsigned)T, (unsigned)ceil_div(m, 256)),
           dim3(256), s, part, splits, (int)T, m, y, ldy);
}
template void join_enqueue<Bf16>(const float*, int, int64_t, int, uint16_t*, int64_t, hipStream_t);
template void join_enqueue<Fp16>(const float*, int, int64_t, int, uint16_t*, int64_t, hipStream_t);

// --------------------------------------------------------------------- host

// How a problem is cut: TA, WR and the workgroups that share a tile's columns.
struct PromptPlan {
    int TA, WR, splits;
    int pieces;
    int64_t lds_, ldc;
    size_t sums, copy, part, bytes;
};

static PromptPlan prompt_plan(int64_t T, int64_t m, int64_t n, int gb)
{
    PromptPlan p;
    // Costs: 4096 tokens x 4096 rows in tiles of 256 x 256 take 128 us, 2048 in
    // 128 x 256 80, 1024 in 128 x 128 49 and 2048 82, 512 in 64 x 128 36.  A large
    // tile expands a code for more tokens; a smaller one wins where the large
    // ones are too few, or a few too many: 3500 tokens x 2500 rows x 3500, 280
    // tiles of 128 x 256, takes 102 us and 87 in 560 of 128 x 128.  A split has two
    // column blocks at least (65 tokens x 4096 x 4096: 16 us with 4 splits, 33
    // without; 128 tokens x 1024 x 1024: 8.5 us with 4, 10.0 with 2).
    static constexpr TileShape shapes[] = {{256, 256, 128.0}, {128, 256, 80.0}, {128, 128, 42.0}, {64, 128, 28.0}};
    const TileChoice c = tile_choose(shapes, T, m, n, std::min<int64_t>(8, ceil_div(n, kQ4Cols) / 2));
    p.TA = shapes[c.shape].tokens / 64;
    p.WR = shapes[c.shape].cols / 64;
    p.splits = c.splits;
    p.lds_ = ceil_div(T, 256) * 256;
    p.ldc = ceil_div(n, 64) * 64;
    p.sums = 0;
    p.pieces = piece_at((int)((n - 1) / 64), gb) + 1;
    p.copy = align_up((size_t)p.lds_ * p.pieces * 4);
    p.part = p.copy + align_up((size_t)T * p.ldc * 2);
    p.bytes = p.part + (p.splits > 1 ? align_up((size_t)p.splits * T * m * 4) : 0);
    return p;
}

size_t q4_prompt_workspace_bytes(int64_t T, int64_t m, int64_t n, int gb) { return prompt_plan(T, m, n, gb).bytes; }

template <class X>
void copy_enqueue(const uint16_t* x, int64_t ldx, int64_t T, int n, uint16_t* copy, int64_t ldc, hipStream_t s)
{
    launch(nullptr, KK_Q4_SUMS, 0.0, 4.0 * T * n, k_q4_sums<X, true>, dim3((unsigned)ceil_div(T, 4)), dim3(256), s, x, ldx,
           (int)T, n, 1, 0, static_cast<float*>(nullptr), (int64_t)0, copy, ldc);
}
template void copy_enqueue<Bf16>(const uint16_t*, int64_t, int64_t, int, uint16_t*, int64_t, hipStream_t);
template void copy_enqueue<Fp16>(const uint16_t*, int64_t, int64_t, int, uint16_t*, int64_t, hipStream_t);

template <class X, int TA, int WR, bool OWN>
static void prompt_launch(const uint16_t* x, int64_t ldx, int64_t T, const Q4Layer& w, const float* sums, int64_t lds_,
                          uint16_t* y, int64_t ldy, int splits, float* part, hipStream_t s)
{
    typedef Prompt<TA, WR> P;
    const int nt = (int)ceil_div(T, P::BT), nr = (int)ceil_div(w.m, P::BR);
    launch(nullptr, KK_Q4_PROMPT, 2.0 * T * w.m * w.n, 0.0, k_q4_prompt<X, TA, WR, OWN>,
           dim3((unsigned)(nt * nr), (unsigned)splits), dim3(128 * WR), s, x, ldx, (int)T, w, sums, lds_, y, ldy, nt, nr, part);
}

template <class X>
static int prompt_run(const void* x, int64_t ldx, int64_t T, const Q4Layer& w, void* y, int64_t ldy, void* ws,
                      hipStream_t s)
{
    const PromptPlan p = prompt_plan(T, w.m, w.n, w.gb);
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    uint16_t* yp = static_cast<uint16_t*>(y);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(ws) + p.sums);
    uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + p.copy);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
    // (the staging offsets of a token block are 31 bits)
    const bool direct = w.n % 64 == 0 && ldx % 8 == 0 && ldx <= (1 << 21) && aligned16(x);
    // Small tiles make X themselves, unless there is a pass that copies and
    // enough of them that their arithmetic counts (900 tokens x 3500 x 3500, a
    // copy: 53 us with products of their own, 49 without; 100 x 300 x 5000,
    // eight splits: 16 and 20).
    const bool own = p.TA == 1 && (direct || p.splits > 1);
    if (!own)
        launch(nullptr, KK_Q4_SUMS, 0.0, 2.0 * T * w.n, direct ? k_q4_sums<X, false> : k_q4_sums<X, true>,
               dim3((unsigned)ceil_div(T, 4)), dim3(256), s, xp, ldx, (int)T, w.n, w.gb, p.pieces, sums, p.lds_, copy, p.ldc);
    else if (!direct) copy_enqueue<X>(xp, ldx, T, w.n, copy, p.ldc, s);
    if (!direct) xp = copy, ldx = p.ldc;
    if (p.TA == 4) prompt_launch<X, 4, 4, false>(xp, ldx, T, w, sums, p.lds_, yp, ldy, p.splits, part, s);
    else if (p.TA == 2 && p.WR == 2) prompt_launch<X, 2, 2, false>(xp, ldx, T, w, sums, p.lds_, yp, ldy, p.splits, part, s);
    else if (p.TA == 2) prompt_launch<X, 2, 4, false>(xp, ldx, T, w, sums, p.lds_, yp, ldy, p.splits, part, s);
    else if (own) prompt_launch<X, 1, 2, true>(xp, ldx, T, w, sums, p.lds_, yp, ldy, p.splits, part, s);
    else prompt_launch<X, 1, 2, false>(xp, ldx, T, w, sums, p.lds_, yp, ldy, p.splits, part, s);
    if (p.splits > 1) join_enqueue<X>(part, p.splits, T, w.m, yp, ldy, s);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int q4_prompt_enqueue(const void* x, int64_t ldx, int64_t T, bool bf16, const Q4Layer& w, void* y, int64_t ldy, void* ws,
                      hipStream_t s)
{
    return bf16 ? prompt_run<Bf16>(x, ldx, T, w, y, ldy, ws, s) : prompt_run<Fp16>(x, ldx, T, w, y, ldy, ws, s);
}

}  // namespace bk
