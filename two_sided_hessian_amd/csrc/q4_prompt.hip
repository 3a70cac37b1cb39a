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
#include "q4_prompt.hpp"

namespace bk {

// The tiles of a launch; gridDim.y workgroups share a tile's columns.
template <class X, int TA, int WR, bool OWN>
__global__ __launch_bounds__(128 * WR, 2) void k_q4_prompt(const uint16_t* __restrict__ x, int64_t ldx, int T, Q4Layer w,
                                                           const float* __restrict__ sums, int64_t lds_,
                                                           uint16_t* __restrict__ y, int64_t ldy, int nt, int nr,
                                                           float* __restrict__ part)
{
    typedef Prompt<TA, WR> P;
    int bt, br;
    tile_of(nt, nr, bt, br);
    prompt_tile<X, TA, WR, OWN>(x, ldx, bt * P::BT, T, w, sums, lds_, y, ldy, br,
                                TileShare{(int)blockIdx.y, (int)gridDim.y, part + (int64_t)blockIdx.y * T * w.m, w.m});
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
