// q4_experts.hip -- each expert's rows times its packed 4-bit layer, and the
// gradient with respect to the rows (gfx950).
//
//     y_p = W_e x_p,   dx_p = dy_p W_e,   offsets[e] <= p < offsets[e + 1]
//
// The products are the linear layer's (q4_few.hpp, q4_prompt.hpp, q4_grad.hpp);
// what is added is which rows meet which layer.  That is known on the device
// only, so a launch has as many blocks of rows as there can be (rows / 64 and
// one more per expert, say): each workgroup reads the offsets, counts the blocks
// of every expert, and takes its own by a prefix sum over the 64 lanes; what is
// past the last block ends there.  A block never holds two experts' rows.
//
//   * few rows per expert (decoding): codes are what is read, and HBM bounds the product.
//     k_q4_experts_few has blocks of up to 32 rows and row tiles of W over workgroups: 16
//     tokens, 6 of 64 experts of 1024 x 2048 in groups of 64: 13.0 us a call, 5.2 TB/s of
//     what has to move, a large copy's rate.  k_q4_experts_grad_few has blocks of 32 rows
//     (16) and 128 columns, and vector instructions bound it: 16 tokens, 2 of 8 of 14336 x 4096:
//     53 us with seven experts in use, 75 - 83 with all eight (floors 44 and 51); tiles of 64
//     rows took 117.  Blocks of 64 rows, two waves a SIMD: 92 us for 103 at 64 tokens, but
//     162 for 139 at 128 and 63 for 54 at 512 tokens, 6 of 64 of 2048 x 1024.
//   * many: k_q4_experts and k_q4_experts_grad, tiles of 64 .. 256 rows, MFMAs.  8192
//     tokens, 2 of 8 of 14336 x 4096: 1676 us and 31 for the rows' sums, 1150 TFLOP/s, MFMAs
//     busy 0.63 of a CU's cycles and vector instructions 0.46 (steps change every second
//     chunk in groups of 128).  Gradient, 2048 tokens: 555 us and 14 to join the
//     tiles that are shared out, MFMAs 0.49, LDS 0.45, vector instructions 0.37, and the rows
//     of tiles that experts' ends cut.  1024 tokens, 6 of 64 of 2048 x 1024, in tiles of
//     128 x 128, two workgroups a CU: 65 us with 40 to 230 rows each, 78 with 4 to 490, whose
//     700 tiles are 1.4 times what fits at once.
#include <algorithm>

#include "moe.hpp"
#include "q4_grad.hpp"
#include "q4_grad_few.hpp"
#include "q4_prompt.hpp"

namespace bk {

constexpr int kExperts = BAKRON_MOE_MAX_EXPERTS;
static_assert(kExperts <= 4 * 64, "four experts a lane");

// Sums of v over lanes 0 .. this one (DPP: shifts within rows of 16 lanes, then
// the rows' last lanes to the rows after them).
__device__ __forceinline__ int lanes_upto(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
}

// The first lane whose `upto` is above `want` (held below the last one's, so that there
// is one); the rest of want there.
__device__ __forceinline__ int lane_of(int upto, int sum, int& want)
{
    want = min(want, __builtin_amdgcn_readlane(upto, 63) - 1);
    const int l = __ffsll((unsigned long long)__ballot(upto > want)) - 1;
    want -= __builtin_amdgcn_readlane(upto - sum, l);
    return l;
}

// A lane's four experts: their first rows, held in [0, R].
struct ExpertLane {
    int o[5];
    __device__ __forceinline__ ExpertLane(const int32_t* __restrict__ offsets, int E, int R)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int u = 0; u < 5; ++u) o[u] = min(max(offsets[min(4 * lane + u, E)], 0), R);
    }
    __device__ __forceinline__ int rows(int u) const { return max(o[u + 1] - o[u], 0); }
};

// Rows of one expert: block k of those that `count` finds in lane l.
struct ExpertRows {
    int e, t0, t1;   // the expert, the block's first row, and the expert's end
};
template <class Count>
__device__ __forceinline__ int expert_at(const ExpertLane& lane, int l, int& k, Count count, ExpertRows& out)
{
    int u = 0;
#pragma unroll
    for (int v = 0; v < 3; ++v) {
        const int n = __builtin_amdgcn_readlane(count(lane.rows(v)), l);
        if (u == v && k >= n) k -= n, ++u;
    }
    int first = 0, last = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (u == v) first = __builtin_amdgcn_readlane(lane.o[v], l), last = __builtin_amdgcn_readlane(lane.o[v + 1], l);
    out = ExpertRows{4 * l + u, first, last};
    return u;
}

// The tiles of a launch.  An expert's rows go into blocks of 64 TA, the last one cut;
// what is cut takes a body for 128 or 64 rows where that is enough.  The order of
// tiles is that of their cost, bodies for more rows first, so that the short ones
// fill up what the long ones leave; `cls` is 0 for 64 TA rows, 1 for half of that, 2
// for a quarter.  nc: tiles beside each other.  A wave's work, the same in every wave.
template <int TA>
struct ExpertTiles {
    static constexpr int BT = 64 * TA;
    ExpertLane lane;
    int bigs, rest, bigs_upto, rest_upto;   // rest: halves, and quarters in the upper 16 bits
    int nb, nh, nq;

    static __device__ __forceinline__ int big(int c) { return c / BT + (TA == 1 ? c % BT > 0 : c % BT > BT / 2); }
    static __device__ __forceinline__ int half(int c) { return TA > 1 && c % BT > BT / 4 * (TA / 4) && c % BT <= BT / 2; }
    static __device__ __forceinline__ int quarter(int c) { return TA == 4 && c % BT > 0 && c % BT <= 64; }

    __device__ __forceinline__ ExpertTiles(const int32_t* __restrict__ offsets, int E, int R) : lane(offsets, E, R), bigs(0), rest(0)
    {
#pragma unroll
        for (int u = 0; u < 4; ++u) bigs += big(lane.rows(u)), rest += half(lane.rows(u)) | quarter(lane.rows(u)) << 16;
        bigs_upto = lanes_upto(bigs);
        rest_upto = lanes_upto(rest);
        nb = __builtin_amdgcn_readlane(bigs_upto, 63);
        nh = __builtin_amdgcn_readlane(rest_upto, 63) & 0xFFFF;
        nq = __builtin_amdgcn_readlane(rest_upto, 63) >> 16;
    }
    __device__ __forceinline__ int64_t count(int nc) const { return (int64_t)(nb + nh + nq) * nc; }
    __device__ __forceinline__ bool find(int64_t b, int nc, ExpertRows& rows, int& bc, int& cls) const
    {
        int bt;
        if (b < (int64_t)nb * nc) {
            cls = 0;
            tile_at((unsigned)b, nb, nc, bt, bc);
            const int l = lane_of(bigs_upto, bigs, bt);
            expert_at(lane, l, bt, big, rows);
            rows.t0 += bt * BT;
            return true;
        }
        b -= (int64_t)nb * nc;
        if (b < nh * nc) {
            cls = 1;
            tile_at((unsigned)b, nh, nc, bt, bc);
            const int l = lane_of(rest_upto & 0xFFFF, rest & 0xFFFF, bt);
            expert_at(lane, l, bt, half, rows);
        } else {
            b -= nh * nc;
            if (b >= nq * nc) return false;
            cls = 2;
            tile_at((unsigned)b, nq, nc, bt, bc);
            const int l = lane_of(rest_upto >> 16, rest >> 16, bt);
            expert_at(lane, l, bt, quarter, rows);
        }
        rows.t0 += (rows.t1 - rows.t0) / BT * BT;
        return true;
    }
};

// Long tiles on 256 CUs, one each: what is left over after whole rounds of them is
// shared out, each tile's depth over as many workgroups as end it soonest, and joined by
// k_q4_experts_tail.  (Whole numbers, so that both kernels find the same.)
constexpr int kTailCUs = 256, kTailParts = 16, kTailUnits = 512;
struct ExpertTail {
    int us;        // hundredths of one that a long tile takes; 0: no tile is shared out
    int deepest;   // parts of a tile at most
    int units;     // and of all of them, that there is room for (whatever the offsets say)
};
struct ExpertTailAt {
    int64_t whole;     // tiles before the tail
    int left, parts;   // of the tail, and workgroups of each
    __device__ __forceinline__ ExpertTailAt(int64_t tiles, const ExpertTail& tail) : whole(tiles), left((int)(tiles % kTailCUs)), parts(1)
    {
        whole -= left;
        int best = tail.us;
        for (int s = 2; s <= tail.deepest && left * s <= tail.units; ++s) {
            // (a launch, and 256 KB there and back at 5.8 TB/s for each part)
            const int us = (left * s + kTailCUs - 1) / kTailCUs * tail.us / s + 200 + 9 * left * s;
            if (us < best) best = us, parts = s;
        }
    }
};

// This workgroup's tile, and its part of it: with a tail that is shared out, or
// (blockIdx.y of gridDim.y) every tile alike.  part: R x cols float32 sums a part, or
// 64 TA x width ones a unit of the tail.
template <int TA>
__device__ __forceinline__ bool expert_tile(const int32_t* __restrict__ offsets, int E, int R, int nc, int cols, int width,
                                            const ExpertTail& tail, float* part, ExpertRows& rows, int& bc, int& cls,
                                            TileShare& share)
{
    const ExpertTiles<TA> tiles(offsets, E, R);
    int64_t b = blockIdx.x;
    int unit = -1;
    share = TileShare{(int)blockIdx.y, (int)gridDim.y, part + (int64_t)blockIdx.y * R * cols, cols};
    if (TA == 4 && tail.us) {
        const ExpertTailAt at(tiles.count(nc), tail);
        if (b >= at.whole && at.parts > 1) {
            unit = (int)(b - at.whole);
            if (unit >= at.left * at.parts) return false;
            share.k = unit / at.left;
            share.of = at.parts;
            b = at.whole + unit % at.left;
        }
    }
    if (!tiles.find(b, nc, rows, bc, cls)) return false;
    if (unit >= 0) {
        share.part = part + ((int64_t)unit * 64 * TA - rows.t0) * width - bc * width;
        share.ld = width;
    }
    return true;
}

// Tiles of up to 64 TA rows by 64 WR of W.  OWN (WR = 2): the rows' sums are made beside the products (q4_prompt.hpp).
template <class X, int TA, int WR, bool OWN>
__global__ __launch_bounds__(128 * WR, 2) void k_q4_experts(const uint16_t* __restrict__ x, int64_t ldx, int R,
                                                            const int32_t* __restrict__ offsets, int E, Q4Layer stack,
                                                            int64_t layer_bytes, const float* __restrict__ sums, int64_t lds_,
                                                            uint16_t* __restrict__ y, int64_t ldy, int nr,
                                                            ExpertTail tail, float* __restrict__ part)
{
    constexpr int HALF = TA > 1 ? TA / 2 : 1, BYTES = std::max(std::max(Prompt<TA, WR>::LDS, Prompt<HALF, WR>::LDS), Prompt<1, WR>::LDS);
    ExpertRows rows;
    int br, cls;
    TileShare share;
    if (!expert_tile<TA>(offsets, E, R, nr, stack.m, 64 * WR, tail, part, rows, br, cls, share)) return;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    if (cls == 0) prompt_tile<X, TA, WR, OWN, BYTES>(x, ldx, rows.t0, rows.t1, w, sums, lds_, y, ldy, br, share);
    else if (cls == 1 && TA > 1) prompt_tile<X, HALF, WR, OWN, BYTES>(x, ldx, rows.t0, rows.t1, w, sums, lds_, y, ldy, br, share);
    else if (TA > 2) prompt_tile<X, 1, WR, OWN, BYTES>(x, ldx, rows.t0, rows.t1, w, sums, lds_, y, ldy, br, share);
}

// Tiles of up to 64 TA rows by 64 WJ columns.
template <class X, int TA, int WJ>
__global__ __launch_bounds__(128 * WJ, 2) void k_q4_experts_grad(const uint16_t* __restrict__ dy, int64_t lddy, int R,
                                                                 const int32_t* __restrict__ offsets, int E, Q4Layer stack,
                                                                 int64_t layer_bytes, uint16_t* __restrict__ dx, int64_t lddx,
                                                                 int nj, ExpertTail tail, float* __restrict__ part)
{
    constexpr int HALF = TA / 2, BYTES = std::max(std::max(Grad<TA, WJ>::LDS, Grad<HALF, WJ>::LDS), Grad<1, WJ>::LDS);
    ExpertRows rows;
    int bj, cls;
    TileShare share;
    if (!expert_tile<TA>(offsets, E, R, nj, stack.n, 64 * WJ, tail, part, rows, bj, cls, share)) return;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    if (cls == 0) grad_tile<X, TA, WJ, BYTES>(dy, lddy, rows.t0, rows.t1, w, dx, lddx, bj, share);
    else if (cls == 1) grad_tile<X, HALF, WJ, BYTES>(dy, lddy, rows.t0, rows.t1, w, dx, lddx, bj, share);
    else if (TA > 2) grad_tile<X, 1, WJ, BYTES>(dy, lddy, rows.t0, rows.t1, w, dx, lddx, bj, share);
}

// The sum of `splits` partial results, in order, for the rows that some expert
// has: four columns a thread, the last ones of a row where they are fewer.  (Rows of
// 4096 x 4096, two parts: 27 us; a column a thread 62.)
template <class X>
__global__ __launch_bounds__(256) void k_q4_experts_join(const float* __restrict__ part, int splits, int R,
                                                         const int32_t* __restrict__ offsets, int E, int m, int log, int chunks,
                                                         uint16_t* __restrict__ y, int64_t ldy)
{
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    const UnitAt at(log, chunks);
    if (4 * at.u >= m) return;
    const int col = max(min(4 * at.u, m - 4), 0);   // (what two threads write they write alike)
    const int64_t all = (int64_t)R * m, first = max(offsets[0], 0), last = min(offsets[E], R);
    for (int64_t row = first + at.r; row < last; row += at.by) {
        const float* p = part + row * m + col;
        uint16_t* to = y + row * ldy + col;
        constexpr int U = 4;
        if (col + 4 <= m) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            for (int u0 = 0; u0 < splits; u0 += U) {
                f32x4 a[U];
#pragma unroll
                for (int u = 0; u < U; ++u) a[u] = *reinterpret_cast<const f32x4_any*>(p + min(u0 + u, splits - 1) * all);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u0 + u < splits) v += a[u];
            }
            *reinterpret_cast<u32x2_any*>(to) = u32x2_any{X::down2(v.x, v.y), X::down2(v.z, v.w)};
        } else {
            for (int e = 0; e < m; ++e) {
                float v = 0.f;
                for (int u = 0; u < splits; ++u) v += p[u * all + e];
                to[e] = X::down(v);
            }
        }
    }
}

// The tail's tiles from their parts, in order; kTailBlocks workgroups a tile.
constexpr int kTailBlocks = 16;
template <class X>
__global__ __launch_bounds__(256) void k_q4_experts_tail(const float* __restrict__ part, ExpertTail tail, int R,
                                                         const int32_t* __restrict__ offsets, int E, int m, int nc,
                                                         uint16_t* __restrict__ y, int64_t ldy)
{
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    const int q = blockIdx.x / kTailBlocks, sub = blockIdx.x % kTailBlocks;
    const ExpertTiles<4> tiles(offsets, E, R);
    const ExpertTailAt at(tiles.count(nc), tail);
    if (q >= at.left || at.parts == 1) return;
    ExpertRows rows;
    int bc, cls;
    if (!tiles.find(at.whole + q, nc, rows, bc, cls)) return;
    const int n = min(256 >> cls, rows.t1 - rows.t0), c = 4 * (threadIdx.x & 63), col = 256 * bc + c;
    if (col >= m) return;
    for (int t = 4 * sub + (threadIdx.x >> 6); t < n; t += 4 * kTailBlocks) {
        const float* p = part + ((int64_t)q * 256 + t) * 256 + c;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < at.parts; k0 += 4) {
            f32x4 a[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                a[u] = *reinterpret_cast<const f32x4*>(p + (int64_t)min(k0 + u, at.parts - 1) * at.left * 65536);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (k0 + u < at.parts) v += a[u];
        }
        uint16_t* to = y + (int64_t)(rows.t0 + t) * ldy + col;
        if (col + 4 <= m) {
            *reinterpret_cast<u32x2_any*>(to) = u32x2_any{X::down2(v.x, v.y), X::down2(v.z, v.w)};
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (col + e < m) to[e] = X::down(v[e]);
        }
    }
}

// Zeros in the rows that some expert has.
__global__ __launch_bounds__(256) void k_q4_experts_zero(uint16_t* __restrict__ y, int64_t ld, int R,
                                                         const int32_t* __restrict__ offsets, int E, int64_t cols)
{
    const int64_t r0 = max(offsets[0], 0), r1 = min(offsets[E], R);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (r1 - r0) * cols; i += (int64_t)gridDim.x * 256)
        y[(r0 + i / cols) * ld + i % cols] = 0;
}

// ------------------------------------------------------------ few rows each
//
// A wave has two row tiles of W, which share the rows' fragments; WS waves share
// the columns of a pair and are joined in wave order.

constexpr int kFewRows = 32;   // of a block
// Up to so many rows per expert on average.  One number for layers of every size is a
// compromise: an expert of more than 32 rows has two blocks, which read its codes twice.
// 2 of 8 of 14336 x 4096, 33 rows each: 100 us, and 106 in tiles of 64 rows; 40: 108 and
// 105; 48: 121 and 106; of 4096 x 4096, 48: 38 and 48.  6 of 64 of 1024 x 2048, 38 uneven
// ones: 52 and 47, 39 nearly even ones: 37 and 44, 48: 41 and 45.
constexpr int kFewMean = 48;
constexpr int kFewLds = 8 * std::max(few_lds(kFewRows / 4), 16 * 64 * 4);   // staged rows, then the joining sums

template <class X, int TQ, int U, int WS, bool HALF>
__device__ __forceinline__ void few_rows_of(const uint16_t* __restrict__ x, int64_t ldx, const Q4Layer& w, int rt0, int t0,
                                            int n, char* lds, uint16_t* __restrict__ y, int64_t ldy)
{
    typedef FewSpan<X, TQ, 2, U, HALF> Span;
    constexpr int NT = Span::NT, N = 2 * NT * 4;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint16_t* xr[TQ];
#pragma unroll
    for (int t = 0; t < TQ; ++t) xr[t] = x + (int64_t)(t0 + min(4 * t + (lane >> 4), n - 1)) * ldx;
    Span span(lds + wave * few_lds(TQ));
    const Q4Layer ws[1] = {w};
    span.template rows<1>(ws, rt0 + 2 * (wave / WS));
    span.tokens(xr);
    span.run(wave % WS, WS, w.KB);
    __syncthreads();   // the joining sums overwrite the staged rows
    float(*red)[N][64] = reinterpret_cast<float(*)[N][64]>(lds);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[wave][4 * (j * NT + i) + e][lane] = span.acc[j][i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 8 / WS * N * 64; o += 512) {
        const int l = o & 63, e = (o >> 6) % N, pair = (o >> 6) / N;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < WS; ++u) v += red[pair * WS + u][e][l];
        const int t = 16 * ((e >> 2) % NT) + 4 * (l >> 4) + (e & 3), row = (rt0 + 2 * pair + (e >> 2) / NT) * 16 + (l & 15);
        if (t < n && row < w.m) y[(int64_t)(t0 + t) * ldy + row] = X::down(v);
    }
}

template <class X, int WS, bool HALF>
__global__ __launch_bounds__(512, 4) void k_q4_experts_few(const uint16_t* __restrict__ x, int64_t ldx, int R,
                                                           const int32_t* __restrict__ offsets, int E, Q4Layer stack,
                                                           int64_t layer_bytes, uint16_t* __restrict__ y, int64_t ldy)
{
    __shared__ __align__(16) char lds[kFewLds];
    const ExpertLane lane(offsets, E, R);
    const auto blocks = [](int c) { return (c + kFewRows - 1) / kFewRows; };
    int sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += blocks(lane.rows(u));
    const int upto = lanes_upto(sum);
    int k = blockIdx.y;
    if (k >= __builtin_amdgcn_readlane(upto, 63)) return;
    ExpertRows rows;
    expert_at(lane, lane_of(upto, sum, k), k, blocks, rows);
    rows.t0 += k * kFewRows;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    const int rt0 = 16 / WS * blockIdx.x, n = min(kFewRows, rows.t1 - rows.t0);
    if (n <= 4) few_rows_of<X, 1, 2, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
    else if (n <= 16) few_rows_of<X, 4, 1, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
    else few_rows_of<X, 8, 1, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
}

// The gradient: a workgroup has a block of up to 16 SETS rows and 128 columns, its
// waves the rows of W in turn; blockIdx.z of gridDim.z shares those.  (Blocks of rows
// are x: there can be more of them than y has room for.)
constexpr int kGradFewWaves = 4;   // (8: 5 to 15 % slower, but for the fewest rows)
inline int grad_few_rows(int gb) { return gb % 2 ? 16 : 32; }   // of a block: its columns may have two grids

template <class X, int SETS, bool HALF>
__global__ __launch_bounds__(64 * kGradFewWaves) void k_q4_experts_grad_few(const uint16_t* __restrict__ dy, int64_t lddy, int R,
                                                                           const int32_t* __restrict__ offsets, int E,
                                                                           Q4Layer stack, int64_t layer_bytes,
                                                                           uint16_t* __restrict__ dx, int64_t lddx,
                                                                           float* __restrict__ part)
{
    constexpr int BT = 16 * SETS;
    __shared__ __align__(16) char lds[kGradFewWaves * std::max(kGradFewStage, kGradFewJoin)];
    const ExpertLane lane(offsets, E, R);
    const auto blocks = [](int c) { return (c + BT - 1) / BT; };
    int sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += blocks(lane.rows(u));
    const int upto = lanes_upto(sum);
    int k = blockIdx.x;
    if (k >= __builtin_amdgcn_readlane(upto, 63)) return;
    ExpertRows rows;
    expert_at(lane, lane_of(upto, sum, k), k, blocks, rows);
    rows.t0 += k * BT;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    const int n = min(BT, rows.t1 - rows.t0), all = (w.m + 31) / 32;
    const int s0 = all * blockIdx.z / gridDim.z, s1 = all * (blockIdx.z + 1) / gridDim.z;
    float* to = gridDim.z > 1 ? part + (int64_t)blockIdx.z * R * w.n : nullptr;
    if (SETS == 1 || n <= 16)
        grad_few<X, 1, HALF, kGradFewWaves>(dy, lddy, w, blockIdx.y, rows.t0, n, s0, s1, lds, dx, lddx, to, w.n);
    else
        grad_few<X, SETS, HALF, kGradFewWaves>(dy, lddy, w, blockIdx.y, rows.t0, n, s0, s1, lds, dx, lddx, to, w.n);
}

// --------------------------------------------------------------------- host

struct ExpertsPlan {
    bool few;
    int TA, WR, splits;
    ExpertTail tail;
    double us;         // that it is expected to take
    int64_t tiles;     // of rows, that there can be
    int pieces;
    int64_t lds_, ldc;
    size_t copy, part, bytes;
};

// Blocks of at most `rows` rows that R rows of E experts can make.
static int64_t blocks_most(int64_t R, int64_t E, int64_t rows) { return R / rows + std::min(R, E); }

// About how many there will be.
static int64_t blocks_about(int64_t R, int64_t E, int64_t rows)
{
    const int64_t some = std::min(R, E);
    return std::max(some, R / rows + some / 2);
}

// A product's tiles: their rows (and halves and quarters of them), columns, and what
// each takes in us for a depth of 4096, the chip full of them.
struct ExpertShape {
    int rows, cols;
    double us[3];
};

// What a launch is expected to take with its depth shared out `splits` times: the work
// over 256 CUs, and two fifths of a long tile for the CUs that finish last.  The rows
// are not dealt out evenly: experts have 0.4 to 1.6 times the mean.
struct ExpertWork {
    double all, tile;   // of a depth of 4096: all tiles over 256 CUs, and the longest
};
static ExpertWork experts_work(const ExpertShape& s, int64_t R, int64_t E, int64_t cols)
{
    const int64_t some = std::min(R, E);
    ExpertWork w{0.0, 0.0};
    for (int q = 0; q < 8; ++q) {
        const int64_t c = std::max<int64_t>(1, (int64_t)((0.475 + 0.15 * q) * R / some)), rest = c % s.rows;
        const double cut = rest == 0 ? 0.0 : s.us[rest <= s.rows / 4 ? 2 : rest <= s.rows / 2 ? 1 : 0];
        w.all += (double)(c / s.rows) * s.us[0] + cut;
        w.tile = std::max(w.tile, c >= s.rows ? s.us[0] : cut);
    }
    w.all *= some * ceil_div(cols, s.cols) / (8.0 * 256);
    return w;
}
static double experts_us(const ExpertWork& w, int64_t R, int64_t cols, int64_t depth, int splits)
{
    // (splits: a launch that joins the parts, which go there and back at 4 TB/s)
    return std::max(w.all + 0.4 * w.tile / splits, w.tile / splits) * depth / 4096 +
           (splits > 1 ? 2.0 + 8.0e-6 / 4 * splits * R * cols : 0.0);
}

// The least of it over shapes and splits, with `deepest` splits at most; or shape 0 with
// its tail shared out (ExpertTail), for tiles of kTailLeast us or more and few rounds of
// them (gradient, 2 of 8 of 14336 x 4096, 1500 tokens: 420 us, and 462 all in equal parts;
// 2048: 543 and 611; 6000, three rounds: 1400 and 1533.  Product, 2048 tokens, four rounds:
// 490 and 484; 8192, fifteen: 1731 and 1706).
struct ExpertsChoice {
    int shape, splits;
    double us;
    ExpertTail tail;
};
constexpr double kTailLeast = 40.0, kTailRounds = 3.5;
template <int N>
static ExpertsChoice experts_choose(const ExpertShape (&shapes)[N], int64_t R, int64_t E, int64_t cols, int64_t depth,
                                    int64_t deepest)
{
    ExpertsChoice best{0, 1, 0.0, {0, 0, 0}};
    for (int i = 0; i < N; ++i) {
        const ExpertWork w = experts_work(shapes[i], R, E, cols);
        const int64_t tiles = blocks_most(R, E, shapes[i].rows) * ceil_div(cols, shapes[i].cols);
        for (int s = 1; s == 1 || (s <= deepest && tiles * s <= 2048); ++s) {
            const double us = experts_us(w, R, cols, depth, s);
            if (best.us == 0.0 || us < best.us) best = {i, s, us, {0, 0, 0}};
        }
    }
    const ExpertWork w = experts_work(shapes[0], R, E, cols);
    const double tile = shapes[0].us[0] * depth / 4096, us = w.all * depth / 4096 + 0.1 * tile + 20.0;
    if (tile >= kTailLeast && w.all <= kTailRounds * w.tile && us < best.us)
        best = {0, 1, us, {(int)std::min(100.0 * tile, 1.0e6), (int)std::min<int64_t>(deepest, kTailParts),
                           (int)std::min<int64_t>(kTailUnits, blocks_most(R, E, 256) * ceil_div(cols, 256) * kTailParts)}};
    return best;
}

// Workgroups of a launch, and the bytes of its parts.
static int64_t experts_grid(const ExpertsPlan& p, int64_t nc) { return p.tiles * nc + p.tail.units; }
static size_t experts_part_bytes(const ExpertsPlan& p, int64_t R, int64_t cols)
{
    if (p.tail.us) return align_up((size_t)p.tail.units * 65536 * 4);
    return p.splits > 1 ? align_up((size_t)p.splits * R * cols * 4) : 0;
}

static ExpertsPlan experts_plan(int64_t R, int64_t E, int64_t m, int64_t n, int gb)
{
    ExpertsPlan p{};
    p.few = R <= kFewMean * E;
    if (p.few) return p;
    static constexpr ExpertShape shapes[] = {
        {256, 256, {128.0, 80.0, 56.0}}, {128, 128, {39.0, 28.0, 28.0}}, {64, 128, {28.0, 28.0, 28.0}}};
    const ExpertsChoice c = experts_choose(shapes, R, E, m, n, std::min<int64_t>(8, ceil_div(n, kQ4Cols) / 2));
    const ExpertShape& s = shapes[c.shape];
    p.splits = c.splits;
    p.tail = c.tail;
    p.us = c.us;
    p.TA = s.rows / 64;
    p.WR = s.cols / 64;
    p.tiles = blocks_most(R, E, s.rows);
    p.lds_ = ceil_div(R, 256) * 256 + 256;   // a block's sums are read as a whole, whichever row it begins at
    p.ldc = ceil_div(n, 64) * 64;
    p.pieces = piece_at((int)((n - 1) / 64), gb) + 1;
    p.copy = align_up((size_t)p.lds_ * p.pieces * 4);
    p.part = p.copy + align_up((size_t)R * p.ldc * 2);
    p.bytes = p.part + experts_part_bytes(p, R, m);
    return p;
}

static ExpertsPlan experts_grad_plan(int64_t R, int64_t E, int64_t m, int64_t n, int gb)
{
    ExpertsPlan p{};
    // 256 x 256 as in q4_grad.hip.  128 x 128: two workgroups of a CU, which take turns with
    // its units where a lone one of eight waves leaves them idle at its barriers, but twice
    // the expansion and LDS writes for a product: where experts have one to two hundred rows, or
    // there are few tiles (1024 tokens, 6 of 64 of 2048 x 1024, 40 to 230 rows each: 65 us, and
    // 73 in 256 x 256; 4 to 490: 79 and 77;
    // 900, 7 of 43 of 1152 x 320: 23 and 32; 512, one of 4096 x 4096: 49 and 60; 2048, 2 of 8
    // of 14336 x 4096: 685 and 606).
    static constexpr ExpertShape shapes[] = {{256, 256, {130.0, 88.0, 64.0}}, {128, 128, {44.0, 32.0, 32.0}}};
    const ExpertsChoice c = experts_choose(shapes, R, E, n, m, std::min<int64_t>(16, ceil_div(m, 64) / 2));
    // Few rows: a block's codes at 5.6 T/s however many rows it has (4.2 where its columns
    // have two grids), where there are two workgroups for every CU; the rows of W are shared
    // out towards that, four steps at least for every wave.  (6 of 64 experts of 2048 x 1024
    // in groups of 128, 48 rows each: 54 us, in tiles 60; 96: 91 and 65; groups of 64, 32
    // rows: 67 and 48.  2 of 8 of 5000 x 3500, 10 rows each: 31 and 65, 100: 101 and 85.)
    const int64_t blocks = blocks_about(R, E, grad_few_rows(gb)), groups = blocks * ceil_div(n, kQ4Cols);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({16, 512 / groups, ceil_div(m, 32) / (4 * kGradFewWaves)}));
    p.few = blocks * (double)m * n / ((gb % 2 ? 4.2e6 : 5.6e6) * std::min(1.0, groups * splits / 512.0)) <= 3.0 + c.us;
    if (p.few) {
        p.splits = (int)splits;
        p.bytes = p.splits > 1 ? align_up((size_t)p.splits * R * n * 4) : 0;
        return p;
    }
    p.splits = c.splits;
    p.tail = c.tail;
    p.TA = shapes[c.shape].rows / 64;
    p.WR = shapes[c.shape].cols / 64;
    p.tiles = blocks_most(R, E, shapes[c.shape].rows);
    p.ldc = ceil_div(m, 64) * 64;
    p.part = align_up((size_t)R * p.ldc * 2);
    p.bytes = p.part + experts_part_bytes(p, R, n);
    return p;
}

struct ExpertsCall {
    const uint16_t* in;
    int64_t ldin, rows;
    const void* packed;
    int64_t E;
    Q4Dims d;
    const int32_t* offsets;
    uint16_t* out;
    int64_t ldout;
    char* ws;
    hipStream_t s;
};

template <class X>
static void experts_join(const ExpertsCall& c, const float* part, int splits, int64_t cols)
{
    const UnitGrid g = unit_grid(c.rows, ceil_div(cols, 4), 0);
    enqueue(k_q4_experts_join<X>, dim3(g.blocks), dim3(256), c.s, part, splits, (int)c.rows, c.offsets, (int)c.E, (int)cols,
            g.log, g.chunks, c.out, c.ldout);
}

// What a product in tiles left in parts.
template <class X>
static void experts_parts(const ExpertsCall& c, const ExpertsPlan& p, int64_t cols)
{
    const float* part = reinterpret_cast<const float*>(c.ws + p.part);
    const int64_t nc = ceil_div(cols, 256);
    if (p.splits > 1) experts_join<X>(c, part, p.splits, cols);
    if (p.tail.us)
        enqueue(k_q4_experts_tail<X>, dim3((unsigned)(std::min<int64_t>(kTailCUs - 1, p.tiles * nc) * kTailBlocks)), dim3(256), c.s,
                part, p.tail, (int)c.rows, c.offsets, (int)c.E, (int)cols, (int)nc, c.out, c.ldout);
}

template <class X, int WS>
static void experts_few(const ExpertsCall& c, const Q4Layer& w)
{
    enqueue(w.gb % 2 ? k_q4_experts_few<X, WS, true> : k_q4_experts_few<X, WS, false>,
            dim3((unsigned)ceil_div(w.RT, 16 / WS), (unsigned)blocks_most(c.rows, c.E, kFewRows)), dim3(512), c.s, c.in, c.ldin,
            (int)c.rows, c.offsets, (int)c.E, w, (int64_t)c.d.bytes, c.out, c.ldout);
}

template <class X, int TA, int WR, bool OWN>
static void experts_launch(const ExpertsCall& c, const ExpertsPlan& p, const Q4Layer& w, const uint16_t* x, int64_t ldx)
{
    const int nr = (int)ceil_div(w.m, 64 * WR);
    enqueue(k_q4_experts<X, TA, WR, OWN>, dim3((unsigned)experts_grid(p, nr), (unsigned)p.splits), dim3(128 * WR), c.s, x, ldx,
            (int)c.rows, c.offsets, (int)c.E, w, (int64_t)c.d.bytes, reinterpret_cast<const float*>(c.ws), p.lds_, c.out,
            c.ldout, nr, p.tail, reinterpret_cast<float*>(c.ws + p.part));
}

template <class X>
static void experts_run(const ExpertsCall& c)
{
    const Q4Layer w = q4_layer(c.packed, c.d);
    const ExpertsPlan p = experts_plan(c.rows, c.E, w.m, w.n, w.gb);
    if (p.few) {
        const int64_t waves = ceil_div(w.RT, 2) * std::min(c.rows, c.E);
        if (8 * waves <= 8192) experts_few<X, 8>(c, w);
        else if (4 * waves <= 8192) experts_few<X, 4>(c, w);
        else experts_few<X, 2>(c, w);
        return;
    }
    // (the staging offsets of a block of rows are 31 bits)
    const bool direct = w.n % 64 == 0 && c.ldin % 8 == 0 && c.ldin <= (1 << 21) && aligned16(c.in);
    // Sums beside the products are half as many more products, and save a launch: only
    // where that is what counts, and for tiles of 64 rows (128 rows: 2048 tokens, 4 of 16 of
    // 2048 x 2048: 102 us, and 92 with the pass).
    const bool own = p.TA == 1 && direct && p.us < 30.0;
    const uint16_t* x = c.in;
    int64_t ldx = c.ldin;
    uint16_t* copy = reinterpret_cast<uint16_t*>(c.ws + p.copy);
    if (!own)
        enqueue(direct ? k_q4_sums<X, false> : k_q4_sums<X, true>, dim3((unsigned)ceil_div(c.rows, 4)), dim3(256), c.s, x, ldx,
                (int)c.rows, w.n, w.gb, p.pieces, reinterpret_cast<float*>(c.ws), p.lds_, copy, p.ldc);
    if (!direct) x = copy, ldx = p.ldc;
    if (p.TA == 4) experts_launch<X, 4, 4, false>(c, p, w, x, ldx);
    else if (p.TA == 2) experts_launch<X, 2, 2, false>(c, p, w, x, ldx);
    else (own ? experts_launch<X, 1, 2, true> : experts_launch<X, 1, 2, false>)(c, p, w, x, ldx);
    experts_parts<X>(c, p, w.m);
}

template <class X>
static void experts_grad_run(const ExpertsCall& c)
{
    const Q4Layer w = q4_layer(c.packed, c.d);
    const ExpertsPlan p = experts_grad_plan(c.rows, c.E, w.m, w.n, w.gb);
    const uint16_t* dy = c.in;
    int64_t lddy = c.ldin;
    if (p.few) {
        const int rows = grad_few_rows(w.gb);
        float* part = reinterpret_cast<float*>(c.ws);
        enqueue(w.gb % 2 ? k_q4_experts_grad_few<X, 1, true> : k_q4_experts_grad_few<X, 2, false>,
                dim3((unsigned)blocks_most(c.rows, c.E, rows), (unsigned)w.KB, (unsigned)p.splits), dim3(64 * kGradFewWaves), c.s,
                dy, lddy, (int)c.rows, c.offsets, (int)c.E, w, (int64_t)c.d.bytes, c.out, c.ldout, part);
        if (p.splits > 1) experts_join<X>(c, part, p.splits, w.n);
        return;
    }
    if (w.m % 64 || lddy % 8 || lddy > (1 << 21) || !aligned16(dy)) {
        copy_enqueue<X>(dy, lddy, c.rows, w.m, reinterpret_cast<uint16_t*>(c.ws), p.ldc, c.s);
        dy = reinterpret_cast<const uint16_t*>(c.ws);
        lddy = p.ldc;
    }
    const int nj = (int)ceil_div(w.n, 64 * p.WR);
    enqueue(p.TA == 4 ? k_q4_experts_grad<X, 4, 4> : k_q4_experts_grad<X, 2, 2>, dim3((unsigned)experts_grid(p, nj), (unsigned)p.splits),
            dim3(128 * p.WR), c.s, dy, lddy, (int)c.rows, c.offsets, (int)c.E, w, (int64_t)c.d.bytes, c.out, c.ldout, nj,
            p.tail, reinterpret_cast<float*>(c.ws + p.part));
    experts_parts<X>(c, p, w.n);
}

static bool experts_size_ok(int64_t rows, int64_t m, int64_t n)
{
    return rows >= 0 && rows <= BAKRON_MOE_MAX_ROWS && m >= 0 && n >= 0 && m <= BAKRON_MAX_DIM && n <= BAKRON_MAX_DIM;
}
static bool experts_arg_ok(int64_t E, int64_t g) { return E >= 1 && E <= kExperts && g >= 0 && g % 64 == 0; }

// The checks that the products and their gradient share, and the call where
// there is something to do.
static int experts_call(bool grad, const void* in, int64_t ldin, int64_t rows, int32_t type, const void* packed, int64_t E,
                        int64_t m, int64_t n, int64_t g, const int32_t* offsets, void* out, int64_t ldout, void* ws,
                        size_t ws_bytes, hipStream_t s)
{
    const int64_t in_cols = grad ? m : n, out_cols = grad ? n : m;
    if (!experts_size_ok(rows, m, n)) return BAKRON_ERR_BAD_SIZE;
    if (!experts_arg_ok(E, g) || !moe_type_ok(type) || !moe_ld_ok(ldin, in_cols) || !moe_ld_ok(ldout, out_cols))
        return BAKRON_ERR_BAD_ARG;
    if (rows == 0 || out_cols == 0) return BAKRON_SUCCESS;
    if (!out || !offsets) return BAKRON_ERR_NULL_POINTER;
    if (!moe_at(out, 2) || !moe_at(offsets, 4)) return BAKRON_ERR_BAD_ARG;
    if (in_cols == 0) {
        enqueue(k_q4_experts_zero, dim3((unsigned)std::min<int64_t>(65536, ceil_div(rows * out_cols, 256))), dim3(256), s,
                static_cast<uint16_t*>(out), ldout, (int)rows, offsets, (int)E, out_cols);
        return moe_done();
    }
    if (!in || !packed) return BAKRON_ERR_NULL_POINTER;
    if (!moe_at(in, 2) || !moe_at(packed, kAlign)) return BAKRON_ERR_BAD_ARG;
    const size_t need = grad ? bakron_q4_experts_grad_workspace_bytes(rows, E, m, n, g)
                             : bakron_q4_experts_workspace_bytes(rows, E, m, n, g);
    if (need && (!ws || ws_bytes < need || !moe_at(ws, kAlign))) return BAKRON_ERR_WORKSPACE;
    const ExpertsCall c{static_cast<const uint16_t*>(in), ldin, rows, packed, E, q4_dims(m, n, g), offsets,
                        static_cast<uint16_t*>(out), ldout, static_cast<char*>(ws), s};
    if (grad) (type == BAKRON_Q4_BF16 ? experts_grad_run<Bf16> : experts_grad_run<Fp16>)(c);
    else (type == BAKRON_Q4_BF16 ? experts_run<Bf16> : experts_run<Fp16>)(c);
    return moe_done();
}

}  // namespace bk

extern "C" {

size_t bakron_q4_experts_workspace_bytes(int64_t rows, int64_t experts, int64_t m, int64_t n, int64_t group_size)
{
    if (!bk::experts_size_ok(rows, m, n) || !bk::experts_arg_ok(experts, group_size) || rows == 0 || m == 0 || n == 0) return 0;
    return bk::experts_plan(rows, experts, m, n, bk::q4_dims(m, n, group_size).gb).bytes;
}

size_t bakron_q4_experts_grad_workspace_bytes(int64_t rows, int64_t experts, int64_t m, int64_t n, int64_t group_size)
{
    if (!bk::experts_size_ok(rows, m, n) || !bk::experts_arg_ok(experts, group_size) || rows == 0 || m == 0 || n == 0) return 0;
    return bk::experts_grad_plan(rows, experts, m, n, bk::q4_dims(m, n, group_size).gb).bytes;
}

int bakron_q4_experts(const void* x, int64_t ldx, int64_t rows, int32_t type, const void* packed, int64_t experts,
                      int64_t m, int64_t n, int64_t group_size, const int32_t* offsets, void* y, int64_t ldy,
                      void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return bk::experts_call(false, x, ldx, rows, type, packed, experts, m, n, group_size, offsets, y, ldy, workspace,
                            workspace_bytes, stream);
}

int bakron_q4_experts_grad(const void* dy, int64_t lddy, int64_t rows, int32_t type, const void* packed,
                           int64_t experts, int64_t m, int64_t n, int64_t group_size, const int32_t* offsets, void* dx,
                           int64_t lddx, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    return bk::experts_call(true, dy, lddy, rows, type, packed, experts, m, n, group_size, offsets, dx, lddx, workspace,
                            workspace_bytes, stream);
}

}  // extern "C"
