// q4_grad.hip -- dx = dy W on 4-bit codes, the input gradient of the linear
// layer (gfx950).
//
//     dx_tj = sum_i dy_ti s_ig (c_ij - z_ig),   g the group of column j.
//
// The sum runs over the rows of W, and step and zero point change with the
// row: they cannot be taken out of it as in the forward product.  So a
// weight is formed in float32, divided by its columns' unit (a power of two,
// q4.hpp) and rounded once to dy's 16-bit type, the product runs on 16-bit
// MFMAs with float32 accumulators, and the unit, a factor of the result's
// column, comes back at the store.  In float16 the largest weight of a group's
// columns is put at 2^15 at most, so that rows down to 2^-29 of it keep every
// bit.  The rounding is half a unit in the last place of each weight, as a
// layer kept in that type would have; independent from weight to weight, it
// adds to a result about what the result's own rounding does.
//
// k_q4_grad: a workgroup of eight waves computes 64 TA tokens x 256 columns;
// a wave owns 32 TA tokens x 64 columns as TA x 2 MFMA tiles of 32 x 32.  dy
// goes through LDS in chunks of 64 rows of W by direct loads.  Of each
// chunk's 64 x 256 weights a thread expands 4 rows x 8 columns (four dwords of
// codes) and writes them to LDS transposed, four rows of a column side by side
// as the MFMA takes them, one chunk ahead of the products that read them, so
// one barrier per chunk orders everything.  Few tiles share out their rows of
// W over several workgroups, joined by k_q4_join.
//
// Measured: 2048 tokens x 4096 x 14336, groups of 128: 239 - 252 us, 950 - 1010
// TFLOP/s (a large 16-bit product of the vendor's library: 1240).  No unit is
// full: of the cycles in which a CU has work MFMAs take 0.50, LDS instructions
// 0.45 (besides the fragments, every weight is written once and read by the
// tiles of two wave rows) and vector instructions 0.36; two waves a SIMD and a
// barrier a chunk overlap them only in part.  300 tokens x 1000 x 1531,
// unaligned: 16.5 us, of which the copy of dy takes 3.4 and the join 3.8.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4_grad.hpp"

namespace bk {

// The tiles of a launch; gridDim.y workgroups share a tile's rows of W.
template <class X, int TA>
__global__ __launch_bounds__(512) void k_q4_grad(const uint16_t* __restrict__ dy, int64_t lddy, int T, Q4Layer w,
                                                 uint16_t* __restrict__ dx, int64_t lddx, int nt, int nj,
                                                 float* __restrict__ part)
{
    typedef Grad<TA> P;
    int bt, bj;
    tile_of(nt, nj, bt, bj);
    grad_tile<X, TA>(dy, lddy, bt * P::BT, T, w, dx, lddx, bj,
                     TileShare{(int)blockIdx.y, (int)gridDim.y, part + (int64_t)blockIdx.y * T * w.n, w.n});
}

// --------------------------------------------------------------------- host

struct GradPlan {
    int TA, splits;
    int64_t ldc;
    size_t part, bytes;
};

static GradPlan grad_plan(int64_t T, int64_t m, int64_t n)
{
    GradPlan p;
    // Costs: 4096 tokens x 4096 columns in tiles of 256 tokens take 135 us, 2048
    // in 128 92, 1024 in 64 71 (and 4096 242).  3500 tokens x 2500 columns x 3500:
    // 139 us with 128, 111 with 256.  A split has two chunks of 64 rows at least.
    static constexpr TileShape shapes[] = {{256, 256, 130.0}, {128, 256, 88.0}, {64, 256, 64.0}};
    const TileChoice c = tile_choose(shapes, T, n, m, std::min<int64_t>(16, ceil_div(m, 64) / 2));
    p.TA = shapes[c.shape].tokens / 64;
    p.splits = c.splits;
    p.ldc = ceil_div(m, 64) * 64;
    p.part = align_up((size_t)T * p.ldc * 2);
    p.bytes = p.part + (p.splits > 1 ? align_up((size_t)p.splits * T * n * 4) : 0);
    return p;
}

size_t q4_grad_workspace_bytes(int64_t T, int64_t m, int64_t n) { return grad_plan(T, m, n).bytes; }

template <class X, int TA>
static void grad_launch(const uint16_t* dy, int64_t lddy, int64_t T, const Q4Layer& w, uint16_t* dx, int64_t lddx,
                        int splits, float* part, hipStream_t s)
{
    typedef Grad<TA> P;
    const int nt = (int)ceil_div(T, P::BT), nj = (int)ceil_div(w.n, P::BJ);
    launch(nullptr, KK_Q4_GRAD, 2.0 * T * w.m * w.n, 0.0, k_q4_grad<X, TA>, dim3((unsigned)(nt * nj), (unsigned)splits),
           dim3(512), s, dy, lddy, (int)T, w, dx, lddx, nt, nj, part);
}

template <class X>
static int grad_run(const void* dy, int64_t lddy, int64_t T, const Q4Layer& w, void* dx, int64_t lddx, void* ws,
                    hipStream_t s)
{
    const GradPlan p = grad_plan(T, w.m, w.n);
    const uint16_t* yp = static_cast<const uint16_t*>(dy);
    uint16_t* xp = static_cast<uint16_t*>(dx);
    uint16_t* copy = static_cast<uint16_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
    // (the staging offsets of a token block are 31 bits)
    if (w.m % 64 || lddy % 8 || lddy > (1 << 21) || !aligned16(dy)) {
        copy_enqueue<X>(yp, lddy, T, w.m, copy, p.ldc, s);
        yp = copy;
        lddy = p.ldc;
    }
    if (p.TA == 4) grad_launch<X, 4>(yp, lddy, T, w, xp, lddx, p.splits, part, s);
    else if (p.TA == 2) grad_launch<X, 2>(yp, lddy, T, w, xp, lddx, p.splits, part, s);
    else grad_launch<X, 1>(yp, lddy, T, w, xp, lddx, p.splits, part, s);
    if (p.splits > 1) join_enqueue<X>(part, p.splits, T, w.n, xp, lddx, s);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int q4_grad_enqueue(const void* dy, int64_t lddy, int64_t T, bool bf16, const Q4Layer& w, void* dx, int64_t lddx, void* ws,
                    hipStream_t s)
{
    return bf16 ? grad_run<Bf16>(dy, lddy, T, w, dx, lddx, ws, s) : grad_run<Fp16>(dy, lddy, T, w, dx, lddx, ws, s);
}

}  // namespace bk
