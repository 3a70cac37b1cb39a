// moe_rows.hip -- tokens' rows into the order of their experts and back,
// weighted, and the gradients of both (gfx950).
//
//   gather        xs[place_tj] = x_t
//   combine       y_t = sum_j w_tj ys[place_tj]
//   combine_grad  dys[place_tj] = w_tj dy_t,   dw_tj = <dy_t, ys[place_tj]>
//
// HBM bounds all three, so every row is moved once: the work is laid out by
// token, whose row (x, y or dy) is in registers while its top_k sorted rows are
// written or read, every load of a lane before its first use.  A place outside
// [0, rows) is no row: loads go to row 0 then, whose value is not used, so that they
// stay in one run.
//
// 8192 tokens of 4096, 2 choices: gather 34 us (5.9 TB/s; what the calls before left
// in the Infinity Cache helps), combine 39 without weights and 44 with (5.1 and 4.6),
// its gradient 56 (6.0).  16 tokens of 2048, 6 choices: 3.3 and 3.8 us, a launch and two
// round trips, place first.
#include <algorithm>

#include "moe.hpp"

namespace bk {

constexpr int kRowsTopK = BAKRON_MOE_MAX_PLACES;

__global__ __launch_bounds__(256) void k_moe_gather(const uint16_t* __restrict__ x, int64_t ldx, int T, int n, int k,
                                                    const int32_t* __restrict__ place, uint16_t* __restrict__ xs,
                                                    int64_t ldxs, int rows, int log, int chunks)
{
    const UnitAt at(log, chunks);
    if (8 * at.u >= n) return;
    for (int64_t t = at.r; t < T; t += at.by) {
        const u32x4 v = load8(x + t * ldx, 8 * at.u, n);
        for (int j = 0; j < k; ++j) {
            const int p = place[t * k + j];
            if ((unsigned)p < (unsigned)rows) store8(xs + (int64_t)p * ldxs, 8 * at.u, n, v);
        }
    }
}

// K: top_k rounded up; W: with weights.
template <class X, int K, bool W>
__global__ __launch_bounds__(256) void k_moe_combine(const uint16_t* __restrict__ ys, int64_t ldys, int rows, int T, int n,
                                                     int k, const int32_t* __restrict__ place,
                                                     const float* __restrict__ weights, uint16_t* __restrict__ y,
                                                     int64_t ldy, int log, int chunks)
{
    const UnitAt at(log, chunks);
    if (8 * at.u >= n) return;
    for (int64_t t = at.r; t < T; t += at.by) {
        u32x4 v[K];
        float w[K];
        bool on[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int64_t c = t * k + min(j, k - 1);
            const int p = place[c];
            on[j] = j < k && (unsigned)p < (unsigned)rows;
            w[j] = W ? weights[c] : 1.f;
            v[j] = load8(ys + (int64_t)(on[j] ? p : 0) * ldys, 8 * at.u, n);
        }
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float f[8];
            up8<X>(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = on[j] ? (W ? fmaf(w[j], f[e], sum[e]) : sum[e] + f[e]) : sum[e];
        }
        store8(y + t * ldy, 8 * at.u, n, down8<X>(sum));
    }
}

// WAVES waves share a token's columns; dw is summed over lanes and waves in
// order.
template <class X, int K, int WAVES>
__global__ __launch_bounds__(256) void k_moe_combine_grad(const uint16_t* __restrict__ dy, int64_t lddy,
                                                          const uint16_t* __restrict__ ys, int64_t ldys, int rows, int T,
                                                          int n, int k, const int32_t* __restrict__ place,
                                                          const float* __restrict__ weights, uint16_t* __restrict__ dys,
                                                          int64_t lddys, float* __restrict__ dweights)
{
    __shared__ float part[4][kRowsTopK];
    constexpr int TOKENS = 4 / WAVES;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, share = wave % WAVES;
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < T; t0 += (int64_t)gridDim.x * TOKENS) {
        const int64_t t = t0 + wave / WAVES;
        if (WAVES == 1 && t >= T) return;
        int p[K];
        float w[K], dot[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int64_t c = t * k + min(j, k - 1);
            p[j] = place[c];
            if (j >= k || (unsigned)p[j] >= (unsigned)rows) p[j] = -1;
            w[j] = weights[c];
            dot[j] = 0.f;
        }
        const uint16_t* row = dy + t * lddy;
        for (int c = 8 * (lane + 64 * share); c < n; c += 512 * WAVES) {
            const u32x4 dv = load8(row, c, n);
            u32x4 v[K];
#pragma unroll
            for (int j = 0; j < K; ++j) v[j] = load8(ys + (int64_t)max(p[j], 0) * ldys, c, n);
            float d[8];
            up8<X>(dv, d);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (p[j] < 0) continue;
                float f[8], g[8];
                up8<X>(v[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot[j] = fmaf(d[e], f[e], dot[j]), g[e] = w[j] * d[e];
                store8(dys + (int64_t)p[j] * lddys, c, n, down8<X>(g));
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
            for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        if (WAVES == 1) {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (lane == 0 && j < k) dweights[t * k + j] = dot[j];
        } else {
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (lane == 0) part[wave][j] = dot[j];
            __syncthreads();
            if (wave == 0 && lane < k) {
                float s = 0.f;
#pragma unroll
                for (int u = 0; u < WAVES; ++u) s += part[u][lane];
                dweights[t * k + lane] = s;
            }
            __syncthreads();
        }
    }
}

// n zeros
__global__ __launch_bounds__(256) void k_moe_zero(float* __restrict__ v, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) v[i] = 0.f;
}

// --------------------------------------------------------------------- host

template <class X, int K>
static void combine_enqueue(const void* ys, int64_t ldys, int64_t rows, int64_t n, int k, const int32_t* place,
                            const float* weights, int64_t T, void* y, int64_t ldy, hipStream_t s)
{
    const UnitGrid g = unit_grid(T, ceil_div(n, 8), 0);
    enqueue(weights ? k_moe_combine<X, K, true> : k_moe_combine<X, K, false>, dim3(g.blocks), dim3(256), s,
            static_cast<const uint16_t*>(ys), ldys, (int)rows, (int)T, (int)n, k, place, weights,
            static_cast<uint16_t*>(y), ldy, g.log, g.chunks);
}

template <class X, int K>
static void combine_grad_enqueue(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows, int64_t n, int k,
                                 const int32_t* place, const float* weights, int64_t T, void* dys, int64_t lddys,
                                 float* dweights, hipStream_t s)
{
    // Four waves share a token wherever a wave's 512 columns do not take a row whole:
    // what is in flight lies together (calls of 8192 tokens of 2 x 4096: 62 us, and 76 with a
    // wave per token; 6 x 2048: 85 and 99; narrow rows would rather have the wave, 2 x 1024: 16
    // and 14, 2 x 640: 14 and 10).
    const bool wide = n > 512;
    enqueue(wide ? k_moe_combine_grad<X, K, 4> : k_moe_combine_grad<X, K, 1>,
            dim3((unsigned)std::min(kUnitBlocks, wide ? T : ceil_div(T, 4))), dim3(256), s,
            static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(ys), ldys, (int)rows, (int)T, (int)n, k,
            place, weights, static_cast<uint16_t*>(dys), lddys, dweights);
}

// What the three calls check alike: 1 where there is nothing to do.
static int rows_check(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t tokens, int64_t rows, int32_t type,
                      int64_t cols, int32_t top_k, const int32_t* place)
{
    if (tokens < 0 || tokens > BAKRON_MOE_MAX_ROWS || rows < 0 || rows > 2 * BAKRON_MOE_MAX_ROWS || cols < 0 ||
        cols > BAKRON_MAX_DIM)
        return BAKRON_ERR_BAD_SIZE;
    if (!moe_type_ok(type) || top_k < 1 || top_k > BAKRON_MOE_MAX_PLACES || !moe_ld_ok(lda, cols) || !moe_ld_ok(ldb, cols))
        return BAKRON_ERR_BAD_ARG;
    if (tokens == 0 || cols == 0) return 1;
    if (!place) return BAKRON_ERR_NULL_POINTER;
    if (!moe_at(place, 4) || !moe_at(a, 2) || !moe_at(b, 2)) return BAKRON_ERR_BAD_ARG;
    return BAKRON_SUCCESS;
}

}  // namespace bk

// K of a launch: top_k rounded up to a power of two
#define BAKRON_BY_TOP_K(run, X, k) \
    ((k) <= 1 ? run<X, 1> : (k) <= 2 ? run<X, 2> : (k) <= 4 ? run<X, 4> : (k) <= 8 ? run<X, 8> : (k) <= 16 ? run<X, 16> : run<X, 32>)

extern "C" {

int bakron_moe_gather(const void* x, int64_t ldx, int64_t tokens, int32_t type, int64_t cols, int32_t top_k,
                      const int32_t* place, void* xs, int64_t ldxs, int64_t rows, hipStream_t stream)
{
    const int c = bk::rows_check(x, ldx, xs, ldxs, tokens, rows, type, cols, top_k, place);
    if (c < 0) return c;
    if (c == 1 || rows == 0) return BAKRON_SUCCESS;
    if (!x || !xs) return BAKRON_ERR_NULL_POINTER;
    const bk::UnitGrid g = bk::unit_grid(tokens, bk::ceil_div(cols, 8), 0);
    bk::enqueue(bk::k_moe_gather, dim3(g.blocks), dim3(256), stream, static_cast<const uint16_t*>(x), ldx, (int)tokens, (int)cols,
                top_k, place, static_cast<uint16_t*>(xs), ldxs, (int)rows, g.log, g.chunks);
    return bk::moe_done();
}

int bakron_moe_combine(const void* ys, int64_t ldys, int64_t rows, int32_t type, int64_t cols, int32_t top_k,
                       const int32_t* place, const float* weights, int64_t tokens, void* y, int64_t ldy,
                       hipStream_t stream)
{
    const int c = bk::rows_check(ys, ldys, y, ldy, tokens, rows, type, cols, top_k, place);
    if (c < 0) return c;
    if (c == 1) return BAKRON_SUCCESS;
    if (!y || (rows > 0 && !ys)) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(weights, 4)) return BAKRON_ERR_BAD_ARG;
    if (rows == 0) {   // no place is a row: zeros, by reading y's own first row unused
        ys = y;
        ldys = 0;
    }
    auto* run = type == BAKRON_Q4_BF16 ? BAKRON_BY_TOP_K(bk::combine_enqueue, bk::Bf16, top_k)
                                       : BAKRON_BY_TOP_K(bk::combine_enqueue, bk::Fp16, top_k);
    run(ys, ldys, rows, cols, top_k, place, weights, tokens, y, ldy, stream);
    return bk::moe_done();
}

int bakron_moe_combine_grad(const void* dy, int64_t lddy, const void* ys, int64_t ldys, int64_t rows, int32_t type,
                            int64_t cols, int32_t top_k, const int32_t* place, const float* weights, int64_t tokens,
                            void* dys, int64_t lddys, float* dweights, hipStream_t stream)
{
    const int c = bk::rows_check(dy, lddy, ys, ldys, tokens, rows, type, cols, top_k, place);
    if (c < 0) return c;
    if (!bk::moe_ld_ok(lddys, cols)) return BAKRON_ERR_BAD_ARG;
    if (tokens == 0) return BAKRON_SUCCESS;
    if (!dweights) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(dweights, 4)) return BAKRON_ERR_BAD_ARG;
    if (c == 1 || rows == 0) {
        const int64_t all = tokens * top_k;
        bk::enqueue(bk::k_moe_zero, dim3((unsigned)std::min<int64_t>(bk::ceil_div(all, 256), 4096)), dim3(256), stream,
                    dweights, all);
        return bk::moe_done();
    }
    if (!dy || !ys || !dys || !weights) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(dys, 2) || !bk::moe_at(weights, 4)) return BAKRON_ERR_BAD_ARG;
    auto* run = type == BAKRON_Q4_BF16 ? BAKRON_BY_TOP_K(bk::combine_grad_enqueue, bk::Bf16, top_k)
                                       : BAKRON_BY_TOP_K(bk::combine_grad_enqueue, bk::Fp16, top_k);
    run(dy, lddy, ys, ldys, rows, cols, top_k, place, weights, tokens, dys, lddys, dweights, stream);
    return bk::moe_done();
}

}  // extern "C"
