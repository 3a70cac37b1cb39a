// q4_moe.hip -- a whole mixture-of-experts layer on packed 4-bit experts, for
// a few tokens.
//
// Launches: k_q4_router (logits, the top_k choices and their softmax),
// k_q4_moe_up (gate and up rows of every chosen expert, silu(gate) * up),
// k_q4_moe_down (down rows per choice), k_q4_moe_join (the weighted sum).
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4.hpp"

namespace bk {

constexpr int kMoeTokens = BAKRON_Q4_MOE_MAX_TOKENS;
constexpr int kMoeTopK = BAKRON_Q4_MOE_MAX_TOP_K;
constexpr int kMoeExperts = BAKRON_Q4_MAX_LAYERS;

// One workgroup per token: a wave per expert in turn for the logits, then
// wave 0 picks top_k times the largest logit left (the lowest index among
// equals; NaN counts as -infinity) and forms the softmax over them.
template <class X>
__global__ __launch_bounds__(512) void k_q4_router(const uint16_t* __restrict__ x, int64_t ldx, int h,
                                                   const uint16_t* __restrict__ router, int E, int k,
                                                   int32_t* __restrict__ ids, float* __restrict__ weights)
{
    __shared__ float logit[kMoeExperts];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t* xr = x + (int64_t)t * ldx;
    for (int e = wave; e < E; e += 8) {
        const uint16_t* w = router + (int64_t)e * h;
        float s = 0.f;
        for (int j = lane; j < h; j += 64) s = fmaf(X::up(xr[j]), X::up(w[j]), s);
        for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
        if (lane == 0) logit[e] = s;
    }
    __syncthreads();
    if (wave != 0) return;
    // lane l holds experts l, l + 64, ...; the key orders, the logit weighs
    float key[kMoeExperts / 64];
    for (int u = 0; u < kMoeExperts / 64; ++u) {
        const int e = lane + 64 * u;
        key[u] = e < E ? (logit[e] == logit[e] ? logit[e] : -INFINITY) : 0.f;
    }
    unsigned taken = 0;   // bit u: expert lane + 64 u is chosen or absent
    for (int u = 0; u < kMoeExperts / 64; ++u)
        if (lane + 64 * u >= E) taken |= 1u << u;
    float top = 0.f, sum = 0.f, mine = 0.f;
    int my_id = 0;
    for (int j = 0; j < k; ++j) {
        float best = -INFINITY;
        int at = 1 << 20;
        for (int u = 0; u < kMoeExperts / 64; ++u) {
            const int e = lane + 64 * u;
            if (!(taken >> u & 1) && (at == 1 << 20 || key[u] > best)) best = key[u], at = e;
        }
        for (int off = 32; off > 0; off >>= 1) {
            const float b = __shfl_xor(best, off);
            const int a = __shfl_xor(at, off);
            if (a < (1 << 20) && (at == 1 << 20 || b > best || (b == best && a < at))) best = b, at = a;
        }
        if (lane == (at & 63)) taken |= 1u << (at >> 6);
        const float l = logit[at];
        if (j == 0) top = l;
        const float ex = expf(l - top);
        sum += ex;
        if (lane == j) mine = ex, my_id = at;
    }
    if (lane < k) {
        ids[t * k + lane] = my_id;
        weights[t * k + lane] = mine / sum;
    }
}

// The choices (t k + j) of expert e, in order, into list; returns how many.
// All threads of the workgroup call it.
__device__ __forceinline__ int moe_list(const int32_t* __restrict__ ids, int pairs, int e, int16_t* list, int* count)
{
    if (threadIdx.x < 64) {
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + (int)threadIdx.x;
            const bool mine = p < pairs && ids[p] == e;
            const unsigned long long b = __ballot(mine);
            if (mine) list[n + __popcll(b & ((1ull << threadIdx.x) - 1))] = (int16_t)p;
            n += __popcll(b);
        }
        if (threadIdx.x == 0) *count = n;
    }
    __syncthreads();
    return *count;
}

// Sum over the columns of one row tile for 16 tokens: acc += s (u x - (16 + z) x).
// WAVES waves take the column blocks in turn; xr is the lane's token row.
template <class X, int WAVES>
__device__ __forceinline__ void moe_tile(const uint16_t* __restrict__ xr, bool wide, const Q4Layer& w, int rt, f32x4& acc)
{
    typedef typename X::vec vec;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane >> 4, r = lane & 15;
    const vec ones = q4_ones<X>();
    for (int kb = wave; kb < w.KB; kb += WAVES) {
        const u32x4 c = w.codes[((int64_t)rt * w.KB + kb) * 64 + lane];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int g = min((2 * kb + hf) / w.gb, w.G - 1);
            const f32x2 sz = w.grid[((int64_t)rt * w.G + g) * 16 + r];
            const int kk = kb * 128 + 64 * hf + 16 * q;
            u32x4 xv[2];
            q4_load16(xr + kk, w.n - kk, wide, xv);
            const vec a0 = __builtin_bit_cast(vec, xv[0]), a1 = __builtin_bit_cast(vec, xv[1]);
            f32x4 t = {0.f, 0.f, 0.f, 0.f}, s = {0.f, 0.f, 0.f, 0.f};
            t = X::mfma16(a0, X::codes(c[2 * hf]), t);
            s = X::mfma16(a0, ones, s);
            t = X::mfma16(a1, X::codes(c[2 * hf + 1]), t);
            s = X::mfma16(a1, ones, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(sz.x, fmaf(-(sz.y + kQ4Offset), s[e], t[e]), acc[e]);
        }
    }
}

// hidden activations a = silu(gate x) * (up x) of one (expert, row tile), per
// choice.  Kept as two bfloat16 terms (a = hi + lo to 16 bits): the range of
// float32 in either activation type, and no rounding that the result sees.
template <class X>
__global__ __launch_bounds__(512) void k_q4_moe_up(const uint16_t* __restrict__ x, int64_t ldx, Q4Layer gate, Q4Layer up,
                                                   int64_t layer_bytes, const int32_t* __restrict__ ids, int pairs, int k,
                                                   uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t lda)
{
    __shared__ float red[8][8][64];
    __shared__ int16_t list[kMoeTokens * kMoeTopK];
    __shared__ int count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
    const int rt = blockIdx.x, e = blockIdx.y;
    const int n = moe_list(ids, pairs, e, list, &count);
    if (n == 0) return;
    const bool wide = ((reinterpret_cast<uintptr_t>(x) & 15) | (ldx & 7)) == 0;
    gate.codes = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(gate.codes) + e * layer_bytes);
    gate.grid = reinterpret_cast<const f32x2*>(reinterpret_cast<const char*>(gate.grid) + e * layer_bytes);
    up.codes = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(up.codes) + e * layer_bytes);
    up.grid = reinterpret_cast<const f32x2*>(reinterpret_cast<const char*>(up.grid) + e * layer_bytes);
    for (int n0 = 0; n0 < n; n0 += 16) {
        const uint16_t* xr = x + (int64_t)(list[min(n0 + r, n - 1)] / k) * ldx;
        f32x4 ga = {0.f, 0.f, 0.f, 0.f}, ua = {0.f, 0.f, 0.f, 0.f};
        moe_tile<X, 8>(xr, wide, gate, rt, ga);
        moe_tile<X, 8>(xr, wide, up, rt, ua);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][i][lane] = ga[i], red[wave][4 + i][lane] = ua[i];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int i = threadIdx.x >> 6, l = lane;
            float a = 0.f, b = 0.f;
            for (int u = 0; u < 8; ++u) a += red[u][i][l], b += red[u][4 + i][l];
            const int c = n0 + 4 * (l >> 4) + i, row = rt * 16 + (l & 15);
            if (c < n) {
                const float v = a / (1.f + expf(-a)) * b;
                const uint16_t vh = Bf16::down(v);
                const int64_t o = (int64_t)list[c] * lda + row;
                hi[o] = vh;
                lo[o] = Bf16::down(v - Bf16::up(vh));
            }
        }
    }
}

// part[choice][row] of the down product, one (expert, row tile) per workgroup.
__global__ __launch_bounds__(512) void k_q4_moe_down(const uint16_t* __restrict__ hi, const uint16_t* __restrict__ lo,
                                                     int64_t lda, Q4Layer down, int64_t layer_bytes,
                                                     const int32_t* __restrict__ ids, int pairs, float* __restrict__ part,
                                                     int h)
{
    __shared__ float red[8][4][64];
    __shared__ int16_t list[kMoeTokens * kMoeTopK];
    __shared__ int count;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
    const int rt = blockIdx.x, e = blockIdx.y;
    const int n = moe_list(ids, pairs, e, list, &count);
    if (n == 0) return;
    down.codes = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(down.codes) + e * layer_bytes);
    down.grid = reinterpret_cast<const f32x2*>(reinterpret_cast<const char*>(down.grid) + e * layer_bytes);
    for (int n0 = 0; n0 < n; n0 += 16) {
        const int64_t o = (int64_t)list[min(n0 + r, n - 1)] * lda;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        moe_tile<Bf16, 8>(hi + o, true, down, rt, acc);
        moe_tile<Bf16, 8>(lo + o, true, down, rt, acc);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int i = threadIdx.x >> 6, l = lane;
            float a = 0.f;
            for (int u = 0; u < 8; ++u) a += red[u][i][l];
            const int c = n0 + 4 * (l >> 4) + i, row = rt * 16 + (l & 15);
            if (c < n && row < h) part[(int64_t)list[c] * h + row] = a;
        }
    }
}

template <class X>
__global__ __launch_bounds__(256) void k_q4_moe_join(const float* __restrict__ part, const float* __restrict__ weights,
                                                     int k, int h, uint16_t* __restrict__ y, int64_t ldy)
{
    const int j = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (j >= h) return;
    float v = 0.f;
    for (int c = 0; c < k; ++c) v = fmaf(weights[t * k + c], part[(int64_t)(t * k + c) * h + j], v);
    y[(int64_t)t * ldy + j] = X::down(v);
}

struct MoeWork {
    int64_t lda;
    size_t hi, lo, part, bytes;
};

static MoeWork moe_work(int64_t T, int64_t h, int64_t f, int k)
{
    MoeWork w;
    w.lda = ceil_div(f, 16) * 16;
    w.hi = 0;
    w.lo = align_up(2 * (size_t)T * k * w.lda);
    w.part = 2 * w.lo;
    w.bytes = w.part + align_up(4 * (size_t)T * k * h);
    return w;
}

int q4_zero_enqueue(void* y, int64_t ld, int64_t rows, int64_t cols, hipStream_t s);

template <class X>
static int moe_enqueue(const void* x, int64_t ldx, int64_t T, const void* router, const void* gate, const void* up,
                       const void* down, int64_t h, int64_t f, int64_t E, int k, int64_t g, void* y, int64_t ldy,
                       int32_t* ids, float* weights, void* ws, hipStream_t s)
{
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    launch(nullptr, KK_Q4_ROUTER, 0.0, 0.0, k_q4_router<X>, dim3((unsigned)T), dim3(512), s, xp, ldx, (int)h,
           static_cast<const uint16_t*>(router), (int)E, k, ids, weights);
    if (f == 0) return q4_zero_enqueue(y, ldy, T, h, s);
    const MoeWork w = moe_work(T, h, f, k);
    char* base = static_cast<char*>(ws);
    uint16_t* hi = reinterpret_cast<uint16_t*>(base + w.hi);
    uint16_t* lo = reinterpret_cast<uint16_t*>(base + w.lo);
    float* part = reinterpret_cast<float*>(base + w.part);
    const Q4Dims du = q4_dims(f, h, g), dd = q4_dims(h, f, g);
    launch(nullptr, KK_Q4_MOE_UP, 0.0, 0.0, k_q4_moe_up<X>, dim3((unsigned)du.RT, (unsigned)E), dim3(512), s, xp, ldx,
           q4_layer(gate, du), q4_layer(up, du), (int64_t)du.bytes, ids, (int)T * k, k, hi, lo, w.lda);
    launch(nullptr, KK_Q4_MOE_DOWN, 0.0, 0.0, k_q4_moe_down, dim3((unsigned)dd.RT, (unsigned)E), dim3(512), s, hi, lo,
           w.lda, q4_layer(down, dd), (int64_t)dd.bytes, ids, (int)T * k, part, (int)h);
    launch(nullptr, KK_Q4_MOE_JOIN, 0.0, 0.0, k_q4_moe_join<X>, dim3((unsigned)ceil_div(h, 256), (unsigned)T), dim3(256),
           s, part, weights, k, (int)h, static_cast<uint16_t*>(y), ldy);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace bk

extern "C" {

size_t bakron_q4_moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t ffn, int64_t experts, int32_t top_k,
                                     int64_t group_size)
{
    if (tokens <= 0 || tokens > BAKRON_Q4_MOE_MAX_TOKENS || hidden <= 0 || hidden > BAKRON_MAX_DIM || ffn <= 0 ||
        ffn > BAKRON_MAX_DIM || experts < 1 || experts > BAKRON_Q4_MAX_LAYERS || top_k < 1 || top_k > experts ||
        top_k > BAKRON_Q4_MOE_MAX_TOP_K || group_size < 0 || group_size % 64)
        return 0;
    return bk::moe_work(tokens, hidden, ffn, top_k).bytes;
}

int bakron_q4_moe(const void* x, int64_t ldx, int64_t tokens, int32_t type, const void* router, const void* gate,
                  const void* up, const void* down, int64_t hidden, int64_t ffn, int64_t experts, int32_t top_k,
                  int64_t group_size, void* y, int64_t ldy, int32_t* ids, float* weights, void* workspace,
                  size_t workspace_bytes, hipStream_t stream)
{
    if (tokens < 0 || tokens > BAKRON_Q4_MOE_MAX_TOKENS || hidden < 0 || hidden > BAKRON_MAX_DIM || ffn < 0 ||
        ffn > BAKRON_MAX_DIM)
        return BAKRON_ERR_BAD_SIZE;
    if ((type != BAKRON_Q4_BF16 && type != BAKRON_Q4_FP16) || experts < 1 || experts > BAKRON_Q4_MAX_LAYERS ||
        top_k < 1 || top_k > experts || top_k > BAKRON_Q4_MOE_MAX_TOP_K || group_size < 0 || group_size % 64 ||
        ldx < hidden || ldy < hidden || ldx >= ((int64_t)1 << 32) || ldy >= ((int64_t)1 << 32))
        return BAKRON_ERR_BAD_ARG;
    if (tokens == 0 || hidden == 0) return BAKRON_SUCCESS;
    if (!x || !router || !y || !ids || !weights || (ffn > 0 && (!gate || !up || !down))) return BAKRON_ERR_NULL_POINTER;
    if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(router) | reinterpret_cast<uintptr_t>(y)) & 1) ||
        ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) & 3) ||
        (ffn > 0 && (reinterpret_cast<uintptr_t>(gate) | reinterpret_cast<uintptr_t>(up) |
                     reinterpret_cast<uintptr_t>(down)) % bk::kAlign))
        return BAKRON_ERR_BAD_ARG;
    const size_t need = bakron_q4_moe_workspace_bytes(tokens, hidden, ffn, experts, top_k, group_size);
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % bk::kAlign))
        return BAKRON_ERR_WORKSPACE;
    const int rc =
        type == BAKRON_Q4_BF16
            ? bk::moe_enqueue<bk::Bf16>(x, ldx, tokens, router, gate, up, down, hidden, ffn, experts, top_k, group_size, y,
                                        ldy, ids, weights, workspace, stream)
            : bk::moe_enqueue<bk::Fp16>(x, ldx, tokens, router, gate, up, down, hidden, ffn, experts, top_k, group_size, y,
                                        ldy, ids, weights, workspace, stream);
    return rc ? BAKRON_ERR_HIP : BAKRON_SUCCESS;
}

}  // extern "C"
