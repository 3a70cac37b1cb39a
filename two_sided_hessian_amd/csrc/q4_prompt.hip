// q4_prompt.hip -- y = x W^T on 4-bit codes for many tokens (gfx950).
//
// Mathematics (q4.hpp): with u = 16 + c,
//     y_ti = sum_g s_ig sum_{j in g} u_ij x_tj  -  sum_g s_ig (16 + z_ig) X_tg,   X_tg = sum_{j in g} x_tj.
// The first sum runs on 16-bit MFMAs with exact operands.  Its accumulators
// are kept in units of the current group's step: on entering group g they are
// multiplied by s_{g-1} / s_g, one float32 multiplication each, so a group
// needs no second set of accumulators.  The second sum is a product over the
// groups alone (n / 128 terms): X and s (16 + z) are split into three
// bfloat16 terms each and the six leading products of every group are six K
// slots of the same MFMAs, run once at the end (error 2^-24 of a term).
//
// k_q4_sums makes X (float32, group-major) in a pass over x of its own, and
// with it, where x's rows are not 16-byte aligned or n is not a multiple of
// 64, a padded copy that the product can stage directly.
//
// k_q4_prompt: a workgroup of 2 x WR waves computes 64 TA tokens x 64 WR rows
// of W; a wave owns 32 TA tokens x 64 rows as TA x 2 MFMA tiles of 32 x 32
// (v_mfma_f32_32x32x16, tokens are its rows).  x goes through LDS in chunks
// of 64 columns by direct loads, two buffers, 16-byte slots permuted so that
// fragment reads spread over the banks.  W never touches LDS: a lane loads
// its fragments' codes from the packed layout (32 bytes per 128 columns and
// tile) and expands them in registers, 7 operations per 8 codes.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4.hpp"

namespace bk {

// ---------------------------------------------------------------- group sums
//
// One wave per token: lanes sum 8 columns, 8 lanes a 64-column half, and the
// halves of a group are added in order.  Columns n .. np - 1 of the copy are
// zero.
constexpr int kSumsHalves = BAKRON_MAX_DIM / 64;

template <class X, bool COPY>
__global__ __launch_bounds__(256) void k_q4_sums(const uint16_t* __restrict__ x, int64_t ldx, int T, int n, int gb, int G,
                                                 float* __restrict__ sums, int64_t lds_, uint16_t* __restrict__ copy,
                                                 int64_t ldc)
{
    __shared__ float half[4][kSumsHalves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    const int halves = (n + 63) / 64;
    if (t < T) {
        const uint16_t* row = x + t * ldx;
        for (int c0 = 0; c0 < 64 * halves; c0 += 512) {
            const int c = c0 + 8 * lane;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (!COPY) {
                if (c < n) v = *reinterpret_cast<const u32x4*>(row + c);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = c + 2 * i < n ? row[c + 2 * i] : 0u;
                    const uint32_t b = c + 2 * i + 1 < n ? row[c + 2 * i + 1] : 0u;
                    v[i] = a | (b << 16);
                }
                if (c < 64 * halves) *reinterpret_cast<u32x4*>(copy + t * ldc + c) = v;
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) s += X::up((uint16_t)v[i]) + X::up((uint16_t)(v[i] >> 16));
            s += __shfl_xor(s, 1);
            s += __shfl_xor(s, 2);
            s += __shfl_xor(s, 4);
            if ((lane & 7) == 0 && c < 64 * halves) half[wave][c >> 6] = s;
        }
    }
    __syncthreads();
    if (t >= T) return;
    for (int g = lane; g < G; g += 64) {
        const int h0 = g * gb, h1 = g == G - 1 ? halves : h0 + gb;   // gb may exceed the halves when G is 1
        float s = 0.f;
        for (int h = h0; h < h1; ++h) s += half[wave][h];
        sums[(int64_t)g * lds_ + t] = s;
    }
}

// ------------------------------------------------------------------ product

template <int TA, int WR>
struct Prompt {
    static constexpr int BT = 64 * TA;           // tokens of a workgroup
    static constexpr int BR = 64 * WR;           // rows of W of a workgroup
    static constexpr int THREADS = 128 * WR;
    static constexpr int BUF = BT * 128;         // bytes of a 64-column chunk of x
    static constexpr int LOADS = BT / 8 / (2 * WR);   // direct loads of a wave per chunk (8 tokens each)
    static_assert(LOADS >= 1, "a wave stages at least eight tokens");
};

// Tokens [t0, t0 + BT) x columns [64 c, 64 c + 64) of x into LDS: token r's
// 16-byte slot v holds columns 8 (v ^ ((r >> 1) & 7)).  Tokens beyond T read
// the last one (their results are not stored).
template <int TA, int WR>
__device__ __forceinline__ void prompt_stage(const uint16_t* __restrict__ x, int64_t ldx, int t0, int T, int c, char* s)
{
    typedef Prompt<TA, WR> P;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < P::LOADS; ++i) {
        const int q = wave * P::LOADS + i;
        const int r = 8 * q + (lane >> 3);
        const uint16_t* src = x + (int64_t)min(t0 + r, T - 1) * ldx + 64 * c + 8 * ((lane & 7) ^ ((r >> 1) & 7));
        __builtin_amdgcn_global_load_lds((global_cptr)src, (lds_ptr)(s + 1024 * q), 16, 0, 0);
    }
}

// The three-term split of a float32 value into bfloat16, v = a + b + c.
__device__ __forceinline__ void split3(float v, uint32_t& a, uint32_t& b, uint32_t& c)
{
    a = Bf16::down(v);
    const float r = v - Bf16::up((uint16_t)a);
    b = Bf16::down(r);
    c = Bf16::down(r - Bf16::up((uint16_t)b));
}

// Workgroups are dealt to the eight XCDs round-robin; each XCD gets a
// contiguous run of the tile order below, so that its L2 sees few tokens and
// rows at a time: runs of 4 token blocks share their rows of W.
__device__ __forceinline__ void prompt_tile(int nt, int nr, int& bt, int& br)
{
    const unsigned total = (unsigned)nt * nr, b = blockIdx.x;
    const unsigned per = total / 8, rest = total % 8, xcd = b % 8;
    const unsigned p = xcd * per + min(xcd, rest) + b / 8;
    const unsigned band = 4u * nr, g = p / band;
    const unsigned h = min(4u, (unsigned)nt - 4 * g);
    bt = (int)(4 * g + (p - g * band) % h);
    br = (int)((p - g * band) / h);
}

template <class X, int TA, int WR>
__global__ __launch_bounds__(128 * WR) void k_q4_prompt(const uint16_t* __restrict__ x, int64_t ldx,
                                                        int T, Q4Layer w,
                                                        const float* __restrict__ sums, int64_t lds_,
                                                        uint16_t* __restrict__ y, int64_t ldy, int nt,
                                                        int nr)
{
    typedef Prompt<TA, WR> P;
    typedef typename X::vec vec;
    __shared__ __align__(16) char lds[2 * P::BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, ml = lane & 31;
    const int wt = wave / WR, wr = wave % WR;
    int bt, br;
    prompt_tile(nt, nr, bt, br);
    const int t0 = bt * P::BT;
    const int nchunk = (w.n + 63) / 64;

    // this lane's row tile and its units (q = h and h + 2) of each 32-row tile
    int64_t unit[2], grid[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int rt = min(br * (P::BR / 16) + wr * 4 + 2 * b + (ml >> 4), w.RT - 1);
        unit[b] = (int64_t)rt * w.KB * 64 + 16 * h + (ml & 15);
        grid[b] = (int64_t)rt * w.G * 16 + (ml & 15);
    }
    f32x16 acc[TA][2];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

    u32x4 next[2][2], cur[2][2];
    float step[2];
    prompt_stage<TA, WR>(x, ldx, t0, T, 0, lds);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        next[b][0] = w.codes[unit[b]];
        next[b][1] = w.codes[unit[b] + 32];
        step[b] = w.grid[grid[b]].x;
    }
    int group = 0;
    for (int kb = 0; kb < w.KB; ++kb) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c = 2 * kb + half;
            if (c < nchunk) {
                wait_direct_loads();
                __syncthreads();
                if (c + 1 < nchunk) prompt_stage<TA, WR>(x, ldx, t0, T, c + 1, lds + ((half + 1) & 1) * P::BUF);
                if (half == 0) {
                    const int kn = min(kb + 1, w.KB - 1);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            cur[b][u] = next[b][u];
                            next[b][u] = w.codes[unit[b] + (int64_t)kn * 64 + 32 * u];
                        }
                }
                const int g = min(c / w.gb, w.G - 1);
                if (g != group) {
                    group = g;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float s = w.grid[grid[b] + (int64_t)g * 16].x;
                        const float ratio = step[b] / s;
                        step[b] = s;
#pragma unroll
                        for (int a = 0; a < TA; ++a)
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[a][b][r] *= ratio;
                    }
                }
                const char* s = lds + half * P::BUF;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        vec wf[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b) wf[b] = X::codes(cur[b][u][2 * half + d]);
                        const int slot = 4 * u + 2 * h + d;
#pragma unroll
                        for (int a = 0; a < TA; ++a) {
                            const int r = 32 * (wt * TA + a) + ml;
                            const vec xf = *reinterpret_cast<const vec*>(s + 128 * r + 16 * (slot ^ ((r >> 1) & 7)));
#pragma unroll
                            for (int b = 0; b < 2; ++b) acc[a][b] = X::mfma32(xf, wf[b], acc[a][b]);
                        }
                    }
            }
        }
    }
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] *= step[b];

    // minus s (16 + z) X: lane half h takes group g0 + h, slots
    // X1 Z1, X1 Z2, X2 Z1, X1 Z3, X2 Z2, X3 Z1
    for (int g0 = 0; g0 < w.G; g0 += 2) {
        const int g = g0 + h;
        bf16x8 zf[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t z1 = 0, z2 = 0, z3 = 0;
            if (g < w.G) {
                const f32x2 sz = w.grid[grid[b] + (int64_t)g * 16];
                split3(-sz.x * (sz.y + kQ4Offset), z1, z2, z3);
            }
            const u32x4 v = {z1 | (z2 << 16), z1 | (z3 << 16), z2 | (z1 << 16), 0u};
            zf[b] = __builtin_bit_cast(bf16x8, v);
        }
#pragma unroll
        for (int a = 0; a < TA; ++a) {
            const int t = min(t0 + 32 * (wt * TA + a) + ml, T - 1);
            uint32_t x1 = 0, x2 = 0, x3 = 0;
            if (g < w.G) split3(sums[(int64_t)g * lds_ + t], x1, x2, x3);
            const u32x4 v = {x1 | (x1 << 16), x2 | (x1 << 16), x2 | (x3 << 16), 0u};
            const bf16x8 xf = __builtin_bit_cast(bf16x8, v);
#pragma unroll
            for (int b = 0; b < 2; ++b) acc[a][b] = Bf16::mfma32(xf, zf[b], acc[a][b]);
        }
    }

#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = br * P::BR + wr * 64 + 32 * b + ml;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = t0 + 32 * (wt * TA + a) + 8 * (r >> 2) + 4 * h + (r & 3);
                if (t < T && row < w.m) y[(int64_t)t * ldy + row] = X::down(acc[a][b][r]);
            }
        }
}

// --------------------------------------------------------------------- host

struct PromptWork {
    int64_t lds_, ldc;
    size_t sums, copy, bytes;
};

static PromptWork prompt_work(int64_t T, int64_t n, int64_t G)
{
    PromptWork p;
    p.lds_ = ceil_div(T, 64) * 64;
    p.ldc = ceil_div(n, 64) * 64;
    p.sums = 0;
    p.copy = align_up((size_t)p.lds_ * G * 4);
    p.bytes = p.copy + align_up((size_t)T * p.ldc * 2);
    return p;
}

size_t q4_prompt_workspace_bytes(int64_t T, int64_t n, int64_t G) { return prompt_work(T, n, G).bytes; }

template <class X, int TA, int WR>
static void prompt_launch(const uint16_t* x, int64_t ldx, int64_t T, const Q4Layer& w, const float* sums, int64_t lds_,
                          uint16_t* y, int64_t ldy, hipStream_t s)
{
    typedef Prompt<TA, WR> P;
    const int nt = (int)ceil_div(T, P::BT), nr = (int)ceil_div(w.m, P::BR);
    launch(nullptr, KK_Q4_PROMPT, 2.0 * T * w.m * w.n, 0.0, k_q4_prompt<X, TA, WR>, dim3((unsigned)(nt * nr)),
           dim3(P::THREADS), s, x, ldx, (int)T, w, sums, lds_, y, ldy, nt, nr);
}

template <class X>
static int prompt_run(const void* x, int64_t ldx, int64_t T, const Q4Layer& w, void* y, int64_t ldy, void* ws,
                      hipStream_t s)
{
    const PromptWork p = prompt_work(T, w.n, w.G);
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    uint16_t* yp = static_cast<uint16_t*>(y);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(ws) + p.sums);
    uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + p.copy);
    const bool direct = w.n % 64 == 0 && ldx % 8 == 0 && aligned16(x);
    launch(nullptr, KK_Q4_SUMS, 0.0, 2.0 * T * w.n, direct ? k_q4_sums<X, false> : k_q4_sums<X, true>,
           dim3((unsigned)ceil_div(T, 4)), dim3(256), s, xp, ldx, (int)T, w.n, w.gb, w.G, sums, p.lds_, copy, p.ldc);
    if (!direct) xp = copy, ldx = p.ldc;
    const int64_t big = ceil_div(T, 256) * ceil_div(w.m, 256), mid = ceil_div(T, 128) * ceil_div(w.m, 256);
    if (big >= 256) prompt_launch<X, 4, 4>(xp, ldx, T, w, sums, p.lds_, yp, ldy, s);
    else if (mid >= 128) prompt_launch<X, 2, 4>(xp, ldx, T, w, sums, p.lds_, yp, ldy, s);
    else prompt_launch<X, 1, 2>(xp, ldx, T, w, sums, p.lds_, yp, ldy, s);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int q4_prompt_enqueue(const void* x, int64_t ldx, int64_t T, bool bf16, const Q4Layer& w, void* y, int64_t ldy, void* ws,
                      hipStream_t s)
{
    return bf16 ? prompt_run<Bf16>(x, ldx, T, w, y, ldy, ws, s) : prompt_run<Fp16>(x, ldx, T, w, y, ldy, ws, s);
}

}  // namespace bk
