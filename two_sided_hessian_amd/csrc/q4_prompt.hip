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
// of 64 columns by direct loads, 16-byte slots permuted so that
// fragment reads spread over the banks.  Codes come through LDS as they are
// (a quarter of the bytes of 16-bit weights); each wave expands its fragments
// in registers, 7 operations per 8 codes.  Two or three chunks are in flight
// at any time: a chunk's products take less than a load's latency.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4_tile.hpp"

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
    static constexpr int BT = 64 * TA;                // tokens of a workgroup
    static constexpr int BR = 64 * WR;                // rows of W of a workgroup
    static constexpr int XBUF = BT * 128;             // bytes of a 64-column chunk of x
    static constexpr int WBUF = BR * 64;              // bytes of a 128-column block of codes
    static constexpr int AHEAD = TA == 4 ? 2 : 3;     // chunks in flight (LDS has no room for 3 of TA = 4)
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
    int nchunk, KB, G, gb, wave;
    int group = 0, in_group = 0;   // of the next chunk staged, and chunks of that group staged before it
    char* lds;

    __device__ __forceinline__ PromptStage(const uint16_t* xp, int64_t ldx, int t0, int T, const Q4Layer& w, int rt0,
                                           char* lds_)
        : x(buffer_of(xp + t0 * ldx, 0x7FFFFFFFu)),
          codes(buffer_of(w.codes + (int64_t)rt0 * w.KB * 64, 0x7FFFFFFFu)),
          grid(buffer_of(w.grid + (int64_t)rt0 * w.G * 16, 0x7FFFFFFFu)),
          nchunk((w.n + 63) / 64), KB(w.KB), G(w.G), gb(w.gb),
          wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), lds(lds_)
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
    // called for c = 0, 1, ... in turn; bx, bw: the buffers of chunk c and of
    // column block c / 2 + 1; part = c & 1
    __device__ __forceinline__ void chunk(int c, int bx, int bw, int part)
    {
        const int cx = min(c, nchunk - 1);
        char* s = lds + bx * P::XBUF + wave * P::XLOADS * 1024;
#pragma unroll
        for (int i = 0; i < P::XLOADS; ++i) load_lds16(x, x_at[i], 128 * cx, s + 1024 * i);
        load_lds4(grid, grid_at, 128 * group, lds + P::GRID + bx * P::GBUF + 256 * wave);
        if (++in_group == gb) in_group = 0, group = min(group + 1, G - 1);
        load_lds16(codes, code_at[part], 1024 * min((c >> 1) + 1, KB - 1),
                     lds + P::CODES + bw * P::WBUF + 1024 * (part * 2 * WR + wave));
    }
    __device__ __forceinline__ void first() const
    {
#pragma unroll
        for (int p = 0; p < 2; ++p) load_lds16(codes, code_at[p], 0, lds + P::CODES + 1024 * (p * 2 * WR + wave));
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

template <class X, int TA, int WR>
__global__ __launch_bounds__(128 * WR, 2) void k_q4_prompt(const uint16_t* __restrict__ x, int64_t ldx, int T, Q4Layer w,
                                                        const float* __restrict__ sums, int64_t lds_,
                                                        uint16_t* __restrict__ y, int64_t ldy, int nt, int nr)
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
    PromptStage<TA, WR> stage(x, ldx, t0, T, w, rt0, lds);
    stage.first();
#pragma unroll
    for (int c = 0; c < P::AHEAD; ++c) stage.chunk(c, c, ((c >> 1) + 1) % P::NW, c & 1);

    f32x16 acc[TA][2];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

    u32x4 codes[2][2];   // [row tile pair][unit h, h + 2]
    float step[2] = {1.f, 1.f};
    int left = 0;        // chunks left of the group whose steps the accumulators count in
    int bx = 0, bw = 0;                                  // buffers of chunk c and block kb
    int px = P::AHEAD, pw = (P::AHEAD / 2 + 1) % P::NW;   // and of the ones staged beside them
    // the lane's parts of the LDS addresses
    uint32_t x_lane[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
        x_lane[v] = 128 * (32 * wt * TA + ml) + 16 * ((4 * (v >> 1) + 2 * h + (v & 1)) ^ ((ml >> 1) & 7));
    const uint32_t w_lane = P::CODES + 1024 * (4 * wr + (ml >> 4)) + 256 * h + 16 * (ml & 15);
    const uint32_t g_lane = P::GRID + 8 * (64 * wr + ml);
    for (int kb = 0; kb < w.KB; ++kb) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c = 2 * kb + half;
            if (c < stage.nchunk) {
                tile_wait<(P::AHEAD - 1) * P::LOADS>();
                stage.chunk(c + P::AHEAD, px, pw, (half + P::AHEAD) & 1);
                px = px + 1 == P::NX ? 0 : px + 1;
                if ((half + P::AHEAD) & 1) pw = pw + 1 == P::NW ? 0 : pw + 1;
                if (half == 0) {
                    const char* s = lds + w_lane + bw * P::WBUF;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            codes[b][u] = *reinterpret_cast<const u32x4*>(s + 2048 * b + 512 * u);
                }
                if (left-- == 0) {
                    left = w.gb - 1;
                    const char* s = lds + g_lane + bx * P::GBUF;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float s1 = *reinterpret_cast<const float*>(s + 256 * b);
                        const float ratio = step[b] * __builtin_amdgcn_rcpf(s1);
                        step[b] = s1;
#pragma unroll
                        for (int a = 0; a < TA; ++a)
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[a][b][r] *= ratio;
                    }
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
#pragma unroll
                    for (int a = 0; a < TA; ++a)
#pragma unroll
                        for (int b = 0; b < 2; ++b) acc[a][b] = X::mfma32(xf[v % (PRE + 1)][a], wf[b], acc[a][b]);
                }
                bx = bx + 1 == P::NX ? 0 : bx + 1;
            }
        }
        bw = bw + 1 == P::NW ? 0 : bw + 1;
    }
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] *= step[b];
    int64_t grid[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
        grid[b] = (int64_t)min(rt0 + wr * 4 + 2 * b + (ml >> 4), w.RT - 1) * w.G * 16 + (ml & 15);

    // minus s (16 + z) X: lane half h takes group g0 + 2 j + h, slots
    // X1 Z1, X1 Z2, X2 Z1, X1 Z3, X2 Z2, X3 Z1; four pairs of groups at a time
    // so that their loads are in flight together
    constexpr int GP = 4;
    for (int g0 = 0; g0 < w.G; g0 += 2 * GP) {
        f32x2 sz[GP][2];
        float xs[GP][TA];
#pragma unroll
        for (int j = 0; j < GP; ++j) {
            const int g = min(g0 + 2 * j + h, w.G - 1);
#pragma unroll
            for (int b = 0; b < 2; ++b) sz[j][b] = w.grid[grid[b] + (int64_t)g * 16];
#pragma unroll
            for (int a = 0; a < TA; ++a)
                xs[j][a] = sums[(int64_t)g * lds_ + min(t0 + 32 * (wt * TA + a) + ml, T - 1)];
        }
#pragma unroll
        for (int j = 0; j < GP; ++j) {
            const float in = g0 + 2 * j + h < w.G ? 1.f : 0.f;   // groups beyond G add nothing
            bf16x8 zf[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t z1, z2, z3;
                split3(in * (-sz[j][b].x * (sz[j][b].y + kQ4Offset)), z1, z2, z3);
                const u32x4 v = {z1 | (z2 << 16), z1 | (z3 << 16), z2 | (z1 << 16), 0u};
                zf[b] = __builtin_bit_cast(bf16x8, v);
            }
#pragma unroll
            for (int a = 0; a < TA; ++a) {
                uint32_t x1, x2, x3;
                split3(xs[j][a], x1, x2, x3);
                const u32x4 v = {x1 | (x1 << 16), x2 | (x1 << 16), x2 | (x3 << 16), 0u};
                const bf16x8 xf = __builtin_bit_cast(bf16x8, v);
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[a][b] = Bf16::mfma32(xf, zf[b], acc[a][b]);
            }
        }
    }

    wait_direct_loads();
    __syncthreads();
    tile_store<X, TA>(acc, 1.f, lds, t0 + 32 * wt * TA, T, br * P::BR + wr * 64, w.m, y, ldy);
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

template <class X>
void copy_enqueue(const uint16_t* x, int64_t ldx, int64_t T, int n, uint16_t* copy, int64_t ldc, hipStream_t s)
{
    launch(nullptr, KK_Q4_SUMS, 0.0, 4.0 * T * n, k_q4_sums<X, true>, dim3((unsigned)ceil_div(T, 4)), dim3(256), s, x, ldx,
           (int)T, n, 1, 0, static_cast<float*>(nullptr), (int64_t)0, copy, ldc);
}
template void copy_enqueue<Bf16>(const uint16_t*, int64_t, int64_t, int, uint16_t*, int64_t, hipStream_t);
template void copy_enqueue<Fp16>(const uint16_t*, int64_t, int64_t, int, uint16_t*, int64_t, hipStream_t);

template <class X, int TA, int WR>
static void prompt_launch(const uint16_t* x, int64_t ldx, int64_t T, const Q4Layer& w, const float* sums, int64_t lds_,
                          uint16_t* y, int64_t ldy, hipStream_t s)
{
    typedef Prompt<TA, WR> P;
    const int nt = (int)ceil_div(T, P::BT), nr = (int)ceil_div(w.m, P::BR);
    launch(nullptr, KK_Q4_PROMPT, 2.0 * T * w.m * w.n, 0.0, k_q4_prompt<X, TA, WR>, dim3((unsigned)(nt * nr)),
           dim3(128 * WR), s, x, ldx, (int)T, w, sums, lds_, y, ldy, nt, nr);
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
    // (the staging offsets of a token block are 31 bits)
    const bool direct = w.n % 64 == 0 && ldx % 8 == 0 && ldx <= (1 << 21) && aligned16(x);
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
