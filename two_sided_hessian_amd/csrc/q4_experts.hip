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
//   * few rows per expert (decoding): codes are what is read.  k_q4_experts_few
//     has blocks of up to 32 rows and row tiles of W over workgroups; HBM bounds it.
//   * many: k_q4_experts and k_q4_experts_grad, tiles of 64 .. 256 rows, MFMAs.
#include <algorithm>

#include "moe.hpp"
#include "q4_grad.hpp"
#include "q4_prompt.hpp"

namespace bk {

constexpr int kExperts = BAKRON_MOE_MAX_EXPERTS;
static_assert(kExperts <= 4 * 64, "four experts a lane");

// The rows of block `block` of BT rows each, counted expert by expert; blocks(total)
// says which one is wanted (-1: none).  A wave's work, the same in every wave.
struct ExpertRows {
    int e, t0, t1;   // the expert, the block's first row, and the expert's end
};
template <class Pick>
__device__ __forceinline__ bool expert_rows(const int32_t* __restrict__ offsets, int E, int R, int BT, Pick pick, ExpertRows& out)
{
    const int lane = threadIdx.x & 63;
    int o[5];
#pragma unroll
    for (int u = 0; u < 5; ++u) o[u] = min(max(offsets[min(4 * lane + u, E)], 0), R);
    int tiles[4], sum = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        tiles[u] = (max(o[u + 1] - o[u], 0) + BT - 1) / BT;
        sum += tiles[u];
    }
    int upto = sum;
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(upto, off);
        if (lane >= off) upto += v;
    }
    const int want = pick(__builtin_amdgcn_readlane(upto, 63));
    if (want < 0) return false;
    const unsigned long long at = __ballot(upto > want);
    if (!at) return false;
    const int l = __ffsll(at) - 1;
    int k = want - __builtin_amdgcn_readlane(upto - sum, l);
    int e = 4 * l, first = __builtin_amdgcn_readlane(o[0], l), last = __builtin_amdgcn_readlane(o[1], l);
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int n = __builtin_amdgcn_readlane(tiles[u], l);
        if (e == 4 * l + u && k >= n) {
            k -= n;
            ++e;
            first = __builtin_amdgcn_readlane(o[u + 1], l);
            last = __builtin_amdgcn_readlane(o[u + 2], l);
        }
    }
    out = ExpertRows{e, first + k * BT, last};
    return true;
}

// The output tile of this workgroup: block of rows and column bc of nc.
template <int BT>
__device__ __forceinline__ bool expert_tile(const int32_t* __restrict__ offsets, int E, int R, int most, int nc,
                                            ExpertRows& rows, int& bc)
{
    return expert_rows(offsets, E, R, BT, [&](int nt) {
        nt = min(nt, most);
        if ((int)blockIdx.x >= nt * nc) return -1;
        int bt;
        tile_of(nt, nc, bt, bc);
        return bt;
    }, rows);
}

template <class X, int TA, int WR, bool OWN>
__global__ __launch_bounds__(128 * WR, 2) void k_q4_experts(const uint16_t* __restrict__ x, int64_t ldx, int R,
                                                            const int32_t* __restrict__ offsets, int E, Q4Layer stack,
                                                            int64_t layer_bytes, const float* __restrict__ sums, int64_t lds_,
                                                            uint16_t* __restrict__ y, int64_t ldy, int most, int nr,
                                                            float* __restrict__ part)
{
    ExpertRows rows;
    int br;
    if (!expert_tile<64 * TA>(offsets, E, R, most, nr, rows, br)) return;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    prompt_tile<X, TA, WR, OWN>(x, ldx, rows.t0, rows.t1, w, sums, lds_, y, ldy, br, part, R);
}

template <class X, int TA>
__global__ __launch_bounds__(512) void k_q4_experts_grad(const uint16_t* __restrict__ dy, int64_t lddy, int R,
                                                         const int32_t* __restrict__ offsets, int E, Q4Layer stack,
                                                         int64_t layer_bytes, uint16_t* __restrict__ dx, int64_t lddx,
                                                         int most, int nj, float* __restrict__ part)
{
    ExpertRows rows;
    int bj;
    if (!expert_tile<64 * TA>(offsets, E, R, most, nj, rows, bj)) return;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    grad_tile<X, TA>(dy, lddy, rows.t0, rows.t1, w, dx, lddx, bj, part, R);
}

// The sum of `splits` partial results, in order, for the rows that some expert
// has.
template <class X>
__global__ __launch_bounds__(256) void k_q4_experts_join(const float* __restrict__ part, int splits, int R,
                                                         const int32_t* __restrict__ offsets, int E, int m,
                                                         uint16_t* __restrict__ y, int64_t ldy)
{
    const int col = blockIdx.y * 256 + threadIdx.x, row = blockIdx.x;
    if (col >= m || row < offsets[0] || row >= offsets[E]) return;
    const int64_t all = (int64_t)R * m;
    const float* p = part + (int64_t)row * m + col;
    constexpr int U = 8;
    float v = 0.f;
    for (int u0 = 0; u0 < splits; u0 += U) {
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = p[min(u0 + u, splits - 1) * all];
#pragma unroll
        for (int u = 0; u < U; ++u) v += u0 + u < splits ? a[u] : 0.f;
    }
    y[row * ldy + col] = X::down(v);
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

constexpr int kFewRows = 32;
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
    ExpertRows rows;
    const int want = blockIdx.y;
    if (!expert_rows(offsets, E, R, kFewRows, [&](int) { return want; }, rows)) return;
    const Q4Layer w = expert_layer(stack, rows.e, layer_bytes);
    const int rt0 = 16 / WS * blockIdx.x, n = min(kFewRows, rows.t1 - rows.t0);
    if (n <= 4) few_rows_of<X, 1, 2, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
    else if (n <= 16) few_rows_of<X, 4, 1, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
    else few_rows_of<X, 8, 1, WS, HALF>(x, ldx, w, rt0, rows.t0, n, lds, y, ldy);
}

// --------------------------------------------------------------------- host

struct ExpertsPlan {
    bool few;
    int TA, WR, splits;
    int64_t most;      // blocks of rows that there can be
    int pieces;
    int64_t lds_, ldc;
    size_t copy, part, bytes;
};

// Blocks of `tokens` rows: at most, and about how many there will be.
static int64_t blocks_most(int64_t R, int64_t E, int64_t tokens) { return R / tokens + std::min(R, E); }
static int64_t blocks_about(int64_t R, int64_t E, int64_t tokens)
{
    const int64_t some = std::min(R, E);
    return std::max(some, R / tokens + some / 2);
}

static ExpertsPlan experts_plan(int64_t R, int64_t E, int64_t m, int64_t n, int gb)
{
    ExpertsPlan p{};
    p.few = R <= kFewRows * E;
    if (p.few) return p;
    // the linear layer's tiles and costs (q4_prompt.hip)
    static constexpr TileShape shapes[] = {{256, 256, 128.0}, {128, 256, 80.0}, {128, 128, 42.0}, {64, 128, 28.0}};
    const TileChoice c = tile_choose_of(shapes, [=](int tokens) { return blocks_about(R, E, tokens); }, R, m, n,
                                        std::min<int64_t>(8, ceil_div(n, kQ4Cols) / 2));
    p.TA = shapes[c.shape].tokens / 64;
    p.WR = shapes[c.shape].cols / 64;
    p.splits = c.splits;
    p.most = blocks_most(R, E, shapes[c.shape].tokens);
    p.lds_ = ceil_div(R, 256) * 256 + 256;   // a block's sums are read as a whole, whichever row it begins at
    p.ldc = ceil_div(n, 64) * 64;
    p.pieces = piece_at((int)((n - 1) / 64), gb) + 1;
    p.copy = align_up((size_t)p.lds_ * p.pieces * 4);
    p.part = p.copy + align_up((size_t)R * p.ldc * 2);
    p.bytes = p.part + (p.splits > 1 ? align_up((size_t)p.splits * R * m * 4) : 0);
    return p;
}

static ExpertsPlan experts_grad_plan(int64_t R, int64_t E, int64_t m, int64_t n)
{
    ExpertsPlan p{};
    static constexpr TileShape shapes[] = {{256, 256, 130.0}, {128, 256, 88.0}, {64, 256, 64.0}};   // as in q4_grad.hip
    const TileChoice c = tile_choose_of(shapes, [=](int tokens) { return blocks_about(R, E, tokens); }, R, n, m,
                                        std::min<int64_t>(16, ceil_div(m, 64) / 2));
    p.TA = shapes[c.shape].tokens / 64;
    p.splits = c.splits;
    p.most = blocks_most(R, E, shapes[c.shape].tokens);
    p.ldc = ceil_div(m, 64) * 64;
    p.part = align_up((size_t)R * p.ldc * 2);
    p.bytes = p.part + (p.splits > 1 ? align_up((size_t)p.splits * R * n * 4) : 0);
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
    enqueue(k_q4_experts_join<X>, dim3((unsigned)c.rows, (unsigned)ceil_div(cols, 256)), dim3(256), c.s, part, splits,
            (int)c.rows, c.offsets, (int)c.E, (int)cols, c.out, c.ldout);
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
    enqueue(k_q4_experts<X, TA, WR, OWN>, dim3((unsigned)(p.most * nr), (unsigned)p.splits), dim3(128 * WR), c.s, x, ldx,
            (int)c.rows, c.offsets, (int)c.E, w, (int64_t)c.d.bytes, reinterpret_cast<const float*>(c.ws), p.lds_, c.out,
            c.ldout, (int)p.most, nr, reinterpret_cast<float*>(c.ws + p.part));
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
    const bool own = p.TA == 1 && (direct || p.splits > 1);   // as in q4_prompt.hip
    const uint16_t* x = c.in;
    int64_t ldx = c.ldin;
    uint16_t* copy = reinterpret_cast<uint16_t*>(c.ws + p.copy);
    if (!own)
        enqueue(direct ? k_q4_sums<X, false> : k_q4_sums<X, true>, dim3((unsigned)ceil_div(c.rows, 4)), dim3(256), c.s, x, ldx,
                (int)c.rows, w.n, w.gb, p.pieces, reinterpret_cast<float*>(c.ws), p.lds_, copy, p.ldc);
    else if (!direct) copy_enqueue<X>(x, ldx, c.rows, w.n, copy, p.ldc, c.s);
    if (!direct) x = copy, ldx = p.ldc;
    if (p.TA == 4) experts_launch<X, 4, 4, false>(c, p, w, x, ldx);
    else if (p.TA == 2 && p.WR == 2) experts_launch<X, 2, 2, false>(c, p, w, x, ldx);
    else if (p.TA == 2) experts_launch<X, 2, 4, false>(c, p, w, x, ldx);
    else if (own) experts_launch<X, 1, 2, true>(c, p, w, x, ldx);
    else experts_launch<X, 1, 2, false>(c, p, w, x, ldx);
    if (p.splits > 1) experts_join<X>(c, reinterpret_cast<const float*>(c.ws + p.part), p.splits, w.m);
}

template <class X, int TA>
static void experts_grad_launch(const ExpertsCall& c, const ExpertsPlan& p, const Q4Layer& w, const uint16_t* dy, int64_t lddy)
{
    const int nj = (int)ceil_div(w.n, 256);
    enqueue(k_q4_experts_grad<X, TA>, dim3((unsigned)(p.most * nj), (unsigned)p.splits), dim3(512), c.s, dy, lddy, (int)c.rows,
            c.offsets, (int)c.E, w, (int64_t)c.d.bytes, c.out, c.ldout, (int)p.most, nj, reinterpret_cast<float*>(c.ws + p.part));
}

template <class X>
static void experts_grad_run(const ExpertsCall& c)
{
    const Q4Layer w = q4_layer(c.packed, c.d);
    const ExpertsPlan p = experts_grad_plan(c.rows, c.E, w.m, w.n);
    const uint16_t* dy = c.in;
    int64_t lddy = c.ldin;
    if (w.m % 64 || lddy % 8 || lddy > (1 << 21) || !aligned16(dy)) {
        copy_enqueue<X>(dy, lddy, c.rows, w.m, reinterpret_cast<uint16_t*>(c.ws), p.ldc, c.s);
        dy = reinterpret_cast<const uint16_t*>(c.ws);
        lddy = p.ldc;
    }
    if (p.TA == 4) experts_grad_launch<X, 4>(c, p, w, dy, lddy);
    else if (p.TA == 2) experts_grad_launch<X, 2>(c, p, w, dy, lddy);
    else experts_grad_launch<X, 1>(c, p, w, dy, lddy);
    if (p.splits > 1) experts_join<X>(c, reinterpret_cast<const float*>(c.ws + p.part), p.splits, w.n);
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
    return bk::experts_grad_plan(rows, experts, m, n).bytes;
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
