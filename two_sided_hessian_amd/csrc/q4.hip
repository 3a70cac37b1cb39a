// q4.hip -- 4-bit layers: packing, the linear layer and its input gradient.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4_few.hpp"

namespace bk {

// ------------------------------------------------------------------ packing
//
// One thread per 16-byte unit: 32 codes of one row, read as two runs of 16
// (four lanes a row's 64 bytes; a wave writes one block of 1 KB).  HBM bounds
// it: 1.5 bytes a code (4096 x 14336: 18.9 us, 4.7 TB/s).

// Rows of codes may start at any byte.
typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// a dword of codes from eight codes, four to a dword
__device__ __forceinline__ uint32_t pack8(uint32_t lo, uint32_t hi)
{
    // even codes to the low half, odd ones to the high half, 4 bits each
    const uint32_t e0 = lo & 0x000F000Fu, o0 = lo >> 8 & 0x000F000Fu, e1 = hi & 0x000F000Fu, o1 = hi >> 8 & 0x000F000Fu;
    const uint32_t e = ((e0 | e0 >> 12) & 0xFFu) | ((e1 | e1 >> 12) & 0xFFu) << 8;
    const uint32_t o = ((o0 | o0 >> 12) & 0xFFu) | ((o1 | o1 >> 12) & 0xFFu) << 8;
    return __builtin_rotateleft32(e | o << 16, 3);
}

__global__ __launch_bounds__(256) void k_q4_pack(const uint8_t* __restrict__ codes, const float* __restrict__ scale,
                                                 int64_t m, int64_t n, int RT, int KB, int G, int gb,
                                                 int64_t layer_bytes, int64_t unit_at, char* __restrict__ packed)
{
    if (blockIdx.x == 0)   // k_q4_pack_grid raises them
        for (int g = threadIdx.x; g < G; g += 256)
            reinterpret_cast<float*>(packed + blockIdx.y * layer_bytes + unit_at)[g] = 0.f;
    const int64_t block = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (block >= (int64_t)RT * KB) return;
    const int64_t layer = blockIdx.y;
    const int q = threadIdx.x & 3, r = threadIdx.x >> 2 & 15;
    const int64_t row = block / KB * kQ4Rows + r;
    const int64_t col0 = block % KB * kQ4Cols + 16 * q;
    u32x4 out = {0u, 0u, 0u, 0u};
    if (row < m) {
        const uint8_t* src = codes + (layer * m + row) * n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c0 = col0 + 64 * h;
            if (c0 >= n) continue;
            const int64_t g = min((int)(c0 >> 6) / gb, G - 1);
            if (scale[(layer * m + row) * G + g] == 0.f) continue;   // weights of 0: see k_q4_pack_grid
            u32x4 v = {0u, 0u, 0u, 0u};
            if (c0 + 16 <= n) {
                v = *reinterpret_cast<const u32x4_byte*>(src + c0);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c0 + e < n) v[e >> 2] |= (uint32_t)src[c0 + e] << (8 * (e & 3));
            }
            out[2 * h] = pack8(v[0], v[1]);
            out[2 * h + 1] = pack8(v[2], v[3]);
        }
    }
    reinterpret_cast<u32x4*>(packed + layer * layer_bytes)[block * 64 + 16 * q + r] = out;
}

// Grids, and the units: the exponent, rounded up, of the largest weight of each
// group's columns (a maximum of integers, which does not depend on the order it
// is taken in).  A row has LANES lanes, as many as it has groups, 16 at most, and
// a workgroup 16 / LANES row tiles at a time; at most so many workgroups per layer
// that few atomics meet at a unit.  4096 x 14336 in groups of 128: 11.8 us (128
// workgroups: 15.5); 65536 rows with a grid each: 5.9 (16 lanes a row: 15.5).
//
// A step of 0 (every weight 0, whatever the codes) is written as the row's
// smallest step, zero point 0, on codes of 0: kernels divide by steps, and
// k_q4_prompt counts a whole row in units of one step after the other, adding
// 16 sum x under the present one and taking it off again.  Under a step above
// the row's others (1, say) that difference's float32 error would bury them.
// Rows without any step take the smallest normal number.
constexpr int kPackGridBlocks = 512;
constexpr float kPackNoStep = 0x1p-126f;

template <int LANES>
__global__ __launch_bounds__(256) void k_q4_pack_grid(const float* __restrict__ scale, const float* __restrict__ zero,
                                                      int64_t m, int RT, int G, int64_t layer_bytes, int64_t grid_at,
                                                      int64_t unit_at, char* __restrict__ packed)
{
    constexpr int TILES = 16 / LANES;
    __shared__ unsigned tops[kQ4MaxHalves];   // floats from 0 on; a group has 64 columns at least
    __shared__ float least[16][kQ4Rows];
    const int64_t layer = blockIdx.y;
    const int r = threadIdx.x & 15, q = threadIdx.x >> 4, g0 = q % LANES;
    for (int g = threadIdx.x; g < G; g += 256) tops[g] = 0u;
    for (int tile0 = blockIdx.x * TILES; tile0 < RT; tile0 += gridDim.x * TILES) {
        const int tile = tile0 + q / LANES;
        const int64_t row = (int64_t)tile * kQ4Rows + r;
        const int64_t at = (layer * m + row) * G;
        float low = INFINITY;
        if (row < m)
            for (int g = g0; g < G; g += LANES) {
                const float s = fabsf(scale[at + g]);
                if (s > 0.f) low = fminf(low, s);
            }
        least[q][r] = low;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LANES; ++i) low = fminf(low, least[q / LANES * LANES + i][r]);
        if (low == INFINITY) low = kPackNoStep;
        f32x2* out = reinterpret_cast<f32x2*>(packed + layer * layer_bytes + grid_at) + (int64_t)tile * G * kQ4Rows + r;
        for (int g = g0; g < G && tile < RT; g += LANES) {
            f32x2 v = {0.f, 0.f};
            float top = 0.f;
            if (row < m) {
                v.x = scale[at + g];
                v.y = zero[at + g];
                if (v.x == 0.f) v = f32x2{low, 0.f};
                else top = fabsf(v.x) * fmaxf(fabsf(v.y), fabsf(15.f - v.y));
            }
            out[g * kQ4Rows] = v;
            for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));   // (16 rows, all here)
            if (r == 0) atomicMax(&tops[g], __float_as_uint(top));
        }
        __syncthreads();   // the next tiles' minima overwrite these
    }
    unsigned* units = reinterpret_cast<unsigned*>(packed + layer * layer_bytes + unit_at);
    for (int g = threadIdx.x; g < G; g += 256) {
        const float top = __uint_as_float(tops[g]);
        if (top > 0.f && top < INFINITY) atomicMax(&units[g], max(min((__float_as_uint(top) >> 23) + 1u, 254u), 1u) << 23);
    }
}

// ------------------------------------------- the linear layer, a few tokens
//
// One workgroup per R tiles of 16 rows of W and 4 TQ tokens; its waves take the
// column blocks in turn (FewSpan) and are joined through LDS in wave order,
// so the result does not depend on timing.
//
// Measured, layers from HBM (1.2 GB of them in turn) and one layer over and over,
// from the Infinity Cache: two tokens x 28672 x 8192, groups of 128: 25.8 us, 5.1
// TB/s (the rate of a 1 GiB copy), and 22.3; one token x 4096 x 14336: 9.4 us, 3.5
// TB/s, and 6.7, of which 2.2 are those of a 1024 x 1024 layer, a launch and a
// round trip; 16 tokens x 14336 x 4096, groups of 64: 12.2 us, 3.0 TB/s, and 9.3;
// 64 tokens x 4096 x 4096: 11.4 us and 10.1: 256 workgroups of 16 rows each read all
// of x, 134 MB through the L2 caches, and expanding for four tiles of tokens at
// once holds too many registers for more waves.
template <class X, int TQ, int R, int WAVES, int U, bool HALF>
__global__ __launch_bounds__(64 * WAVES) void k_q4_few(const uint16_t* __restrict__ x, int64_t ldx, int T, Q4Layer w,
                                                       uint16_t* __restrict__ y, int64_t ldy)
{
    typedef FewSpan<X, TQ, R, U, HALF> Span;
    constexpr int NT = Span::NT, N = R * NT * 4;
    constexpr int STAGE = WAVES * few_lds(TQ), JOIN = WAVES * N * 64 * 4;
    __shared__ __align__(16) char lds[STAGE > JOIN ? STAGE : JOIN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rt = blockIdx.x * R, t0 = blockIdx.y * 4 * TQ;
    const uint16_t* xr[TQ];
#pragma unroll
    for (int t = 0; t < TQ; ++t) xr[t] = x + (int64_t)min(t0 + 4 * t + (lane >> 4), T - 1) * ldx;
    const Q4Layer ws[1] = {w};
    Span span(lds + wave * few_lds(TQ));
    span.template rows<1>(ws, rt);
    span.tokens(xr);
    span.run(wave, WAVES, w.KB);
    __syncthreads();   // the joining sums overwrite the staged tokens
    float(*red)[N][64] = reinterpret_cast<float(*)[N][64]>(lds);
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[wave][4 * (j * NT + i) + e][lane] = span.acc[j][i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < N * 64; o += 64 * WAVES) {
        const int e = o >> 6, l = o & 63;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < WAVES; ++u) v += red[u][e][l];
        const int t = t0 + 16 * ((e >> 2) % NT) + 4 * (l >> 4) + (e & 3), row = (rt + (e >> 2) / NT) * 16 + (l & 15);
        if (t < T && row < w.m) y[(int64_t)t * ldy + row] = X::down(v);
    }
}

// rows x cols zeros of a 2-byte type
__global__ __launch_bounds__(256) void k_q4_zero(uint16_t* __restrict__ y, int64_t ld, int64_t rows, int64_t cols)
{
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * cols; e += (int64_t)gridDim.x * 256)
        y[e / cols * ld + e % cols] = 0;
}

int q4_zero_enqueue(void* y, int64_t ld, int64_t rows, int64_t cols, hipStream_t s)
{
    launch(nullptr, KK_Q4_ZERO, 0.0, 2.0 * rows * cols, k_q4_zero,
           dim3((unsigned)std::min<int64_t>(65536, ceil_div(rows * cols, 256))), dim3(256), s, static_cast<uint16_t*>(y), ld, rows, cols);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <class X, int TQ, int R, int WAVES, int U>
static void few_launch(const uint16_t* x, int64_t ldx, int T, const Q4Layer& w, uint16_t* y, int64_t ldy, hipStream_t s)
{
    // HALF: a group ends inside a block of 128 columns
    launch(nullptr, KK_Q4_FEW, 2.0 * T * w.m * w.n, 0.0,
           w.gb % 2 ? k_q4_few<X, TQ, R, WAVES, U, true> : k_q4_few<X, TQ, R, WAVES, U, false>,
           dim3((unsigned)ceil_div(w.RT, R), (unsigned)ceil_div(T, 4 * TQ)), dim3(64 * WAVES), s, x, ldx, T, w, y, ldy);
}

// Two row tiles per workgroup where that still gives every CU one: they share
// the reads of x (16 tokens x 14336 x 4096: 11.9 us with one, 10.0 with two;
// one token x 4096 x 14336, where two would leave half the CUs idle: 7.7 with
// one, 10.4 with two).  Up to four tokens a lone row tile is spread over 16
// waves, a block each at a time, instead of 8 with two (one token x 4096 x
// 14336: 7.7 us and 8.1; two row tiles, 14336 x 4096: 8.9 and 8.0).
template <class X, int TQ, int WAVES, int U>
static void few_rows(const uint16_t* x, int64_t ldx, int T, const Q4Layer& w, uint16_t* y, int64_t ldy, hipStream_t s)
{
    if (w.RT >= 512) few_launch<X, TQ, 2, 8, WAVES * U / 8>(x, ldx, T, w, y, ldy, s);
    else few_launch<X, TQ, 1, WAVES, U>(x, ldx, T, w, y, ldy, s);
}

template <class X>
static void few_enqueue(const void* x, int64_t ldx, int64_t T, const Q4Layer& w, void* y, int64_t ldy, hipStream_t s)
{
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    uint16_t* yp = static_cast<uint16_t*>(y);
    const int t = (int)T;
    if (T <= 4) few_rows<X, 1, 16, 1>(xp, ldx, t, w, yp, ldy, s);
    else if (T <= 8) few_rows<X, 2, 8, 2>(xp, ldx, t, w, yp, ldy, s);
    else if (T <= 16) few_rows<X, 4, 8, 2>(xp, ldx, t, w, yp, ldy, s);
    else if (T <= 32) few_rows<X, 8, 8, 1>(xp, ldx, t, w, yp, ldy, s);
    else few_rows<X, 16, 8, 1>(xp, ldx, t, w, yp, ldy, s);
}

}  // namespace bk

// ------------------------------------------------------------------- C ABI

static bool q4_shape_ok(int64_t m, int64_t n)
{
    return m >= 0 && n >= 0 && m <= BAKRON_MAX_DIM && n <= BAKRON_MAX_DIM;
}

static bool q4_group_ok(int64_t g) { return g >= 0 && g % 64 == 0; }

extern "C" {

size_t bakron_q4_packed_bytes(int64_t count, int64_t m, int64_t n, int64_t group_size)
{
    if (!q4_shape_ok(m, n) || !q4_group_ok(group_size) || count < 0 || count > BAKRON_Q4_MAX_LAYERS) return 0;
    if (m == 0 || n == 0) return 0;
    return (size_t)count * bk::q4_dims(m, n, group_size).bytes;
}

int bakron_q4_pack(const uint8_t* codes, const float* scale, const float* zero, int64_t count, int64_t m, int64_t n,
                   int64_t group_size, void* packed, hipStream_t stream)
{
    if (!q4_shape_ok(m, n) || count < 0 || count > BAKRON_Q4_MAX_LAYERS) return BAKRON_ERR_BAD_SIZE;
    if (!q4_group_ok(group_size)) return BAKRON_ERR_BAD_ARG;
    if (m == 0 || n == 0 || count == 0) return BAKRON_SUCCESS;
    if (!codes || !scale || !zero || !packed) return BAKRON_ERR_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(packed) % bk::kAlign) return BAKRON_ERR_BAD_ARG;
    const bk::Q4Dims d = bk::q4_dims(m, n, group_size);
    char* out = static_cast<char*>(packed);
    const double mn = (double)count * m * n;
    bk::launch(nullptr, bk::KK_Q4_PACK, 0.0, 1.5 * mn, bk::k_q4_pack,
               dim3((unsigned)bk::ceil_div((int64_t)d.RT * d.KB, 4), (unsigned)count), dim3(256), stream, codes, scale,
               m, n, d.RT, d.KB, d.G, d.gb, (int64_t)d.bytes, (int64_t)d.unit_at, out);
    const int lanes = d.G > 8 ? 16 : d.G > 4 ? 8 : d.G > 2 ? 4 : d.G;
    auto* grids = lanes == 16 ? bk::k_q4_pack_grid<16> : lanes == 8 ? bk::k_q4_pack_grid<8>
                : lanes == 4 ? bk::k_q4_pack_grid<4> : lanes == 2 ? bk::k_q4_pack_grid<2> : bk::k_q4_pack_grid<1>;
    bk::launch(nullptr, bk::KK_Q4_PACK_GRID, 0.0, 16.0 * count * m * d.G, grids,
               dim3((unsigned)std::min<int64_t>(bk::kPackGridBlocks, bk::ceil_div(d.RT, 16 / lanes)), (unsigned)count),
               dim3(256), stream, scale, zero, m, d.RT, d.G, (int64_t)d.bytes, (int64_t)d.grid_at, (int64_t)d.unit_at, out);
    return hipGetLastError() == hipSuccess ? BAKRON_SUCCESS : BAKRON_ERR_HIP;
}

// The argument checks that the layer and its gradient share: `in` rows of
// `in_cols` values, `out` rows of `out_cols`.  1: nothing to do, 2: zeros.
static int check_q4(const void* in, int64_t ldin, int64_t in_cols, int64_t tokens, int32_t type, const void* packed,
                    int64_t m, int64_t n, int64_t group_size, const void* out, int64_t ldout, int64_t out_cols,
                    const void* ws, size_t ws_bytes, size_t need)
{
    if (!q4_shape_ok(m, n) || tokens < 0 || tokens > BAKRON_Q4_MAX_TOKENS) return BAKRON_ERR_BAD_SIZE;
    if (!q4_group_ok(group_size) || (type != BAKRON_Q4_BF16 && type != BAKRON_Q4_FP16)) return BAKRON_ERR_BAD_ARG;
    if (ldin < in_cols || ldout < out_cols || ldin >= ((int64_t)1 << 32) || ldout >= ((int64_t)1 << 32))
        return BAKRON_ERR_BAD_ARG;
    if (out_cols == 0 || tokens == 0) return 1;
    if (!out) return BAKRON_ERR_NULL_POINTER;
    if (reinterpret_cast<uintptr_t>(out) & 1) return BAKRON_ERR_BAD_ARG;
    if (in_cols == 0) return 2;
    if (!in || !packed) return BAKRON_ERR_NULL_POINTER;
    if ((reinterpret_cast<uintptr_t>(in) & 1) || reinterpret_cast<uintptr_t>(packed) % bk::kAlign)
        return BAKRON_ERR_BAD_ARG;
    if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % bk::kAlign)) return BAKRON_ERR_WORKSPACE;
    return BAKRON_SUCCESS;
}

size_t bakron_q4_linear_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int64_t group_size)
{
    if (!q4_shape_ok(m, n) || !q4_group_ok(group_size) || tokens <= bk::kQ4Few || tokens > BAKRON_Q4_MAX_TOKENS ||
        m == 0 || n == 0)
        return 0;
    return bk::q4_prompt_workspace_bytes(tokens, m, n, bk::q4_dims(m, n, group_size).gb);
}

int bakron_q4_linear(const void* x, int64_t ldx, int64_t tokens, int32_t type, const void* packed, int64_t m, int64_t n,
                     int64_t group_size, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                     hipStream_t stream)
{
    const int c = check_q4(x, ldx, n, tokens, type, packed, m, n, group_size, y, ldy, m, workspace, workspace_bytes,
                           bakron_q4_linear_workspace_bytes(tokens, m, n, group_size));
    if (c < 0) return c;
    if (c == 1) return BAKRON_SUCCESS;
    if (c == 2) return bk::q4_zero_enqueue(y, ldy, tokens, m, stream) ? BAKRON_ERR_HIP : BAKRON_SUCCESS;
    const bk::Q4Layer w = bk::q4_layer(packed, bk::q4_dims(m, n, group_size));
    if (tokens > bk::kQ4Few)
        return bk::q4_prompt_enqueue(x, ldx, tokens, type == BAKRON_Q4_BF16, w, y, ldy, workspace, stream)
                   ? BAKRON_ERR_HIP
                   : BAKRON_SUCCESS;
    if (type == BAKRON_Q4_BF16) bk::few_enqueue<bk::Bf16>(x, ldx, tokens, w, y, ldy, stream);
    else bk::few_enqueue<bk::Fp16>(x, ldx, tokens, w, y, ldy, stream);
    return hipGetLastError() == hipSuccess ? BAKRON_SUCCESS : BAKRON_ERR_HIP;
}

size_t bakron_q4_linear_grad_workspace_bytes(int64_t tokens, int64_t m, int64_t n, int64_t group_size)
{
    if (!q4_shape_ok(m, n) || !q4_group_ok(group_size) || tokens <= 0 || tokens > BAKRON_Q4_MAX_TOKENS || m == 0 ||
        n == 0)
        return 0;
    return bk::q4_grad_workspace_bytes(tokens, m, n);
}

int bakron_q4_linear_grad(const void* dy, int64_t lddy, int64_t tokens, int32_t type, const void* packed, int64_t m,
                          int64_t n, int64_t group_size, void* dx, int64_t lddx, void* workspace,
                          size_t workspace_bytes, hipStream_t stream)
{
    const int c = check_q4(dy, lddy, m, tokens, type, packed, m, n, group_size, dx, lddx, n, workspace, workspace_bytes,
                           bakron_q4_linear_grad_workspace_bytes(tokens, m, n, group_size));
    if (c < 0) return c;
    if (c == 1) return BAKRON_SUCCESS;
    if (c == 2) return bk::q4_zero_enqueue(dx, lddx, tokens, n, stream) ? BAKRON_ERR_HIP : BAKRON_SUCCESS;
    const bk::Q4Layer w = bk::q4_layer(packed, bk::q4_dims(m, n, group_size));
    return bk::q4_grad_enqueue(dy, lddy, tokens, type == BAKRON_Q4_BF16, w, dx, lddx, workspace, stream)
               ? BAKRON_ERR_HIP
               : BAKRON_SUCCESS;
}

}  // extern "C"
