// q4_grad.hip -- dx = dy W on 4-bit codes, the input gradient of the linear
// layer (gfx950).
//
//     dx_tj = sum_i dy_ti s_ig (c_ij - z_ig),   g the group of column j.
//
// The sum runs over the rows of W, and step and zero point change with the
// row: they cannot be taken out of it as in the forward product.  So a
// weight is formed in float32, divided by the layer's unit (a power of two,
// q4.hpp) and rounded once to dy's 16-bit type, the product runs on 16-bit
// MFMAs with float32 accumulators, and the unit comes back at the store.
// The rounding is half a unit in the last place of each weight, as a layer
// kept in that type would have; independent from weight to weight, it adds
// to a result about what the result's own rounding does.
//
// k_q4_grad: a workgroup of eight waves computes 64 TA tokens x 256 columns;
// a wave owns 32 TA tokens x 64 columns as TA x 2 MFMA tiles of 32 x 32.  dy
// goes through LDS in chunks of 64 rows of W by direct loads.  Of each
// chunk's 64 x 256 weights a thread expands 4 rows x 8 columns (four dwords of
// codes, loaded two chunks ahead) and writes them to LDS transposed, four
// rows of a column side by side as the MFMA takes them, one chunk ahead of
// the products that read them, so one barrier per chunk orders everything.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4_tile.hpp"

namespace bk {

template <int TA>
struct Grad {
    static constexpr int BT = 64 * TA;              // tokens of a workgroup
    static constexpr int BJ = 256;                  // columns of a workgroup
    static constexpr int XBUF = BT * 128;           // bytes of a 64-row chunk of dy
    static constexpr int PITCH = 144;               // bytes of a column's 64 rows in LDS: 9 x 16, spreads the banks
    static constexpr int WBUF = BJ * PITCH;
    static constexpr int AHEAD = TA == 4 ? 1 : 2;   // chunks of dy in flight (a chunk of TA = 4 outlasts a load)
    static constexpr int NX = AHEAD + 1;
    static constexpr int XLOADS = BT / 64;
    static constexpr int WEIGHTS = NX * XBUF, LDS = WEIGHTS + 2 * WBUF;
};

// Eight bytes to LDS byte address at + OFFSET.  Written out because the
// compiler would have every direct load in flight land before a store to LDS,
// whose target here is never theirs; tile_wait orders it before the barrier.
template <int OFFSET>
__device__ __forceinline__ void write64(uint32_t at, uint32_t lo, uint32_t hi)
{
    const uint64_t v = (uint64_t)hi << 32 | lo;
    asm volatile("ds_write_b64 %0, %1 offset:%2" ::"v"(at), "v"(v), "n"(OFFSET));
}

template <class X, int TA>
__global__ __launch_bounds__(512) void k_q4_grad(const uint16_t* __restrict__ dy, int64_t lddy, int T, Q4Layer w,
                                                 uint16_t* __restrict__ dx, int64_t lddx, int nt, int nj)
{
    typedef Grad<TA> P;
    typedef typename X::vec vec;
    __shared__ __align__(16) char lds[P::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, ml = lane & 31;
    const int wt = wave >> 2, wj = wave & 3;
    int bt, bj;
    tile_of(nt, nj, bt, bj);
    const int t0 = bt * P::BT, j0 = bj * P::BJ;
    const int nchunk = (w.m + 63) / 64;
    const float unit = *w.unit > 0.f ? *w.unit : 1.f;
    const float down = 1.f / unit;

    // staging of dy
    const Rsrc x = buffer_of(dy + (int64_t)t0 * lddy, 0x7FFFFFFFu);
    uint32_t x_at[P::XLOADS];
#pragma unroll
    for (int i = 0; i < P::XLOADS; ++i) {
        const int r = 8 * (wave * P::XLOADS + i) + (lane >> 3);
        x_at[i] = (uint32_t)(min(r, T - 1 - t0) * lddy * 2) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
    auto stage = [&](int c, int bx) {
#pragma unroll
        for (int i = 0; i < P::XLOADS; ++i)
            load_lds16(x, x_at[i], 128 * min(c, nchunk - 1), lds + bx * P::XBUF + (wave * P::XLOADS + i) * 1024);
    };

    // expansion: rows 4 a .. 4 a + 3 of the chunk, the eight columns of dword d
    // of unit column q of block kb
    const int a4 = lane & 15, d = lane >> 4, q = wave & 3;
    const int kb = min(2 * bj + (wave >> 2), w.KB - 1);
    const int g = min((2 * kb + (d >> 1)) / w.gb, w.G - 1);
    const int col = 128 * (wave >> 2) + 64 * (d >> 1) + 16 * q + 8 * (d & 1);
    const uint32_t* code_at = reinterpret_cast<const uint32_t*>(w.codes + (int64_t)kb * 64 + 16 * q) + 16 * (a4 & 3) + d;
    const f32x4* grid_at = reinterpret_cast<const f32x4*>(w.grid + (int64_t)g * 16 + 4 * (a4 & 3));
    const uint32_t w_at = (uint32_t)(uintptr_t)(lds_ptr)lds + P::WEIGHTS + col * P::PITCH + 8 * a4;
    struct Raw {
        uint32_t c[4];
        f32x4 g[2];
    };
    auto fetch = [&](int c, Raw& v) {
        const int64_t rt = min(4 * min(c, nchunk - 1) + (a4 >> 2), w.RT - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.c[i] = code_at[rt * w.KB * 256 + 4 * i];
        v.g[0] = grid_at[rt * w.G * 8];
        v.g[1] = grid_at[rt * w.G * 8 + 1];
    };
    auto expand = [&](const Raw& v, int buf) {
        float f[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = v.g[i >> 1][2 * (i & 1)] * down, b = -s * v.g[i >> 1][2 * (i & 1) + 1];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                // two codes in bytes 0 and 2, which convert in one instruction
                // each (the empty statement hides that they are nibbles)
                uint32_t two = __builtin_rotateright32(v.c[i], 3 + 4 * p) & 0x000F000Fu;
                asm("" : "+v"(two));
                f[i][2 * p] = fmaf(s, (float)(two & 0xFFu), b);
                f[i][2 * p + 1] = fmaf(s, (float)(two >> 16 & 0xFFu), b);
            }
        }
        const uint32_t s = w_at + buf * P::WBUF;
        write64<0 * P::PITCH>(s, X::down2(f[0][0], f[1][0]), X::down2(f[2][0], f[3][0]));
        write64<1 * P::PITCH>(s, X::down2(f[0][1], f[1][1]), X::down2(f[2][1], f[3][1]));
        write64<2 * P::PITCH>(s, X::down2(f[0][2], f[1][2]), X::down2(f[2][2], f[3][2]));
        write64<3 * P::PITCH>(s, X::down2(f[0][3], f[1][3]), X::down2(f[2][3], f[3][3]));
        write64<4 * P::PITCH>(s, X::down2(f[0][4], f[1][4]), X::down2(f[2][4], f[3][4]));
        write64<5 * P::PITCH>(s, X::down2(f[0][5], f[1][5]), X::down2(f[2][5], f[3][5]));
        write64<6 * P::PITCH>(s, X::down2(f[0][6], f[1][6]), X::down2(f[2][6], f[3][6]));
        write64<7 * P::PITCH>(s, X::down2(f[0][7], f[1][7]), X::down2(f[2][7], f[3][7]));
    };

    f32x16 acc[TA][2];
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

    Raw raw;
    fetch(0, raw);
#pragma unroll
    for (int c = 0; c < P::AHEAD; ++c) stage(c, c);
    expand(raw, 0);
    fetch(1, raw);
    uint32_t x_lane[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) x_lane[v] = 128 * (32 * wt * TA + ml) + 16 * ((2 * v + h) ^ ((ml >> 1) & 7));
    const uint32_t b_lane = P::WEIGHTS + (64 * wj + ml) * P::PITCH + 16 * h;
    int bx = 0, px = P::AHEAD % P::NX;
    for (int c = 0; c < nchunk; ++c) {
        // chunk c of dy and the weights of chunk c are in LDS for every wave,
        // and every wave is done with chunk c - 1
        tile_wait<(P::AHEAD - 1) * P::XLOADS>();
        Raw now = raw;
        fetch(c + 2, raw);
        stage(c + P::AHEAD, px);
        px = px + 1 == P::NX ? 0 : px + 1;
        const char* xs = lds + bx * P::XBUF;
        const char* ws = lds + b_lane + (c & 1) * P::WBUF;
        expand(now, (c + 1) & 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            vec wf[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) wf[b] = *reinterpret_cast<const vec*>(ws + 32 * v + 32 * b * P::PITCH);
#pragma unroll
            for (int a = 0; a < TA; ++a) {
                const vec xf = *reinterpret_cast<const vec*>(xs + x_lane[v] + 4096 * a);
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[a][b] = X::mfma32(xf, wf[b], acc[a][b]);
            }
        }
        bx = bx + 1 == P::NX ? 0 : bx + 1;
    }
    wait_direct_loads();
    __syncthreads();
    tile_store<X, TA>(acc, unit, lds, t0 + 32 * wt * TA, T, j0 + wj * 64, w.n, dx, lddx);
}

// --------------------------------------------------------------------- host

size_t q4_grad_workspace_bytes(int64_t T, int64_t m) { return align_up((size_t)T * ceil_div(m, 64) * 64 * 2); }

template <class X, int TA>
static void grad_launch(const uint16_t* dy, int64_t lddy, int64_t T, const Q4Layer& w, uint16_t* dx, int64_t lddx,
                        hipStream_t s)
{
    typedef Grad<TA> P;
    const int nt = (int)ceil_div(T, P::BT), nj = (int)ceil_div(w.n, P::BJ);
    launch(nullptr, KK_Q4_GRAD, 2.0 * T * w.m * w.n, 0.0, k_q4_grad<X, TA>, dim3((unsigned)(nt * nj)), dim3(512), s, dy,
           lddy, (int)T, w, dx, lddx, nt, nj);
}

template <class X>
static int grad_run(const void* dy, int64_t lddy, int64_t T, const Q4Layer& w, void* dx, int64_t lddx, void* ws,
                    hipStream_t s)
{
    const uint16_t* yp = static_cast<const uint16_t*>(dy);
    uint16_t* xp = static_cast<uint16_t*>(dx);
    if (w.m % 64 || lddy % 8 || lddy > (1 << 21) || !aligned16(dy)) {
        const int64_t ldc = ceil_div(w.m, 64) * 64;
        copy_enqueue<X>(yp, lddy, T, w.m, static_cast<uint16_t*>(ws), ldc, s);
        yp = static_cast<const uint16_t*>(ws);
        lddy = ldc;
    }
    const int64_t nj = ceil_div(w.n, 256);
    if (ceil_div(T, 256) * nj >= 256) grad_launch<X, 4>(yp, lddy, T, w, xp, lddx, s);
    else if (ceil_div(T, 128) * nj >= 128) grad_launch<X, 2>(yp, lddy, T, w, xp, lddx, s);
    else grad_launch<X, 1>(yp, lddy, T, w, xp, lddx, s);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int q4_grad_enqueue(const void* dy, int64_t lddy, int64_t T, bool bf16, const Q4Layer& w, void* dx, int64_t lddx, void* ws,
                    hipStream_t s)
{
    return bf16 ? grad_run<Bf16>(dy, lddy, T, w, dx, lddx, ws, s) : grad_run<Fp16>(dy, lddy, T, w, dx, lddx, ws, s);
}

}  // namespace bk
