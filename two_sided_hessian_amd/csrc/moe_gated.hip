// moe_gated.hip -- 8-bit checkpoints, and the experts' inner activation
// act(a) b that keeps its inputs in them for the backward pass (gfx950).
//
// A checkpoint's block is 32 columns of a row, four lanes of 8.  Its step is a
// power of two, so every operation on the way is exact but for the one rounding
// of each code: with m the bits of the block's largest |v| (an integer maximum,
// in which infinities and NaN are larger than any number),
//     s + 127 = ((m + 0x10000) >> 23) - 6
// puts max / 2^s into [63.75, 127.5): the exponent of max less 6, one more where
// the mantissa is from 127.5 / 64 on, which would round to 128.  The code is the
// low byte of v / 2^s + 1.5 * 2^23, one fused operation that rounds to an
// integer, ties to even.
//
// act(v) = v p, p = sigmoid(t(v)), and act'(v) = p + v p (1 - p) t'(v), with
// t(v) = v (SiLU) or 2 sqrt(2/pi) (v + 0.044715 v^3) (GELU, tanh form), whose v is
// held within +-64 there: p is 0 or 1 beyond, and the cube stays finite.
// Exponential and reciprocal are the hardware's (1 unit in the last place of
// float32 each), a few parts in 10^6 at most where p is far below 1: the results
// are rounded to 16 bits.  They hold no numbers below 2^-126: there, beyond t = -87.3, p
// is 0.
//
// HBM bounds all of it, and next the vector instructions (0.65 of a CU's cycles):
// 16384 x 14336, forward with checkpoints 332 us, backward 324, 5.7 and 5.8 TB/s; a
// checkpoint alone, packed 127, unpacked 126 (to float32 198), 5.6 to 6.0 TB/s.
// 96 x 1024 without: 2.6 us, a launch and a round trip.
#include <algorithm>

#include "moe.hpp"

namespace bk {

constexpr int kCkBlock = 32;     // columns of a step
constexpr int kCkNaN = 255;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A checkpoint's rows: `units` 8-column units of codes, units / 4 steps.
struct Ck8 {
    u32x2* codes;
    uint8_t* steps;
};
static Ck8 ck8_of(void* ck, int64_t rows, int64_t cols)
{
    const int64_t blocks = ceil_div(cols, kCkBlock);
    return Ck8{static_cast<u32x2*>(ck), static_cast<uint8_t*>(ck) + align_up((size_t)rows * blocks * kCkBlock)};
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));          // lanes 1 0 3 2
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));       // lanes 2 3 0 1
}

// Codes of a lane's 8 values (four lanes a block), and the block's step byte.
__device__ __forceinline__ u32x2 ck8_codes(const float (&f)[8], uint32_t& step)
{
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    m = quad_max(m);
    step = (uint32_t)max((int)((m + 0x10000u) >> 23) - 6, 1);
    if (m >= 0x7F800000u) step = kCkNaN;
    const float inv = __uint_as_float((254u - min(step, 253u)) << 23);
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(fmaf(f[e], inv, 12582912.f));
    // the low bytes of four values each
    const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                              __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
    const uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[7], b[6], 0x0C0C0400u),
                                              __builtin_amdgcn_perm(b[5], b[4], 0x0C0C0400u), 0x05040100u);
    return step == kCkNaN ? u32x2{0u, 0u} : u32x2{lo, hi};
}

__device__ __forceinline__ void ck8_values(u32x2 c, uint32_t step, float (&f)[8])
{
    const float s = step == kCkNaN ? __uint_as_float(0x7FC00000u) : __uint_as_float(step << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * i + e] = (float)(int8_t)(c[i] >> 8 * e) * s;
}

__device__ __forceinline__ int64_t rows_of(int64_t rows, const int32_t* __restrict__ count)
{
    return count ? min(rows, (int64_t)max(*count, 0)) : rows;
}

__device__ __forceinline__ void ck8_store(const Ck8& ck, int64_t row, int units, int u, const float (&f)[8])
{
    uint32_t step;
    const u32x2 c = ck8_codes(f, step);
    ck.codes[row * units + u] = c;
    if (u % 4 == 0) ck.steps[row * (units / 4) + u / 4] = (uint8_t)step;
}

template <class X>
__global__ __launch_bounds__(256) void k_ck8_pack(const uint16_t* __restrict__ x, int64_t ldx, int64_t rows, int n, int units,
                                                  int log, int chunks, Ck8 ck)
{
    const UnitAt at(log, chunks);
    if (at.u >= units) return;
    for (int64_t r = at.r; r < rows; r += at.by) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (8 * at.u < n) v = load8(x + r * ldx, 8 * at.u, n);
        float f[8];
        up8<X>(v, f);
        ck8_store(ck, r, units, at.u, f);
    }
}

template <class X>
__global__ __launch_bounds__(256) void k_ck8_unpack(Ck8 ck, int64_t rows, int n, int units, int log, int chunks,
                                                    typename RawOf<X>::type* __restrict__ x, int64_t ldx)
{
    const UnitAt at(log, chunks);
    if (8 * at.u >= n) return;
    for (int64_t r = at.r; r < rows; r += at.by) {
        float f[8];
        ck8_values(ck.codes[r * units + at.u], ck.steps[r * (units / 4) + at.u / 4], f);
        typename RawOf<X>::type* row = x + r * ldx;
        if constexpr (sizeof(*row) == 2) {
            store8(row, 8 * at.u, n, down8<X>(f));
        } else {
            typedef u32x4 u32x4_word __attribute__((aligned(4)));
            if (8 * at.u + 8 <= n) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<u32x4_word*>(row + 8 * at.u + 4 * i) =
                        u32x4{X::down(f[4 * i]), X::down(f[4 * i + 1]), X::down(f[4 * i + 2]), X::down(f[4 * i + 3])};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (8 * at.u + e < n) row[8 * at.u + e] = X::down(f[e]);
            }
        }
    }
}

// act(v) = v p, and the slope of t
template <bool GELU>
__device__ __forceinline__ float gate_p(float v, float& dt)
{
    constexpr float kLog2e = 1.44269504088896341f, kC = 1.59576912160573071f /* 2 sqrt(2 / pi) */, kCube = 0.044715f;
    float t = v;
    dt = 1.f;
    if (GELU) {
        const float c = __builtin_amdgcn_fmed3f(v, -64.f, 64.f), c2 = c * c;
        t = kC * c * fmaf(kCube, c2, 1.f);
        dt = fmaf(3.f * kC * kCube, c2, kC);
    }
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * t));
}

template <class X, bool GELU, bool KEEP>
__global__ __launch_bounds__(256) void k_gated_act(const uint16_t* __restrict__ a, int64_t lda, const uint16_t* __restrict__ b,
                                                   int64_t ldb, int64_t rows, int n, int units, int log, int chunks,
                                                   const int32_t* __restrict__ count, uint16_t* __restrict__ h, int64_t ldh,
                                                   Ck8 cka, Ck8 ckb)
{
    const UnitAt at(log, chunks);
    const int c = 8 * at.u;
    if (at.u >= units) return;
    rows = rows_of(rows, count);
    for (int64_t r = at.r; r < rows; r += at.by) {
        u32x4 av = {0u, 0u, 0u, 0u}, bv = av;
        if (c < n) av = load8(a + r * lda, c, n), bv = load8(b + r * ldb, c, n);
        float fa[8], fb[8], v[8];
        up8<X>(av, fa);
        up8<X>(bv, fb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float dt;
            v[e] = fa[e] * gate_p<GELU>(fa[e], dt) * fb[e];
        }
        if (c < n) store8(h + r * ldh, c, n, down8<X>(v));
        if (KEEP) {
            ck8_store(cka, r, units, at.u, fa);
            ck8_store(ckb, r, units, at.u, fb);
        }
    }
}

template <class X, bool GELU>
__global__ __launch_bounds__(256) void k_gated_grad(const uint16_t* __restrict__ dh, int64_t lddh, Ck8 cka, Ck8 ckb,
                                                    int64_t rows, int n, int units, int log, int chunks,
                                                    const int32_t* __restrict__ count, uint16_t* __restrict__ da, int64_t ldda,
                                                    uint16_t* __restrict__ db, int64_t lddb)
{
    const UnitAt at(log, chunks);
    const int c = 8 * at.u;
    if (c >= n) return;
    rows = rows_of(rows, count);
    for (int64_t r = at.r; r < rows; r += at.by) {
        const u32x4 dv = load8(dh + r * lddh, c, n);
        const int64_t u = r * units + at.u, s = r * (units / 4) + at.u / 4;
        const u32x2 ca = cka.codes[u], cb = ckb.codes[u];
        const uint32_t sa = cka.steps[s], sb = ckb.steps[s];
        float d[8], fa[8], fb[8], va[8], vb[8];
        up8<X>(dv, d);
        ck8_values(ca, sa, fa);
        ck8_values(cb, sb, fb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float dt;
            const float p = gate_p<GELU>(fa[e], dt), ap = fa[e] * p;
            va[e] = d[e] * fb[e] * fmaf(ap * (1.f - p), dt, p);
            vb[e] = d[e] * ap;
        }
        store8(da + r * ldda, c, n, down8<X>(va));
        store8(db + r * lddb, c, n, down8<X>(vb));
    }
}

// --------------------------------------------------------------------- host

struct GatedGrid {
    int units;
    UnitGrid at;
};
static GatedGrid gated_grid(int64_t rows, int64_t cols)
{
    const int units = (int)ceil_div(cols, kCkBlock) * 4;
    return {units, unit_grid(rows, units, 2)};
}

static bool gated_size_ok(int64_t rows, int64_t cols)
{
    return rows >= 0 && rows <= BAKRON_MOE_MAX_ROWS && cols >= 0 && cols <= BAKRON_MAX_DIM;
}

template <class X>
static void gated_enqueue(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols, bool gelu,
                          const int32_t* count, void* h, int64_t ldh, void* ck_a, void* ck_b, hipStream_t s)
{
    const GatedGrid g = gated_grid(rows, cols);
    auto* kernel = gelu ? (ck_a ? k_gated_act<X, true, true> : k_gated_act<X, true, false>)
                        : (ck_a ? k_gated_act<X, false, true> : k_gated_act<X, false, false>);
    enqueue(kernel, dim3(g.at.blocks), dim3(256), s, static_cast<const uint16_t*>(a), lda, static_cast<const uint16_t*>(b), ldb, rows,
            (int)cols, g.units, g.at.log, g.at.chunks, count, static_cast<uint16_t*>(h), ldh, ck8_of(ck_a, rows, cols),
            ck8_of(ck_b, rows, cols));
}

template <class X>
static void gated_grad_enqueue(const void* dh, int64_t lddh, const void* ck_a, const void* ck_b, int64_t rows, int64_t cols,
                               bool gelu, const int32_t* count, void* da, int64_t ldda, void* db, int64_t lddb, hipStream_t s)
{
    const GatedGrid g = gated_grid(rows, cols);
    enqueue(gelu ? k_gated_grad<X, true> : k_gated_grad<X, false>, dim3(g.at.blocks), dim3(256), s, static_cast<const uint16_t*>(dh),
            lddh, ck8_of(const_cast<void*>(ck_a), rows, cols), ck8_of(const_cast<void*>(ck_b), rows, cols), rows, (int)cols,
            g.units, g.at.log, g.at.chunks, count, static_cast<uint16_t*>(da), ldda, static_cast<uint16_t*>(db), lddb);
}

template <class X>
static void unpack_enqueue(const void* ck, int64_t rows, int64_t cols, void* x, int64_t ldx, hipStream_t s)
{
    const GatedGrid g = gated_grid(rows, cols);
    enqueue(k_ck8_unpack<X>, dim3(g.at.blocks), dim3(256), s, ck8_of(const_cast<void*>(ck), rows, cols), rows, (int)cols, g.units, g.at.log, g.at.chunks,
            static_cast<typename RawOf<X>::type*>(x), ldx);
}

}  // namespace bk

extern "C" {

size_t bakron_ck8_bytes(int64_t rows, int64_t cols)
{
    if (!bk::gated_size_ok(rows, cols) || rows == 0 || cols == 0) return 0;
    const size_t blocks = (size_t)rows * bk::ceil_div(cols, bk::kCkBlock);
    return bk::align_up(blocks * bk::kCkBlock) + bk::align_up(blocks);
}

int bakron_ck8_pack(const void* x, int64_t ldx, int64_t rows, int32_t type, int64_t cols, void* ck, hipStream_t stream)
{
    if (!bk::gated_size_ok(rows, cols)) return BAKRON_ERR_BAD_SIZE;
    if (!bk::moe_type_ok(type) || !bk::moe_ld_ok(ldx, cols)) return BAKRON_ERR_BAD_ARG;
    if (rows == 0 || cols == 0) return BAKRON_SUCCESS;
    if (!x || !ck) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(x, 2) || !bk::moe_at(ck, bk::kAlign)) return BAKRON_ERR_BAD_ARG;
    const bk::GatedGrid g = bk::gated_grid(rows, cols);
    bk::enqueue(type == BAKRON_Q4_BF16 ? bk::k_ck8_pack<bk::Bf16> : bk::k_ck8_pack<bk::Fp16>, dim3(g.at.blocks), dim3(256), stream,
                static_cast<const uint16_t*>(x), ldx, rows, (int)cols, g.units, g.at.log, g.at.chunks, bk::ck8_of(ck, rows, cols));
    return bk::moe_done();
}

int bakron_ck8_unpack(const void* ck, int64_t rows, int64_t cols, int32_t type, void* x, int64_t ldx, hipStream_t stream)
{
    if (!bk::gated_size_ok(rows, cols)) return BAKRON_ERR_BAD_SIZE;
    if ((!bk::moe_type_ok(type) && type != BAKRON_MOE_F32) || !bk::moe_ld_ok(ldx, cols)) return BAKRON_ERR_BAD_ARG;
    if (rows == 0 || cols == 0) return BAKRON_SUCCESS;
    if (!x || !ck) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(x, type == BAKRON_MOE_F32 ? 4 : 2) || !bk::moe_at(ck, bk::kAlign)) return BAKRON_ERR_BAD_ARG;
    auto* run = type == BAKRON_MOE_F32 ? bk::unpack_enqueue<bk::Fp32>
              : type == BAKRON_Q4_BF16 ? bk::unpack_enqueue<bk::Bf16> : bk::unpack_enqueue<bk::Fp16>;
    run(ck, rows, cols, x, ldx, stream);
    return bk::moe_done();
}

int bakron_gated_act(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int32_t type, int64_t cols,
                     int32_t act, const int32_t* count, void* h, int64_t ldh, void* ck_a, void* ck_b,
                     hipStream_t stream)
{
    if (!bk::gated_size_ok(rows, cols)) return BAKRON_ERR_BAD_SIZE;
    if (!bk::moe_type_ok(type) || (act != BAKRON_MOE_SILU && act != BAKRON_MOE_GELU) || !bk::moe_ld_ok(lda, cols) ||
        !bk::moe_ld_ok(ldb, cols) || !bk::moe_ld_ok(ldh, cols) || !ck_a != !ck_b)
        return BAKRON_ERR_BAD_ARG;
    if (rows == 0 || cols == 0) return BAKRON_SUCCESS;
    if (!a || !b || !h) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(a, 2) || !bk::moe_at(b, 2) || !bk::moe_at(h, 2) || !bk::moe_at(count, 4) ||
        !bk::moe_at(ck_a, bk::kAlign) || !bk::moe_at(ck_b, bk::kAlign))
        return BAKRON_ERR_BAD_ARG;
    auto* run = type == BAKRON_Q4_BF16 ? bk::gated_enqueue<bk::Bf16> : bk::gated_enqueue<bk::Fp16>;
    run(a, lda, b, ldb, rows, cols, act == BAKRON_MOE_GELU, count, h, ldh, ck_a, ck_b, stream);
    return bk::moe_done();
}

int bakron_gated_act_grad(const void* dh, int64_t lddh, const void* ck_a, const void* ck_b, int64_t rows, int32_t type,
                          int64_t cols, int32_t act, const int32_t* count, void* da, int64_t ldda, void* db,
                          int64_t lddb, hipStream_t stream)
{
    if (!bk::gated_size_ok(rows, cols)) return BAKRON_ERR_BAD_SIZE;
    if (!bk::moe_type_ok(type) || (act != BAKRON_MOE_SILU && act != BAKRON_MOE_GELU) || !bk::moe_ld_ok(lddh, cols) ||
        !bk::moe_ld_ok(ldda, cols) || !bk::moe_ld_ok(lddb, cols))
        return BAKRON_ERR_BAD_ARG;
    if (rows == 0 || cols == 0) return BAKRON_SUCCESS;
    if (!dh || !ck_a || !ck_b || !da || !db) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(dh, 2) || !bk::moe_at(da, 2) || !bk::moe_at(db, 2) || !bk::moe_at(count, 4) ||
        !bk::moe_at(ck_a, bk::kAlign) || !bk::moe_at(ck_b, bk::kAlign))
        return BAKRON_ERR_BAD_ARG;
    auto* run = type == BAKRON_Q4_BF16 ? bk::gated_grad_enqueue<bk::Bf16> : bk::gated_grad_enqueue<bk::Fp16>;
    run(dh, lddh, ck_a, ck_b, rows, cols, act == BAKRON_MOE_GELU, count, da, ldda, db, lddb, stream);
    return bk::moe_done();
}

}  // extern "C"
