// q4.hpp -- packed 4-bit layers: the layout and the device pieces that the
// q4 kernels share (gfx950).
//
// Layout of one packed layer (m x n, RT = ceil(m / 16) row tiles, KB =
// ceil(n / 128) column blocks, G grids per row):
//   codes: RT x KB blocks of 1 KB, each 16 rows x 128 columns, as 64 units of
//          16 bytes; unit u = 16 q + r belongs to row r of the tile and holds
//          four dwords d of 8 columns each,
//              column = 64 (d >> 1) + 16 q + 8 (d & 1) + e,  e = 0 .. 7,
//          so lane u of a wave loads a unit, a wave instruction one block, and
//          dword pair d = 0, 1 (2, 3) of all units is the block's first (last)
//          64 columns: a group of 64 columns never shares an MFMA with the
//          next.  A 16 x 16 x 32 MFMA takes dword d of lane (q, r) as its
//          fragment; a 32 x 32 x 16 one takes two tiles and units q, q + 2.
//   dword: column pair p (e = 2p, 2p + 1) has its codes in bits 4p .. 4p + 3
//          and 16 + 4p .. 16 + 4p + 3, and the whole is rotated left by 3,
//          which puts pair 0 where a bfloat16's mantissa wants it.
//   grids: RT x G x 16 pairs (scale, zero), at the next 256 bytes after the
//          codes; rows beyond m have scale = zero = 0.
//   units: one float per grid, the power of two at or above the largest weight
//          |s (c - z)| of its columns, at the next 256 bytes after the grids:
//          kernels that round weights to 16 bits divide by it first, so that
//          no columns' weights leave float16's normal range as a whole.
// Codes of rows beyond m and columns beyond n are 0; their products are kept
// out by zeros of the activations.
//
// A code becomes the exact number u = 16 + c in one operation per pair: in
// bfloat16, 16 has the bits 0x4180 and four mantissa bits of weight 1 at bits
// 3 .. 6; in float16, 0x4C00 and bits 6 .. 9.  The products of u with
// activations are exact in the MFMA's float32, and
//     sum_j s (c_j - z) x_j = s ( sum_j u_j x_j - (16 + z) sum_j x_j )
// over a group (or a piece of one) applies step and zero point once, in
// float32.  The offset of 16 costs about 16 / 5 of the sum's float32 rounding,
// 2 bits of 24, where x has no mean.  With one, sum_j u_j x_j grows with the
// columns and the result with their root: kernels take zero points off after
// 128 columns (few tokens) or at most 1024 (many), not at the row's end.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm.hpp"
#include "internal.hpp"

namespace bk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kQ4Rows = 16;       // rows of a code block
constexpr int kQ4Cols = 128;      // columns of a code block
constexpr float kQ4Offset = 16.f; // u = c + 16

struct Q4Dims {
    int64_t m, n;
    int RT, KB, G;
    int gb;                       // 64-column halves per grid (>= 2 KB when one grid per row)
    size_t grid_at, unit_at;      // byte offsets of the grids and the units
    size_t bytes;                 // bytes of one layer
};

inline Q4Dims q4_dims(int64_t m, int64_t n, int64_t group_size)
{
    Q4Dims d;
    d.m = m;
    d.n = n;
    d.RT = (int)ceil_div(m, kQ4Rows);
    d.KB = (int)ceil_div(n, kQ4Cols);
    d.G = group_size ? (int)ceil_div(n, group_size) : 1;
    if (d.G < 1) d.G = 1;
    d.gb = group_size ? (int)(group_size / 64 < (1 << 20) ? group_size / 64 : (1 << 20)) : (1 << 20);
    d.grid_at = align_up((size_t)d.RT * d.KB * 1024);
    d.unit_at = align_up(d.grid_at + (size_t)d.RT * d.G * kQ4Rows * 8);
    d.bytes = d.unit_at + align_up((size_t)d.G * 4);
    return d;
}

// One packed layer as the kernels take it.
struct Q4Layer {
    const u32x4* codes;
    const f32x2* grid;
    const float* unit;
    int m, n, RT, KB, G, gb;
    uint32_t gm;                  // ceil(2^21 / gb), for group_of
};

// The group of 64-column half h (< 1024): h / gb as one multiplication, exact
// since h (gm gb - 2^21) < 2^21.  An integer division, ahead of the loads that
// wait for it, costs 0.2 us of a few-token kernel's step.
constexpr int kQ4MaxHalves = BAKRON_MAX_DIM / 64;
static_assert(kQ4MaxHalves <= 1024, "group_of's range");
__device__ __forceinline__ int group_of(uint32_t h, uint32_t gm, int G) { return (int)min(h * gm >> 21, (uint32_t)G - 1); }

inline Q4Layer q4_layer(const void* packed, const Q4Dims& d)
{
    const char* p = static_cast<const char*>(packed);
    return Q4Layer{reinterpret_cast<const u32x4*>(p), reinterpret_cast<const f32x2*>(p + d.grid_at),
                   reinterpret_cast<const float*>(p + d.unit_at), (int)d.m, (int)d.n, d.RT, d.KB, d.G, d.gb,
                   (uint32_t)ceil_div(1 << 21, std::min(d.gb, kQ4MaxHalves))};
}

// (w & mask) | base.  The constants pass through empty asm statements so that
// the compiler keeps them in registers, the mask in a vector one, and takes
// its one instruction for both (which reads no literal and at most one scalar
// register) instead of two with literals.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t base)
{
    asm("" : "+v"(mask));
    asm("" : "+s"(base));
    return (w & mask) | base;
}

// Rows may start at any 2-byte address: global loads and stores need no
// alignment here.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The activation types: raw 16-bit storage, MFMA forms and roundings.
struct Bf16 {
    typedef bf16x8 vec;
    static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t down(float v)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)v);   // to nearest, ties to even
    }
    // two values, a in the low half
    static __device__ __forceinline__ uint32_t down2(float a, float b)
    {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        const v2 v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ f32x4 mfma16(vec a, vec b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(vec a, vec b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // u of the 8 codes of a dword
    static __device__ __forceinline__ vec codes(uint32_t w)
    {
        u32x4 v;
        v.x = and_or(w, 0x00780078u, 0x41804180u);
        v.y = and_or(__builtin_rotateright32(w, 4), 0x00780078u, 0x41804180u);
        v.z = and_or(__builtin_rotateright32(w, 8), 0x00780078u, 0x41804180u);
        v.w = and_or(__builtin_rotateright32(w, 12), 0x00780078u, 0x41804180u);
        return __builtin_bit_cast(vec, v);
    }
    static constexpr uint16_t kOne = 0x3F80;
    static constexpr float kUnit = 1.f;        // of a packed layer's units, what weights are rounded in
};

struct Fp16 {
    typedef f16x8 vec;
    static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
    static __device__ __forceinline__ uint32_t down2(float a, float b)
    {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        const v2 v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ f32x4 mfma16(vec a, vec b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(vec a, vec b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vec codes(uint32_t w)
    {
        u32x4 v;
        v.x = and_or(__builtin_rotateright32(w, 29), 0x03C003C0u, 0x4C004C00u);
        v.y = and_or(__builtin_rotateright32(w, 1), 0x03C003C0u, 0x4C004C00u);
        v.z = and_or(__builtin_rotateright32(w, 5), 0x03C003C0u, 0x4C004C00u);
        v.w = and_or(__builtin_rotateright32(w, 9), 0x03C003C0u, 0x4C004C00u);
        return __builtin_bit_cast(vec, v);
    }
    static constexpr uint16_t kOne = 0x3C00;
    static constexpr float kUnit = 0x1p-15f;   // (2^15 is the largest power of two, 2^-14 the smallest normal)
};

template <class X>
__device__ __forceinline__ typename X::vec q4_ones()
{
    const uint32_t o = (uint32_t)X::kOne * 0x10001u;
    const u32x4 v = {o, o, o, o};
    return __builtin_bit_cast(typename X::vec, v);
}

// Direct loads to LDS through a buffer descriptor: per-lane byte offsets
// `lane_at` that never change, a scalar one that does, no vector arithmetic
// per load.  Lane l's 16 (4) bytes land at s + 16 l (4 l).
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc buffer_of(const void* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
__device__ __forceinline__ void load_lds16(Rsrc r, uint32_t lane_at, uint32_t at, char* s)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)s, 16, lane_at, at, 0, 0);
}
__device__ __forceinline__ void load_lds4(Rsrc r, uint32_t lane_at, uint32_t at, char* s)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)s, 4, lane_at, at, 0, 0);
}

// Many tokens (q4_prompt.hip)
constexpr int64_t kQ4Few = 64;   // up to so many tokens the few-token kernel runs
size_t q4_prompt_workspace_bytes(int64_t T, int64_t m, int64_t n, int gb);
int q4_prompt_enqueue(const void* x, int64_t ldx, int64_t T, bool bf16, const Q4Layer& w, void* y, int64_t ldy, void* ws,
                      hipStream_t s);

// Input gradient (q4_grad.hip)
size_t q4_grad_workspace_bytes(int64_t T, int64_t m, int64_t n);
int q4_grad_enqueue(const void* dy, int64_t lddy, int64_t T, bool bf16, const Q4Layer& w, void* dx, int64_t lddx, void* ws,
                    hipStream_t s);

}  // namespace bk
