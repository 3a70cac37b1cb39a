// moe.hpp -- what the calls of the expert layer for many tokens share (gfx950).
#pragma once

#include "../../include/bakron_moe.h"
#include "q4_few.hpp"

namespace bk {

// A third activation type beside Bf16 and Fp16 (q4.hpp), for logits and
// unpacked checkpoints: raw 32-bit storage.
struct Fp32 {
    static __device__ __forceinline__ float up(uint32_t v) { return __uint_as_float(v); }
    static __device__ __forceinline__ uint32_t down(float v) { return __float_as_uint(v); }
};
template <class X>
struct RawOf {
    typedef uint16_t type;
};
template <>
struct RawOf<Fp32> {
    typedef uint32_t type;
};

// A row of 16 lanes is what a token's choice is made in: value v combined with
// that of the lane N places round the row (DPP, no LDS).
template <int N>
__device__ __forceinline__ uint32_t row_turn(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, row_turn<8>(v));
    v = max(v, row_turn<4>(v));
    v = max(v, row_turn<2>(v));
    return max(v, row_turn<1>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v)
{
    v = min(v, row_turn<8>(v));
    v = min(v, row_turn<4>(v));
    v = min(v, row_turn<2>(v));
    return min(v, row_turn<1>(v));
}
// (every lane adds the same pairs, so all get the same bits)
__device__ __forceinline__ float row_sum(float v)
{
    v += __uint_as_float(row_turn<8>(__float_as_uint(v)));
    v += __uint_as_float(row_turn<4>(__float_as_uint(v)));
    v += __uint_as_float(row_turn<2>(__float_as_uint(v)));
    return v + __uint_as_float(row_turn<1>(__float_as_uint(v)));
}

// Eight columns c .. c + 7 of a row of n, zeros beyond n.  No access beyond n.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ row, int c, int n)
{
    if (c + 8 <= n) return *reinterpret_cast<const u32x4_any*>(row + c);
    return few_x_cut(row, c, n);
}
// and their store, columns beyond n left alone
__device__ __forceinline__ void store8(uint16_t* __restrict__ row, int c, int n, u32x4 v)
{
    if (c + 8 <= n) {
        *reinterpret_cast<u32x4_any*>(row + c) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < n) row[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}
template <class X>
__device__ __forceinline__ void up8(u32x4 v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = X::up((uint16_t)v[i]), f[2 * i + 1] = X::up((uint16_t)(v[i] >> 16));
}
template <class X>
__device__ __forceinline__ u32x4 down8(const float (&f)[8])
{
    return u32x4{X::down2(f[0], f[1]), X::down2(f[2], f[3]), X::down2(f[4], f[5]), X::down2(f[6], f[7])};
}

// Rows of 8-column units over threads: 2^log lanes a run of a row's units, a row's
// runs (`chunks` of them) in workgroups beside each other, so that what is in flight
// lies together in memory.
struct UnitAt {
    int64_t r, by;   // the first row and the step to the next
    int u;
    __device__ __forceinline__ UnitAt(int log, int chunks)
    {
        const unsigned chunk = blockIdx.x % chunks, group = blockIdx.x / chunks;
        r = ((int64_t)group << (8 - log)) + (threadIdx.x >> log);
        by = (int64_t)(gridDim.x / chunks) << (8 - log);
        u = (int)(threadIdx.x & ((1u << log) - 1)) + (int)(chunk << log);
    }
};
constexpr int64_t kUnitBlocks = 1 << 22;   // of a launch; more rows are taken in turn
struct UnitGrid {
    int log, chunks;
    unsigned blocks;   // of 256 threads, a multiple of chunks
};
// As many lanes a run as leave one in 16 idle at most: 256 where they fit (16384 x
// 14336, forward with checkpoints and backward: 322 + 319 us with 256 lanes, 334 + 314
// with 64; with a workgroup's four rows below each other and runs of rows as the faster
// index 407 + 400).
inline UnitGrid unit_grid(int64_t rows, int64_t units, int least)
{
    UnitGrid g;
    g.log = least;
    while (g.log < 6 && (1 << g.log) < units) ++g.log;
    for (int log = 8; log > 6; --log)
        if (g.log == 6 && (ceil_div(units, 1 << log) << log) - units <= units / 16) g.log = log;
    g.chunks = (int)ceil_div(units, 1 << g.log);
    g.blocks = (unsigned)(std::min(kUnitBlocks / g.chunks, ceil_div(rows, 256 >> g.log)) * g.chunks);
    return g;
}

// Layer e of a stack
__device__ __forceinline__ Q4Layer expert_layer(Q4Layer w, int e, int64_t layer_bytes)
{
    w.codes = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(w.codes) + e * layer_bytes);
    w.grid = reinterpret_cast<const f32x2*>(reinterpret_cast<const char*>(w.grid) + e * layer_bytes);
    w.unit = reinterpret_cast<const float*>(reinterpret_cast<const char*>(w.unit) + e * layer_bytes);
    return w;
}

// Host-side checks
inline bool moe_type_ok(int32_t type) { return type == BAKRON_Q4_BF16 || type == BAKRON_Q4_FP16; }
inline bool moe_ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld < ((int64_t)1 << 32); }
inline bool moe_at(const void* p, size_t align) { return reinterpret_cast<uintptr_t>(p) % align == 0; }
inline int moe_done() { return hipGetLastError() == hipSuccess ? BAKRON_SUCCESS : BAKRON_ERR_HIP; }

}  // namespace bk
