// q4_grad_few.hpp -- dx = dy W for a few rows of dy on packed codes (gfx950).
//
//     dx_tj = sum_i dy_ti s_ig (c_ij - z_ig) = sum_i a_ti u_ij - sum_i a_ti (16 + z_ig),
//     a_ti = dy_ti s_ig,   u = 16 + c,   g the group of column j.
//
// With few rows of dy the codes are what is read, and a weight formed for each code
// would take most of the time: the step goes to dy's side instead, once per row of dy
// and group, and the codes enter the MFMAs as the exact numbers u.  a is rounded to 16
// bits, which two bfloat16 terms hold exactly, and both sums are of that number: what the
// rounding leaves (2^-16 of a at most) is weighted by c - z then.  With a itself in the
// second sum it is weighted by 16 + c, which rows of W that are alike do not average out
// (14336 of them: 0.77 of a float16 result's rounding).  The second sum, one number per row of dy and
// group, is float32; it comes off after at most 256 rows of W of a wave, since the first
// one grows with the mean of a where the result does not.
//
// The sum runs over W's rows, and a packed dword holds eight columns of one row.  A lane
// takes the dwords of eight rows at one place (columns 8 n ..): joined two rows at a
// time, even and odd columns apart (4 operations), each is again a dword that expands
// in 7 operations, into pairs of rows now: 72 operations make the operands of eight
// MFMAs, one per column of the eight, for 64 codes a lane.
//
// Codes and grids go through LDS by direct loads, two steps of 32 rows ahead, in an order
// in which the eight dwords of a lane are 256 bytes apart and the 64 lanes' lie in
// different banks.  The LDS is a wave's own: no barrier is involved.
//
// Vector instructions bound it (0.82 of the busy cycles), those that expand codes for the
// fewest rows and those that split a for more; HBM is next.  Groups of 128, 2 of 8 experts
// of 14336 x 4096: 16 tokens 53 us while at most seven experts have rows (4.4 TB/s of codes
// and grids, partly from the Infinity Cache), 75 - 83 where all eight have (3.2 - 3.5); 64 tokens
// 82 - 88 with 16 rows each, 109 with 4 to 30.  A weight formed for every code, as with many
// rows, took 117 us of 16 tokens.
#pragma once

#include "moe.hpp"

namespace bk {

constexpr int kGradFewStep = 2048 + 512;             // LDS of a step: codes of 32 rows x 128 columns, grids of two halves
constexpr int kGradFewStage = 2 * kGradFewStep;      // and of a wave
constexpr int kGradFewPitch = 132;                   // floats of a row of dx in the joining sums
constexpr int kGradFewJoin = 16 * kGradFewPitch * 4;
constexpr int kGradFewTake = 8;                      // steps after which the second sum comes off

typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int LEFT>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory");
}

// What two bfloat16 terms hold of a value: its first 16 bits, rounded to nearest.
__device__ __forceinline__ uint32_t two_terms(float v) { return (__float_as_uint(v) + 0x80u) & 0xFFFFFF00u; }

// 16 SETS rows of dy, the 128 columns of block kb of W.  HALF: the block's halves have
// grids of their own.  acc[.][.][e]: columns 64 (d >> 1) + 16 q + 8 (d & 1) + e, q = lane / 4
// % 4, d = lane % 4, rows 4 (lane / 16) + r of dy.
template <class X, int SETS, bool HALF>
struct GradFew {
    static constexpr int NG = HALF ? 2 : 1;
    static constexpr int LOADS = 2 + NG + SETS;      // of a step
    f32x4 acc[SETS][NG][8];
    float off[SETS][NG];                             // the lane's part of the second sum
    const uint16_t* xr[SETS];                        // the lane's row of dy
    const char *codes, *grid[NG];                    // block kb, and its groups, of row tile 0
    uint32_t code_at, grid_at, code_step, grid_step; // the lane's part of a load; bytes of a row tile
    uint32_t code_lane, grid_lane;                   // and of the reads of LDS
    int m, RT;
    char* lds;

    __device__ __forceinline__ GradFew(const Q4Layer& w, int kb, const uint16_t* const (&rows)[SETS], char* wave_lds)
        : code_step(w.KB * 1024u), grid_step(w.G * 128u), m(w.m), RT(w.RT), lds(wave_lds)
    {
        const uint32_t lane = threadIdx.x & 63, kq = lane >> 4;
        codes = reinterpret_cast<const char*>(w.codes) + (int64_t)kb * 1024;
#pragma unroll
        for (int h = 0; h < NG; ++h)
            grid[h] = reinterpret_cast<const char*>(w.grid) + 128 * group_of(2 * kb + h, w.gm, w.G);
#pragma unroll
        for (int s = 0; s < SETS; ++s) {
            xr[s] = rows[s] + 8 * kq;
#pragma unroll
            for (int h = 0; h < NG; ++h) {
                off[s][h] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[s][h][e] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
        // slot 16 i + q + 4 half + 8 t of a step's codes is the unit of row 16 t + 8 half + i
        code_at = (lane >> 3 & 1) * code_step + 16 * (16 * (lane & 3) + 8 * (lane >> 2 & 1) + (lane >> 4));
        grid_at = (lane >> 5) * grid_step + 4 * (lane & 31);
        code_lane = 16 * ((lane >> 2 & 3) + 4 * kq) + 4 * (lane & 3);   // (kq = half + 2 t)
        grid_lane = 2048 + 64 * kq;
    }
    // step s: rows 32 s .. 32 s + 31, that is row tiles 2 s and 2 s + 1 (where there is none,
    // 2 s again: dy is zero there)
    __device__ __forceinline__ void stage(int s, int buf) const
    {
        char* to = lds + buf * kGradFewStep;
        const bool one = 2 * s + 1 >= RT;
        const uint32_t lane = threadIdx.x & 63;
        const Rsrc c = buffer_of(codes + 2ll * s * code_step, 0x7FFFFFFFu);
        const uint32_t ca = one && (lane & 8) ? code_at - code_step : code_at, ga = one && lane >= 32 ? grid_at - grid_step : grid_at;
        load_lds16(c, ca, 0, to);
        load_lds16(c, ca, 64, to + 1024);
#pragma unroll
        for (int h = 0; h < NG; ++h)
            load_lds4(buffer_of(grid[h] + 2ll * s * grid_step, 0x7FFFFFFFu), ga, 0, to + 2048 + 256 * h);
    }
    __device__ __forceinline__ void load(int s, u32x4 (&x)[SETS]) const
    {
#pragma unroll
        for (int t = 0; t < SETS; ++t) x[t] = *reinterpret_cast<const u32x4_any*>(xr[t] + 32 * s);
    }
    __device__ __forceinline__ void load_cut(int s, u32x4 (&x)[SETS]) const
    {
        const int kq = threadIdx.x >> 4 & 3;
#pragma unroll
        for (int t = 0; t < SETS; ++t) x[t] = few_x_cut(xr[t] - 8 * kq, 32 * s + 8 * kq, m);
    }
    // What a step has of LDS: the lane's eight dwords; and a of its groups, as two terms.
    struct Step {
        uint32_t v[8];
        bf16x8 hi[SETS][NG], lo[SETS][NG];
    };
    __device__ __forceinline__ void take(int buf, const u32x4 (&x)[SETS], Step& st)
    {
        const char* s = lds + buf * kGradFewStep;
#pragma unroll
        for (int i = 0; i < 8; ++i) st.v[i] = *reinterpret_cast<const uint32_t*>(s + code_lane + 256 * i);
        float f[SETS][8];
#pragma unroll
        for (int t = 0; t < SETS; ++t) up8<X>(x[t], f[t]);
#pragma unroll
        for (int h = 0; h < NG; ++h) {
            f32x4 sz[4];   // (s, z) of rows 2 i and 2 i + 1
#pragma unroll
            for (int i = 0; i < 4; ++i) sz[i] = *reinterpret_cast<const f32x4*>(s + grid_lane + 256 * h + 16 * i);
#pragma unroll
            for (int t = 0; t < SETS; ++t) {
                u32x4 hi, lo;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = f[t][2 * i] * sz[i].x, b = f[t][2 * i + 1] * sz[i].z;
                    const uint32_t a16 = two_terms(a), b16 = two_terms(b);
                    const float ha = __uint_as_float(a16 & 0xFFFF0000u), hb = __uint_as_float(b16 & 0xFFFF0000u);
                    const float la = __uint_as_float(a16) - ha, lb = __uint_as_float(b16) - hb;   // (8 bits each)
                    hi[i] = __builtin_amdgcn_perm(b16, a16, 0x07060302u);   // the upper halves
                    lo[i] = __builtin_amdgcn_perm(__float_as_uint(lb), __float_as_uint(la), 0x07060302u);
                    off[t][h] = fmaf(__uint_as_float(a16), sz[i].y + kQ4Offset, off[t][h]);
                    off[t][h] = fmaf(__uint_as_float(b16), sz[i].w + kQ4Offset, off[t][h]);
                }
                st.hi[t][h] = __builtin_bit_cast(bf16x8, hi);
                st.lo[t][h] = __builtin_bit_cast(bf16x8, lo);
            }
        }
    }
    __device__ __forceinline__ void add(const Step& st)
    {
        u32x4 even[4], odd[4];   // [two rows], columns 0 2 4 6 and 1 3 5 7
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a = st.v[2 * j], b = st.v[2 * j + 1], mask = 0x0007FFF8u;   // (a half, where the rotation by 3 has it)
            even[j] = __builtin_bit_cast(u32x4, Bf16::codes((a & mask) | (__builtin_rotateleft32(b, 16) & ~mask)));
            odd[j] = __builtin_bit_cast(u32x4, Bf16::codes((__builtin_rotateleft32(a, 16) & mask) | (b & ~mask)));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const u32x4(&u)[4] = e & 1 ? odd : even;
            const bf16x8 w = __builtin_bit_cast(bf16x8, u32x4{u[0][e >> 1], u[1][e >> 1], u[2][e >> 1], u[3][e >> 1]});
#pragma unroll
            for (int t = 0; t < SETS; ++t)
#pragma unroll
                for (int h = 0; h < NG; ++h) {
                    acc[t][h][e] = Bf16::mfma16(st.hi[t][h], w, acc[t][h][e]);
                    acc[t][h][e] = Bf16::mfma16(st.lo[t][h], w, acc[t][h][e]);
                }
        }
    }
    // The second sum off the first.
    __device__ __forceinline__ void take_off()
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int t = 0; t < SETS; ++t)
#pragma unroll
            for (int h = 0; h < NG; ++h) {
                float c = off[t][h];
                c += __shfl_xor(c, 16);
                c += __shfl_xor(c, 32);   // lane % 16 is the row of dy
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = __shfl(c, 4 * (lane >> 4) + r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[t][h][e][r] -= v;
                }
                off[t][h] = 0.f;
            }
    }
    // Steps first, first + by, ... below end, of rows that all exist but in the last step
    // of a layer.
    __device__ __forceinline__ void run(int first, int by, int end)
    {
        const int whole = min(m / 32, end), count = whole > first ? (whole - first + by - 1) / by : 0;
        if (count) {
            u32x4 x[2][SETS];
            stage(first, 0);
            load(first, x[0]);
            __builtin_amdgcn_sched_barrier(0);   // (what is waited for goes by the order of the loads)
            const int second = first + by * min(1, count - 1);
            stage(second, 1);
            load(second, x[1]);
            __builtin_amdgcn_sched_barrier(0);
            // past the last step it is loaded again: every step counts the same loads
            auto step = [&](int k, int buf) {
                wait_loads<LOADS>();
                Step st;
                take(buf, x[buf], st);
                // the reads have to be over before the loads that go to the same place
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                const int next = first + by * min(k + 2, count - 1);
                stage(next, buf);
                load(next, x[buf]);
                __builtin_amdgcn_sched_barrier(0);
                add(st);
                if (k % kGradFewTake == kGradFewTake - 1) take_off();
            };
            int k = 0;
            for (; k + 2 <= count; k += 2) {
                step(k, 0);
                step(k + 1, 1);
            }
            if (k < count) step(k, 0);   // (outside: in the loop it would make every first wait one for all loads)
            wait_loads<0>();
        }
        if (whole < end && whole >= first && (whole - first) % by == 0) {
            u32x4 x[SETS];
            stage(whole, 0);
            load_cut(whole, x);
            wait_loads<0>();
            Step st;
            take(0, x, st);
            add(st);
        }
        take_off();
    }
    // Set t to LDS as 16 rows of 128 columns
    __device__ __forceinline__ void put(int t, float* to) const
    {
        const int lane = threadIdx.x & 63, d = lane & 3;
        const bool h = HALF && d >> 1;
        float* p = to + 64 * (d >> 1) + 16 * (lane >> 2 & 3) + 8 * (d & 1);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = h ? acc[t][NG - 1][e + i][r] : acc[t][0][e + i][r];
                *reinterpret_cast<f32x4*>(p + (4 * (lane >> 4) + r) * kGradFewPitch + e) = v;
            }
    }
};

// Rows t0 .. t0 + n - 1 (n <= 16 SETS) of dy, columns 128 kb .., steps [s0, s1) shared by
// WAVES waves and joined in their order.  part: null, or where float32 sums go instead of
// dx (row t, column j at t ldp + j).
template <class X, int SETS, bool HALF, int WAVES>
__device__ __forceinline__ void grad_few(const uint16_t* __restrict__ dy, int64_t lddy, const Q4Layer& w, int kb, int t0, int n,
                                         int s0, int s1, char* lds, uint16_t* __restrict__ dx, int64_t lddx,
                                         float* __restrict__ part, int64_t ldp)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint16_t* rows[SETS];
#pragma unroll
    for (int s = 0; s < SETS; ++s) rows[s] = dy + (int64_t)(t0 + min(16 * s + (lane & 15), n - 1)) * lddy;
    GradFew<X, SETS, HALF> span(w, kb, rows, lds + wave * kGradFewStage);
    span.run(s0 + wave, WAVES, s1);
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        __syncthreads();   // the joining sums overwrite the staged codes, or the set before
        span.put(s, red + wave * 16 * kGradFewPitch);
        __syncthreads();
        for (int o = threadIdx.x; o < 256; o += 64 * WAVES) {
            const int t = 16 * s + (o >> 4), c = 8 * (o & 15), j = 128 * kb + c;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < WAVES; ++u) {
                const f32x4* p = reinterpret_cast<const f32x4*>(red + (u * 16 + (o >> 4)) * kGradFewPitch + c);
                const f32x4 a = p[0], b = p[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += a[e], v[4 + e] += b[e];
            }
            if (t >= n || j >= w.n) continue;
            if (part) {
                float* p = part + (int64_t)(t0 + t) * ldp + j;
                if (j + 8 <= w.n) {
                    *reinterpret_cast<f32x4_any*>(p) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4_any*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j + e < w.n) p[e] = v[e];
                }
            } else {
                store8(dx + (int64_t)(t0 + t) * lddx, j, w.n, down8<X>(v));
            }
        }
    }
}

}  // namespace bk
