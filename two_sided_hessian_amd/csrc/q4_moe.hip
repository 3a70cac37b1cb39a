// q4_moe.hip -- a whole mixture-of-experts layer on packed 4-bit experts, for
// a few tokens (gfx950).
//
//   l = x router^T;  token t chooses the top_k experts of largest l_t, shares
//   p_te = softmax of l over them;
//   y_t = sum_e p_te down_e ( silu(gate_e x_t) * (up_e x_t) ).
//
// Three launches, since every expert's inner activations have to be complete
// before the down products and the logits before the choice (logits made by
// every workgroup for itself, in two launches, were slower: 61 us against 55
// for one token and 8 experts of 4096 x 14336, 44 against 36 for 16 tokens
// and 16 experts of 2048 x 1024):
//   k_q4_router: the logits.
//   k_q4_moe_up: one workgroup per (row tiles of ffn, expert).  It ranks its
//     own expert among each token's logits (a token chooses it if fewer than
//     top_k logits are larger, or equal with a lower index), so no selection
//     has to come first; workgroups of experts that no token chose end there.
//     Gate and up rows share the tokens' fragments.  One more workgroup writes
//     ids, weights and the choices sorted by expert.
//   k_q4_moe_down: one workgroup per row tile of hidden (and per split of the
//     work, where there are fewer tiles than CUs): its waves share the column
//     blocks of all chosen experts evenly, keep their sums per token in LDS and
//     are joined in wave order; splits are joined by the last one to finish, in
//     split order.  No result depends on timing.
// HBM bounds it: the chosen experts' codes and grids are read once.  Measured,
// router, up and down in turn: one token, 2 of 8 experts of 4096 x 14336, groups
// of 128: 5, 29 (4.5 TB/s) and 16 us, the call 50; 16 tokens, 6 of 64 experts of
// 2048 x 1024, groups of 64: 6, 40 (3.5 TB/s) and 27, the call 69 - 72:
// choosing, first round trips and the joins weigh more in short rows, and grids
// are a fifth of the bytes; 16 tokens, 2 of 16 experts of 4096 x 14336: 309 us,
// 4.5 TB/s over all.
#include <algorithm>

#include "../../include/bakron_q4.h"
#include "q4_few.hpp"

namespace bk {

constexpr int kMoeTokens = BAKRON_Q4_MOE_MAX_TOKENS;
constexpr int kMoeTopK = BAKRON_Q4_MOE_MAX_TOP_K;
constexpr int kMoeExperts = BAKRON_Q4_MAX_LAYERS;
constexpr int kMoePairs = kMoeTokens * kMoeTopK;

// A choice: p = t k + j, the j-th of token t, with its token beside it (a
// division by k, 20 instructions, where it is made and not where it is used).
__device__ __forceinline__ int32_t moe_choice(int t, int p) { return t << 16 | p; }
__device__ __forceinline__ int choice_token(int32_t c) { return c >> 16; }
__device__ __forceinline__ int choice_place(int32_t c) { return c & 0xFFFF; }

// The choices sorted by expert, as k_q4_moe_up leaves them for k_q4_moe_down.
struct MoePlan {
    int32_t active;                    // experts that some token chose, ascending:
    int32_t expert[kMoeExperts];
    int32_t start[kMoeExperts + 1];    // their choices: pair[start[a]] .. pair[start[a + 1] - 1]
    int32_t pair[kMoePairs];
};

// ------------------------------------------------------------------- router
//
// logits[t][e], 16 tokens x 16 experts per workgroup, its waves the 32-column
// steps in turn (four steps' loads in flight), joined in wave order.
template <class X>
__global__ __launch_bounds__(1024) void k_q4_router(const uint16_t* __restrict__ x, int64_t ldx, int T, int h,
                                                    const uint16_t* __restrict__ router, int E, float* __restrict__ logits,
                                                    int32_t* __restrict__ done, int ndone)
{
    typedef typename X::vec vec;
    __shared__ float red[16][4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, q = lane >> 4, r = lane & 15;
    if (blockIdx.x == 0 && blockIdx.y == 0)   // the counters of k_q4_moe_down's splits
        for (int i = threadIdx.x; i < ndone; i += 1024) done[i] = 0;
    const uint16_t* xr = x + (int64_t)min(t0 + r, T - 1) * ldx;
    const uint16_t* wr = router + (int64_t)min(e0 + r, E - 1) * h;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int whole = h / 32;
    constexpr int U = 4;
    for (int s0 = wave; s0 < whole; s0 += 16 * U) {
        u32x4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = 32 * min(s0 + 16 * u, whole - 1) + 8 * q;
            a[u] = *reinterpret_cast<const u32x4_any*>(xr + k);
            b[u] = *reinterpret_cast<const u32x4_any*>(wr + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + 16 * u < whole)
                acc = X::mfma16(__builtin_bit_cast(vec, a[u]), __builtin_bit_cast(vec, b[u]), acc);
    }
    if (32 * whole < h && whole % 16 == wave)
        acc = X::mfma16(__builtin_bit_cast(vec, few_x_cut(xr, 32 * whole + 8 * q, h)),
                        __builtin_bit_cast(vec, few_x_cut(wr, 32 * whole + 8 * q, h)), acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int i = threadIdx.x >> 6;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) v += red[u][i][lane];
        const int t = t0 + 4 * q + i, e = e0 + r;
        if (t < T && e < E) logits[(int64_t)t * E + e] = v;
    }
}

// NaN counts as -infinity in the order of logits
__device__ __forceinline__ float moe_key(float l) { return l == l ? l : -INFINITY; }

// Rank of expert e among the E logits l of a token (a wave's work, every lane
// gets the result).
__device__ __forceinline__ int moe_rank(const float* __restrict__ l, int E, int e)
{
    const int lane = threadIdx.x & 63;
    const float mine = moe_key(l[e]);
    int n = 0;
    for (int f0 = 0; f0 < E; f0 += 64) {
        const int f = f0 + lane;
        const float v = moe_key(l[min(f, E - 1)]);
        n += __popcll(__ballot(f < E && (v > mine || (v == mine && f < e))));
    }
    return n;
}

// ids, weights and the plan: one workgroup of 8 waves, a wave per token in turn.
__device__ void moe_choose(const float* __restrict__ logits, int T, int E, int k, int32_t* __restrict__ ids,
                           float* __restrict__ weights, MoePlan* __restrict__ plan)
{
    __shared__ int16_t chosen[kMoePairs];
    __shared__ float keys[8][kMoeExperts];
    __shared__ int count[kMoeExperts], slot[kMoeExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int t = wave; t < T; t += 8) {
        const float* l = logits + (int64_t)t * E;
        for (int f = lane; f < E; f += 64) keys[wave][f] = moe_key(l[f]);
        __builtin_amdgcn_wave_barrier();
        for (int f = lane; f < E; f += 64) {
            const float v = keys[wave][f];
            int rank = 0;
            for (int g = 0; g < E; ++g) {
                const float u = keys[wave][g];
                rank += u > v || (u == v && g < f);
            }
            if (rank < k) chosen[t * k + rank] = (int16_t)f;
        }
        __builtin_amdgcn_wave_barrier();
        const int e = lane < k ? chosen[t * k + lane] : 0;
        const float top = l[chosen[t * k]];
        const float ex = lane < k ? expf(l[e] - top) : 0.f;
        float sum = ex;
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor(sum, off);   // top_k <= 16 lanes
        if (lane < k) ids[t * k + lane] = e, weights[t * k + lane] = ex / sum;
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    const int pairs = T * k;
    for (int e = wave; e < E; e += 8) {
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64)
            n += __popcll(__ballot(p0 + lane < pairs && chosen[min(p0 + lane, pairs - 1)] == e));
        if (lane == 0) count[e] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int a = 0, at = 0;
        for (int e = 0; e < E; ++e) {
            if (!count[e]) continue;
            plan->expert[a] = e;
            plan->start[a] = at;
            slot[e] = at;
            at += count[e];
            ++a;
        }
        plan->start[a] = at;
        plan->active = a;
    }
    __syncthreads();
    for (int e = wave; e < E; e += 8) {
        if (!count[e]) continue;
        int at = slot[e];
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const bool in = p0 + lane < pairs && chosen[min(p0 + lane, pairs - 1)] == e;
            const unsigned long long b = __ballot(in);
            if (in) plan->pair[at + __popcll(b & ((1ull << lane) - 1))] = moe_choice((p0 + lane) / k, p0 + lane);
            at += __popcll(b);
        }
    }
}

// ---------------------------------------------------------- gate, up, silu

__device__ __forceinline__ Q4Layer moe_layer(Q4Layer w, int e, int64_t layer_bytes)
{
    w.codes = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(w.codes) + e * layer_bytes);
    w.grid = reinterpret_cast<const f32x2*>(reinterpret_cast<const char*>(w.grid) + e * layer_bytes);
    return w;
}

// a = silu(gate x) * (up x) of row tiles rt0 .. rt0 + 8 / WS - 1, for the choices
// list[0 .. n) of an expert, at most 4 TQ; WS waves share a tile's columns.
// Kept as two bfloat16 terms (a = hi + lo to 16 bits): the range of float32 in
// either activation type, and no rounding that the result sees.
template <class X, int TQ, int U, int WS, bool HALF>
__device__ __forceinline__ void moe_up(const uint16_t* __restrict__ x, int64_t ldx, const Q4Layer (&w)[2], int rt0,
                                       const int32_t* list, int n, char* lds, uint16_t* __restrict__ hi,
                                       uint16_t* __restrict__ lo, int64_t lda)
{
    typedef FewSpan<X, TQ, 2, U, HALF> Span;
    static_assert(Span::NT == 1, "one MFMA tile of tokens");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint16_t* xr[TQ];
#pragma unroll
    for (int t = 0; t < TQ; ++t) xr[t] = x + (int64_t)choice_token(list[min(4 * t + (lane >> 4), n - 1)]) * ldx;
    Span span(lds + wave * few_lds(4));
    span.template rows<2>(w, rt0 + wave / WS);
    span.tokens(xr);
    span.run(wave % WS, WS, w[0].KB);
    __syncthreads();
    float(*red)[8][64] = reinterpret_cast<float(*)[8][64]>(lds);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[wave][4 * j + e][lane] = span.acc[j][0][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 8 / WS * 256; o += 512) {
        const int tile = o >> 8, e = o >> 6 & 3;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int u = 0; u < WS; ++u) a += red[tile * WS + u][e][lane], b += red[tile * WS + u][4 + e][lane];
        const int c = 4 * (lane >> 4) + e;
        if (c < n && rt0 + tile < w[0].RT) {
            const float v = a / (1.f + expf(-a)) * b;
            const uint16_t vh = Bf16::down(v);
            const int64_t at = (int64_t)choice_place(list[c]) * lda + (rt0 + tile) * 16 + (lane & 15);
            hi[at] = vh;
            lo[at] = Bf16::down(v - Bf16::up(vh));
        }
    }
    __syncthreads();
}

// The expert of rank j among a token's logits (a wave's work on an array of E
// keys of its own; every lane gets the result).
__device__ __forceinline__ int moe_nth(const float* __restrict__ l, int E, int j, float* keys)
{
    const int lane = threadIdx.x & 63;
    for (int f = lane; f < E; f += 64) keys[f] = moe_key(l[f]);
    __builtin_amdgcn_wave_barrier();
    int found = 0;
    for (int f0 = 0; f0 < E; f0 += 64) {
        const int f = f0 + lane;
        const float v = keys[min(f, E - 1)];
        int rank = 0;
        for (int g = 0; g < E; ++g) {
            const float u = keys[g];
            rank += u > v || (u == v && g < f);
        }
        const unsigned long long b = __ballot(f < E && rank == j);
        if (b) found = f0 + __ffsll(b) - 1;
    }
    return found;
}

// grid: groups of 8 / WS row tiles of ffn (and one for ids, weights and the plan) x slots.  A
// slot is an expert, or, where the tokens make fewer choices than there are
// experts, a choice; the first choice of an expert stands for it.
template <class X, int WS, bool HALF>
__global__ __launch_bounds__(512, 4) void k_q4_moe_up(const uint16_t* __restrict__ x, int64_t ldx, int T, Q4Layer gate,
                                                      Q4Layer up, int64_t layer_bytes, const float* __restrict__ logits,
                                                      int E, int k, uint16_t* __restrict__ hi,
                                                      uint16_t* __restrict__ lo, int64_t lda, int32_t* __restrict__ ids,
                                                      float* __restrict__ weights, MoePlan* __restrict__ plan)
{
    __shared__ __align__(16) char lds[8 * few_lds(4)];
    __shared__ int32_t list[kMoeTokens];
    __shared__ int rank[kMoeTokens];
    __shared__ int expert;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rt = blockIdx.x, slot = blockIdx.y;
    if (rt == (int)gridDim.x - 1) {
        if (slot == 0) moe_choose(logits, T, E, k, ids, weights, plan);
        return;
    }
    int e = slot, first = 0;
    if ((int)gridDim.y < E) {   // slots are choices
        first = slot / k;
        if (wave == 0) {
            const int f = moe_nth(logits + (int64_t)first * E, E, slot - first * k, reinterpret_cast<float*>(lds));
            if (lane == 0) expert = f;
        }
        __syncthreads();
        e = expert;
    }
    for (int t = wave; t < T; t += 8) {
        const int n = moe_rank(logits + (int64_t)t * E, E, e);
        if (lane == 0) rank[t] = n;
    }
    __syncthreads();
    const bool mine = lane < T && rank[min(lane, T - 1)] < k;
    const unsigned long long b = __ballot(mine);
    const int n = __popcll(b);
    if (n == 0 || ((int)gridDim.y < E && __ffsll(b) - 1 < first)) return;
    if (wave == 0 && mine) list[__popcll(b & ((1ull << lane) - 1))] = moe_choice(lane, lane * k + rank[lane]);
    __syncthreads();
    const Q4Layer w[2] = {moe_layer(gate, e, layer_bytes), moe_layer(up, e, layer_bytes)};
    for (int n0 = 0; n0 < n; n0 += 16) {
        const int nn = min(16, n - n0);
        if (nn <= 4) moe_up<X, 1, 2, WS, HALF>(x, ldx, w, 8 / WS * rt, list + n0, nn, lds, hi, lo, lda);
        else moe_up<X, 4, 1, WS, HALF>(x, ldx, w, 8 / WS * rt, list + n0, nn, lds, hi, lo, lda);
    }
}

// --------------------------------------------------------------- down, join

// Column blocks [kb0, kb1) of one expert's row tile for its choices pair[0 .. n),
// at most 2 TQ: rows hi and lo of a choice are two tokens of the span.  Adds
// p times the sums to the wave's ys[token][row].
template <int TQ, bool HALF>
__device__ __forceinline__ void moe_down(const uint16_t* __restrict__ hi, const uint16_t* __restrict__ lo, int64_t lda,
                                         const Q4Layer& w, int rt, int kb0, int kb1, const int32_t* pair, int n,
                                         const float* weights, char* lds, float (*ys)[16])
{
    typedef FewSpan<Bf16, TQ, 1, 2, HALF> Span;
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const uint16_t* xr[TQ];
#pragma unroll
    for (int t = 0; t < TQ; ++t) {
        const int c = min(4 * t + q, 2 * n - 1);
        xr[t] = (c < n ? hi : lo) + (int64_t)choice_place(pair[c < n ? c : c - n]) * lda;
    }
    Span span(lds);
    const Q4Layer ws[1] = {w};
    span.template rows<1>(ws, rt);
    span.tokens(xr);
    span.run(kb0, 1, kb1);
    // hi and lo of a choice are different lanes' adds to one place: one after
    // the other
#pragma unroll
    for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 4 * q + e - part * n;
            if (c >= 0 && c < n) {
                ys[choice_token(pair[c])][r] += weights[choice_place(pair[c])] * span.acc[0][0][e];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

constexpr int kDownWaves = 16;
constexpr int kMoeSplits = 4;

template <class X, int TMAX, bool HALF>
__global__ __launch_bounds__(64 * kDownWaves) void k_q4_moe_down(const uint16_t* __restrict__ hi,
                                                                 const uint16_t* __restrict__ lo, int64_t lda,
                                                                 Q4Layer down, int64_t layer_bytes,
                                                                 const MoePlan* __restrict__ plan,
                                                                 const float* __restrict__ weights, int T, int k,
                                                                 float* __restrict__ part, int32_t* __restrict__ done,
                                                                 uint16_t* __restrict__ y, int64_t ldy)
{
    __shared__ __align__(16) char stage[kDownWaves][few_lds(4)];
    __shared__ float sums[kDownWaves][TMAX][16];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rt = blockIdx.x, split = blockIdx.y, splits = gridDim.y;
    // the plan and the shares, in one round trip
    __shared__ MoePlan pl;
    __shared__ float share[kMoePairs];
    for (int i = threadIdx.x; i < (int)(sizeof(MoePlan) / 4); i += 64 * kDownWaves)
        reinterpret_cast<int32_t*>(&pl)[i] = reinterpret_cast<const int32_t*>(plan)[i];
    for (int i = threadIdx.x; i < T * k; i += 64 * kDownWaves) share[i] = weights[i];
    __syncthreads();
    float(*ys)[16] = sums[wave];
    for (int i = lane; i < 16 * T; i += 64) ys[i >> 4][i & 15] = 0.f;
    __builtin_amdgcn_wave_barrier();

    // this wave's share of the active experts' column blocks
    const int active = pl.active, total = active * down.KB;
    const int parts = splits * kDownWaves, me = split * kDownWaves + wave;
    const int i0 = (int)((int64_t)total * me / parts), i1 = (int)((int64_t)total * (me + 1) / parts);
    for (int i = i0; i < i1;) {
        const int a = i / down.KB, kb0 = i - a * down.KB, kb1 = min(down.KB, kb0 + i1 - i);
        const int s0 = pl.start[a], s1 = pl.start[a + 1];
        const Q4Layer w = moe_layer(down, pl.expert[a], layer_bytes);
        for (int s = s0; s < s1; s += 8) {
            const int n = min(8, s1 - s);
            if (n <= 2)
                moe_down<1, HALF>(hi, lo, lda, w, rt, kb0, kb1, pl.pair + s, n, share, stage[wave], ys);
            else
                moe_down<4, HALF>(hi, lo, lda, w, rt, kb0, kb1, pl.pair + s, n, share, stage[wave], ys);
        }
        i += kb1 - kb0;
    }
    __syncthreads();
    const int h = down.m;
    for (int i = threadIdx.x; i < 16 * T; i += 64 * kDownWaves) {
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kDownWaves; ++u) v += sums[u][i >> 4][i & 15];
        const int t = i >> 4, row = rt * 16 + (i & 15);
        if (row >= h) continue;
        if (splits == 1) y[(int64_t)t * ldy + row] = X::down(v);
        else __hip_atomic_store(&part[((int64_t)split * T + t) * h + row], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (splits == 1) return;
    // The last split of a row tile to get here adds all of them, in split
    // order.  Partial sums are stored and loaded past the XCD's own cache
    // (device-scope atomics), and each wave's stores have completed before the
    // tile's counter (cleared by k_q4_router) is raised.  That order is this
    // chip's, not the language's: a device-scope store counts as complete
    // (vmcnt) once it has reached the memory that all XCDs read, device-scope
    // loads read there, and the loads below are issued after the counter's
    // answer.  The language's model asks for a release and an acquire, which
    // write back and drop the whole cache (measured at 80 us for a launch).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(&done[rt], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
    __syncthreads();
    if (!last) return;
    for (int i = threadIdx.x; i < 16 * T; i += 64 * kDownWaves) {
        const int t = i >> 4, row = rt * 16 + (i & 15);
        if (row >= h) continue;
        float v = 0.f;
        for (int u = 0; u < splits; ++u)
            v += __hip_atomic_load(&part[((int64_t)u * T + t) * h + row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        y[(int64_t)t * ldy + row] = X::down(v);
    }
}

struct MoeWork {
    int64_t lda;
    size_t logits, plan, done, hi, lo, part, bytes;
};

static MoeWork moe_work(int64_t T, int64_t h, int64_t f, int64_t E, int k)
{
    MoeWork w;
    w.lda = ceil_div(f, 16) * 16;
    w.logits = 0;
    w.plan = align_up(4 * (size_t)T * E);
    w.done = w.plan + align_up(sizeof(MoePlan));
    w.hi = w.done + align_up(4 * (size_t)ceil_div(h, 16));
    w.lo = w.hi + align_up(2 * (size_t)T * k * w.lda);
    w.part = w.lo + align_up(2 * (size_t)T * k * w.lda);
    w.bytes = w.part + align_up(4 * (size_t)kMoeSplits * T * h);
    return w;
}

int q4_zero_enqueue(void* y, int64_t ld, int64_t rows, int64_t cols, hipStream_t s);

template <class X, bool HALF>
static int moe_enqueue(const void* x, int64_t ldx, int64_t T, const void* router, const void* gate, const void* up,
                       const void* down, int64_t h, int64_t f, int64_t E, int k, int64_t g, void* y, int64_t ldy,
                       int32_t* ids, float* weights, void* ws, hipStream_t s)
{
    const uint16_t* xp = static_cast<const uint16_t*>(x);
    const MoeWork w = moe_work(T, h, f, E, k);
    char* base = static_cast<char*>(ws);
    float* logits = reinterpret_cast<float*>(base + w.logits);
    MoePlan* plan = reinterpret_cast<MoePlan*>(base + w.plan);
    int32_t* done = reinterpret_cast<int32_t*>(base + w.done);
    uint16_t* hi = reinterpret_cast<uint16_t*>(base + w.hi);
    uint16_t* lo = reinterpret_cast<uint16_t*>(base + w.lo);
    float* part = reinterpret_cast<float*>(base + w.part);
    const Q4Dims du = q4_dims(f, h, g), dd = q4_dims(h, f, g);
    launch(nullptr, KK_Q4_ROUTER, 2.0 * T * E * h, 0.0, k_q4_router<X>,
           dim3((unsigned)ceil_div(E, 16), (unsigned)ceil_div(T, 16)), dim3(1024), s, xp, ldx, (int)T, (int)h,
           static_cast<const uint16_t*>(router), (int)E, logits, done, dd.RT);
    const int64_t slots = std::min<int64_t>(E, T * k);
    // Waves per row tile: as many as keep the launch to two rounds of the 4096
    // waves that fit the chip at this kernel's registers, at least two (16
    // tokens, 64 experts of 2048 x 1024: 40 us with 2 waves, 65 with 8; one
    // token, 2 of 8 experts of 4096 x 14336: 28 us with 4, 37 with 8; 16 tokens,
    // 16 experts of 4096 x 14336, whole call: 303 us with 2, 333 with 1).
    const int64_t waves = du.RT * slots;
    auto* kup = k_q4_moe_up<X, 2, HALF>;
    int per = 2;
    if (8 * waves <= 8192) kup = k_q4_moe_up<X, 8, HALF>, per = 8;
    else if (4 * waves <= 8192) kup = k_q4_moe_up<X, 4, HALF>, per = 4;
    launch(nullptr, KK_Q4_MOE_UP, 4.0 * T * k * h * f, 0.0, kup,
           dim3((unsigned)(ceil_div(du.RT, 8 / per) + 1), (unsigned)slots), dim3(512), s, xp, ldx, (int)T,
           q4_layer(gate, du), q4_layer(up, du), (int64_t)du.bytes, logits, (int)E, k, hi, lo, w.lda, ids, weights, plan);
    if (f == 0) return q4_zero_enqueue(y, ldy, T, h, s);
    // Splits of the down products: a workgroup per CU where there are fewer row
    // tiles, but two column blocks at least for every wave (3 tokens, 5 experts
    // of 1003 x 1501: 17.4 us with one split, 18.7 with four).
    const int64_t blocks = slots * dd.KB / (2 * kDownWaves);
    const int splits = (int)std::max<int64_t>(1, std::min<int64_t>({kMoeSplits, ceil_div(256, dd.RT), blocks}));
    launch(nullptr, KK_Q4_MOE_DOWN, 2.0 * T * k * h * f, 0.0,
           T <= 16 ? k_q4_moe_down<X, 16, HALF> : k_q4_moe_down<X, 64, HALF>,
           dim3((unsigned)dd.RT, (unsigned)splits), dim3(64 * kDownWaves), s, hi, lo, w.lda, q4_layer(down, dd),
           (int64_t)dd.bytes, plan, weights, (int)T, k, part, done, static_cast<uint16_t*>(y), ldy);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace bk

extern "C" {

size_t bakron_q4_moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t ffn, int64_t experts, int32_t top_k,
                                     int64_t group_size)
{
    if (tokens <= 0 || tokens > BAKRON_Q4_MOE_MAX_TOKENS || hidden <= 0 || hidden > BAKRON_MAX_DIM || ffn < 0 ||
        ffn > BAKRON_MAX_DIM || experts < 1 || experts > BAKRON_Q4_MAX_LAYERS || top_k < 1 || top_k > experts ||
        top_k > BAKRON_Q4_MOE_MAX_TOP_K || group_size < 0 || group_size % 64)
        return 0;
    return bk::moe_work(tokens, hidden, ffn, experts, top_k).bytes;
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
    const bool half = group_size / 64 % 2;   // a group ends inside a block of 128 columns
    auto* run = type == BAKRON_Q4_BF16 ? (half ? bk::moe_enqueue<bk::Bf16, true> : bk::moe_enqueue<bk::Bf16, false>)
                                       : (half ? bk::moe_enqueue<bk::Fp16, true> : bk::moe_enqueue<bk::Fp16, false>);
    return run(x, ldx, tokens, router, gate, up, down, hidden, ffn, experts, top_k, group_size, y, ldy, ids, weights,
               workspace, stream)
               ? BAKRON_ERR_HIP
               : BAKRON_SUCCESS;
}

}  // extern "C"
