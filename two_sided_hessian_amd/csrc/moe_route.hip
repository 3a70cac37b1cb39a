// moe_route.hip -- the choice of experts for any number of tokens, the choices
// sorted by expert, and the shares' gradient (gfx950).
//
// Choosing.  A token has 16 lanes, lane l the logits 16 i + l.  Logits become
// unsigned keys of the same order (0 for -infinity and NaN, which are never
// chosen; the two zeros are one key), and each of top_k rounds takes the
// largest key of the row of lanes and, of those equal to it, the lowest index.
//
// Sorting.  A stable counting sort: choices have at most 257 different keys (the
// experts, and "none" behind them).  A workgroup takes its tokens 64 at a time,
// a choice per thread; its place among the workgroup's choices of that expert
// is a count of equal keys below it: in the wave by comparing the bits of all
// keys at once (a ballot per bit), over the waves by a table in LDS.  That
// order does not depend on timing.  One workgroup does all of up to 64 tokens; more
// write their counts, and k_moe_place adds, for every choice, the counts of the
// experts and workgroups before it.
//
// Latency bounds it: a launch and its round trips, twice where there is more
// than one workgroup.  One token, 2 of 8: 3.2 us; 16 tokens, 6 of 64: 4.1; 64: 5.4; 256:
// 8.6; 8192: 10.4; 16384, 8 of 128: 14.2.  (One workgroup for 256 tokens, a pass after
// the other: 16.6.)
#include <algorithm>

#include "moe.hpp"

namespace bk {

constexpr int kRouteTokens = 64;   // tokens of a workgroup's pass: 16 lanes each
constexpr int kRouteWaves = 16;
constexpr int kRouteBlocks = 256;  // workgroups at most (16384 tokens, 8 of 128: 14.2 us, with 128 18.8)
constexpr int kRouteKeys = BAKRON_MOE_MAX_EXPERTS + 1;
static_assert(kRouteTokens * BAKRON_MOE_MAX_TOP_K == 64 * kRouteWaves, "a choice per thread");

__device__ __forceinline__ uint32_t route_key(float l)
{
    if (!(l > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(l + 0.f);   // (-0 becomes +0)
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float route_value(uint32_t key)
{
    return __uint_as_float(key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

// Exclusive sums of v[0 .. n) in LDS, n <= 320, by the first wave; `total` past
// the end.
__device__ __forceinline__ void route_scan(int* v, int n)
{
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x, per = (n + 63) / 64;
    int own[5], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        own[i] = i < per && lane * per + i < n ? v[lane * per + i] : 0;
        sum += own[i];
    }
    int before = sum;
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(before, off);
        if (lane >= off) before += o;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        if (i < per && lane * per + i < n) v[lane * per + i] = before;
        before += own[i];
    }
}

// Workgroup b: tokens [b per, min((b + 1) per, T)), per a multiple of 64 where
// there is more than one.  A lone workgroup (counts null, 64 tokens at most) finishes
// place, order and offsets; otherwise place gets a choice's place among the workgroup's of its
// expert, and counts[b][0 .. E] how many there are.
template <class L, int NV>
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(const typename RawOf<L>::type* __restrict__ logits, int64_t ld,
                                                               int T, int per, int E, int k, int bits,
                                                               int32_t* __restrict__ ids, float* __restrict__ weights,
                                                               int32_t* __restrict__ place, int32_t* __restrict__ order,
                                                               int32_t* __restrict__ offsets, int32_t* __restrict__ counts,
                                                               int pitch)
{
    __shared__ int table[kRouteWaves][kRouteKeys];
    __shared__ int hist[kRouteKeys];
    __shared__ int16_t key_of[kRouteTokens * BAKRON_MOE_MAX_TOP_K];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = tid & 15;
    const int first = blockIdx.x * per, last = min(T, first + per);
    for (int e = tid; e <= E; e += 64 * kRouteWaves) hist[e] = 0;
    for (int t0 = first; t0 < last; t0 += kRouteTokens) {
        const int t = t0 + (tid >> 4), here = min(kRouteTokens, last - t0);
        if (t < last) {   // (whole rows of lanes)
            uint32_t key[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = 16 * i + l;
                key[i] = e < E ? route_key(L::up(logits[t * ld + e])) : 0u;
            }
            uint32_t top = 0u, mine = 0u, id = (uint32_t)E;
            for (int j = 0; j < k; ++j) {
                uint32_t m = key[0];
#pragma unroll
                for (int i = 1; i < NV; ++i) m = max(m, key[i]);
                m = row_max(m);
                uint32_t at = 0xFFFFu;
#pragma unroll
                for (int i = NV - 1; i >= 0; --i) at = key[i] == m ? 16 * i + l : at;
                at = row_min(at);
#pragma unroll
                for (int i = 0; i < NV; ++i) key[i] = (uint32_t)(16 * i + l) == at ? 0u : key[i];
                if (j == 0) top = m;
                if (l == j) mine = m, id = m ? at : (uint32_t)E;
            }
            // equal to the largest: a difference of 0, also of infinities
            float ex = mine == top ? 1.f : expf(route_value(mine) - route_value(top));
            if (l >= k || mine == 0u) ex = 0.f;
            const float sum = row_sum(ex);
            if (l < k) {
                const int64_t p = (int64_t)t * k + l;
                ids[p] = id == (uint32_t)E ? -1 : (int32_t)id;
                weights[p] = ex > 0.f ? ex / sum : 0.f;
                key_of[(t - t0) * k + l] = (int16_t)id;
            }
        }
        for (int i = tid; i < kRouteWaves * kRouteKeys; i += 64 * kRouteWaves) (&table[0][0])[i] = 0;
        __syncthreads();
        // a choice per thread
        const int n = here * k;
        const bool on = tid < n;
        const int key = on ? key_of[tid] : 0;
        unsigned long long same = __ballot(on);
        for (int b = 0; b < bits; ++b) {
            const unsigned long long set = __ballot(key >> b & 1);
            same &= key >> b & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (on && rank == 0) table[wave][key] = __popcll(same);
        __syncthreads();
        if (tid <= E) {
            int c[kRouteWaves], s = hist[tid];
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) c[w] = table[w][tid];
#pragma unroll
            for (int w = 0; w < kRouteWaves; ++w) table[w][tid] = s, s += c[w];
            hist[tid] = s;
        }
        __syncthreads();
        if (counts) {
            if (on) place[(int64_t)t0 * k + tid] = table[wave][key] + rank;
            __syncthreads();   // the next pass clears the table and writes key_of
            continue;
        }
        // alone, and this was the only pass
        route_scan(hist, E + 1);
        __syncthreads();
        if (tid <= E) offsets[tid] = hist[tid];
        if (on) {
            const int at = hist[key] + table[wave][key] + rank;
            order[at] = key < E ? tid : -1;
            place[tid] = key < E ? at : -1;
        }
    }
    if (counts && tid < pitch) counts[(int64_t)blockIdx.x * pitch + tid] = tid <= E ? hist[tid] : 0;
}

// The same workgroups again: counts before, four keys (a 16-byte load) per thread
// and the workgroups shared out over the rest.
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_place(const int32_t* __restrict__ counts, int pitch, int blocks,
                                                               int T, int per, int E, int k, const int32_t* __restrict__ ids,
                                                               int32_t* __restrict__ place, int32_t* __restrict__ order,
                                                               int32_t* __restrict__ offsets)
{
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    constexpr int N = 64 * kRouteWaves;
    __shared__ i32x4 before[N], total[N];
    __shared__ int base[kRouteKeys + 3], start[kRouteKeys + 3];
    const int tid = threadIdx.x, quads = pitch / 4, groups = N / quads;
    const int q = tid % quads, g = tid / quads, me = blockIdx.x;
    const int first = me * per * k, last = (int)min((int64_t)T, (int64_t)(me + 1) * per) * k;
    int p = first + tid, id = -1, local = 0;   // the first choice, read beside the counts
    if (p < last) id = ids[p], local = place[p];
    i32x4 b = {0, 0, 0, 0}, a = {0, 0, 0, 0};
    if (g < groups) {
#pragma unroll 8
        for (int i = g; i < blocks; i += groups) {
            const i32x4 c = reinterpret_cast<const i32x4*>(counts)[(int64_t)i * quads + q];
            a += c;
            if (i < me) b += c;
        }
        before[tid] = b;
        total[tid] = a;
    }
    __syncthreads();
    if (tid <= E) {
        int s = 0, t = 0;
#pragma unroll 8
        for (int i = 0; i < groups; ++i) {
            s += reinterpret_cast<const int*>(before)[i * pitch + tid];
            t += reinterpret_cast<const int*>(total)[i * pitch + tid];
        }
        base[tid] = s;
        start[tid] = t;
    }
    __syncthreads();
    route_scan(start, E + 1);
    __syncthreads();
    if (me == 0 && tid <= E) offsets[tid] = start[tid];
    while (p < last) {
        const int e = id < 0 ? E : id, at = start[e] + base[e] + local;
        order[at] = id < 0 ? -1 : p;
        place[p] = id < 0 ? -1 : at;
        p += N;
        if (p < last) id = ids[p], local = place[p];
    }
}

// What a wave's lanes have in LDS before and after, kept apart for the compiler (the
// LDS itself answers a wave in order).
__device__ __forceinline__ void row_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 16 lanes a token; its row is put together in LDS (a wave's own part).
template <class L>
__global__ __launch_bounds__(256) void k_moe_route_grad(const float* __restrict__ dweights, const float* __restrict__ weights,
                                                        const int32_t* __restrict__ ids, int T, int E, int k,
                                                        typename RawOf<L>::type* __restrict__ dlogits, int64_t ld)
{
    __shared__ float rows[16][BAKRON_MOE_MAX_EXPERTS];
    const int l = threadIdx.x & 15;
    float* row = rows[threadIdx.x >> 4];
    for (int64_t t0 = (int64_t)blockIdx.x * 16; t0 < T; t0 += (int64_t)gridDim.x * 16) {
        const int64_t t = t0 + (threadIdx.x >> 4);
        if (t >= T) return;
        int id = -1;
        float w = 0.f, g = 0.f;
        if (l < k) {
            id = ids[t * k + l];
            if (id >= 0 && id < E) w = weights[t * k + l], g = dweights[t * k + l];
            else id = -1;
        }
        const float d = w * (g - row_sum(id < 0 ? 0.f : w * g));
        for (int e = l; e < E; e += 16) row[e] = 0.f;
        row_order();
        if (id >= 0) row[id] = d;
        row_order();
        for (int e = l; e < E; e += 16) dlogits[t * ld + e] = L::down(row[e]);
        row_order();
    }
}

// --------------------------------------------------------------------- host

struct RoutePlan {
    int blocks, per, pitch;   // workgroups, tokens each, ints of a workgroup's counts
};

static RoutePlan route_plan(int64_t T, int64_t E)
{
    RoutePlan p;
    p.pitch = (int)ceil_div(E + 1, 4) * 4;
    const int64_t passes = ceil_div(T, kRouteTokens);
    p.per = (int)ceil_div(passes, kRouteBlocks) * kRouteTokens;
    p.blocks = (int)ceil_div(T, p.per);
    return p;
}

template <class L>
static void route_enqueue(const void* logits, int64_t ld, int64_t T, int64_t E, int k, int32_t* ids, float* weights,
                          int32_t* place, int32_t* order, int32_t* offsets, int32_t* counts, hipStream_t s)
{
    const RoutePlan p = route_plan(T, E);
    int bits = 0;
    while (E >> bits) ++bits;
    auto* kernel = E <= 16 ? k_moe_route<L, 1> : E <= 32 ? k_moe_route<L, 2> : E <= 64 ? k_moe_route<L, 4>
                 : E <= 128 ? k_moe_route<L, 8> : k_moe_route<L, 16>;
    if (p.blocks == 1) counts = nullptr;
    enqueue(kernel, dim3((unsigned)p.blocks), dim3(64 * kRouteWaves), s,
            static_cast<const typename RawOf<L>::type*>(logits), ld, (int)T, p.per, (int)E, k, bits, ids, weights, place,
            order, offsets, counts, p.pitch);
    if (counts)
        enqueue(k_moe_place, dim3((unsigned)p.blocks), dim3(64 * kRouteWaves), s, counts, p.pitch, p.blocks, (int)T, p.per,
                (int)E, k, ids, place, order, offsets);
}

template <class L>
static void route_grad_enqueue(const float* dweights, const float* weights, const int32_t* ids, int64_t T, int64_t E, int k,
                               void* dlogits, int64_t ld, hipStream_t s)
{
    enqueue(k_moe_route_grad<L>, dim3((unsigned)std::min<int64_t>(ceil_div(T, 16), 4096)), dim3(256), s, dweights, weights,
            ids, (int)T, (int)E, k, static_cast<typename RawOf<L>::type*>(dlogits), ld);
}

__global__ __launch_bounds__(64) void k_moe_no_rows(int32_t* __restrict__ offsets, int n)
{
    for (int e = threadIdx.x; e < n; e += 64) offsets[e] = 0;
}

static bool route_size_ok(int64_t T, int32_t k)
{
    return T >= 0 && T <= BAKRON_MOE_MAX_ROWS && T * std::max(k, 1) <= BAKRON_MOE_MAX_ROWS;
}
static bool route_arg_ok(int64_t E, int32_t k)
{
    return E >= 1 && E <= BAKRON_MOE_MAX_EXPERTS && k >= 1 && k <= E && k <= BAKRON_MOE_MAX_TOP_K;
}

}  // namespace bk

extern "C" {

size_t bakron_moe_route_workspace_bytes(int64_t tokens, int64_t experts, int32_t top_k)
{
    if (!bk::route_arg_ok(experts, top_k) || !bk::route_size_ok(tokens, top_k) || tokens == 0) return 0;
    const bk::RoutePlan p = bk::route_plan(tokens, experts);
    return p.blocks == 1 ? 0 : bk::align_up(4 * (size_t)p.blocks * p.pitch);
}

int bakron_moe_route(const void* logits, int64_t ld, int64_t tokens, int32_t type, int64_t experts, int32_t top_k,
                     int32_t* ids, float* weights, int32_t* place, int32_t* order, int32_t* offsets, void* workspace,
                     size_t workspace_bytes, hipStream_t stream)
{
    if (top_k < 0 || top_k > BAKRON_MOE_MAX_TOP_K) return BAKRON_ERR_BAD_ARG;
    if (!bk::route_size_ok(tokens, top_k)) return BAKRON_ERR_BAD_SIZE;
    if (!bk::route_arg_ok(experts, top_k) || (!bk::moe_type_ok(type) && type != BAKRON_MOE_F32) ||
        !bk::moe_ld_ok(ld, experts))
        return BAKRON_ERR_BAD_ARG;
    if (!offsets) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(offsets, 4)) return BAKRON_ERR_BAD_ARG;
    if (tokens == 0) {
        bk::enqueue(bk::k_moe_no_rows, dim3(1), dim3(64), stream, offsets, (int)experts + 1);
        return bk::moe_done();
    }
    if (!logits || !ids || !weights || !place || !order) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(logits, type == BAKRON_MOE_F32 ? 4 : 2) || !bk::moe_at(ids, 4) || !bk::moe_at(weights, 4) ||
        !bk::moe_at(place, 4) || !bk::moe_at(order, 4))
        return BAKRON_ERR_BAD_ARG;
    const size_t need = bakron_moe_route_workspace_bytes(tokens, experts, top_k);
    if (need && (!workspace || workspace_bytes < need || !bk::moe_at(workspace, bk::kAlign))) return BAKRON_ERR_WORKSPACE;
    auto* run = type == BAKRON_MOE_F32 ? bk::route_enqueue<bk::Fp32>
              : type == BAKRON_Q4_BF16 ? bk::route_enqueue<bk::Bf16> : bk::route_enqueue<bk::Fp16>;
    run(logits, ld, tokens, experts, top_k, ids, weights, place, order, offsets, static_cast<int32_t*>(workspace), stream);
    return bk::moe_done();
}

int bakron_moe_route_grad(const float* dweights, const float* weights, const int32_t* ids, int64_t tokens,
                          int64_t experts, int32_t top_k, void* dlogits, int64_t ld, int32_t type, hipStream_t stream)
{
    if (top_k < 0 || top_k > BAKRON_MOE_MAX_TOP_K) return BAKRON_ERR_BAD_ARG;
    if (!bk::route_size_ok(tokens, top_k)) return BAKRON_ERR_BAD_SIZE;
    if (!bk::route_arg_ok(experts, top_k) || (!bk::moe_type_ok(type) && type != BAKRON_MOE_F32) ||
        !bk::moe_ld_ok(ld, experts))
        return BAKRON_ERR_BAD_ARG;
    if (tokens == 0) return BAKRON_SUCCESS;
    if (!dweights || !weights || !ids || !dlogits) return BAKRON_ERR_NULL_POINTER;
    if (!bk::moe_at(dlogits, type == BAKRON_MOE_F32 ? 4 : 2) || !bk::moe_at(ids, 4) || !bk::moe_at(weights, 4) ||
        !bk::moe_at(dweights, 4))
        return BAKRON_ERR_BAD_ARG;
    auto* run = type == BAKRON_MOE_F32 ? bk::route_grad_enqueue<bk::Fp32>
              : type == BAKRON_Q4_BF16 ? bk::route_grad_enqueue<bk::Bf16> : bk::route_grad_enqueue<bk::Fp16>;
    run(dweights, weights, ids, tokens, experts, top_k, dlogits, ld, stream);
    return bk::moe_done();
}

}  // extern "C"
