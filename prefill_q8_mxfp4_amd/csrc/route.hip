// Rows sorted by expert and back: the counting sort of the router's choices,
// rows moved to their sorted places, the weighted sum back, and the gradients
// of both moves.
#include "int8.h"

namespace qg {

// ================================================================ route
// f = t * topk + j, e = ids[f], kept when 0 <= e < E:
//   off[e] = #{f : 0 <= ids[f] < e},   pos[f] = off[e] + #{f' < f : ids[f'] = e}.
//
// One launch, no memory shared between workgroups: each counts every choice
// into LDS (all of them, and those before its own run of choices), scans the
// totals over the experts, and gives its own run its places.  A run's rank
// order is the flat order: waves take their parts in turn of 64 choices, a
// lane's rank among the equal ids of its 64 from ballots over the id's bits.
// Counting is by LDS adds of whole numbers, so the order in which they land
// changes nothing.
constexpr int RT_THREADS = 1024;
constexpr int RT_WAVES = RT_THREADS / 64;

__global__ __launch_bounds__(RT_THREADS) void route_kernel(RouteArgs a, int run, int bits)
{
    extern __shared__ int lds[];
    int *tot = lds;           // [E] every choice, then off[e]
    int *mine = lds + a.E;    // [E] choices before this run, then the next place
    __shared__ int wsum[RT_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int lo = min((int)blockIdx.x * run, a.n), hi = min(lo + run, a.n);

    for (int e = tid; e < 2 * a.E; e += RT_THREADS)
        lds[e] = 0;
    __syncthreads();
    auto count = [&](int f, int e) {
        if (e >= 0 && e < a.E) {
            atomicAdd(&tot[e], 1);
            if (f < lo)
                atomicAdd(&mine[e], 1);
        }
    };
    // four ids a load, four loads in flight
    const int quads = a.vec ? a.n / 4 : 0;
    for (int q0 = tid; q0 < quads; q0 += 4 * RT_THREADS) {
        typedef int i32x4v __attribute__((ext_vector_type(4)));
        i32x4v v[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int q = q0 + k * RT_THREADS;
            v[k] = q < quads ? ((const i32x4v *)a.ids)[q] : i32x4v{-1, -1, -1, -1};
        }
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                count((q0 + k * RT_THREADS) * 4 + i, v[k][i]);
    }
    for (int f = quads * 4 + tid; f < a.n; f += RT_THREADS)
        count(f, a.ids[f]);
    __syncthreads();
    // exclusive scan of tot over the experts, RT_THREADS of them at a time
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += RT_THREADS) {
        const int e = e0 + tid;
        const int v = e < a.E ? tot[e] : 0;
        int s = v;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d)
                s += o;
        }
        if (lane == 63)
            wsum[wid] = s;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < RT_WAVES; w++) {
            before += w < wid ? wsum[w] : 0;
            all += wsum[w];
        }
        if (e < a.E) {
            const int off = carry + before + s - v;
            mine[e] += off;
            if (blockIdx.x == 0)
                a.off[e] = off;
        }
        carry += all;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        a.off[a.E] = carry;
    // places of this run's choices, 64 at a time in order
    for (int f0 = lo; f0 < hi; f0 += RT_THREADS) {
        const int f = f0 + tid;
        const int id = f < hi ? a.ids[f] : -1;
        const bool kept = id >= 0 && id < a.E;
        unsigned long long same = __ballot(kept);
        for (int b = 0; b < bits; b++) {
            const unsigned long long m = __ballot((id >> b) & 1);
            same &= (id >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const bool first = kept && rank == 0;
        int base = 0;
        const int waves = min(RT_WAVES, (hi - f0 + 63) / 64);
        for (int w = 0; w < waves; w++) {  // waves in order
            if (w == wid && first)
                base = atomicAdd(&mine[id], __popcll(same));
            __syncthreads();
        }
        base = __shfl(base, __ffsll(same) - 1);
        if (f < hi)
            a.pos[f] = kept ? base + rank : -1;
    }
}

hipError_t launch_route(RouteArgs a, hipStream_t st)
{
    int bits = 0;
    while (bits < 31 && (1 << bits) < a.E)
        bits++;
    // runs of 256 choices, up to 256 of them: the count of all choices, which every
    // workgroup makes, is most of the time, the places of a run the rest
    int run = (a.n + 255) / 256;
    run = run < 256 ? 256 : (run + 63) / 64 * 64;
    const int wgs = a.n > 0 ? (a.n + run - 1) / run : 1;
    a.vec = ((uintptr_t)a.ids & 15u) == 0;
    const int lds = 2 * a.E * 4;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void *)route_kernel,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(route_kernel, dim3(wgs), dim3(RT_THREADS), lds, st, a, run, bits);
    return hipGetLastError();
}

// ================================================================ moves
// A row is cut into 16-byte vectors; rows whose size is no multiple of 16
// start off alignment, which gfx950's global loads and stores take, and end in
// single elements.  Moving bytes is the bound: a wave owns 64 vectors of a token
// and has the loads of several of its rows in flight.
template <int DT>
struct Elem {
    typedef float T;
    static constexpr int V = 4;
};
template <>
struct Elem<OUT_BF16> {
    typedef __bf16 T;
    static constexpr int V = 8;
};

// A vector as it is, its first `left` elements (the others zero).
template <int DT>
__device__ __forceinline__ u32x4 load_raw(const typename Elem<DT>::T *p, int left)
{
    u32x4 r = u32x4{0u, 0u, 0u, 0u};
    if (left >= Elem<DT>::V) {
        __builtin_memcpy(&r, p, 16);
    } else {
        for (int i = 0; i < Elem<DT>::V - 1; i++) {
            if (i < left) {
                if constexpr (DT == OUT_F32)
                    r[i] = __float_as_uint(p[i]);
                else
                    r[i / 2] |= (uint32_t)((const uint16_t *)p)[i] << (16 * (i & 1));
            }
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ float elem_of(u32x4 r, int i)
{
    if constexpr (DT == OUT_F32)
        return __uint_as_float(r[i]);
    else
        return __uint_as_float(i & 1 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
}

template <int DT>
__device__ __forceinline__ void store_raw(typename Elem<DT>::T *p, int left, u32x4 r)
{
    if (left >= Elem<DT>::V) {
        __builtin_memcpy(p, &r, 16);
    } else {
        for (int i = 0; i < Elem<DT>::V - 1; i++) {
            if (i < left) {
                if constexpr (DT == OUT_F32)
                    p[i] = __uint_as_float(r[i]);
                else
                    ((uint16_t *)p)[i] = (uint16_t)(r[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ u32x4 pack_vec(const float *v)
{
    typename Elem<DT>::T e[Elem<DT>::V];
#pragma unroll
    for (int i = 0; i < Elem<DT>::V; i++)
        e[i] = (typename Elem<DT>::T)v[i];
    u32x4 r;
    __builtin_memcpy(&r, e, 16);
    return r;
}

// The row a choice names: -1 for a dropped one; one past the rows is reported
// and treated as dropped.
__device__ __forceinline__ int row_of(const MoveArgs &a, int64_t f)
{
    const int p = a.pos[f];
    if (p >= a.R) {
        __hip_atomic_fetch_or(a.status, DEV_BAD_ROUTE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return -1;
    }
    return p < 0 ? -1 : p;
}

// dispatch: xs[pos[t][j]] = x[t].  One load, topk stores; lane j reads choice j.
template <int DT>
__global__ __launch_bounds__(256) void dispatch_kernel(MoveArgs a, int chunks)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V;
    const int lane = threadIdx.x & 63;
    const int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = u / chunks;
    if (t >= a.T)
        return;
    const int64_t h = (u % chunks * 64 + lane) * V;
    const int left = (int)min((int64_t)V, a.H - h);
    const int mine = lane < a.topk ? row_of(a, t * a.topk + lane) : -1;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (left > 0)
        v = load_raw<DT>((const E *)a.src + t * a.H + h, left);
    for (int j = 0; j < a.topk; j++) {
        const int p = __builtin_amdgcn_readlane(mine, j);
        if (p >= 0 && left > 0)
            store_raw<DT>((E *)a.dst + (int64_t)p * a.H + h, left, v);
    }
}

// combine: y[t] = sum_j w[t][j] ys[pos[t][j]], j in order, fp32, one rounding.
// Eight choices' loads in flight; lane j reads choice j and its weight.
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(MoveArgs a, int chunks)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V, G = 8;
    const int lane = threadIdx.x & 63;
    const int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = u / chunks;
    if (t >= a.T)
        return;
    const int64_t h = (u % chunks * 64 + lane) * V;
    const int left = (int)min((int64_t)V, a.H - h);
    const int64_t f = t * a.topk + lane;
    const int mine = lane < a.topk ? row_of(a, f) : -1;
    const float wl = a.weights && lane < a.topk ? a.weights[f] : 1.f;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        sum[i] = 0.f;
    for (int j0 = 0; j0 < a.topk; j0 += G) {
        u32x4 v[G];
        int p[G];
#pragma unroll
        for (int g = 0; g < G; g++) {
            p[g] = j0 + g < a.topk ? __builtin_amdgcn_readlane(mine, j0 + g) : -1;
            if (p[g] >= 0 && left > 0)
                v[g] = load_raw<DT>((const E *)a.src + (int64_t)p[g] * a.H + h, left);
        }
#pragma unroll
        for (int g = 0; g < G; g++)
            if (p[g] >= 0) {
                const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), (j0 + g) & 63));
#pragma unroll
                for (int i = 0; i < V; i++)
                    sum[i] = fmaf(w, elem_of<DT>(v[g], i), sum[i]);
            }
    }
    if (left > 0)
        store_raw<DT>((E *)a.dst + t * a.H + h, left, pack_vec<DT>(sum));
}

// combine_grad, one wave a choice: dys[p] = w dy[t], dw = sum_h dy[t][h] ys[p][h].
// Two vectors of both rows in flight; neighbouring waves share dy in L1.
template <int DT>
__global__ __launch_bounds__(256) void combine_grad_kernel(MoveArgs a)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V, G = 2;
    const int64_t f = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (f >= a.T * a.topk)
        return;
    const int64_t t = f / a.topk;
    const int64_t p = __builtin_amdgcn_readfirstlane(row_of(a, f));
    float dot = 0.f;
    if (p >= 0) {
        const float w = a.weights[f];
        const E *dy = (const E *)a.src + t * a.H;
        const E *ys = (const E *)a.src2 + p * a.H;
        E *dys = (E *)a.dst + p * a.H;
        for (int64_t h0 = lane * V; h0 < a.H; h0 += 64 * V * G) {
            u32x4 g[G], y[G];
            int left[G];
#pragma unroll
            for (int k = 0; k < G; k++) {
                const int64_t h = h0 + 64 * V * k;
                left[k] = (int)min((int64_t)V, a.H - h);
                if (left[k] > 0) {
                    g[k] = load_raw<DT>(dy + h, left[k]);
                    y[k] = load_raw<DT>(ys + h, left[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < G; k++) {
                if (left[k] > 0) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        const float d = elem_of<DT>(g[k], i);
                        if (i < left[k])
                            dot = fmaf(d, elem_of<DT>(y[k], i), dot);
                        o[i] = w * d;
                    }
                    store_raw<DT>(dys + h0 + 64 * V * k, left[k], pack_vec<DT>(o));
                }
            }
        }
    }
    for (int d = 32; d; d >>= 1)
        dot += __shfl_xor(dot, d);
    if (lane == 0)
        a.dw[f] = dot;
}

template <int DT, typename K>
static void go_by_vectors(K kernel, const MoveArgs &a, hipStream_t st)
{
    const int64_t per = 64 * Elem<DT>::V, chunks = (a.H + per - 1) / per;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T * chunks + 3) / 4)), dim3(256), 0, st, a, (int)chunks);
}

hipError_t launch_dispatch(int dt, const MoveArgs &a, hipStream_t st)
{
    if (dt == OUT_F32)
        go_by_vectors<OUT_F32>(dispatch_kernel<OUT_F32>, a, st);
    else
        go_by_vectors<OUT_BF16>(dispatch_kernel<OUT_BF16>, a, st);
    return hipGetLastError();
}

hipError_t launch_combine(int dt, const MoveArgs &a, hipStream_t st)
{
    if (dt == OUT_F32)
        go_by_vectors<OUT_F32>(combine_kernel<OUT_F32>, a, st);
    else
        go_by_vectors<OUT_BF16>(combine_kernel<OUT_BF16>, a, st);
    return hipGetLastError();
}

hipError_t launch_combine_grad(int dt, const MoveArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.T * a.topk + 3) / 4));
    if (dt == OUT_F32)
        hipLaunchKernelGGL(combine_grad_kernel<OUT_F32>, grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(combine_grad_kernel<OUT_BF16>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace qg
