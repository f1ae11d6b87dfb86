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
    for (int f = tid; f < a.n; f += RT_THREADS) {
        const int e = a.ids[f];
        if (e >= 0 && e < a.E) {
            atomicAdd(&tot[e], 1);
            if (f < lo)
                atomicAdd(&mine[e], 1);
        }
    }
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
        for (int w = 0; w < RT_WAVES; w++) {  // waves in order
            if (w == wid && first)
                base = atomicAdd(&mine[id], __popcll(same));
            __syncthreads();
        }
        base = __shfl(base, __ffsll(same) - 1);
        if (f < hi)
            a.pos[f] = kept ? base + rank : -1;
    }
}

hipError_t launch_route(const RouteArgs &a, hipStream_t st)
{
    int bits = 0;
    while (bits < 31 && (1 << bits) < a.E)
        bits++;
    const int runs = a.n < 64 * RT_THREADS ? (a.n + RT_THREADS - 1) / RT_THREADS : 64;
    const int wgs = runs < 1 ? 1 : runs;
    const int run = (a.n + wgs - 1) / wgs;
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
// single elements.
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

template <int DT>
__device__ __forceinline__ void load_vec(const typename Elem<DT>::T *p, int left, float *v)
{
    constexpr int V = Elem<DT>::V;
    typename Elem<DT>::T e[V];
    if (left >= V) {
        __builtin_memcpy(e, p, 16);
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = (float)e[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = i < left ? (float)p[i] : 0.f;
    }
}

template <int DT>
__device__ __forceinline__ void store_vec(typename Elem<DT>::T *p, int left, const float *v)
{
    constexpr int V = Elem<DT>::V;
    typename Elem<DT>::T e[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        e[i] = (typename Elem<DT>::T)v[i];
    if (left >= V) {
        __builtin_memcpy(p, e, 16);
    } else {
        for (int i = 0; i < V; i++)
            if (i < left)
                p[i] = e[i];
    }
}

// The row a choice names: -1 for a dropped one; one past the rows is reported
// and treated as dropped.
__device__ __forceinline__ int64_t row_of(const MoveArgs &a, int64_t f)
{
    const int p = a.pos[f];
    if (p < 0)
        return -1;
    if (p >= a.R) {
        __hip_atomic_fetch_or(a.status, DEV_BAD_ROUTE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return -1;
    }
    return p;
}

// dispatch: xs[pos[t][j]] = x[t].  A wave owns 64 vectors of one token's row:
// one load, topk stores.
template <int DT>
__global__ __launch_bounds__(64) void dispatch_kernel(MoveArgs a)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V;
    const int64_t t = blockIdx.x;
    const int64_t h = ((int64_t)blockIdx.y * 64 + threadIdx.x) * V;
    const int left = (int)min((int64_t)V, a.H - h);
    float v[V];
    if (left > 0)
        load_vec<DT>((const E *)a.src + t * a.H + h, left, v);
    for (int j = 0; j < a.topk; j++) {
        const int64_t p = row_of(a, t * a.topk + j);
        if (p >= 0 && left > 0)
            store_vec<DT>((E *)a.dst + p * a.H + h, left, v);
    }
}

// combine: y[t] = sum_j w[t][j] ys[pos[t][j]], j in order, fp32, one rounding.
template <int DT>
__global__ __launch_bounds__(64) void combine_kernel(MoveArgs a)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V;
    const int64_t t = blockIdx.x;
    const int64_t h = ((int64_t)blockIdx.y * 64 + threadIdx.x) * V;
    const int left = (int)min((int64_t)V, a.H - h);
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; i++)
        sum[i] = 0.f;
    for (int j = 0; j < a.topk; j++) {
        const int64_t p = row_of(a, t * a.topk + j);
        if (p >= 0 && left > 0) {
            const float w = a.weights ? a.weights[t * a.topk + j] : 1.f;
            float v[V];
            load_vec<DT>((const E *)a.src + p * a.H + h, left, v);
#pragma unroll
            for (int i = 0; i < V; i++)
                sum[i] = fmaf(w, v[i], sum[i]);
        }
    }
    if (left > 0)
        store_vec<DT>((E *)a.dst + t * a.H + h, left, sum);
}

// combine_grad, one wave a choice: dys[p] = w dy[t], dw = sum_h dy[t][h] ys[p][h].
template <int DT>
__global__ __launch_bounds__(256) void combine_grad_kernel(MoveArgs a)
{
    typedef typename Elem<DT>::T E;
    constexpr int V = Elem<DT>::V;
    const int64_t f = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (f >= a.T * a.topk)
        return;
    const int64_t t = f / a.topk;
    const int64_t p = row_of(a, f);
    float dot = 0.f;
    if (p >= 0) {
        const float w = a.weights[f];
        const E *dy = (const E *)a.src + t * a.H;
        const E *ys = (const E *)a.src2 + p * a.H;
        E *dys = (E *)a.dst + p * a.H;
        for (int64_t h = lane * V; h < a.H; h += 64 * V) {
            const int left = (int)min((int64_t)V, a.H - h);
            float g[V], y[V];
            load_vec<DT>(dy + h, left, g);
            load_vec<DT>(ys + h, left, y);
#pragma unroll
            for (int i = 0; i < V; i++) {
                if (i < left)
                    dot = fmaf(g[i], y[i], dot);
                g[i] *= w;
            }
            store_vec<DT>(dys + h, left, g);
        }
    }
    for (int d = 32; d; d >>= 1)
        dot += __shfl_xor(dot, d);
    if (lane == 0)
        a.dw[f] = dot;
}

template <int DT>
static dim3 vec_grid(const MoveArgs &a)
{
    const int64_t per = 64 * Elem<DT>::V;
    return dim3((unsigned)a.T, (unsigned)((a.H + per - 1) / per));
}

hipError_t launch_dispatch(int dt, const MoveArgs &a, hipStream_t st)
{
    if (dt == OUT_F32)
        hipLaunchKernelGGL(dispatch_kernel<OUT_F32>, vec_grid<OUT_F32>(a), dim3(64), 0, st, a);
    else
        hipLaunchKernelGGL(dispatch_kernel<OUT_BF16>, vec_grid<OUT_BF16>(a), dim3(64), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_combine(int dt, const MoveArgs &a, hipStream_t st)
{
    if (dt == OUT_F32)
        hipLaunchKernelGGL(combine_kernel<OUT_F32>, vec_grid<OUT_F32>(a), dim3(64), 0, st, a);
    else
        hipLaunchKernelGGL(combine_kernel<OUT_BF16>, vec_grid<OUT_BF16>(a), dim3(64), 0, st, a);
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
