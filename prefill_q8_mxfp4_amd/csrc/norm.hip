// The norm in front of a projection, with the residual's addition, and its
// gradients.
//
//   h = rt(x + residual),  r = (mean_k h_k^2 + eps)^(-1/2),  y = dt(h r w)
//
// or the rows h r w as 8-bit codes.  r is common to a row, so it has no part in
// its codes: they are those of u = fp32(h w) as quantize_rows makes them, and
// the scale is u's times r.  The codes' bits then do not depend on the order
// of the sum in r.
//
// The norm of h as it is stored (rounded to the residual's type), not of the
// unrounded sum: it is what the next layer adds to and what the gradient reads.
#include "int8_quant.h"
#include "layer.h"

namespace qg {

constexpr int NV_E = RQ_V;  // elements of a thread's vector

// How a row of H elements lies: whole vectors of eight; or ragged, its rows at any
// alignment; or shorter than a vector.
enum { ROW_WHOLE, ROW_RAGGED, ROW_TINY };

// Ragged rows: a vector past the last whole one is loaded from the row's last eight
// elements, like any other without a branch (a branch around loads makes each wait
// for itself: 2048 rows of 5119 in bf16 took 33.0 us, gradients 66.4), and moved down
// by the elements that belong to the vector before; zeros behind the row.
__device__ __forceinline__ void move_down(float *v, int d)
{
    // by masks: of selections the compiler makes places that the lane computes
#pragma unroll
    for (int step = 4; step; step >>= 1) {
        const uint32_t m = (d & step) ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < NV_E; i++) {
            const uint32_t next = i + step < NV_E ? __float_as_uint(v[i + step < NV_E ? i + step : i]) : 0u;
            v[i] = __uint_as_float((next & m) | (__float_as_uint(v[i]) & ~m));
        }
    }
    const uint32_t in = d >= NV_E ? 0u : 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < NV_E; i++)
        v[i] = __uint_as_float(__float_as_uint(v[i]) & in);
}

// The first element of a ragged vector, and how far it has to move; vectors of whole
// waves inside the row do not (uniform).
__device__ __forceinline__ int64_t ragged_at(int64_t k, int64_t H) { return k < H - NV_E ? k : H - NV_E; }
__device__ __forceinline__ bool ragged_wave(int64_t k, int64_t H)
{
    return __builtin_amdgcn_readfirstlane((int)k) + 64 * NV_E > H;
}

template <int T>
__device__ __forceinline__ void raw_load(Raw8<T> &r, const void *base, int64_t at)
{
    __builtin_memcpy(&r, (const uint8_t *)base + at * Raw8<T>::ESZ, sizeof r);
}

// Eight elements of a row, zeros behind it; nothing looks at them before floats().
template <int T, int M>
struct Vec {
    Raw8<T> raw;
    float v[M == ROW_TINY ? NV_E : 1];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, const void *base, int64_t row, int64_t k, int64_t H)
    {
        if constexpr (M == ROW_WHOLE)
            raw.load(rs, (int)k * Raw8<T>::ESZ);  // the resource ends with the row
        else if constexpr (M == ROW_RAGGED)
            raw_load<T>(raw, base, row * H + ragged_at(k, H));
        else
            load8<T>(base, row * H + k, H - k, v);
    }
    __device__ __forceinline__ void floats(float *o, int64_t k, int64_t H) const
    {
        if constexpr (M == ROW_TINY) {
#pragma unroll
            for (int i = 0; i < NV_E; i++)
                o[i] = v[i];
        } else {
            raw.floats(o);
            if (M == ROW_RAGGED && ragged_wave(k, H))
                move_down(o, (int)(k - ragged_at(k, H)));
        }
    }
    // What floats() gave is made again when it is next asked for, not kept in twice as
    // many registers.
    __device__ __forceinline__ void keep()
    {
        if constexpr (M != ROW_TINY && T == ACT_BF16)
            asm volatile("" : "+v"(raw.r[0]));
    }
};

template <int T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void *base, int64_t row, int64_t H)
{
    return make_rsrc((const uint8_t *)base + row * H * Raw8<T>::ESZ, base ? H * Raw8<T>::ESZ : 0);
}

// Ragged rows' vectors behind the row are not stored, a part of one by elements.
template <int T, int M>
__device__ __forceinline__ void store8(void *base, int64_t at, int64_t left, const float *v)
{
    if (M == ROW_WHOLE || left >= NV_E) {
        if constexpr (T == ACT_F32) {
            __builtin_memcpy((float *)base + at, v, 32);
        } else {
            __bf16 h[NV_E];
#pragma unroll
            for (int i = 0; i < NV_E; i++)
                h[i] = (__bf16)v[i];
            __builtin_memcpy((__bf16 *)base + at, h, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV_E - 1; i++)
            if (i < left)
                store_out<T == ACT_F32 ? OUT_F32 : OUT_BF16>(base, at + i, v[i]);
    }
}

// Eight elements of the weight (zeros behind it), ones where there is none.
template <int T, int M>
__device__ __forceinline__ void weight_of(const void *w, int64_t k, int64_t H, float *o)
{
    Vec<T, M> v;
    v.load(make_rsrc(w, H * Raw8<T>::ESZ), w, 0, k, H);
    v.floats(o, k, H);
}

template <int M>
__device__ __forceinline__ void weight8(const void *w, int wt, int64_t k, int64_t H, float *o)
{
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < NV_E; i++)
            o[i] = 1.f;
    } else if (wt == QGEMM_F32) {
        weight_of<ACT_F32, M>(w, k, H, o);
    } else {
        weight_of<ACT_BF16, M>(w, k, H, o);
    }
}

// The value as it is held in type T.
template <int T>
__device__ __forceinline__ float held(float v)
{
    return T == ACT_F32 ? v : (float)(__bf16)v;
}

// TPR threads a row, which stays in NV vectors of registers a thread as far as it
// fits; the rest is read again for the output.  A workgroup takes every G-th row (four
// neighbours with 64 threads a row), the next one's loads on their way while the
// present one is reduced and written, so that reads and writes of memory overlap.
template <int DT, int RT, bool CODES, int TPR, int NV, int M>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_norm_kernel(NormArgs a)
{
    constexpr int RPW = TPR > 256 ? 1 : 256 / TPR;
    const int tid = threadIdx.x % TPR;
    int64_t row = (int64_t)blockIdx.x * RPW + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    if (row >= a.B)
        return;  // whole waves, and whole workgroups where there is a barrier
    Vec<DT, M> x[NV];
    Vec<RT, M> res[NV];
    auto fetch = [&](int64_t row) {
        const __amdgpu_buffer_rsrc_t xr = row_rsrc<DT>(a.x, row, a.H), rr = row_rsrc<RT>(a.res, row, a.H);
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            x[j].load(xr, a.x, row, k, a.H);
            if (a.res)
                res[j].load(rr, a.res, row, k, a.H);
        }
    };
    fetch(row);
    float w[NV][NV_E];
#pragma unroll
    for (int j = 0; j < NV; j++)
        weight8<M>(a.w, a.wt, ((int64_t)j * TPR + tid) * NV_E, a.H, w[j]);
    for (int turn = 0; row < a.B; turn ^= 1) {
        const int64_t base = row * a.H;
        float v[NV][NV_E];
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            x[j].floats(v[j], k, a.H);
            if (a.res) {
                float o[NV_E];
                res[j].floats(o, k, a.H);
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    v[j][i] = held<RT>(v[j][i] + o[i]);
            }
        }
        const int64_t next = row + (int64_t)gridDim.x * RPW;
        if (next < a.B)
            fetch(next);
        // past the registers: h to memory (or x as it is), to be read again
        auto far = [&](int64_t k, float *o) {
            load8<DT>(a.x, base + k, a.H - k, o);
            if (a.res) {
                float r[NV_E];
                load8<RT>(a.res, base + k, a.H - k, r);
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    o[i] = held<RT>(o[i] + r[i]);
            }
        };
        auto far_again = [&](int64_t k, float *o) {
            if (a.h)  // the residual may have been its place
                load8<RT>(a.h, base + k, a.H - k, o);
            else
                far(k, o);
        };
        float sum = 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
#pragma unroll
            for (int i = 0; i < NV_E; i++)
                sum = fmaf(v[j][i], v[j][i], sum);
            if (a.h && k < a.H)
                store8<RT, M>(a.h, base + k, a.H - k, v[j]);
            if constexpr (CODES) {
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    v[j][i] *= w[j][i];  // zeros behind the row
                top = top8(v[j], top);
            }
        }
        for (int64_t k = ((int64_t)NV * TPR + tid) * NV_E; k < a.H; k += TPR * NV_E) {
            float o[NV_E];
            far(k, o);
#pragma unroll
            for (int i = 0; i < NV_E; i++)
                sum = fmaf(o[i], o[i], sum);
            if (a.h)
                store8<RT, M>(a.h, base + k, a.H - k, o);
            if constexpr (CODES) {
                float g[NV_E];
                weight8<M>(a.w, a.wt, k, a.H, g);
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    o[i] *= g[i];
                top = top8(o, top);
            }
        }
        sum = wave_total(sum);
        if constexpr (CODES)
            top = wave_top(top);
        if constexpr (TPR > 64) {
            __shared__ float sums[2][TPR / 64];
            __shared__ uint32_t tops[2][TPR / 64];
            if ((threadIdx.x & 63) == 0) {
                sums[turn][threadIdx.x >> 6] = sum;
                if constexpr (CODES)
                    tops[turn][threadIdx.x >> 6] = top;
            }
            __syncthreads();  // the other half is the next row's
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; i++) {
                sum += sums[turn][i];
                if constexpr (CODES)
                    top = max(top, tops[turn][i]);
            }
        }
        const float r = 1.f / __builtin_sqrtf(sum / (float)a.H + a.eps);

        if constexpr (CODES) {
            const RowScale sc(top);
            if (tid == 0)
                a.scales[row] = sc.s * r;
            int8_t *to = a.codes + row * a.ldc;
#pragma unroll
            for (int j = 0; j < NV; j++) {
                const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
                if (k < a.ldc)
                    *(u32x2 *)(to + k) = sc.codes(v[j]);
            }
            for (int64_t k = ((int64_t)NV * TPR + tid) * NV_E; k < a.ldc; k += TPR * NV_E) {
                float o[NV_E];
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    o[i] = 0.f;
                if (k < a.H) {
                    float g[NV_E];
                    far_again(k, o);
                    weight8<M>(a.w, a.wt, k, a.H, g);
#pragma unroll
                    for (int i = 0; i < NV_E; i++)
                        o[i] *= g[i];
                }
                *(u32x2 *)(to + k) = sc.codes(o);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; j++) {
                const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
                if (k < a.H) {
                    float o[NV_E];
#pragma unroll
                    for (int i = 0; i < NV_E; i++)
                        o[i] = v[j][i] * r * w[j][i];
                    store8<DT, M>(a.y, base + k, a.H - k, o);
                }
            }
            for (int64_t k = ((int64_t)NV * TPR + tid) * NV_E; k < a.H; k += TPR * NV_E) {
                float o[NV_E], g[NV_E];
                far_again(k, o);
                weight8<M>(a.w, a.wt, k, a.H, g);
#pragma unroll
                for (int i = 0; i < NV_E; i++)
                    o[i] = o[i] * r * g[i];
                store8<DT, M>(a.y, base + k, a.H - k, o);
            }
        }
        row = next;
    }
}

template <int DT, int RT, bool CODES, int TPR, int NV>
static void norm_go(const NormArgs &a, hipStream_t st)
{
    constexpr int RPW = TPR > 256 ? 1 : 256 / TPR;
    const int64_t rows = (a.B + RPW - 1) / RPW;
    // 16 waves of the chip's CUs each, or one workgroup of 16 waves (2048 rows of 5120,
    // bf16 with a residual: 16.4 us with 256 workgroups, 14.2 with 1024, 16.5 with a
    // workgroup a row; 600 rows of 17408: 15.9 with 256, 20.1 with 600)
    const int64_t most = TPR > 256 ? 256 : 1024;
    const dim3 g((unsigned)(rows < most ? rows : most)), blk(TPR > 256 ? TPR : 256);
    if (a.H % NV_E == 0)
        hipLaunchKernelGGL((rms_norm_kernel<DT, RT, CODES, TPR, NV, ROW_WHOLE>), g, blk, 0, st, a);
    else if (TPR > 64 || a.H > NV_E)
        hipLaunchKernelGGL((rms_norm_kernel<DT, RT, CODES, TPR, NV, ROW_RAGGED>), g, blk, 0, st, a);
    else
        hipLaunchKernelGGL((rms_norm_kernel<DT, RT, CODES, TPR, NV, TPR == 64 ? ROW_TINY : ROW_RAGGED>), g, blk, 0, st, a);
}

// Rows of 8193 and more: three vectors a thread are more than 128 registers hold beside
// the next row's unless both types are bf16; 40 to 116 bytes a lane go to scratch there,
// 12 of ragged bf16 rows (600 x 17408 with a residual: bf16 15.8 us, bf16 with fp32 35.5,
// fp32 44.6, its codes 51.6, where their bytes take 16.4, 24.7, 32.9 and 26.7; 17407 fp32
// 58.5).  Rows up to 1024 take a wave whatever their length, so short ones leave lanes
// idle (81920 x 128 bf16 without a residual: 23.7 us, its bytes 8.3).
template <int DT, int RT, bool CODES>
static void norm_shape(const NormArgs &a, hipStream_t st)
{
    if (a.H <= 64 * NV_E * 2)
        norm_go<DT, RT, CODES, 64, 2>(a, st);
    else if (a.H <= 256 * NV_E)
        norm_go<DT, RT, CODES, 256, 1>(a, st);
    else if (a.H <= 256 * NV_E * 3 && a.B > 256)
        norm_go<DT, RT, CODES, 256, 3>(a, st);
    else if (a.H <= 1024 * NV_E)
        norm_go<DT, RT, CODES, 1024, 1>(a, st);
    else
        norm_go<DT, RT, CODES, 1024, 3>(a, st);
}

hipError_t launch_rms_norm(int dt, int rt, const NormArgs &a, hipStream_t st)
{
#define QG_NORM(D, R) \
    (a.codes ? norm_shape<D, R, true>(a, st) : norm_shape<D, R, false>(a, st))
    if (dt == QGEMM_F32)
        rt == QGEMM_F32 ? QG_NORM(ACT_F32, ACT_F32) : QG_NORM(ACT_F32, ACT_BF16);
    else
        rt == QGEMM_F32 ? QG_NORM(ACT_BF16, ACT_F32) : QG_NORM(ACT_BF16, ACT_BF16);
#undef QG_NORM
    return hipGetLastError();
}

// ---------------------------------------------------------------- gradients
// With c1 = sum_k h_k^2 and c2 = sum_k dy_k w_k h_k:
//   dx_k = r dy_k w_k - (h_k r) (r (r c2 / H)) + dh_k,   dw_k = sum_b dy_k h_k r.
// In this order every factor is of the size of h r or of dy: r^3 leaves fp32's normal
// range for rows of 10^13 and larger (a row of 10^15 lost half of its second term) and
// of 10^-13 and smaller.
// r comes from h again, which is read anyway.  A workgroup takes every G-th row
// and keeps its sums of dw in registers; the G partial rows are added, in order,
// by a second launch.
// Workgroups: a row of them in flight for every CU, more of short rows, as long as
// their partial rows of dw are few bytes beside the rows (2048 rows of 5120 in bf16,
// both launches: 22.7 us with 256, 25.8 with 512, 34.7 with 1024; 8192 rows of 1024: 35.8,
// 25.8, 21.8).  Always 256 threads and a barrier a row: short rows leave most idle
// (81920 x 128 in bf16: 139 us, its bytes 12).
static int norm_grad_groups(int64_t B, int64_t H)
{
    // at least two rows each, where there are enough of them
    int64_t most = H < 1280 ? 1024 : H < 5120 ? 1310720 / H : 256;
    most = B / 2 < most ? B / 2 : most;
    most = most < 256 ? 256 : most;
    return (int)(B < most ? B : most);
}

template <int DT, int RT, int TPR, int NV, int M>
__global__ __launch_bounds__(TPR) void rms_norm_grad_kernel(NormGradArgs a)
{
    // the next row's loads on their way during this one's work, and the weight kept in
    // registers: where they have room for it
    constexpr bool AHEAD = NV <= 3;
    const int tid = threadIdx.x;
    __shared__ float s1[2][TPR / 64], s2[2][TPR / 64];
    // a row's vectors as they are in memory
    struct Rows {
        Vec<DT, M> g[NV];
        Vec<RT, M> h[NV], e[NV];
    };
    auto fetch = [&](Rows &r, int64_t row) {
        const __amdgpu_buffer_rsrc_t gr = row_rsrc<DT>(a.dy, row, a.H), hr = row_rsrc<RT>(a.h, row, a.H),
                                     er = row_rsrc<RT>(a.dh, row, a.H);
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            r.g[j].load(gr, a.dy, row, k, a.H);
            r.h[j].load(hr, a.h, row, k, a.H);
            if (a.dh)
                r.e[j].load(er, a.dh, row, k, a.H);
        }
    };
    Rows now;
    int64_t row = blockIdx.x;
    fetch(now, row);
    float acc[NV][NV_E], w[AHEAD ? NV : 1][NV_E];
#pragma unroll
    for (int j = 0; j < NV; j++) {
        if constexpr (AHEAD)
            weight8<M>(a.w, a.wt, ((int64_t)j * TPR + tid) * NV_E, a.H, w[j]);
#pragma unroll
        for (int i = 0; i < NV_E; i++)
            acc[j][i] = 0.f;
    }
    for (int turn = 0; row < a.B; turn ^= 1) {
        const int64_t base = row * a.H, next = row + gridDim.x;
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            float gv[NV_E], hv[NV_E], *wv = w[AHEAD ? j : 0];
            if constexpr (!AHEAD)
                weight8<M>(a.w, a.wt, k, a.H, wv);
            now.g[j].floats(gv, k, a.H);
            now.h[j].floats(hv, k, a.H);
#pragma unroll
            for (int i = 0; i < NV_E; i++) {
                c1 = fmaf(hv[i], hv[i], c1);
                c2 = fmaf(gv[i] * wv[i], hv[i], c2);
            }
            now.g[j].keep();
            now.h[j].keep();
        }
        Rows coming;
        if (AHEAD && next < a.B)
            fetch(coming, next);
        for (int64_t k = ((int64_t)NV * TPR + tid) * NV_E; k < a.H; k += TPR * NV_E) {
            float gv[NV_E], hv[NV_E], wv[NV_E];
            load8<DT>(a.dy, base + k, a.H - k, gv);
            load8<RT>(a.h, base + k, a.H - k, hv);
            weight8<M>(a.w, a.wt, k, a.H, wv);
#pragma unroll
            for (int i = 0; i < NV_E; i++) {
                c1 = fmaf(hv[i], hv[i], c1);
                c2 = fmaf(gv[i] * wv[i], hv[i], c2);
            }
        }
        c1 = wave_total(c1);
        c2 = wave_total(c2);
        if ((tid & 63) == 0) {
            s1[turn][tid >> 6] = c1;
            s2[turn][tid >> 6] = c2;
        }
        __syncthreads();  // the other half of s1, s2 is the next row's
        c1 = c2 = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; i++) {
            c1 += s1[turn][i];
            c2 += s2[turn][i];
        }
        const float r = 1.f / __builtin_sqrtf(c1 / (float)a.H + a.eps);
        const float t = r * (r * (c2 / (float)a.H));
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            float gv[NV_E], hv[NV_E], ev[NV_E], o[NV_E], *wv = w[AHEAD ? j : 0];
            if constexpr (!AHEAD)
                weight8<M>(a.w, a.wt, k, a.H, wv);
            now.g[j].floats(gv, k, a.H);
            now.h[j].floats(hv, k, a.H);
            if (a.dh)
                now.e[j].floats(ev, k, a.H);
#pragma unroll
            for (int i = 0; i < NV_E; i++) {
                const float n = hv[i] * r;
                o[i] = r * (gv[i] * wv[i]) - n * t + (a.dh ? ev[i] : 0.f);
                acc[j][i] = fmaf(gv[i], n, acc[j][i]);
            }
            if (k < a.H) {
                if (a.dx)
                    store8<DT, M>(a.dx, base + k, a.H - k, o);
                if (a.dr)
                    store8<RT, M>(a.dr, base + k, a.H - k, o);
            }
        }
        for (int64_t k = ((int64_t)NV * TPR + tid) * NV_E; k < a.H; k += TPR * NV_E) {
            float gv[NV_E], hv[NV_E], wv[NV_E], o[NV_E], ev[NV_E];
            load8<DT>(a.dy, base + k, a.H - k, gv);
            load8<RT>(a.h, base + k, a.H - k, hv);
            if (a.dh)
                load8<RT>(a.dh, base + k, a.H - k, ev);
            weight8<M>(a.w, a.wt, k, a.H, wv);
            float p[NV_E];  // dw so far: this thread's own place
            const bool first = row == blockIdx.x;
            if (a.part && !first)
                load8<ACT_F32>(a.part, blockIdx.x * a.pitch + k, a.H - k, p);
#pragma unroll
            for (int i = 0; i < NV_E; i++) {
                const float n = hv[i] * r;
                o[i] = r * (gv[i] * wv[i]) - n * t + (a.dh ? ev[i] : 0.f);
                p[i] = fmaf(gv[i], n, first ? 0.f : p[i]);
            }
            if (a.part)
                store8<ACT_F32, M>(a.part, blockIdx.x * a.pitch + k, a.H - k, p);
            if (a.dx)
                store8<DT, M>(a.dx, base + k, a.H - k, o);
            if (a.dr)
                store8<RT, M>(a.dr, base + k, a.H - k, o);
        }
        if constexpr (AHEAD)
            now = coming;
        else if (next < a.B)
            fetch(now, next);
        row = next;
    }
    if (a.part) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * NV_E;
            if (k < a.H)
                store8<ACT_F32, M>(a.part, blockIdx.x * a.pitch + k, a.H - k, acc[j]);
        }
    }
}

// dw = the sum of G partial rows: sixteen columns a workgroup, four a lane, 64
// threads down the rows with all their loads in flight (512 rows of 5120: 64
// columns a workgroup and 16 threads down the rows took 8.2 us, this 5.3).
__global__ __launch_bounds__(256) void norm_dw_kernel(const float *part, float *dw, int G, int64_t H, int64_t pitch)
{
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const float *p = part + (int64_t)blockIdx.x * 16 + (lane & 3) * 4;
    __shared__ f32x4 sh[4][4];
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int g = threadIdx.x >> 2; g < G; g += 64)
        s += *(const f32x4 *)(p + g * pitch);
#pragma unroll
    for (int i = 0; i < 4; i++)
        for (int d = 4; d < 64; d <<= 1)
            s[i] += __shfl_xor(s[i], d);
    if (lane < 4)
        sh[wid][lane] = s;
    __syncthreads();
    const int64_t k = (int64_t)blockIdx.x * 16 + threadIdx.x;
    if (threadIdx.x < 16 && k < H) {
        const int c = threadIdx.x >> 2, i = threadIdx.x & 3;
        dw[k] = sh[0][c][i] + sh[1][c][i] + sh[2][c][i] + sh[3][c][i];
    }
}

// Floats from one partial row of dw to the next: whole vectors.
static int64_t dw_pitch(int64_t H) { return (H + 15) / 16 * 16; }

int64_t norm_grad_bytes(int64_t B, int64_t H) { return norm_grad_groups(B, H) * dw_pitch(H) * 4; }


template <int DT, int RT, int TPR, int NV>
static void grad_go(const NormGradArgs &a, int G, hipStream_t st)
{
    constexpr bool SHORT = TPR == 256 && NV == 1;
    if (a.H % NV_E == 0)
        hipLaunchKernelGGL((rms_norm_grad_kernel<DT, RT, TPR, NV, ROW_WHOLE>), dim3(G), dim3(TPR), 0, st, a);
    else if (!SHORT || a.H > NV_E)
        hipLaunchKernelGGL((rms_norm_grad_kernel<DT, RT, TPR, NV, ROW_RAGGED>), dim3(G), dim3(TPR), 0, st, a);
    else
        hipLaunchKernelGGL((rms_norm_grad_kernel<DT, RT, TPR, NV, SHORT ? ROW_TINY : ROW_RAGGED>), dim3(G), dim3(TPR), 0,
                           st, a);
}

template <int DT, int RT>
static void grad_shape(const NormGradArgs &a, int G, hipStream_t st)
{
    if (a.H <= 256 * NV_E)
        grad_go<DT, RT, 256, 1>(a, G, st);
    else if (a.H <= 256 * NV_E * 3)
        grad_go<DT, RT, 256, 3>(a, G, st);
    else if constexpr (DT == ACT_BF16 && RT == ACT_BF16)
        grad_go<DT, RT, 512, 5>(a, G, st);
    else  // what five vectors of fp32 take, registers do not have
        grad_go<DT, RT, 512, 4>(a, G, st);
    // (ragged rows of more than 6144 do not fit either: 140 to 440 bytes a lane go to scratch;
    // 512 x 17407: bf16 36.8 us, fp32 71.0, where 17408 take 25.7 and 39.0)
}

hipError_t launch_rms_norm_grad(int dt, int rt, NormGradArgs a, hipStream_t st)
{
    a.pitch = dw_pitch(a.H);
    const int G = norm_grad_groups(a.B, a.H);
    if (G == 0)
        ;  // no rows: dw is zeros
    else if (dt == QGEMM_F32)
        rt == QGEMM_F32 ? grad_shape<ACT_F32, ACT_F32>(a, G, st) : grad_shape<ACT_F32, ACT_BF16>(a, G, st);
    else
        rt == QGEMM_F32 ? grad_shape<ACT_BF16, ACT_F32>(a, G, st) : grad_shape<ACT_BF16, ACT_BF16>(a, G, st);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.dw) {
        hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((a.H + 15) / 16)), dim3(256), 0, st, a.part, a.dw, G, a.H,
                           a.pitch);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace qg
