// Rows to 8-bit codes with one fp32 scale a row, in place order or straight
// to the rows' sorted places, and the packed layout of 8-bit weights.
//
//   s = fp32(max_k |x_k| / 127),  q_k = clamp(rne(fp32(x_k / s)), -127, 127)
//
// with both quotients correctly rounded; s = 0 gives q = 0, and a row that
// holds a NaN or an infinity gets s = NaN and q = 0, so that its products are
// NaN.  Columns K .. ldc-1 of the codes are written as zero.
#include "int8.h"

namespace qg {

constexpr int RQ_V = 8;  // elements of a thread's vector

template <int ACT>
__device__ __forceinline__ void load8(const void *x, int64_t at, int64_t left, float *v)
{
    if (left >= RQ_V) {
        if constexpr (ACT == ACT_F32) {
            __builtin_memcpy(v, (const float *)x + at, 32);
        } else {
            uint16_t h[RQ_V];
            __builtin_memcpy(h, (const uint16_t *)x + at, 16);
#pragma unroll
            for (int i = 0; i < RQ_V; i++)
                v[i] = __uint_as_float((uint32_t)h[i] << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < RQ_V; i++) {
            v[i] = 0.f;
            if (i < left)
                v[i] = ACT == ACT_F32 ? ((const float *)x)[at + i]
                                      : __uint_as_float((uint32_t)((const uint16_t *)x)[at + i] << 16);
        }
    }
}

__device__ __forceinline__ uint32_t pack_codes4(const float *v, float s)
{
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float r = __builtin_rintf(v[i] / s);
        const int c = (int)fminf(fmaxf(r, -127.f), 127.f);
        o |= ((uint32_t)c & 0xFFu) << (8 * i);
    }
    return o;
}

// TPR threads a row (64: four rows a workgroup, no barrier; 256: one row), the
// row held in NV vectors of registers a thread when it fits, else read twice.
template <int ACT, int TPR, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(RowsArgs a)
{
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (row >= a.B)
        return;  // whole waves
    const int64_t base = row * a.K;
    float v[NV][RQ_V];
    uint32_t top = 0;  // largest |x| as bits: infinities and NaNs above all finite values
#pragma unroll
    for (int j = 0; j < NV; j++) {
        const int64_t k = ((int64_t)j * TPR + tid) * RQ_V;
        load8<ACT>(a.x, base + k, a.K - k, v[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
        for (int i = 0; i < RQ_V; i++)
            top = max(top, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
    for (int64_t k = ((int64_t)NV * TPR + tid) * RQ_V; k < a.K; k += TPR * RQ_V) {
        float w[RQ_V];
        load8<ACT>(a.x, base + k, a.K - k, w);
#pragma unroll
        for (int i = 0; i < RQ_V; i++)
            top = max(top, __float_as_uint(w[i]) & 0x7FFFFFFFu);
    }
    for (int d = 32; d; d >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if constexpr (TPR > 64) {
        __shared__ uint32_t tops[TPR / 64];
        if ((threadIdx.x & 63) == 0)
            tops[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; w++)
            top = max(top, tops[w]);
    }
    const bool bad = top >= 0x7F800000u;
    const float s = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 127.f;
    const bool zero = bad || s == 0.f;

    const int reps = a.pos ? a.topk : 1;
    for (int r = 0; r < reps; r++) {
        int64_t to = row;
        if (a.pos) {
            to = a.pos[row * a.topk + r];
            if (to < 0)
                continue;
            if (to >= a.R) {
                if (tid == 0)
                    __hip_atomic_fetch_or(a.status, DEV_BAD_ROUTE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                continue;
            }
        }
        int8_t *o = a.codes + to * a.ldc;
        if (tid == 0)
            a.scales[to] = s;
        auto put = [&](int64_t k, const float *w) {
            u32x2 c = u32x2{pack_codes4(w, s), pack_codes4(w + 4, s)};
            if (zero)
                c = u32x2{0u, 0u};
            *(u32x2 *)(o + k) = c;
        };
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * RQ_V;
            if (k < a.ldc)
                put(k, v[j]);
        }
        for (int64_t k = ((int64_t)NV * TPR + tid) * RQ_V; k < a.ldc; k += TPR * RQ_V) {
            float w[RQ_V];
            load8<ACT>(a.x, base + k, a.K - k, w);
            put(k, w);
        }
    }
}

hipError_t launch_quantize_rows(int act, const RowsArgs &a, hipStream_t st)
{
    const bool f32 = act == QGEMM_F32;
#define QROWS(TPR, NV)                                                                                              \
    do {                                                                                                            \
        const dim3 g((unsigned)((a.B + 256 / TPR - 1) / (256 / TPR)));                                              \
        if (f32)                                                                                                    \
            hipLaunchKernelGGL((quantize_rows_kernel<ACT_F32, TPR, NV>), g, dim3(256), 0, st, a);                   \
        else                                                                                                        \
            hipLaunchKernelGGL((quantize_rows_kernel<ACT_BF16, TPR, NV>), g, dim3(256), 0, st, a);                  \
    } while (0)
    if (a.K <= 64 * RQ_V * 2)
        QROWS(64, 2);
    else if (a.K <= 256 * RQ_V * 4)
        QROWS(256, 4);
    else
        QROWS(256, 9);
#undef QROWS
    return hipGetLastError();
}

// One thread a 16-byte chunk: 16 codes of one row (zero past N and K); the
// scales follow.
__global__ __launch_bounds__(256) void i8_pack_kernel(Layout L, const int8_t *codes, const float *scales, uint8_t *out)
{
    const int64_t chunks = L.RT * L.S * 64;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < chunks) {
        const int64_t slab = i >> 6, rt = slab / L.S, s = slab % L.S;
        const int lane = (int)(i & 63);
        const int64_t n = rt * 16 + (lane & 15), k = s * 64 + (lane >> 4) * 16;
        u32x4 c = u32x4{0u, 0u, 0u, 0u};
        if (n < L.N && k < L.K) {
            const int8_t *p = codes + n * L.K + k;
            if (k + 16 <= L.K) {
                __builtin_memcpy(&c, p, 16);
            } else {
                for (int j = 0; j < (int)(L.K - k); j++)
                    c[j >> 2] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
            }
        }
        *(u32x4 *)(out + i * 16) = c;
    }
    const int64_t ns = (L.total - L.scale_off) / 4;
    if (i < ns)
        ((float *)(out + L.scale_off))[i] = i < L.N ? scales[i] : 0.f;
}

hipError_t launch_i8_pack(const Layout &L, const int8_t *codes, const float *scales, uint8_t *out, hipStream_t st)
{
    const int64_t chunks = L.RT * L.S * 64, ns = (L.total - L.scale_off) / 4;
    const int64_t n = chunks > ns ? chunks : ns;
    hipLaunchKernelGGL(i8_pack_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, L, codes, scales, out);
    return hipGetLastError();
}

}  // namespace qg
