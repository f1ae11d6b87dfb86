// Rows to 8-bit codes with one fp32 scale a row, in place order or straight
// to the rows' sorted places, and the packed layout of 8-bit weights.
//
//   s = fp32(max_k |x_k| / 127),  q_k = clamp(rne(fp32(x_k / s)), -127, 127)
//
// with both quotients correctly rounded; s = 0 gives q = 0, and a row that
// holds a NaN or an infinity gets s = NaN and q = 0, so that its products are
// NaN.  Columns K .. ldc-1 of the codes are written as zero.
#include "int8_quant.h"

namespace qg {

// TPR threads a row (64: four rows a workgroup and no barrier), the row held in
// NV vectors of registers a thread as far as it fits, the rest read twice.
// WHOLE: K is a multiple of 8, so a row is whole vectors, all of them loaded
// before the first is looked at; past the row the resource ends: zeros.
template <int ACT, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void quantize_rows_kernel(RowsArgs a)
{
    constexpr int RPW = TPR > 256 ? 1 : 256 / TPR;  // rows a workgroup
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPW + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    if (row >= a.B)
        return;  // whole waves
    const int64_t base = row * a.K;
    float v[NV][RQ_V];
    if constexpr (WHOLE) {
        Raw8<ACT> raw[NV];
        const __amdgpu_buffer_rsrc_t xr =
            make_rsrc((const uint8_t *)a.x + base * Raw8<ACT>::ESZ, a.K * Raw8<ACT>::ESZ);
#pragma unroll
        for (int j = 0; j < NV; j++)
            raw[j].load(xr, (j * TPR + tid) * RQ_V * Raw8<ACT>::ESZ);
#pragma unroll
        for (int j = 0; j < NV; j++)
            raw[j].floats(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * RQ_V;
            if (j == 0 || (int64_t)j * TPR * RQ_V < a.K)  // uniform
                load8<ACT>(a.x, base + k, a.K - k, v[j]);
            else
#pragma unroll
                for (int i = 0; i < RQ_V; i++)
                    v[j][i] = 0.f;
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; j++)
        top = top8(v[j], top);
    for (int64_t k = ((int64_t)NV * TPR + tid) * RQ_V; k < a.K; k += TPR * RQ_V) {
        float w[RQ_V];
        load8<ACT>(a.x, base + k, a.K - k, w);
        top = top8(w, top);
    }
    top = wave_max(top);
    if constexpr (TPR > 64) {
        __shared__ uint32_t tops[TPR / 64];
        if ((threadIdx.x & 63) == 0)
            tops[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; w++)
            top = max(top, tops[w]);
    }
    const RowScale sc(top);

    // the registers' codes once, then to every row they go to
    u32x2 c[NV];
#pragma unroll
    for (int j = 0; j < NV; j++)
        c[j] = sc.codes(v[j]);
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
            a.scales[to] = sc.s;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int64_t k = ((int64_t)j * TPR + tid) * RQ_V;
            if (k < a.ldc)
                *(u32x2 *)(o + k) = c[j];
        }
        for (int64_t k = ((int64_t)NV * TPR + tid) * RQ_V; k < a.ldc; k += TPR * RQ_V) {
            float w[RQ_V];
            load8<ACT>(a.x, base + k, a.K - k, w);
            *(u32x2 *)(o + k) = sc.codes(w);
        }
    }
}

template <int TPR, int NV>
static void rows_go(bool f32, const RowsArgs &a, hipStream_t st)
{
    constexpr int RPW = TPR > 256 ? 1 : 256 / TPR;
    const dim3 g((unsigned)((a.B + RPW - 1) / RPW)), blk(TPR > 256 ? TPR : 256);
    const bool whole = a.K % RQ_V == 0;
    if (f32 && whole)
        hipLaunchKernelGGL((quantize_rows_kernel<ACT_F32, TPR, NV, true>), g, blk, 0, st, a);
    else if (f32)
        hipLaunchKernelGGL((quantize_rows_kernel<ACT_F32, TPR, NV, false>), g, blk, 0, st, a);
    else if (whole)
        hipLaunchKernelGGL((quantize_rows_kernel<ACT_BF16, TPR, NV, true>), g, blk, 0, st, a);
    else
        hipLaunchKernelGGL((quantize_rows_kernel<ACT_BF16, TPR, NV, false>), g, blk, 0, st, a);
}

// As few threads a row as hold it in registers; long rows of which there are not
// enough for the chip get four times as many (70 rows of 17408 floats: 6.6 us
// with 256 threads, 6.0 with 1024).
hipError_t launch_quantize_rows(int act, const RowsArgs &a, hipStream_t st)
{
    const bool f32 = act == QGEMM_F32;
    if (a.K <= 64 * RQ_V * 2)
        rows_go<64, 2>(f32, a, st);
    else if (a.K <= 256 * RQ_V * 1)
        rows_go<256, 1>(f32, a, st);
    else if (a.B <= 256)
        rows_go<1024, 3>(f32, a, st);
    else if (a.K <= 256 * RQ_V * 3)
        rows_go<256, 3>(f32, a, st);
    else
        rows_go<256, 9>(f32, a, st);
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
