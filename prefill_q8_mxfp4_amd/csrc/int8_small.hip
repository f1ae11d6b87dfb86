// 8-bit products with few rows: each weight byte is read once, straight into
// the matrix cores' operands, with the rows' codes beside it.
//
// A packed slab of 16 channels x 64 k is 1 KB whose chunk L is the A operand of
// lane L of v_mfma_i32_16x16x64_i8, and lane L's 16 bytes of a row's codes
// (row L % 16, k group L / 16) are the B operand, so nothing is decoded or
// shuffled.  The waves of a workgroup take the slabs of its R row tiles in
// turn, and their int32 sums meet in LDS: sums of whole numbers, so the split
// changes no bit.  A lane ends with four neighbouring channels of one row.
#include "int8.h"

namespace qg {

constexpr int SM_W = 8;  // waves a workgroup
constexpr int SM_R = 2;  // row tiles a workgroup (with SwiGLU a gate tile and its up tile)

// Row tile of a workgroup's r'th tile: with SwiGLU the gate tiles first, then
// the up tiles; past the last one a copy of it (computed, never stored).
template <bool DUAL>
__device__ __forceinline__ int sm_tile(const I8Args &a, int g, int r)
{
    if constexpr (DUAL) {
        constexpr int H = SM_R / 2;
        const int last = a.Nh / 16 - 1;
        return (r < H ? 0 : a.Nh / 16) + min(g * H + r % H, last);
    } else {
        return min(g * SM_R + r, a.RT - 1);
    }
}

template <int CG, bool DUAL, int OUTT>
__device__ __forceinline__ void sm_body(const I8Args &a, const uint8_t *w, int g, int64_t row0, int rows, i32x4 *red)
{
    constexpr int R = SM_R;
    constexpr int D = CG >= 4 ? 2 : 4;  // slabs loaded ahead of their products
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, kg = lane >> 4;
    const int64_t tile_bytes = (int64_t)a.S << 10;
    const uint8_t *wt[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        wt[r] = w + sm_tile<DUAL>(a, g, r) * tile_bytes;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.codes + row0 * a.ldc, (int64_t)rows * a.ldc);
    int xo[CG];
#pragma unroll
    for (int c = 0; c < CG; c++)  // rows past the last read row 0: their columns are never stored
        xo[c] = (c * 16 + c16 < rows ? (c * 16 + c16) * a.ldc : 0) + kg * 16;
    i32x4 acc[R][CG];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int c = 0; c < CG; c++)
            acc[r][c] = i32x4{0, 0, 0, 0};
    for (int s0 = wid; s0 < a.S; s0 += SM_W * D) {
        i32x4 wv[D][R], xv[D][CG];
#pragma unroll
        for (int d = 0; d < D; d++) {
            // past the last slab the weights come as zeros from an empty
            // resource; the codes then come from anywhere in the rows, or as zeros
            const int s = s0 + d * SM_W;
            const bool live = s < a.S;
#pragma unroll
            for (int r = 0; r < R; r++)
                wv[d][r] = __builtin_bit_cast(
                    i32x4, bload16_nt(make_rsrc(wt[r], live ? tile_bytes : 0), lane * 16, live ? s << 10 : 0));
#pragma unroll
            for (int c = 0; c < CG; c++)
                xv[d][c] = __builtin_bit_cast(i32x4, bload16(xr, xo[c] + (s << 6), 0));
        }
#pragma unroll
        for (int d = 0; d < D; d++)
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int c = 0; c < CG; c++)
                    acc[r][c] = mfma_i8(wv[d][r], xv[d][c], acc[r][c]);
    }
    __syncthreads();  // the previous pass has read its sums
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int c = 0; c < CG; c++)
            red[((wid * R + r) * CG + c) * 64 + lane] = acc[r][c];
    __syncthreads();
    constexpr int RO = DUAL ? R / 2 : R;  // output tiles a workgroup
    const bool vec = (a.ncols & 3) == 0;
    const float *ws = (const float *)(w + a.scale_off);
    for (int o = wid; o < RO * CG; o += SM_W) {
        const int r = o / CG, c = o % CG;
        auto sum = [&](int rr) {
            i32x4 s = red[(rr * CG + c) * 64 + lane];
#pragma unroll
            for (int v = 1; v < SM_W; v++)
                s += red[((v * R + rr) * CG + c) * 64 + lane];
            return s;
        };
        const int t0 = g * RO + r;  // output tile
        const int n = t0 * 16 + kg * 4;
        const int b = c * 16 + c16;
        const bool live = b < rows && n < a.ncols;
        const float xs = live ? a.xs[row0 + b] : 0.f;
        f32x4 out;
        const i32x4 s = sum(r);
        i32x4 u = s;
        if constexpr (DUAL)
            u = sum(r + R / 2);
        if (live) {
            const f32x4 t = *(const f32x4 *)(ws + n);
#pragma unroll
            for (int i = 0; i < 4; i++)
                out[i] = (float)s[i] * xs * t[i];
            if constexpr (DUAL) {
                const f32x4 tu = *(const f32x4 *)(ws + a.Nh + n);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    out[i] = silu(out[i]) * ((float)u[i] * xs * tu[i]);
            }
            i8_store4<OUTT>(a.y, row0 + b, a.ncols, n, vec, out);
        }
    }
}

template <int CG, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * SM_W) void i8_small_kernel(I8Args a)
{
    __shared__ i32x4 red[SM_W * SM_R * CG * 64];
    const int row0 = blockIdx.y * 16 * CG;
    sm_body<CG, DUAL, OUTT>(a, a.w, blockIdx.x, row0, min(16 * CG, a.B - row0), red);
}

// One workgroup a (expert, row group); an expert's rows are taken 64 at a time.
template <bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * SM_W) void i8_small_grouped_kernel(I8Args a, I8Groups grp, int groups)
{
    __shared__ i32x4 red[SM_W * SM_R * 4 * 64];
    const int e = blockIdx.x / groups, g = blockIdx.x % groups;
    const int lo = __builtin_amdgcn_readfirstlane(grp.off[e]);
    const int hi = __builtin_amdgcn_readfirstlane(grp.off[e + 1]);
    if (lo < 0 || hi < lo || hi > a.B || (e == 0 && lo != 0)) {
        if (g == 0 && threadIdx.x == 0)
            __hip_atomic_fetch_or(grp.status, DEV_BAD_OFFSETS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }
    if (lo == hi)
        return;
    const uint8_t *w = uniform_ptr(grp.wtab[e]);
    for (int r0 = lo; r0 < hi; r0 += 64) {
        const int rows = min(64, hi - r0);
        if (rows <= 16)
            sm_body<1, DUAL, OUTT>(a, w, g, r0, rows, red);
        else if (rows <= 32)
            sm_body<2, DUAL, OUTT>(a, w, g, r0, rows, red);
        else
            sm_body<4, DUAL, OUTT>(a, w, g, r0, rows, red);
    }
}

static int sm_groups(const I8Args &a)
{
    return a.Nh ? (a.Nh / 16 + SM_R / 2 - 1) / (SM_R / 2) : (a.RT + SM_R - 1) / SM_R;
}

template <int CG>
static void small_cg(const I8Args &a, int outt, hipStream_t st)
{
    const dim3 grid((unsigned)sm_groups(a), (unsigned)((a.B + 16 * CG - 1) / (16 * CG)));
    const dim3 blk(64 * SM_W);
    if (a.Nh && outt == OUT_F32)
        hipLaunchKernelGGL((i8_small_kernel<CG, true, OUT_F32>), grid, blk, 0, st, a);
    else if (a.Nh)
        hipLaunchKernelGGL((i8_small_kernel<CG, true, OUT_BF16>), grid, blk, 0, st, a);
    else if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_small_kernel<CG, false, OUT_F32>), grid, blk, 0, st, a);
    else
        hipLaunchKernelGGL((i8_small_kernel<CG, false, OUT_BF16>), grid, blk, 0, st, a);
}

hipError_t launch_i8_small(const I8Args &a, int outt, hipStream_t st)
{
    if (a.B <= 16)
        small_cg<1>(a, outt, st);
    else if (a.B <= 32)
        small_cg<2>(a, outt, st);
    else
        small_cg<4>(a, outt, st);
    return hipGetLastError();
}

hipError_t launch_i8_small_grouped(const I8Args &a, const I8Groups &g, int outt, hipStream_t st)
{
    const int groups = sm_groups(a);
    const dim3 grid((unsigned)((int64_t)g.E * groups)), blk(64 * SM_W);
    if (a.Nh && outt == OUT_F32)
        hipLaunchKernelGGL((i8_small_grouped_kernel<true, OUT_F32>), grid, blk, 0, st, a, g, groups);
    else if (a.Nh)
        hipLaunchKernelGGL((i8_small_grouped_kernel<true, OUT_BF16>), grid, blk, 0, st, a, g, groups);
    else if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_small_grouped_kernel<false, OUT_F32>), grid, blk, 0, st, a, g, groups);
    else
        hipLaunchKernelGGL((i8_small_grouped_kernel<false, OUT_BF16>), grid, blk, 0, st, a, g, groups);
    return hipGetLastError();
}

}  // namespace qg
