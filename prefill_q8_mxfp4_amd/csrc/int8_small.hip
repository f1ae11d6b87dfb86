// 8-bit products with few rows: each weight byte is read once, straight into
// the matrix cores' operands, with the rows' codes beside it.
//
// A packed slab of 16 channels x 64 k is 1 KB whose chunk L is the A operand of
// lane L of v_mfma_i32_16x16x64_i8, and lane L's 16 bytes of a row's codes
// (row L % 16, k group L / 16) are the B operand, so nothing is decoded or
// shuffled.  Reading the weights is the bound: a workgroup owns R row tiles and
// 16 rows, its waves take the slabs of those tiles two at a time (the codes' two
// 64-byte halves of a cache line) and keep SLOTS such pairs in flight in
// registers.  The waves' int32 sums meet in LDS: sums of whole numbers, so the
// split changes no bit.  A lane ends with four neighbouring channels of one row.
#include "int8_quant.h"

namespace qg {

constexpr int SM_W = 8;  // waves a workgroup

// Row tile of a workgroup's r'th tile: with SwiGLU the gate tiles first, then
// the up tiles; past the last one a copy of it (computed, never stored).
template <int R, bool DUAL>
__device__ __forceinline__ int sm_tile(const I8Args &a, int g, int r)
{
    if constexpr (DUAL) {
        constexpr int H = R / 2;
        const int last = a.Nh / 16 - 1;
        return (r < H ? 0 : a.Nh / 16) + min(g * H + r % H, last);
    } else {
        return min(g * R + r, a.RT - 1);
    }
}

// FUSED: up to SM_FUSED_B rows come as floats of type ACT (xf), which every
// workgroup quantises for itself into LDS while its first weights are on their
// way: a row is 10 KB to read from L2, a launch of its own costs more (1 x 5120 x
// 5120: 10.0 us in two launches, 6.9 in one).  Rows longer than SM_FUSED_BYTES
// in all would take the registers that let two workgroups share a CU (20 us).
constexpr int SM_FUSED_B = 2, SM_FUSED_BYTES = 8 * 1024, SM_FUSED_NV = SM_FUSED_BYTES / (64 * SM_W * RQ_V);

template <int R, int SLOTS, bool DUAL, int OUTT, bool FUSED, int ACT>
__global__ __launch_bounds__(64 * SM_W, 2) void i8_small_kernel(I8Args a, const void *xf)
{
    __shared__ uint8_t xq[FUSED ? SM_FUSED_BYTES : 16];  // [rows][64 S] codes
    __shared__ uint32_t tops[SM_W];
    __shared__ i32x4 red[SM_W * R * 64];
    const int g = blockIdx.x, row0 = blockIdx.y * 16;
    const int rows = min(16, a.B - row0);
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, kg = lane >> 4;
    const int64_t tile_bytes = (int64_t)a.S << 10;
    const uint8_t *wt[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        wt[r] = a.w + sm_tile<R, DUAL>(a, g, r) * tile_bytes;
    const uint8_t *xbase = (const uint8_t *)a.codes + (int64_t)row0 * a.ldc;
    const int64_t xbytes = (int64_t)rows * a.ldc;
    const int xo = (c16 < rows ? c16 * a.ldc : 0) + kg * 16;  // rows past the last: row 0, never stored
    i32x4 acc[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        acc[r] = i32x4{0, 0, 0, 0};

    // The i'th pair of slabs of this wave (S is even) into a slot; past the
    // last one zeros from empty resources, so that every step issues the same
    // loads and the waits for the slots are exact.
    i32x4 wv[SLOTS][2][R], xv[FUSED ? 1 : SLOTS][2];
    // FUSED: all threads on one row, or half of them on each of two
    const int tpr = rows == 2 ? 32 * SM_W : 64 * SM_W, xr_ = rows == 2 ? threadIdx.x / tpr : 0;
    const int tt = threadIdx.x - xr_ * tpr, kp = a.S * 64;
    Raw8<ACT> fv[FUSED ? SM_FUSED_NV : 1];  // K is a multiple of 8
    if constexpr (FUSED) {                  // before the weights: loads come back in order
        constexpr int ESZ = Raw8<ACT>::ESZ;
        const __amdgpu_buffer_rsrc_t fr = make_rsrc(xf, (int64_t)rows * a.K * ESZ);
#pragma unroll
        for (int j = 0; j < SM_FUSED_NV; j++) {
            const int k = (j * tpr + tt) * RQ_V;  // past the row: past the resource, zeros
            fv[j].load(fr, k < a.K ? (xr_ * a.K + k) * ESZ : 0x7FFFFF00);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    auto load = [&](int i, int slot) {
        const int s = (i * SM_W + wid) * 2;
        const bool live = s < a.S;
        const __amdgpu_buffer_rsrc_t xr = make_rsrc(xbase, live ? xbytes : 0);
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int r = 0; r < R; r++)
                wv[slot][h][r] = __builtin_bit_cast(
                    i32x4, bload16_nt(make_rsrc(wt[r], live ? tile_bytes : 0), lane * 16, live ? (s + h) << 10 : 0));
            if constexpr (!FUSED)
                xv[slot][h] = __builtin_bit_cast(i32x4, bload16(xr, xo + ((s + h) << 6), 0));
        }
    };
    const int n = (a.S / 2 + SM_W - 1) / SM_W;
#pragma unroll
    for (int u = 0; u < SLOTS; u++) {
        load(u, u);
        __builtin_amdgcn_sched_barrier(0);  // in the order of the loop
    }
    [[maybe_unused]] float own_scale = 0.f;
    if constexpr (FUSED) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < SM_FUSED_NV; j++) {
            float v[RQ_V];
            fv[j].floats(v);
            top = top8(v, top);
        }
        top = wave_max(top);
        if (lane == 0)
            tops[wid] = top;
        __syncthreads();
        uint32_t top0 = 0, top1 = 0;
#pragma unroll
        for (int k = 0; k < SM_W / 2; k++) {
            top0 = max(top0, tops[k]);
            top1 = max(top1, tops[SM_W / 2 + k]);
        }
        if (rows == 1)
            top0 = max(top0, top1);
        const RowScale sc(xr_ ? top1 : top0);
        own_scale = RowScale(c16 ? top1 : top0).s;  // of the row that this lane stores
#pragma unroll
        for (int j = 0; j < SM_FUSED_NV; j++) {
            const int k = (j * tpr + tt) * RQ_V;
            if (k < kp) {  // with the padding's zeros
                float v[RQ_V];
                fv[j].floats(v);
                *(u32x2 *)(xq + xr_ * kp + k) = sc.codes(v);
            }
        }
        __syncthreads();
    }
    auto multiply = [&](int i, int u) {  // the i'th pair, in slot u
        const int s = (i * SM_W + wid) * 2;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            i32x4 x;
            if constexpr (FUSED)
                x = *(const i32x4 *)(xq + (c16 < rows ? c16 * kp : 0) + (s < a.S ? (s + h) << 6 : 0) + kg * 16);
            else
                x = xv[u][h];
#pragma unroll
            for (int r = 0; r < R; r++)
                acc[r] = mfma_i8(wv[u][h][r], x, acc[r]);
        }
    };
    int i = SLOTS;
    for (; i < n; i += SLOTS) {
#pragma unroll
        for (int u = 0; u < SLOTS; u++) {
            multiply(i - SLOTS + u, u);
            __builtin_amdgcn_sched_barrier(0);
            load(i + u, u);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int u = 0; u < SLOTS; u++)
        multiply(i - SLOTS + u, u);

#pragma unroll
    for (int r = 0; r < R; r++)
        red[(wid * R + r) * 64 + lane] = acc[r];
    __syncthreads();
    constexpr int RO = DUAL ? R / 2 : R;  // output tiles of a workgroup
    const float *ws = (const float *)(a.w + a.scale_off);
    if (wid < RO) {
        auto sum = [&](int r) {
            i32x4 v = red[r * 64 + lane];
#pragma unroll
            for (int k = 1; k < SM_W; k++)
                v += red[(k * R + r) * 64 + lane];
            return v;
        };
        const int n = (g * RO + wid) * 16 + kg * 4;
        const i32x4 s = sum(wid);
        i32x4 up = s;
        if constexpr (DUAL)
            up = sum(wid + RO);
        if (c16 < rows && n < a.ncols) {
            const float xs = FUSED ? own_scale : a.xs[row0 + c16];
            const f32x4 t = *(const f32x4 *)(ws + n);
            f32x4 out;
#pragma unroll
            for (int i = 0; i < 4; i++)
                out[i] = (float)s[i] * xs * t[i];
            if constexpr (DUAL) {
                const f32x4 tu = *(const f32x4 *)(ws + a.Nh + n);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    out[i] = silu(out[i]) * ((float)up[i] * xs * tu[i]);
            }
            i8_put4_part<OUTT>((uint8_t *)a.y + ((int64_t)(row0 + c16) * a.ncols + n) * (OUTT == OUT_F32 ? 4 : 2),
                               out, a.ncols - n);
        }
    }
}

template <int R, int SLOTS, bool DUAL, bool FUSED, int ACT>
static void small_go(const I8Args &a, const void *xf, int outt, hipStream_t st)
{
    const int groups = DUAL ? a.Nh / 16 : (a.RT + R - 1) / R;
    const dim3 grid((unsigned)groups, (unsigned)((a.B + 15) / 16)), blk(64 * SM_W);
    if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_small_kernel<R, SLOTS, DUAL, OUT_F32, FUSED, ACT>), grid, blk, 0, st, a, xf);
    else
        hipLaunchKernelGGL((i8_small_kernel<R, SLOTS, DUAL, OUT_BF16, FUSED, ACT>), grid, blk, 0, st, a, xf);
}

template <bool FUSED, int ACT>
static void small_shape(const I8Args &a, const void *xf, int outt, hipStream_t st)
{
    if (a.Nh)
        small_go<2, 4, true, FUSED, ACT>(a, xf, outt, st);
    else if (a.N >= 8192)
        small_go<2, 4, false, FUSED, ACT>(a, xf, outt, st);
    else
        small_go<1, 5, false, FUSED, ACT>(a, xf, outt, st);
}

// Up to two rows any weight, up to 16 rows one of 8192 channels or more.
// Measured against the tiled kernel's best shape, us: 5120 x 5120 at B = 1, 2, 4,
// 16: 7.4, 7.5, 8.2, 10.5 against 7.7 throughout; 34816 x 5120 at B = 2, 8, 16:
// 32.1, 33.3, 35.5 against 35.7, 37.2, 39.5, and at 24 51 against 40.
bool i8_small_wins(int64_t B, int64_t N) { return B <= 2 || (B <= 16 && N >= 8192); }

hipError_t launch_i8_small(const I8Args &a, int outt, hipStream_t st)
{
    small_shape<false, ACT_F32>(a, nullptr, outt, st);
    return hipGetLastError();
}

bool i8_small_fuses(int64_t B, int64_t K, int64_t S)
{
    return B <= SM_FUSED_B && K % RQ_V == 0 && B * S * 64 <= SM_FUSED_BYTES;
}

hipError_t launch_i8_small_fused(const I8Args &a, const void *x, int act, int outt, hipStream_t st)
{
    if (act == QGEMM_F32)
        small_shape<true, ACT_F32>(a, x, outt, st);
    else
        small_shape<true, ACT_BF16>(a, x, outt, st);
    return hipGetLastError();
}

}  // namespace qg
