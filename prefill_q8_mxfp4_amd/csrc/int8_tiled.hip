// 8-bit products with many rows: BM batch rows x BN channels a workgroup, both
// operands staged through LDS by gfx950's direct loads, int32 accumulators.
//
// LDS holds matrix-core operands as they are fed: a 1 KB chunk is 16 channels
// (or 16 rows) x 64 k, lane L's 16 bytes at 16 L.  A packed weight slab is
// such a chunk already; a row group's chunk is gathered by the load itself
// (lane L: row L % 16, k group L / 16), so every LDS access is a wave-wide
// contiguous KB and no shuffle, decode or register staging is left.  A step is
// 128 k (two chunks of each tile), two steps in LDS: the next one is loaded
// while the current one is multiplied.
#include "int8.h"

namespace qg {

constexpr int I8_STEP = 128;  // k a step

template <int WM_, int WN_, int TM_, int TN_>
struct TiShape {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;  // waves, and 16-wide tiles a wave
    static constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
    static constexpr int XC = BM / 16 * 2, WC = BN / 16 * 2;  // chunks a step
    static constexpr int XPW = XC / NW, WPW = WC / NW;        // of them a wave loads
    static constexpr int STAGE = (XC + WC) * 1024;
    static_assert(XC % NW == 0 && WC % NW == 0, "whole chunks a wave");
};
using TiBig = TiShape<2, 4, 8, 4>;    // 256 x 256, 8 waves of 128 x 64
using TiMid = TiShape<2, 2, 4, 4>;    // 128 x 128, 4 waves of 64 x 64

typedef __attribute__((address_space(3))) uint8_t lds_byte;

__device__ __forceinline__ void load_chunk(__amdgpu_buffer_rsrc_t r, uint8_t *lds, int voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 0);
}

// Row tile (16 channels) of a workgroup's i'th tile.  With SwiGLU a wave's
// tiles are TN / 2 gate tiles and the matching up tiles, so that a lane holds
// both; tiles past the last are copies of it (computed, never stored).
template <typename S, bool DUAL>
__device__ __forceinline__ int ti_tile(const I8Args &a, int nt, int i)
{
    if constexpr (DUAL) {
        const int wn = i / S::TN, j = i % S::TN, H = S::TN / 2;
        const int t = nt * (S::BN / 32) + wn * H + j % H;
        const int last = a.Nh / 16 - 1;
        return (j < H ? 0 : a.Nh / 16) + min(t, last);
    } else {
        return min(nt * (S::BN / 16) + i, a.RT - 1);
    }
}

// Outputs of one lane for row group i: tiles j in acc (int32 sums).
template <typename S, bool DUAL, int OUTT>
__device__ __forceinline__ void ti_store(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int wm,
                                         int wn, int lane, int i, const i32x4 (&acc)[S::TN])
{
    const int b = (wm * S::TM + i) * 16 + (lane & 15);
    if (b >= rows)
        return;
    const bool vec = (a.ncols & 3) == 0;
    const float xs = a.xs[row0 + b];
    const float *ws = (const float *)(w + a.scale_off);
    constexpr int TO = DUAL ? S::TN / 2 : S::TN;
#pragma unroll
    for (int j = 0; j < TO; j++) {
        const int n = ((nt * S::WN + wn) * TO + j) * 16 + (lane >> 4) * 4;
        if (n >= a.ncols)
            continue;
        const f32x4 t = *(const f32x4 *)(ws + n);
        f32x4 o;
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = (float)acc[j][k] * xs * t[k];
        if constexpr (DUAL) {
            const f32x4 tu = *(const f32x4 *)(ws + a.Nh + n);
#pragma unroll
            for (int k = 0; k < 4; k++)
                o[k] = silu(o[k]) * ((float)acc[j + TO][k] * xs * tu[k]);
        }
        i8_store4<OUTT>(a.y, row0 + b, a.ncols, n, vec, o);
    }
}

// One tile: rows row0 .. row0+rows-1 (at most BM), weight tile nt, steps k0 .. k1-1.
template <typename S, bool DUAL>
__device__ __forceinline__ void ti_tile_sums(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int k0,
                                             int k1, uint8_t *st0, uint8_t *st1, i32x4 (&acc)[S::TM][S::TN])
{
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid / S::WN, wn = wid % S::WN;
    const int64_t tile_bytes = (int64_t)a.S << 10;

    // what this wave loads: row groups and weight tiles, both chunks of each
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.codes + row0 * a.ldc, (int64_t)rows * a.ldc);
    int xo[S::XPW / 2];
#pragma unroll
    for (int c = 0; c < S::XPW / 2; c++) {
        const int b = min((wid * (S::XPW / 2) + c) * 16 + (lane & 15), rows - 1);
        xo[c] = b * a.ldc + (lane >> 4) * 16;
    }
    __amdgpu_buffer_rsrc_t wr[S::WPW / 2];
#pragma unroll
    for (int c = 0; c < S::WPW / 2; c++)
        wr[c] = make_rsrc(w + ti_tile<S, DUAL>(a, nt, wid * (S::WPW / 2) + c) * tile_bytes, tile_bytes);

    auto load = [&](int kt, uint8_t *st) {
        uint8_t *xl = st + wid * S::XPW * 1024, *wl = st + (S::XC + wid * S::WPW) * 1024;
#pragma unroll
        for (int c = 0; c < S::XPW; c++)
            load_chunk(xr, xl + c * 1024, xo[c / 2] + (c & 1) * 64, kt * I8_STEP);
#pragma unroll
        for (int c = 0; c < S::WPW; c++)
            load_chunk(wr[c / 2], wl + c * 1024, lane * 16, (kt * 2 + (c & 1)) << 10);
    };
    auto compute = [&](const uint8_t *st) {
        const uint8_t *xl = st + wm * S::TM * 2048 + lane * 16;
        const uint8_t *wl = st + S::XC * 1024 + wn * S::TN * 2048 + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            i32x4 xf[S::TM], wf[S::TN];
#pragma unroll
            for (int j = 0; j < S::TN; j++)
                wf[j] = *(const i32x4 *)(wl + j * 2048 + h * 1024);
#pragma unroll
            for (int i = 0; i < S::TM; i++)
                xf[i] = *(const i32x4 *)(xl + i * 2048 + h * 1024);
#pragma unroll
            for (int i = 0; i < S::TM; i++)
#pragma unroll
                for (int j = 0; j < S::TN; j++)
                    acc[i][j] = mfma_i8(wf[j], xf[i], acc[i][j]);
        }
    };
#pragma unroll
    for (int i = 0; i < S::TM; i++)
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            acc[i][j] = i32x4{0, 0, 0, 0};
    load(k0, st0);
    __syncthreads();
    for (int kt = k0; kt < k1; kt += 2) {
        if (kt + 1 < k1)
            load(kt + 1, st1);
        compute(st0);
        __syncthreads();
        if (kt + 1 < k1) {
            if (kt + 2 < k1)
                load(kt + 2, st0);
            compute(st1);
            __syncthreads();
        }
    }
}

// Workgroup id -> tile: consecutive ids go to the 8 XCDs in turn, so an XCD's
// share is made one run of tiles, batch tiles fastest: the tiles an XCD works
// on together share their weight tiles in its L2.
__device__ __forceinline__ int xcd_order(int id, int n)
{
    const int per = (n + 7) / 8, xcd = id % 8, loc = id / 8;
    const int full = n % 8 == 0 ? 8 : n % 8;
    return xcd < full ? xcd * per + loc : full * per + (xcd - full) * (per - 1) + loc;
}

template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * S::NW, S::NW == 8 ? 2 : 2) void i8_tiled_kernel(I8Args a, int mtiles, int ntiles,
                                                                                int split, int32_t *part)
{
    __shared__ __attribute__((aligned(1024))) uint8_t st0[S::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[S::STAGE];
    const int t = xcd_order(blockIdx.x, gridDim.x);
    const int tile = t / split, piece = t % split;
    const int mt = tile % mtiles, nt = tile / mtiles;
    const int steps = a.S / 2, per = (steps + split - 1) / split;
    const int k0 = piece * per, k1 = min(steps, k0 + per);
    const int64_t row0 = (int64_t)mt * S::BM;
    const int rows = min(S::BM, (int)(a.B - row0));
    i32x4 acc[S::TM][S::TN];
    ti_tile_sums<S, DUAL>(a, a.w, row0, rows, nt, k0, k1, st0, st1, acc);
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    if (split > 1) {
        i32x4 *p = (i32x4 *)part + ((int64_t)t * S::NW + wid) * S::TM * S::TN * 64;
#pragma unroll
        for (int i = 0; i < S::TM; i++)
#pragma unroll
            for (int j = 0; j < S::TN; j++)
                p[(i * S::TN + j) * 64 + lane] = acc[i][j];
        return;
    }
#pragma unroll
    for (int i = 0; i < S::TM; i++)
        ti_store<S, DUAL, OUTT>(a, a.w, row0, rows, nt, wid / S::WN, wid % S::WN, lane, i, acc[i]);
}

// The split's partial tiles, a wave a row group of a wave's part of a tile.
template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64) void i8_tiled_reduce_kernel(I8Args a, int mtiles, int split, const int32_t *part)
{
    const int lane = threadIdx.x;
    const int i = blockIdx.x % S::TM, wid = blockIdx.x / S::TM % S::NW;
    const int tile = blockIdx.x / (S::TM * S::NW);
    const int mt = tile % mtiles, nt = tile / mtiles;
    const int64_t row0 = (int64_t)mt * S::BM;
    const int rows = min(S::BM, (int)(a.B - row0));
    i32x4 acc[S::TN];
#pragma unroll
    for (int j = 0; j < S::TN; j++)
        acc[j] = i32x4{0, 0, 0, 0};
    if ((wid / S::WN * S::TM + i) * 16 >= rows)
        return;
    for (int p = 0; p < split; p++) {
        const i32x4 *q = (const i32x4 *)part + (((int64_t)tile * split + p) * S::NW + wid) * S::TM * S::TN * 64;
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            acc[j] += q[(i * S::TN + j) * 64 + lane];
    }
    ti_store<S, DUAL, OUTT>(a, a.w, row0, rows, nt, wid / S::WN, wid % S::WN, lane, i, acc);
}

// Rows sorted by expert: workgroup t of the grid's bound takes the t'th
// (expert, row tile, weight tile), weight tiles fastest, found by a scan of the
// experts' row-tile counts; those past the real count leave.
template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * S::NW, 2) void i8_tiled_grouped_kernel(I8Args a, I8Groups grp, int ntiles)
{
    __shared__ __attribute__((aligned(1024))) uint8_t st0[S::STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[S::STAGE];
    __shared__ int wsum[S::NW], found[4];
    constexpr int NT = 64 * S::NW;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int t = xcd_order(blockIdx.x, gridDim.x);
    const int mt = t / ntiles, nt = t % ntiles;  // row tile over all experts
    if (tid == 0)
        found[0] = -1;
    int carry = 0;
    for (int e0 = 0; e0 < grp.E; e0 += NT) {
        const int e = e0 + tid;
        int lo = 0, hi = 0;
        if (e < grp.E) {
            lo = grp.off[e];
            hi = grp.off[e + 1];
            if (lo < 0 || hi < lo || hi > a.B || (e == 0 && lo != 0)) {
                lo = hi = 0;
                if (blockIdx.x == 0)
                    __hip_atomic_fetch_or(grp.status, DEV_BAD_OFFSETS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        const int v = (hi - lo + S::BM - 1) / S::BM;
        int s = v;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d)
                s += o;
        }
        if (lane == 63)
            wsum[wid] = s;
        __syncthreads();
        int before = carry;
        for (int k = 0; k < S::NW; k++) {
            before += k < wid ? wsum[k] : 0;
            carry += wsum[k];
        }
        const int first = before + s - v;
        if (mt >= first && mt < first + v) {
            found[0] = e;
            found[1] = lo + (mt - first) * S::BM;
            found[2] = hi;
        }
        __syncthreads();
        if (found[0] >= 0)
            break;  // uniform
    }
    const int e = __builtin_amdgcn_readfirstlane(found[0]);
    if (e < 0)
        return;
    const int row0 = __builtin_amdgcn_readfirstlane(found[1]);
    const int rows = min(S::BM, __builtin_amdgcn_readfirstlane(found[2]) - row0);
    const uint8_t *w = uniform_ptr(grp.wtab[e]);
    i32x4 acc[S::TM][S::TN];
    ti_tile_sums<S, DUAL>(a, w, row0, rows, nt, 0, a.S / 2, st0, st1, acc);
#pragma unroll
    for (int i = 0; i < S::TM; i++)
        ti_store<S, DUAL, OUTT>(a, w, row0, rows, nt, wid / S::WN, wid % S::WN, lane, i, acc[i]);
}

// ------------------------------------------------------------------ host

// Whole tiles of the larger shape when they fill the chip, else the smaller
// one, K split so that at least a round of tiles runs.
I8TiCfg i8_tiled_cfg(const I8Args &a, bool split)
{
    I8TiCfg c;
    const int cols = a.Nh ? 2 * a.Nh : a.N;
    const int64_t big = (int64_t)((a.B + 255) / 256) * ((cols + 255) / 256);
    c.BM = c.BN = big >= 192 ? 256 : 128;
    c.mtiles = (a.B + c.BM - 1) / c.BM;
    c.ntiles = (cols + c.BN - 1) / c.BN;
    const int64_t tiles = (int64_t)c.mtiles * c.ntiles;
    const int steps = a.S / 2;
    c.split = 1;
    if (split && tiles < 256) {
        int s = (int)(512 / tiles);
        s = s > steps / 4 ? steps / 4 : s;
        s = s < 1 ? 1 : s;
        const int per = (steps + s - 1) / s;
        c.split = (steps + per - 1) / per;  // no empty piece
    }
    c.part_bytes = c.split > 1 ? tiles * c.split * c.BM * c.BN * 4 : 0;
    return c;
}

template <typename S, bool DUAL, int OUTT>
static void tiled_go(const I8Args &a, const I8TiCfg &c, int32_t *part, hipStream_t st)
{
    const int tiles = c.mtiles * c.ntiles;
    hipLaunchKernelGGL((i8_tiled_kernel<S, DUAL, OUTT>), dim3((unsigned)(tiles * c.split)), dim3(64 * S::NW), 0, st, a,
                       c.mtiles, c.ntiles, c.split, part);
    if (c.split > 1)
        hipLaunchKernelGGL((i8_tiled_reduce_kernel<S, DUAL, OUTT>), dim3((unsigned)(tiles * S::TM * S::NW)), dim3(64),
                           0, st, a, c.mtiles, c.split, part);
}

template <typename S>
static void tiled_shape(const I8Args &a, const I8TiCfg &c, int32_t *part, int outt, hipStream_t st)
{
    if (a.Nh && outt == OUT_F32)
        tiled_go<S, true, OUT_F32>(a, c, part, st);
    else if (a.Nh)
        tiled_go<S, true, OUT_BF16>(a, c, part, st);
    else if (outt == OUT_F32)
        tiled_go<S, false, OUT_F32>(a, c, part, st);
    else
        tiled_go<S, false, OUT_BF16>(a, c, part, st);
}

hipError_t launch_i8_tiled(const I8Args &a, const I8TiCfg &c, int32_t *part, int outt, hipStream_t st)
{
    if (c.BM == 256)
        tiled_shape<TiBig>(a, c, part, outt, st);
    else
        tiled_shape<TiMid>(a, c, part, outt, st);
    return hipGetLastError();
}

hipError_t launch_i8_tiled_grouped(const I8Args &a, const I8Groups &g, int outt, hipStream_t st)
{
    using S = TiMid;
    const int cols = a.Nh ? 2 * a.Nh : a.N;
    const int ntiles = (cols + S::BN - 1) / S::BN;
    // an expert adds at most one partial tile, and at most B experts have rows
    const int64_t tiles = a.B / S::BM + (g.E < a.B ? g.E : a.B);
    const dim3 grid((unsigned)(tiles * ntiles)), blk(64 * S::NW);
    if (a.Nh && outt == OUT_F32)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, true, OUT_F32>), grid, blk, 0, st, a, g, ntiles);
    else if (a.Nh)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, true, OUT_BF16>), grid, blk, 0, st, a, g, ntiles);
    else if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, false, OUT_F32>), grid, blk, 0, st, a, g, ntiles);
    else
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, false, OUT_BF16>), grid, blk, 0, st, a, g, ntiles);
    return hipGetLastError();
}

}  // namespace qg
