// 8-bit products with many rows: BM batch rows x BN channels a workgroup, both
// operands staged through LDS by gfx950's direct loads, int32 accumulators.
//
// A step is 64 k.  A packed weight slab is 1 KB in the order in which the lanes
// of a wave take it, so its load and its read are a contiguous KB each.  Rows of
// codes are loaded 128 k at a time, whole cache lines (64-byte halves of them,
// one a step, cost each line twice: 400 against 330 us at 2048 x 34816 x 5120):
// a KB holds 8 rows x 128 k, with the eight 16-byte pieces of row r in the order
// p ^ swizzle(r), so that the 16 lanes that read one k group of 16 rows together
// find 16 different bank groups.  Nothing is decoded, shuffled or staged in
// registers on the way.
//
// Four steps of weights and two double steps of codes are in LDS.  While a step
// is multiplied, the next one's operands are read into registers and the loads
// of the ones after it are in flight: a step's matrix time is far below the
// latency of a load.  One barrier a step: it says that the next step has landed
// (each wave waits for its own loads of it, and leaves the later ones in flight)
// and that the present one is in every wave's registers, so that its place can
// be loaded into again.  The same loads are issued in every fourth step, those
// past the last step from an empty resource, so the counts waited for are exact.
#include "int8.h"

namespace qg {

template <int WM_, int WN_, int TM_, int TN_>
struct TiShape {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;  // waves, and 16-wide tiles a wave
    static constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
    // KBs of a double step of codes (the same number for each wave: copies of
    // the last row past BM) and of a step of weights
    static constexpr int XC = (BM / 8 + NW - 1) / NW * NW, WC = BN / 16;
    static constexpr int XPW = XC / NW, WPW = WC / NW;  // of them a wave loads
    static constexpr int XST = XC * 1024, WST = WC * 1024;
    static_assert(XC % NW == 0 && WC % NW == 0, "whole KBs a wave");
};
using TiBig = TiShape<2, 4, 8, 4>;  // 256 x 256, 8 waves of 128 x 64
using TiMid = TiShape<2, 2, 4, 4>;  // 128 x 128, 4 waves of 64 x 64
using TiWide = TiShape<1, 4, 5, 4>;  // 80 x 256, 4 waves of 80 x 64
using TiLow = TiShape<2, 2, 2, 4>;  // 64 x 128, 4 waves of 32 x 64
using TiFew = TiShape<1, 4, 2, 2>;  // 32 x 128, 4 waves of 32 x 32
using TiOne = TiShape<1, 4, 1, 2>;  // 16 x 128, 4 waves of 16 x 32

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

// Waits until at most N of this wave's loads are in flight and its LDS reads are
// done, then for the other waves.  Nothing moves across it.
template <int N>
__device__ __forceinline__ void step_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The order of a step's instructions: its loads (as many as wanted), then a read
// every other matrix instruction, so that neither waits for the other.
template <int LOADS, int READS, int MFMAS>
__device__ __forceinline__ void ti_interleave()
{
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // a load
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction
    }
    constexpr int PER = (MFMAS - LOADS) / READS > 0 ? (MFMAS - LOADS) / READS : 1;
#pragma unroll
    for (int i = 0; i < READS; i++) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// LDS of a workgroup.  Every buffer is an array of its own in the kernels: the
// compiler tells the loads into one from the reads of another by the array.
struct TiLds {
    uint8_t *x[2], *w[4];
};
#define TI_LDS(S, L)                                                                      \
    __shared__ __attribute__((aligned(1024))) uint8_t ldx0[S::XST], ldx1[S::XST];         \
    __shared__ __attribute__((aligned(1024))) uint8_t ldw0[S::WST], ldw1[S::WST];         \
    __shared__ __attribute__((aligned(1024))) uint8_t ldw2[S::WST], ldw3[S::WST];         \
    const TiLds L = {{ldx0, ldx1}, {ldw0, ldw1, ldw2, ldw3}}

__device__ __forceinline__ int x_swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// One tile: rows row0 .. row0+rows-1 (at most BM), weight tile nt, steps k0 .. k1-1
// (a multiple of 4).
template <typename S, bool DUAL>
__device__ __forceinline__ void ti_tile_sums(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int k0,
                                             int k1, const TiLds &lds, i32x4 (&acc)[S::TM][S::TN])
{
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid / S::WN, wn = wid % S::WN;
    const int64_t tile_bytes = (int64_t)a.S << 10;

    // what this wave loads: KBs of codes (rows past the last are copies of it)
    // and weight tiles
    const uint8_t *xbase = (const uint8_t *)a.codes + row0 * a.ldc;
    const int64_t xbytes = (int64_t)rows * a.ldc;
    int xo[S::XPW];
#pragma unroll
    for (int c = 0; c < S::XPW; c++) {
        const int r = (wid * S::XPW + c) * 8 + (lane >> 3);
        xo[c] = min(r, rows - 1) * a.ldc + (((lane & 7) ^ x_swizzle(r)) << 4);
    }
    const uint8_t *wbase[S::WPW];
#pragma unroll
    for (int c = 0; c < S::WPW; c++)
        wbase[c] = w + ti_tile<S, DUAL>(a, nt, wid * S::WPW + c) * tile_bytes;

    auto load_x = [&](int kt, uint8_t *to) {  // the double step kt, kt + 1
        const bool live = kt < k1;
        const __amdgpu_buffer_rsrc_t xr = make_rsrc(xbase, live ? xbytes : 0);
#pragma unroll
        for (int c = 0; c < S::XPW; c++)
            load_chunk(xr, to + (wid * S::XPW + c) * 1024, xo[c], live ? kt << 6 : 0);
    };
    auto load_w = [&](int kt, uint8_t *to) {
        const bool live = kt < k1;
#pragma unroll
        for (int c = 0; c < S::WPW; c++)
            load_chunk(make_rsrc(wbase[c], live ? tile_bytes : 0), to + (wid * S::WPW + c) * 1024, lane * 16,
                       live ? kt << 10 : 0);
    };
    i32x4 xf[2][S::TM], wf[2][S::TN];
    // row r = lane % 16 of a group of 16 and its k group, in the even step; the
    // odd step's piece is 4 further on, which the swizzle leaves a flip of one bit
    const int r16 = lane & 15;
    const int xl = wm * S::TM * 2048 + r16 * 128 + (((lane >> 4) ^ x_swizzle(r16)) << 4);
    auto read = [&](const uint8_t *x, const uint8_t *wt, int odd, int to) {
        const uint8_t *wl = wt + wn * S::TN * 1024 + lane * 16;
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            wf[to][j] = *(const i32x4 *)(wl + j * 1024);
#pragma unroll
        for (int i = 0; i < S::TM; i++)
            xf[to][i] = *(const i32x4 *)(x + (xl ^ (odd << 6)) + i * 2048);
    };
#pragma unroll
    for (int i = 0; i < S::TM; i++)
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            acc[i][j] = i32x4{0, 0, 0, 0};
    // in the order that the loop keeps: a step's weights, then (odd steps) codes
    load_x(k0, lds.x[0]);
    load_w(k0, lds.w[0]);
    load_w(k0 + 1, lds.w[1]);
    load_x(k0 + 2, lds.x[1]);
    load_w(k0 + 2, lds.w[2]);
    load_w(k0 + 3, lds.w[3]);
    step_barrier<S::XPW + 3 * S::WPW>();
    read(lds.x[0], lds.w[0], 0, 0);
    for (int kt = k0; kt < k1; kt += 4) {
#pragma unroll
        for (int u = 0; u < 4; u++) {
            // Even steps wait for the next step's weights, with two steps'
            // weights and one load of codes issued after them; odd steps for
            // the next double step of codes too, with one step's weights after.
            if (u & 1)
                step_barrier<S::WPW>();
            else
                step_barrier<S::XPW + 2 * S::WPW>();
            load_w(kt + u + 4, lds.w[u]);
            if (u & 1)
                load_x(kt + u + 3, lds.x[u / 2]);
            read(lds.x[(u + 1) / 2 % 2], lds.w[(u + 1) % 4], (u + 1) & 1, (u + 1) & 1);
#pragma unroll
            for (int i = 0; i < S::TM; i++)
#pragma unroll
                for (int j = 0; j < S::TN; j++)
                    acc[i][j] = mfma_i8(wf[u & 1][j], xf[u & 1][i], acc[i][j]);
            if (u & 1)
                ti_interleave<S::WPW + S::XPW, S::TM + S::TN, S::TM * S::TN>();
            else
                ti_interleave<S::WPW, S::TM + S::TN, S::TM * S::TN>();
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load outlives the workgroup's LDS
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
__global__ __launch_bounds__(64 * S::NW, 2) void i8_tiled_kernel(I8Args a, int mtiles, int ntiles,
                                                                                int split, int32_t *part)
{
    TI_LDS(S, lds);
    const int t = xcd_order(blockIdx.x, gridDim.x);
    const int tile = t / split, piece = t % split;
    const int mt = tile % mtiles, nt = tile / mtiles;
    const int steps = a.S, per = (steps / 4 + split - 1) / split * 4;
    const int k0 = piece * per, k1 = min(steps, k0 + per);
    const int64_t row0 = (int64_t)mt * S::BM;
    const int rows = min(S::BM, (int)(a.B - row0));
    i32x4 acc[S::TM][S::TN];
    ti_tile_sums<S, DUAL>(a, a.w, row0, rows, nt, k0, k1, lds, acc);
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

// Rows sorted by expert: the grid covers a bound on the experts' row tiles, each
// with its weight tiles; a workgroup finds its expert by a scan of the experts'
// row-tile counts, and those past the real count leave.  Row tiles are dealt to
// the XCDs in turn (the real ones are the first of the bound, so runs of them
// would leave half of the XCDs idle), a row tile's weight tiles to one XCD.
template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * S::NW, 2) void i8_tiled_grouped_kernel(I8Args a, I8Groups grp, int ntiles)
{
    TI_LDS(S, lds);
    __shared__ int wsum[S::NW], found[4];
    constexpr int NT = 64 * S::NW;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int loc = blockIdx.x / 8;
    const int mt = loc / ntiles * 8 + blockIdx.x % 8, nt = loc % ntiles;  // row tile over all experts
    // PER neighbouring experts a thread: up to NT * PER of them with one wait for
    // their offsets
    constexpr int PER = 4;
    if (tid == 0)
        found[0] = -1;
    int carry = 0;
    for (int e0 = 0; e0 < grp.E; e0 += NT * PER) {
        int off[PER + 1], cnt[PER], v = 0;
#pragma unroll
        for (int k = 0; k <= PER; k++)
            off[k] = grp.off[min(e0 + tid * PER + k, grp.E)];
#pragma unroll
        for (int k = 0; k < PER; k++) {
            const int e = e0 + tid * PER + k;
            if (e < grp.E && (off[k] < 0 || off[k + 1] < off[k] || off[k + 1] > a.B || (e == 0 && off[k] != 0))) {
                cnt[k] = 0;
                if (blockIdx.x == 0)
                    __hip_atomic_fetch_or(grp.status, DEV_BAD_OFFSETS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            } else {
                cnt[k] = (off[k + 1] - off[k] + S::BM - 1) / S::BM;  // 0 past the last expert
            }
            v += cnt[k];
        }
        int s = v;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d)
                s += o;
        }
        if (lane == 63)
            wsum[wid] = s;
        __syncthreads();
        int first = carry + s - v;
        for (int k = 0; k < S::NW; k++) {
            first += k < wid ? wsum[k] : 0;
            carry += wsum[k];
        }
#pragma unroll
        for (int k = 0; k < PER; k++) {
            if (mt >= first && mt < first + cnt[k]) {
                found[0] = e0 + tid * PER + k;
                found[1] = off[k] + (mt - first) * S::BM;
                found[2] = off[k + 1];
            }
            first += cnt[k];
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
    ti_tile_sums<S, DUAL>(a, w, row0, rows, nt, 0, a.S, lds, acc);
#pragma unroll
    for (int i = 0; i < S::TM; i++)
        ti_store<S, DUAL, OUTT>(a, w, row0, rows, nt, wid / S::WN, wid % S::WN, lane, i, acc[i]);
}

// ------------------------------------------------------------------ host

// Whole tiles of the larger shape when they fill the chip, else the smaller
// one, K split so that at least a round of tiles runs.
I8TiCfg i8_tiled_cfg(const I8Args &a, bool split, int bm, int forced)
{
    I8TiCfg c;
    const int cols = a.Nh ? 2 * a.Nh : a.N;
    const int64_t big = (int64_t)((a.B + 255) / 256) * ((cols + 255) / 256);
    c.BM = bm ? bm : big >= 192 ? 256 : 128;
    c.BN = c.BM == 80 || c.BM == 256 ? 256 : 128;
    c.mtiles = (a.B + c.BM - 1) / c.BM;
    c.ntiles = (cols + c.BN - 1) / c.BN;
    const int64_t tiles = (int64_t)c.mtiles * c.ntiles;
    const int steps = a.S / 4;  // in fours, as the kernel walks them
    c.split = 1;
    if (split && tiles < 256) {
        int s = (int)(512 / tiles);
        s = s > steps / 2 ? steps / 2 : s;
        s = s < 1 ? 1 : s;
        if (forced) s = forced > steps ? steps : forced;
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
    switch (c.BM) {
    case 32: tiled_shape<TiFew>(a, c, part, outt, st); break;
    case 64: tiled_shape<TiLow>(a, c, part, outt, st); break;
    case 80: tiled_shape<TiWide>(a, c, part, outt, st); break;
    case 128: tiled_shape<TiMid>(a, c, part, outt, st); break;
    default: tiled_shape<TiBig>(a, c, part, outt, st); break;
    }
    return hipGetLastError();
}

template <typename S>
static void grouped_go(const I8Args &a, const I8Groups &g, int outt, hipStream_t st)
{
    const int cols = a.Nh ? 2 * a.Nh : a.N;
    const int ntiles = (cols + S::BN - 1) / S::BN;
    // an expert adds at most one partial tile, and at most B experts have rows
    const int64_t tiles = a.B / S::BM + (g.E < a.B ? g.E : a.B);
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8 * ntiles)), blk(64 * S::NW);
    if (a.Nh && outt == OUT_F32)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, true, OUT_F32>), grid, blk, 0, st, a, g, ntiles);
    else if (a.Nh)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, true, OUT_BF16>), grid, blk, 0, st, a, g, ntiles);
    else if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, false, OUT_F32>), grid, blk, 0, st, a, g, ntiles);
    else
        hipLaunchKernelGGL((i8_tiled_grouped_kernel<S, false, OUT_BF16>), grid, blk, 0, st, a, g, ntiles);
}

hipError_t launch_i8_grouped(const I8Args &a, const I8Groups &g, int bm, int outt, hipStream_t st)
{
    switch (bm) {
    case 16: grouped_go<TiOne>(a, g, outt, st); break;
    case 32: grouped_go<TiFew>(a, g, outt, st); break;
    case 64: grouped_go<TiLow>(a, g, outt, st); break;
    default: grouped_go<TiMid>(a, g, outt, st); break;
    }
    return hipGetLastError();
}

}  // namespace qg
