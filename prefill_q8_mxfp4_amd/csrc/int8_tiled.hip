// 8-bit products with many rows: BM batch rows x BN channels a workgroup, both
// operands staged through LDS by gfx950's direct loads, int32 accumulators.
//
// A step is 64 k.  A packed weight slab is 1 KB in the order in which the lanes
// of a wave take it, so its load and its read are a contiguous KB each.  Rows of
// codes are loaded 128 k at a time, whole cache lines (64-byte halves of them,
// one a step, cost each line twice: 401 against 345 us at 2048 x 34816 x 5120):
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

template <int WM_, int WN_, int TM_, int TN_, int NE_ = 0>
struct TiShape {
    static constexpr int NE = NE_;  // double steps of the ring, 0: the large tile's loop
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;  // waves, and 16-wide tiles a wave
    static constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
    // KBs of a double step of codes (the same number for each wave: copies of
    // the last row past BM) and of a step of weights
    static constexpr int XC = (BM / 8 + NW - 1) / NW * NW, WC = BN / 16;
    static constexpr int XPW = XC / NW, WPW = WC / NW;  // of them a wave loads
    static constexpr int XST = XC * 1024, WST = WC * 1024;
    // LDS that a wave has to itself for its outputs, and the row groups that fit
    static constexpr int OUT = NE ? (NW > NE ? (XST + 2 * WST) / 2 : XST + 2 * WST)
                             : NW > 4 ? (WST < XST / 2 ? WST : XST / 2) : WST;
    static constexpr int FIT = OUT / (TN * 1024) < 4 ? OUT / (TN * 1024) : 4, GP = FIT < TM ? FIT : TM;
    static_assert(GP >= 1 && GP <= 4 && TM % GP == 0 && (TN == 2 || TN == 4), "whole passes of at most 64 rows");
    static_assert(XC % NW == 0 && WC % NW == 0, "whole KBs a wave");
};
// Rows x channels; see i8_tiled_cfg and i8_grouped_shape for which is taken when.
using T32x32 = TiShape<2, 1, 1, 2, 8>;
using T32x64 = TiShape<2, 2, 1, 2, 8>;
using T64x64 = TiShape<2, 2, 2, 2, 8>;
using T64x128 = TiShape<2, 2, 2, 4>;
using T64x128R = TiShape<2, 4, 2, 2, 4>;
using T128x128R = TiShape<2, 4, 4, 2, 4>;
using T128x256 = TiShape<2, 4, 4, 4>;
using T256x256 = TiShape<2, 4, 8, 4>;
using T32x128 = TiShape<1, 4, 2, 2>;   // routed rows only
using T128x128 = TiShape<2, 4, 4, 2>;  // routed rows only

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

// Outputs of one lane for row group i, straight from its sums.
template <typename S, bool DUAL, int OUTT>
__device__ __forceinline__ void ti_store(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int wm,
                                         int wn, int lane, int i, const i32x4 (&acc)[S::TN])
{
    const float *ws = (const float *)(w + a.scale_off);
    constexpr int TO = DUAL ? S::TN / 2 : S::TN;
    const int b = (wm * S::TM + i) * 16 + (lane & 15);
    const int n0 = (nt * S::WN + wn) * TO * 16 + (lane >> 4) * 4;
    if (b >= rows)
        return;
    const float xs = a.xs[row0 + b];
    f32x4 t[TO], tu[TO];  // all read before the first store, which a later read would wait for
#pragma unroll
    for (int j = 0; j < TO; j++) {
        const int n = n0 + j * 16 < a.ncols ? n0 + j * 16 : 0;
        t[j] = *(const f32x4 *)(ws + n);
        if constexpr (DUAL)
            tu[j] = *(const f32x4 *)(ws + a.Nh + n);
    }
#pragma unroll
    for (int j = 0; j < TO; j++) {
        const int n = n0 + j * 16;
        f32x4 o;
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = (float)acc[j][k] * xs * t[j][k];
        if constexpr (DUAL) {
#pragma unroll
            for (int k = 0; k < 4; k++)
                o[k] = silu(o[k]) * ((float)acc[j + TO][k] * xs * tu[j][k]);
        }
        i8_put4_part<OUTT>((uint8_t *)a.y + ((row0 + b) * a.ncols + n) * (OUTT == OUT_F32 ? 4 : 2), o, a.ncols - n);
    }
}

// The scales of a wave's outputs: of its lane's four channels (the same in every
// pass) and of the rows of each pass, a row a lane.  Read before the sums, so that
// no read waits behind a store.
template <typename S, bool DUAL>
struct TiScales {
    static constexpr int TO = DUAL ? S::TN / 2 : S::TN, LPR = TO * 4, GR = S::GP * 16;
    f32x4 t, tu;
    float xs[S::TM / S::GP];
    __device__ __forceinline__ TiScales(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt)
    {
        const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
        const int n = (nt * S::WN + wid % S::WN) * TO * 16 + lane % LPR * 4;
        const float *ws = (const float *)(w + a.scale_off) + (n < a.ncols ? n : 0);
        t = tu = *(const f32x4 *)ws;
        if constexpr (DUAL)
            tu = *(const f32x4 *)(ws + a.Nh);
#pragma unroll
        for (int p = 0; p < S::TM / S::GP; p++)
            xs[p] = a.xs[row0 + min((wid / S::WN * S::TM + p * S::GP) * 16 + (lane < GR ? lane : 0), rows - 1)];
    }
};

// A wave's outputs, GP row groups at a time through its own LDS `own`: the lanes
// give their sums there (row by row, the 16-byte pieces of a row swizzled so that
// neither side meets bank conflicts) and take them back a row of the tile after
// the other, so that a store is whole cache lines and the code for it is a short
// loop.  A call of one 256 x 256 tile over K = 256 took 12.8 us straight from the
// accumulators (some 6 KB of code that runs once) and takes 10.0 so.
template <typename S, bool DUAL, int OUTT>
__device__ __forceinline__ void ti_finish(const I8Args &a, const TiScales<S, DUAL> &sc, int64_t row0, int rows, int nt,
                                          uint8_t *own, const i32x4 (&acc)[S::TM][S::TN])
{
    constexpr int TO = DUAL ? S::TN / 2 : S::TN, OSZ = OUTT == OUT_F32 ? 4 : 2;
    constexpr int PITCH = S::TN * 64, LPR = TO * 4, RPI = 64 / LPR, GR = S::GP * 16;
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid / S::WN, wn = wid % S::WN;
    const int c = lane % LPR, r = lane / LPR;
    const int n = (nt * S::WN + wn) * TO * 16 + c * 4, left = a.ncols - n;
    const f32x4 t = sc.t, tu = sc.tu;
    auto piece = [](int row, int q) { return row * PITCH + ((q ^ (S::TN == 4 ? row & 15 : (row >> 1) & 7)) << 4); };
#pragma unroll
    for (int p = 0; p < S::TM / S::GP; p++) {
        const int b0 = (wm * S::TM + p * S::GP) * 16;
        if (b0 >= rows)
            break;  // uniform
#pragma unroll
        for (int i = 0; i < S::GP; i++)
#pragma unroll
            for (int j = 0; j < S::TN; j++)
                *(i32x4 *)(own + piece(i * 16 + (lane & 15), j * 4 + (lane >> 4))) = acc[p * S::GP + i][j];
        uint8_t *to = (uint8_t *)a.y + ((row0 + b0 + r) * a.ncols + n) * OSZ;
        const int64_t next = (int64_t)a.ncols * RPI * OSZ;
        auto out = [&](int row) {
            const i32x4 g = *(const i32x4 *)(own + piece(row, c));
            const float xs = __shfl(sc.xs[p], row);
            f32x4 o;
#pragma unroll
            for (int e = 0; e < 4; e++)
                o[e] = (float)g[e] * xs * t[e];
            if constexpr (DUAL) {
                const i32x4 u = *(const i32x4 *)(own + piece(row, c + LPR));
#pragma unroll
                for (int e = 0; e < 4; e++)
                    o[e] = silu(o[e]) * ((float)u[e] * xs * tu[e]);
            }
            return o;
        };
        if (b0 + GR <= rows && n - c * 4 + TO * 16 <= a.ncols) {  // uniform: all inside, four rows' reads at once
#pragma unroll 4
            for (int k = 0; k < GR / RPI; k++, to += next)
                i8_put4<OUTT>(to, out(k * RPI + r));
        } else {
            for (int k = 0; k < GR / RPI; k++, to += next) {
                const f32x4 o = out(k * RPI + r);
                if (b0 + k * RPI + r < rows)
                    i8_put4_part<OUTT>(to, o, left);
            }
        }
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

// Rows 2 m and 2 m + 1 take m: then the pieces of one k group of 16 rows lie in 16
// different 16-byte bank groups, and so do those of rows 0-3 and 12-15 of one k
// group with rows 4-11 of the next, which a 16-byte read takes together.
// (r & 7 with r's bit 3 flipping the lowest does only the first: 39 % of the LDS
// cycles were conflicts.)
__device__ __forceinline__ int x_swizzle(int r) { return (r >> 1) & 7; }

// What a wave loads of a tile: KBs of codes (rows past the last are copies of it)
// and weight tiles; steps from `end` on come from an empty resource.
template <typename S, bool DUAL>
struct TiLoads {
    const uint8_t *xbase, *wbase[S::WPW];
    int64_t xbytes, tile_bytes;
    int xo[S::XPW], wo, wid, end;

    __device__ __forceinline__ TiLoads(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int end_)
        : xbase((const uint8_t *)a.codes + row0 * a.ldc), xbytes((int64_t)rows * a.ldc),
          tile_bytes((int64_t)a.S << 10), wo((threadIdx.x & 63) * 16),
          wid(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), end(end_)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int c = 0; c < S::XPW; c++) {
            const int r = (wid * S::XPW + c) * 8 + (lane >> 3);
            xo[c] = min(r, rows - 1) * a.ldc + (((lane & 7) ^ x_swizzle(r)) << 4);
        }
#pragma unroll
        for (int c = 0; c < S::WPW; c++)
            wbase[c] = w + ti_tile<S, DUAL>(a, nt, wid * S::WPW + c) * tile_bytes;
    }
    // the codes of the double step kt, kt + 1
    __device__ __forceinline__ void x(int kt, uint8_t *to) const
    {
        const bool live = kt < end;
        const __amdgpu_buffer_rsrc_t xr = make_rsrc(xbase, live ? xbytes : 0);
#pragma unroll
        for (int c = 0; c < S::XPW; c++)
            load_chunk(xr, to + (wid * S::XPW + c) * 1024, xo[c], live ? kt << 6 : 0);
    }
    // the weights of step kt
    __device__ __forceinline__ void w(int kt, uint8_t *to) const
    {
        const bool live = kt < end;
#pragma unroll
        for (int c = 0; c < S::WPW; c++)
            load_chunk(make_rsrc(wbase[c], live ? tile_bytes : 0), to + (wid * S::WPW + c) * 1024, wo,
                       live ? kt << 10 : 0);
    }
};

// One tile: rows row0 .. row0+rows-1 (at most BM), weight tile nt, steps k0 .. k1-1
// (a multiple of 4).
template <typename S, bool DUAL>
__device__ __forceinline__ void ti_tile_sums(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int k0,
                                             int k1, const TiLds &lds, i32x4 (&acc)[S::TM][S::TN])
{
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid / S::WN, wn = wid % S::WN;
    const TiLoads<S, DUAL> ld(a, w, row0, rows, nt, k1);
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
    ld.x(k0, lds.x[0]);
    ld.w(k0, lds.w[0]);
    ld.w(k0 + 1, lds.w[1]);
    ld.x(k0 + 2, lds.x[1]);
    ld.w(k0 + 2, lds.w[2]);
    ld.w(k0 + 3, lds.w[3]);
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
            ld.w(kt + u + 4, lds.w[u]);
            if (u & 1)
                ld.x(kt + u + 3, lds.x[u / 2]);
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
    step_barrier<0>();  // no load outlives this, and every wave is done with the stages
}

// The same sums for small tiles, whose steps take less time than a barrier and an
// LDS read: a ring of NE double steps, all but one of them in flight, one barrier
// a double step.
template <typename S, bool DUAL, int NE>
__device__ __forceinline__ void ti_deep_sums(const I8Args &a, const uint8_t *w, int64_t row0, int rows, int nt, int k0,
                                             int k1, uint8_t *const (&ring)[NE], i32x4 (&acc)[S::TM][S::TN])
{
    constexpr int LPE = S::XPW + 2 * S::WPW;  // loads a wave issues each double step
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wid / S::WN, wn = wid % S::WN;
    const TiLoads<S, DUAL> ld(a, w, row0, rows, nt, k1);
    auto load = [&](int kt, uint8_t *to) {
        ld.x(kt, to);
        ld.w(kt, to + S::XST);
        ld.w(kt + 1, to + S::XST + S::WST);
    };
    const int r16 = lane & 15;
    const int xl = wm * S::TM * 2048 + r16 * 128 + (((lane >> 4) ^ x_swizzle(r16)) << 4);
    const int wl = S::XST + wn * S::TN * 1024 + lane * 16;
#pragma unroll
    for (int i = 0; i < S::TM; i++)
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < NE - 1; u++)
        load(k0 + 2 * u, ring[u]);
    auto step = [&](int kt, int u) {  // double step kt, in ring[u]
        step_barrier<LPE *(NE - 2)>();
        load(kt + 2 * (NE - 1), ring[(u + NE - 1) % NE]);
        const uint8_t *at = ring[u];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            i32x4 xf[S::TM], wf[S::TN];
#pragma unroll
            for (int j = 0; j < S::TN; j++)
                wf[j] = *(const i32x4 *)(at + wl + h * S::WST + j * 1024);
#pragma unroll
            for (int i = 0; i < S::TM; i++)
                xf[i] = *(const i32x4 *)(at + (xl ^ (h << 6)) + i * 2048);
#pragma unroll
            for (int i = 0; i < S::TM; i++)
#pragma unroll
                for (int j = 0; j < S::TN; j++)
                    acc[i][j] = mfma_i8(wf[j], xf[i], acc[i][j]);
        }
    };
    int kt = k0;
    for (; kt + 2 * NE <= k1; kt += 2 * NE) {
#pragma unroll
        for (int u = 0; u < NE; u++)
            step(kt + 2 * u, u);
    }
    // the rest, in pairs of double steps
#pragma unroll
    for (int u = 0; u < NE - 2; u += 2) {
        if (kt + 2 * u < k1) {  // uniform
            step(kt + 2 * u, u);
            step(kt + 2 * u + 2, u + 1);
        }
    }
    step_barrier<0>();  // no load outlives this, and every wave is done with the stages
}

// A wave's own LDS once the stages are done with.
template <typename S>
__device__ __forceinline__ uint8_t *ti_own(const TiLds &l, int wid)
{
    if (wid < 4)
        return wid == 0 ? l.w[0] : wid == 1 ? l.w[1] : wid == 2 ? l.w[2] : l.w[3];
    return (wid < 6 ? l.x[0] : l.x[1]) + (wid & 1) * (S::XST / 2);
}

// The sums of one tile in the way its shape has them, and the wave's own LDS after.
#define TI_SUMS(S, DUAL, ...)                                                                                       \
    uint8_t *own;                                                                                                   \
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);                                              \
    if constexpr (S::NE == 0) {                                                                                     \
        TI_LDS(S, lds);                                                                                             \
        ti_tile_sums<S, DUAL>(__VA_ARGS__, lds, acc);                                                               \
        own = ti_own<S>(lds, wave);                                                                                 \
    } else {                                                                                                        \
        constexpr int RB = S::XST + 2 * S::WST, R8 = S::NE > 4 ? RB : 16;                                           \
        __shared__ __attribute__((aligned(1024))) uint8_t r0[RB], r1[RB], r2[RB], r3[RB];                           \
        __shared__ __attribute__((aligned(1024))) uint8_t r4[R8], r5[R8], r6[R8], r7[R8];                           \
        if constexpr (S::NE == 4) {                                                                                 \
            uint8_t *const ring[4] = {r0, r1, r2, r3};                                                              \
            ti_deep_sums<S, DUAL, 4>(__VA_ARGS__, ring, acc);                                                       \
        } else {                                                                                                    \
            uint8_t *const ring[8] = {r0, r1, r2, r3, r4, r5, r6, r7};                                              \
            ti_deep_sums<S, DUAL, 8>(__VA_ARGS__, ring, acc);                                                       \
        }                                                                                                           \
        const int at = S::NW > S::NE ? wave / 2 : wave;                                                             \
        own = (at == 0 ? r0 : at == 1 ? r1 : at == 2 ? r2 : r3) + (S::NW > S::NE ? (wave & 1) * (RB / 2) : 0);      \
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

// One whole tile of shape S in LDS made for a shape at least as large.
template <typename S, bool DUAL, int OUTT>
__device__ __forceinline__ void ti_whole(const I8Args &a, int mt, int nt, const TiLds &lds)
{
    const int64_t row0 = (int64_t)mt * S::BM;
    const int rows = min(S::BM, (int)(a.B - row0));
    if (rows <= 0 || nt * (S::BN / (DUAL ? 2 : 1)) >= a.ncols)
        return;  // uniform: a piece of a tile that lies outside
    i32x4 acc[S::TM][S::TN];
    const TiScales<S, DUAL> sc(a, a.w, row0, rows, nt);
    ti_tile_sums<S, DUAL>(a, a.w, row0, rows, nt, 0, a.S, lds, acc);
    ti_finish<S, DUAL, OUTT>(a, sc, row0, rows, nt,
                             ti_own<S>(lds, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), acc);
}

// 256 x 256 tiles: the first `full` whole, the others as PIECES (1, 2 or 4)
// smaller ones each.  Whole rounds of 256 tiles run first; a last, partial round
// of whole tiles would leave most of the chip idle for a tile's time, its pieces
// share it out.
template <int PIECES, bool DUAL, int OUTT>
__global__ __launch_bounds__(512, 2) void i8_big_kernel(I8Args a, int mtiles, int ntiles, int full)
{
    TI_LDS(T256x256, lds);
    using P = TiShape<2, 4, PIECES == 1 ? 8 : 4, PIECES == 4 ? 2 : 4>;
    constexpr int PM = T256x256::BM / P::BM, PN = T256x256::BN / P::BN;
    if (blockIdx.x < full) {
        const int t = xcd_order(blockIdx.x, full);
        ti_whole<T256x256, DUAL, OUTT>(a, t % mtiles, t / mtiles, lds);
    } else {
        const int t = xcd_order(blockIdx.x - full, gridDim.x - full), tile = full + t / PIECES, p = t % PIECES;
        ti_whole<P, DUAL, OUTT>(a, tile % mtiles * PM + p % PM, tile / mtiles * PN + p / PM, lds);
    }
}

template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * S::NW, 2) void i8_tiled_kernel(I8Args a, int mtiles, int ntiles,
                                                                                int split, int32_t *part)
{
    const int t = xcd_order(blockIdx.x, gridDim.x);
    const int tile = t / split, piece = t % split;
    const int mt = tile % mtiles, nt = tile / mtiles;
    const int steps = a.S, per = (steps / 4 + split - 1) / split * 4;
    const int k0 = piece * per, k1 = min(steps, k0 + per);
    const int64_t row0 = (int64_t)mt * S::BM;
    const int rows = min(S::BM, (int)(a.B - row0));
    i32x4 acc[S::TM][S::TN];
    const TiScales<S, DUAL> sc(a, a.w, row0, rows, nt);
    TI_SUMS(S, DUAL, a, a.w, row0, rows, nt, k0, k1)
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
    ti_finish<S, DUAL, OUTT>(a, sc, row0, rows, nt, own, acc);
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
    i32x4 acc[1][S::TN];
#pragma unroll
    for (int j = 0; j < S::TN; j++)
        acc[0][j] = i32x4{0, 0, 0, 0};
    if ((wid / S::WN * S::TM + i) * 16 >= rows)
        return;
    for (int p = 0; p < split; p++) {
        const i32x4 *q = (const i32x4 *)part + (((int64_t)tile * split + p) * S::NW + wid) * S::TM * S::TN * 64;
#pragma unroll
        for (int j = 0; j < S::TN; j++)
            acc[0][j] += q[(i * S::TN + j) * 64 + lane];
    }
    ti_store<S, DUAL, OUTT>(a, a.w, row0, rows, nt, wid / S::WN, wid % S::WN, lane, i, acc[0]);
}

// Rows sorted by expert: the grid covers a bound on the experts' row tiles, each
// with its weight tiles; a workgroup finds its expert by a scan of the experts'
// row-tile counts, and those past the real count leave.  Row tiles are dealt to
// the XCDs in turn (the real ones are the first of the bound, so runs of them
// would leave half of the XCDs idle), a row tile's weight tiles to one XCD, `per`
// of them to a workgroup.
template <typename S, bool DUAL, int OUTT>
__global__ __launch_bounds__(64 * S::NW, 2) void i8_grouped_kernel(I8Args a, I8Groups grp, int ntiles,
                                                                     int per)
{
    __shared__ int wsum[S::NW], found[4];
    constexpr int NT = 64 * S::NW;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
    const int loc = blockIdx.x / 8;
    const int groups = (ntiles + per - 1) / per;
    const int mt = loc / groups * 8 + blockIdx.x % 8;  // row tile over all experts
    const int nt0 = loc % groups * per;
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
        if (found[0] >= 0 && blockIdx.x)
            break;  // uniform; the first workgroup looks at every expert's offsets
    }
    const int e = __builtin_amdgcn_readfirstlane(found[0]);
    if (e < 0)
        return;
    const int row0 = __builtin_amdgcn_readfirstlane(found[1]);
    const int rows = min(S::BM, __builtin_amdgcn_readfirstlane(found[2]) - row0);
    if (rows <= 0)
        return;  // bad offsets whose counts passed 32 bits
    const uint8_t *w = uniform_ptr(grp.wtab[e]);
    TI_LDS(S, lds);
    for (int nt = nt0; nt < min(nt0 + per, ntiles); nt++) {
        if (nt > nt0)
            __syncthreads();  // every wave is done with its outputs' LDS
        i32x4 acc[S::TM][S::TN];
        const TiScales<S, DUAL> sc(a, w, row0, rows, nt);
        ti_tile_sums<S, DUAL>(a, w, row0, rows, nt, 0, a.S, lds, acc);
        ti_finish<S, DUAL, OUTT>(a, sc, row0, rows, nt,
                                 ti_own<S>(lds, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), acc);
    }
}

// ------------------------------------------------------------------ host

// What a call costs with a shape, in us, fitted to times on MI355X (K = 256 to
// 17408; 5 to 35000 channels, 1 to 4096 rows; within 10 % of nearly all of them).
// A workgroup takes `fixed` for its first loads and its outputs and a step's time
// for each 64 k; that time grows with the workgroups at work, for their share of
// L2 and of the clock: step[0] with up to 128 of them, step[1] with 256, step[2]
// with all that the CUs hold.  Choices it makes, with the runner-up: 16 x 5120 x
// 5120 32x32 7.5 (32x64 8.4); 70 x 5120 x 17408 32x64 28 (128x128R, split, 28;
// 64x64 31); 128 x 5120 x 5120 64x64 11.2 (64x128R 13.9); 256: 64x128R 14.6
// (128x128R 19); 512: 128x128R 20 (64x128 24); 1024: 128x256 32 (64x128 39); 2048:
// 256x256 54 (128x128R 64).
struct ShapeCost {
    int BM, BN, resident;  // workgroups a CU holds
    float fixed, step[3];
};
static const ShapeCost COST[] = {
    {0, 0, 0, 0.f, {0.f, 0.f, 0.f}},
    {32, 32, 2, 1.0f, {0.067f, 0.075f, 0.110f}},    // I8_32x32
    {32, 64, 1, 0.3f, {0.085f, 0.092f, 0.092f}},    // I8_32x64
    {64, 64, 1, 0.8f, {0.103f, 0.112f, 0.112f}},    // I8_64x64
    {64, 128, 3, 1.0f, {0.225f, 0.250f, 0.520f}},   // I8_64x128
    {64, 128, 1, 0.5f, {0.145f, 0.165f, 0.165f}},   // I8_64x128R
    {128, 128, 1, 1.0f, {0.200f, 0.280f, 0.280f}},  // I8_128x128R
    {128, 256, 1, 2.0f, {0.300f, 0.520f, 0.520f}},  // I8_128x256
    {256, 256, 1, 5.0f, {0.540f, 0.820f, 0.820f}},  // I8_256x256
};

// One round of n workgroups (n <= 256 * resident) of `steps` steps.
static float round_us(const ShapeCost &p, int64_t n, int steps)
{
    float t = p.step[0];
    if (n > 256)
        t = p.step[1] + (p.step[2] - p.step[1]) * (float)(n - 256) / (256.f * (p.resident - 1));
    else if (n > 128)
        t += (p.step[1] - t) * (float)(n - 128) / 128.f;
    return p.fixed + t * steps;
}

// Pieces of each 256 x 256 tile of the last, partial round: as many as still fit
// one round.
static int big_pieces(int64_t tiles)
{
    const int64_t rem = tiles % 256;
    return tiles < 256 || rem == 0 || rem > 128 ? 1 : rem > 64 ? 2 : 4;
}

I8TiCfg i8_tiled_cfg(const I8Args &a, bool split, int shape, int pieces)
{
    const int cols = a.Nh ? 2 * a.Nh : a.N, fours = a.S / 4;
    I8TiCfg best = {};
    float best_us = 1e30f;
    for (int k = I8_32x32; k <= I8_256x256; k++) {
        if (shape >= I8_32x32 && shape <= I8_256x256 && k != shape)
            continue;
        const ShapeCost &p = COST[k];
        I8TiCfg c;
        c.shape = k;
        c.mtiles = (a.B + p.BM - 1) / p.BM;
        c.ntiles = (cols + p.BN - 1) / p.BN;
        const int64_t tiles = (int64_t)c.mtiles * c.ntiles;
        for (int s = 1; s <= 16 && s <= fours; s *= 2) {
            if (s > 1 && (!split || tiles >= 256))
                break;  // enough workgroups as it is
            const int want = split && pieces > 0 ? (pieces < fours ? pieces : fours) : s;
            const int per = (fours + want - 1) / want;
            c.split = (fours + per - 1) / per;  // no empty piece
            c.part_bytes = c.split > 1 ? tiles * c.split * p.BM * p.BN * 4 : 0;
            const int64_t wgs = tiles * c.split, round = 256 * p.resident, rest = wgs % round;
            float us = (float)(wgs / round) * round_us(p, round, 4 * per);
            if (rest && k == I8_256x256 && c.split == 1 && big_pieces(tiles) > 1)
                us += round_us(COST[big_pieces(tiles) == 4 ? I8_128x128R : I8_128x256], rest * big_pieces(tiles), 4 * per);
            else if (rest)
                us += round_us(p, rest, 4 * per);
            if (c.split > 1)  // a second launch, and the partial tiles written and read
                us += 4.f + 0.5e-6f * (float)c.part_bytes;
            if (us < best_us) {
                best_us = us;
                best = c;
            }
        }
    }
    return best;
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

template <bool DUAL, int OUTT>
static void big_go(const I8Args &a, const I8TiCfg &c, hipStream_t st)
{
    const int tiles = c.mtiles * c.ntiles, pieces = big_pieces(tiles);
    const int full = pieces == 1 ? tiles : tiles / 256 * 256;
    const dim3 grid((unsigned)(full + (tiles - full) * pieces)), blk(512);
    if (pieces == 4)
        hipLaunchKernelGGL((i8_big_kernel<4, DUAL, OUTT>), grid, blk, 0, st, a, c.mtiles, c.ntiles, full);
    else if (pieces == 2)
        hipLaunchKernelGGL((i8_big_kernel<2, DUAL, OUTT>), grid, blk, 0, st, a, c.mtiles, c.ntiles, full);
    else
        hipLaunchKernelGGL((i8_big_kernel<1, DUAL, OUTT>), grid, blk, 0, st, a, c.mtiles, c.ntiles, full);
}

template <bool DUAL, int OUTT>
static void tiled_shape(const I8Args &a, const I8TiCfg &c, int32_t *part, hipStream_t st)
{
    switch (c.shape) {
    case I8_32x32: tiled_go<T32x32, DUAL, OUTT>(a, c, part, st); break;
    case I8_32x64: tiled_go<T32x64, DUAL, OUTT>(a, c, part, st); break;
    case I8_64x64: tiled_go<T64x64, DUAL, OUTT>(a, c, part, st); break;
    case I8_64x128: tiled_go<T64x128, DUAL, OUTT>(a, c, part, st); break;
    case I8_64x128R: tiled_go<T64x128R, DUAL, OUTT>(a, c, part, st); break;
    case I8_128x128R: tiled_go<T128x128R, DUAL, OUTT>(a, c, part, st); break;
    case I8_128x256: tiled_go<T128x256, DUAL, OUTT>(a, c, part, st); break;
    default:
        if (c.split > 1)
            tiled_go<T256x256, DUAL, OUTT>(a, c, part, st);
        else
            big_go<DUAL, OUTT>(a, c, st);
    }
}

hipError_t launch_i8_tiled(const I8Args &a, const I8TiCfg &c, int32_t *part, int outt, hipStream_t st)
{
    if (a.Nh && outt == OUT_F32)
        tiled_shape<true, OUT_F32>(a, c, part, st);
    else if (a.Nh)
        tiled_shape<true, OUT_BF16>(a, c, part, st);
    else if (outt == OUT_F32)
        tiled_shape<false, OUT_F32>(a, c, part, st);
    else
        tiled_shape<false, OUT_BF16>(a, c, part, st);
    return hipGetLastError();
}

template <typename S>
static void grouped_go(const I8Args &a, const I8Groups &g, int outt, hipStream_t st)
{
    const int cols = a.Nh ? 2 * a.Nh : a.N;
    const int ntiles = (cols + S::BN - 1) / S::BN;
    // an expert adds at most one partial tile, and at most B experts have rows
    const int64_t tiles = a.B / S::BM + (g.E < a.B ? g.E : a.B);
    // Two weight tiles a workgroup where a tile is little work, so that finding
    // the expert and its weights is less of it: one against two, 20480 rows over
    // 512 experts of 2048 x 512 144 against 123 us, 160 rows of 1024 x 2048 40.5
    // against 38; four leave the rounds uneven (51).
    const int per = S::BM == 32 || a.S <= 16 ? 2 : 1, groups = (ntiles + per - 1) / per;
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8 * groups)), blk(64 * S::NW);
    if (a.Nh && outt == OUT_F32)
        hipLaunchKernelGGL((i8_grouped_kernel<S, true, OUT_F32>), grid, blk, 0, st, a, g, ntiles, per);
    else if (a.Nh)
        hipLaunchKernelGGL((i8_grouped_kernel<S, true, OUT_BF16>), grid, blk, 0, st, a, g, ntiles, per);
    else if (outt == OUT_F32)
        hipLaunchKernelGGL((i8_grouped_kernel<S, false, OUT_F32>), grid, blk, 0, st, a, g, ntiles, per);
    else
        hipLaunchKernelGGL((i8_grouped_kernel<S, false, OUT_BF16>), grid, blk, 0, st, a, g, ntiles, per);
}

// Rows of a tile by the mean rows of an expert.  Measured with 128 experts of
// 1024 x 2048, rows dealt evenly and unevenly, us for 32 / 64 / 128 rows a tile:
// mean 8: 57 / 57 / 54 and 55 / 55 / 51; 24: 61 / 62 / 58 and 63 / 61 / 63;
// 48: 93 / 64 / 61 and 88 / 69 / 71; 96: 128 / 98 / 70 and 130 / 97 / 83; of
// 2048 x 512: mean 8: 33 / 35 / 39 and 32 / 35 / 38; 24: 37 / 40 / 43 and
// 43 / 40 / 45; 48: 60 / 43 / 48 and 62 / 50 / 52; 96: 93 / 74 / 60 and 90 / 74 / 69.
// Where the two weights disagree, at means of 8 and 24, the rule follows the one
// with short K: it gives away 3 to 4 us of 57 there to save 3 to 6 of 33 to 43 here.
int i8_grouped_shape(int64_t E, int64_t T)
{
    return T < 16 * E ? I8_32x128 : T < 36 * E ? I8_64x128 : I8_128x128;
}

hipError_t launch_i8_grouped(const I8Args &a, const I8Groups &g, int shape, int outt, hipStream_t st)
{
    switch (shape) {
    case I8_32x128: grouped_go<T32x128>(a, g, outt, st); break;
    case I8_64x128: grouped_go<T64x128>(a, g, outt, st); break;
    default: grouped_go<T128x128>(a, g, outt, st); break;
    }
    return hipGetLastError();
}

}  // namespace qg
