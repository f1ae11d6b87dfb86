// 8-bit integer weights with one scale a channel (QGEMM_INT8), 8-bit
// activations with one scale a token, and rows sorted by expert: types and
// launch interface of int8_rows.hip, int8_small.hip, int8_tiled.hip and
// route.hip.
//
//   y[b][n] = float(sum_k q[b][k] c[n][k]) * s[b] * t[n]
//
// The sum is exact in int32 (|q|, |c| <= 128, K <= I8_MAX_K), so it does not
// depend on the order: every kernel, tile and K split gives the same bits.
#pragma once
#include "common.h"

namespace qg {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 128 * 128 * K < 2^31
constexpr int64_t I8_MAX_K = 131071;

struct I8Args {
    const uint8_t *w;     // packed weights (dense calls)
    const int8_t *codes;  // [B][ldc]
    const float *xs;      // [B] scales of the rows
    void *y;              // [B][ncols]
    int64_t scale_off;    // of the channel scales in w
    int B, N, K, S, RT;
    int Nh;               // fused gate+up: rows of the gate half (N = 2 Nh), else 0
    int ncols;            // Nh or N
    int ldc;              // bytes from row to row of codes, a multiple of 16
};

// Rows sorted by expert: rows off[e] .. off[e+1]-1 use wtab[e].  An expert
// whose own two offsets are out of order or outside 0..B is left out and sets
// DEV_BAD_OFFSETS; rows from off[E] on are neither read nor written.
struct I8Groups {
    const uint8_t *const *wtab;
    const int *off;
    int E;
    uint32_t *status;
};

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A uniform pointer read from memory, in scalar registers.
__device__ __forceinline__ const uint8_t *uniform_ptr(const uint8_t *p)
{
    const uint64_t v = (uint64_t)p;
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    return (const uint8_t *)(((uint64_t)hi << 32) | lo);
}

// Four neighbouring outputs of one lane: one store, which gfx950 takes at any
// alignment; _part: only the first `left` of them are inside.
template <int OUTT>
__device__ __forceinline__ void i8_put4(void *to, f32x4 v)
{
    if constexpr (OUTT == OUT_F32) {
        __builtin_memcpy(to, &v, 16);
    } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        bf16x4 o;
        o[0] = (__bf16)v[0]; o[1] = (__bf16)v[1]; o[2] = (__bf16)v[2]; o[3] = (__bf16)v[3];
        __builtin_memcpy(to, &o, 8);
    }
}

template <int OUTT>
__device__ __forceinline__ void i8_put4_part(void *to, f32x4 v, int left)
{
    if (left >= 4) {
        i8_put4<OUTT>(to, v);
    } else {
#pragma unroll
        for (int i = 0; i < 3; i++)
            if (i < left)
                store_out<OUTT>(to, i, v[i]);
    }
}

// ---- int8_rows.hip
// x [B][K] (act) -> codes [B][ldc] and scales [B]; pos null, or [B][topk]:
// row t's codes and scale go to the rows pos[t][j] < R instead (a negative
// position is no row, one past R sets DEV_BAD_ROUTE).
struct RowsArgs {
    const void *x;
    int8_t *codes;
    float *scales;
    const int *pos;
    uint32_t *status;
    int64_t B, K, ldc, R;
    int topk;
};
hipError_t launch_quantize_rows(int act, const RowsArgs &a, hipStream_t st);
// codes [N][K] and scales [N] on the device -> the packed layout
hipError_t launch_i8_pack(const Layout &L, const int8_t *codes, const float *scales, uint8_t *out, hipStream_t st);

// ---- int8_small.hip: few rows, weights streamed into the operands
hipError_t launch_i8_small(const I8Args &a, int outt, hipStream_t st);
bool i8_small_wins(int64_t B, int64_t N);  // the automatic choice
// rows x of type act, quantised on the way (codes and xs are not read)
bool i8_small_fuses(int64_t B, int64_t K, int64_t S);
hipError_t launch_i8_small_fused(const I8Args &a, const void *x, int act, int outt, hipStream_t st);

// ---- int8_tiled.hip: many rows, tiles through LDS
enum I8Shape {  // batch rows x channels of a tile
    I8_32x32 = 1, I8_32x64, I8_64x64, I8_64x128, I8_64x128R, I8_128x128R, I8_128x256, I8_256x256,
    I8_32x128, I8_128x128,  // routed rows (and 64 x 128)
};
struct I8TiCfg {
    int shape;
    int mtiles, ntiles;
    int split;           // workgroups along K for each tile
    int64_t part_bytes;  // int32 partial tiles (0 without a split)
};
// The shape and K split of least cost; shape, pieces: forced where they name a
// shape of dense calls and a positive number (a split only with `split`: room for
// its partial tiles).
I8TiCfg i8_tiled_cfg(const I8Args &a, bool split, int shape, int pieces);
hipError_t launch_i8_tiled(const I8Args &a, const I8TiCfg &c, int32_t *part, int outt, hipStream_t st);
int i8_grouped_shape(int64_t E, int64_t T);
hipError_t launch_i8_grouped(const I8Args &a, const I8Groups &g, int shape, int outt, hipStream_t st);

// ---- route.hip
constexpr uint32_t DEV_BAD_ROUTE = 4u;  // a position past the rows
constexpr int ROUTE_MAX_E = 16384;      // two counters an expert in 128 KB of LDS
struct RouteArgs {
    const int *ids;
    int *off, *pos;
    int n, E;
    bool vec;  // ids are 16-byte aligned
};
hipError_t launch_route(RouteArgs a, hipStream_t st);

struct MoveArgs {
    const void *src, *src2;  // dispatch: x; combine: ys; combine_grad: dy, ys
    void *dst;               // dispatch: xs; combine: y; combine_grad: dys
    const float *weights;    // [T][topk] or null (ones)
    float *dw;
    const int *pos;
    uint32_t *status;
    int64_t T, H, R;
    int topk;
};
hipError_t launch_dispatch(int dt, const MoveArgs &a, hipStream_t st);
hipError_t launch_combine(int dt, const MoveArgs &a, hipStream_t st);
hipError_t launch_combine_grad(int dt, const MoveArgs &a, hipStream_t st);

}  // namespace qg
