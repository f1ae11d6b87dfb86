// A row's elements to its codes: the steps that the kernels of int8_rows.hip and
// the fused form of int8_small.hip share, so that both give the same bits.
#pragma once
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

// Eight elements as they are in memory, through a resource; a load that nothing
// looks at yet.
template <int ACT>
struct Raw8 {
    static constexpr int ESZ = ACT == ACT_F32 ? 4 : 2;
    u32x4 r[ACT == ACT_F32 ? 2 : 1];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, int at)
    {
        r[0] = bload16(x, at, 0);
        if constexpr (ACT == ACT_F32)
            r[1] = bload16(x, at + 16, 0);
    }
    __device__ __forceinline__ void floats(float *v) const
    {
#pragma unroll
        for (int i = 0; i < RQ_V; i++) {
            if constexpr (ACT == ACT_F32)
                v[i] = __uint_as_float(r[i / 4][i % 4]);
            else
                v[i] = __uint_as_float(i & 1 ? r[0][i / 2] & 0xFFFF0000u : r[0][i / 2] << 16);
        }
    }
};

// Eight codes.  Where 1 / s is finite, s has 22 bits at least (it may be
// subnormal), |x / s| is below 127.01 and x * (1 / s) within 2^-15 of the quotient
// that the definition rounds: three roundings of 2^-24 of it.  So only a value
// within 10^-4 of a border between codes, or one that is no number or infinite
// because 1 / s overflowed (s of 2^-128 and below, where |x / s| reaches 190),
// takes the division (ten instructions each: 15.5 against 13.9 us for 2048 rows
// of 5120).
__device__ __forceinline__ u32x2 pack_codes8(const float *v, float s, float inv)
{
    float n[RQ_V];
    bool near = false;
#pragma unroll
    for (int i = 0; i < RQ_V; i++) {
        const float r = v[i] * inv;
        n[i] = __builtin_rintf(r);
        near |= !(__builtin_fabsf(r - n[i]) < 0.4999f);
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < RQ_V; i++)
            n[i] = __builtin_rintf(v[i] / s);
    }
    u32x2 o = u32x2{0u, 0u};
#pragma unroll
    for (int i = 0; i < RQ_V; i++) {
        const int c = (int)fminf(fmaxf(n[i], -127.f), 127.f);
        o[i / 4] |= ((uint32_t)c & 0xFFu) << (8 * (i % 4));
    }
    return o;
}

// The scale of a row from the bits of its largest |x|, and what pack_codes8 takes;
// zero: its codes are 0 (a row of zeros, or one that holds a NaN or an infinity,
// whose scale is NaN).
struct RowScale {
    float s, inv;
    bool zero;
    __device__ __forceinline__ explicit RowScale(uint32_t top)
    {
        const bool bad = top >= 0x7F800000u;
        s = bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / 127.f;
        zero = bad || s == 0.f;
        inv = zero ? 0.f : 1.f / s;
    }
    __device__ __forceinline__ u32x2 codes(const float *v) const
    {
        return zero ? u32x2{0u, 0u} : pack_codes8(v, s, inv);
    }
};

// Largest |x| of eight elements as bits: infinities and NaNs above all finite
// values, whatever the order.
__device__ __forceinline__ uint32_t top8(const float *v, uint32_t top)
{
#pragma unroll
    for (int i = 0; i < RQ_V; i++)
        top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return top;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t top)
{
    for (int d = 32; d; d >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    return top;
}

}  // namespace qg
