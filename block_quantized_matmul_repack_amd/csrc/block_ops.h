// Sums, scans and order keys shared by the serving-step kernels (plan.hip,
// resnorm.hip, sample.hip, sparse.hip).
#pragma once

#include "tq_internal.h"

namespace tq {

template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t dpp_bits(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, true);
}

template <int CTRL, int ROWS> __device__ __forceinline__ uint64_t dpp_bits(uint64_t x)
{
    return ((uint64_t)dpp_bits<CTRL, ROWS>((uint32_t)(x >> 32)) << 32) |
           dpp_bits<CTRL, ROWS>((uint32_t)x);
}

template <int CTRL, int ROWS> __device__ __forceinline__ float dpp_bits(float x)
{
    return __builtin_bit_cast(float, dpp_bits<CTRL, ROWS>(__builtin_bit_cast(uint32_t, x)));
}

template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_bits(double x)
{
    return __builtin_bit_cast(double, dpp_bits<CTRL, ROWS>(__builtin_bit_cast(uint64_t, x)));
}

// Running sum over each row of 16 lanes: shifts by 1, 2, 4, 8.  Lanes that a step
// brings nothing to add 0.
template <typename T> __device__ __forceinline__ T scan_row(T v)
{
    v += dpp_bits<0x111, 0xF>(v);
    v += dpp_bits<0x112, 0xF>(v);
    v += dpp_bits<0x114, 0xF>(v);
    v += dpp_bits<0x118, 0xF>(v);
    return v;
}

// Running sum over the lanes of a wave: in rows, then the last lane of a row added to
// the rows behind it.
template <typename T> __device__ __forceinline__ T scan_wave(T v)
{
    v = scan_row(v);
    v += dpp_bits<0x142, 0xA>(v);
    v += dpp_bits<0x143, 0xC>(v);
    return v;
}

// Lane k's value, k uniform.
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int k)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)x, k);
}

__device__ __forceinline__ uint64_t lane_value(uint64_t x, int k)
{
    return ((uint64_t)lane_value((uint32_t)(x >> 32), k) << 32) | lane_value((uint32_t)x, k);
}

__device__ __forceinline__ float lane_value(float x, int k)
{
    return __builtin_bit_cast(float, lane_value(__builtin_bit_cast(uint32_t, x), k));
}

__device__ __forceinline__ double lane_value(double x, int k)
{
    return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, x), k));
}

template <typename T> __device__ __forceinline__ T wave_sum(T v)
{
    return lane_value(scan_wave(v), 63);
}

// Largest over the lanes.
__device__ __forceinline__ float wave_max(float v)
{
    for (int m = 1; m < 64; m <<= 1)
        v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Running sum over a workgroup of WAVES waves, before this thread, and the sum
// of all.  `lds` holds WAVES values; it may be used again after the next barrier
// that all threads pass.
template <int WAVES, typename T>
__device__ __forceinline__ T scan_before(T v, T *lds, T &all)
{
    static_assert(WAVES <= 16, "");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T run = scan_wave(v);
    if (lane == 63)
        lds[wave] = run;
    __syncthreads();
    // the waves' sums by lanes: fewer instructions than reading all of them in turn
    const T upto = scan_row(lane < WAVES ? lds[lane] : T(0));
    all = lane_value(upto, WAVES - 1);
    const int w = __builtin_amdgcn_readfirstlane(wave);
    return (w ? lane_value(upto, w - 1) : T(0)) + run - v;
}

// The sum of what lanes 0 .. n - 1 hold, n up to 16, in every lane.
template <typename T> __device__ __forceinline__ T sum_lanes(T v, int n)
{
    return lane_value(scan_row((int)(threadIdx.x & 63) < n ? v : T(0)), 15);
}

// Unsigned numbers in the order of the floats; a NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x != x ? -__builtin_inff() : x + 0.0f);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Nearest whole number of v * inv, halves away from zero: quant_quad's rounding.
__device__ __forceinline__ int round_away(float v, float inv)
{
#pragma clang fp contract(off)
    const float y = v * inv;
    return (int)(y + copysignf(0.49999997f, y));
}

// One element of a run-time type.
__device__ __forceinline__ float load_one(const void *x, int dtype, int64_t i)
{
    if (dtype == TQ_F32)
        return ((const float *)x)[i];
    const uint16_t h = ((const uint16_t *)x)[i];
    return dtype == TQ_BF16 ? __builtin_bit_cast(float, (uint32_t)h << 16) : f16_bits_to_f32(h);
}

}  // namespace tq
