// The norm after a block, its gate and residual scale, and the norm before the
// next block in one pass (tq_residual_norm).
//
//   p = y * w_post / sqrt(mean(y^2) + eps)            (w_post null: p = y)
//   x' = round(scale * x + gate * p)                  (gate null: 1)
//   z = x' * w_pre / sqrt(mean(x'^2) + eps)           (w_pre null: z = x')
//
// z leaves in a float type, or quantized as the products take their activations
// (quant_quad, from the fp32 z: not rounded to a 16-bit type on the way).  The
// second norm is of x' as it is stored, so that the pass gives what the two
// steps by themselves would.  Sums, products and statistics are fp32.
//
// Bound: HBM; y and x are read, x' and z written once.  A token's elements stay in
// registers, eight a lane in a row (a quad of lanes holds one quantization block),
// of a workgroup with as many waves as they fill, or of a part of a wave.  8191
// tokens of 4096, bf16, norms on both sides: 51.5 us, 5.2 TB/s; copies of as many
// bytes run at 4.93.  One token: 2.7 us.
#include <algorithm>

#include "block_ops.h"

namespace tq {
namespace {

// Eight elements from index i of a row of n; zeros past its end.
template <int DT>
__device__ __forceinline__ void load_part(float (&v)[8], const void *x, int64_t row, int i, int n)
{
    if (i + 8 <= n) {
        load_x8<DT>(v, x, row + i);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = i + e < n ? load_one(x, DT, row + i + e) : 0.0f;
}

__device__ __forceinline__ void load_any(float (&v)[8], const void *x, int dtype, int64_t row,
                                         int i, int n)
{
    if (dtype == TQ_F32)
        load_part<TQ_F32>(v, x, row, i, n);
    else if (dtype == TQ_BF16)
        load_part<TQ_BF16>(v, x, row, i, n);
    else
        load_part<TQ_F16>(v, x, row, i, n);
}

template <int DT>
__device__ __forceinline__ void store_part(void *y, int64_t row, int i, int n, const float (&v)[8])
{
    if (i + 8 <= n) {
        store_x8<DT>(y, row + i, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (i + e < n) {
            if constexpr (DT == TQ_F32)
                ((float *)y)[row + i + e] = v[e];
            else
                ((uint16_t *)y)[row + i + e] = f32_to_16<DT>(v[e]);
        }
}

// v as an fp32 value: else a product or sum may be rounded to fp16 as it is formed in
// one kernel and after fp32 in another.
__device__ __forceinline__ float held(float v)
{
    asm("" : "+v"(v));
    return v;
}

template <int DT> __device__ __forceinline__ float rounded(float v)
{
    v = held(v);
    if constexpr (DT == TQ_F32)
        return v;
    else if constexpr (DT == TQ_BF16)
        return __builtin_bit_cast(float, (uint32_t)f32_to_16<DT>(v) << 16);
    else
        return f16_bits_to_f32(f32_to_16<DT>(v));
}

// One token, held by `lanes` lanes of which this is number `li`, U units of eight
// elements each; sum(x, k): the k-th sum over them.  Lanes past the last token hold
// it again and do not store.
template <int DT, int U, typename F>
__device__ __forceinline__ void norm_token(const ResNormArgs &a, int64_t t, bool live, int li,
                                           int lanes, F sum)
{
    const int n = a.n;
    float y[U][8], x[U][8];
    float squares = 0.0f;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * lanes + li) * 8;
        load_any(y[u], a.y, a.y_dtype, t * a.y_ts, i, n);
        load_part<DT>(x[u], a.x, t * a.x_ts, i, n);
    }
    float post = 1.0f;
    if (a.post) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int e = 0; e < 8; e++)
                squares += y[u][e] * y[u][e];
        post = 1.0f / sqrtf(sum(squares, 0) / (float)n + a.eps);
    }
    squares = 0.0f;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * lanes + li) * 8;
        float w[8];
        if (a.post) {
            load_any(w, a.post, a.w_dtype, 0, i, n);
#pragma unroll
            for (int e = 0; e < 8; e++)
                y[u][e] *= post * w[e];
        }
        if (a.gate) {
            if (a.gate_es) {
                load_any(w, a.gate, a.w_dtype, t * a.gate_ts, i, n);
            } else {
                const float g = load_one(a.gate, a.w_dtype, t * a.gate_ts);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    w[e] = g;
            }
#pragma unroll
            for (int e = 0; e < 8; e++)
                y[u][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            x[u][e] = rounded<DT>(fmaf(a.scale, x[u][e], y[u][e]));
            if (i + e >= n)
                x[u][e] = 0.0f;                  // an infinite gate makes NaN of a 0
            squares += x[u][e] * x[u][e];
        }
        if (live && i < n)
            store_part<DT>(a.x_out, t * a.xo_ts, i, n, x[u]);
    }
    float pre = 1.0f;
    if (a.pre)
        pre = 1.0f / sqrtf(sum(squares, 1) / (float)n + a.eps);
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * lanes + li) * 8;
        if (a.pre) {
            float w[8];
            load_any(w, a.pre, a.w_dtype, 0, i, n);
#pragma unroll
            for (int e = 0; e < 8; e++)
                x[u][e] = held(x[u][e] * (pre * w[e]));
        }
        if (a.q) {
            // n is a multiple of 32: the lanes of a quad are inside or outside together
            uint2 code;
            uint16_t d;
            quant_quad(x[u], code, d);
            if (live && i < n) {
                *(u32x2u *)(a.q + t * n + i) = u32x2u{code.x, code.y};
                if ((li & 3) == 0)
                    a.d[(t * n + i) >> 5] = d;
            }
        } else if (live && i < n) {
            store_part<DT>(a.z, t * a.z_ts, i, n, x[u]);
        }
    }
}

// A workgroup of as many waves as a token fills.
template <int DT, int U> __global__ __launch_bounds__(1024) void k_residual_norm(ResNormArgs a)
{
    __shared__ float red[2][16];
    const int waves = blockDim.x >> 6;
    norm_token<DT, U>(a, blockIdx.x, true, threadIdx.x, blockDim.x, [&](float v, int k) {
        v = wave_sum(v);
        if (waves == 1)
            return v;
        if ((threadIdx.x & 63) == 0)
            red[k][threadIdx.x >> 6] = v;
        __syncthreads();
        return sum_lanes(red[k][threadIdx.x & 15], waves);
    });
}

// Eight elements as they lie in memory.
struct Raw8 {
    uint32_t w[8];
};

__device__ __forceinline__ void load_raw(Raw8 &r, const void *x, int dtype, int64_t row, int i, int n)
{
    if (i + 8 <= n) {
        if (dtype == TQ_F32) {
            float v[8];
            load_x8<TQ_F32>(v, x, row + i);
#pragma unroll
            for (int e = 0; e < 8; e++)
                r.w[e] = __builtin_bit_cast(uint32_t, v[e]);
        } else {
            const u16x8u h = *(const u16x8u *)((const uint16_t *)x + row + i);
#pragma unroll
            for (int e = 0; e < 4; e++)
                r.w[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        r.w[e] = 0;
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (i + e < n) {
            if (dtype == TQ_F32)
                r.w[e] = ((const uint32_t *)x)[row + i + e];
            else
                r.w[e >> 1] |= (uint32_t)((const uint16_t *)x)[row + i + e] << (16 * (e & 1));
        }
}

__device__ __forceinline__ void convert(float (&v)[8], const Raw8 &r, int dtype)
{
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const uint32_t h = (r.w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        v[e] = dtype == TQ_F32 ? __builtin_bit_cast(float, r.w[e])
                               : (dtype == TQ_BF16 ? __builtin_bit_cast(float, h << 16)
                                                   : f16_bits_to_f32((uint16_t)h));
    }
}

// The same for many tokens of up to 8192 elements, two waves and more: a workgroup
// takes every gridDim-th token, has the weights in registers, and the next token on
// its way while it works on one.  bf16, norms on both sides, three sets of inputs in
// turn, a workgroup for each token / so, us: 8192 x 4096 51.2 / 53.0, with one gate for
// all tokens 55.1 / 52.5, quantized 50.6 / 49.7, of fp32 y 60.0 / 62.9; 8192 x 5120
// 77.7 / 66.8, with the gate 85.5 / 67.5; 32768 x 1024 49.4 / 52.0, with the gate 53.8 /
// 52.8; 4096 x 8192 53.1 / 54.9, with the gate 56.6 / 54.9, quantized 56.3 / 64.3.  A wave
// each of 512 is faster alone (50.2, so 53.8, for 65536 tokens).
template <int DT> __global__ __launch_bounds__(1024) void k_residual_norm_many(ResNormArgs a)
{
    __shared__ float red[2][2][16];
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6, n = a.n, i = tid * 8;
    int64_t t = blockIdx.x;
    Raw8 next_y, next_x;
    load_raw(next_y, a.y, a.y_dtype, t * a.y_ts, i, n);
    load_raw(next_x, a.x, DT, t * a.x_ts, i, n);
    float post_w[8] = {}, pre_w[8] = {}, gate[8] = {};
    if (a.post)
        load_any(post_w, a.post, a.w_dtype, 0, i, n);
    if (a.pre)
        load_any(pre_w, a.pre, a.w_dtype, 0, i, n);
    const bool one_gate = a.gate && a.gate_ts == 0;
    auto load_gate = [&](int64_t token) {
        if (a.gate_es) {
            load_any(gate, a.gate, a.w_dtype, token * a.gate_ts, i, n);
        } else {
            const float g = load_one(a.gate, a.w_dtype, token * a.gate_ts);
#pragma unroll
            for (int e = 0; e < 8; e++)
                gate[e] = g;
        }
    };
    if (one_gate)
        load_gate(0);
    for (int turn = 0; t < a.tokens; t += gridDim.x, turn ^= 1) {
        auto sum = [&](float v, int k) {
            v = wave_sum(v);
            if (lane == 0)
                red[turn][k][tid >> 6] = v;
            __syncthreads();
            return sum_lanes(red[turn][k][tid & 15], waves);
        };
        float y[8], x[8], squares = 0.0f;
        convert(y, next_y, a.y_dtype);
        convert(x, next_x, DT);
        if (a.gate && !one_gate)
            load_gate(t);
        const int64_t then = t + gridDim.x;
        if (then < a.tokens) {
            load_raw(next_y, a.y, a.y_dtype, then * a.y_ts, i, n);
            load_raw(next_x, a.x, DT, then * a.x_ts, i, n);
        }
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8; e++)
                squares += y[e] * y[e];
            const float f = 1.0f / sqrtf(sum(squares, 0) / (float)n + a.eps);
#pragma unroll
            for (int e = 0; e < 8; e++)
                y[e] *= f * post_w[e];
        }
        squares = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if (a.gate)
                y[e] *= gate[e];
            x[e] = rounded<DT>(fmaf(a.scale, x[e], y[e]));
            if (i + e >= n)
                x[e] = 0.0f;
            squares += x[e] * x[e];
        }
        if (i < n)
            store_part<DT>(a.x_out, t * a.xo_ts, i, n, x);
        if (a.pre) {
            const float f = 1.0f / sqrtf(sum(squares, 1) / (float)n + a.eps);
#pragma unroll
            for (int e = 0; e < 8; e++)
                x[e] = held(x[e] * (f * pre_w[e]));
        }
        if (a.q) {
            uint2 code;
            uint16_t d;
            quant_quad(x, code, d);
            if (i < n) {
                *(u32x2u *)(a.q + t * n + i) = u32x2u{code.x, code.y};
                if ((tid & 3) == 0)
                    a.d[(t * n + i) >> 5] = d;
            }
        } else if (i < n) {
            store_part<DT>(a.z, t * a.z_ts, i, n, x);
        }
    }
}

// Several tokens a wave, 2^log_lanes lanes each.
constexpr int SMALL_WAVES = 4;

template <int DT>
__global__ __launch_bounds__(64 * SMALL_WAVES) void k_residual_norm_small(ResNormArgs a, int log_lanes)
{
    const int lanes = 1 << log_lanes, li = threadIdx.x & (lanes - 1);
    const int64_t t = (int64_t)blockIdx.x * (64 * SMALL_WAVES >> log_lanes) + (threadIdx.x >> log_lanes);
    norm_token<DT, 1>(a, min(t, a.tokens - 1), t < a.tokens, li, lanes, [&](float v, int) {
        for (int m = 1; m < lanes; m <<= 1)
            v += __shfl_xor(v, m);
        return v;
    });
}

constexpr int MANY_WAVES = 24;                   // of a unit, by the kernel's registers

template <int DT> hipError_t launch_dt(const ResNormArgs &a, hipStream_t s)
{
    if (!grid_fits(a.tokens, 1024))
        return hipErrorInvalidConfiguration;
    // Half a wave and less: 131072 tokens of 256 take 56 us so, 90 with a wave each.
    int log_lanes = 2;                           // a quantization block at least
    while ((8 << log_lanes) < a.n)
        log_lanes++;
    if (log_lanes < 6) {
        const int64_t each = 64 * SMALL_WAVES >> log_lanes;
        k_residual_norm_small<DT><<<dim3((unsigned)((a.tokens + each - 1) / each)), 64 * SMALL_WAVES, 0,
                                    s>>>(a, log_lanes);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)a.tokens);
    const int units = (a.n + 511) / 512;         // of a wave
    const int64_t resident = (int64_t)256 * std::max(1, MANY_WAVES / units);
    if (units > 1 && units <= 16 && a.tokens >= 2 * resident)
        k_residual_norm_many<DT><<<dim3((unsigned)resident), 64 * units, 0, s>>>(a);
    else if (units <= 16)
        k_residual_norm<DT, 1><<<grid, 64 * units, 0, s>>>(a);
    else if (units <= 32)
        k_residual_norm<DT, 2><<<grid, 64 * ((units + 1) / 2), 0, s>>>(a);
    else
        k_residual_norm<DT, 4><<<grid, 64 * ((units + 3) / 4), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(int dtype, const ResNormArgs &a, hipStream_t s)
{
    switch (dtype) {
    case TQ_F32: return launch_dt<TQ_F32>(a, s);
    case TQ_BF16: return launch_dt<TQ_BF16>(a, s);
    case TQ_F16: return launch_dt<TQ_F16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace tq
