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
// Bound: HBM; y and x are read, x' and z written once.  A workgroup has a token
// at a time, its elements in registers, eight a lane in a row: a quad of lanes
// holds one quantization block.
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

template <int DT> __device__ __forceinline__ float rounded(float v)
{
    if constexpr (DT == TQ_F32)
        return v;
    else if constexpr (DT == TQ_BF16)
        return __builtin_bit_cast(float, (uint32_t)f32_to_16<DT>(v) << 16);
    else
        return f16_bits_to_f32(f32_to_16<DT>(v));
}

template <int WAVES> __device__ __forceinline__ float sum_all(float v, float *lds)
{
    v = wave_sum(v);
    if constexpr (WAVES == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    const int lane = threadIdx.x & 63;
    return sum_lanes(lane < WAVES ? lds[lane] : 0.0f, WAVES);
}

// WAVES waves hold a token, U units of eight elements a lane.
template <int DT, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void k_residual_norm(ResNormArgs a)
{
    constexpr int THREADS = 64 * WAVES;
    __shared__ float red[2][WAVES];
    const int tid = threadIdx.x, n = a.n;
    const int64_t t = blockIdx.x;
    float y[U][8], x[U][8];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * THREADS + tid) * 8;
        load_any(y[u], a.y, a.y_dtype, t * a.y_ts, i, n);
        load_part<DT>(x[u], a.x, t * a.x_ts, i, n);
    }
    float post = 1.0f;
    if (a.post) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int e = 0; e < 8; e++)
                sum += y[u][e] * y[u][e];
        post = 1.0f / sqrtf(sum_all<WAVES>(sum, red[0]) / (float)n + a.eps);
    }
    sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * THREADS + tid) * 8;
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
                x[u][e] = 0.0f;              // an infinite gate makes NaN of a 0
            sum += x[u][e] * x[u][e];
        }
        if (i < n)
            store_part<DT>(a.x_out, t * a.xo_ts, i, n, x[u]);
    }
    float pre = 1.0f;
    if (a.pre)
        pre = 1.0f / sqrtf(sum_all<WAVES>(sum, red[1]) / (float)n + a.eps);
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int i = (u * THREADS + tid) * 8;
        if (a.pre) {
            float w[8];
            load_any(w, a.pre, a.w_dtype, 0, i, n);
#pragma unroll
            for (int e = 0; e < 8; e++)
                x[u][e] *= pre * w[e];
        }
        if (a.q) {
            // n is a multiple of 32: the lanes of a quad are inside or outside together
            uint2 code;
            uint16_t d;
            quant_quad(x[u], code, d);
            if (i < n) {
                *(u32x2u *)(a.q + t * n + i) = u32x2u{code.x, code.y};
                if ((tid & 3) == 0)
                    a.d[(t * n + i) >> 5] = d;
            }
        } else if (a.z && i < n) {
            store_part<DT>(a.z, t * a.z_ts, i, n, x[u]);
        }
    }
}

template <int DT> hipError_t launch_dt(const ResNormArgs &a, hipStream_t s)
{
    if (!grid_fits(a.tokens, 1024))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)a.tokens);
    if (a.n <= 512)
        k_residual_norm<DT, 1, 1><<<grid, 64, 0, s>>>(a);
    else if (a.n <= 2048)
        k_residual_norm<DT, 4, 1><<<grid, 256, 0, s>>>(a);
    else if (a.n <= 4096)
        k_residual_norm<DT, 8, 1><<<grid, 512, 0, s>>>(a);
    else if (a.n <= 8192)
        k_residual_norm<DT, 16, 1><<<grid, 1024, 0, s>>>(a);
    else if (a.n <= 16384)
        k_residual_norm<DT, 16, 2><<<grid, 1024, 0, s>>>(a);
    else
        k_residual_norm<DT, 16, 4><<<grid, 1024, 0, s>>>(a);
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
