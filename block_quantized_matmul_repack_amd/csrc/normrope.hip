// Per-head RMS norm of queries and keys with their position rotation, in one
// pass over both (tq_qk_norm_rope).
//
//   z = x * w / sqrt(mean(x^2) + eps)                 (w null: z = x)
//   pair (a, b) at angle t = pos * freq[i]: (a cos t - b sin t, b cos t + a sin t)
//
// The kernel is a read and a write of every element; statistics, products and
// angles stay in fp32 (angles in fp64 turns) and each output is rounded once.
// A wave owns one token and several heads: its angles are the same for every
// head, so each is computed once, by one lane, and passed on through LDS (each
// lane computing the angles of its own elements, eight times as many, took
// 44 us where this took 40, both with one wave a token).  8192 tokens, 32 + 8
// heads of 128, bf16, nothing in the caches, two waves a token: 36.8 us, 4.6
// TB/s; copies of the two tensors 35.  Called again and again on the same
// tensors, half of which the caches then hold: 32.
#include <algorithm>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;
constexpr int MAX_D = 512;

// V consecutive elements from index i.
template <int DT, int V>
__device__ __forceinline__ void load_v(float (&v)[V], const void *x, int64_t i)
{
    if constexpr (V == 8) {
        load_x8<DT>(v, x, i);
    } else {
        static_assert(V == 1, "");
        if constexpr (DT == TQ_F32)
            v[0] = ((const float *)x)[i];
        else if constexpr (DT == TQ_BF16)
            v[0] = __builtin_bit_cast(float, (uint32_t)((const uint16_t *)x)[i] << 16);
        else
            v[0] = f16_bits_to_f32(((const uint16_t *)x)[i]);
    }
}

template <int DT, int V>
__device__ __forceinline__ void store_v(void *y, int64_t i, const float (&v)[V])
{
    if constexpr (V == 8) {
        store_x8<DT>(y, i, v);
    } else if constexpr (DT == TQ_F32) {
        ((float *)y)[i] = v[0];
    } else {
        ((uint16_t *)y)[i] = f32_to_16<DT>(v[0]);
    }
}

template <int V>
__device__ __forceinline__ void load_w(float (&v)[V], const void *w, int dtype, int64_t i)
{
    if (dtype == TQ_F32)
        load_v<TQ_F32, V>(v, w, i);
    else if (dtype == TQ_BF16)
        load_v<TQ_BF16, V>(v, w, i);
    else
        load_v<TQ_F16, V>(v, w, i);
}

// A head is cut into units of 2 V elements: V rotation pairs (halves: V
// elements of each half; interleaved: 2 V neighbours), or 2 V elements past
// the rotated part.  2^log_lanes lanes hold a head, U units each (U > 1 only
// for V = 1).  Heads are numbered queries first, then keys; a wave takes
// `groups` = 64 >> log_lanes heads at a time.
template <int DT, int V, int U>
__global__ __launch_bounds__(THREADS) void k_norm_rope(NormRopeArgs a, int log_lanes, int parts)
{
    const int64_t id = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    const int64_t t = id / parts;
    const int part = (int)(id - t * parts);
    if (t >= a.tokens)
        return;
    const int lane = threadIdx.x & 63;
    const int lanes = 1 << log_lanes, groups = 64 >> log_lanes;
    const int li = lane & (lanes - 1), gi = lane >> log_lanes;
    const int half = a.rot >> 1, rot_units = half / V, units = a.D / (2 * V);

    int o0[U], o1[U];
    bool live[U];
    float cs[U][V], sn[U][V];
    __shared__ __align__(16) float turn[WAVES][2][MAX_D / 2];
    float *cosines = turn[threadIdx.x >> 6][0], *sines = turn[threadIdx.x >> 6][1];
    const double pos = (double)a.pos[t] * 0.15915494309189533577;   // 1 / (2 pi)
    for (int i = lane; i < half; i += 64) {
        // the angle in turns, reduced to [-1/2, 1/2] before it leaves fp64
        const double turns = pos * (double)a.freq[i];
        float c, s;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cosines[i] = c;
        sines[i] = s;
    }
    wave_handover();
#pragma unroll
    for (int k = 0; k < U; k++) {
        const int u = li + k * lanes;
        live[k] = u < units;
        const bool rotated = u < rot_units;
        if (!rotated) {
            o0[k] = a.rot + 2 * (u - rot_units) * V;
            o1[k] = o0[k] + V;
        } else if (a.interleaved) {
            o0[k] = 2 * u * V;
            o1[k] = o0[k] + V;
        } else {
            o0[k] = u * V;
            o1[k] = half + o0[k];
        }
#pragma unroll
        for (int e = 0; e < V; e++) {
            cs[k][e] = live[k] && rotated ? cosines[u * V + e] : 1.0f;
            sn[k][e] = live[k] && rotated ? sines[u * V + e] : 0.0f;
        }
    }

    const int all = a.heads[0] + a.heads[1];
    for (int hb = part * groups; hb < all; hb += parts * groups) {
        const int hh = hb + gi;
        if (hh >= all)
            continue;                            // uniform across the lanes of a head
        const int which = hh >= a.heads[0];
        const int h = hh - (which ? a.heads[0] : 0);
        const void *x = which ? a.x[1] : a.x[0];
        const void *w = which ? a.w[1] : a.w[0];
        const int64_t xi = t * (which ? a.xts[1] : a.xts[0]) + h * (which ? a.xhs[1] : a.xhs[0]);
        const int64_t yi = t * (which ? a.yts[1] : a.yts[0]) + h * (which ? a.yhs[1] : a.yhs[0]);
        float v0[U][V], v1[U][V];
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < U; k++)
            if (live[k]) {
                load_v<DT, V>(v0[k], x, xi + o0[k]);
                load_v<DT, V>(v1[k], x, xi + o1[k]);
#pragma unroll
                for (int e = 0; e < V; e++)
                    sum += v0[k][e] * v0[k][e] + v1[k][e] * v1[k][e];
            }
        float inv = 1.0f;
        if (w) {
            for (int m = 1; m < lanes; m <<= 1)
                sum += __shfl_xor(sum, m);
            inv = 1.0f / sqrtf(sum / (float)a.D + a.eps);
        }
#pragma unroll
        for (int k = 0; k < U; k++)
            if (live[k]) {
                if (w) {
                    float w0[V], w1[V];
                    load_w<V>(w0, w, a.w_dtype, o0[k]);
                    load_w<V>(w1, w, a.w_dtype, o1[k]);
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        v0[k][e] *= inv * w0[e];
                        v1[k][e] *= inv * w1[e];
                    }
                }
                float r0[V], r1[V];
                if (a.interleaved && V > 1) {
                    // neighbours are pairs: elements 0, 1 of v0 are pair 0, ...
#pragma unroll
                    for (int e = 0; e + 1 < V; e += 2) {
                        const float c0 = cs[k][e / 2], s0 = sn[k][e / 2];
                        const float c1 = cs[k][V / 2 + e / 2], s1 = sn[k][V / 2 + e / 2];
                        r0[e] = v0[k][e] * c0 - v0[k][e + 1] * s0;
                        r0[e + 1] = v0[k][e + 1] * c0 + v0[k][e] * s0;
                        r1[e] = v1[k][e] * c1 - v1[k][e + 1] * s1;
                        r1[e + 1] = v1[k][e + 1] * c1 + v1[k][e] * s1;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        r0[e] = v0[k][e] * cs[k][e] - v1[k][e] * sn[k][e];
                        r1[e] = v1[k][e] * cs[k][e] + v0[k][e] * sn[k][e];
                    }
                }
                void *y = which ? a.y[1] : a.y[0];
                store_v<DT, V>(y, yi + o0[k], r0);
                store_v<DT, V>(y, yi + o1[k], r1);
            }
    }
}

template <int DT>
hipError_t launch_dt(const NormRopeArgs &a, hipStream_t s)
{
    // 8 pairs per lane wherever the halves and the rest are whole eights
    const bool wide = (a.rot / 2) % 8 == 0 && (a.D - a.rot) % 16 == 0;
    const int units = a.D / (wide ? 16 : 2);
    int log_lanes = 0;
    while (log_lanes < 6 && (1 << log_lanes) < units)
        log_lanes++;
    const int groups = 64 >> log_lanes;
    const int64_t rounds = (a.heads[0] + a.heads[1] + groups - 1) / groups;
    // Few tokens: a token's heads are spread over waves, one round each, as far
    // as that fills the chip twice (256 units, 32 waves each).  Many: a wave has a
    // few rounds, since its angles cost as much as one or two, and with all of
    // them the last waves run alone.  5 rounds of 16-byte loads (32 + 8 heads of
    // 128, bf16, caches flushed, one call): two waves a token 49.9, 67.3, 83.9 and
    // 502 us for 8193, 12000, 16384 and 131072 tokens, one 54.0, 70.2, 88.5 and
    // 503, five 48.0, 65.0, 82.5 and 533; 9 rounds: three 80.3 and 869 us for 8193
    // and 131072, one 91.7 and 922.  Rounds of single elements are an eighth as
    // long: 40 of them (32 + 8 heads of 72), four waves 115 and 789 us for 8193 and
    // 65536, one 149 and 780, ten 120 and 873.
    const int64_t least = (rounds + (wide ? 2 : 9)) / (wide ? 3 : 10);
    int64_t parts = std::max(least, std::min<int64_t>(rounds, 16384 / a.tokens));
    parts = std::max<int64_t>(1, std::min(parts, (int64_t(1) << 25) / a.tokens));  // the grid's limit
    const int64_t blocks = (a.tokens * parts + WAVES - 1) / WAVES;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks);
    if (wide)
        k_norm_rope<DT, 8, 1><<<grid, THREADS, 0, s>>>(a, log_lanes, (int)parts);
    else
        k_norm_rope<DT, 1, 4><<<grid, THREADS, 0, s>>>(a, log_lanes, (int)parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(int dtype, const NormRopeArgs &a, hipStream_t s)
{
    switch (dtype) {
    case TQ_F32: return launch_dt<TQ_F32>(a, s);
    case TQ_BF16: return launch_dt<TQ_BF16>(a, s);
    case TQ_F16: return launch_dt<TQ_F16>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace tq
