// Paged key / value cache held in 32-element quantized blocks: tokens are
// quantized as they are written (tq_cache_write) and read back as the values
// their blocks stand for (tq_cache_read).  The layout is cache_layout.h.
//
// Both kernels only move data (about 3 bytes of traffic per bf16 element
// stored, one pass).  A quad of lanes holds one 32-element block, 8 elements
// per lane, as in the activation quantization.
#include <type_traits>

#include "cache_layout.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int THREADS = 256;

// The largest magnitude a cache block stands for: 65472 / 127 rounds to the
// fp16 scale 515.5 and 127 * 515.5 = 65468.5, 65472 / 8 = 8184 exactly, so
// every dequantized element stays a finite fp16 number.
constexpr float CACHE_LIMIT = 65472.0f;

// NaN counts as 0, magnitudes past CACHE_LIMIT (infinities too) as
// CACHE_LIMIT, so that nothing a cache holds is NaN or infinite.
__device__ __forceinline__ float cache_clean(float x)
{
    return x == x ? fminf(fmaxf(x, -CACHE_LIMIT), CACHE_LIMIT) : 0.0f;
}

// GGML's Q4_0 rule for the block of a quad of lanes (8 elements per lane):
// m = the first element of the largest magnitude, d = m / -8, code =
// min(15, trunc(x * (1 / d) + 8.5)), fp32 steps, d stored as fp16.  Lane c's
// codes come back as nibbles in element order.
__device__ __forceinline__ void quant_quad_q4(const float (&v)[8], int c, uint32_t &codes,
                                              uint16_t &dbits)
{
#pragma clang fp contract(off)
    float m = v[0];
#pragma unroll
    for (int e = 1; e < 8; e++)
        if (fabsf(v[e]) > fabsf(m))
            m = v[e];
    // the earlier lane wins ties: lane c takes the other's only where larger,
    // or equal and the other comes first
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        const float o = __shfl_xor(m, s);
        const bool first = (c & s) != 0;
        if (fabsf(o) > fabsf(m) || (first && fabsf(o) == fabsf(m)))
            m = o;
    }
    const float dd = m * -0.125f;
    const float id = dd != 0.0f ? 1.0f / dd : 0.0f;
    codes = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float y = v[e] * id;
        const int q = (int)(y + 8.5f);
        codes |= (uint32_t)min(max(q, 0), 15) << (4 * e);
    }
    dbits = f32_to_f16_bits(dd);
}

// Codes of one lane: 8 biased bytes (Q8_0) or 8 nibbles in x (Q4_0).
template <int CT>
__device__ __forceinline__ uint2 quantize_lane(float (&v)[8], int c, uint16_t &dbits)
{
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = cache_clean(v[e]);
    uint2 q = make_uint2(0, 0);
    if constexpr (CT == TQ_Q8_0) {
        quant_quad(v, q, dbits);
        q.x ^= 0x80808080u;
        q.y ^= 0x80808080u;
    } else {
        quant_quad_q4(v, c, q.x, dbits);
    }
    return q;
}

struct WriteArgs {
    const void *x[2];            // keys, values
    int64_t ts[2], hs[2];        // token and head strides, elements
    uint8_t *cache[2];
    const int32_t *slots;
    int64_t tokens, slots_total;
    int heads, log_page;
};

// One unit (8 elements) per lane; blockIdx.y picks keys or values.
template <int CT, int DT, int D>
__global__ __launch_bounds__(THREADS) void k_cache_write(WriteArgs a)
{
    constexpr int UPH = D / 8;                   // units per head
    const int which = blockIdx.y;
    const int64_t u = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t th = u / UPH;
    const int uu = (int)(u - th * UPH), s = uu >> 2, c = uu & 3;
    const int64_t t = th / a.heads;
    const int h = (int)(th - t * a.heads);
    if (t >= a.tokens)
        return;                                  // uniform across the quad of a block
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.slots_total)
        return;
    float v[8];
    load_x8<DT>(v, a.x[which], t * a.ts[which] + h * a.hs[which] + 8 * uu);
    uint16_t db;
    const uint2 q = quantize_lane<CT>(v, c, db);

    const int P = 1 << a.log_page;
    const int64_t page = slot >> a.log_page;
    const int pos = (int)(slot & (P - 1));
    constexpr int TB = (int)token_code_bytes(CT, D);
    uint8_t *chunk = a.cache[which] + (page * a.heads + h) * chunk_bytes(CT, D, P);
    uint16_t *scales = (uint16_t *)(chunk + P * TB);
    if (which == 0) {
        uint8_t *p = chunk + k_offset<CT, D>(pos, s, c);
        if constexpr (CT == TQ_Q8_0) {
            *(uint2 *)p = q;
        } else {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; e++)
                w |= ((q.x >> (4 * e)) & 15u) << k4_shift(e);
            *(uint32_t *)p = w;
        }
        if (c == 0)
            scales[pos * (D / 32) + s] = db;
    } else {
        if constexpr (CT == TQ_Q8_0) {
            uint8_t *p = chunk + ((pos >> 2) * D + 8 * uu) * 4 + (pos & 3);
#pragma unroll
            for (int e = 0; e < 8; e++)
                p[4 * e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
        } else {
            uint8_t *p = chunk + ((pos >> 2) * (D / 2) + 4 * uu) * 4 + v4_byte(pos & 3);
#pragma unroll
            for (int e = 0; e < 4; e++)
                p[4 * e] = (uint8_t)(q.x >> (8 * e));
        }
        if (c == 0)
            scales[s * P + pos] = db;
    }
}

struct ReadArgs {
    const uint8_t *cache[2];
    void *y[2];                  // [tokens][heads][D], contiguous
    const int32_t *slots;
    int64_t tokens, slots_total;
    int heads, log_page;
};

// A slot outside the cache reads as zeros.
template <int CT, int DT, int D>
__global__ __launch_bounds__(THREADS) void k_cache_read(ReadArgs a)
{
    constexpr int UPH = D / 8;
    const int which = blockIdx.y;
    const int64_t u = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    const int64_t th = u / UPH;
    const int uu = (int)(u - th * UPH), s = uu >> 2, c = uu & 3;
    const int64_t t = th / a.heads;
    const int h = (int)(th - t * a.heads);
    if (t >= a.tokens)
        return;
    const int64_t slot = a.slots[t];
    float v[8] = {};
    if (slot >= 0 && slot < a.slots_total) {
        const int P = 1 << a.log_page;
        const int64_t page = slot >> a.log_page;
        const int pos = (int)(slot & (P - 1));
        constexpr int TB = (int)token_code_bytes(CT, D);
        const uint8_t *chunk = a.cache[which] + (page * a.heads + h) * chunk_bytes(CT, D, P);
        const uint16_t *scales = (const uint16_t *)(chunk + P * TB);
        const float d =
            f16_bits_to_f32(which == 0 ? scales[pos * (D / 32) + s] : scales[s * P + pos]);
        int code[8];
        if (which == 0) {
            const uint8_t *p = chunk + k_offset<CT, D>(pos, s, c);
            if constexpr (CT == TQ_Q8_0) {
                const uint2 q = *(const uint2 *)p;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    code[e] = (int)(((e < 4 ? q.x : q.y) >> (8 * (e & 3))) & 255u) - 128;
            } else {
                const uint32_t w = *(const uint32_t *)p;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    code[e] = (int)((w >> k4_shift(e)) & 15u) - 8;
            }
        } else if constexpr (CT == TQ_Q8_0) {
            const uint8_t *p = chunk + ((pos >> 2) * D + 8 * uu) * 4 + (pos & 3);
#pragma unroll
            for (int e = 0; e < 8; e++)
                code[e] = (int)p[4 * e] - 128;
        } else {
            const uint8_t *p = chunk + ((pos >> 2) * (D / 2) + 4 * uu) * 4 + v4_byte(pos & 3);
#pragma unroll
            for (int e = 0; e < 8; e++)
                code[e] = (int)((p[4 * (e >> 1)] >> (4 * (e & 1))) & 15u) - 8;
        }
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = d * (float)code[e];           // 19 bits at most: exact in fp32
    }
    store_x8<DT>(a.y[which], th * D + 8 * uu, v);
}

template <int CT, int DT>
hipError_t write_d(int D, dim3 grid, const WriteArgs &a, hipStream_t s)
{
    switch (D) {
    case 64: k_cache_write<CT, DT, 64><<<grid, THREADS, 0, s>>>(a); break;
    case 96: k_cache_write<CT, DT, 96><<<grid, THREADS, 0, s>>>(a); break;
    case 128: k_cache_write<CT, DT, 128><<<grid, THREADS, 0, s>>>(a); break;
    case 256: k_cache_write<CT, DT, 256><<<grid, THREADS, 0, s>>>(a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int CT, int DT>
hipError_t read_d(int D, dim3 grid, const ReadArgs &a, hipStream_t s)
{
    switch (D) {
    case 64: k_cache_read<CT, DT, 64><<<grid, THREADS, 0, s>>>(a); break;
    case 96: k_cache_read<CT, DT, 96><<<grid, THREADS, 0, s>>>(a); break;
    case 128: k_cache_read<CT, DT, 128><<<grid, THREADS, 0, s>>>(a); break;
    case 256: k_cache_read<CT, DT, 256><<<grid, THREADS, 0, s>>>(a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int CT, typename A>
hipError_t by_dtype(int dtype, int D, dim3 grid, const A &a, hipStream_t s)
{
    if constexpr (std::is_same_v<A, WriteArgs>) {
        switch (dtype) {
        case TQ_F32: return write_d<CT, TQ_F32>(D, grid, a, s);
        case TQ_BF16: return write_d<CT, TQ_BF16>(D, grid, a, s);
        case TQ_F16: return write_d<CT, TQ_F16>(D, grid, a, s);
        }
    } else {
        switch (dtype) {
        case TQ_F32: return read_d<CT, TQ_F32>(D, grid, a, s);
        case TQ_BF16: return read_d<CT, TQ_BF16>(D, grid, a, s);
        case TQ_F16: return read_d<CT, TQ_F16>(D, grid, a, s);
        }
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_write(const CacheShape &c, int dtype, const void *k, int64_t k_ts,
                              int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs,
                              int64_t tokens, const int32_t *slots, void *k_cache, void *v_cache,
                              hipStream_t s)
{
    const int64_t blocks = (tokens * c.heads * (c.D / 8) + THREADS - 1) / THREADS;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    WriteArgs a{{k, v}, {k_ts, v_ts}, {k_hs, v_hs}, {(uint8_t *)k_cache, (uint8_t *)v_cache},
                slots, tokens, c.pages * c.page_size, c.heads, log2_of(c.page_size)};
    const dim3 grid((unsigned)blocks, 2);
    return c.type == TQ_Q8_0 ? by_dtype<TQ_Q8_0>(dtype, c.D, grid, a, s)
                             : by_dtype<TQ_Q4_0>(dtype, c.D, grid, a, s);
}

hipError_t launch_cache_read(const CacheShape &c, int dtype, const void *k_cache,
                             const void *v_cache, const int32_t *slots, int64_t tokens, void *k,
                             void *v, hipStream_t s)
{
    const int64_t blocks = (tokens * c.heads * (c.D / 8) + THREADS - 1) / THREADS;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    ReadArgs a{{(const uint8_t *)k_cache, (const uint8_t *)v_cache}, {k, v}, slots, tokens,
               c.pages * c.page_size, c.heads, log2_of(c.page_size)};
    const dim3 grid((unsigned)blocks, 2);
    return c.type == TQ_Q8_0 ? by_dtype<TQ_Q8_0>(dtype, c.D, grid, a, s)
                             : by_dtype<TQ_Q4_0>(dtype, c.D, grid, a, s);
}

}  // namespace tq
