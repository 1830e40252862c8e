// Paged key / value cache held in 32-element quantized blocks: tokens are
// quantized as they are written (tq_cache_write) and read back as the values
// their blocks stand for (tq_cache_read).  The layout is cache_layout.h.
//
// Both kernels only move data (about 3 bytes of traffic per bf16 element
// stored, one pass).  A quad of lanes holds one 32-element block, 8 elements
// per lane, as in the activation quantization, of four tokens in a row: where
// those fill one group of four positions (a prompt's do), the values' bytes of
// four tokens leave and enter as whole dwords, 32 bytes a lane, and the two
// lanes that share pieces of Q8_0 keys trade tokens for whole pieces, 32 bytes
// a lane too; else one by one.  8192 tokens of 8 heads of 128 in bf16: 13.4 us
// written (key halves apart and loads after the slots: 16; byte by byte 33),
// 10.7 us read (14, 24); a copy of as many bytes takes 10.6.
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

// Four tokens in a row: those of one group of four positions if the slots run
// on from the first call's first slot.
struct Group {
    int64_t t0;                      // first token, may lie before 0
    int64_t slot[4];                 // -1: no such token or slot
    bool whole;                      // slots 4n, 4n + 1, 4n + 2, 4n + 3
};

__device__ __forceinline__ Group group_at(const int32_t *slots, int64_t tokens, int64_t slots_total,
                                          int64_t n)
{
    Group q;
    q.t0 = 4 * n - (slots[0] & 3);
    q.whole = true;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t t = q.t0 + i;
        const int64_t s = t >= 0 && t < tokens ? (int64_t)slots[t] : -1;
        q.slot[i] = s >= 0 && s < slots_total ? s : -1;
        q.whole = q.whole && q.slot[i] >= 0 && q.slot[i] == (q.slot[0] & ~int64_t(3)) + i;
    }
    return q;
}

// Which (group, head, unit of 8 elements) a lane has.
template <int D> struct Unit {
    int64_t group;
    int h, uu;
    bool live;
    __device__ __forceinline__ Unit(int64_t tokens, int heads, uint32_t block)
    {
        constexpr uint32_t UPH = D / 8;
        const uint32_t u = block * (uint32_t)THREADS + threadIdx.x, per = heads * UPH;
        const uint32_t g = u / per, rest = u - g * per;
        group = g;
        h = (int)(rest / UPH);
        uu = (int)(rest % UPH);
        live = group < (tokens + 6) / 4;
    }
};

// One token's codes of a lane: element order, but for a Q4_0 key's shifts.
template <int CT> __device__ __forceinline__ uint2 key_codes(uint2 code)
{
    if constexpr (CT == TQ_Q8_0)
        return code;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; e++)
        w |= ((code.x >> (4 * e)) & 15u) << k4_shift(e);
    return make_uint2(w, 0);
}

template <int CT, int D>
__device__ __forceinline__ void store_key(uint8_t *chunk, int pos, int s, int c, uint2 code)
{
    code = key_codes<CT>(code);
    uint8_t *p = chunk + k_offset<CT, D>(pos, s, c);
    if constexpr (CT == TQ_Q8_0)
        *(uint2 *)p = code;
    else
        *(uint32_t *)p = code.x;
}

// Q8_0 pieces of two blocks' codes.
template <int CT, int D> constexpr bool shared_piece()
{
    return CT == TQ_Q8_0 && k_piece<CT, D>() == 16;
}

// Four tokens in a row of one block: the two lanes whose blocks share pieces
// exchange tokens, and each stores two whole pieces.
template <int CT, int D>
__device__ __forceinline__ void store_keys(uint8_t *chunk, int pos, int s, int c,
                                           const uint2 (&code)[4])
{
    if constexpr (shared_piece<CT, D>()) {
        const bool odd = s & 1;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint2 keep = odd ? code[2 + j] : code[j], give = odd ? code[j] : code[2 + j];
            const uint2 got = make_uint2(__shfl_xor(give.x, 4), __shfl_xor(give.y, 4));
            uint4 w = odd ? make_uint4(got.x, got.y, keep.x, keep.y)
                          : make_uint4(keep.x, keep.y, got.x, got.y);
            *(uint4 *)(chunk + k_offset<CT, D>(pos + 2 * odd + j, s & ~1, c)) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            store_key<CT, D>(chunk, pos + i, s, c, code[i]);
    }
}

// blockIdx.y picks keys or values.
template <int CT, int DT, int D>
__global__ __launch_bounds__(THREADS) void k_cache_write(WriteArgs a)
{
    const int which = blockIdx.y;
    const Unit<D> u(a.tokens, a.heads, blockIdx.x);
    if (!u.live)
        return;                                  // uniform across the quad of a block
    const int s = u.uu >> 2, c = u.uu & 3;
    const Group q = group_at(a.slots, a.tokens, a.slots_total, u.group);
    const int P = 1 << a.log_page;
    constexpr int TB = (int)token_code_bytes(CT, D);
    uint2 code[4];
    uint16_t db[4];
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        // whatever the slot, so that the loads do not wait for it
        const int64_t t = min(max(q.t0 + i, (int64_t)0), a.tokens - 1);
        load_x8<DT>(v[i], a.x[which], t * a.ts[which] + u.h * a.hs[which] + 8 * u.uu);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (q.slot[i] < 0)
            continue;
        code[i] = quantize_lane<CT>(v[i], c, db[i]);
        if (q.whole)
            continue;
        const int64_t page = q.slot[i] >> a.log_page;
        const int pos = (int)(q.slot[i] & (P - 1));
        uint8_t *chunk = a.cache[which] + (page * a.heads + u.h) * chunk_bytes(CT, D, P);
        uint16_t *scales = (uint16_t *)(chunk + P * TB);
        if (which == 0) {
            store_key<CT, D>(chunk, pos, s, c, code[i]);
            if (c == 0)
                scales[pos * (D / 32) + s] = db[i];
        } else {
            if constexpr (CT == TQ_Q8_0) {
                uint8_t *p = chunk + ((pos >> 2) * D + 8 * u.uu) * 4 + (pos & 3);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    p[4 * e] = (uint8_t)((e < 4 ? code[i].x : code[i].y) >> (8 * (e & 3)));
            } else {
                uint8_t *p = chunk + ((pos >> 2) * (D / 2) + 4 * u.uu) * 4 + v4_byte(pos & 3);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    p[4 * e] = (uint8_t)(code[i].x >> (8 * e));
            }
            if (c == 0)
                scales[s * P + pos] = db[i];
        }
    }
    if (!q.whole)
        return;
    const int64_t page = q.slot[0] >> a.log_page;
    const int pos = (int)(q.slot[0] & (P - 1));
    uint8_t *chunk = a.cache[which] + (page * a.heads + u.h) * chunk_bytes(CT, D, P);
    uint16_t *scales = (uint16_t *)(chunk + P * TB);
    if (which == 0) {
        store_keys<CT, D>(chunk, pos, s, c, code);
        scales[(pos + c) * (D / 32) + s] = c < 2 ? (c ? db[1] : db[0]) : (c == 2 ? db[2] : db[3]);
        return;
    }
    // byte b of the four tokens' dwords, in the order the layout asks for
    auto column = [&](uint32_t t0, uint32_t t1, uint32_t t2, uint32_t t3, int b) {
        const uint32_t pick = (uint32_t)(0x0C0C0400 + 0x0101 * b);
        const uint32_t lo = __builtin_amdgcn_perm(t1, t0, pick), hi = __builtin_amdgcn_perm(t3, t2, pick);
        return lo | (hi << 16);
    };
    if constexpr (CT == TQ_Q8_0) {
        uint4 *p = (uint4 *)(chunk + ((pos >> 2) * D + 8 * u.uu) * 4);
        p[0] = make_uint4(column(code[0].x, code[1].x, code[2].x, code[3].x, 0),
                          column(code[0].x, code[1].x, code[2].x, code[3].x, 1),
                          column(code[0].x, code[1].x, code[2].x, code[3].x, 2),
                          column(code[0].x, code[1].x, code[2].x, code[3].x, 3));
        p[1] = make_uint4(column(code[0].y, code[1].y, code[2].y, code[3].y, 0),
                          column(code[0].y, code[1].y, code[2].y, code[3].y, 1),
                          column(code[0].y, code[1].y, code[2].y, code[3].y, 2),
                          column(code[0].y, code[1].y, code[2].y, code[3].y, 3));
    } else {
        // tokens 0, 2, 1, 3 (v4_byte)
        uint4 *p = (uint4 *)(chunk + ((pos >> 2) * (D / 2) + 4 * u.uu) * 4);
        p[0] = make_uint4(column(code[0].x, code[2].x, code[1].x, code[3].x, 0),
                          column(code[0].x, code[2].x, code[1].x, code[3].x, 1),
                          column(code[0].x, code[2].x, code[1].x, code[3].x, 2),
                          column(code[0].x, code[2].x, code[1].x, code[3].x, 3));
    }
    if (c == 0)
        *(uint2 *)(scales + s * P + pos) =
            make_uint2(db[0] | ((uint32_t)db[1] << 16), db[2] | ((uint32_t)db[3] << 16));
}

struct ReadArgs {
    const uint8_t *cache[2];
    void *y[2];                  // [tokens][heads][D], contiguous
    const int32_t *slots;
    int64_t tokens, slots_total;
    int heads, log_page;
};

// One token's codes of a lane, as store_key left them.
template <int CT, int D>
__device__ __forceinline__ uint2 load_key(const uint8_t *chunk, int pos, int s, int c)
{
    const uint8_t *p = chunk + k_offset<CT, D>(pos, s, c);
    if constexpr (CT == TQ_Q8_0)
        return *(const uint2 *)p;
    else
        return make_uint2(*(const uint32_t *)p, 0);
}

// Four tokens in a row of one block: store_keys the other way round.
template <int CT, int D>
__device__ __forceinline__ void load_keys(uint2 (&code)[4], const uint8_t *chunk, int pos, int s,
                                          int c)
{
    if constexpr (shared_piece<CT, D>()) {
        const bool odd = s & 1;
        uint4 w[2];
#pragma unroll
        for (int j = 0; j < 2; j++)
            w[j] = *(const uint4 *)(chunk + k_offset<CT, D>(pos + 2 * odd + j, s & ~1, c));
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint2 lo = make_uint2(w[j].x, w[j].y), hi = make_uint2(w[j].z, w[j].w);
            const uint2 keep = odd ? hi : lo, give = odd ? lo : hi;
            const uint2 got = make_uint2(__shfl_xor(give.x, 4), __shfl_xor(give.y, 4));
            code[j] = odd ? got : keep;
            code[2 + j] = odd ? keep : got;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            code[i] = load_key<CT, D>(chunk, pos + i, s, c);
    }
}

// One token's value codes: 8 bytes, or nibbles in element order.
template <int CT, int D>
__device__ __forceinline__ uint2 load_value(const uint8_t *chunk, int pos, int uu)
{
    uint2 w = make_uint2(0, 0);
    if constexpr (CT == TQ_Q8_0) {
        const uint8_t *p = chunk + ((pos >> 2) * D + 8 * uu) * 4 + (pos & 3);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            w.x |= (uint32_t)p[4 * e] << (8 * e);
            w.y |= (uint32_t)p[4 * (e + 4)] << (8 * e);
        }
    } else {
        const uint8_t *p = chunk + ((pos >> 2) * (D / 2) + 4 * uu) * 4 + v4_byte(pos & 3);
#pragma unroll
        for (int e = 0; e < 4; e++)
            w.x |= (uint32_t)p[4 * e] << (8 * e);
    }
    return w;
}

// A slot outside the cache reads as zeros.
template <int CT, int DT, int D>
__global__ __launch_bounds__(THREADS) void k_cache_read(ReadArgs a)
{
    const int which = blockIdx.y;
    // workgroups go round the eight dies: each takes a run of tokens, so that a
    // line of scales, which several share, is read by one die (17.6 MB read for
    // 8192 tokens instead of 31, 10.7 us instead of 12.1; writes took 14.1
    // instead of 13.2 so)
    const Unit<D> u(a.tokens, a.heads, (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3));
    if (!u.live)
        return;
    const int s = u.uu >> 2, c = u.uu & 3;
    const Group q = group_at(a.slots, a.tokens, a.slots_total, u.group);
    const int P = 1 << a.log_page;
    constexpr int TB = (int)token_code_bytes(CT, D);
    float v[4][8] = {};
    if (which && q.whole) {
        const int64_t page = q.slot[0] >> a.log_page;
        const int pos = (int)(q.slot[0] & (P - 1));
        const uint8_t *chunk = a.cache[1] + (page * a.heads + u.h) * chunk_bytes(CT, D, P);
        const uint2 sc = *(const uint2 *)((const uint16_t *)(chunk + P * TB) + s * P + pos);
        uint32_t w[8];
        const uint4 *p = (const uint4 *)(chunk + (pos >> 2) * (4 * TB) + u.uu * (CT == TQ_Q8_0 ? 32 : 16));
        const uint4 x = p[0];
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        if constexpr (CT == TQ_Q8_0) {
            const uint4 y = p[1];
            w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float d = f16_bits_to_f32((uint16_t)((i < 2 ? sc.x : sc.y) >> (16 * (i & 1))));
#pragma unroll
            for (int e = 0; e < 8; e++) {
                int code;
                if constexpr (CT == TQ_Q8_0)
                    code = (int)((w[e] >> (8 * i)) & 255u) - 128;
                else
                    code = (int)((w[e >> 1] >> (8 * v4_byte(i) + 4 * (e & 1))) & 15u) - 8;
                v[i][e] = d * (float)code;       // 19 bits at most: exact in fp32
            }
        }
    } else {
        // all four tokens' loads are on their way before the first is used
        uint2 code[4];
        uint16_t db[4];
        if (q.whole) {
            const int64_t page = q.slot[0] >> a.log_page;
            const int pos = (int)(q.slot[0] & (P - 1));
            const uint8_t *chunk = a.cache[0] + (page * a.heads + u.h) * chunk_bytes(CT, D, P);
            const int d = ((const uint16_t *)(chunk + P * TB))[(pos + c) * (D / 32) + s];
            load_keys<CT, D>(code, chunk, pos, s, c);
#pragma unroll
            for (int i = 0; i < 4; i++)
                db[i] = (uint16_t)__shfl(d, (int)(threadIdx.x & 60) + i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                code[i] = make_uint2(0, 0);
                db[i] = 0;
                if (q.slot[i] < 0)
                    continue;
                const int64_t page = q.slot[i] >> a.log_page;
                const int pos = (int)(q.slot[i] & (P - 1));
                const uint8_t *chunk =
                    a.cache[which] + (page * a.heads + u.h) * chunk_bytes(CT, D, P);
                db[i] = ((const uint16_t *)(chunk +
                                            P * TB))[which == 0 ? pos * (D / 32) + s : s * P + pos];
                code[i] = which == 0 ? load_key<CT, D>(chunk, pos, s, c)
                                     : load_value<CT, D>(chunk, pos, u.uu);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float d = f16_bits_to_f32(db[i]);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                int x;
                if constexpr (CT == TQ_Q8_0)
                    x = (int)(((e < 4 ? code[i].x : code[i].y) >> (8 * (e & 3))) & 255u) - 128;
                else
                    x = (int)((code[i].x >> (which == 0 ? k4_shift(e) : 4 * e)) & 15u) - 8;
                v[i][e] = d * (float)x;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t t = q.t0 + i;
        if (t >= 0 && t < a.tokens)
            store_x8<DT>(a.y[which], (t * a.heads + u.h) * D + 8 * u.uu, v[i]);
    }
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

// Groups of four tokens, the first of which may begin up to three before.
int64_t blocks_of(int64_t tokens, const CacheShape &c)
{
    return ((tokens + 6) / 4 * c.heads * (c.D / 8) + THREADS - 1) / THREADS;
}

}  // namespace

hipError_t launch_cache_write(const CacheShape &c, int dtype, const void *k, int64_t k_ts,
                              int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs,
                              int64_t tokens, const int32_t *slots, void *k_cache, void *v_cache,
                              hipStream_t s)
{
    const int64_t blocks = blocks_of(tokens, c);
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
    const int64_t blocks = (blocks_of(tokens, c) + 7) / 8 * 8;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    ReadArgs a{{(const uint8_t *)k_cache, (const uint8_t *)v_cache}, {k, v}, slots, tokens,
               c.pages * c.page_size, c.heads, log2_of(c.page_size)};
    const dim3 grid((unsigned)blocks, 2);
    return c.type == TQ_Q8_0 ? by_dtype<TQ_Q8_0>(dtype, c.D, grid, a, s)
                             : by_dtype<TQ_Q4_0>(dtype, c.D, grid, a, s);
}

}  // namespace tq
