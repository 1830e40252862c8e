// Attention of new tokens (one, a chain or a tree of drafted ones) over the
// paged block-quantized cache (tq_tree_attention).
//
//   o[t] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q[t] . k_j),
//
// over the keys j that token t sees: all cached keys before the new tokens,
// and the new tokens its mask row names.  One pass over the keys with a
// running reference m in the exponent: p_j = 2^(c s_j - m), m raised (and the
// sums rescaled) only when some score passes it by 2^RAISE.
//
// Bound: a single token's step reads every cached byte once and is bound by
// HBM; trees multiply each dequantized key with many rows and are bound by
// the matrix cores and the vector work around them.
//
// Split: rows are (token, query head) pairs of one key head, 16 per matrix
// tile, QT tiles per wave, so a cached byte serves all the query heads and
// tokens of its head.  The four waves of a workgroup take every fourth group
// of 32 keys of the workgroup's key range; the ranges of a long cache go to
// several workgroups, whose sums k_attn_combine joins.
//
// Keys and values go from memory through registers into the matrix cores
// (v_mfma_f32_16x16x32_f16), without LDS: S^T = K Q^T leaves query columns in
// lanes and keys in registers, which is the operand layout of O^T = V^T P^T
// once lane group g's tokens are 4g..4g+3 of each 16 (cache_layout.h places
// the codes to match).
//
// Rounding: the queries enter as fp16 after a scaling of each row by a power
// of two that puts its largest element in [2^14, 2^15) (bf16 elements down to
// 2^-17 of that stay exact, below it they err by at most 2^-40 of the
// largest); code * scale of a key or value rounds once to fp16 (2^-11), as do
// the probabilities (taken times 2^BIAS against underflow: exact to 2^-11
// down to 2^-24 of the reference).  Scores, sums and outputs are fp32.
#include <algorithm>

#include "cache_layout.h"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;
constexpr int STEP = 32;                         // keys per wave and step
constexpr int STRIDE = STEP * WAVES;
constexpr float RAISE = 4.0f, BIAS = 10.0f;      // p <= 2^(RAISE + BIAS) = 2^14
constexpr float NO_REF = -1e30f;
constexpr int RED = 8;                           // fragments joined at a time

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

template <int CT, int D> struct Geo {
    static constexpr int NB = D / 32;            // 32-element blocks = matrix steps of Q K^T
    static constexpr int NT = D / 16;            // 16-element tiles of the output
    static constexpr int KW = CT == TQ_Q8_0 ? D / 16 : D / 32;   // code dwords per lane and 16 keys
    // values: elements next to each other in a lane, and 16 * CW apart
    static constexpr int CW = CT == TQ_Q8_0 ? (D % 64 == 0 ? 4 : 2)
                                            : (D % 128 == 0 ? 8 : (D % 64 == 0 ? 4 : 2));
    static constexpr int NH = D / (16 * CW);
    static constexpr int VL = CT == TQ_Q8_0 ? CW : CW / 2;       // code dwords per load
    static constexpr int TB = (int)token_code_bytes(CT, D);
};

// 32 keys' codes and scales as one lane loads them (two 16-key tiles).
template <int CT, int D> struct Raw {
    using G = Geo<CT, D>;
    uint32_t k[2][G::KW], ks[2][(G::NB + 1) / 2];
    uint32_t v[2][G::KW];
    uint2 vs[2][G::NH];
};

template <int N> __device__ __forceinline__ void load_words(uint32_t *w, const uint8_t *p)
{
    if constexpr (N == 4) {
        const uint4 x = *(const uint4 *)p;
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (N == 3) {
        const uint32_t *q = (const uint32_t *)p;
        w[0] = q[0]; w[1] = q[1]; w[2] = q[2];
    } else if constexpr (N == 2) {
        const uint2 x = *(const uint2 *)p;
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = *(const uint32_t *)p;
    }
}

// Tile T (16 keys at position pos of its page) of a step.
template <int CT, int D, int T>
__device__ __forceinline__ void load_tile(Raw<CT, D> &raw, const uint8_t *kc, const uint8_t *vc,
                                          int pos, int P, int lane)
{
    using G = Geo<CT, D>;
    const int r = lane & 15, g = lane >> 4;
    const int key = pos + r;
    if constexpr (CT == TQ_Q8_0 && D % 64 != 0) {
#pragma unroll
        for (int s = 0; s < G::NB; s++)
            load_words<2>(raw.k[T] + 2 * s, kc + key * G::TB + k_piece_off<CT, D>(s, g));
    } else if constexpr (CT == TQ_Q4_0 && D % 128 != 0) {
        load_words<G::KW>(raw.k[T], kc + key * G::TB + k_piece_off<CT, D>(0, g));
    } else {
        constexpr int PER = CT == TQ_Q8_0 ? 2 : 4;           // blocks per 16 bytes
#pragma unroll
        for (int s = 0; s < G::NB; s += PER)
            load_words<4>(raw.k[T] + s * (4 / PER), kc + key * G::TB + k_piece_off<CT, D>(s, g));
    }
    const uint8_t *ks = kc + P * G::TB + key * (G::NB * 2);
    if constexpr (G::NB == 3) {
        const uint16_t *q = (const uint16_t *)ks;
        raw.ks[T][0] = q[0] | ((uint32_t)q[1] << 16);
        raw.ks[T][1] = q[2];
    } else {
        load_words<G::NB / 2>(raw.ks[T], ks);
    }
    const int quad = (pos >> 2) + g;
    const uint8_t *vs = vc + P * G::TB;
#pragma unroll
    for (int h = 0; h < G::NH; h++) {
        load_words<G::VL>(raw.v[T] + h * G::VL,
                          vc + (quad * (4 * G::TB) + (16 * h + r) * (G::VL * 4)));
        const int block = (16 * G::CW * h + G::CW * r) / 32;
        raw.vs[T][h] = *(const uint2 *)(vs + (block * P + pos + 4 * g) * 2);
    }
}

__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ uint32_t as_u32(h2 h) { return __builtin_bit_cast(uint32_t, h); }

// Codes to fp16 pairs: with 0x64 above it a byte u reads 1024 + u, so one
// subtraction gives the signed code exactly.
__device__ __forceinline__ void codes8(uint32_t w, h2 &a, h2 &b)
{
    const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    a = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
    b = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
}

__device__ __forceinline__ h2 codes4(uint32_t w)
{
    const h2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
    return as_h2((w & 0x000f000fu) | 0x64006400u) - off;
}

union Frag {
    h2 p[4];
    h8 v;
};

// Block s of the lane's key in tile T: 8 elements.
template <int CT, int D>
__device__ __forceinline__ h8 key_frag(const Raw<CT, D> &raw, int T, int s)
{
    Frag f;
    if constexpr (CT == TQ_Q8_0) {
        codes8(raw.k[T][2 * s], f.p[0], f.p[1]);
        codes8(raw.k[T][2 * s + 1], f.p[2], f.p[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            f.p[i] = codes4(raw.k[T][s] >> (4 * i));
    }
    const h2 two = as_h2(raw.ks[T][s >> 1]);
    const _Float16 d = s & 1 ? two.y : two.x;
    const h2 dd = {d, d};
#pragma unroll
    for (int i = 0; i < 4; i++)
        f.p[i] *= dd;
    return f.v;
}

// Element j of the lane's group h of values: 8 tokens (4 of each tile).
template <int CT, int D>
__device__ __forceinline__ h8 value_frag(const Raw<CT, D> &raw, int h, int j)
{
    using G = Geo<CT, D>;
    Frag f;
#pragma unroll
    for (int T = 0; T < 2; T++) {
        if constexpr (CT == TQ_Q8_0) {
            codes8(raw.v[T][h * G::VL + j], f.p[2 * T], f.p[2 * T + 1]);
        } else {
            const uint32_t w = raw.v[T][h * G::VL + (j >> 1)] >> (4 * (j & 1));
            f.p[2 * T] = codes4(w);
            f.p[2 * T + 1] = codes4(w >> 8);
        }
        f.p[2 * T] *= as_h2(raw.vs[T][h].x);
        f.p[2 * T + 1] *= as_h2(raw.vs[T][h].y);
    }
    return f.v;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ float load_16(const void *p, int64_t i, int dtype)
{
    const uint16_t b = ((const uint16_t *)p)[i];
    return dtype == TQ_BF16 ? __builtin_bit_cast(float, (uint32_t)b << 16) : f16_bits_to_f32(b);
}

// The rows of one workgroup: sequence b, key head h, row block rb; row r is
// (token r / group, query head h * group + r % group).
struct Rows {
    int b, h, rb, group, T, ctx, L;
    int64_t tok0;
};

__device__ __forceinline__ Rows rows_of(const AttnArgs &a, int row_blocks, int64_t unit)
{
    Rows w;
    w.rb = (int)(unit % row_blocks);
    const int64_t bh = unit / row_blocks;
    w.h = (int)(bh % a.kv_heads);
    w.b = (int)(bh / a.kv_heads);
    w.group = a.heads / a.kv_heads;
    // lengths and starts are held inside the buffers whatever they say
    const int64_t s0 = min(max((int64_t)uniform(a.starts[w.b]), (int64_t)0), a.tokens);
    const int64_t s1 = min((int64_t)uniform(a.starts[w.b + 1]), a.tokens);
    w.tok0 = s0;
    w.T = (int)min(max(s1 - s0, (int64_t)0), (int64_t)a.max_nodes);
    w.ctx = max(uniform(a.ctx[w.b]), 0);
    const int64_t most = (int64_t)a.table_pages << a.log_page;
    w.L = (int)min((int64_t)w.ctx + w.T, most);
    return w;
}

// Ranges of keys that sequence w is cut into: range 0 always counts, the last
// takes what the launch did not foresee.
__device__ __forceinline__ int ranges_of(const Rows &w, int splits, int chunk)
{
    return (int)max((int64_t)1, min((int64_t)splits, ((int64_t)w.L + chunk - 1) / chunk));
}

// Fragment (query tile qt, output tile t) of a row block, as every wave holds
// it: lane's query column lane & 15, elements of rows 4 (lane >> 4) + 0..3.
template <int CT, int D>
__device__ __forceinline__ void store_frag(const AttnArgs &a, const Rows &w, int QT, int qt, int t,
                                           int lane, f4 o)
{
    using G = Geo<CT, D>;
    const int r = (w.rb * QT + qt) * 16 + (lane & 15);
    if (r >= w.T * w.group)
        return;
    const int node = r / w.group;
    const int64_t at = (w.tok0 + node) * a.yts + (w.h * w.group + r - node * w.group) * a.yhs;
    const int d0 = 16 * G::CW * (t / G::CW) + t % G::CW + 4 * (lane >> 4) * G::CW;
    uint16_t *y = (uint16_t *)a.y + at + d0;
#pragma unroll
    for (int e = 0; e < 4; e++)
        y[G::CW * e] = a.dtype == TQ_BF16 ? f32_to_16<TQ_BF16>(o[e]) : f32_to_16<TQ_F16>(o[e]);
}

template <int CT, int D, int QT>
__global__ __launch_bounds__(THREADS) void k_attn(AttnArgs a, int row_blocks, int splits, int chunk,
                                                  float *__restrict__ part,
                                                  float *__restrict__ part_ml)
{
    using G = Geo<CT, D>;
    __shared__ f4 red[WAVES][RED][64];
    __shared__ float ml[WAVES][QT * 16][2];

    // consecutive workgroups go to the 8 dies in turn: the row blocks of one
    // key range follow each other on one die, whose cache then serves them
    const int64_t keyed = (int64_t)a.batch * a.kv_heads * splits;    // (b, h, range)
    const int64_t id = blockIdx.x;
    int64_t kr;
    int rb;
    if (id < keyed / 8 * 8 * row_blocks) {
        const int64_t q = id >> 3;
        kr = q / row_blocks * 8 + (id & 7);
        rb = (int)(q % row_blocks);
    } else {
        const int64_t left = id - keyed / 8 * 8 * row_blocks;
        kr = keyed / 8 * 8 + left / row_blocks;
        rb = (int)(left % row_blocks);
    }
    const int range = (int)(kr % splits);
    const int64_t unit = kr / splits * row_blocks + rb;
    const Rows w = rows_of(a, row_blocks, unit);
    if (rb * (16 * QT) >= w.T * w.group)
        return;
    const int ranges = ranges_of(w, splits, chunk);
    if (range >= ranges)
        return;
    const int begin = range * chunk;
    const int end = range == ranges - 1 ? w.L : begin + chunk;

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int P = 1 << a.log_page;
    const int64_t cb = chunk_bytes(CT, D, P);
    const int32_t *table = a.table + w.b * a.table_stride;

    // queries: fp16 after the row's power of two, c = what a score is times
    h8 q[QT][G::NB];
    float c[QT], m[QT], l[QT];
    int node[QT];
    f4 o[QT][G::NT];
#pragma unroll
    for (int i = 0; i < QT; i++) {
        const int r = (rb * QT + i) * 16 + col;
        const bool live = r < w.T * w.group;
        node[i] = live ? r / w.group : 0;
        const int64_t at =
            (w.tok0 + node[i]) * a.qts + (w.h * w.group + (live ? r - node[i] * w.group : 0)) * a.qhs;
        float x[G::NB][8], big = 0.0f;
#pragma unroll
        for (int s = 0; s < G::NB; s++)
#pragma unroll
            for (int e = 0; e < 8; e++) {
                x[s][e] = live ? load_16(a.q, at + 32 * s + 8 * g + e, a.dtype) : 0.0f;
                big = fmaxf(big, fabsf(x[s][e]));
            }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        // 2^k with big * 2^k in [2^14, 2^15); 1 for a row of zeros or with an infinity
        const int ex = (int)(__builtin_bit_cast(uint32_t, big) >> 23);
        const int k = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -126), 126);
        const float up = __builtin_bit_cast(float, (uint32_t)(127 + k) << 23);
        const float down = __builtin_bit_cast(float, (uint32_t)(127 - k) << 23);
#pragma unroll
        for (int s = 0; s < G::NB; s++)
#pragma unroll
            for (int e = 0; e < 8; e++)
                q[i][s][e] = (_Float16)(x[s][e] * up);
        c[i] = a.scale * 1.44269504088896f * down;
        m[i] = NO_REF;
        l[i] = 0.0f;
#pragma unroll
        for (int t = 0; t < G::NT; t++)
            o[i][t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // page of each of the two tiles at key kb; -1 where the table has none
    auto page_at = [&](int key) {
        const int i = key >> a.log_page;
        return i < a.table_pages && key < end ? table[i] : -1;
    };
    auto mapped = [&](int page) { return page >= 0 && page < a.pages; };
    struct Pages {
        int a, b;
    };
    auto pages_at = [&](int kb) { return Pages{page_at(kb), page_at(kb + 16)}; };

    auto load = [&](Raw<CT, D> &raw, Pages &pg, int kb) {
        pg.a = uniform(pg.a);
        pg.b = uniform(pg.b);
        if (kb >= end)
            return;
        // an unmapped tile's loads go to page 0; its keys are masked
        const int64_t pa = mapped(pg.a) ? pg.a : 0, pb = mapped(pg.b) ? pg.b : 0;
        const int64_t oa = (pa * a.kv_heads + w.h) * cb, ob = (pb * a.kv_heads + w.h) * cb;
        load_tile<CT, D, 0>(raw, a.kc + oa, a.vc + oa, kb & (P - 1), P, lane);
        load_tile<CT, D, 1>(raw, a.kc + ob, a.vc + ob, (kb + 16) & (P - 1), P, lane);
    };

    auto compute = [&](Raw<CT, D> &raw, const Pages &pg, int kb) {
        f4 s[QT][2];
#pragma unroll
        for (int T = 0; T < 2; T++) {
#pragma unroll
            for (int i = 0; i < QT; i++)
                s[i][T] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int b = 0; b < G::NB; b++) {
                const h8 kf = key_frag<CT, D>(raw, T, b);
#pragma unroll
                for (int i = 0; i < QT; i++)
                    s[i][T] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[i][b], s[i][T], 0, 0, 0);
            }
        }
        const bool oka = mapped(pg.a), okb = mapped(pg.b);
        if (kb + STEP > w.ctx || !oka || !okb) {
            // some keys are new tokens, past the end or unmapped
#pragma unroll
            for (int T = 0; T < 2; T++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int key = kb + 16 * T + 4 * g + e;
                    const bool there = key < w.L && (T ? okb : oka);
                    const int n = key - w.ctx;
#pragma unroll
                    for (int i = 0; i < QT; i++) {
                        bool see = there;
                        if (there && n >= 0) {
                            if (!a.mask)
                                see = n <= node[i];
                            else
                                see = (n >> 5) < a.mask_words &&
                                      ((a.mask[(w.tok0 + node[i]) * a.mask_stride + (n >> 5)] >>
                                        (n & 31)) & 1u);
                        }
                        if (!see)
                            s[i][T][e] = -__builtin_inff();
                    }
                    // what a value block holds where no token was written
                    // must not meet a probability of 0 as NaN
#pragma unroll
                    for (int h = 0; h < G::NH; h++) {
                        uint32_t &word = e < 2 ? raw.vs[T][h].x : raw.vs[T][h].y;
                        const int sh = 16 * (e & 1);
                        const bool odd = ((word >> sh) & 0x7C00u) == 0x7C00u;
                        if (!there || (n >= 0 && odd))
                            word &= ~(0xFFFFu << sh);
                    }
                }
        }
        h8 p[QT];
#pragma unroll
        for (int i = 0; i < QT; i++) {
            float top = fmaxf(fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3])),
                              fmaxf(fmaxf(s[i][1][0], s[i][1][1]), fmaxf(s[i][1][2], s[i][1][3])));
            top *= c[i];
            if (__any(top > m[i] + RAISE)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float mn = fmaxf(m[i], top);
                const float f = __builtin_amdgcn_exp2f(m[i] - mn);
                m[i] = mn;
                l[i] *= f;
#pragma unroll
                for (int t = 0; t < G::NT; t++)
                    o[i][t] *= f;
            }
            const float ref = BIAS - m[i];
#pragma unroll
            for (int T = 0; T < 2; T++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float x = __builtin_amdgcn_exp2f(fmaf(s[i][T][e], c[i], ref));
                    l[i] += x;
                    p[i][4 * T + e] = (_Float16)x;
                }
        }
#pragma unroll
        for (int t = 0; t < G::NT; t++) {
            const h8 vf = value_frag<CT, D>(raw, t / G::CW, t % G::CW);
#pragma unroll
            for (int i = 0; i < QT; i++)
                o[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[i], o[i][t], 0, 0, 0);
        }
    };

    // two steps in flight: one computed, the next one's codes and the page
    // numbers of the one after that being loaded
    int kb = begin + wave * STEP;
    if (kb < end) {
        Raw<CT, D> ra, rb2;
        Pages pa = pages_at(kb), pb = pages_at(kb + STRIDE);
        load(ra, pa, kb);
        for (;;) {
            load(rb2, pb, kb + STRIDE);
            Pages pn = pages_at(kb + 2 * STRIDE);
            compute(ra, pa, kb);
            pa = pn;
            kb += STRIDE;
            if (kb >= end)
                break;
            load(ra, pa, kb + STRIDE);
            pn = pages_at(kb + 2 * STRIDE);
            compute(rb2, pb, kb);
            pb = pn;
            kb += STRIDE;
            if (kb >= end)
                break;
        }
    }

    // join the four waves: references, then the outputs RED fragments at a time
#pragma unroll
    for (int i = 0; i < QT; i++) {
        l[i] += __shfl_xor(l[i], 16);
        l[i] += __shfl_xor(l[i], 32);
        if (g == 0) {
            ml[wave][i * 16 + col][0] = m[i];
            ml[wave][i * 16 + col][1] = l[i];
        }
    }
    __syncthreads();
    float all_m[QT], all_l[QT], f[QT];
#pragma unroll
    for (int i = 0; i < QT; i++) {
        float mm = NO_REF;
#pragma unroll
        for (int k = 0; k < WAVES; k++)
            mm = fmaxf(mm, ml[k][i * 16 + col][0]);
        float ll = 0.0f;
#pragma unroll
        for (int k = 0; k < WAVES; k++)
            ll += ml[k][i * 16 + col][1] * __builtin_amdgcn_exp2f(ml[k][i * 16 + col][0] - mm);
        all_m[i] = mm;
        all_l[i] = ll;
        f[i] = __builtin_amdgcn_exp2f(m[i] - mm);
    }
    constexpr int F = QT * G::NT;
    const int64_t slot = unit * splits + range;
    if (ranges > 1 && wave == 0 && g == 0) {
#pragma unroll
        for (int i = 0; i < QT; i++) {
            part_ml[(slot * (QT * 16) + i * 16 + col) * 2] = all_m[i];
            part_ml[(slot * (QT * 16) + i * 16 + col) * 2 + 1] = all_l[i];
        }
    }
#pragma unroll
    for (int f0 = 0; f0 < F; f0 += RED) {
        if (f0)
            __syncthreads();
#pragma unroll
        for (int k = 0; k < RED; k++)
            if (f0 + k < F)
                red[wave][k][lane] = o[(f0 + k) / G::NT][(f0 + k) % G::NT] * f[(f0 + k) / G::NT];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RED / WAVES; k++) {
            const int kk = wave * (RED / WAVES) + k, ff = f0 + kk;
            if (ff >= F)
                continue;
            const f4 sum = (red[0][kk][lane] + red[1][kk][lane]) +
                           (red[2][kk][lane] + red[3][kk][lane]);
            if (ranges > 1) {
                *(f4 *)(part + ((slot * F + ff) * 64 + lane) * 4) = sum;
            } else {
                float ll = all_l[0];
#pragma unroll
                for (int i = 1; i < QT; i++)
                    ll = ff / G::NT == i ? all_l[i] : ll;
                // nothing seen: zeros
                store_frag<CT, D>(a, w, QT, ff / G::NT, ff % G::NT, lane,
                                  ll == 0.0f ? f4{0, 0, 0, 0} : sum * (1.0f / ll));
            }
        }
    }
}

// One wave per fragment: the ranges' sums, each rescaled to the largest
// reference, in range order.
template <int CT, int D>
__global__ __launch_bounds__(THREADS) void k_attn_combine(AttnArgs a, int QT, int row_blocks,
                                                          int splits, int chunk,
                                                          const float *__restrict__ part,
                                                          const float *__restrict__ part_ml)
{
    using G = Geo<CT, D>;
    const int64_t unit = blockIdx.x;
    const Rows w = rows_of(a, row_blocks, unit);
    if (w.rb * (16 * QT) >= w.T * w.group)
        return;
    const int ranges = ranges_of(w, splits, chunk);
    const int F = QT * G::NT;
    const int lane = threadIdx.x & 63, ff = blockIdx.y * WAVES + (threadIdx.x >> 6);
    if (ranges == 1 || ff >= F)
        return;
    const int qt = ff / G::NT;
    const float *mlp = part_ml + (unit * splits * (QT * 16) + qt * 16 + (lane & 15)) * 2;
    const int64_t ms = QT * 32;
    float mm = NO_REF;
    for (int k = 0; k < ranges; k++)
        mm = fmaxf(mm, mlp[k * ms]);
    float ll = 0.0f;
    f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < ranges; k++) {
        const float f = __builtin_amdgcn_exp2f(mlp[k * ms] - mm);
        ll += f * mlp[k * ms + 1];
        sum += f * *(const f4 *)(part + (((unit * splits + k) * F + ff) * 64 + lane) * 4);
    }
    store_frag<CT, D>(a, w, QT, qt, ff % G::NT, lane,
                      ll == 0.0f ? f4{0, 0, 0, 0} : sum * (1.0f / ll));
}

template <int CT, int D>
hipError_t launch_cd(const AttnArgs &a, const AttnPlan &p, void *scratch, hipStream_t s)
{
    const int64_t units = (int64_t)a.batch * a.kv_heads * p.row_blocks;
    const int64_t blocks = units * p.splits;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    const int F = p.qt * (D / 16);
    float *part = (float *)scratch;
    float *ml = part ? part + (size_t)units * p.splits * F * 256 : nullptr;
    const dim3 grid((unsigned)blocks);
    switch (p.qt) {
    case 1: k_attn<CT, D, 1><<<grid, THREADS, 0, s>>>(a, p.row_blocks, p.splits, p.chunk, part, ml); break;
    case 2: k_attn<CT, D, 2><<<grid, THREADS, 0, s>>>(a, p.row_blocks, p.splits, p.chunk, part, ml); break;
    default:
        if constexpr (D <= 128) {
            k_attn<CT, D, 4><<<grid, THREADS, 0, s>>>(a, p.row_blocks, p.splits, p.chunk, part, ml);
            break;
        } else {
            return hipErrorInvalidValue;
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const dim3 cgrid((unsigned)units, (unsigned)((F + WAVES - 1) / WAVES));
    k_attn_combine<CT, D><<<cgrid, THREADS, 0, s>>>(a, p.qt, p.row_blocks, p.splits, p.chunk, part, ml);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_c(int D, const AttnArgs &a, const AttnPlan &p, void *scratch, hipStream_t s)
{
    switch (D) {
    case 64: return launch_cd<CT, 64>(a, p, scratch, s);
    case 96: return launch_cd<CT, 96>(a, p, scratch, s);
    case 128: return launch_cd<CT, 128>(a, p, scratch, s);
    case 256: return launch_cd<CT, 256>(a, p, scratch, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

AttnPlan attn_plan(int D, int64_t batch, int64_t heads, int64_t kv_heads, int64_t max_nodes,
                   int64_t max_keys)
{
    AttnPlan p;
    const int64_t rows = max_nodes * (heads / kv_heads);
    p.qt = rows <= 16 ? 1 : (rows <= 32 || D > 128 ? 2 : 4);
    p.row_blocks = (int)((rows + 16 * p.qt - 1) / (16 * p.qt));
    const int64_t units = batch * kv_heads * p.row_blocks;
    const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(units, 1));
    const int64_t most = std::max<int64_t>(1, (max_keys + 255) / 256);
    const int64_t s = std::min(want, most);
    const int64_t chunk = ((max_keys + s - 1) / s + STRIDE - 1) / STRIDE * STRIDE;
    p.chunk = (int)std::max<int64_t>(chunk, STRIDE);
    p.splits = (int)std::max<int64_t>(1, (max_keys + p.chunk - 1) / p.chunk);
    return p;
}

size_t attn_scratch_bytes(const AttnPlan &p, int D, int64_t batch, int64_t kv_heads)
{
    if (p.splits == 1)
        return 0;
    const size_t units = (size_t)batch * kv_heads * p.row_blocks * p.splits;
    return units * ((size_t)p.qt * (D / 16) * 256 + p.qt * 32) * sizeof(float);
}

hipError_t launch_attention(int cache_type, int D, const AttnArgs &a, const AttnPlan &p,
                            uint32_t *, void *scratch, hipStream_t s)
{
    return cache_type == TQ_Q8_0 ? launch_c<TQ_Q8_0>(D, a, p, scratch, s)
                                 : launch_c<TQ_Q4_0>(D, a, p, scratch, s);
}

}  // namespace tq
