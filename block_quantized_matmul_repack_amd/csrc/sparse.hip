// Attention over the pages that promise the most: bounds of each page's keys
// (tq_cache_bounds), and from them the pages that a step reads
// (tq_select_pages); attention.hip then takes the pages of each key head.
//
// Of each page and key head the bounds hold the largest and smallest key of each
// channel, quantized as Q8_0 blocks that both share a scale in: 32 + 32 codes
// and an fp16 scale for 32 channels, 1.5 % of a page of 64 tokens.  A page's score
// for a query row is sum_d max(q_d hi_d, q_d lo_d), which no key of the page
// passes but for the rounding; as q+ . hi + q- . lo (the positive and the negative
// part of q, in int8 blocks, too) a block is one v_mfma_i32_16x16x64_i8 for 16
// pages and 16 rows, exact, and only the scales' products and the sum over the
// D / 32 blocks are fp64: the choice of pages does not hang on rounding.  A page's
// score is the largest over the rows (new tokens times query heads of the key
// head), rounded to fp32; equal scores go to the earlier page.
#include <algorithm>

#include "block_ops.h"
#include "cache_layout.h"

namespace tq {
namespace {

typedef int i4 __attribute__((ext_vector_type(4)));

constexpr int WAVES = 4, THREADS = 64 * WAVES;
constexpr int SEL_WAVES = 16, SEL_THREADS = 64 * SEL_WAVES;

// ---- bounds ----------------------------------------------------------------

// A wave has one block of one page and head: lane (g, r) the elements 8g ..
// 8g+7 of every 16th token from r.
template <int CT, int D>
__global__ __launch_bounds__(THREADS) void k_bounds(BoundsArgs a, int pages)
{
    constexpr int NB = D / 32, TB = (int)token_code_bytes(CT, D);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const uint32_t unit = __builtin_amdgcn_readfirstlane(blockIdx.x * WAVES + (threadIdx.x >> 6));
    const int s = unit % NB, h = unit / NB % a.kv_heads, j = unit / NB / a.kv_heads;
    const int b = blockIdx.y, P = 1 << a.log_page;
    if (j >= pages)
        return;
    const int64_t begin = max(a.begin[b], 0);
    const int64_t end = min((int64_t)a.end[b], (int64_t)a.table_pages << a.log_page);
    const int64_t page = (begin >> a.log_page) + j, first = page << a.log_page;
    if (begin >= end || first >= end)
        return;
    const int64_t id = a.table[b * a.table_stride + page];
    if (id < 0 || id >= a.pages)
        return;
    const int n = (int)min(end - first, (int64_t)P);
    const uint8_t *chunk = a.k_cache + (id * a.kv_heads + h) * chunk_bytes(CT, D, P);
    const uint16_t *scales = (const uint16_t *)(chunk + P * TB);
    float hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        hi[e] = -__builtin_inff();
        lo[e] = __builtin_inff();
    }
#pragma unroll 4
    for (int pos = r; pos < n; pos += 16) {
        const uint8_t *p = chunk + k_offset<CT, D>(pos, s, g);
        const float d = f16_bits_to_f32(scales[pos * NB + s]);
        uint2 code;
        if constexpr (CT == TQ_Q8_0)
            code = *(const uint2 *)p;
        else
            code = make_uint2(*(const uint32_t *)p, 0);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            int x;
            if constexpr (CT == TQ_Q8_0)
                x = (int)(((e < 4 ? code.x : code.y) >> (8 * (e & 3))) & 255u) - 128;
            else
                x = (int)((code.x >> k4_shift(e)) & 15u) - 8;
            const float v = d * (float)x;        // 19 bits: exact
            hi[e] = fmaxf(hi[e], v);
            lo[e] = fminf(lo[e], v);
        }
    }
    float big = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        for (int m = 1; m < 16; m <<= 1) {
            hi[e] = fmaxf(hi[e], __shfl_xor(hi[e], m));
            lo[e] = fminf(lo[e], __shfl_xor(lo[e], m));
        }
        big = fmaxf(big, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
    }
    big = fmaxf(big, __shfl_xor(big, 16));
    big = fmaxf(big, __shfl_xor(big, 32));
    const float d = big / 127.0f, inv = d != 0.0f ? 1.0f / d : 0.0f;
    // lane (g, 0) writes the largest, lane (g, 1) the smallest
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e++)
        w[e >> 2] |= ((uint32_t)round_away((r ? lo[e] : hi[e]), inv) & 0xFFu) << (8 * (e & 3));
    const int64_t block = (id * a.kv_heads + h) * NB + s;
    if (r < 2)
        *(uint2 *)(a.codes + block * 64 + r * 32 + g * 8) = make_uint2(w[0], w[1]);
    if (lane == 0)
        a.scales[block] = f32_to_f16_bits(d);
}

// ---- scores ----------------------------------------------------------------

// What a step keeps of a sequence's pages: [0, first), those chosen among
// [first, tail), and [tail, total).
struct Span {
    int64_t tok0;
    int T, ctx, first, tail, total, keep;
};

__device__ __forceinline__ Span span_of(const SelectArgs &a, int b)
{
    Span s;
    const int64_t t0 = min(max((int64_t)a.starts[b], (int64_t)0), a.tokens);
    const int64_t t1 = min((int64_t)a.starts[b + 1], a.tokens);
    s.tok0 = t0;
    s.T = (int)min(max(t1 - t0, (int64_t)0), (int64_t)a.max_nodes);
    s.ctx = max(a.ctx[b], 0);
    const int64_t P = int64_t(1) << a.log_page;
    const int64_t total = min(((int64_t)s.ctx + s.T + P - 1) >> a.log_page, (int64_t)a.table_pages);
    const int64_t fresh = min((int64_t)s.ctx >> a.log_page, total);
    s.total = (int)total;
    s.tail = (int)max(fresh - a.last, (int64_t)0);
    s.first = min(a.first, s.tail);
    s.keep = min(a.keep, s.tail - s.first);
    return s;
}

// The scores of 16 pages a wave and turn, written as order keys.
template <int DT, int D> __global__ __launch_bounds__(THREADS) void k_scores(SelectArgs a, uint32_t *keys)
{
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = blockIdx.x / a.kv_heads, h = blockIdx.x - b * a.kv_heads;
    const Span sp = span_of(a, b);
    if (sp.keep == sp.tail - sp.first)
        return;                                  // all of them are read
    const int32_t *table = a.table + b * a.table_stride;
    uint32_t *out = keys + (int64_t)blockIdx.x * a.table_pages;
    const int rows = sp.T * a.group;
    for (int64_t p0 = sp.first + ((int64_t)blockIdx.y * WAVES + wave) * 16; p0 < sp.tail;
         p0 += (int64_t)gridDim.y * WAVES * 16) {
        // lane (g, r): bytes 16g .. of the codes of page p0 + r
        const int64_t page = min(p0 + r, (int64_t)sp.tail - 1);
        int64_t id = table[page];
        const bool there = id >= 0 && id < a.pages;
        id = there ? id : 0;
        const int64_t block = (id * a.kv_heads + h) * NB;
        i4 codes[NB];
        float scale[NB];
#pragma unroll
        for (int s = 0; s < NB; s++) {
            codes[s] = *(const i4 *)(a.codes + (block + s) * 64 + g * 16);
            scale[s] = f16_bits_to_f32(a.scales[block + s]);
        }
        double best[4];
#pragma unroll
        for (int e = 0; e < 4; e++)
            best[e] = -__builtin_inf();
        for (int r0 = 0; r0 < rows; r0 += 16) {
            const int row = min(r0 + r, rows - 1);                   // the last one again
            const int node = row / a.group;
            const int64_t at = (sp.tok0 + node) * a.qts + (h * a.group + row - node * a.group) * a.qhs;
            double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int s = 0; s < NB; s++) {
                // lane (g, r): elements 16 (g & 1) .. of block s of row r; g < 2
                // their positive parts, to meet the largest keys, else the negative
                float v[16], big = 0.0f;
                {
                    float x[8];
                    load_x8<DT>(x, a.q, at + 32 * s + 16 * (g & 1));
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        v[e] = x[e];
                    load_x8<DT>(x, a.q, at + 32 * s + 16 * (g & 1) + 8);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        v[8 + e] = x[e];
                }
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    v[e] = v[e] != v[e] ? 0.0f : fminf(fmaxf(v[e], -3.0e38f), 3.0e38f);
                    big = fmaxf(big, fabsf(v[e]));
                }
                big = fmaxf(big, __shfl_xor(big, 16));
                const float d = big / 127.0f, inv = d > 0x1p-100f ? 1.0f / d : 0.0f;
                i4 q;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    uint32_t x = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int c = round_away(v[4 * w + e], inv);
                        x |= ((uint32_t)(g < 2 ? max(c, 0) : min(c, 0)) & 0xFFu) << (8 * e);
                    }
                    q[w] = (int)x;
                }
                // pages in the rows of the result, queries in its columns (lanes)
                const i4 dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(codes[s], q, i4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float ds = __shfl(scale[s], 4 * g + e);
                    sum[e] += (double)dot[e] * ((double)d * (double)ds);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; e++)
                best[e] = fmax(best[e], sum[e]);
        }
        const uint64_t mapped = __ballot(there);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            for (int m = 1; m < 16; m <<= 1)
                best[e] = fmax(best[e], __shfl_xor(best[e], m));
            const int64_t p = p0 + 4 * g + e;
            // a page that is not there comes last
            if (r == 0 && p < sp.tail)
                out[p] = (mapped >> (4 * g + e)) & 1 ? order_key((float)best[e]) : 0u;
        }
    }
}

// ---- choice ----------------------------------------------------------------

// One workgroup for each sequence and key head: the key of the last page that
// is kept, eight bits at a time, then the pages in order.
__global__ __launch_bounds__(SEL_THREADS) void k_select(SelectArgs a, const uint32_t *all_keys)
{
    __shared__ uint32_t count[256], scan[SEL_WAVES];
    __shared__ int hit;
    __shared__ uint32_t before_hit;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.kv_heads, h = blockIdx.x - b * a.kv_heads;
    const Span sp = span_of(a, b);
    const int32_t *table = a.table + b * a.table_stride;
    const uint32_t *keys = all_keys + (int64_t)blockIdx.x * a.table_pages;
    int32_t *out = a.out + ((int64_t)b * a.kv_heads + h) * a.width;
    const int cand = sp.tail - sp.first;
    uint32_t key = 0, need = sp.keep;            // pages with larger keys, and `need` of this key
    if (sp.keep < cand && sp.keep > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256)
                count[tid] = 0;
            __syncthreads();
            for (int i = sp.first + tid; i < sp.tail; i += SEL_THREADS) {
                const uint32_t k = keys[i];
                if (shift == 24 || (k >> (shift + 8)) == key >> (shift + 8))
                    atomicAdd(&count[(k >> shift) & 255], 1u);
            }
            __syncthreads();
            const uint32_t own = tid < 256 ? count[255 - tid] : 0;
            uint32_t all;
            const uint32_t before = scan_before<SEL_WAVES>(own, scan, all);
            if (before < need && before + own >= need) {
                hit = 255 - tid;
                before_hit = before;
            }
            __syncthreads();
            key |= (uint32_t)hit << shift;
            need -= before_hit;
            __syncthreads();
        }
    }
    // pages in order: all up to `first` and from `tail` on
    uint32_t written = 0, ties = 0;
    for (int base = 0; base < sp.total; base += SEL_THREADS) {
        const int i = base + tid;
        bool take = i < sp.total;
        uint32_t tie = 0;
        if (take && i >= sp.first && i < sp.tail && sp.keep < cand) {
            const uint32_t k = keys[i];
            tie = sp.keep > 0 && k == key;
            take = sp.keep > 0 && k > key;
        }
        uint32_t all;
        const uint32_t tb = ties + scan_before<SEL_WAVES>(tie, scan, all);
        ties += all;
        __syncthreads();
        take = take || (tie && tb < need);
        const uint32_t at = written + scan_before<SEL_WAVES>((uint32_t)take, scan, all);
        written += all;
        __syncthreads();
        if (take && at < (uint32_t)a.width)
            out[at] = table[i];
    }
    for (int i = written + tid; i < a.width; i += SEL_THREADS)
        out[i] = -1;
    if (h == 0 && tid == 0)
        a.ctx_out[b] = sp.ctx - (int)((int64_t)(cand - sp.keep) << a.log_page);
}

template <int CT>
hipError_t bounds_d(int D, dim3 grid, const BoundsArgs &a, int pages, hipStream_t s)
{
    switch (D) {
    case 64: k_bounds<CT, 64><<<grid, THREADS, 0, s>>>(a, pages); break;
    case 96: k_bounds<CT, 96><<<grid, THREADS, 0, s>>>(a, pages); break;
    case 128: k_bounds<CT, 128><<<grid, THREADS, 0, s>>>(a, pages); break;
    case 256: k_bounds<CT, 256><<<grid, THREADS, 0, s>>>(a, pages); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int DT> hipError_t scores_d(int D, dim3 grid, const SelectArgs &a, uint32_t *keys, hipStream_t s)
{
    switch (D) {
    case 64: k_scores<DT, 64><<<grid, THREADS, 0, s>>>(a, keys); break;
    case 96: k_scores<DT, 96><<<grid, THREADS, 0, s>>>(a, keys); break;
    case 128: k_scores<DT, 128><<<grid, THREADS, 0, s>>>(a, keys); break;
    case 256: k_scores<DT, 256><<<grid, THREADS, 0, s>>>(a, keys); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_bounds(int cache_type, int D, const BoundsArgs &a, int64_t max_new, hipStream_t s)
{
    // pages that max_new positions in a row can touch
    const int64_t P = int64_t(1) << a.log_page;
    const int64_t pages = std::min<int64_t>((max_new + P - 2) / P + 1, a.table_pages);
    const int64_t blocks = (pages * a.kv_heads * (D / 32) + WAVES - 1) / WAVES;
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks, (unsigned)a.batch);
    return cache_type == TQ_Q8_0 ? bounds_d<TQ_Q8_0>(D, grid, a, (int)pages, s)
                                 : bounds_d<TQ_Q4_0>(D, grid, a, (int)pages, s);
}

size_t select_scratch_bytes(int64_t batch, int64_t kv_heads, int64_t table_pages)
{
    return (size_t)batch * kv_heads * table_pages * sizeof(uint32_t);
}

hipError_t launch_select(int D, const SelectArgs &a, int64_t max_ctx, void *scratch, hipStream_t s)
{
    const int64_t units = (int64_t)a.batch * a.kv_heads;
    const int64_t pages = std::min<int64_t>((max_ctx >> a.log_page) + 1, a.table_pages);
    const int64_t y = std::min<int64_t>((pages + 16 * WAVES - 1) / (16 * WAVES), 65535);
    if (!grid_fits(units, SEL_THREADS))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)units, (unsigned)y);
    hipError_t e = a.dtype == TQ_BF16 ? scores_d<TQ_BF16>(D, grid, a, (uint32_t *)scratch, s)
                                      : scores_d<TQ_F16>(D, grid, a, (uint32_t *)scratch, s);
    if (e != hipSuccess)
        return e;
    k_select<<<dim3((unsigned)units), SEL_THREADS, 0, s>>>(a, (const uint32_t *)scratch);
    return hipGetLastError();
}

}  // namespace tq
