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
constexpr int SEL_WAVES = 8, SEL_THREADS = 64 * SEL_WAVES;
constexpr int CHOOSE_WAVES = 16;
constexpr int MOST_KEYS = 8192;                  // pages whose keys LDS holds
// Heads of more than two turns of pages, as long as they are fewer than half the
// compute units, have their pages spread over workgroups.  One workgroup a head /
// spread, one query row group, us: 8 heads, 128 pages 6.4 / 7.7, 256 8.3 / 8.0, 512 11.0 / 8.6,
// 2048 27 / 11.3; 120 heads, 512 pages 11.2 / 10.6, 2048 34.8 / 29.1; 128 heads 11.6 / 10.5,
// 35 / 30; 192 heads 12.4 / 14.0 (1024 pages 21.3 / 23.0); 512 heads 20 / 27.  124 query rows:
// 32 heads, 64 pages 12.8 / 14.0, 256 17.8 / 15.0, 1024 39.5 / 17.1.  Tables past MOST_KEYS take
// two launches whatever lies in them: 8 heads of 2047 pages 11.4, in a table of 8192 11.1.
constexpr int SPREAD_TURNS = 2, SPREAD_UNITS = 128;
constexpr int COUNTER_STRIDE = 64;               // words: a cache line for each head

// ---- bounds ----------------------------------------------------------------

// A wave has one block of one page and head: lane (g, r) the elements 8g ..
// 8g+7 of every 16th token from r.  Bound: four dependent reads (length, page,
// scales and codes); 64 sequences' last pages of 64 take 5.8 us, the pages of two
// prompts of 8191 tokens 11.4, 8 heads of 128 (7.0 and 12.2 with the codes made signed
// first, a token at a time).
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
    // The codes are unsigned: code * d - offset * d, one fma of a value that fp32 holds
    // (19 bits).  Two tokens at a time, for maxima and minima of three; past the end the
    // last one again.
#pragma unroll 2
    for (int pos = r; pos < n; pos += 32) {
        uint2 code[2];
        float d[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int at = pos + 16 * k < n ? pos + 16 * k : pos;
            const uint8_t *p = chunk + k_offset<CT, D>(at, s, g);
            d[k] = f16_bits_to_f32(scales[at * NB + s]);
            if constexpr (CT == TQ_Q8_0) {
                code[k] = *(const uint2 *)p;
            } else {
                const uint32_t w = *(const uint32_t *)p;
                code[k] = make_uint2(w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            // element of byte e % 4 of the low or high nibbles, or e itself
            constexpr float offset = CT == TQ_Q8_0 ? 128.0f : 8.0f;
            const float u = fmaf((float)(((e < 4 ? code[0].x : code[0].y) >> (8 * (e & 3))) & 255u), d[0],
                                 -offset * d[0]);
            const float v = fmaf((float)(((e < 4 ? code[1].x : code[1].y) >> (8 * (e & 3))) & 255u), d[1],
                                 -offset * d[1]);
            hi[e] = fmaxf(fmaxf(hi[e], u), v);
            lo[e] = fminf(fminf(lo[e], u), v);
        }
    }
    if constexpr (CT == TQ_Q4_0) {
        // from the places of the nibbles to the elements
        float h[8], l[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int at = ((k4_shift(e) & 4) ? 4 : 0) + (k4_shift(e) >> 3);
            h[e] = hi[at];
            l[e] = lo[at];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            hi[e] = h[e];
            lo[e] = l[e];
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

// Query rows that are in LDS at a time: as 16-row operands of the matrix cores, and
// their blocks' scales.
constexpr int row_tiles(int D) { return D <= 128 ? 8 : 4; }

template <int D> struct QueryLds {
    i4 code[row_tiles(D)][D / 32][64];
    double scale[row_tiles(D)][D / 32][16];
};

// Quantizes rows r0 .. of a head's query rows, a 16-row tile's block a wave at a
// time.  Lane (g, r): elements 16 (g & 1) .. of the block of row r; g < 2 their
// positive parts, to meet the largest keys, else the negative.  Rows past the last
// repeat it.
template <int DT, int D, int W>
__device__ __forceinline__ void quantize_rows(QueryLds<D> &l, const SelectArgs &a, const Span &sp,
                                              int h, int r0, int tiles)
{
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int rows = sp.T * a.group;
    for (int item = threadIdx.x >> 6; item < tiles * NB; item += W) {
        const int tile = item / NB, s = item % NB;
        const int row = min(r0 + tile * 16 + r, rows - 1), node = row / a.group;
        const int64_t at = (sp.tok0 + node) * a.qts + (h * a.group + row - node * a.group) * a.qhs +
                           32 * s + 16 * (g & 1);
        float v[2][8], big = 0.0f;
        load_x8<DT>(v[0], a.q, at);
        load_x8<DT>(v[1], a.q, at + 8);
#pragma unroll
        for (int e = 0; e < 16; e++) {
            float &x = v[e >> 3][e & 7];
            x = x != x ? 0.0f : fminf(fmaxf(x, -3.0e38f), 3.0e38f);
            big = fmaxf(big, fabsf(x));
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        const float d = big / 127.0f, inv = d > 0x1p-100f ? 1.0f / d : 0.0f;
        i4 q;
#pragma unroll
        for (int w = 0; w < 4; w++) {
            uint32_t x = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int c = round_away(v[w >> 1][4 * (w & 1) + e], inv);
                x |= ((uint32_t)(g < 2 ? max(c, 0) : min(c, 0)) & 0xFFu) << (8 * e);
            }
            q[w] = (int)x;
        }
        l.code[tile][s][lane] = q;
        if (g == 0)
            l.scale[tile][s][r] = (double)d;
    }
}

// One page a lane r: bytes 16g .. of its blocks' codes, and the scales.
template <int D> struct PageBounds {
    i4 code[D / 32];
    uint16_t scale[D / 32];
    bool there;
};

template <int D>
__device__ __forceinline__ void load_bounds(PageBounds<D> &p, const SelectArgs &a, int64_t id, int h,
                                            int g)
{
    constexpr int NB = D / 32;
    p.there = id >= 0 && id < a.pages;
    const int64_t block = ((p.there ? id : 0) * a.kv_heads + h) * NB;
#pragma unroll
    for (int s = 0; s < NB; s++) {
        p.code[s] = *(const i4 *)(a.codes + (block + s) * 64 + g * 16);
        p.scale[s] = a.scales[block + s];
    }
}

// Scores of pages [begin, end), 16 a wave and turn, as order keys: put(page, key,
// again), again where the page has one of earlier rows.  The next turn's bounds are
// on their way while this one's are scored.
template <int DT, int D, int W, typename F>
__device__ __forceinline__ void score_pages(QueryLds<D> &l, const SelectArgs &a, const Span &sp, int h,
                                            int begin, int end, F put)
{
    constexpr int NB = D / 32, RT = row_tiles(D);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t *table = a.table + (blockIdx.x / a.kv_heads) * a.table_stride;
    const int rows = sp.T * a.group;
    for (int r0 = 0; r0 < max(rows, 1); r0 += 16 * RT) {
        const int tiles = min((rows - r0 + 15) / 16, RT);
        int p0 = begin + wave * 16;
        PageBounds<D> now, next;
        if (p0 < end)
            load_bounds<D>(now, a, table[min(p0 + r, end - 1)], h, g);
        if (r0)
            __syncthreads();                     // the rows before have been read
        quantize_rows<DT, D, W>(l, a, sp, h, r0, tiles);
        __syncthreads();
        for (; p0 < end; p0 += W * 16) {
            const int p1 = p0 + W * 16;
            if (p1 < end)
                load_bounds<D>(next, a, table[min(p1 + r, end - 1)], h, g);
            double best = -__builtin_inf();
            for (int t = 0; t < tiles; t++) {
                double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
                for (int s = 0; s < NB; s++) {
                    // queries in the rows of the result, pages in its columns (lanes)
                    const i4 dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(l.code[t][s][lane], now.code[s],
                                                                       i4{0, 0, 0, 0}, 0, 0, 0);
                    const double page = (double)f16_bits_to_f32(now.scale[s]);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        sum[e] += (double)dot[e] * (l.scale[t][s][4 * g + e] * page);
                }
#pragma unroll
                for (int e = 0; e < 4; e++)
                    best = fmax(best, sum[e]);
            }
            // rounding keeps the order: the largest is rounded, whatever comes first
            float score = (float)best;
            score = fmaxf(score, __shfl_xor(score, 16));
            score = fmaxf(score, __shfl_xor(score, 32));
            if (g == 0 && p0 + r < end) {
                // a page that is not there comes last
                put(p0 + r, now.there ? order_key(score) : 0u, r0 > 0);
            }
            now = next;
        }
    }
}

// ---- choice ----------------------------------------------------------------

template <int W> struct ChoiceLds {
    uint32_t count[64 * W], scan[2][W];
    uint32_t least, most, before, own;
    int sub;
};

// The pages that are kept, in order, by a workgroup: those of the span's ends, and
// the `keep` largest keys of the others.  Sub-bins of the keys' range, one a thread,
// bring it down to the one that the last kept page is in, and so on inside that, until it is
// kept whole or its keys are all equal: two turns as a rule.
template <int W>
__device__ __forceinline__ void choose(ChoiceLds<W> &l, const SelectArgs &a, const Span &sp, int b,
                                       int h, const uint32_t *keys)
{
    constexpr int THREADS = 64 * W, SUBS = THREADS, LOG_SUBS = W == 16 ? 10 : (W == 8 ? 9 : 8);
    static_assert(1 << LOG_SUBS == SUBS, "");
    const int tid = threadIdx.x;
    const int32_t *table = a.table + b * a.table_stride;
    int32_t *out = a.out + ((int64_t)b * a.kv_heads + h) * a.width;
    const int cand = sp.tail - sp.first;
    // kept: keys of lo and more but the last `drop` of those equal to lo
    uint32_t lo = 0, need = sp.keep, ties = 0;
    if (sp.keep < cand && sp.keep > 0) {
        if (tid == 0) {
            l.least = ~0u;
            l.most = 0;
        }
        __syncthreads();
        uint32_t least = ~0u, most = 0;
        for (int i = sp.first + tid; i < sp.tail; i += THREADS) {
            least = min(least, keys[i]);
            most = max(most, keys[i]);
        }
        for (int d = 1; d < 64; d <<= 1) {
            least = min(least, (uint32_t)__shfl_xor(least, d));
            most = max(most, (uint32_t)__shfl_xor(most, d));
        }
        if ((tid & 63) == 0) {
            atomicMin(&l.least, least);
            atomicMax(&l.most, most);
        }
        __syncthreads();
        lo = l.least;
        most = l.most;                           // keys lo .. most are in question
        for (;;) {
            const uint32_t span = most - lo;
            const int shift = max(32 - __builtin_clz(span | 1) - LOG_SUBS, 0);
            l.count[tid] = 0;
            __syncthreads();
            for (int i = sp.first + tid; i < sp.tail; i += THREADS) {
                const uint32_t k = keys[i];
                if (k >= lo && k <= most)
                    atomicAdd(&l.count[(k - lo) >> shift], 1u);
            }
            __syncthreads();
            // from the highest sub-bin down, one a thread
            const uint32_t own = l.count[SUBS - 1 - tid];
            uint32_t all;
            const uint32_t before = scan_before<W>(own, l.scan[0], all);
            if (before < need && before + own >= need) {
                l.sub = SUBS - 1 - tid;
                l.before = before;
                l.own = own;
            }
            __syncthreads();
            need -= l.before;
            lo += (uint32_t)l.sub << shift;
            ties = l.own;
            const bool done = shift == 0 || ties == need;
            most = shift == 0 ? lo : min(most, lo + ((1u << shift) - 1));
            __syncthreads();
            if (done)
                break;
        }
    }
    // with ties: keys above `most` are kept, of those in lo .. most (all equal, or
    // all kept) the first `need`
    const bool partly = ties != need;
    uint32_t written = 0, met = 0;
    for (int base = 0; base < sp.total; base += THREADS) {
        const int i = base + tid;
        bool take = i < sp.total;
        uint32_t tie = 0;
        if (take && i >= sp.first && i < sp.tail && sp.keep < cand) {
            const uint32_t k = sp.keep > 0 ? keys[i] : 0;
            take = sp.keep > 0 && k >= lo;
            tie = take && partly && k == lo;
        }
        uint32_t all;
        if (partly) {
            const uint32_t rank = met + scan_before<W>(tie, l.scan[0], all);
            met += all;
            take = take && (!tie || rank < need);
        }
        const uint32_t at = written + scan_before<W>((uint32_t)take, l.scan[1], all);
        written += all;
        if (take && at < (uint32_t)a.width)
            out[at] = table[i];
        __syncthreads();
    }
    for (int i = written + tid; i < a.width; i += THREADS)
        out[i] = -1;
    if (h == 0 && tid == 0)
        a.ctx_out[b] = sp.ctx - (int)((int64_t)(cand - sp.keep) << a.log_page);
}

// A workgroup for each sequence and key head scores its pages and chooses; their
// keys stay in LDS.  64 sequences of up to 16384 keys in pages of 64, 8 key heads:
// 11.9 us for 26 MB of bounds (sixteen waves a workgroup: 16.7).
template <int DT, int D>
__global__ __launch_bounds__(SEL_THREADS) void k_select(SelectArgs a)
{
    __shared__ QueryLds<D> q;
    __shared__ uint32_t keys[MOST_KEYS];
    __shared__ ChoiceLds<SEL_WAVES> l;
    const int b = blockIdx.x / a.kv_heads, h = blockIdx.x - b * a.kv_heads;
    const Span sp = span_of(a, b);
    if (sp.keep < sp.tail - sp.first && sp.keep > 0)
        score_pages<DT, D, SEL_WAVES>(q, a, sp, h, sp.first, sp.tail,
                                      [&](int page, uint32_t key, bool again) {
                                          keys[page] = again ? max(keys[page], key) : key;
                                      });
    choose<SEL_WAVES>(l, a, sp, b, h, keys);
}

// A head's pages spread over gridDim.y workgroups.  LAST: the last of them to end
// chooses; the keys are exchanged into memory (device-scope atomics act there, past
// the dies' caches) and have come back before the head's count rises, so it reads
// them whole.  Else k_choose does, in a launch of its own.  One sequence of 131000
// keys: 11.6 us, where scores and choice apart take 7 + 7.
template <int DT, int D, bool LAST>
__global__ __launch_bounds__(SEL_THREADS) void k_scores(SelectArgs a, uint32_t *all_keys,
                                                        uint32_t *counters)
{
    __shared__ QueryLds<D> q;
    __shared__ uint32_t own[LAST ? MOST_KEYS : 1];
    __shared__ ChoiceLds<SEL_WAVES> l;
    __shared__ bool last;
    const int b = blockIdx.x / a.kv_heads, h = blockIdx.x - b * a.kv_heads;
    const Span sp = span_of(a, b);
    const int cand = sp.tail - sp.first;
    uint32_t *keys = all_keys + (int64_t)blockIdx.x * a.table_pages;
    if (sp.keep == cand || sp.keep == 0) {       // nothing to compare
        if constexpr (LAST) {
            if (blockIdx.y == 0)
                choose<SEL_WAVES>(l, a, sp, b, h, own);
        }
        return;
    }
    // whole turns of 16 pages a wave
    const int turns = (cand + SEL_WAVES * 16 - 1) / (SEL_WAVES * 16);
    const int64_t each = (int64_t)((turns + gridDim.y - 1) / gridDim.y) * (SEL_WAVES * 16);
    const int64_t begin = sp.first + blockIdx.y * each;
    uint32_t was = 0;
    if (begin < sp.tail)
        score_pages<DT, D, SEL_WAVES>(
            q, a, sp, h, (int)begin, (int)min(begin + each, (int64_t)sp.tail),
            [&](int page, uint32_t key, bool again) {
                if constexpr (LAST)
                    was |= again ? __hip_atomic_fetch_max(keys + page, key, __ATOMIC_RELAXED,
                                                          __HIP_MEMORY_SCOPE_AGENT)
                                 : __hip_atomic_exchange(keys + page, key, __ATOMIC_RELAXED,
                                                         __HIP_MEMORY_SCOPE_AGENT);
                else
                    keys[page] = again ? max(keys[page], key) : key;
            });
    if constexpr (LAST) {
        asm volatile("s_waitcnt vmcnt(0)" : : "v"(was) : "memory");
        __syncthreads();
        uint32_t *count = counters + (int64_t)blockIdx.x * COUNTER_STRIDE;
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   gridDim.y - 1;
        __syncthreads();
        if (!last)
            return;
        for (int i = sp.first + threadIdx.x; i < sp.tail; i += SEL_THREADS)
            own[i] = __hip_atomic_load(keys + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        choose<SEL_WAVES>(l, a, sp, b, h, own);
        if (threadIdx.x == 0)                    // zero again for the next call
            __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

__global__ __launch_bounds__(64 * CHOOSE_WAVES) void k_choose(SelectArgs a, const uint32_t *keys)
{
    __shared__ ChoiceLds<CHOOSE_WAVES> l;
    const int b = blockIdx.x / a.kv_heads, h = blockIdx.x - b * a.kv_heads;
    choose<CHOOSE_WAVES>(l, a, span_of(a, b), b, h, keys + (int64_t)blockIdx.x * a.table_pages);
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

// How a step's pages are chosen: by a workgroup for each head; by several, of which
// the last one chooses; or in two launches, where LDS does not hold a head's keys.
enum Form { ALONE, SPREAD, APART };

template <int DT, int D>
hipError_t select_dd(Form form, const SelectArgs &a, int64_t pages, uint32_t *counters,
                     uint32_t *keys, hipStream_t s)
{
    const int64_t y = std::min<int64_t>((pages + SEL_WAVES * 16 - 1) / (SEL_WAVES * 16), 65535);
    const dim3 units((unsigned)(a.batch * a.kv_heads)), spread(units.x, (unsigned)y);
    if (form == ALONE) {
        k_select<DT, D><<<units, SEL_THREADS, 0, s>>>(a);
    } else if (form == SPREAD) {
        k_scores<DT, D, true><<<spread, SEL_THREADS, 0, s>>>(a, keys, counters);
    } else {
        k_scores<DT, D, false><<<spread, SEL_THREADS, 0, s>>>(a, keys, nullptr);
        k_choose<<<units, 64 * CHOOSE_WAVES, 0, s>>>(a, keys);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t select_d(int D, Form form, const SelectArgs &a, int64_t pages, uint32_t *counters,
                    uint32_t *keys, hipStream_t s)
{
    switch (D) {
    case 64: return select_dd<DT, 64>(form, a, pages, counters, keys, s);
    case 96: return select_dd<DT, 96>(form, a, pages, counters, keys, s);
    case 128: return select_dd<DT, 128>(form, a, pages, counters, keys, s);
    case 256: return select_dd<DT, 256>(form, a, pages, counters, keys, s);
    }
    return hipErrorInvalidValue;
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
    // with more units than that a workgroup has each, and the keys in LDS
    const int64_t units = batch * kv_heads;
    return (size_t)(table_pages > MOST_KEYS ? units : std::min<int64_t>(units, SPREAD_UNITS)) *
           table_pages * sizeof(uint32_t);
}

hipError_t launch_select(int D, const SelectArgs &a, int64_t max_ctx, uint32_t *counters,
                         void *scratch, hipStream_t s)
{
    const int64_t units = (int64_t)a.batch * a.kv_heads;
    if (!grid_fits(units, 64 * CHOOSE_WAVES))
        return hipErrorInvalidConfiguration;
    const int64_t pages = std::min<int64_t>((max_ctx >> a.log_page) + 1, a.table_pages);
    const int64_t turns = (pages + SEL_WAVES * 16 - 1) / (SEL_WAVES * 16) *
                          (((int64_t)a.max_nodes * a.group + 15) / 16);
    const Form form = a.table_pages > MOST_KEYS                            ? APART
                      : turns <= SPREAD_TURNS || units >= SPREAD_UNITS ? ALONE
                                                                           : SPREAD;
    uint32_t *keys = (uint32_t *)scratch;
    return a.dtype == TQ_BF16 ? select_d<TQ_BF16>(D, form, a, pages, counters, keys, s)
                              : select_d<TQ_F16>(D, form, a, pages, counters, keys, s);
}

}  // namespace tq
