// Tokens drawn from logits with temperature, top-k, top-p and min-p from given
// uniform numbers (tq_sample), and the distribution that they are drawn from
// (tq_sample_probs).
//
// A row's weights are w_i = exp((x_i - max) / T), each rounded to a whole
// multiple of 2^-s (s = 45 for vocabularies up to 2^17, less for larger ones: 62
// bits hold a whole row), so that a sum of them is exact and the same in every
// order; fp64 up to that rounding.  In the order of falling x, ties by rising index,
// top-k keeps the first k, top-p of those the shortest prefix that holds p of
// their sum; min-p keeps w >= min_p.  All three are prefixes, so what is kept is
// described by one key and how many of its ties count.  The token is the first
// index whose running sum of kept weights exceeds u times their sum.
#include <algorithm>

#include "block_ops.h"

namespace tq {
namespace {

constexpr int WAVES = 16, THREADS = 64 * WAVES;
constexpr int DIGITS = 256;

// The settings of a row.
struct Setting {
    double rate;                                 // log2(e) / T; 0 or less: the likeliest token
    double p;                                    // >= 1: off
    uint64_t min_w;                              // the least weight that min-p keeps
    int64_t k;                                   // <= 0: off
    float u;
    int bits;                                    // s
};

__device__ __forceinline__ Setting setting_of(const SampleArgs &a, int64_t row)
{
    Setting s;
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    s.rate = t > 0.0f ? 1.4426950408889634074 / (double)t : 0.0;
    if (!(t > 0.0f))
        s.rate = -1.0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    s.p = p < 1.0f ? (double)p : 1.0;            // NaN: off
    const float m = a.min_p ? a.min_p[row] : 0.0f;
    s.min_w = m > 0.0f ? (uint64_t)ceil(ldexp((double)fminf(m, 1.0f), a.bits)) : 0;
    s.k = a.top_k ? a.top_k[row] : 0;
    s.u = a.u ? a.u[row] : 0.0f;
    s.bits = a.bits;
    return s;
}

// 2^t as a whole number, nearest, for t <= 51: 2^n times a polynomial for 2^f, |f| <=
// 1/2 (interpolated in Chebyshev's points, off by 2^-51), whose bits come to the
// low end of a mantissa by adding 2^52.
__device__ __forceinline__ uint64_t whole_exp2(double t)
{
    const double n = rint(t), f = t - n;
    double p = 7.072585949269223e-09;
    p = fma(p, f, 1.0208690299958306e-07);
    p = fma(p, f, 1.321544258792169e-06);
    p = fma(p, f, 1.5252657260200837e-05);
    p = fma(p, f, 0.0001540353044173605);
    p = fma(p, f, 0.0013333558230164974);
    p = fma(p, f, 0.009618129107606888);
    p = fma(p, f, 0.05550410866444772);
    p = fma(p, f, 0.24022650695910097);
    p = fma(p, f, 0.69314718055995);
    p = fma(p, f, 1.0);
    const uint64_t scaled = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(int64_t)(int)n << 52);
    const double magic = __builtin_bit_cast(double, scaled) + 0x1p52;
    return __builtin_bit_cast(uint64_t, magic) & 0xFFFFFFFFFFFFFull;
}

// A weight in units of 2^-bits; 0 for what is no number, or -infinity.
__device__ __forceinline__ uint64_t weight(float x, float top, const Setting &s)
{
    const double t = ((double)x - (double)top) * s.rate + (double)s.bits;
    const uint64_t w = whole_exp2(fmax(t, -2.0));                // 1/4: rounds to 0; so does NaN
    const uint64_t got = x > -__builtin_inff() ? w : 0;
    return x == top ? uint64_t(1) << s.bits : got;
}

// Whether an element with `before` weights in front of it is inside top-p's
// prefix of `total`; the first one always is.
__device__ __forceinline__ bool inside(uint64_t before, double p, uint64_t total)
{
    return p >= 1.0 || before == 0 || (double)before < p * (double)total;
}

// What is kept of a row: keys above `key`, and those equal to it up to `last`.
struct Cut {
    uint32_t key;
    int64_t last;
};

__device__ __forceinline__ bool kept(const Cut &c, uint32_t key, int64_t i)
{
    return key > c.key || (key == c.key && i <= c.last);
}

struct RowLds {
    uint32_t count[DIGITS];
    uint64_t mass[DIGITS];
    uint64_t scan[WAVES];
    uint32_t scan32[WAVES];
    uint64_t mass_before;
    uint32_t count_before;
    int hit;
    float top[WAVES];
    int64_t index[WAVES];
};

// Walks over all of a row by one workgroup.
struct Walker {
    const void *x;
    int64_t at, vocab;
    int dtype;
    float top;

    __device__ __forceinline__ float get(int64_t i) const { return load_one(x, dtype, at + i); }
};

struct Found {
    uint32_t key;                                // of the last element kept
    uint32_t ties;                               // elements with it
    uint32_t count_before;                       // elements, and weights, above it
    uint64_t mass_before;
    bool all;                                    // nothing is left out
};

// The key where the order passes a limit, eight bits at a time: the k-th
// element (K), or the last one inside top-p's prefix of `total`.  Elements of no
// weight do not count.
template <bool K>
__device__ __forceinline__ Found find_key(const Walker &r, const Setting &s, RowLds &l,
                                          uint64_t total)
{
    const int tid = threadIdx.x;
    Found f{0, 0, 0, 0, false};
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < DIGITS; i += THREADS) {
            l.count[i] = 0;
            l.mass[i] = 0;
        }
        if (tid == 0)
            l.hit = -1;
        __syncthreads();
        for (int64_t i = tid; i < r.vocab; i += THREADS) {
            const float x = r.get(i);
            const uint32_t key = order_key(x);
            if (shift < 24 && (key >> (shift + 8)) != f.key >> (shift + 8))
                continue;
            const uint64_t w = weight(x, r.top, s);
            if (w == 0)
                continue;
            atomicAdd(&l.count[(key >> shift) & 255], 1u);
            atomicAdd((unsigned long long *)&l.mass[(key >> shift) & 255], (unsigned long long)w);
        }
        __syncthreads();
        // digits in falling order, one a thread
        const uint32_t own = tid < DIGITS ? l.count[255 - tid] : 0;
        const uint64_t mass = tid < DIGITS ? l.mass[255 - tid] : 0;
        uint32_t all_count;
        uint64_t all_mass;
        const uint32_t cb = f.count_before + scan_before<WAVES>(own, l.scan32, all_count);
        const uint64_t mb = f.mass_before + scan_before<WAVES>(mass, l.scan, all_mass);
        const bool last = own && (K ? cb < s.k : inside(mb, s.p, total));
        if (last)
            atomicMax(&l.hit, tid);
        __syncthreads();
        const int hit = l.hit;
        if (tid == hit) {
            l.count_before = cb;
            l.mass_before = mb;
        }
        __syncthreads();
        const uint32_t digit = 255 - hit;        // a row has an element of weight: its largest
        f.key |= digit << shift;
        f.ties = l.count[digit];
        if (K && shift == 24 && (int64_t)all_count <= s.k)
            f.all = true;
        f.count_before = l.count_before;
        f.mass_before = l.mass_before;
        __syncthreads();
        if (f.all)
            return f;
    }
    return f;
}

// How many of `ties` equal weights w behind `before` are inside top-p's prefix.
__device__ __forceinline__ uint32_t ties_inside(uint64_t before, uint64_t w, uint32_t ties,
                                                double p, uint64_t total)
{
    const double about = (p * (double)total - (double)before) / (double)w;
    uint32_t m = about >= (double)ties ? ties : (about > 1.0 ? (uint32_t)about : 1);
    while (m < ties && inside(before + m * w, p, total))
        m++;
    while (m > 1 && !inside(before + (m - 1) * w, p, total))
        m--;
    return m;
}

// Index of the m-th element (from 1) with a key.
__device__ __forceinline__ int64_t find_tie(const Walker &r, RowLds &l, uint32_t key, uint32_t m)
{
    const int tid = threadIdx.x;
    uint32_t before = 0;
    if (tid == 0)
        l.index[0] = r.vocab;
    for (int64_t base = 0; base < r.vocab && before < m; base += THREADS) {
        const int64_t i = base + tid;
        const uint32_t is = i < r.vocab && order_key(r.get(i)) == key;
        uint32_t all;
        const uint32_t b = before + scan_before<WAVES>(is, l.scan32, all);
        if (is && b + 1 == m)
            l.index[0] = i;
        before += all;
        __syncthreads();
    }
    __syncthreads();
    const int64_t at = l.index[0];
    __syncthreads();
    return at;
}

// What top-k and top-p keep of a row.
__device__ __forceinline__ Cut find_cut(const Walker &r, const Setting &s, RowLds &l)
{
    Cut c{0, r.vocab};
    Found f{};
    uint64_t total = 0;
    uint32_t m = 0;
    bool cut = false;
    if (s.k > 0) {
        f = find_key<true>(r, s, l, 0);
        if (!f.all) {
            m = (uint32_t)(s.k - f.count_before);
            total = f.mass_before + m * weight(key_value(f.key), r.top, s);
            cut = true;
        }
    }
    if (s.p < 1.0) {
        if (!cut) {
            uint64_t mine = 0;
            for (int64_t i = threadIdx.x; i < r.vocab; i += THREADS)
                mine += weight(r.get(i), r.top, s);
            __syncthreads();
            scan_before<WAVES>(mine, l.scan, total);
            __syncthreads();
        }
        f = find_key<false>(r, s, l, total);
        m = ties_inside(f.mass_before, weight(key_value(f.key), r.top, s), f.ties, s.p, total);
        cut = true;
    }
    if (cut) {
        c.key = f.key;
        if (m < f.ties)
            c.last = find_tie(r, l, f.key, m);
    }
    return c;
}

// The kept weight of element i.
__device__ __forceinline__ uint64_t kept_weight(const Walker &r, const Setting &s, const Cut &c,
                                                int64_t i)
{
    const float x = r.get(i);
    if (!kept(c, order_key(x), i))
        return 0;
    const uint64_t w = weight(x, r.top, s);
    return w >= s.min_w ? w : 0;
}

// The place of u in a sum: at most its last unit; below 0 or NaN counts as 0.
__device__ __forceinline__ uint64_t place_in(float u, uint64_t all)
{
    const double v = u > 0.0f ? fmin((double)u, 1.0) : 0.0;
    return all ? min((uint64_t)(v * (double)all), all - 1) : 0;
}

// A token (r.top set, a row of some weight) from its cut by one workgroup, for rows that the
// tiles below do not serve; or the sum of what is kept.
__device__ __forceinline__ uint64_t walk_row(const SampleArgs &a, const Walker &r, const Setting &s,
                                             const Cut &c, int64_t row, RowLds &l)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // a wave has a run of the row
    const int64_t run = (a.vocab + THREADS - 1) / THREADS * 64, begin = run * wave;
    const int64_t end = min(begin + run, a.vocab);
    uint64_t sum = 0;
    for (int64_t i = begin + lane; i < end; i += 64)
        sum += kept_weight(r, s, c, i);
    sum = wave_sum(sum);
    __syncthreads();
    if (lane == 0)
        l.scan[wave] = sum;
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (int i = 0; i < WAVES; i++) {
        before += i < wave ? l.scan[i] : 0;
        all += l.scan[i];
    }
    const uint64_t thr = place_in(s.u, all);
    if (a.probs || !(before <= thr && thr < before + sum))
        return all;
    for (int64_t base = begin; base < end; base += 64) {
        const int64_t i = base + lane;
        const uint64_t upto = before + scan_wave(i < end ? kept_weight(r, s, c, i) : 0);
        const uint64_t hit = __ballot(upto > thr);
        if (hit) {
            if (lane == __builtin_ctzll(hit))
                a.tokens[row] = (int32_t)i;
            break;
        }
        before = lane_value(upto, 63);
    }
    return all;
}

__device__ __forceinline__ float max_all(float v, float *lds)
{
    for (int m = 1; m < 64; m <<= 1)
        v = fmaxf(v, __shfl_xor(v, m));
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    for (int i = 0; i < WAVES; i++)
        v = fmaxf(v, lds[i]);
    return v;
}

// One workgroup a row: vocabularies of more than MOST_TILES tiles.
__global__ __launch_bounds__(THREADS) void k_sample_row(SampleArgs a)
{
    __shared__ RowLds l;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    Setting s = setting_of(a, row);
    Walker r{a.logits, row * a.stride, a.vocab, a.dtype, 0.0f};
    float top = -__builtin_inff();
    for (int64_t i = tid; i < a.vocab; i += THREADS)
        top = fmaxf(top, r.get(i));
    r.top = max_all(top, l.top);
    const bool none = r.top == -__builtin_inff();
    Cut c{0, a.vocab};
    uint64_t all = 0;
    if (!none) {
        if (s.rate < 0.0) {                      // greedy: the first of the largest
            c.key = order_key(r.top);
            c.last = find_tie(r, l, c.key, 1);
            s.rate = 1.0;
            s.min_w = 0;
        } else {
            c = find_cut(r, s, l);
        }
        all = walk_row(a, r, s, c, row, l);
    } else if (!a.probs && tid == 0) {
        a.tokens[row] = -1;
    }
    if (a.probs) {
        const double inv = none ? 0.0 : 1.0 / (double)all;
        for (int64_t i = tid; i < a.vocab; i += THREADS)
            a.probs[row * a.probs_stride + i] =
                none ? 0.0f : (float)((double)kept_weight(r, s, c, i) * inv);
    }
}

// ---- rows cut into tiles -----------------------------------------------------
//
// k_bins: each workgroup finds the largest logit of its tile and counts its
// elements by their place below it, in bins of 1 / BIN_RATE in the exponent on a
// grid that all tiles share.  A bin's count and its mass come from one 64-bit add in
// LDS: the mass, in the low half, in fixed point relative to the bin, whose
// weights lie within 7 % of each other.
// k_gather: each workgroup adds up the bins of the row and learns in which of them
// top-k and top-p cut (the masses err by a known margin, so at times two come into
// question), sums the exact weights of what is surely kept, and lists the elements
// of the bins in question.
// k_cut: one workgroup a row ranks the list, which gives the cut, and draws.
// k_probs writes the distribution instead.
// A vocabulary of one tile takes one launch (k_one) and no scratch.  Rows that the
// grid does not suit (a largest logit or a rate past what fp32 holds) or whose list
// does not fit (thousands of equal logits) are left to the search through the whole
// row, by k_cut's workgroup.

constexpr int BINS = 512;
// 32 in the exponent and more weigh nothing (2^-46); a bin more for the grid.
constexpr float BIN_RATE = 15.0f;
constexpr int MASS_BITS = 17;                    // of a bin's first weight: 16384 elements fit 32 bits
constexpr int MOST_TILES = 64;
constexpr int LIST = 4096, SUBS = THREADS;
constexpr int MOST_ROWS = 4096;                  // of one launch; more take several

// Exact weights: kept: surely, and heavy enough for min-p; below: surely inside
// top-p, were there no min-p; limit: what top-p is a part of.  All without the list.
struct Sums {
    uint64_t kept, below, limit;
};

// Which bins count: those under lo are kept; lo .. hi and kbin (BINS: no top-k)
// are listed.  odd: not for the grid.
struct Range {
    int lo, hi, kbin;
    uint32_t k_before;                           // elements above kbin
    int odd;
};

// What a row has in scratch.
struct RowScratch {
    float top[MOST_TILES];                       // of each tile
    int first[MOST_TILES];                       // its first place
    Sums sums[MOST_TILES];
    uint64_t list[LIST];                         // entry()
    Range range;
    uint32_t listed;
    uint32_t key;                                // the cut, and the sum of what is kept
    int32_t last;
    uint64_t sum;
};

// An element in the order of what is kept: falling logits, rising index.
__device__ __forceinline__ uint64_t entry(float x, uint32_t i)
{
    return ((uint64_t)~order_key(x) << 32) | i;
}

__device__ __forceinline__ float entry_value(uint64_t e) { return key_value(~(uint32_t)(e >> 32)); }

__device__ __forceinline__ float grid_rate(const Setting &s)
{
    return (float)(s.rate * (BIN_RATE * 0.69314718055994531));
}

// Whether fp32 resolves the grid around a row's largest logit: places there err by
// less than half a bin.
__device__ __forceinline__ bool on_grid(float top, float rate)
{
    return rate < 0x1p100f && fabsf(top * rate) < 0x1p22f;
}

// The bin of x, `place` being the largest's; BINS: of no weight.  It falls as x
// rises, or stays.
__device__ __forceinline__ int bin_of(float x, float place, float rate)
{
    const float d = place - floorf(x * rate);
    return d < (float)BINS ? (int)d : BINS;      // NaN: none
}

__device__ __forceinline__ bool cuts(const Setting &s) { return s.k > 0 || s.p < 1.0; }

template <int PER, int DT>
__device__ __forceinline__ void load_tile(float (&x)[PER], const SampleArgs &a, int64_t row,
                                          int64_t i0)
{
#pragma unroll
    for (int e = 0; e < PER; e += 8) {
        float v[8];
        if (i0 + e + 8 <= a.vocab) {
            load_x8<DT>(v, a.logits, row * a.stride + i0 + e);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++)
                v[k] = i0 + e + k < a.vocab ? load_one(a.logits, DT, row * a.stride + i0 + e + k)
                                            : -__builtin_inff();
        }
#pragma unroll
        for (int k = 0; k < 8; k++)
            x[e + k] = v[k] != v[k] ? -__builtin_inff() : v[k];
    }
}

template <int PER>
__device__ __forceinline__ float top_of(const float (&x)[PER], float *red)
{
    float top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < PER; e++)
        top = fmaxf(top, x[e]);
    return max_all(top, red);
}

// The row's largest logit from its tiles'.
__device__ __forceinline__ float top_of(const RowScratch &r, int tiles)
{
    const int lane = threadIdx.x & 63;
    float top = lane < tiles ? r.top[lane] : -__builtin_inff();
    for (int m = 1; m < 64; m <<= 1)
        top = fmaxf(top, __shfl_xor(top, m));
    return top;
}

// Adds a tile's elements to its bins (zeroed, and a barrier since).
template <int PER>
__device__ __forceinline__ void add_bins(const float (&x)[PER], float top, float rate, uint64_t *bins)
{
    const float place = floorf(top * rate);
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const float whole = floorf(x[e] * rate), d = place - whole;
        if (d < (float)BINS) {
            const float part = fmaf(x[e], rate, -whole);
            const float m = __builtin_amdgcn_exp2f(part * (1.44269504f / BIN_RATE));
            atomicAdd((unsigned long long *)&bins[(int)d],
                      (1ull << 32) | (uint32_t)fmaf(m, (float)(1 << MASS_BITS), 0.5f));
        }
    }
}

// First place of the largest in a tile; the others' is 2^31 - 1.
template <int PER>
__device__ __forceinline__ void note_first(const float (&x)[PER], float top, int64_t i0, int *first)
{
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int e = PER - 1; e >= 0; e--)
        at = x[e] == top ? (int)(i0 + e) : at;
    if (at != 0x7FFFFFFF)
        atomicMin(first, at);
}

template <int PER, int DT>
__global__ __launch_bounds__(THREADS) void k_bins(SampleArgs a, RowScratch *scratch, uint64_t *planes)
{
    __shared__ uint64_t bins[BINS];
    __shared__ float red[WAVES];
    __shared__ int first;
    const int tid = threadIdx.x, tile = blockIdx.x;
    const int64_t row = blockIdx.y, i0 = ((int64_t)tile * THREADS + tid) * PER;
    const Setting s = setting_of(a, row);
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    if (tid < BINS)
        bins[tid] = 0;
    if (tid == 0)
        first = 0x7FFFFFFF;
    const float top = top_of(x, red);
    RowScratch &r = scratch[row];
    if (s.rate < 0.0) {                          // greedy: its place is all there is to know
        note_first(x, top, i0, &first);
        __syncthreads();
    } else if (cuts(s)) {
        add_bins(x, top, grid_rate(s), bins);
        __syncthreads();
        if (tid < BINS)
            planes[(row * gridDim.x + tile) * BINS + tid] = bins[tid];
    }
    if (tid == 0) {
        r.top[tile] = top;
        r.first[tile] = first;
        if (tile == 0)
            r.listed = 0;
    }
}

struct RangeLds {
    uint32_t half_count[BINS];
    uint64_t half_units[BINS];
    int shift[MOST_TILES];
    uint32_t scan32[WAVES];
    double scan[WAVES];
    int lo, hi, kbin;
    uint32_t k_before;
    double mass_k, mass_through;
};

// From the bins of all tiles (or of this one, in LDS) to those that cut.
template <bool ALONE>
__device__ __forceinline__ Range find_range(RangeLds &l, const Setting &s, const RowScratch *r,
                                            const uint64_t *planes, int tiles, float top)
{
    const int tid = threadIdx.x, b = tid & (BINS - 1), half = tid / BINS;
    const float rate = grid_rate(s), place = floorf(top * rate);
    Range g{BINS, -1, BINS, 0, 0};
    if (!on_grid(top, rate)) {
        g.odd = 1;
        return g;
    }
    uint32_t count = 0;
    uint64_t units = 0;
    if constexpr (ALONE) {
        if (half == 0) {
            count = (uint32_t)(planes[b] >> 32);
            units = (uint32_t)planes[b];
        }
    } else {
        if (tid < tiles)
            l.shift[tid] = bin_of(r->top[tid], place, rate);
        __syncthreads();
        // by fours: the loads of four tiles are on their way together
        for (int c0 = half * 4; c0 < tiles; c0 += 8) {
            uint64_t v[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int c = min(c0 + k, tiles - 1), i = b - l.shift[c];
                v[k] = planes[c * BINS + max(i, 0)];
                if (i < 0 || c0 + k >= tiles)
                    v[k] = 0;
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                count += (uint32_t)(v[k] >> 32);
                units += (uint32_t)v[k];
            }
        }
        if (half) {
            l.half_count[b] = count;
            l.half_units[b] = units;
        }
        __syncthreads();
        if (!half) {
            count += l.half_count[b];
            units += l.half_units[b];
        }
    }
    if (half) {
        count = 0;
        units = 0;
    }
    if (tid == 0)
        l.lo = l.hi = l.kbin = -1;
    uint32_t all;
    double total;
    const double mass = (double)units * (double)exp2f((float)b * (-1.44269504f / BIN_RATE));
    const uint32_t before = scan_before<WAVES>(count, l.scan32, all);
    const double mass_before = scan_before<WAVES>(mass, l.scan, total);
    const bool k_cuts = s.k > 0 && (int64_t)all > s.k;
    if (k_cuts && count && before < s.k)
        atomicMax(&l.kbin, b);
    __syncthreads();
    g.kbin = k_cuts ? l.kbin : BINS;
    if (!half && b == g.kbin) {
        l.k_before = before;
        l.mass_k = mass_before;
        l.mass_through = mass_before + mass;
    }
    __syncthreads();
    if (k_cuts) {
        g.lo = g.hi = g.kbin;
        g.k_before = l.k_before;
    }
    if (s.p < 1.0) {
        const double least = k_cuts ? l.mass_k : total, most = k_cuts ? l.mass_through : total;
        // A weight's part of its bin is rounded to 2^-18 of it; the grid's rate and a
        // place on it err by 2^-24 of the place, yet the part stays within its bin.
        const double margin = 0x1p-15 + fmin((double)(fabsf(place) + BINS) * 0x1p-22, 0.08);
        if (count && (before == 0 ||
                      mass_before * (1.0 + margin) < s.p * least * (1.0 - margin)))
            atomicMax(&l.lo, b);
        if (count && (before == 0 ||
                      mass_before * (1.0 - margin) <= s.p * most * (1.0 + margin)))
            atomicMax(&l.hi, b);
        __syncthreads();
        g.lo = l.lo;
        g.hi = min(l.hi, g.kbin);
    }
    return g;
}

// A workgroup's sums, to all of its threads.
__device__ __forceinline__ Sums sum_up(Sums v, uint64_t (&lds)[3][WAVES])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = {wave_sum(v.kept), wave_sum(v.below), wave_sum(v.limit)};
    if (lane == 0) {
        lds[0][wave] = v.kept;
        lds[1][wave] = v.below;
        lds[2][wave] = v.limit;
    }
    __syncthreads();
    Sums all{0, 0, 0};
    for (int i = 0; i < WAVES; i++) {
        all.kept += lds[0][i];
        all.below += lds[1][i];
        all.limit += lds[2][i];
    }
    return all;
}

// Sums of a tile's elements by the range, and the list of those in question (of
// which `most` fit), counted in *listed.
template <int PER>
__device__ __forceinline__ Sums gather(const float (&x)[PER], int64_t i0, float top, const Setting &s,
                                       const Range &g, uint64_t *list, uint32_t most, uint32_t *listed)
{
    const float rate = grid_rate(s), place = floorf(top * rate);
    Sums mine{0, 0, 0};
    if (g.odd)
        return mine;
    const bool cut = g.hi >= 0 || g.kbin < BINS;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const int bin = cut || on_grid(top, rate) ? bin_of(x[e], place, rate) : 0;
        if (bin >= BINS || (bin > g.kbin))
            continue;
        const uint64_t w = weight(x[e], top, s);
        mine.limit += bin < g.kbin ? w : 0;
        if (bin < g.lo) {
            mine.below += w;
            mine.kept += w >= s.min_w ? w : 0;
        } else if (w && (bin <= g.hi || bin == g.kbin)) {
            const uint32_t at = atomicAdd(listed, 1u);
            if (at < most)
                list[at] = entry(x[e], (uint32_t)(i0 + e));
        }
    }
    return mine;
}

template <int PER, int DT>
__global__ __launch_bounds__(THREADS) void k_gather(SampleArgs a, RowScratch *scratch,
                                                    const uint64_t *planes)
{
    constexpr int MOST = PER * THREADS < LIST ? PER * THREADS : LIST;
    __shared__ RangeLds range;
    __shared__ uint64_t list[MOST], sums[3][WAVES];
    __shared__ uint32_t listed, base;
    const int tid = threadIdx.x, tile = blockIdx.x, tiles = gridDim.x;
    const int64_t row = blockIdx.y, i0 = ((int64_t)tile * THREADS + tid) * PER;
    const Setting s = setting_of(a, row);
    RowScratch &r = scratch[row];
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    const float top = top_of(r, tiles);
    if (top == -__builtin_inff() || s.rate < 0.0)
        return;
    if (tid == 0)
        listed = 0;
    __syncthreads();
    Range g{BINS, -1, BINS, 0, 0};
    if (cuts(s))
        g = find_range<false>(range, s, &r, planes + row * tiles * BINS, tiles, top);
    const Sums all = sum_up(gather(x, i0, top, s, g, list, MOST, &listed), sums);
    const uint32_t n = listed;
    if (tid == 0) {
        r.sums[tile] = all;
        if (tile == 0)
            r.range = g;
        if (n)
            base = atomicAdd(&r.listed, n);
    }
    if (n) {
        __syncthreads();
        for (uint32_t i = tid; i < min(n, (uint32_t)MOST) && base + i < LIST; i += THREADS)
            r.list[base + i] = list[i];
    }
}

struct CutLds {
    uint64_t list[LIST], weight[LIST];
    uint32_t sub_count[SUBS];
    uint64_t sub_mass[SUBS];
    uint64_t in_sub[LIST];                       // those of one sub-bin
    uint64_t tile_kept[MOST_TILES];
    uint64_t scan[WAVES];
    uint32_t scan32[WAVES];
    unsigned long long cut, low_mass, part;
    uint32_t low, least, most, n_in;
    int k_sub, p_sub;
    uint32_t sub_before;
    uint64_t sub_mass_before;
};

// How many entries of the list, and how much, come before one.
struct Ranked {
    uint32_t rank;
    uint64_t before;
};

// Entries of sub-bin `sub` and, for each that a thread has (list[tid + ...]), how
// many and how much of them come before it.
template <typename F>
__device__ __forceinline__ void rank_in(CutLds &l, uint32_t n, int sub, uint32_t least, int shift,
                                        float top, const Setting &s, F f)
{
    const int tid = threadIdx.x;
    if (tid == 0)
        l.n_in = 0;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += THREADS)
        if ((int)(((uint32_t)(l.list[i] >> 32) - least) >> shift) == sub)
            l.in_sub[atomicAdd(&l.n_in, 1u)] = l.list[i];
    __syncthreads();
    const uint32_t m = l.n_in, rank0 = l.sub_before;
    const uint64_t before0 = l.sub_mass_before;
    for (uint32_t i = tid; i < m; i += THREADS) {
        const uint64_t e = l.in_sub[i];
        uint32_t rank = rank0, same = 0;
        uint64_t before = before0;
        for (uint32_t j = 0; j < m; j++) {
            const uint64_t o = l.in_sub[j];
            const bool ahead = o < e;
            rank += ahead;
            // equal logits weigh alike; the others are looked up
            const bool alike = (uint32_t)(o >> 32) == (uint32_t)(e >> 32);
            same += ahead && alike;
            if (ahead && !alike)
                before += weight(entry_value(o), top, s);
        }
        const uint64_t w = weight(entry_value(e), top, s);
        f(e, w, Ranked{rank, before + same * w});
    }
}

// The cut, from the list in LDS (n entries); adds what is kept of it to the tiles'
// sums.  Sub-bins of the list's own range, in falling order, bring it down to the
// few elements around a cut; those are ranked one by one.
__device__ __forceinline__ Cut rank_list(CutLds &l, const Setting &s, const Range &g, uint32_t n,
                                         const Sums &all, float top, int tile_size)
{
    const int tid = threadIdx.x;
    const float rate = grid_rate(s), place = floorf(top * rate);
    const bool k_cuts = g.kbin < BINS;
    l.sub_count[tid] = 0;
    l.sub_mass[tid] = 0;
    if (tid == 0) {
        l.cut = l.low_mass = l.part = 0;
        l.low = l.most = 0;
        l.least = ~0u;
        l.k_sub = l.p_sub = -1;
    }
    __syncthreads();
    uint32_t least = ~0u, most = 0, low = 0;
    uint64_t low_mass = 0;
    for (uint32_t i = tid; i < n; i += THREADS) {
        const uint32_t k = (uint32_t)(l.list[i] >> 32);
        const float x = key_value(~k);
        const uint64_t w = weight(x, top, s);
        l.weight[i] = w;
        least = min(least, k);
        most = max(most, k);
        if (k_cuts && bin_of(x, place, rate) < g.kbin) {
            low++;
            low_mass += w;
        }
    }
    if (most) {
        atomicMin(&l.least, least);
        atomicMax(&l.most, most);
    }
    if (low) {
        atomicAdd(&l.low, low);
        atomicAdd(&l.low_mass, (unsigned long long)low_mass);
    }
    __syncthreads();
    least = l.least;
    const uint32_t span = l.most - least;
    const int shift = max(32 - __builtin_clz(span | 1) - 10, 0);     // SUBS = 2^10
    for (uint32_t i = tid; i < n; i += THREADS) {
        const int sub = (int)(((uint32_t)(l.list[i] >> 32) - least) >> shift);
        atomicAdd(&l.sub_count[sub], 1u);
        atomicAdd((unsigned long long *)&l.sub_mass[sub], (unsigned long long)l.weight[i]);
    }
    __syncthreads();
    const uint32_t count = l.sub_count[tid];
    const uint64_t mass = l.sub_mass[tid];
    uint32_t all_count;
    uint64_t all_mass;
    const uint32_t before = scan_before<WAVES>(count, l.scan32, all_count);
    const uint64_t mass_before = scan_before<WAVES>(mass, l.scan, all_mass);
    // top-k keeps k_rank entries of the list: those above kbin and some in it
    const uint32_t k_rank = k_cuts ? (uint32_t)(s.k - g.k_before) + l.low : ~0u;
    uint64_t total = all.limit;
    if (k_cuts) {
        if (count && before < k_rank)
            atomicMax(&l.k_sub, tid);
        __syncthreads();
        if (tid == l.k_sub) {
            l.sub_before = before;
            l.sub_mass_before = mass_before;
        }
        if (s.p < 1.0) {
            rank_in(l, n, l.k_sub, least, shift, top, s, [&](uint64_t, uint64_t w, const Ranked &r) {
                if (r.rank < k_rank)
                    atomicAdd(&l.part, (unsigned long long)w);
            });
            __syncthreads();
            total += l.sub_mass_before + l.part - l.low_mass;
        }
    }
    if (count && before < k_rank && inside(all.below + mass_before, s.p, total))
        atomicMax(&l.p_sub, tid);
    __syncthreads();
    if (tid == l.p_sub) {
        l.sub_before = before;
        l.sub_mass_before = mass_before;
    }
    rank_in(l, n, l.p_sub, least, shift, top, s, [&](uint64_t e, uint64_t, const Ranked &r) {
        if (r.rank < k_rank && inside(all.below + r.before, s.p, total))
            atomicMax(&l.cut, (unsigned long long)e);
    });
    __syncthreads();
    const uint64_t cut = l.cut;
    for (uint32_t i = tid; i < n; i += THREADS)
        if (l.list[i] <= cut && l.weight[i] >= s.min_w)
            atomicAdd((unsigned long long *)&l.tile_kept[(uint32_t)l.list[i] / tile_size],
                      (unsigned long long)l.weight[i]);
    __syncthreads();
    return Cut{~(uint32_t)(cut >> 32), (int64_t)(uint32_t)cut};
}

// A row's end: from the sums (in tile_kept, too) and the list in LDS to its token, or
// to its cut and the sum of what is kept.  x: tile `mine`'s elements, or none (-1).
template <int PER, int DT>
__device__ __forceinline__ uint64_t finish(const SampleArgs &a, int64_t row, CutLds &l, RowLds &rl,
                                           const Setting &s, const Range &g, const Sums &all,
                                           uint32_t n, float top, int tiles, Cut &c,
                                           float (&x)[PER], int mine)
{
    const int tid = threadIdx.x, lane = tid & 63;
    if (g.odd || n > LIST) {
        const Walker walker{a.logits, row * a.stride, a.vocab, a.dtype, top};
        c = find_cut(walker, s, rl);
        return walk_row(a, walker, s, c, row, rl);
    }
    if (n)
        c = rank_list(l, s, g, n, all, top, PER * THREADS);
    // the tile, then the element in it, where the running sum passes u
    const uint64_t v = lane < tiles ? l.tile_kept[lane] : 0, run = scan_wave(v);
    const uint64_t sum = lane_value(run, 63), thr = place_in(s.u, sum);
    if (a.probs)
        return sum;
    const int tile = __builtin_ctzll(__ballot(run > thr));
    const int64_t j0 = ((int64_t)tile * THREADS + tid) * PER;
    if (tile != mine)
        load_tile<PER, DT>(x, a, row, j0);
    uint64_t w[PER], own = 0, whole;
#pragma unroll
    for (int e = 0; e < PER; e++) {
        w[e] = kept(c, order_key(x[e]), j0 + e) ? weight(x[e], top, s) : 0;
        w[e] = w[e] >= s.min_w ? w[e] : 0;
        own += w[e];
    }
    __syncthreads();
    uint64_t at = lane_value(run - v, tile) + scan_before<WAVES>(own, l.scan, whole);
    if (at <= thr && thr < at + own) {
        int hit = 0;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            at += w[e];
            hit += at <= thr;
        }
        a.tokens[row] = (int32_t)(j0 + hit);
    }
    return sum;
}

template <int PER, int DT>
__global__ __launch_bounds__(THREADS) void k_cut(SampleArgs a, RowScratch *scratch, int tiles)
{
    __shared__ CutLds l;
    __shared__ RowLds rl;
    __shared__ uint64_t sums[3][WAVES];
    __shared__ int first;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    Setting s = setting_of(a, row);
    RowScratch &r = scratch[row];
    const float top = top_of(r, tiles);
    const bool none = top == -__builtin_inff();
    Cut c{0, a.vocab};
    uint64_t sum = 0;
    if (none || s.rate < 0.0) {
        // an empty row, or greedy: the first of the largest
        if (!none) {
            if (tid == 0)
                first = 0x7FFFFFFF;
            __syncthreads();
            if (tid < tiles && r.top[tid] == top)
                atomicMin(&first, r.first[tid]);
            __syncthreads();
            c = {order_key(top), first};
            sum = uint64_t(1) << s.bits;
        }
        if (tid == 0 && !a.probs)
            a.tokens[row] = none ? -1 : (int32_t)c.last;
    } else {
        Sums v{0, 0, 0};
        const uint32_t n = r.listed;
        const Range g = r.range;
        if (tid < tiles) {
            v = r.sums[tid];
            l.tile_kept[tid] = v.kept;
        }
        for (uint32_t i = tid; i < min(n, (uint32_t)LIST); i += THREADS)
            l.list[i] = r.list[i];
        const Sums all = sum_up(v, sums);
        float x[PER];
        sum = finish<PER, DT>(a, row, l, rl, s, g, all, n, top, tiles, c, x, -1);
    }
    if (a.probs && tid == 0) {
        r.key = c.key;
        r.last = (int32_t)min(c.last, (int64_t)0x7FFFFFFF);
        r.sum = sum;
    }
}

// The kept part of eight elements' distribution.
template <int PER>
__device__ __forceinline__ void write_probs(const SampleArgs &a, int64_t row, int64_t i0,
                                            const float (&x)[PER], float top, const Setting &s,
                                            const Cut &c, uint64_t sum)
{
    const double inv = sum ? 1.0 / (double)sum : 0.0;
#pragma unroll
    for (int e0 = 0; e0 < PER; e0 += 8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[e] = 0.0f;
            if (sum && kept(c, order_key(x[e0 + e]), i0 + e0 + e)) {
                const uint64_t w = weight(x[e0 + e], top, s);
                v[e] = w >= s.min_w ? (float)((double)w * inv) : 0.0f;
            }
        }
        if (i0 + e0 + 8 <= a.vocab) {
            store_x8<TQ_F32>(a.probs, row * a.probs_stride + i0 + e0, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (i0 + e0 + e < a.vocab)
                    a.probs[row * a.probs_stride + i0 + e0 + e] = v[e];
        }
    }
}

// Greedy takes one element, whatever min-p says.
__device__ __forceinline__ void set_greedy(Setting &s)
{
    if (s.rate < 0.0) {
        s.rate = 1.0;
        s.min_w = 0;
    }
}

template <int PER, int DT>
__global__ __launch_bounds__(THREADS) void k_probs(SampleArgs a, const RowScratch *scratch)
{
    const int64_t row = blockIdx.y, i0 = ((int64_t)blockIdx.x * THREADS + threadIdx.x) * PER;
    Setting s = setting_of(a, row);
    set_greedy(s);
    const RowScratch &r = scratch[row];
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    const float top = top_of(r, gridDim.x);
    write_probs(a, row, i0, x, top, s, Cut{r.key, r.last}, r.sum);
}

// A vocabulary of one tile.
template <int PER, int DT> __global__ __launch_bounds__(THREADS) void k_one(SampleArgs a)
{
    __shared__ CutLds l;
    __shared__ RowLds rl;
    __shared__ RangeLds range;
    __shared__ uint64_t bins[BINS], sums[3][WAVES];
    __shared__ int first;
    __shared__ uint32_t listed;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, i0 = (int64_t)tid * PER;
    Setting s = setting_of(a, row);
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    if (tid < BINS)
        bins[tid] = 0;
    if (tid == 0) {
        first = 0x7FFFFFFF;
        listed = 0;
    }
    const float top = top_of(x, rl.top);
    const bool none = top == -__builtin_inff();
    Cut c{0, a.vocab};
    uint64_t sum = 0;
    if (none || s.rate < 0.0) {
        if (!none) {
            note_first(x, top, i0, &first);
            __syncthreads();
            c = {order_key(top), first};
            sum = uint64_t(1) << s.bits;
        }
        if (tid == 0 && !a.probs)
            a.tokens[row] = none ? -1 : (int32_t)c.last;
        set_greedy(s);
    } else {
        Range g{BINS, -1, BINS, 0, 0};
        if (cuts(s)) {
            add_bins(x, top, grid_rate(s), bins);
            __syncthreads();
            g = find_range<true>(range, s, nullptr, bins, 1, top);
        }
        const Sums all = sum_up(gather(x, i0, top, s, g, l.list, LIST, &listed), sums);
        const uint32_t n = listed;
        if (tid == 0)
            l.tile_kept[0] = all.kept;
        __syncthreads();
        sum = finish<PER, DT>(a, row, l, rl, s, g, all, n, top, 1, c, x, 0);
    }
    if (a.probs)
        write_probs(a, row, i0, x, top, s, c, sum);
}

constexpr int PER = 8;

int64_t tiles_of(int64_t vocab) { return (vocab + PER * THREADS - 1) / (PER * THREADS); }

template <int DT> hipError_t launch_dt(SampleArgs a, void *scratch, hipStream_t s)
{
    const int64_t tiles = tiles_of(a.vocab), rows = a.rows;
    if (tiles == 1 || tiles > MOST_TILES) {
        if (!grid_fits(rows, THREADS))
            return hipErrorInvalidConfiguration;
        if (tiles == 1)
            k_one<PER, DT><<<dim3((unsigned)rows), THREADS, 0, s>>>(a);
        else
            k_sample_row<<<dim3((unsigned)rows), THREADS, 0, s>>>(a);
        return hipGetLastError();
    }
    RowScratch *r = (RowScratch *)scratch;
    uint64_t *planes = (uint64_t *)(r + std::min<int64_t>(rows, MOST_ROWS));
    const int64_t size = DT == TQ_F32 ? 4 : 2;
    for (int64_t at = 0; at < rows; at += MOST_ROWS) {
        const int64_t n = std::min<int64_t>(rows - at, MOST_ROWS);
        const dim3 grid((unsigned)tiles, (unsigned)n);
        k_bins<PER, DT><<<grid, THREADS, 0, s>>>(a, r, planes);
        k_gather<PER, DT><<<grid, THREADS, 0, s>>>(a, r, planes);
        k_cut<PER, DT><<<dim3((unsigned)n), THREADS, 0, s>>>(a, r, (int)tiles);
        if (a.probs)
            k_probs<PER, DT><<<grid, THREADS, 0, s>>>(a, r);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        a.logits = (const uint8_t *)a.logits + MOST_ROWS * a.stride * size;
        a.temperature += a.temperature ? MOST_ROWS : 0;
        a.top_k += a.top_k ? MOST_ROWS : 0;
        a.top_p += a.top_p ? MOST_ROWS : 0;
        a.min_p += a.min_p ? MOST_ROWS : 0;
        a.u += a.u ? MOST_ROWS : 0;
        a.tokens += a.tokens ? MOST_ROWS : 0;
        a.probs += a.probs ? MOST_ROWS * a.probs_stride : 0;
    }
    return hipSuccess;
}

}  // namespace

size_t sample_scratch_bytes(int64_t rows, int64_t vocab)
{
    const int64_t tiles = tiles_of(vocab), n = std::min<int64_t>(rows, MOST_ROWS);
    return tiles == 1 || tiles > MOST_TILES
               ? 0
               : (size_t)n * (sizeof(RowScratch) + tiles * BINS * sizeof(uint64_t));
}

hipError_t launch_sample(const SampleArgs &a, void *scratch, hipStream_t s)
{
    switch (a.dtype) {
    case TQ_F32: return launch_dt<TQ_F32>(a, scratch, s);
    case TQ_BF16: return launch_dt<TQ_BF16>(a, scratch, s);
    case TQ_F16: return launch_dt<TQ_F16>(a, scratch, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace tq
