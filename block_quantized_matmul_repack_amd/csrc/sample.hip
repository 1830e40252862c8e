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
//
// Of rows of several tiles four launches read the logits twice: bins (k_bins),
// the bins that the cuts are in (k_range), those bins' elements and the tiles' sums
// of the others (k_gather), the cuts and the token (k_cut); distributions are a
// third reading (k_probs).  us of each, rows of 128001: one, all filters, 4.1 + 5.8 +
// 3.8 + 6.0, latency; 64, top-p, 10.2 + 4.2 + 15.8 + 10.5, where 11 of k_gather's are
// its vector instructions, most of them the fp64 of the weights (two readings from
// memory are 9); 128 of bf16, top-k and top-p, 16.6 + 6.0 + 12.2 + 5.8 and
// k_probs 21.9, 4.5 TB/s.  The launches of one workgroup a row are bound by its own
// instructions (400 to 800 a wave, sixteen waves on a unit: 3 to 6 us), whence a pair
// of bins and few elements a thread there.  A workgroup for each row that does it all took 418 us for
// one row and 493 for 64.
#include <algorithm>
#include <type_traits>

#include "block_ops.h"

namespace tq {
namespace {

constexpr int WAVES = 16, THREADS = 64 * WAVES;
constexpr int DIGITS = 256;

// Bins of the exponent (see k_bins): 60 to one of it.
constexpr float BIN_RATE = 60.0f;

// The settings of a row.
struct Setting {
    double rate;                                 // log2(e) / T; below 0: the likeliest token
    double p;                                    // >= 1: off
    uint64_t min_w;                              // the least weight that min-p keeps
    int k;                                       // <= 0: off
    int bits;                                    // s
    float u;
    float grid;                                  // bins for one of a logit
};

__device__ __forceinline__ float temperature_of(const SampleArgs &a, int64_t row)
{
    return a.temperature ? a.temperature[row] : 1.0f;
}

__device__ __forceinline__ Setting setting_of(const SampleArgs &a, int64_t row)
{
    Setting s;
    const float t = temperature_of(a, row), p = a.top_p ? a.top_p[row] : 1.0f;
    const float m = a.min_p ? a.min_p[row] : 0.0f;
    s.rate = t > 0.0f ? 1.4426950408889634074 / (double)t : -1.0;
    s.p = p < 1.0f ? (double)p : 1.0;            // NaN: off
    s.min_w = m > 0.0f ? (uint64_t)ceil(ldexp((double)fminf(m, 1.0f), a.bits)) : 0;
    s.k = a.top_k ? a.top_k[row] : 0;
    s.bits = a.bits;
    s.u = a.u ? a.u[row] : 0.0f;
    s.grid = BIN_RATE / t;
    return s;
}

// 2^52 + 2^t, rounded to a whole number, for -1000 < t < 52: 2^n times a polynomial
// for 2^f, |f| <= 1/2 (interpolated in Chebyshev's points, off by 2^-51).
__device__ __forceinline__ double whole_exp2(double t)
{
    // the coefficients in scalar registers: as literals each takes two moves
    double c[10] = {7.072585949269223e-09, 1.0208690299958306e-07, 1.321544258792169e-06, 1.5252657260200837e-05,
                    0.0001540353044173605, 0.0013333558230164974, 0.009618129107606888,
                    0.05550410866444772, 0.24022650695910097, 0.69314718055995};
#pragma unroll
    for (int i = 0; i < 10; i++)
        asm("" : "+s"(c[i]));
    // with 1.5 * 2^52 added the whole part is in the low bits: no conversion
    const double near = t + 0x1.8p52, f = t - (near - 0x1.8p52);
    const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, near);
    double p = c[0];
#pragma unroll
    for (int i = 1; i < 10; i++)
        p = fma(p, f, c[i]);
    p = fma(p, f, 1.0);
    const uint64_t scaled = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(uint32_t)n << 52);
    return __builtin_bit_cast(double, scaled) + 0x1p52;
}

constexpr uint64_t LOW52 = (uint64_t(1) << 52) - 1;

// w of 2^52 + w.
__device__ __forceinline__ uint64_t whole_bits(double v)
{
    return __builtin_bit_cast(uint64_t, v) & LOW52;
}

// A weight in units of 2^-bits; 0 for what is no number, or -infinity.
__device__ __forceinline__ uint64_t weight(float x, float top, const Setting &s)
{
    const double t = ((double)x - (double)top) * s.rate + (double)s.bits;
    // 1/4 rounds to 0, and so do NaN and what is far below
    const uint64_t w = whole_bits(whole_exp2(fmax(t, -2.0)));
    const uint64_t got = x > -__builtin_inff() ? w : 0;
    return x == top ? uint64_t(1) << s.bits : got;
}

// The same as a double, for an element that is in a bin (below): then -16 < t.
__device__ __forceinline__ double weight_in_bin(float x, float top, const Setting &s)
{
    return whole_exp2(((double)x - (double)top) * s.rate + (double)s.bits) - 0x1p52;
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
        const bool last = own && (K ? cb < (uint32_t)s.k : inside(mb, s.p, total));
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
        if (K && shift == 24 && all_count <= (uint32_t)s.k)
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
            m = (uint32_t)s.k - f.count_before;
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
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[threadIdx.x & (WAVES - 1)];
    for (int m = 1; m < WAVES; m <<= 1)
        v = fmaxf(v, __shfl_xor(v, m));
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
// weights lie within 2 % of each other.
// k_range: one workgroup a row adds up its bins and learns in which of them top-k and
// top-p cut (the masses err by a known margin, so at times two come into question).
// k_gather: each workgroup, a quarter of a tile (a part), sums the exact weights of what
// is surely kept, and lists the elements of the bins in question.
// k_cut: one workgroup a row ranks the list, which gives the cut, and draws.
// k_probs writes the distribution instead.
// A vocabulary of one tile takes one launch (k_one) and no scratch.  Rows that the
// grid does not suit (largest logit * 60 / T past 2^22) or whose list does not fit are
// left to the search through the whole row, by k_cut's workgroup, 0.3 to 1.8 ms for
// 128001.  A list does not fit with tens of thousands of logits within 2 % at a
// cut, thousands of unlike ones within 2e-5, or with top-p so near 1 that find_range's
// margin, 5e-4 of the sum for logits of a few tens, takes the tail in: 64 rows of
// 128001, spread 2.5, take 41 us with p = 0.95, 46 with 0.99, 80 with 0.999, 460 with
// 0.9995; of a mean of 20, 590 from 0.999 on; with T = 1e-4, off the grid, 335.

// 32 in the exponent and more weigh nothing (2^-46); a bin more for the grid.
constexpr int BINS = 2048, EACH = BINS / THREADS;
static_assert(EACH == 2, "a pair of bins a thread");
// e^(-1 / BIN_RATE): from a bin to the next.
constexpr float STEP = 0.98347145f;
constexpr int GUARD = 4, PLANE = GUARD + BINS;   // a tile's bins in scratch, behind entries of nothing
constexpr int MASS_BITS = 17;                    // of a bin's first weight: 16384 elements fit 32 bits
constexpr int MOST_TILES = 64;
// More tiles than are on the chip at once (two a unit): two of them share their bins. 63
// rows of 128001, top-p / bf16, top-k and top-p: 38.2 / 30.5 us, 39.7 / 33.0 apart.
constexpr int RESIDENT = 512;
constexpr int LIST = 32768;                      // entries of a row
constexpr int GATHER_THREADS = 256;
constexpr int PARTS = THREADS / GATHER_THREADS, MOST_PARTS = MOST_TILES * PARTS;    // of a tile, a row
constexpr int SHORT = 128, SUBS = THREADS, MOST_ALIKE = 4096;

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
    Setting setting;
    Range range;
    float row_top;
    uint32_t listed;
    uint32_t key;                                // the cut, and the sum of what is kept
    int32_t last;
    uint64_t sum;
    float top[MOST_TILES];                       // of each tile
    int first[MOST_TILES];                       // its first place
    Sums sums[MOST_PARTS];
    uint64_t list[LIST];                         // entry()
};

// An element in the order of what is kept: falling logits, rising index.
__device__ __forceinline__ uint64_t entry(float x, uint32_t i)
{
    return ((uint64_t)~order_key(x) << 32) | i;
}

__device__ __forceinline__ float entry_value(uint64_t e) { return key_value(~(uint32_t)(e >> 32)); }

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

// -infinity past the row's end.  A NaN has no bin, no weight and the key of -infinity.
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
            x[e + k] = v[k];
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

// Adds a tile's elements to its bins (zeroed, and a barrier since).  Without top-k
// only the masses are asked for, and 32-bit adds meet in half as many banks.
template <int PER>
__device__ __forceinline__ void add_bins(const float (&x)[PER], float top, float rate, bool counted,
                                         uint64_t *bins)
{
    constexpr float ONE = 1 << MASS_BITS;
    const float place = floorf(top * rate);
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const float whole = floorf(x[e] * rate), d = place - whole;
        if (d < (float)BINS) {
            // e^(part / BIN_RATE) of 0 <= part < 1: a square's error is below 2^-20
            const float part = fmaf(x[e], rate, -whole);
            const float more = fmaf(part, ONE / (2 * BIN_RATE * BIN_RATE), ONE / BIN_RATE);
            const uint32_t units = (uint32_t)fmaf(part, more, ONE + 0.5f);
            if (counted)
                atomicAdd((unsigned long long *)&bins[(int)d], (1ull << 32) | units);
            else
                atomicAdd((uint32_t *)bins + (int)d, units);
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
    const float t = temperature_of(a, row);
    const int k = a.top_k ? a.top_k[row] : 0;
    const bool counted = k > 0, cut = counted || (a.top_p && a.top_p[row] < 1.0f);
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
#pragma unroll
    for (int i = 0; i < EACH; i++)
        bins[i * THREADS + tid] = 0;
    if (tid == 0)
        first = 0x7FFFFFFF;
    const float top = top_of(x, red);
    RowScratch &r = scratch[row];
    if (!(t > 0.0f)) {                           // greedy: its place is all there is to know
        note_first(x, top, i0, &first);
        __syncthreads();
    } else if (cut) {
        add_bins(x, top, BIN_RATE / t, counted, bins);
        __syncthreads();
        // without counts: 32-bit masses in the first half of its place
        uint64_t *out = planes + (row * gridDim.x + tile) * PLANE;
        const int at = counted ? GUARD : GUARD / 2;
#pragma unroll
        for (int i = 0; i < EACH; i++)
            if (counted || i < EACH / 2)
                out[at + i * THREADS + tid] = bins[i * THREADS + tid];
        if (tid < at)
            out[tid] = 0;
    }
    if (tid == 0) {
        r.top[tile] = top;
        r.first[tile] = first;
    }
}

struct RangeLds {
    uint32_t scan32[WAVES];
    float scan[WAVES];
    int lo, hi, kbin;
    uint32_t k_before;
    float mass_k, mass_through;
};

// The largest number of the threads with `is`, into *p: one add to it a wave.
__device__ __forceinline__ void note_last(bool is, int number, int *p)
{
    const uint64_t some = __ballot(is);
    if (some && (int)(threadIdx.x & 63) == 63 - __builtin_clzll(some))
        atomicMax(p, number);
}

// The same of a pair of neighbours.
__device__ __forceinline__ void note_last(const bool (&is)[2], int number, int *p)
{
    note_last(is[0] || is[1], number + is[1], p);
}

// From the bins of the row (thread t: bins 2t and 2t + 1) to those that cut.
__device__ __forceinline__ Range find_range(RangeLds &l, const uint32_t (&count)[2],
                                            const uint64_t (&units)[2], const Setting &s, float top)
{
    const int tid = threadIdx.x;
    const float place = floorf(top * s.grid);
    Range g{BINS, -1, BINS, 0, 0};
    if (tid == 0)
        l.lo = l.hi = l.kbin = -1;
    const int b = 2 * tid;
    const float first = __builtin_amdgcn_exp2f((float)b * (-1.44269504f / BIN_RATE));
    const float mass[2] = {(float)units[0] * first, (float)units[1] * (first * STEP)};
    float total;
    const float ahead0 = scan_before<WAVES>(mass[0] + mass[1], l.scan, total);
    const float ahead[2] = {ahead0, ahead0 + mass[0]};
    float least = total, most = total;
    uint32_t all = 0, before[2] = {};
    if (s.k > 0) {
        before[0] = scan_before<WAVES>(count[0] + count[1], l.scan32, all);
        before[1] = before[0] + count[0];
    }
    if (s.k > 0 && all > (uint32_t)s.k) {
        note_last({count[0] && before[0] < (uint32_t)s.k, count[1] && before[1] < (uint32_t)s.k}, b,
                  &l.kbin);
        __syncthreads();
        g.kbin = g.lo = g.hi = l.kbin;
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (b + i == g.kbin) {
                l.k_before = before[i];
                l.mass_k = ahead[i];
                l.mass_through = ahead[i] + mass[i];
            }
        __syncthreads();
        g.k_before = l.k_before;
        least = l.mass_k;
        most = l.mass_through;
    }
    if (s.p < 1.0) {
        // A weight's part of its bin is rounded to 2^-18 of it, sums of 2048 bins to
        // 2^-19 (by lanes and waves); the grid's rate and a place on it err by 2^-24
        // of the place, yet the part stays within its bin.
        const float margin = 0x1p-15f + fminf((fabsf(place) + BINS) * 0x1p-23f, 0.02f);
        const float p = (float)s.p, sure = p * least * (1.0f - margin), some = p * most * (1.0f + margin);
        bool lo[2], hi[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            lo[i] = count[i] && (b + i == 0 || ahead[i] * (1.0f + margin) < sure);
            hi[i] = count[i] && (b + i == 0 || ahead[i] * (1.0f - margin) <= some);
        }
        note_last(lo, b, &l.lo);
        note_last(hi, b, &l.hi);
        __syncthreads();
        g.lo = max(l.lo, 0);
        g.hi = min(l.hi, g.kbin);
    }
    return g;
}

// COUNTED: the tiles' bins hold counts, too; else a count is what is not 0.  shift: of
// lane's tile, the bins that its own lie behind the row's; before them a pair is read
// from the guard.
template <bool COUNTED>
__device__ __forceinline__ void add_tiles(uint32_t (&count)[2], uint64_t (&units)[2],
                                          const uint64_t *from, int tiles, int shift)
{
    typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(4)));
    typedef uint64_t u64x2a __attribute__((ext_vector_type(2), aligned(8)));
    using T = std::conditional_t<COUNTED, u64x2a, u32x2a>;
    constexpr int TOGETHER = 8;                  // loads of so many tiles
    const int b = 2 * (int)threadIdx.x;
    for (int c0 = 0; c0 < tiles; c0 += TOGETHER) {
        T v[TOGETHER];
#pragma unroll
        for (int k = 0; k < TOGETHER; k++) {
            // past the last tile the guard of the last one
            const int c = min(c0 + k, tiles - 1);
            const int down = c0 + k < tiles ? __builtin_amdgcn_readlane(shift, c) : BINS;
            const int at = max(b - down, -2) + GUARD;
            if constexpr (COUNTED)
                v[k] = *(const T *)(from + c * PLANE + at);
            else
                v[k] = *(const T *)((const uint32_t *)(from + c * PLANE) + at);
        }
#pragma unroll
        for (int k = 0; k < TOGETHER; k++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if constexpr (COUNTED)
                    count[i] += (uint32_t)(v[k][i] >> 32);
                else
                    count[i] |= v[k][i];
                units[i] += (uint32_t)v[k][i];
            }
    }
}

__global__ __launch_bounds__(THREADS) void k_range(SampleArgs a, RowScratch *scratch,
                                                   const uint64_t *planes, int tiles)
{
    __shared__ RangeLds l;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    RowScratch &r = scratch[row];
    const float tile_top = lane < tiles ? r.top[lane] : -__builtin_inff();
    const Setting s = setting_of(a, row);
    const float top = wave_max(tile_top);
    Range g{BINS, -1, BINS, 0, 0};
    if (top > -__builtin_inff() && s.rate >= 0.0 && cuts(s)) {
        if (on_grid(top, s.grid)) {
            const int shift = bin_of(tile_top, floorf(top * s.grid), s.grid);    // of lane's tile
            const uint64_t *from = planes + row * tiles * PLANE;
            uint32_t count[2] = {};
            uint64_t units[2] = {};
            if (s.k > 0)
                add_tiles<true>(count, units, from, tiles, shift);
            else
                add_tiles<false>(count, units, from, tiles, shift);
            g = find_range(l, count, units, s, top);
        } else {
            g.odd = 1;
        }
    }
    if (tid == 0) {
        r.setting = s;
        r.range = g;
        r.row_top = top;
        r.listed = 0;
    }
}

// A workgroup's sums, to all of its threads.
__device__ __forceinline__ Sums sum_up(Sums v, uint64_t (&lds)[3][WAVES])
{
    const int lane = threadIdx.x & 63;
    v = {wave_sum(v.kept), wave_sum(v.below), wave_sum(v.limit)};
    if (lane == 0) {
        lds[0][threadIdx.x >> 6] = v.kept;
        lds[1][threadIdx.x >> 6] = v.below;
        lds[2][threadIdx.x >> 6] = v.limit;
    }
    __syncthreads();
    const int i = lane & (WAVES - 1);
    return {sum_lanes(lds[0][i], WAVES), sum_lanes(lds[1][i], WAVES), sum_lanes(lds[2][i], WAVES)};
}

// Sums of a tile's elements by the range, and the list of those in question (of
// which `most` fit), counted in *listed.
template <int PER>
__device__ __forceinline__ Sums gather(const float (&x)[PER], int64_t i0, float top, const Setting &s,
                                       const Range &g, uint64_t *list, uint32_t most, uint32_t *listed)
{
    const float rate = s.grid, place = floorf(top * rate);
    Sums mine{0, 0, 0};
    if (g.odd)
        return mine;
    if (g.lo == BINS && !on_grid(top, rate)) {
        // nothing cuts: any element may be kept
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const uint64_t w = weight(x[e], top, s);
            mine.kept += w >= s.min_w ? w : 0;
            mine.below += w;
        }
        return mine;
    }
    const float lo = (float)g.lo, hi = (float)g.hi;
    float d[PER];
#pragma unroll
    for (int e = 0; e < PER; e++)
        d[e] = place - floorf(x[e] * rate);
    uint32_t question = 0;
    if (g.kbin < BINS) {                         // top-k leaves few
        const float kbin = (float)g.kbin, end = kbin + 1.0f;
        bool some = false;
#pragma unroll
        for (int e = 0; e < PER; e++)
            some = some || d[e] < end;
        if (!__any(some))
            return mine;                         // a wave of what top-k leaves out
        // whole numbers below 2^50: exact in any order
        const double min_w = (double)s.min_w;
        double kept = 0.0, below = 0.0, limit = 0.0;
#pragma unroll
        for (int e = 0; e < PER; e++)
            if (d[e] < end) {
                const double w = weight_in_bin(x[e], top, s), b = d[e] < lo ? w : 0.0;
                limit += d[e] < kbin ? w : 0.0;
                below += b;
                kept += b >= min_w ? b : 0.0;
                question |= w > 0.0 && ((d[e] >= lo && d[e] <= hi) || d[e] == kbin) ? 1u << e : 0u;
            }
        mine = {whole_bits(kept + 0x1p52), whole_bits(below + 0x1p52), whole_bits(limit + 0x1p52)};
    } else {
        // Without branches, for the weights' instructions to overlap.  Each is 2^52 + w,
        // whose bits as whole numbers add up to the sum of w in their low 52.  What is
        // in no bin weighs nothing; what weighs nothing is in no prefix, listed or not.
        double w[PER];
        uint64_t below = 0, limit = 0;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            w[e] = whole_exp2(fmax(((double)x[e] - (double)top) * s.rate + (double)s.bits, -2.0));
            const uint64_t bits = __builtin_bit_cast(uint64_t, w[e]);
            const bool under = d[e] < lo;
            limit += bits;
            below += under ? bits : 0;
            question |= (uint32_t)(!under && d[e] <= hi) << e;
        }
        uint64_t kept = below;
        if (s.min_w) {
            const double least = 0x1p52 + (double)s.min_w;
            kept = 0;
#pragma unroll
            for (int e = 0; e < PER; e++)
                kept += d[e] < lo && w[e] >= least ? __builtin_bit_cast(uint64_t, w[e]) : 0;
        }
        mine = {kept & LOW52, below & LOW52, limit & LOW52};
    }
    if (question) {
        uint32_t at = atomicAdd(listed, (uint32_t)__builtin_popcount(question));
#pragma unroll
        for (int e = 0; e < PER; e++)
            if (question >> e & 1) {
                if (at < most)
                    list[at] = entry(x[e], (uint32_t)(i0 + e));
                at++;
            }
    }
    return mine;
}

// Small workgroups, four for a tile, so that some load while others compute (128
// rows of 128001, top-k and top-p: 13 us, one for a tile 17; 64 rows, top-p alone,
// level).
template <int PER, int DT>
__global__ __launch_bounds__(GATHER_THREADS, PER == 8 ? 8 : 4) void k_gather(SampleArgs a, RowScratch *scratch)
{
    constexpr int MOST = PER * GATHER_THREADS;
    __shared__ uint64_t list[MOST];
    __shared__ Sums sums[GATHER_THREADS / 64];
    __shared__ uint32_t listed, base;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.y, i0 = ((int64_t)blockIdx.x * GATHER_THREADS + tid) * PER;
    RowScratch &r = scratch[row];
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    const Setting s = r.setting;
    const Range g = r.range;
    const float top = r.row_top;
    if (top == -__builtin_inff() || s.rate < 0.0)
        return;
    if (tid == 0)
        listed = 0;
    __syncthreads();
    Sums v = gather(x, i0, top, s, g, list, MOST, &listed);
    v.below = wave_sum(v.below);
    v.kept = s.min_w ? wave_sum(v.kept) : v.below;
    v.limit = wave_sum(v.limit);
    if ((tid & 63) == 0)
        sums[tid >> 6] = v;
    __syncthreads();
    const uint32_t n = listed;
    if (tid == 0) {
        for (int i = 1; i < GATHER_THREADS / 64; i++)
            v = {v.kept + sums[i].kept, v.below + sums[i].below, v.limit + sums[i].limit};
        r.sums[blockIdx.x] = v;
    }
    if (n == 0)
        return;
    if (tid == 0)
        base = atomicAdd(&r.listed, n);
    __syncthreads();
    for (uint32_t i = tid; i < n && base + i < LIST; i += GATHER_THREADS)
        r.list[base + i] = list[i];
}

struct CutLds {
    uint64_t list[THREADS];                      // the first entries
    uint64_t weight[SHORT];
    uint32_t sub_count[SUBS];
    uint64_t sub_mass[SUBS];
    uint64_t in_sub[MOST_ALIKE];                 // those of one sub-bin
    uint64_t part_kept[MOST_PARTS];
    uint64_t scan[WAVES];
    uint32_t scan32[WAVES];
    unsigned long long cut, low_mass, part;
    uint32_t low, least, most, n_in, sub_least, sub_most;
    int k_sub, p_sub;
    uint32_t sub_before;
    uint64_t sub_mass_before;
};

// How many entries of the list, and how much, come before one.
struct Ranked {
    uint32_t rank;
    uint64_t before;
};

// Brings the entries of sub-bin `sub` together, as far as they fit, and says whether
// their logits are all equal.
__device__ __forceinline__ bool collect(CutLds &l, const uint64_t *list, uint32_t n, int sub,
                                        uint32_t least, int shift)
{
    const int tid = threadIdx.x;
    if (tid == 0) {
        l.n_in = l.sub_most = 0;
        l.sub_least = ~0u;
    }
    __syncthreads();
    for (uint32_t i = tid; i < n; i += THREADS) {
        const uint64_t e = list[i];
        const uint32_t key = (uint32_t)(e >> 32);
        if ((int)((key - least) >> shift) == sub) {
            const uint32_t at = atomicAdd(&l.n_in, 1u);
            if (at < MOST_ALIKE)
                l.in_sub[at] = e;
            atomicMin(&l.sub_least, key);
            atomicMax(&l.sub_most, key);
        }
    }
    __syncthreads();
    return l.sub_least == l.sub_most;
}

// The m-th entry (from 1) of equal logits, key in the list, into l.cut: by sub-bins of
// the index, then among the few of one (vocabularies of tiles: up to 2048).
__device__ __forceinline__ void nth_alike(CutLds &l, const uint64_t *list, uint32_t n, uint32_t key,
                                          uint32_t m, int64_t vocab)
{
    const int tid = threadIdx.x;
    const int shift = max(32 - __builtin_clz((uint32_t)vocab | 1) - 10, 0);
    l.sub_count[tid] = 0;
    if (tid == 0)
        l.n_in = 0;
    __syncthreads();
    for (uint32_t i = tid; i < n; i += THREADS)
        if ((uint32_t)(list[i] >> 32) == key)
            atomicAdd(&l.sub_count[(uint32_t)list[i] >> shift], 1u);
    __syncthreads();
    const uint32_t own = l.sub_count[tid];
    uint32_t all;
    const uint32_t before = scan_before<WAVES>(own, l.scan32, all);
    if (before < m && m <= before + own) {
        l.low = tid;
        l.sub_before = before;
    }
    __syncthreads();
    const uint32_t sub = l.low, need = m - l.sub_before;
    for (uint32_t i = tid; i < n; i += THREADS)
        if ((uint32_t)(list[i] >> 32) == key && (uint32_t)list[i] >> shift == sub)
            l.in_sub[atomicAdd(&l.n_in, 1u)] = list[i];
    __syncthreads();
    const uint32_t few = l.n_in;
    for (uint32_t i = tid; i < few; i += THREADS) {
        const uint64_t e = l.in_sub[i];
        uint32_t rank = 1;
        for (uint32_t j = 0; j < few; j++)
            rank += l.in_sub[j] < e;
        if (rank == need)
            l.cut = e;
    }
    __syncthreads();
}

// The entries collected of a sub-bin, each with how many and how much of the list come
// before it; false (nothing done) if they do not fit.
template <typename F>
__device__ __forceinline__ bool rank_in(CutLds &l, float top, const Setting &s, F f)
{
    const int tid = threadIdx.x;
    const uint32_t m = l.n_in, rank0 = l.sub_before;
    const uint64_t before0 = l.sub_mass_before;
    if (m > MOST_ALIKE)
        return false;
    // sorted by exchanges: each stretch of k entries is made a rising or falling one of
    // two halves that are (1024 equal logits: 20 us; counting for each what comes
    // before it takes 100)
    uint32_t P = 1;
    while (P < m)
        P *= 2;
    for (uint32_t i = m + tid; i < P; i += THREADS)
        l.in_sub[i] = ~uint64_t(0);
    for (uint32_t k = 2; k <= P; k *= 2)
        for (uint32_t j = k / 2; j; j /= 2) {
            __syncthreads();
            for (uint32_t t = tid; t < P / 2; t += THREADS) {
                const uint32_t i = 2 * t - (t & (j - 1));
                const uint64_t x = l.in_sub[i], y = l.in_sub[i + j];
                if ((x > y) == ((i & k) == 0)) {
                    l.in_sub[i] = y;
                    l.in_sub[i + j] = x;
                }
            }
        }
    __syncthreads();
    const uint32_t each = (P + THREADS - 1) / THREADS;
    uint64_t own = 0, sum;
    for (uint32_t i = tid * each; i < min((tid + 1) * each, m); i++)
        own += weight(entry_value(l.in_sub[i]), top, s);
    uint64_t before = before0 + scan_before<WAVES>(own, l.scan, sum);
    for (uint32_t i = tid * each; i < min((tid + 1) * each, m); i++) {
        const uint64_t e = l.in_sub[i], w = weight(entry_value(e), top, s);
        f(e, w, Ranked{rank0 + i, before});
        before += w;
    }
    __syncthreads();
    return true;
}

// What a short list's cut is: threads in a row share an entry and count what comes
// before it.
__device__ __forceinline__ Cut rank_short(CutLds &l, const Setting &s, const Range &g, uint32_t n,
                                          const Sums &all, float top, int part_size)
{
    const int tid = threadIdx.x;
    const float rate = s.grid, place = floorf(top * rate);
    const bool k_cuts = g.kbin < BINS;
    int P = THREADS / SHORT;
    while (P < 64 && n * P * 2 <= THREADS)
        P *= 2;
    if (tid == 0) {
        l.cut = l.part = 0;
        l.low = 0;
    }
    __syncthreads();
    if (tid < n) {
        const float x = entry_value(l.list[tid]);
        l.weight[tid] = weight(x, top, s);
        if (k_cuts && bin_of(x, place, rate) < g.kbin)
            atomicAdd(&l.low, 1u);
    }
    __syncthreads();
    const uint32_t i = (uint32_t)tid / P;
    const bool in = i < n && !(tid & (P - 1));
    const uint64_t e = i < n ? l.list[i] : 0, w = i < n ? l.weight[i] : 0;
    uint32_t rank = 0;
    uint64_t before = 0;
    if (i < n) {
#pragma unroll 4
        for (uint32_t j = tid & (P - 1); j < n; j += P) {
            const bool ahead = l.list[j] < e;
            rank += ahead;
            before += ahead ? l.weight[j] : 0;
        }
    }
    for (int d = 1; d < P; d <<= 1) {
        rank += __shfl_xor(rank, d);
        before += __shfl_xor((unsigned long long)before, d);
    }
    const int bin = bin_of(entry_value(e), place, rate);
    const bool in_k = !k_cuts || bin < g.kbin || rank - l.low < (uint32_t)s.k - g.k_before;
    uint64_t total = all.limit;
    if (k_cuts && s.p < 1.0) {
        if (in && in_k && bin == g.kbin)
            atomicAdd(&l.part, (unsigned long long)w);
        __syncthreads();
        total += l.part;
    }
    if (in && in_k && bin <= g.hi && inside(all.below + before, s.p, total)) {
        atomicMax(&l.cut, (unsigned long long)e);
        if (w >= s.min_w)
            atomicAdd((unsigned long long *)&l.part_kept[(uint32_t)e / part_size],
                      (unsigned long long)w);
    }
    __syncthreads();
    return Cut{~(uint32_t)(l.cut >> 32), (int64_t)(uint32_t)l.cut};
}

// The cut, from the list (n entries); adds what is kept of it to the parts' sums.
// Sub-bins of the list's own range, in falling order, bring it down to the few
// elements around a cut; those are ranked one by one.  false: too many are alike.
__device__ __forceinline__ bool rank_list(CutLds &l, const Setting &s, const Range &g,
                                          const uint64_t *list, uint32_t n, const Sums &all, float top,
                                          int part_size, int64_t vocab, Cut &c)
{
    const int tid = threadIdx.x;
    const float rate = s.grid, place = floorf(top * rate);
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
        const uint32_t k = (uint32_t)(list[i] >> 32);
        least = min(least, k);
        most = max(most, k);
        const float x = key_value(~k);
        if (k_cuts && bin_of(x, place, rate) < g.kbin) {
            low++;
            low_mass += weight(x, top, s);
        }
    }
    for (int d = 1; d < 64; d <<= 1) {
        least = min(least, (uint32_t)__shfl_xor(least, d));
        most = max(most, (uint32_t)__shfl_xor(most, d));
    }
    low = wave_sum(low);
    low_mass = wave_sum(low_mass);
    if ((tid & 63) == 0) {
        atomicMin(&l.least, least);
        atomicMax(&l.most, most);
        if (low) {
            atomicAdd(&l.low, low);
            atomicAdd(&l.low_mass, (unsigned long long)low_mass);
        }
    }
    __syncthreads();
    least = l.least;
    const uint32_t span = l.most - least;
    const int shift = max(32 - __builtin_clz(span | 1) - 10, 0);     // SUBS = 2^10
    for (uint32_t i = tid; i < n; i += THREADS) {
        const uint64_t e = list[i];
        const int sub = (int)(((uint32_t)(e >> 32) - least) >> shift);
        atomicAdd(&l.sub_count[sub], 1u);
        atomicAdd((unsigned long long *)&l.sub_mass[sub],
                  (unsigned long long)weight(entry_value(e), top, s));
    }
    __syncthreads();
    const uint32_t count = l.sub_count[tid];
    const uint64_t mass = l.sub_mass[tid];
    uint32_t all_count;
    uint64_t all_mass;
    const uint32_t before = scan_before<WAVES>(count, l.scan32, all_count);
    const uint64_t mass_before = scan_before<WAVES>(mass, l.scan, all_mass);
    // top-k keeps k_rank entries of the list: those above kbin and some in it
    const uint32_t k_rank = k_cuts ? (uint32_t)s.k - g.k_before + l.low : ~0u;
    uint64_t total = all.limit;
    if (k_cuts && s.p < 1.0) {
        note_last(count && before < k_rank, tid, &l.k_sub);
        __syncthreads();
        if (tid == l.k_sub) {
            l.sub_before = before;
            l.sub_mass_before = mass_before;
        }
        if (collect(l, list, n, l.k_sub, least, shift)) {
            const uint64_t w = weight(key_value(~l.sub_least), top, s);
            total += min(l.n_in, k_rank - l.sub_before) * w;
        } else {
            if (!rank_in(l, top, s, [&](uint64_t, uint64_t w, const Ranked &r) {
                    if (r.rank < k_rank)
                        atomicAdd(&l.part, (unsigned long long)w);
                }))
                return false;
            total += l.part;
        }
        total += l.sub_mass_before - l.low_mass;
    }
    note_last(count && before < k_rank && inside(all.below + mass_before, s.p, total), tid, &l.p_sub);
    __syncthreads();
    if (tid == l.p_sub) {
        l.sub_before = before;
        l.sub_mass_before = mass_before;
    }
    if (collect(l, list, n, l.p_sub, least, shift)) {
        const uint32_t key = l.sub_least, m = min(l.n_in, k_rank - l.sub_before);
        const uint64_t w = weight(key_value(~key), top, s), ahead = all.below + l.sub_mass_before;
        const uint32_t in = s.p < 1.0 ? ties_inside(ahead, w, m, s.p, total) : m;
        __syncthreads();
        nth_alike(l, list, n, key, in, vocab);
    } else if (!rank_in(l, top, s, [&](uint64_t e, uint64_t, const Ranked &r) {
                   if (r.rank < k_rank && inside(all.below + r.before, s.p, total))
                       atomicMax(&l.cut, (unsigned long long)e);
               })) {
        return false;
    }
    const uint64_t cut = l.cut;
    for (uint32_t i = tid; i < n; i += THREADS) {
        const uint64_t e = list[i];
        const uint64_t w = e <= cut ? weight(entry_value(e), top, s) : 0;
        if (w && w >= s.min_w)
            atomicAdd((unsigned long long *)&l.part_kept[(uint32_t)e / part_size],
                      (unsigned long long)w);
    }
    __syncthreads();
    c = Cut{~(uint32_t)(cut >> 32), (int64_t)(uint32_t)cut};
    return true;
}

// A row's end: from the sums of its parts (part_kept, too) and the list (its first
// entries in LDS, too) to its token, or to its cut and the sum of what is kept.  A
// part holds E elements a thread; x: the only part's, or not loaded.
template <int E, int DT>
__device__ __forceinline__ uint64_t finish(const SampleArgs &a, int64_t row, CutLds &l, RowLds &rl,
                                           const Setting &s, const Range &g, const Sums &all,
                                           const uint64_t *list, uint32_t n, uint32_t most,
                                           float top, int parts, Cut &c, float (&x)[E],
                                           bool loaded)
{
    const int tid = threadIdx.x, lane = tid & 63;
    bool ranked = !g.odd && n <= most;
    if (ranked && n) {
        if (n <= SHORT)
            c = rank_short(l, s, g, n, all, top, E * THREADS);
        else
            ranked = rank_list(l, s, g, n <= THREADS ? l.list : list, n, all, top, E * THREADS,
                               a.vocab, c);
    }
    if (!ranked) {
        const Walker walker{a.logits, row * a.stride, a.vocab, a.dtype, top};
        c = find_cut(walker, s, rl);
        return walk_row(a, walker, s, c, row, rl);
    }
    // the part, then the element in it, where the running sum passes u
    const int each = (parts + 63) / 64;          // of a lane
    uint64_t v = 0;
    for (int i = lane * each; i < min(lane * each + each, parts); i++)
        v += l.part_kept[i];
    const uint64_t run = scan_wave(v);
    const uint64_t sum = lane_value(run, 63), thr = place_in(s.u, sum);
    if (a.probs)
        return sum;
    const int at_lane = __builtin_ctzll(__ballot(run > thr));
    int part = at_lane * each;
    uint64_t at = lane_value(run - v, at_lane);
    for (int i = 1; i < each; i++)
        if (at + l.part_kept[part] <= thr)
            at += l.part_kept[part++];
    const int64_t j0 = ((int64_t)part * THREADS + tid) * E;
    if (!loaded) {
#pragma unroll
        for (int e = 0; e < E; e++)
            x[e] = j0 + e < a.vocab ? load_one(a.logits, DT, row * a.stride + j0 + e)
                                    : -__builtin_inff();
    }
    uint64_t w[E] = {}, own = 0, whole;
    uint32_t in = 0;
#pragma unroll
    for (int e = 0; e < E; e++)
        in |= kept(c, order_key(x[e]), j0 + e) ? 1u << e : 0u;
    if (__any(in)) {
#pragma unroll
        for (int e = 0; e < E; e++) {
            w[e] = weight(x[e], top, s);
            w[e] = (in >> e & 1) && w[e] >= s.min_w ? w[e] : 0;
            own += w[e];
        }
    }
    __syncthreads();
    at += scan_before<WAVES>(own, l.scan, whole);
    if (at <= thr && thr < at + own) {
        int hit = 0;
#pragma unroll
        for (int e = 0; e < E; e++) {
            at += w[e];
            hit += at <= thr;
        }
        a.tokens[row] = (int32_t)(j0 + hit);
    }
    return sum;
}

template <int PER, int DT>
__global__ __launch_bounds__(THREADS) void k_cut(SampleArgs a, RowScratch *scratch, int tiles,
                                                 int parts)
{
    __shared__ CutLds l;
    __shared__ RowLds rl;
    __shared__ uint64_t sums[3][WAVES];
    __shared__ int first;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    RowScratch &r = scratch[row];
    const uint64_t e0 = r.list[tid];             // before it is known how many there are
    const Setting s = r.setting;
    const float top = r.row_top;
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
        if (tid < parts) {
            v = r.sums[tid];
            l.part_kept[tid] = v.kept;
        }
        l.list[tid] = e0;
        const Sums all = sum_up(v, sums);
        float x[PER / PARTS];
        sum = finish<PER / PARTS, DT>(a, row, l, rl, s, g, all, r.list, n, LIST, top, parts, c, x,
                                      false);
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
    const RowScratch &r = scratch[row];
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
    Setting s = r.setting;
    set_greedy(s);
    write_probs(a, row, i0, x, r.row_top, s, Cut{r.key, r.last}, r.sum);
}

// A vocabulary of one tile.
template <int PER, int DT> __global__ __launch_bounds__(THREADS) void k_one(SampleArgs a)
{
    __shared__ CutLds l;
    __shared__ RowLds rl;
    __shared__ RangeLds range;
    __shared__ uint64_t bins[BINS], sums[3][WAVES], list[PER * THREADS];
    __shared__ int first;
    __shared__ uint32_t listed;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, i0 = (int64_t)tid * PER;
    Setting s = setting_of(a, row);
    float x[PER];
    load_tile<PER, DT>(x, a, row, i0);
#pragma unroll
    for (int i = 0; i < EACH; i++)
        bins[i * THREADS + tid] = 0;
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
            if (on_grid(top, s.grid)) {
                const bool counted = s.k > 0;
                add_bins(x, top, s.grid, counted, bins);
                __syncthreads();
                uint32_t count[2];
                uint64_t units[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int b = 2 * tid + i;
                    units[i] = counted ? (uint32_t)bins[b] : ((const uint32_t *)bins)[b];
                    count[i] = counted ? (uint32_t)(bins[b] >> 32) : units[i] != 0;
                }
                g = find_range(range, count, units, s, top);
            } else {
                g.odd = 1;
            }
        }
        const Sums all = sum_up(gather(x, i0, top, s, g, list, PER * THREADS, &listed), sums);
        const uint32_t n = listed;
        if (tid == 0)
            l.part_kept[0] = all.kept;
        if (tid < n)
            l.list[tid] = list[tid];
        __syncthreads();
        sum = finish<PER, DT>(a, row, l, rl, s, g, all, list, n, PER * THREADS, top, 1, c, x, true);
    }
    if (a.probs)
        write_probs(a, row, i0, x, top, s, c, sum);
}

// Elements a thread: 8, or 16 where the tiles were too many else.  (16 for 64 rows
// of 128001: 64 us a call, 60 with 8.)
bool large_tiles(int64_t vocab) { return vocab > (int64_t)8 * THREADS * MOST_TILES; }

int64_t tiles_of(int64_t vocab)
{
    const int64_t size = (large_tiles(vocab) ? 16 : 8) * THREADS;
    return (vocab + size - 1) / size;
}

// Rows of one launch: those whose scratch takes up to 256 MiB (several hundred).
size_t row_bytes(int64_t tiles) { return sizeof(RowScratch) + tiles * PLANE * sizeof(uint64_t); }

int64_t rows_a_launch(int64_t rows, int64_t tiles)
{
    return std::min<int64_t>(rows, std::max<int64_t>(1, (int64_t(256) << 20) / row_bytes(tiles)));
}

template <int PER, int DT>
hipError_t launch_tiles(SampleArgs a, int64_t tiles, void *scratch, hipStream_t s)
{
    const int64_t rows = a.rows, most = rows_a_launch(rows, tiles), size = DT == TQ_F32 ? 4 : 2;
    RowScratch *r = (RowScratch *)scratch;
    uint64_t *planes = (uint64_t *)(r + most);
    for (int64_t at = 0; at < rows; at += most) {
        const int64_t n = std::min(rows - at, most);
        const dim3 grid((unsigned)tiles, (unsigned)n);
        const bool pairs = PER == 8 && n * tiles > RESIDENT;
        const int64_t binned = pairs ? (tiles + 1) / 2 : tiles;
        if (pairs)
            k_bins<16, DT><<<dim3((unsigned)binned, (unsigned)n), THREADS, 0, s>>>(a, r, planes);
        else
            k_bins<PER, DT><<<grid, THREADS, 0, s>>>(a, r, planes);
        k_range<<<dim3((unsigned)n), THREADS, 0, s>>>(a, r, planes, (int)binned);
        k_gather<PER, DT><<<dim3((unsigned)(tiles * PARTS), (unsigned)n),
                            GATHER_THREADS, 0, s>>>(a, r);
        k_cut<PER, DT><<<dim3((unsigned)n), THREADS, 0, s>>>(a, r, (int)binned, (int)tiles * PARTS);
        if (a.probs)
            k_probs<PER, DT><<<grid, THREADS, 0, s>>>(a, r);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        a.logits = (const uint8_t *)a.logits + most * a.stride * size;
        a.temperature += a.temperature ? most : 0;
        a.top_k += a.top_k ? most : 0;
        a.top_p += a.top_p ? most : 0;
        a.min_p += a.min_p ? most : 0;
        a.u += a.u ? most : 0;
        a.tokens += a.tokens ? most : 0;
        a.probs += a.probs ? most * a.probs_stride : 0;
    }
    return hipSuccess;
}

template <int DT> hipError_t launch_dt(const SampleArgs &a, void *scratch, hipStream_t s)
{
    const int64_t tiles = tiles_of(a.vocab);
    if (tiles > 1 && tiles <= MOST_TILES)
        return large_tiles(a.vocab) ? launch_tiles<16, DT>(a, tiles, scratch, s)
                                            : launch_tiles<8, DT>(a, tiles, scratch, s);
    if (!grid_fits(a.rows, THREADS))
        return hipErrorInvalidConfiguration;
    if (tiles == 1)
        k_one<8, DT><<<dim3((unsigned)a.rows), THREADS, 0, s>>>(a);
    else
        k_sample_row<<<dim3((unsigned)a.rows), THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t sample_scratch_bytes(int64_t rows, int64_t vocab)
{
    const int64_t tiles = tiles_of(vocab);
    return tiles == 1 || tiles > MOST_TILES ? 0 : rows_a_launch(rows, tiles) * row_bytes(tiles);
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
