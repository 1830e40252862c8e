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
    double min_w;                                // in units of the weights
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
    s.min_w = m > 0.0f ? ldexp((double)fminf(m, 1.0f), a.bits) : 0.0;
    s.k = a.top_k ? a.top_k[row] : 0;
    s.u = a.u ? a.u[row] : 0.0f;
    s.bits = a.bits;
    return s;
}

// A weight in units of 2^-bits; 0 for what is no number, or -infinity.
__device__ __forceinline__ uint64_t weight(float x, float top, const Setting &s)
{
    if (x == top)
        return uint64_t(1) << s.bits;
    const double t = ((double)x - (double)top) * s.rate + (double)s.bits;
    if (!(t > -2.0) || !(x > -__builtin_inff()))
        return 0;
    return (uint64_t)rint(exp2(t));
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

// One workgroup a row.
template <bool PROBS> __global__ __launch_bounds__(THREADS) void k_sample_row(SampleArgs a)
{
    __shared__ RowLds l;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    Setting s = setting_of(a, row);
    Walker r{a.logits, row * a.stride, a.vocab, a.dtype, 0.0f};
    float top = -__builtin_inff();
    for (int64_t i = tid; i < a.vocab; i += THREADS)
        top = fmaxf(top, r.get(i));
    for (int m = 1; m < 64; m <<= 1)
        top = fmaxf(top, __shfl_xor(top, m));
    if (lane == 0)
        l.top[wave] = top;
    __syncthreads();
    for (int i = 0; i < WAVES; i++)
        top = fmaxf(top, l.top[i]);
    r.top = top;
    const bool none = top == -__builtin_inff();
    Cut c{0, a.vocab};
    if (s.rate < 0.0) {                          // greedy: the first of the largest
        c.key = order_key(top);
        if (!none)
            c.last = find_tie(r, l, c.key, 1);
        s.rate = 1.0;
    } else if (!none) {
        c = find_cut(r, s, l);
    }
    auto kept_weight = [&](int64_t i) {
        const float x = r.get(i);
        const uint64_t w = none || !kept(c, order_key(x), i) ? 0 : weight(x, r.top, s);
        return (double)w >= s.min_w ? w : 0;
    };
    // a wave has a run of the row
    const int64_t run = (a.vocab + THREADS - 1) / THREADS * 64, begin = run * wave;
    const int64_t end = min(begin + run, a.vocab);
    uint64_t sum = 0;
    for (int64_t i = begin + lane; i < end; i += 64)
        sum += kept_weight(i);
    sum = wave_sum(sum);
    if (lane == 0)
        l.scan[wave] = sum;
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (int i = 0; i < WAVES; i++) {
        before += i < wave ? l.scan[i] : 0;
        all += l.scan[i];
    }
    if constexpr (PROBS) {
        const double inv = all ? 1.0 / (double)all : 0.0;
        for (int64_t i = tid; i < a.vocab; i += THREADS)
            a.probs[row * a.probs_stride + i] = (float)((double)kept_weight(i) * inv);
    } else {
        // u below 0 or NaN counts as 0, 1 and above as just below it
        const double u = s.u > 0.0f ? fmin((double)s.u, 1.0) : 0.0;
        const uint64_t thr = all ? min((uint64_t)(u * (double)all), all - 1) : 0;
        if (tid == 0 && all == 0)
            a.tokens[row] = -1;
        if (!(before <= thr && thr < before + sum))
            return;
        for (int64_t base = begin; base < end; base += 64) {
            const int64_t i = base + lane;
            const uint64_t w = i < end ? kept_weight(i) : 0;
            const uint64_t upto = before + scan_wave(w);
            const uint64_t hit = __ballot(upto > thr);
            if (hit) {
                if (lane == __builtin_ctzll(hit))
                    a.tokens[row] = (int32_t)i;
                break;
            }
            before = lane_value(upto, 63);
        }
    }
}

}  // namespace

size_t sample_scratch_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleArgs &a, void *, hipStream_t s)
{
    const dim3 grid((unsigned)a.rows);
    if (a.probs)
        k_sample_row<true><<<grid, THREADS, 0, s>>>(a);
    else
        k_sample_row<false><<<grid, THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace tq
