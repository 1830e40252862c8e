// Verification of drafted tokens against the target's probabilities from
// given uniform numbers (tq_verify_draft).
//
// Nodes of one sequence are in drafting order, node 0 the last token that is
// already certain; row n of `target` is the target's distribution after node
// n, row n of `draft` the one that n's children were drawn from.  From node
// n, with w = target[n], the children c are tried in order:
//     accepted when u[c] * q(x_c) < w(x_c): go on from c;
//     else w <- max(w - q, 0) / sum max(w - q, 0)    (draft given), or
//          w(x_c) <- 0, the threshold u * (1 - what was removed)   (none).
// After the last one the next token is the first index whose running sum of w
// passes r times the sum.  After j rejections w = max(a p - b q, 0) for two
// scalars a, b, so no row is ever written.  Everything is fp64: an index then
// depends on the order of a sum with a probability of about 1e-13.
//
// Bound: the rows the last token is drawn from are read once; for few
// sequences, latency (starts -> nodes -> their probabilities -> the row -> the
// tile).  A sequence's row is cut into tiles of TILE elements, one a wave;
// the first wave of every workgroup of 16 walks the drafted nodes, 64 at a
// time in its lanes (a ballot finds the children: a turn per child tried, not
// per node), the waves sum their tiles, and the last workgroup of the
// sequence finds the tile that holds the threshold and the element in it.
// Reductions are DPP adds, not LDS permutes; one device-scope count per
// workgroup, on a cache line of its sequence's own, since such atomics on one
// line follow each other (with one per wave on a shared line 32 trees took 44
// us).  One sequence of
// 5 nodes over 128001 tokens: 12.0 us; 32 trees of up to 31 nodes: 21.8 us.
// Trees drafted with probabilities need whole-row sums during the walk and
// run as one workgroup per sequence instead: one of 31 nodes 32 us, 32 of them
// 105.
#include <algorithm>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int TILE = 512;                        // 8 elements a lane
constexpr int PER = TILE / 64;
constexpr int WAVES = 16, THREADS = 64 * WAVES;
constexpr int MOST_TILES = 64;                   // of one workgroup

template <int DT> __device__ __forceinline__ double prob(const void *p, int64_t i)
{
    if constexpr (DT == TQ_F32)
        return (double)((const float *)p)[i];
    else if constexpr (DT == TQ_BF16)
        return (double)__builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
    else
        return (double)f16_bits_to_f32(((const uint16_t *)p)[i]);
}

__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }

// What a p - b q leaves, q a draft probability of `positive`.  A row that
// does not count (b = 0) may hold anything, infinities too.
__device__ __forceinline__ double residual(double a, double p, double b, double q)
{
    return positive(b != 0.0 ? a * p - b * q : a * p);
}

// Lane k's value, k uniform.
__device__ __forceinline__ int lane_of(int x, int k) { return __builtin_amdgcn_readlane(x, k); }

__device__ __forceinline__ double lane_of(double x, int k)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)lane_of((int)(uint32_t)b, k), hi = (uint32_t)lane_of((int)(b >> 32), k);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int CTRL, int ROWS> __device__ __forceinline__ double dpp(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive running sum over the lanes: shifts by 1, 2, 4, 8 in each row of
// 16, then the last lane of a row added to the rows behind it.
__device__ __forceinline__ double scan_wave(double v)
{
    v += dpp<0x111, 0xF>(v);
    v += dpp<0x112, 0xF>(v);
    v += dpp<0x114, 0xF>(v);
    v += dpp<0x118, 0xF>(v);
    v += dpp<0x142, 0xA>(v);                     // row 0 -> 1, 2 -> 3
    v += dpp<0x143, 0xC>(v);                     // rows 0, 1 -> 2, 3
    return v;
}

__device__ __forceinline__ double wave_sum(double v) { return lane_of(scan_wave(v), 63); }

struct Seq {
    int64_t n0;
    int T;
};

__device__ __forceinline__ Seq seq_of(const VerifyArgs &a, int b)
{
    const int64_t s0 = min(max((int64_t)a.starts[b], (int64_t)0), a.nodes);
    const int64_t s1 = min((int64_t)a.starts[b + 1], a.nodes);
    return {s0, (int)min(max(s1 - s0, (int64_t)0), (int64_t)a.width)};
}

// Result of a walk.  took: the accepted nodes, a bit each; gone: the tokens
// refused at the last node (no draft probabilities only).
struct Found {
    int taken, rejected, node;
    double a, b;                                 // last token from max(a p - b q, 0), ...
    double a0, b0;                               // ... or, where that is all zero, this one
};

struct Record {
    uint64_t *took;                              // [width / 64 rounded up], LDS
    int *gone;                                   // [width], LDS
};

__host__ __device__ constexpr size_t record_bytes(int width)
{
    return (size_t)((width + 63) / 64) * 8 + (size_t)((width + 1) / 2) * 8;
}

extern __shared__ uint64_t record_lds[];

__device__ __forceinline__ Record record_of(int width)
{
    return {record_lds, (int *)(record_lds + (width + 63) / 64)};
}

// The walk, by a whole wave: one pass over the nodes, since children come
// after their parents.  row_sum(node, a, b): sum of max(a p - b q, 0), called
// only for a sibling after a rejection with draft probabilities given.  Waves
// that walk alike to join in it share the record: they write the same words,
// and `gone` is not used then.
template <int DT, typename F>
__device__ __forceinline__ Found walk(const VerifyArgs &a, const Seq &s, const Record &rec,
                                      F row_sum)
{
    Found f{0, 0, 0, 1.0, 0.0, 1.0, 0.0};
    const int lane = threadIdx.x & 63;
    double left = 1.0;
    bool pending = false;                        // the last rejection's sum is not taken yet
    for (int base = 0; base < s.T; base += 64) {
        const int i = base + lane;
        const bool in = i > 0 && i < s.T;
        const int64_t at = s.n0 + (in ? i : 0);
        int parent = a.parents ? a.parents[at] : i - 1;
        int x = a.tokens[at];
        const float ul = a.u[at];
        // a child after its parent and inside the vocabulary, or never accepted
        const bool ok = in && parent >= 0 && parent < i && x >= 0 && x < a.vocab;
        parent = ok ? parent : -1;
        x = ok ? x : 0;
        const int64_t row = s.n0 + max(parent, 0);
        const double pl = positive(prob<DT>(a.target, row * a.target_stride + x));
        const double ql = a.draft ? positive(prob<DT>(a.draft, row * a.draft_stride + x)) : 0.0;
        uint64_t took = 0, children = __ballot(parent == f.node);
        while (children) {
            const int c = __builtin_ctzll(children);
            children &= children - 1;
            const int token = lane_of(x, c);
            double p = lane_of(pl, c);
            const double q = lane_of(ql, c);
            const double u = (double)__builtin_bit_cast(float, lane_of(__builtin_bit_cast(int, ul), c));
            bool good;
            if (a.draft) {
                if (pending) {
                    const double z = row_sum(f.node, f.a, f.b);
                    if (z > 0.0) {
                        f.a /= z;
                        f.b /= z;
                    } else {
                        f.a = f.a0;
                        f.b = f.b0;
                    }
                    pending = false;
                }
                good = u * q < residual(f.a, p, f.b, q);
            } else {
                // a sibling with the same token has taken its probability along
                for (int k = 0; k < f.rejected; k += 64)
                    if (__any(k + lane < f.rejected && rec.gone[k + lane] == token))
                        p = 0.0;
                good = p > 0.0 && u * left < p;
            }
            if (good) {
                f.node = base + c;
                took |= uint64_t(1) << c;
                f.taken++;
                f.rejected = 0;
                f.a = f.a0 = 1.0;
                f.b = f.b0 = 0.0;
                left = 1.0;
                pending = false;
                children = __ballot(parent == f.node);
            } else if (a.draft) {
                f.a0 = f.a;
                f.b0 = f.b;
                f.b += 1.0;
                pending = true;
            } else {
                if (lane == 0)
                    rec.gone[f.rejected] = token;
                wave_handover();                 // all lanes read it for the next sibling
                f.rejected++;
                left -= p;
            }
        }
        if (lane == 0)
            rec.took[base >> 6] = took;
    }
    return f;
}

// Weight of vocabulary entry x at node row `row`, and the fallback's.
struct Sums {
    double now, before;
};

template <int DT>
__device__ __forceinline__ Sums weights(const VerifyArgs &a, const Record &rec, const Found &f,
                                        int64_t row, int64_t x)
{
    const double p = prob<DT>(a.target, row * a.target_stride + x);
    if (a.draft) {
        // nothing was refused after this node: its draft row has no say
        if (f.b == 0.0)
            return {positive(f.a * p), positive(f.a0 * p)};
        const double q = positive(prob<DT>(a.draft, row * a.draft_stride + x));
        return {residual(f.a, p, f.b, q), residual(f.a0, p, f.b0, q)};
    }
    double now = positive(p);
    for (int k = 0; k < f.rejected; k++)
        if (rec.gone[k] == x)
            now = 0.0;
    return {now, 0.0};
}

// One wave: a tile's sums.
template <int DT>
__device__ __forceinline__ Sums tile_sums(const VerifyArgs &a, const Seq &s, const Record &rec,
                                          const Found &f, int tile)
{
    const int lane = threadIdx.x & 63;
    Sums t{0.0, 0.0};
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const int64_t x = (int64_t)tile * TILE + e * 64 + lane;
        if (x < a.vocab) {
            const Sums w = weights<DT>(a, rec, f, s.n0 + f.node, x);
            t.now += w.now;
            t.before += w.before;
        }
    }
    return {wave_sum(t.now), a.draft ? wave_sum(t.before) : 0.0};
}

// One wave: from the tile sums that sums(i) gives, which of the two weights
// counts and the tile where the running sum passes r times the total; then the
// element in it; and the sequence's outputs.
template <int DT, typename F>
__device__ __forceinline__ void finish(const VerifyArgs &a, int b, const Seq &s, const Record &rec,
                                       const Found &f, int tiles, F sums)
{
    const int lane = threadIdx.x & 63;
    int next = -1;
    if (s.T > 0) {
        const Sums mine = lane < tiles ? sums(lane) : Sums{0.0, 0.0};   // the first 64 stay here
        Sums t = mine;
        for (int i = 64 + lane; i < tiles; i += 64) {
            const Sums v = sums(i);
            t.now += v.now;
            t.before += v.before;
        }
        t.now = wave_sum(t.now);
        t.before = wave_sum(t.before);
        const bool use_before = !(t.now > 0.0);
        const double total = use_before ? t.before : t.now, thr = (double)a.r[b] * total;
        int tile = -1;                           // else the last tile of positive sum
        double from = 0.0, before = 0.0;
        for (int base = 0; base < tiles; base += 64) {
            Sums v = mine;
            if (base)
                v = base + lane < tiles ? sums(base + lane) : Sums{0.0, 0.0};
            const double w = use_before ? v.before : v.now;
            const double run = scan_wave(w), prev = before + (run - w);
            const uint64_t hit = __ballot(w > 0.0 && before + run > thr), some = __ballot(w > 0.0);
            if (hit | some) {
                const int k = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
                tile = base + k;
                from = lane_of(prev, k);
                if (hit)
                    break;
            }
            before += lane_of(run, 63);
        }
        if (tile >= 0) {
            double v[PER], sum = 0.0;
            const int64_t x0 = (int64_t)tile * TILE + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; e++) {
                Sums w{0.0, 0.0};
                if (x0 + e < a.vocab)
                    w = weights<DT>(a, rec, f, s.n0 + f.node, x0 + e);
                v[e] = use_before ? w.before : w.now;
                sum += v[e];
            }
            double at = from + (scan_wave(sum) - sum);
            int hit = -1, last = -1;
#pragma unroll
            for (int e = 0; e < PER; e++) {
                at += v[e];
                if (v[e] > 0.0) {
                    last = e;
                    if (at > thr && hit < 0)
                        hit = e;
                }
            }
            const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
            if (hits) {
                const int k = __builtin_ctzll(hits);
                next = tile * TILE + k * PER + lane_of(hit, k);
            } else if (some) {
                const int k = 63 - __builtin_clzll(some);
                next = tile * TILE + k * PER + lane_of(last, k);
            }
        }
    }
    int32_t *tokens = a.out_tokens + (int64_t)b * a.width, *nodes = a.out_nodes + (int64_t)b * a.width;
    int done = 0;
    for (int base = 0; base < s.T; base += 64) {
        const uint64_t took = rec.took[base >> 6];
        if ((took >> lane) & 1) {
            const int at = done + __builtin_popcountll(took & ((uint64_t(1) << lane) - 1));
            nodes[at] = base + lane;
            tokens[at] = a.tokens[s.n0 + base + lane];
        }
        done += __builtin_popcountll(took);
    }
    for (int i = f.taken + lane; i < a.width; i += 64) {
        nodes[i] = -1;
        tokens[i] = i == f.taken ? next : -1;
    }
    if (lane == 0)
        a.count[b] = f.taken;
}

// Chains, and trees without draft probabilities: `per` tiles a wave.
template <int DT>
__global__ __launch_bounds__(THREADS) void k_verify(VerifyArgs a, int tiles, int per,
                                                    uint32_t *counters, int counter_stride,
                                                    double *sums)
{
    __shared__ Found found;
    __shared__ double mine[MOST_TILES * 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = blockIdx.y, own = WAVES * per, first = blockIdx.x * own;
    const Record rec = record_of(a.width);
    const Seq s = seq_of(a, b);
    if (wave == 0) {
        const Found f = walk<DT>(a, s, rec, [](int, double, double) { return 1.0; });
        if (lane == 0)
            found = f;
    }
    __syncthreads();
    const Found f = found;
    for (int i = wave; i < own; i += WAVES) {
        Sums t{0.0, 0.0};
        if (s.T > 0 && first + i < tiles)
            t = tile_sums<DT>(a, s, rec, f, first + i);
        if (lane < 2)
            mine[2 * i + lane] = lane ? t.before : t.now;
    }
    __syncthreads();
    if (wave)
        return;
    // The sums are exchanged into memory (device-scope atomics act there, past
    // the dies' caches) and have come back before the count rises, so whoever
    // sees the last count reads them whole.  A release at device scope would
    // do as well, but it writes back and drops a die's whole L2 (32 trees: 58
    // us instead of 35, everything else alike).
    uint64_t *all = (uint64_t *)(sums + (int64_t)b * tiles * 2);
    const int n = 2 * min(own, tiles - first);
    uint64_t was = 0;
    for (int i = lane; i < n; i += 64)
        was |= __hip_atomic_exchange(all + 2 * first + i, __builtin_bit_cast(uint64_t, mine[i]),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" : : "v"(was) : "memory");
    uint32_t *count = counters + (int64_t)b * counter_stride;
    uint32_t done = 0;
    if (lane == 0)
        done = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (lane_of((int)done, 0) != (int)gridDim.x - 1)
        return;
    finish<DT>(a, b, s, rec, f, tiles, [&](int i) {
        const double *p = (const double *)all + 2 * i;
        return Sums{__hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                    __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
    });
    if (lane == 0)                               // zero again for the next call
        __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Trees with draft probabilities: one workgroup per sequence, its waves walk
// alike and share the row sums.
template <int DT>
__global__ __launch_bounds__(THREADS) void k_verify_tree(VerifyArgs a, int tiles, double *sums)
{
    __shared__ double red[WAVES];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Record rec = record_of(a.width);
    const Seq s = seq_of(a, b);
    const Found f = walk<DT>(a, s, rec, [&](int node, double fa, double fb) {
        double v = 0.0;
        const int64_t row = s.n0 + node;
#pragma unroll 8
        for (int64_t x = tid; x < a.vocab; x += THREADS)
            v += residual(fa, prob<DT>(a.target, row * a.target_stride + x), fb,
                          positive(prob<DT>(a.draft, row * a.draft_stride + x)));
        v = wave_sum(v);
        __syncthreads();                         // red is free
        if (lane == 0)
            red[wave] = v;
        __syncthreads();
        double z = 0.0;
        for (int k = 0; k < WAVES; k++)
            z += red[k];
        return z;
    });
    double *mine = sums + (int64_t)b * tiles * 2;
    for (int tile = wave; tile < tiles; tile += WAVES) {
        Sums t{0.0, 0.0};
        if (s.T > 0)
            t = tile_sums<DT>(a, s, rec, f, tile);
        if (lane < 2)
            mine[2 * tile + lane] = lane ? t.before : t.now;
    }
    __syncthreads();
    if (wave == 0)
        finish<DT>(a, b, s, rec, f, tiles, [&](int i) { return Sums{mine[2 * i], mine[2 * i + 1]}; });
}

int tiles_of(int64_t vocab) { return (int)((vocab + TILE - 1) / TILE); }

template <int DT>
hipError_t launch_dt(const VerifyArgs &a, uint32_t *counters, double *sums, hipStream_t s)
{
    const int tiles = tiles_of(a.vocab);
    const size_t rec = record_bytes(a.width);
    if (a.parents && a.draft) {
        k_verify_tree<DT><<<dim3((unsigned)a.batch), THREADS, rec, s>>>(a, tiles, sums);
        return hipGetLastError();
    }
    // one tile a wave, or up to four where that gives more than 512 workgroups:
    // two for each of 256 compute units, of which its registers let one run at a
    // time (66 a lane; 64 would let two)
    const int64_t groups = (int64_t)a.batch * ((tiles + WAVES - 1) / WAVES);
    const int per = (int)std::min<int64_t>(MOST_TILES / WAVES, (groups + 511) / 512);
    const int x = (tiles + WAVES * per - 1) / (WAVES * per);
    // counts 256 bytes apart, closer where TQ_NOALLOC_SCRATCH_BYTES asks for it
    const int stride = (int)std::min<int64_t>(64, TQ_NOALLOC_SCRATCH_BYTES / 4 / a.batch);
    k_verify<DT><<<dim3((unsigned)x, (unsigned)a.batch), THREADS, rec, s>>>(a, tiles, per, counters,
                                                                           stride, sums);
    return hipGetLastError();
}

}  // namespace

size_t verify_scratch_bytes(int64_t batch, int64_t vocab)
{
    return (size_t)batch * tiles_of(vocab) * 2 * sizeof(double);
}

hipError_t launch_verify(int dtype, const VerifyArgs &a, uint32_t *counters, void *scratch,
                         hipStream_t s)
{
    switch (dtype) {
    case TQ_F32: return launch_dt<TQ_F32>(a, counters, (double *)scratch, s);
    case TQ_BF16: return launch_dt<TQ_BF16>(a, counters, (double *)scratch, s);
    case TQ_F16: return launch_dt<TQ_F16>(a, counters, (double *)scratch, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace tq
